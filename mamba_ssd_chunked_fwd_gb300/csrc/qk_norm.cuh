// qk_norm.cuh -- parameters of the norm of queries and keys.
#pragma once

#include "scan_common.cuh"

namespace ssd {

struct QkNormParams {
    int B, L, H, G, N, half;  // half: rotated pairs
    const void *q, *k;
    const float *w_q, *w_k, *freqs;
    const int32_t *positions;
    void *q_out, *k_out;
    long long qs[2], ks[2];  // strides (batch, token) in elements
    int l2, interleaved;
    float eps;
    // backward
    const void *dq_out, *dk_out;
    void *dq, *dk;
    float *dw_q, *dw_k;
    float *part;  // [qk_norm_parts, N]
};
int qk_norm_parts(const QkNormParams &p);
cudaError_t launch_qk_norm(const QkNormParams &p, int io, cudaStream_t s);
cudaError_t launch_qk_norm_bwd(const QkNormParams &p, int io, cudaStream_t s);

}  // namespace ssd

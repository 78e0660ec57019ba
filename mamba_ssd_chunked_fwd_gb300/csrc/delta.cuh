// delta.cuh -- what the kernels of the gated delta rule share.
//
//   S' = exp(g_t) S_{t-1},  u_t = beta_t (v_t - S' k_t),  S_t = S' + u_t k_t^T,  y_t = scale S_t q_t
//
// with S a state of P x N for every head, and the queries and keys of group h / (H/G).
#pragma once

#include "scan_common.cuh"

namespace ssd {

constexpr int kDeltaChunk = 64;  // tokens of a chunk

struct DeltaParams {
    int B, L, H, G, N, P;
    const void *q, *k, *v, *g, *beta;
    const float *h0;
    const int32_t *lengths;
    void *y;
    float *final_state;
    long long qs[2], ks[2], vs[2], gs[2], bs[2];  // strides (batch, token) in elements
    int g32, b32;                                 // g, beta are fp32
    float scale;
    int nc;  // chunks of a row
    // segments: tokens [s seg_len, (s+1) seg_len) of every row; seg_len a multiple of 64
    int nseg, seg_len;
    bool chunked;  // by the kernels of delta_tc.cu
    float *seg_states;  // [B,H,nseg,P,N] state entering a segment (slot 0 unused)
    unsigned char *ops;  // [B,H,nc] a chunk's operands (delta_tc.cuh)
    float *seg_trans;   // [B,H,nseg-1,N,N] a segment's transition: the state after it is S trans + (its own); slot 0 unused
    // backward
    const void *dy;
    const float *dfinal;
    void *dq, *dk, *dv, *dg, *dbeta;
    float *dh0;
    // (in chunks on the tensor cores these four are operands of the same size, N and P rounded up: delta_tc.cuh)
    float *states;  // [B,H,nc,P,N] state before a chunk
    float *adj;     // [B,H,nc,P,N] adjoint of the state after a chunk
    float *u, *dr;  // [B,H,64 nc,P] u, and the gradient of v_t - S' k_t over beta
    float *dqh, *dkh;  // [B,L,H,N] a head's share of dq, dk (H > G)
    float *units;  // fp16 in chunks, [B,H,nc,P tiles of 128][4]: the powers of two that states, u, adjoint and r are held times
};

struct DeltaStepParams {
    int B, H, G, N, P;
    long long nslots;
    const void *q, *k, *v, *g, *beta;
    const float *state;
    float *state_out;
    const int32_t *slots;
    void *y;
    long long q_row, k_row, v_row, g_row, b_row;
    int g32, b32;
    float scale;
};

cudaError_t launch_delta_walk(const DeltaParams &p, int io, cudaStream_t s);          // y, final_state
size_t delta_op_bytes(bool pure);
cudaError_t launch_delta_prep(const DeltaParams &p, int io, bool pure, cudaStream_t s);   // a chunk's operands for the next three
cudaError_t launch_delta_grad_tc(const DeltaParams &p, int io, cudaStream_t s);           // as launch_delta_grad
cudaError_t launch_delta_tc_walks(const DeltaParams &p, int io, cudaStream_t s);          // as launch_delta_walks
void delta_segments(DeltaParams &p);
bool delta_tc_takes(const DeltaParams &p, int io);
cudaError_t launch_delta_tc(const DeltaParams &p, int io, cudaStream_t s);            // the same in chunks
cudaError_t launch_delta_bwd(const DeltaParams &p, int io, cudaStream_t s);
cudaError_t launch_delta_walks(const DeltaParams &p, int io, cudaStream_t s);        // states, u; adj, dr, dv, dh0
cudaError_t launch_delta_grad(const DeltaParams &p, int io, cudaStream_t s);          // the other gradients
cudaError_t launch_delta_step(const DeltaStepParams &p, int io, cudaStream_t s);

// An element of g or beta: fp32 or the tensors' type.
template <int IO>
__device__ __forceinline__ float load_gate(const void *base, long long i, int f32, bool ok) {
    if (IO == IO_F32) return load_one<IO_F32>(base, i, ok);
    const float a = load_one<IO>(base, i, ok && !f32), b = load_one<IO_F32>(base, i, ok && f32);
    return f32 ? b : a;
}
template <int IO>
__device__ __forceinline__ void store_gate(void *base, long long i, int f32, float v) {
    if (IO == IO_F32 || f32) static_cast<float *>(base)[i] = v;
    else st_io<IO>(base, i, v);
}

__device__ __forceinline__ int delta_length(const DeltaParams &p, int b) {
    return p.lengths ? min(max(__ldg(p.lengths + b), 0), p.L) : p.L;
}

}  // namespace ssd

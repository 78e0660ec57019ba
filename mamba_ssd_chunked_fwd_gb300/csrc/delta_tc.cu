// delta_tc.cu -- the gated delta rule of 16-bit prompts in chunks: the walks of delta_walk_tc.cuh, whole or
// cut into segments, and the fold between.
#include <math.h>

#include "delta_walk_tc.cuh"

namespace ssd {

namespace {

using delta_walk::LOCAL_STATE;
using delta_walk::Y;

template <int IO, int NN, int MODE>
__global__ void __launch_bounds__(delta_walk::kThreads, 1)
delta_tc_kernel(const __grid_constant__ DeltaParams p) {
    delta_walk::walk<IO, NN, MODE>(p, blockIdx.x);
}

// The state entering each segment from the third on: S_{s+1} = S_s trans_s + own_s, row by row; `own` lies where the
// result goes.  A CTA takes 16 rows of a head; the next transition is copied while one is multiplied.  A thread has four rows of
// two columns, so that a column's float2 and a row's float4 from shared memory feed eight multiply-adds each: 16 heads of
// 128 x 128 in 9 segments 29 us (eight rows of one column a thread, and a transition more: 41).
constexpr int kFoldRows = 16, kFoldThreads = 256;
constexpr int kFoldBytes = 2 * 128 * 128 * 4 + kFoldRows * 132 * 4;
__global__ void __launch_bounds__(kFoldThreads)
delta_fold_kernel(const __grid_constant__ DeltaParams p) {
    extern __shared__ __align__(16) float fold_mem[];
    float *trans = fold_mem, *state = fold_mem + 2 * 128 * 128;
    const int tiles = (p.P + kFoldRows - 1) / kFoldRows, bh = blockIdx.x / tiles, p0 = (blockIdx.x % tiles) * kFoldRows;
    const int tid = threadIdx.x, n = 2 * (tid & 63), r0 = (tid >> 6) * 4, N = p.N;
    const size_t pn = (size_t)p.P * N, nn = (size_t)N * N;
    auto copy = [&](int s) {
        const float *src = p.seg_trans + ((size_t)bh * (p.nseg - 1) + s) * nn;
        for (int e = 4 * tid; e < (int)nn; e += 4 * kFoldThreads) cp_async16(trans + (s & 1) * 128 * 128 + e, src + e, 16);
        cp_commit();
    };
    auto entering = [&](int s, int r) { return reinterpret_cast<float2 *>(p.seg_states + ((size_t)bh * p.nseg + s) * pn + (size_t)(p0 + r0 + r) * N + n); };
    copy(1);
#pragma unroll
    for (int r = 0; r < 4; ++r)
        *reinterpret_cast<float2 *>(state + (r0 + r) * 132 + n) = n < N && p0 + r0 + r < p.P ? *entering(1, r) : make_float2(0.f, 0.f);
    for (int s = 1; s + 1 < p.nseg; ++s) {
        if (s + 2 < p.nseg) copy(s + 1);
        else cp_commit();
        float2 acc[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] = n < N && p0 + r0 + r < p.P ? *entering(s + 1, r) : make_float2(0.f, 0.f);
        cp_wait<1>();
        __syncthreads();
        const float *t = trans + (s & 1) * 128 * 128 + n;
#pragma unroll 4
        for (int m = 0; m < N; m += 4) {
            float2 f[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = n < N ? *reinterpret_cast<const float2 *>(t + (m + j) * N) : make_float2(0.f, 0.f);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float4 x = *reinterpret_cast<const float4 *>(state + (r0 + r) * 132 + m);
                acc[r] = __ffma2_rn(dup(x.x), f[0], __ffma2_rn(dup(x.y), f[1], __ffma2_rn(dup(x.z), f[2], __ffma2_rn(dup(x.w), f[3], acc[r]))));
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            *reinterpret_cast<float2 *>(state + (r0 + r) * 132 + n) = acc[r];
            if (n < N && p0 + r0 + r < p.P) *entering(s + 1, r) = acc[r];
        }
        __syncthreads();
    }
}

template <int IO, int NN, int MODE>
cudaError_t tc_as(const DeltaParams &p, cudaStream_t s) {
    const long long tiles = (p.P + 127) / 128, heads = (long long)p.B * p.H;
    auto *kernel = delta_tc_kernel<IO, NN, MODE>;
    const cudaError_t e = allow_smem<delta_walk::Smem<NN>::BYTES>(kernel);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(MODE == LOCAL_STATE ? heads * (p.nseg - 1) * (tiles + 1) : heads * p.nseg * tiles), delta_walk::kThreads, delta_walk::Smem<NN>::BYTES, s>>>(p);
    return cudaGetLastError();
}
template <int IO, int MODE>
cudaError_t tc_mode(const DeltaParams &p, cudaStream_t s) {
    return p.N <= 64 ? tc_as<IO, 64, MODE>(p, s) : tc_as<IO, 128, MODE>(p, s);
}

template <int IO>
cudaError_t tc_io(const DeltaParams &p, cudaStream_t s) {
    cudaError_t e = launch_delta_prep(p, IO, false, s);
    if (e == cudaSuccess && p.nseg > 1) {
        e = tc_mode<IO, LOCAL_STATE>(p, s);
    }
    if (e == cudaSuccess && p.nseg > 2) {
        e = allow_smem<kFoldBytes>(delta_fold_kernel);
        if (e != cudaSuccess) return e;
        delta_fold_kernel<<<(unsigned)((long long)p.B * p.H * ((p.P + kFoldRows - 1) / kFoldRows)), kFoldThreads, kFoldBytes, s>>>(p);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? tc_mode<IO, Y>(p, s) : e;
}

bool by_eights(const void *p, long long s0, long long s1) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && s0 % 8 == 0 && s1 % 8 == 0;
}

}  // namespace

// 16-byte pieces of k, q and v, and float4 of the states.  What is not taken is walked token by token, [4,4096] with 32 heads of
// 128 rows in bf16 (and its gradients, [4,2048] with 16 heads): N = 128 in chunks 347 us (424), N = 124 by tokens 2231 us (2321); fp32
// with N = 128 by tokens 2137 us (2318).  One chunk of one row takes 6 us longer than its 64 tokens, 512 tokens half as long; the rule
// has no term for the length.
bool delta_tc_takes(const DeltaParams &p, int io) {
    return io != IO_F32 && p.N % 8 == 0 && p.P % 8 == 0 && by_eights(p.k, p.ks[0], p.ks[1]) && by_eights(p.q, p.qs[0], p.qs[1]) &&
           by_eights(p.v, p.vs[0], p.vs[1]) && by_eights(p.y, 0, 0) && by_eights(p.h0, 0, 0) && by_eights(p.final_state, 0, 0) &&
           by_eights(p.dy, 0, 0) && by_eights(p.dq, 0, 0) && by_eights(p.dk, 0, 0) && by_eights(p.dv, 0, 0) && by_eights(p.dfinal, 0, 0) && by_eights(p.dh0, 0, 0);
}

// The cut of the rows into segments.  A walk takes an SM for itself, and a chunk about 3.3 us of it (a pass of a segment's own
// state and of its transition 2.6), both measured with 128 x 128 in bf16 and taken for every N and P; few heads are cut until there are walks for the SMs.  The cut costs that first pass, a
// fold (a state through a segment's transition, about 1.5 us) and two launches.
void delta_segments(DeltaParams &p) {
    const double sms = scan_sm_count(), heads = (double)p.B * p.H, tiles = (p.P + 127) / 128;
    auto cost = [&](int m) {
        const int len = (p.nc + m - 1) / m, n = (p.nc + len - 1) / len;
        const double walk = ceil(heads * tiles * n / sms) * 3.3 * len;
        return n == 1 ? walk : walk + ceil(heads * ((tiles + 1) * (n - 1) - 1) / sms) * 2.6 * len + 1.5 * n + 10.;
    };
    int best = 1;
    for (int m = 2; m <= 64 && m <= p.nc; ++m)
        if (cost(m) < cost(best)) best = m;
    const int len = (p.nc + best - 1) / best;
    p.seg_len = len * kC;
    p.nseg = (p.nc + len - 1) / len;
}

cudaError_t launch_delta_tc(const DeltaParams &p, int io, cudaStream_t s) {
    return io == IO_BF16 ? tc_io<IO_BF16>(p, s) : tc_io<IO_F16>(p, s);
}

}  // namespace ssd

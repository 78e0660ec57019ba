// block_norm.cu -- the end of one block and the norm before the next:
//
//   p = o / rms(o) * w_post,  r' = r + scale gate p,  n = r' / rms(r') * w_pre
//
// and its backward.  With a = d o / rms(o) (the normalised rows hat_o, hat_r):
//   dr     = dr_out + (v - hat_r mean(v hat_r)) / rms(r'),       v = dn w_pre
//   d_o    = (u - hat_o mean(u hat_o)) / rms(o),                 u = dr scale gate w_post
//   dgate  = dr scale w_post hat_o,   dw_pre = sum dn hat_r,
//   dscale = w_post s,  dw_post = scale s,                       s = sum dr gate hat_o
//
// About 11 (backward 30) operations per element against 8 to 16 bytes: bound by
// HBM.  The threads of a row own runs of four elements, K per thread, which they
// copy into slots of their own in shared memory a row ahead, so that the loads of
// one row run beside the reductions and stores of the one before, need no
// registers, and every tensor moves once.  Backwards the two column sums and the
// weights stay in registers over a chunk of rows.
#include "scan_common.cuh"

namespace ssd {

namespace {

// Sums of v over the row's TPR threads (blockDim.x), for every one of them.  One
// barrier: consecutive calls must use different `slot`s.
template <int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float (*slot)[32]) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return;  // rows of one warp are independent of each other
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < NV; ++i) slot[i][w] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        v[i] = lane < nw ? slot[i][lane] : 0.f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    }
}

template <int IO, bool VEC>
__device__ __forceinline__ void unpack_pairs(const Raw4 &r, float2 (&v)[2]) {
    float f[4];
    unpack4<IO, VEC>(r, f);
    v[0] = make_float2(f[0], f[1]);
    v[1] = make_float2(f[2], f[3]);
}
template <int IO, bool VEC>
__device__ __forceinline__ void store_pairs(void *base, long long i, int nv, const float2 (&v)[2]) {
    const float f[4] = {v[0].x, v[0].y, v[1].x, v[1].y};
    store4_io<IO, VEC>(base, i, nv, f);
}
// Four of a weight vector [D], or ones.
template <bool VEC>
__device__ __forceinline__ void weights(const float *w, int c, int nv, float2 (&v)[2]) {
    unpack_pairs<IO_F32, VEC>(load_raw4<IO_F32, VEC>(w, c, w && nv > 0, nv), v);
    if (!w) v[0] = v[1] = dup(1.f);
}
// scale w_post
template <bool VEC>
__device__ __forceinline__ void post_weights(const BlockNormParams &p, int c, int nv, float2 (&v)[2]) {
    float2 s[2];
    weights<VEC>(p.w_post, c, nv, v);
    weights<VEC>(p.scale, c, nv, s);
    v[0] = __fmul2_rn(v[0], s[0]);
    v[1] = __fmul2_rn(v[1], s[1]);
}

// The slots of a CTA's threads for one row: NI tensors in the block's type, then NS in the stream's.
template <int IO, int SIO, int K, int NI, int NS>
struct NormSlots {
    static constexpr int kQi = IO == IO_F32 ? 16 : 8, kQs = SIO == IO_F32 ? 16 : 8;
    static constexpr int kPerThread = K * (NI * kQi + NS * kQs);
    // of thread `tid` of n: tensor i's quad k
    static __device__ __forceinline__ int block(int i, int k, int tid, int n) { return (i * K + k) * kQi * n + tid * kQi; }
    static __device__ __forceinline__ int stream(int i, int k, int tid, int n) {
        return NI * K * kQi * n + (i * K + k) * kQs * n + tid * kQs;
    }
};

template <int IO, int SIO, int K, bool VEC>
__global__ void __launch_bounds__(1024)
block_norm_kernel(BlockNormParams p, int stages) {
    using S = NormSlots<IO, SIO, K, 2, 1>;  // o, gate; r
    extern __shared__ __align__(16) char ring[];
    __shared__ float red[2][1][32];
    constexpr int kEi = IO == IO_F32 ? 4 : 2, kEs = SIO == IO_F32 ? 4 : 2;
    const int tx = threadIdx.x, tpr = blockDim.x, nthr = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + tx;
    const float inv_d = 1.f / (float)p.D;
    const long long step = (long long)gridDim.x * blockDim.y;
    auto copy = [&](long long row, char *slot) {
        if (row < p.rows) {
            const long long base = row * p.D + tx * 4, gbase = p.gate ? row / p.rows_per_gate * p.D + tx * 4 : 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int nv = min(4, p.D - (tx + tpr * k) * 4), c = tpr * k * 4;
                copy_quad<SIO, VEC>(slot + S::stream(0, k, tid, nthr), static_cast<const char *>(p.r) + (base + c) * kEs, nv);
                if (p.o) copy_quad<IO, VEC>(slot + S::block(0, k, tid, nthr), static_cast<const char *>(p.o) + (base + c) * kEi, nv);
                if (p.gate) copy_quad<IO, VEC>(slot + S::block(1, k, tid, nthr), static_cast<const char *>(p.gate) + (gbase + c) * kEi, nv);
            }
        }
        cp_commit();
    };
    long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    char *slot = ring, *next = stages == 2 ? ring + nthr * S::kPerThread : ring;
    if (stages == 2) copy(row, slot);
    for (; row < p.rows; row += step) {
        if (stages == 2) {
            copy(row + step, next);
            cp_wait<1>();
        } else {
            copy(row, slot);
            cp_wait<0>();
        }
        const long long base = row * p.D + tx * 4;
        float inv = 1.f;
        if (p.o && p.w_post) {
            float2 s2 = dup(0.f);
#pragma unroll
            for (int k = 0; k < K; ++k) {  // zeros past the row's end
                float2 o[2];
                read_quad<IO>(slot + S::block(0, k, tid, nthr), o);
                s2 = __ffma2_rn(o[0], o[0], s2);
                s2 = __ffma2_rn(o[1], o[1], s2);
            }
            float ss[1] = {s2.x + s2.y};
            row_sum(ss, red[0]);
            inv = rsqrtf(ss[0] * inv_d + p.eps);
        }
        float2 s2 = dup(0.f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (tx + tpr * k) * 4, nv = min(4, p.D - c);
            float2 r[2];
            read_quad<SIO>(slot + S::stream(0, k, tid, nthr), r);
            if (p.o) {
                float2 o[2], ws[2];
                post_weights<VEC>(p, c, nv, ws);
                read_quad<IO>(slot + S::block(0, k, tid, nthr), o);
                if (p.gate) {
                    float2 g[2];
                    read_quad<IO>(slot + S::block(1, k, tid, nthr), g);
                    ws[0] = __fmul2_rn(ws[0], g[0]);
                    ws[1] = __fmul2_rn(ws[1], g[1]);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) r[j] = __ffma2_rn(ws[j], __fmul2_rn(o[j], dup(inv)), r[j]);
                write_quad<SIO>(slot + S::stream(0, k, tid, nthr), r);  // rounded as it is stored
                if (nv > 0) store_pairs<SIO, VEC>(p.r_out, base + tpr * k * 4, nv, r);
                read_quad<SIO>(slot + S::stream(0, k, tid, nthr), r);
            }
            s2 = __ffma2_rn(r[0], r[0], s2);
            s2 = __ffma2_rn(r[1], r[1], s2);
        }
        float ss[1] = {s2.x + s2.y};
        row_sum(ss, red[1]);
        const float2 inv2 = dup(rsqrtf(ss[0] * inv_d + p.eps));
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (tx + tpr * k) * 4, nv = min(4, p.D - c);
            float2 r[2], wp[2];
            weights<VEC>(p.w_pre, c, nv, wp);
            read_quad<SIO>(slot + S::stream(0, k, tid, nthr), r);
            r[0] = __fmul2_rn(__fmul2_rn(r[0], inv2), wp[0]);
            r[1] = __fmul2_rn(__fmul2_rn(r[1], inv2), wp[1]);
            if (nv > 0) store_pairs<IO, VEC>(p.n, base + tpr * k * 4, nv, r);
        }
        if (!(p.o && p.w_post) && blockDim.x > 32) __syncthreads();  // one reduction per row only: its slot is free again
        char *t = slot;
        slot = next;
        next = t;
    }
}

// MAXT: the threads a row may take (fewer leave each more registers).  whole: the
// slots hold dr_out and the gate too; rows too wide for that load them where they are used.
template <int IO, int SIO, int K, bool VEC, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 128 ? 4 : 1)
block_norm_bwd_kernel(BlockNormParams p, int stages, int whole) {
    using S = NormSlots<IO, SIO, K, 3, 2>;   // o, dn, gate; r', dr_out
    using T = NormSlots<IO, SIO, K, 2, 1>;   // o, dn; r'
    extern __shared__ __align__(16) char ring[];
    __shared__ float red[2][3][32];
    constexpr int kEi = IO == IO_F32 ? 4 : 2, kEs = SIO == IO_F32 ? 4 : 2;
    const int tx = threadIdx.x, tpr = blockDim.x, nthr = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + tx;
    const long long chunk = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    if (chunk >= p.chunks) return;  // blockDim.y > 1 only for rows of one warp
    const bool seq_gate = p.gate && p.rows_per_gate > 1;
    long long r0, r1;
    if (seq_gate) {
        const long long per = (p.rows_per_gate + p.chunk_rows - 1) / p.chunk_rows, gi = chunk / per;
        r0 = gi * p.rows_per_gate + chunk % per * p.chunk_rows;
        r1 = min((gi + 1) * p.rows_per_gate, r0 + p.chunk_rows);
    } else {
        r0 = chunk * p.chunk_rows;
        r1 = min(p.rows, r0 + p.chunk_rows);
    }
    auto off_o = [&](int k) { return whole ? S::block(0, k, tid, nthr) : T::block(0, k, tid, nthr); };
    auto off_n = [&](int k) { return whole ? S::block(1, k, tid, nthr) : T::block(1, k, tid, nthr); };
    auto off_r = [&](int k) { return whole ? S::stream(0, k, tid, nthr) : T::stream(0, k, tid, nthr); };
    auto copy = [&](long long row, char *slot) {
        if (row < r1) {
            const long long base = row * p.D + tx * 4, gbase = p.gate ? row / p.rows_per_gate * p.D + tx * 4 : 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int nv = min(4, p.D - (tx + tpr * k) * 4), c = tpr * k * 4;
                copy_quad<SIO, VEC>(slot + off_r(k), static_cast<const char *>(p.r_out) + (base + c) * kEs, nv);
                copy_quad<IO, VEC>(slot + off_n(k), static_cast<const char *>(p.dn) + (base + c) * kEi, nv);
                if (p.o) copy_quad<IO, VEC>(slot + off_o(k), static_cast<const char *>(p.o) + (base + c) * kEi, nv);
                if (!whole) continue;
                if (p.dr_out) copy_quad<SIO, VEC>(slot + S::stream(1, k, tid, nthr), static_cast<const char *>(p.dr_out) + (base + c) * kEs, nv);
                if (p.gate) copy_quad<IO, VEC>(slot + S::block(2, k, tid, nthr), static_cast<const char *>(p.gate) + (gbase + c) * kEi, nv);
            }
        }
        cp_commit();
    };
    char *slot = ring, *next = stages == 2 ? ring + nthr * (whole ? S::kPerThread : T::kPerThread) : ring;
    if (stages == 2) copy(r0, slot);
    float2 acc1[K][2], acc2[K][2], wp[K][2], ws[K][2];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (tx + tpr * k) * 4, nv = min(4, p.D - c);
        acc1[k][0] = acc1[k][1] = acc2[k][0] = acc2[k][1] = dup(0.f);
        weights<VEC>(p.w_pre, c, nv, wp[k]);
        post_weights<VEC>(p, c, nv, ws[k]);
    }
    const float inv_d = 1.f / (float)p.D;
    for (long long row = r0; row < r1; ++row) {
        if (stages == 2) {
            copy(row + 1, next);
            cp_wait<1>();
        } else {
            copy(row, slot);
            cp_wait<0>();
        }
        const long long base = row * p.D + tx * 4;
        float2 s0 = dup(0.f), s1 = dup(0.f), s2 = dup(0.f);
#pragma unroll
        for (int k = 0; k < K; ++k) {  // zeros past the row's end
            float2 r[2], n[2], o[2];
            read_quad<SIO>(slot + off_r(k), r);
            read_quad<IO>(slot + off_n(k), n);
            if (p.o) read_quad<IO>(slot + off_o(k), o);
            else o[0] = o[1] = dup(0.f);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                s0 = __ffma2_rn(r[j], r[j], s0);
                s1 = __ffma2_rn(__fmul2_rn(n[j], wp[k][j]), r[j], s1);
                s2 = __ffma2_rn(o[j], o[j], s2);
            }
        }
        float s[3] = {s0.x + s0.y, s1.x + s1.y, s2.x + s2.y};  // |r'|^2, dn w_pre . r', |o|^2
        row_sum(s, red[0]);
        const float inv2 = rsqrtf(s[0] * inv_d + p.eps), m2 = s[1] * inv_d * inv2 * inv2;
        const float inv = p.w_post ? rsqrtf(s[2] * inv_d + p.eps) : 1.f;
        float2 t2 = dup(0.f), u[K][2];  // u . o
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (tx + tpr * k) * 4, nv = min(4, p.D - c);
            const long long at = base + tpr * k * 4;
            float2 dr[2], r[2], n[2];
            read_quad<SIO>(slot + off_r(k), r);
            read_quad<IO>(slot + off_n(k), n);
            if (!p.dr_out) dr[0] = dr[1] = dup(0.f);
            else if (whole) read_quad<SIO>(slot + S::stream(1, k, tid, nthr), dr);
            else unpack_pairs<SIO, VEC>(load_raw4<SIO, VEC>(p.dr_out, at, nv, nv), dr);
#pragma unroll
            for (int j = 0; j < 2; ++j) {  // dr = (v - r' inv2^2 mean(v r')) inv2 + dr_out
                const float2 v = __ffma2_rn(r[j], dup(-m2), __fmul2_rn(n[j], wp[k][j]));
                dr[j] = __ffma2_rn(v, dup(inv2), dr[j]);
                acc2[k][j] = __ffma2_rn(n[j], __fmul2_rn(r[j], dup(inv2)), acc2[k][j]);
            }
            if (nv > 0) store_pairs<SIO, VEC>(p.dr, at, nv, dr);
            if (!p.o) continue;
            float2 o[2], g[2], dg[2];
            read_quad<IO>(slot + off_o(k), o);
            if (!p.gate) g[0] = g[1] = dup(1.f);
            else if (whole) read_quad<IO>(slot + S::block(2, k, tid, nthr), g);
            else unpack_pairs<IO, VEC>(load_raw4<IO, VEC>(p.gate, row / p.rows_per_gate * p.D + c, nv, nv), g);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 dh = __fmul2_rn(dr[j], __fmul2_rn(o[j], dup(inv)));  // dr hat_o
                dg[j] = __fmul2_rn(dh, ws[k][j]);
                u[k][j] = __fmul2_rn(__fmul2_rn(g[j], dr[j]), ws[k][j]);
                t2 = __ffma2_rn(u[k][j], o[j], t2);
                acc1[k][j] = seq_gate ? __fadd2_rn(acc1[k][j], dh) : __ffma2_rn(dh, g[j], acc1[k][j]);
            }
            if (p.gate && !seq_gate && nv > 0) store_pairs<IO, VEC>(p.dgate, at, nv, dg);
        }
        if (p.o) {
            float t[1] = {t2.x + t2.y};
            row_sum(t, red[1]);
            const float m = p.w_post ? t[0] * inv_d * inv * inv : 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int nv = min(4, p.D - (tx + tpr * k) * 4);
                float2 o[2];
                read_quad<IO>(slot + off_o(k), o);
#pragma unroll
                for (int j = 0; j < 2; ++j) o[j] = __fmul2_rn(__ffma2_rn(o[j], dup(-m), u[k][j]), dup(inv));
                if (nv > 0) store_pairs<IO, VEC>(p.d_o, base + tpr * k * 4, nv, o);
            }
        } else if (blockDim.x > 32) {
            __syncthreads();  // the slot of the sums is free again
        }
        char *t = slot;
        slot = next;
        next = t;
    }
    float *part = p.part + chunk * 2 * p.D;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = (tx + tpr * k) * 4 + j;
            if (c < p.D) {
                part[c] = j & 1 ? acc1[k][j / 2].y : acc1[k][j / 2].x;
                part[p.D + c] = j & 1 ? acc2[k][j / 2].y : acc2[k][j / 2].x;
            }
        }
}

// The column sums over the chunks, in a fixed order: 32 interleaved sums per column, then those in turn.
template <int IO>
__global__ void __launch_bounds__(1024)
block_norm_sum_kernel(BlockNormParams p) {
    __shared__ float red[2][32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    const bool seq_gate = p.gate && p.rows_per_gate > 1, in = c < p.D;
    const float wpost = in && p.w_post ? __ldg(p.w_post + c) : 1.f, scale = in && p.scale ? __ldg(p.scale + c) : 1.f;
    float s1 = 0.f, s2 = 0.f;
    if (in) {
        if (seq_gate) {
            const long long per = (p.rows_per_gate + p.chunk_rows - 1) / p.chunk_rows, gates = p.rows / p.rows_per_gate;
            for (long long gi = threadIdx.y; gi < gates; gi += 32) {
                float s = 0.f;
                for (long long q = gi * per; q < (gi + 1) * per; ++q) {
                    s += p.part[q * 2 * p.D + c];
                    s2 += p.part[(q * 2 + 1) * p.D + c];
                }
                st_io<IO>(p.dgate, (size_t)(gi * p.D + c), s * (wpost * scale));
                s1 = fmaf(ld_io<IO>(p.gate, (size_t)(gi * p.D + c)), s, s1);
            }
        } else {
            for (long long q = threadIdx.y; q < p.chunks; q += 32) {
                s1 += p.part[q * 2 * p.D + c];
                s2 += p.part[(q * 2 + 1) * p.D + c];
            }
        }
    }
    red[0][threadIdx.y][threadIdx.x] = s1;
    red[1][threadIdx.y][threadIdx.x] = s2;
    __syncthreads();
    if (threadIdx.y != 0 || !in) return;
    for (int y = 1; y < 32; ++y) {
        s1 += red[0][y][threadIdx.x];
        s2 += red[1][y][threadIdx.x];
    }
    p.dw_pre[c] = s2;
    if (p.dw_post) p.dw_post[c] = scale * s1;
    if (p.dscale) p.dscale[c] = wpost * s1;
}

// Threads of a row and rows of a CTA for K runs of four elements per thread.
dim3 row_block(int D, int K) {
    const int tpr = ((D + 4 * K - 1) / (4 * K) + 31) / 32 * 32;
    return dim3(tpr, tpr == 32 ? 4 : 1);
}

// Runs of four elements per thread: the fewest that a warp's row takes, up to 4 (backwards 8 for rows
// past 8192, whose registers would not allow more threads); wider rows take more warps.
int norm_k(int D, bool backward) { return D <= 128 ? 1 : D <= 256 ? 2 : backward && D > 8192 ? 8 : 4; }

constexpr int kNormSmem = 227 * 1024 - 1024;  // the most a CTA may hold, less the sums

bool norm_vec(const BlockNormParams &p, int io, int sio) {
    auto ok = [](const void *q, int t) { return reinterpret_cast<uintptr_t>(q) % (t == IO_F32 ? 16 : 8) == 0; };
    return p.D % 4 == 0 && ok(p.o, io) && ok(p.r, sio) && ok(p.gate, io) && ok(p.n, io) && ok(p.r_out, sio) &&
           ok(p.dn, io) && ok(p.dr_out, sio) && ok(p.d_o, io) && ok(p.dr, sio) && ok(p.dgate, io) &&
           ok(p.w_post, IO_F32) && ok(p.w_pre, IO_F32) && ok(p.scale, IO_F32);
}

template <int IO, int SIO, int K>
cudaError_t launch_norm_as(const BlockNormParams &p, cudaStream_t s) {
    const dim3 block = row_block(p.D, K);
    auto *kernel = norm_vec(p, IO, SIO) ? block_norm_kernel<IO, SIO, K, true> : block_norm_kernel<IO, SIO, K, false>;
    const int row = (int)(block.x * block.y) * NormSlots<IO, SIO, K, 2, 1>::kPerThread;
    const int stages = 2 * row <= kNormSmem ? 2 : 1, bytes = stages * row;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const long long need = (p.rows + block.y - 1) / block.y;
    long long grid = scan_sm_count();
    if (need > grid) {  // as many CTAs as the SMs hold, each walking rows
        int per_sm = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, block.x * block.y, bytes);
        if (e != cudaSuccess) return e;
        grid *= per_sm > 0 ? per_sm : 1;
    }
    kernel<<<(unsigned)(need < grid ? need : grid), block, bytes, s>>>(p, stages);
    return cudaGetLastError();
}

template <int IO, int SIO>
cudaError_t launch_norm_io(const BlockNormParams &p, cudaStream_t s) {
    switch (norm_k(p.D, false)) {
        case 1: return launch_norm_as<IO, SIO, 1>(p, s);
        case 2: return launch_norm_as<IO, SIO, 2>(p, s);
        default: return launch_norm_as<IO, SIO, 4>(p, s);
    }
}

template <int IO, int SIO, int K, int MAXT>
cudaError_t launch_norm_bwd_as(const BlockNormParams &p, cudaStream_t s) {
    const dim3 block = row_block(p.D, K);
    auto *kernel = norm_vec(p, IO, SIO) ? block_norm_bwd_kernel<IO, SIO, K, true, MAXT> : block_norm_bwd_kernel<IO, SIO, K, false, MAXT>;
    const int n = block.x * block.y, row = n * NormSlots<IO, SIO, K, 3, 2>::kPerThread;
    const int whole = row <= kNormSmem, mine = whole ? row : n * NormSlots<IO, SIO, K, 2, 1>::kPerThread;
    const int stages = 2 * mine <= kNormSmem ? 2 : 1, bytes = stages * mine;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)((p.chunks + block.y - 1) / block.y), block, bytes, s>>>(p, stages, whole);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    block_norm_sum_kernel<IO><<<(p.D + 31) / 32, dim3(32, 32), 0, s>>>(p);
    return cudaGetLastError();
}

template <int IO, int SIO>
cudaError_t launch_norm_bwd_io(const BlockNormParams &p, cudaStream_t s) {
    switch (norm_k(p.D, true)) {
        case 1: return launch_norm_bwd_as<IO, SIO, 1, 128>(p, s);
        case 2: return launch_norm_bwd_as<IO, SIO, 2, 128>(p, s);
        case 4: return p.D <= 2048 ? launch_norm_bwd_as<IO, SIO, 4, 128>(p, s) : launch_norm_bwd_as<IO, SIO, 4, 512>(p, s);
        default: return launch_norm_bwd_as<IO, SIO, 8, 512>(p, s);
    }
}

}  // namespace

// Chunks for about 16 warps per SM, two at least; a chunk never spans two gates of several rows.
void block_norm_chunks(BlockNormParams &p) {
    const int warps = row_block(p.D, norm_k(p.D, true)).x / 32;
    const long long target = (warps < 8 ? 16 / warps : 2) * (long long)scan_sm_count();
    const bool seq_gate = p.gate && p.rows_per_gate > 1;
    const long long span = seq_gate ? p.rows_per_gate : p.rows, spans = p.rows / span;
    long long per = (target + spans - 1) / spans;  // chunks per span
    if (per > span) per = span;
    p.chunk_rows = (span + per - 1) / per;
    p.chunks = spans * ((span + p.chunk_rows - 1) / p.chunk_rows);
}

#define SSD_NORM_DISPATCH(FN)                                                     \
    if (io == IO_F32 && sio == IO_F32) return FN<IO_F32, IO_F32>(p, s);  \
    if (io == IO_F16 && sio == IO_F16) return FN<IO_F16, IO_F16>(p, s);  \
    if (io == IO_F16 && sio == IO_F32) return FN<IO_F16, IO_F32>(p, s);  \
    if (io == IO_BF16 && sio == IO_BF16) return FN<IO_BF16, IO_BF16>(p, s); \
    if (io == IO_BF16 && sio == IO_F32) return FN<IO_BF16, IO_F32>(p, s); \
    return cudaErrorInvalidValue;

cudaError_t launch_block_norm(const BlockNormParams &p, int io, int sio, cudaStream_t s) {
    SSD_NORM_DISPATCH(launch_norm_io)
}

cudaError_t launch_block_norm_bwd(const BlockNormParams &p, int io, int sio, cudaStream_t s) {
    SSD_NORM_DISPATCH(launch_norm_bwd_io)
}

}  // namespace ssd

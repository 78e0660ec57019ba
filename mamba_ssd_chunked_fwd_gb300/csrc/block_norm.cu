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
// HBM.  The threads of a row own units of eight elements, K per thread, which they
// copy into slots of their own in shared memory a row ahead, so that the loads of
// one row run beside the reductions and stores of the one before, need no
// registers, and every tensor moves once.  The weights, and backwards the two column
// sums, stay in registers over the rows that the threads walk.
// Measured: [8,4096,2048], bf16 with an fp32 stream and a gate per sequence, 143 us (5.65 TB/s,
// 83 % of the copy rate); backwards [4,2048,2048] in bf16 with a gate per token 59 us
// (4.6 TB/s), 8 of it the column sums: 128 registers a thread, 13.7 warps active per SM.  A gate per sequence: 58 us (80 while one thread per column
// summed a gate's partial rows; one sequence of 500 rows 25 and 109).
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

template <int SIO>
__device__ __forceinline__ float round_io(float v) {
    return IoTraits<SIO>::to_f(IoTraits<SIO>::from_f(v));
}

// Eight elements of a row as four pairs, the unit a thread deals in.  VEC: aligned and
// whole, one chunk of 16 bytes of a 16-bit type, two of fp32, beside its neighbours' chunks.
// Otherwise the pairs lie `step` elements apart, each beside the neighbours' pairs, so
// that a warp's accesses stay dense, and n elements are left in the row from the first
// pair on.  32768 rows of 2048, 2046 and 2047 bf16 elements: 136, 206 and 242 us (396 for
// 2047 with a thread's eight elements side by side); backwards, 8192 rows: 64, 100 and 129.
template <int IO>
struct Eight {
    static constexpr int kEs = IO == IO_F32 ? 4 : 2, kBytes = 8 * kEs;
};
// Pairs from a 4-byte boundary, and fp32 elements, are copied asynchronously; other 16-bit
// elements have no asynchronous form and are loaded, all at once, and stored.
template <int IO, bool VEC>
__device__ __forceinline__ void copy8(char *dst, const char *src, int n, int step) {
    if (VEC || IO == IO_F32) {
#pragma unroll
        for (int j = 0; j < (VEC ? Eight<IO>::kBytes / 16 : 8); ++j) {
            if (VEC) {
                copy_chunk<IO, true>(dst + 16 * j, src + 16 * j, n);
            } else {
                const int e = j / 2 * step + j % 2;
                cp_async4(dst + 4 * j, e < n ? src + 4LL * e : nullptr, e < n ? 4 : 0);
            }
        }
        return;
    }
    const bool even = (reinterpret_cast<size_t>(src) & 3) == 0;  // so are the other pairs: step is even
    uint16_t e[8];
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int left = n - j * step;
        const char *at = src + 2LL * j * step;
        cp_async4_if(even, dst + 4 * j, left > 0 ? at : nullptr, min(max(2 * left, 0), 4));
        e[2 * j] = e[2 * j + 1] = 0;
        ldg_u16(e[2 * j], at, !even && left > 0);
        ldg_u16(e[2 * j + 1], at + 2, !even && left > 1);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = e[2 * j] | ((uint32_t)e[2 * j + 1] << 16);
    if (!even) *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <int IO>
__device__ __forceinline__ void read8(const char *src, float2 (&v)[4]) {
    read_chunk<IO>(src, v);
    if (IO == IO_F32) read_chunk<IO>(src + 16, v + 2);
}
template <int IO, bool VEC>
__device__ __forceinline__ void store8(char *dst, int n, int step, const float2 (&v)[4]) {
    if (VEC) {
        store_chunk<IO, VEC>(dst, n, v);
        if (IO == IO_F32) store_chunk<IO, VEC>(dst + 16, n, v + 2);
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int left = n - j * step;
        char *at = dst + (long long)j * step * Eight<IO>::kEs;
        if (IO != IO_F32 && left > 1 && (reinterpret_cast<size_t>(at) & 3) == 0) {
            *reinterpret_cast<uint32_t *>(at) = pack16<IO>(v[j]);
        } else {
            if (left > 0) st_io<IO>(at, 0, v[j].x);
            if (left > 1) st_io<IO>(at, 1, v[j].y);
        }
    }
}
// Straight from global memory: a weight vector (ones when absent), or a tensor that has no slot.
template <int IO, bool VEC>
__device__ __forceinline__ void load8(const void *base, long long i, int n, int step, float2 (&v)[4]) {
    if (!base) n = 0;
    if (VEC) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[4];
            unpack4<IO, VEC>(load_raw4<IO, VEC>(base, i + 4 * h, n, n - 4 * h), f);
            v[2 * h] = make_float2(f[0], f[1]);
            v[2 * h + 1] = make_float2(f[2], f[3]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int left = n - j * step;
            v[j].x = left > 0 ? ld_io<IO>(base, (size_t)(i + j * step)) : 0.f;
            v[j].y = left > 1 ? ld_io<IO>(base, (size_t)(i + j * step + 1)) : 0.f;
        }
    }
}
template <bool VEC>
__device__ __forceinline__ void weights(const float *w, int c, int n, int step, float2 (&v)[4]) {
    load8<IO_F32, VEC>(w, c, n, step, v);
    if (!w)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = dup(1.f);
}
// scale w_post
template <bool VEC>
__device__ __forceinline__ void post_weights(const BlockNormParams &p, int c, int n, int step, float2 (&v)[4]) {
    float2 s[4];
    weights<VEC>(p.w_post, c, n, step, v);
    weights<VEC>(p.scale, c, n, step, s);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __fmul2_rn(v[j], s[j]);
}

// The slots of a CTA's threads for one row, K units each: NI tensors in the
// block's type, then NS in the stream's. A unit lies in one piece, 16 bytes of a 16-bit type or 32 of fp32 per thread.
template <int IO, int SIO, int K, int NI, int NS>
struct NormSlots {
    static constexpr int kPerThread = K * (NI * Eight<IO>::kBytes + NS * Eight<SIO>::kBytes);
};

template <int IO, int SIO, int K, bool VEC, int MAXT>
__global__ void __launch_bounds__(MAXT)
block_norm_kernel(BlockNormParams p, int stages) {
    using S = NormSlots<IO, SIO, K, 2, 1>;  // o, gate; r
    extern __shared__ __align__(16) char ring[];
    __shared__ float red[2][1][32];
    constexpr int kEi = Eight<IO>::kEs, kEs = Eight<SIO>::kEs, kBi = Eight<IO>::kBytes, kBs = Eight<SIO>::kBytes;
    const int tx = threadIdx.x, tpr = blockDim.x, nthr = blockDim.x * blockDim.y;
    const int cx = tx * (VEC ? 8 : 2), ps = VEC ? 2 : 2 * tpr;  // the first element of unit 0; from pair to pair
    char *mine = ring + (threadIdx.y * blockDim.x + tx) * kBi;                   // + (i K + k) line
    char *mine_s = ring + 2 * K * kBi * nthr + (threadIdx.y * blockDim.x + tx) * kBs;  // + k line_s
    const int line = nthr * kBi, line_s = nthr * kBs, stage = nthr * S::kPerThread;
    const float inv_d = 1.f / (float)p.D;
    const long long step = (long long)gridDim.x * blockDim.y;
    auto copy = [&](long long row, int at) {
        if (row < p.rows) {
            const long long base = row * p.D + cx, gbase = p.gate ? row / p.rows_per_gate * p.D + cx : 0;
            const char *r = static_cast<const char *>(p.r) + base * kEs, *o = static_cast<const char *>(p.o) + base * kEi,
                       *g = static_cast<const char *>(p.gate) + gbase * kEi;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int n = p.D - cx - tpr * k * 8;
                copy8<SIO, VEC>(mine_s + at + k * line_s, r + tpr * k * kBs, n, ps);
                if (p.o) copy8<IO, VEC>(mine + at + k * line, o + tpr * k * kBi, n, ps);
                if (p.gate) copy8<IO, VEC>(mine + at + (K + k) * line, g + tpr * k * kBi, n, ps);
            }
        }
        cp_commit();
    };
    long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    int at = 0;
    if (stages == 2) copy(row, 0);
    float2 wp[K][4], ws[K][4];  // w_pre; scale w_post
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = cx + tpr * k * 8, n = p.D - c;
        weights<VEC>(p.w_pre, c, n, ps, wp[k]);
        post_weights<VEC>(p, c, n, ps, ws[k]);
    }
    for (; row < p.rows; row += step) {
        if (stages == 2) {
            copy(row + step, stage - at);
            cp_wait<1>();
        } else {
            copy(row, 0);
            cp_wait<0>();
        }
        const long long base = row * p.D + cx;
        float inv = 1.f;
        if (p.o && p.w_post) {
            float2 s2 = dup(0.f);
#pragma unroll
            for (int k = 0; k < K; ++k) {  // zeros past the row's end
                float2 o[4];
                read8<IO>(mine + at + k * line, o);
#pragma unroll
                for (int j = 0; j < 4; ++j) s2 = __ffma2_rn(o[j], o[j], s2);
            }
            float ss[1] = {s2.x + s2.y};
            row_sum(ss, red[0]);
            inv = rsqrtf(ss[0] * inv_d + p.eps);
        }
        float2 r[K][4], s2 = dup(0.f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int n = p.D - cx - tpr * k * 8;
            read8<SIO>(mine_s + at + k * line_s, r[k]);
            if (p.o) {
                float2 o[4];
                read8<IO>(mine + at + k * line, o);
                if (p.gate) {
                    float2 g[4];
                    read8<IO>(mine + at + (K + k) * line, g);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = __fmul2_rn(o[j], g[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = __ffma2_rn(ws[k][j], __fmul2_rn(o[j], dup(inv)), r[k][j]);
                    r[k][j] = make_float2(round_io<SIO>(v.x), round_io<SIO>(v.y));  // as it is stored
                }
                store8<SIO, VEC>(static_cast<char *>(p.r_out) + (base + tpr * k * 8) * kEs, n, ps, r[k]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) s2 = __ffma2_rn(r[k][j], r[k][j], s2);
        }
        float ss[1] = {s2.x + s2.y};
        row_sum(ss, red[1]);
        const float2 inv2 = dup(rsqrtf(ss[0] * inv_d + p.eps));
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int j = 0; j < 4; ++j) r[k][j] = __fmul2_rn(__fmul2_rn(r[k][j], inv2), wp[k][j]);
            store8<IO, VEC>(static_cast<char *>(p.n) + (base + tpr * k * 8) * kEi, p.D - cx - tpr * k * 8, ps, r[k]);
        }
        if (!(p.o && p.w_post) && blockDim.x > 32) __syncthreads();  // one reduction per row only: its slot is free again
        if (stages == 2) at = stage - at;
    }
}

// MAXT: the threads a row may take (fewer leave each more registers).  WHOLE: the
// slots hold dr_out and the gate too; rows too wide for that load them where they are used.
template <int IO, int SIO, int K, bool VEC, int MAXT, bool WHOLE>
__global__ void __launch_bounds__(MAXT, MAXT == 128 ? 4 : 1)
block_norm_bwd_kernel(BlockNormParams p, int stages) {
    tc::pdl_launch_dependents();
    constexpr int NI = WHOLE ? 3 : 2;
    using S = NormSlots<IO, SIO, K, NI, WHOLE ? 2 : 1>;  // o, dn, gate; r', dr_out
    extern __shared__ __align__(16) char ring[];
    __shared__ float red[2][3][32];
    constexpr int kEi = Eight<IO>::kEs, kEs = Eight<SIO>::kEs, kBi = Eight<IO>::kBytes, kBs = Eight<SIO>::kBytes;
    const int tx = threadIdx.x, tpr = blockDim.x, nthr = blockDim.x * blockDim.y;
    const int cx = tx * (VEC ? 8 : 2), ps = VEC ? 2 : 2 * tpr;  // the first element of unit 0; from pair to pair
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
    char *mine = ring + (threadIdx.y * blockDim.x + tx) * kBi;                          // + (i K + k) line
    char *mine_s = ring + NI * K * kBi * nthr + (threadIdx.y * blockDim.x + tx) * kBs;  // + (i K + k) line_s
    const int line = nthr * kBi, line_s = nthr * kBs, stage = nthr * S::kPerThread;
    auto copy = [&](long long row, int at) {
        if (row < r1) {
            const long long base = row * p.D + cx, gbase = p.gate ? row / p.rows_per_gate * p.D + cx : 0;
            const char *r = static_cast<const char *>(p.r_out) + base * kEs, *n = static_cast<const char *>(p.dn) + base * kEi,
                       *o = static_cast<const char *>(p.o) + base * kEi, *d = static_cast<const char *>(p.dr_out) + base * kEs,
                       *g = static_cast<const char *>(p.gate) + gbase * kEi;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int nv = p.D - cx - tpr * k * 8;
                copy8<SIO, VEC>(mine_s + at + k * line_s, r + tpr * k * kBs, nv, ps);
                copy8<IO, VEC>(mine + at + (K + k) * line, n + tpr * k * kBi, nv, ps);
                if (p.o) copy8<IO, VEC>(mine + at + k * line, o + tpr * k * kBi, nv, ps);
                if (WHOLE && p.dr_out) copy8<SIO, VEC>(mine_s + at + (K + k) * line_s, d + tpr * k * kBs, nv, ps);
                if (WHOLE && p.gate) copy8<IO, VEC>(mine + at + (2 * K + k) * line, g + tpr * k * kBi, nv, ps);
            }
        }
        cp_commit();
    };
    int at = 0;
    if (stages == 2) copy(r0, 0);
    float2 acc1[K][4], acc2[K][4], wp[K][4], ws[K][4];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = cx + tpr * k * 8, n = p.D - c;
#pragma unroll
        for (int j = 0; j < 4; ++j) acc1[k][j] = acc2[k][j] = dup(0.f);
        weights<VEC>(p.w_pre, c, n, ps, wp[k]);
        post_weights<VEC>(p, c, n, ps, ws[k]);
    }
    const float inv_d = 1.f / (float)p.D;
    for (long long row = r0; row < r1; ++row) {
        if (stages == 2) {
            copy(row + 1, stage - at);
            cp_wait<1>();
        } else {
            copy(row, 0);
            cp_wait<0>();
        }
        const long long base = row * p.D + cx;
        float2 s0 = dup(0.f), s1 = dup(0.f), s2 = dup(0.f);
#pragma unroll
        for (int k = 0; k < K; ++k) {  // zeros past the row's end
            float2 r[4], n[4];
            read8<SIO>(mine_s + at + k * line_s, r);
            read8<IO>(mine + at + (K + k) * line, n);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s0 = __ffma2_rn(r[j], r[j], s0);
                s1 = __ffma2_rn(__fmul2_rn(n[j], wp[k][j]), r[j], s1);
            }
            if (p.o) {
                read8<IO>(mine + at + k * line, n);
#pragma unroll
                for (int j = 0; j < 4; ++j) s2 = __ffma2_rn(n[j], n[j], s2);
            }
        }
        float s[3] = {s0.x + s0.y, s1.x + s1.y, s2.x + s2.y};  // |r'|^2, dn w_pre . r', |o|^2
        row_sum(s, red[0]);
        const float inv2 = rsqrtf(s[0] * inv_d + p.eps), m2 = s[1] * inv_d * inv2 * inv2;
        const float inv = p.w_post ? rsqrtf(s[2] * inv_d + p.eps) : 1.f;
        float2 t2 = dup(0.f), u[K][4];  // u . o
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = cx + tpr * k * 8, nv = p.D - c;
            const long long to = base + tpr * k * 8;
            float2 dr[4], r[4], n[4];
            read8<SIO>(mine_s + at + k * line_s, r);
            read8<IO>(mine + at + (K + k) * line, n);
            if (WHOLE && p.dr_out) read8<SIO>(mine_s + at + (K + k) * line_s, dr);
            else load8<SIO, VEC>(p.dr_out, to, nv, ps, dr);  // zeros when absent
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // dr = (v - r' inv2^2 mean(v r')) inv2 + dr_out
                const float2 v = __ffma2_rn(r[j], dup(-m2), __fmul2_rn(n[j], wp[k][j]));
                dr[j] = __ffma2_rn(v, dup(inv2), dr[j]);
                acc2[k][j] = __ffma2_rn(n[j], __fmul2_rn(r[j], dup(inv2)), acc2[k][j]);
            }
            store8<SIO, VEC>(static_cast<char *>(p.dr) + to * kEs, nv, ps, dr);
            if (!p.o) continue;
            float2 o[4];
            read8<IO>(mine + at + k * line, o);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                r[j] = __fmul2_rn(dr[j], __fmul2_rn(o[j], dup(inv)));  // dr hat_o
                u[k][j] = __fmul2_rn(dr[j], ws[k][j]);
            }
            if (p.gate) {
                if (!seq_gate) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) n[j] = __fmul2_rn(r[j], ws[k][j]);
                    store8<IO, VEC>(static_cast<char *>(p.dgate) + to * kEi, nv, ps, n);
                }
                if (WHOLE) read8<IO>(mine + at + (2 * K + k) * line, n);
                else load8<IO, VEC>(p.gate, row / p.rows_per_gate * p.D + c, nv, ps, n);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u[k][j] = __fmul2_rn(u[k][j], n[j]);
                    if (!seq_gate) r[j] = __fmul2_rn(r[j], n[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                t2 = __ffma2_rn(u[k][j], o[j], t2);
                acc1[k][j] = __fadd2_rn(acc1[k][j], r[j]);
            }
        }
        if (p.o) {
            float t[1] = {t2.x + t2.y};
            row_sum(t, red[1]);
            const float m = p.w_post ? t[0] * inv_d * inv * inv : 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float2 o[4];
                read8<IO>(mine + at + k * line, o);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = __fmul2_rn(__ffma2_rn(o[j], dup(-m), u[k][j]), dup(inv));
                store8<IO, VEC>(static_cast<char *>(p.d_o) + (base + tpr * k * 8) * kEi, p.D - cx - tpr * k * 8, ps, o);
            }
        } else if (blockDim.x > 32) {
            __syncthreads();  // the slot of the sums is free again
        }
        if (stages == 2) at = stage - at;
    }
    float *part = p.part + chunk * 2 * p.D;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = cx + tpr * k * 8 + j / 2 * ps + j % 2;
            if (c < p.D) {
                part[c] = j & 1 ? acc1[k][j / 2].y : acc1[k][j / 2].x;
                part[p.D + c] = j & 1 ? acc2[k][j / 2].y : acc2[k][j / 2].x;
            }
        }
}

// The column sums over the chunks, in a fixed order: 64 interleaved sums per column,
// then those over a warp.  16 columns per CTA, so that 2048 of them reach 128 SMs.
// With fewer than 64 gates of several rows, the threads of a column share a gate's chunks.
constexpr int kSumX = 16, kSumY = 64;

// Rows q0, q0 + step, .. below q1 of the partial sums, four rows' loads together.
__device__ __forceinline__ void sum_chunks(const BlockNormParams &p, int c, long long q0, long long q1, int step, float &s1,
                                           float &s2) {
    for (long long q = q0; q < q1; q += 4 * step) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool ok = q + step * j < q1;
            v[j] = ok ? p.part[(q + step * j) * 2 * p.D + c] : 0.f;
            v[4 + j] = ok ? p.part[((q + step * j) * 2 + 1) * p.D + c] : 0.f;
        }
        s1 += (v[0] + v[1]) + (v[2] + v[3]);
        s2 += (v[4] + v[5]) + (v[6] + v[7]);
    }
}

template <int IO>
__global__ void __launch_bounds__(kSumX * kSumY)
block_norm_sum_kernel(BlockNormParams p) {
    __shared__ float red[2][kSumY][kSumX + 1];
    tc::pdl_wait();
    const int x = threadIdx.x, y = threadIdx.y, c = blockIdx.x * kSumX + x;
    const bool in = c < p.D;
    float s1 = 0.f, s2 = 0.f;
    if (p.gate && p.rows_per_gate > 1) {
        const long long per = (p.rows_per_gate + p.chunk_rows - 1) / p.chunk_rows, gates = p.rows / p.rows_per_gate;
        int split = 1;  // threads per gate
        while (2 * split * gates <= kSumY) split *= 2;
        const int sub = y % split;
        const float w = in ? (p.w_post ? __ldg(p.w_post + c) : 1.f) * (p.scale ? __ldg(p.scale + c) : 1.f) : 0.f;
        for (long long g0 = 0; g0 < gates; g0 += kSumY / split) {  // more than once only with a thread per gate
            const long long gi = g0 + y / split;
            float s = 0.f;
            if (in && gi < gates) sum_chunks(p, c, gi * per + sub, (gi + 1) * per, split, s, s2);
            if (split > 1) {
                red[0][y][x] = s;
                __syncthreads();
                if (sub == 0)
                    for (int k = 1; k < split; ++k) s += red[0][y + k][x];
                __syncthreads();
            }
            if (in && gi < gates && sub == 0) {
                st_io<IO>(p.dgate, (size_t)(gi * p.D + c), s * w);
                s1 = fmaf(ld_io<IO>(p.gate, (size_t)(gi * p.D + c)), s, s1);
            }
        }
    } else if (in) {
        sum_chunks(p, c, y, p.chunks, kSumY, s1, s2);
    }
    red[0][y][x] = s1;
    red[1][y][x] = s2;
    __syncthreads();
    // a warp per column and sum
    const int lane = (y * kSumX + x) & 31, job = (y * kSumX + x) >> 5, which = job / kSumX, col = blockIdx.x * kSumX + job % kSumX;
    float s = red[which][lane][job % kSumX] + red[which][lane + 32][job % kSumX];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane != 0 || col >= p.D) return;
    if (which == 1) {
        p.dw_pre[col] = s;
        return;
    }
    if (p.dw_post) p.dw_post[col] = (p.scale ? __ldg(p.scale + col) : 1.f) * s;
    if (p.dscale) p.dscale[col] = (p.w_post ? __ldg(p.w_post + col) : 1.f) * s;
}

// Threads of a row and rows of a CTA for K units of eight elements per thread.
dim3 row_block(int D, int K) {
    const int tpr = ((D + 8 * K - 1) / (8 * K) + 31) / 32 * 32;
    return dim3(tpr, tpr == 32 ? 4 : 1);
}

// Units per thread: two, but one for rows that a warp takes so, and backwards four for rows past 8192,
// whose registers would not allow more threads; wider rows take more warps.  Rows of 256 with one
// unit and two: 148 and 154 us (262144 rows).  One unit and two are level at rows of 512 and 1024 (49.8 and
// 88.7 us, 65536 rows) and within 2 % at 2048 (132 and 134 us; four 138), and with two 512 threads
// take rows of up to 8192.  Four units backwards do not fit the registers: 488 to 656 bytes a thread are
// spilled, and 2048 rows of 10240 take 168 us (148 and the sums 20; 49 for their bytes).
int norm_k(int D, bool backward) { return D <= 256 ? 1 : backward && D > 8192 ? 4 : 2; }

// Whether every tensor moves in whole, aligned units (absent ones do).
bool norm_vec(const BlockNormParams &p) {
    bool ok = p.D % 8 == 0;
    for (const void *q : {p.o, p.r, p.gate, (const void *)p.n, (const void *)p.r_out, p.dn, p.dr_out, (const void *)p.d_o,
                          (const void *)p.dr, (const void *)p.dgate, (const void *)p.w_post, (const void *)p.w_pre,
                          (const void *)p.scale})
        ok = ok && chunk_aligned(q);
    return ok;
}

template <int IO, int SIO, int K, int MAXT>
cudaError_t launch_norm_as(const BlockNormParams &p, cudaStream_t s) {
    const dim3 block = row_block(p.D, K);
    auto *kernel = norm_vec(p) ? block_norm_kernel<IO, SIO, K, true, MAXT> : block_norm_kernel<IO, SIO, K, false, MAXT>;
    const int row = (int)(block.x * block.y) * NormSlots<IO, SIO, K, 2, 1>::kPerThread;
    const int stages = 2 * row <= kSmemMost ? 2 : 1, bytes = stages * row;
    cudaError_t e = allow_smem<kSmemMost>(kernel);  // bytes depend on D
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
    if (norm_k(p.D, false) == 1) return launch_norm_as<IO, SIO, 1, 128>(p, s);
    return p.D <= 8192 ? launch_norm_as<IO, SIO, 2, 512>(p, s) : launch_norm_as<IO, SIO, 2, 1024>(p, s);
}

template <int IO, int SIO, int K, int MAXT, bool WHOLE>
cudaError_t launch_norm_bwd_as(const BlockNormParams &p, cudaStream_t s) {
    const dim3 block = row_block(p.D, K);
    auto *kernel = norm_vec(p) ? block_norm_bwd_kernel<IO, SIO, K, true, MAXT, WHOLE>
                               : block_norm_bwd_kernel<IO, SIO, K, false, MAXT, WHOLE>;
    const int row = block.x * block.y * NormSlots<IO, SIO, K, WHOLE ? 3 : 2, WHOLE ? 2 : 1>::kPerThread;
    const int stages = 2 * row <= kSmemMost ? 2 : 1, bytes = stages * row;
    cudaError_t e = allow_smem<kSmemMost>(kernel);  // bytes depend on D
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)((p.chunks + block.y - 1) / block.y), block, bytes, s>>>(p, stages);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_kernel(true, block_norm_sum_kernel<IO>, dim3((p.D + kSumX - 1) / kSumX), dim3(kSumX, kSumY), 0, s, p);
}

template <int IO, int SIO>
cudaError_t launch_norm_bwd_io(const BlockNormParams &p, cudaStream_t s) {
    switch (norm_k(p.D, true)) {
        case 1: return launch_norm_bwd_as<IO, SIO, 1, 128, true>(p, s);
        case 2: return p.D <= 2048 ? launch_norm_bwd_as<IO, SIO, 2, 128, true>(p, s) : launch_norm_bwd_as<IO, SIO, 2, 512, true>(p, s);
        // 512 threads' whole slots: 160 KB of 16-bit tensors, too much with fp32 ones
        // (2048 rows of 10240: 168 us whole, 201 not)
        default: return launch_norm_bwd_as<IO, SIO, 4, 512, IO != IO_F32 && SIO != IO_F32>(p, s);
    }
}

}  // namespace

// Chunks for about 16 warps per SM, two at least; a chunk never spans two gates of several rows.
// (8192 rows of 2048: 66 us with eight warps, 64 with 16, 70 with 32.)
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

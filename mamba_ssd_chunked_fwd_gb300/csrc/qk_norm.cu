// qk_norm.cu -- norm of queries and keys, head by head, with the rotation by
// position in the same pass; forward and backward.
//
//   v = x / sqrt(mean(x^2) + eps) * w         (l2: the sum in place of the mean; w optional)
//   pair i of v turns by the angle a = position * freqs[i]:  (v1, v2) -> (v1 cos a - v2 sin a, v2 cos a + v1 sin a)
//
// Backward, with d the incoming gradient turned by -a, r the inverse root and m the
// divisor of the mean (N or 1):  dw = sum d x r,  dx = r (d w - x r^2 (d w . x) / m).
//
// Bound by HBM: each value is read once and written once.  A group of LPR lanes
// holds a head's vector, two runs of Q elements to a lane, chosen so that both
// members of a pair lie in one lane: no exchange but the sums.  The angles are worked out once
// for a tile of tokens and shared by its heads through shared memory.  [8,4096] with 32 and 8 heads of 128, bf16, rotated: 121 us,
// 82 % of a plain copy's rate; gradients of [4,2048] with 16 and 16: 65 us (50 %: registers leave two rows to a warp in flight).
#include "qk_norm.cuh"

namespace ssd {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = 128;
constexpr int kTokens = 16;  // most tokens of a tile (forward 8)

// The position's turns are kept as a fraction of 2^64: position times
// freq / (2 pi), whole turns dropped by the overflow.  The product loses nothing, however far
// the position; freq / (2 pi) is off by 2^-52 of itself, 4e-10 of a turn at position 10^6.
__device__ __forceinline__ unsigned long long turn_of(float freq) {
    double f = (double)freq * 0.15915494309189535;  // 1 / (2 pi)
    f -= floor(f);
    return (unsigned long long)(f * 18446744073709551616.0);
}
__device__ __forceinline__ float2 cos_sin(unsigned long long turn, int position) {
    const unsigned long long a = turn * (unsigned long long)(long long)position;
    float c, s;
    sincospif((float)(int)(a >> 32) * 4.656612873077393e-10f, &s, &c);  // half turns in [-1, 1)
    return make_float2(c, s);
}

// Where unit u of a vector lies: its two runs of Q elements, and whether they are turned.
struct Unit {
    int a, b, f;  // first elements of the runs, first frequency
    bool rot;
};
template <int Q>
__device__ __forceinline__ Unit unit_of(int u, int half, int interleaved) {
    Unit x;
    if (interleaved) {
        x.a = 2 * u * Q, x.b = x.a + Q, x.f = u * Q, x.rot = u * Q < half;
    } else if (u * Q < half) {
        x.a = u * Q, x.b = half + u * Q, x.f = u * Q, x.rot = true;
    } else {
        x.a = 2 * u * Q, x.b = x.a + Q, x.f = 0, x.rot = false;
    }
    return x;
}

// A run of Q elements: 16 or 8 bytes, or one element.
template <int IO, int Q>
__device__ __forceinline__ Raw4 load_run(const void *base, long long i, bool ok) {
    if (Q == 1) return load_raw4<IO, false, false>(base, i, ok, 1);
    Raw4 r = {{0u, 0u, 0u, 0u}};
    const char *at = static_cast<const char *>(base) + i * (IO == IO_F32 ? 4 : 2);
    if (IO == IO_F32 || Q == 8) ld_v4(r.w, at, ok);
    else ld_v2(r.w, at, ok);
    return r;
}
template <int IO>
__device__ __forceinline__ float first_of(uint32_t w) {
    return IO == IO_F32 ? __uint_as_float(w) : IO == IO_BF16 ? __uint_as_float(w << 16) : __half2float(__ushort_as_half((unsigned short)w));
}
template <int IO>
__device__ __forceinline__ float second_of(uint32_t w) {
    return IO == IO_BF16 ? __uint_as_float(w & 0xffff0000u) : __half2float(__ushort_as_half((unsigned short)(w >> 16)));
}
// Two runs as pairs, element j of both side by side: what follows is packed arithmetic, one instruction to a pair.
template <int IO, int Q>
__device__ __forceinline__ void unpack_runs(const Raw4 &a, const Raw4 &b, float2 (&v)[Q]) {
#pragma unroll
    for (int j = 0; j < Q; ++j) {
        if (IO == IO_F32 || Q == 1) v[j] = make_float2(first_of<IO>(a.w[j & 3]), first_of<IO>(b.w[j & 3]));
        else if (j % 2 == 0) v[j] = make_float2(first_of<IO>(a.w[(j / 2) & 3]), first_of<IO>(b.w[(j / 2) & 3]));
        else v[j] = make_float2(second_of<IO>(a.w[(j / 2) & 3]), second_of<IO>(b.w[(j / 2) & 3]));
    }
}
// The first (second) of the pairs as a run in memory.
template <int IO, int Q>
__device__ __forceinline__ void store_run(void *base, long long i, const float2 (&v)[Q], bool second) {
    auto of = [&](int j) { return second ? v[j % Q].y : v[j % Q].x; };
    if (Q == 1) {
        st_io<IO>(base, i, of(0));
    } else if (IO == IO_F32) {
        reinterpret_cast<float4 *>(static_cast<float *>(base) + i)[0] = make_float4(of(0), of(1), of(2), of(3));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack16<IO>(make_float2(of(2 * j), of(2 * j + 1)));
        if (Q == 8) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + i) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(base) + i) = make_uint2(w[0], w[1]);
    }
}

// The pairs of a unit turned by their angles (sign -1: back).  Angle j of the unit lies at cs[j step], so that lanes read
// neighbours.
template <int Q>
__device__ __forceinline__ void turn_unit(float2 (&v)[Q], const float2 *cs, int step, bool interleaved, float sign) {
    if (Q == 1 || !interleaved) {  // the partners are the pair
#pragma unroll
        for (int j = 0; j < Q; ++j) {
            const float2 t = cs[j * step];
            const float s = sign * t.y;
            v[j] = __ffma2_rn(make_float2(v[j].y, v[j].x), make_float2(-s, s), __fmul2_rn(v[j], dup(t.x)));
        }
    } else {  // partners are neighbours of each run
#pragma unroll
        for (int j = 0; j < Q / 2; ++j) {
            const float2 t = cs[j * step], u = cs[(j + Q / 2) * step];
            const float2 c = make_float2(t.x, u.x), s = make_float2(sign * t.y, sign * u.y), x = v[2 * j], y = v[2 * j + 1];
            v[2 * j] = __ffma2_rn(y, make_float2(-s.x, -s.y), __fmul2_rn(x, c));
            v[2 * j + 1] = __ffma2_rn(x, s, __fmul2_rn(y, c));
        }
    }
}

template <int LPR>
__device__ __forceinline__ float sum_group(float v) {
#pragma unroll
    for (int m = 1; m < LPR; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// One tensor's rows of a tile: `heads` of each of nt tokens, RU rows in flight so that their loads overlap.
// `from`: where the tile's tokens begin; `magic`: ceil(2^32 / heads), for r / heads (0: one head).
template <int IO, int Q, int M, int LPR, bool BWD>
__device__ __forceinline__ void rows_of(const QkNormParams &p, int which, long long tok0, int nt, const float2 *table, const long long *from,
                                        uint32_t magic, float2 (&dw)[M][Q]) {
    constexpr int kGroups = kThreads / LPR, RU = M > 1 ? 1 : BWD || Q == 8 ? 2 : 4;
    const int heads = which ? p.G : p.H, ln = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const void *x = which ? p.k : p.q, *dy = which ? p.dk_out : p.dq_out;
    const float *w = which ? p.w_k : p.w_q;
    void *out = BWD ? (which ? p.dk : p.dq) : (which ? p.k_out : p.q_out);
    const float div = p.l2 ? 1.f : 1.f / p.N;
    Unit un[M];
    bool oka[M], okb[M];
    float2 wt[M][Q];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        un[m] = unit_of<Q>(ln + LPR * m, p.half, p.interleaved);
        oka[m] = un[m].a < p.N, okb[m] = un[m].b < p.N;
#pragma unroll
        for (int j = 0; j < Q; ++j) {
            wt[m][j] = make_float2(w && oka[m] ? __ldg(w + un[m].a + j) : 1.f, w && okb[m] ? __ldg(w + un[m].b + j) : 1.f);
        }
    }
    const int rows = nt * heads;
    Raw4 xa[RU][M], xb[RU][M], da[RU][M], db[RU][M];
    long long to[RU];
    int tk[RU];
    bool ok[RU];
    auto load = [&](int i, int r) {
        ok[i] = r < rows;
        tk[i] = ok[i] ? (magic ? (int)__umulhi((uint32_t)r, magic) : r) : 0;
        const long long at = from[tk[i]] + (long long)(r - tk[i] * heads) * p.N;
        to[i] = (tok0 * heads + r) * p.N;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            xa[i][m] = load_run<IO, Q>(x, at + un[m].a, ok[i] && oka[m]);
            xb[i][m] = load_run<IO, Q>(x, at + un[m].b, ok[i] && okb[m]);
            if (BWD) {
                da[i][m] = load_run<IO, Q>(dy, to[i] + un[m].a, ok[i] && oka[m]);
                db[i][m] = load_run<IO, Q>(dy, to[i] + un[m].b, ok[i] && okb[m]);
            }
        }
    };
    const int apart = p.half / Q;  // the units that turn
    auto work = [&](int i) {
        float2 v[M][Q], sq = make_float2(0.f, 0.f);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            unpack_runs<IO, Q>(xa[i][m], xb[i][m], v[m]);
#pragma unroll
            for (int j = 0; j < Q; ++j) sq = __ffma2_rn(v[m][j], v[m][j], sq);
        }
        const float inv = rsqrtf(fmaf(sum_group<LPR>(sq.x + sq.y), div, p.eps));
        const float2 *cs = table + tk[i] * p.half;
        if constexpr (!BWD) {
#pragma unroll
            for (int m = 0; m < M; ++m) {
#pragma unroll
                for (int j = 0; j < Q; ++j) v[m][j] = __fmul2_rn(v[m][j], __fmul2_rn(dup(inv), wt[m][j]));
                if (un[m].rot) turn_unit<Q>(v[m], cs + un[m].f / Q, apart, p.interleaved, 1.f);
                if (ok[i] && oka[m]) store_run<IO, Q>(out, to[i] + un[m].a, v[m], false);
                if (ok[i] && okb[m]) store_run<IO, Q>(out, to[i] + un[m].b, v[m], true);
            }
        } else {
            float2 g[M][Q], dot = make_float2(0.f, 0.f);
            const float2 part = dup(ok[i] ? inv : 0.f);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                unpack_runs<IO, Q>(da[i][m], db[i][m], g[m]);
                if (un[m].rot) turn_unit<Q>(g[m], cs + un[m].f / Q, apart, p.interleaved, -1.f);
#pragma unroll
                for (int j = 0; j < Q; ++j) {
                    const float2 x = __fmul2_rn(g[m][j], v[m][j]);
                    dw[m][j] = __ffma2_rn(x, part, dw[m][j]);
                    dot = __ffma2_rn(x, wt[m][j], dot);
                    g[m][j] = __fmul2_rn(g[m][j], wt[m][j]);
                }
            }
            // r^3 alone leaves fp32's range where rows are near 1e-13 or 1e13; with the sum, which has their size, r^2 is the most
            const float2 f = dup(-inv * (inv * (inv * (div * sum_group<LPR>(dot.x + dot.y)))));
#pragma unroll
            for (int m = 0; m < M; ++m) {
#pragma unroll
                for (int j = 0; j < Q; ++j) g[m][j] = __ffma2_rn(f, v[m][j], __fmul2_rn(dup(inv), g[m][j]));
                if (ok[i] && oka[m]) store_run<IO, Q>(out, to[i] + un[m].a, g[m], false);
                if (ok[i] && okb[m]) store_run<IO, Q>(out, to[i] + un[m].b, g[m], true);
            }
        }
    };
    // r0 - grp < rows: the same number of rounds for every lane of a warp
    if constexpr (BWD && RU == 2) {  // a row's loads run while the one before is worked on
        load(0, grp);
        for (int r0 = grp; r0 - grp < rows; r0 += 2 * kGroups) {
            load(1, r0 + kGroups);
            work(0);
            load(0, r0 + 2 * kGroups);
            work(1);
        }
    } else {
        for (int r0 = grp; r0 - grp < rows; r0 += kGroups * RU) {
#pragma unroll
            for (int i = 0; i < RU; ++i) load(i, r0 + i * kGroups);
#pragma unroll
            for (int i = 0; i < RU; ++i) work(i);
        }
    }
}

// The CTA's sums of dw, the groups one after another.
template <int Q, int M, int LPR>
__device__ __forceinline__ void store_sums(const QkNormParams &p, const float2 (&dw)[M][Q]) {
    __shared__ float sums[2 * kMaxHalf];
    for (int i = threadIdx.x; i < p.N; i += kThreads) sums[i] = 0.f;
    for (int g = 0; g < kThreads / LPR; ++g) {
        __syncthreads();
        if ((int)threadIdx.x / LPR != g) continue;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const Unit un = unit_of<Q>(threadIdx.x % LPR + LPR * m, p.half, p.interleaved);
#pragma unroll
            for (int j = 0; j < Q; ++j) {
                if (un.a < p.N) sums[un.a + j] += dw[m][j].x;
                if (un.b < p.N) sums[un.b + j] += dw[m][j].y;
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.N; i += kThreads) p.part[(size_t)blockIdx.x * p.N + i] = sums[i];
}

// Backward a CTA takes one of the two tensors (the first nq of them the queries), so that one set of sums lies in registers.
template <int IO, int Q, int M, int LPR, bool BWD>
__global__ void __launch_bounds__(kThreads, M > 1 || BWD ? 2 : 3)
qk_norm_kernel(const __grid_constant__ QkNormParams p, int tile, int nq, uint32_t magic_q, uint32_t magic_k) {
    __shared__ __align__(16) float2 table[kTokens * kMaxHalf];
    __shared__ unsigned long long turn[kMaxHalf];
    __shared__ long long from[2][kTokens];
    const long long tokens = (long long)p.B * p.L;
    float2 dw[M][Q];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < Q; ++j) dw[m][j] = make_float2(0.f, 0.f);
    for (int i = threadIdx.x; i < p.half; i += kThreads) turn[i] = turn_of(__ldg(p.freqs + i));
    const int which = BWD && (int)blockIdx.x >= nq, first = blockIdx.x - which * nq, step = BWD ? (which ? gridDim.x - nq : nq) : gridDim.x;
    for (long long tok0 = (long long)first * tile; tok0 < tokens; tok0 += (long long)step * tile) {
        const int nt = (int)min((long long)tile, tokens - tok0);
        __syncthreads();
        if ((int)threadIdx.x < 2 * nt) {
            const long long tok = tok0 + (threadIdx.x >> 1), row = tok / p.L, t = tok - row * p.L;
            from[threadIdx.x & 1][threadIdx.x >> 1] = threadIdx.x & 1 ? row * p.ks[0] + t * p.ks[1] : row * p.qs[0] + t * p.qs[1];
        }
        for (int e = threadIdx.x; e < nt * p.half; e += kThreads) {
            const int t = e / p.half;
            const long long tok = tok0 + t;
            const int f = e - t * p.half;  // angle f % Q of unit f / Q
            table[t * p.half + (f % Q) * (p.half / Q) + f / Q] = cos_sin(turn[f], p.positions ? __ldg(p.positions + tok) : (int)(tok % p.L));
        }
        __syncthreads();
        if (!BWD || which == 0) rows_of<IO, Q, M, LPR, BWD>(p, 0, tok0, nt, table, from[0], magic_q, dw);
        if (!BWD || which == 1) rows_of<IO, Q, M, LPR, BWD>(p, 1, tok0, nt, table, from[1], magic_k, dw);
    }
    if constexpr (BWD) tc::pdl_launch_dependents();
    if constexpr (BWD) if (which ? p.w_k : p.w_q) store_sums<Q, M, LPR>(p, dw);
}

// dw_q, dw_k: the CTAs' sums, 32 threads to a column, each over every 32nd row.
__global__ void __launch_bounds__(1024)
qk_norm_weights_kernel(const __grid_constant__ QkNormParams p, int nq, int parts) {
    __shared__ float s[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, col = blockIdx.x * 32 + x, which = blockIdx.y;
    float *out = which ? p.dw_k : p.dw_q;
    tc::pdl_wait();
    if (!out) return;
    float v = 0.f;
    if (col < p.N)
#pragma unroll 4
        for (int i = (which ? nq : 0) + y; i < (which ? parts : nq); i += 32) v += p.part[(size_t)i * p.N + col];
    s[y][x] = v;
    __syncthreads();
    v = s[x][y];  // a warp to a column
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if (x == 0 && blockIdx.x * 32 + y < p.N) out[blockIdx.x * 32 + y] = v;
}

// Tokens of a tile: as many as leave every SM two CTAs, and rows that the division by a product serves (65536).
int tile_of(const QkNormParams &p, bool bwd) {
    if (p.H > 2048 || p.G > 2048) return 1;
    const long long tokens = (long long)p.B * p.L, most = tokens / (2LL * scan_sm_count());
    int t = 1;
    while (t < (bwd ? kTokens : kTokens / 2) && 2 * t <= most) t *= 2;
    return t;
}

// Of the backward's CTAs, two to an SM, those that take the queries: their share of the heads.
int parts_of_q(const QkNormParams &p, int parts) {
    const int q = (int)((long long)parts * p.H / (p.H + p.G));
    return q < 1 ? 1 : q > parts - 1 ? parts - 1 : q;
}

template <int IO, int Q, int M, int LPR>
cudaError_t norm_as(const QkNormParams &p, bool bwd, cudaStream_t s) {
    const int tile = tile_of(p, bwd);
    const uint32_t mq = (uint32_t)((0x100000000ull + p.H - 1) / p.H), mk = (uint32_t)((0x100000000ull + p.G - 1) / p.G);
    if (!bwd) {
        const long long tiles = ((long long)p.B * p.L + tile - 1) / tile;
        qk_norm_kernel<IO, Q, M, LPR, false><<<(unsigned)min(tiles, (long long)1 << 30), kThreads, 0, s>>>(p, tile, 0, mq, mk);
        return cudaGetLastError();
    }
    const int parts = qk_norm_parts(p), nq = parts_of_q(p, parts);
    qk_norm_kernel<IO, Q, M, LPR, true><<<parts, kThreads, 0, s>>>(p, tile, nq, mq, mk);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!p.w_q && !p.w_k)) return e;
    return launch_kernel(true, qk_norm_weights_kernel, dim3((p.N + 31) / 32, 2), dim3(1024), 0, s, p, nq, parts);
}

template <int IO>
cudaError_t norm_io(const QkNormParams &p, bool bwd, cudaStream_t s) {
    // Runs of 16 bytes, of 8 (16-bit elements), or elements: what every row begins and the rotated part ends at.
    auto by = [&](int q) {
        auto aligned = [&](const void *x) { return reinterpret_cast<uintptr_t>(x) % (q * (IO == IO_F32 ? 4 : 2)) == 0; };
        auto strided = [&](const void *x, const long long (&st)[2]) { return aligned(x) && st[0] % q == 0 && st[1] % q == 0; };
        return p.N % q == 0 && p.half % q == 0 && strided(p.q, p.qs) && strided(p.k, p.ks) &&
               (bwd ? aligned(p.dq_out) && aligned(p.dk_out) && aligned(p.dq) && aligned(p.dk) : aligned(p.q_out) && aligned(p.k_out));
    };
    if (IO != IO_F32 && by(8)) {
        constexpr int Q = IO == IO_F32 ? 4 : 8;
        if (p.N <= 64) return norm_as<IO, Q, 1, 32 / Q>(p, bwd, s);
        if (p.N <= 128) return norm_as<IO, Q, 1, 64 / Q>(p, bwd, s);
        return norm_as<IO, Q, 1, 128 / Q>(p, bwd, s);
    }
    if (!by(4)) return norm_as<IO, 1, 4, 32>(p, bwd, s);
    if (p.N <= 64) return norm_as<IO, 4, 1, 8>(p, bwd, s);
    if (p.N <= 128) return norm_as<IO, 4, 1, 16>(p, bwd, s);
    return norm_as<IO, 4, 1, 32>(p, bwd, s);
}

cudaError_t norm(const QkNormParams &p, int io, bool bwd, cudaStream_t s) {
    switch (io) {
        case IO_F32: return norm_io<IO_F32>(p, bwd, s);
        case IO_F16: return norm_io<IO_F16>(p, bwd, s);
        case IO_BF16: return norm_io<IO_BF16>(p, bwd, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

int qk_norm_parts(const QkNormParams &p) {
    const long long tiles = ((long long)p.B * p.L + tile_of(p, true) - 1) / tile_of(p, true), most = scan_sm_count();
    return (int)(2 * (tiles < most ? tiles : most));
}
cudaError_t launch_qk_norm(const QkNormParams &p, int io, cudaStream_t s) { return norm(p, io, false, s); }
cudaError_t launch_qk_norm_bwd(const QkNormParams &p, int io, cudaStream_t s) { return norm(p, io, true, s); }

}  // namespace ssd

// delta_walk.cu -- the gated delta rule token by token in fp32: forward, and the
// adjoint of the state backwards.  Any N <= 128 and any P: fp32 tensors, and 16-bit ones that
// delta_tc.cu does not take.
//
// The rows of a head's state (one for each of the P values) do not mix: row p
// needs the keys, the gates and v[p].  So a warp keeps its rows in registers, R to
// a lane with N / 8 columns each, and walks the tokens with no word to other
// warps but the tile of 16 tokens that the CTA loads for its four.
// Forward, with S the state before the token:
//     u = beta (v - a (S k)),  y = scale (a (S q) + u (k . q)),  S <- a S + u k^T,    a = exp(g)
// so that both sums over the state's columns come from the same S, side by side.
// Backward, with D the adjoint of the state after the token:
//     r = D k + d (q . k),  d = scale dy,  D <- a (D + d q^T - beta r k^T),  dv = beta r
// A tile's tokens behind the row's end have a = 1 and zeros elsewhere, which leaves a state as it is, so that
// every tile takes the same steps, laid out four at a time.
//
// Bound by the latency of a token's sums over eight lanes, so few heads get more warps with
// a row to a lane (R = 1), many heads R = 4.  [3,517] with 6 heads of 72 x 100: 98 us, 0.19 us a token (R = 4: 180).
#include "delta.cuh"

namespace ssd {

namespace {

constexpr int kTile = 16, kThreads = 128;

// A tile of `kTile` tokens as loaded, four elements at a time.
template <int NP, int R>
struct Staged {
    Raw4 k[NP / 32], q[NP / 32], v[(R + 1) / 2];
    float gate;
};

// ROWS = 16 R rows of the state to a CTA.
template <int NP, int R>
struct Tile {
    static constexpr int ROWS = 16 * R;
    float k[kTile][NP], q[kTile][NP], v[kTile][ROWS], out[kTile][ROWS], dv[kTile][ROWS];
    float a[kTile], beta[kTile], kq[kTile];
};

template <int IO, int NP, int R, bool VEC>
__device__ __forceinline__ void load_tile(const DeltaParams &p, const void *vals, const long long (&vst)[2], int b, int h, int p0, int t0,
                                          int len, Staged<NP, R> &r) {
    const int tid = threadIdx.x, gn = (h / (p.H / p.G)) * p.N;
#pragma unroll
    for (int i = 0; i < NP / 32; ++i) {
        const int e = tid + kThreads * i, t = t0 + e / (NP / 4), n = (e % (NP / 4)) * 4;
        const int ok = t < len && n < p.N;
        r.k[i] = load_raw4<IO, VEC>(p.k, b * p.ks[0] + t * p.ks[1] + gn + n, ok, p.N - n);
        r.q[i] = load_raw4<IO, VEC>(p.q, b * p.qs[0] + t * p.qs[1] + gn + n, ok, p.N - n);
    }
#pragma unroll
    for (int i = 0; i < (R + 1) / 2; ++i) {
        const int e = tid + kThreads * i, t = t0 + e / (4 * R), c = p0 + (e % (4 * R)) * 4;
        r.v[i] = load_raw4<IO, VEC>(vals, b * vst[0] + t * vst[1] + (long long)h * p.P + c, e < kTile * 4 * R && t < len && c < p.P, p.P - c);
    }
    const int t = t0 + (tid & 15);
    if (tid < 16) r.gate = load_gate<IO>(p.g, b * p.gs[0] + t * p.gs[1] + h, p.g32, t < len);
    else if (tid < 32) r.gate = load_gate<IO>(p.beta, b * p.bs[0] + t * p.bs[1] + h, p.b32, t < len);
}

template <int IO, int NP, int R, bool VEC>
__device__ __forceinline__ void put_tile(const Staged<NP, R> &r, Tile<NP, R> &s) {
    const int tid = threadIdx.x;
    float f[4];
#pragma unroll
    for (int i = 0; i < NP / 32; ++i) {
        const int e = tid + kThreads * i, t = e / (NP / 4), n = (e % (NP / 4)) * 4;
        unpack4<IO, VEC>(r.k[i], f);
        *reinterpret_cast<float4 *>(&s.k[t][n]) = make_float4(f[0], f[1], f[2], f[3]);
        unpack4<IO, VEC>(r.q[i], f);
        *reinterpret_cast<float4 *>(&s.q[t][n]) = make_float4(f[0], f[1], f[2], f[3]);
    }
#pragma unroll
    for (int i = 0; i < (R + 1) / 2; ++i) {
        const int e = tid + kThreads * i;
        unpack4<IO, VEC>(r.v[i], f);
        if (e < kTile * 4 * R) *reinterpret_cast<float4 *>(&s.v[e / (4 * R)][(e % (4 * R)) * 4]) = make_float4(f[0], f[1], f[2], f[3]);
    }
    if (tid < 16) s.a[tid] = expf(r.gate);
    else if (tid < 32) s.beta[tid - 16] = r.gate;
}

// k . q of the tile's tokens, eight lanes to each.
template <int NP, int R>
__device__ __forceinline__ void dot_tile(Tile<NP, R> &s) {
    const int t = threadIdx.x >> 3, ln = threadIdx.x & 7;
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < NP / 32; ++j) {
        const float4 a = *reinterpret_cast<const float4 *>(&s.k[t][32 * j + 4 * ln]), c = *reinterpret_cast<const float4 *>(&s.q[t][32 * j + 4 * ln]);
        v = fmaf(a.x, c.x, fmaf(a.y, c.y, fmaf(a.z, c.z, fmaf(a.w, c.w, v))));
    }
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if (ln == 0) s.kq[t] = v;
}

__device__ __forceinline__ float sum8(float2 v) {
    float r = v.x + v.y;
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) r += __shfl_xor_sync(0xffffffffu, r, m);
    return r;
}

// A lane's columns of a row with those of k or q, in two sums side by side.
template <int NP>
__device__ __forceinline__ float2 dot_row(const float2 (&s)[NP / 16], const float2 (&x)[NP / 16]) {
    float2 a = __fmul2_rn(s[0], x[0]), b = __fmul2_rn(s[1], x[1]);
#pragma unroll
    for (int m = 2; m < NP / 16; m += 2) {
        a = __ffma2_rn(s[m], x[m], a);
        b = __ffma2_rn(s[m + 1], x[m + 1], b);
    }
    return __fadd2_rn(a, b);
}

// Rows of a state in registers: lane ln of a group of eight holds columns 32 j + 4 ln + 0..3.
template <int NP, int R, bool VEC>
__device__ __forceinline__ void load_state(const float *src, int P, int N, int row0, int ln, float2 (&S)[R][NP / 16]) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < NP / 32; ++j) {
            const int n = 32 * j + 4 * ln;
            float f[4] = {0.f, 0.f, 0.f, 0.f};
            if (src) unpack4<IO_F32, VEC>(load_raw4<IO_F32, VEC>(src, (long long)(row0 + r) * N + n, row0 + r < P && n < N, N - n), f);
            S[r][2 * j] = make_float2(f[0], f[1]);
            S[r][2 * j + 1] = make_float2(f[2], f[3]);
        }
}
template <int NP, int R, bool VEC>
__device__ __forceinline__ void store_state(float *dst, int P, int N, int row0, int ln, const float2 (&S)[R][NP / 16]) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < NP / 32; ++j) {
            const int n = 32 * j + 4 * ln;
            const float f[4] = {S[r][2 * j].x, S[r][2 * j].y, S[r][2 * j + 1].x, S[r][2 * j + 1].y};
            if (row0 + r < P && n < N) store4_io<IO_F32, VEC>(dst, (long long)(row0 + r) * N + n, min(4, N - n), f);
        }
}

template <int NP>
__device__ __forceinline__ void read_row(const float *src, int ln, float2 (&v)[NP / 16]) {
#pragma unroll
    for (int j = 0; j < NP / 32; ++j) {
        const float4 f = *reinterpret_cast<const float4 *>(src + 32 * j + 4 * ln);
        v[2 * j] = make_float2(f.x, f.y);
        v[2 * j + 1] = make_float2(f.z, f.w);
    }
}

// A lane's R values of a token's.
template <int R>
__device__ __forceinline__ void read_rows(const float *src, float (&v)[R]) {
    if (R == 4) {
        const float4 f = *reinterpret_cast<const float4 *>(src);
        v[0] = f.x, v[R > 1] = f.y, v[R > 2 ? 2 : 0] = f.z, v[R > 3 ? 3 : 0] = f.w;
    } else {
        v[0] = src[0];
    }
}
template <int R>
__device__ __forceinline__ void write_rows(float *dst, const float (&v)[R]) {
    if (R == 4) *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[R > 1], v[R > 2 ? 2 : 0], v[R > 3 ? 3 : 0]);
    else dst[0] = v[0];
}

// STATES: for the gradients, the state before every chunk and u, in place of y.
template <int IO, int NP, int R, bool VEC, bool STATES>
__device__ __forceinline__ void walk_rows(const DeltaParams &p, int block, Tile<NP, R> &s) {
    constexpr int kRows = 16 * R;
    const int tiles = (p.P + kRows - 1) / kRows, p0 = (block % tiles) * kRows;
    const int bh = block / tiles, h = bh % p.H, b = bh / p.H;
    const int tid = threadIdx.x, lane = tid & 31, ln = lane & 7, lrow = (tid >> 5) * 4 * R + (lane >> 3) * R, row0 = p0 + lrow;
    const int len = delta_length(p, b);
    const size_t pn = (size_t)p.P * p.N;
    float2 S[R][NP / 16];
    load_state<NP, R, VEC>(p.h0 ? p.h0 + bh * pn : nullptr, p.P, p.N, row0, ln, S);
    Staged<NP, R> next;
    load_tile<IO, NP, R, VEC>(p, p.v, p.vs, b, h, p0, 0, len, next);
    for (int t0 = 0; t0 < len; t0 += kTile) {
        __syncthreads();
        put_tile<IO, NP, R, VEC>(next, s);
        load_tile<IO, NP, R, VEC>(p, p.v, p.vs, b, h, p0, t0 + kTile, len, next);
        __syncthreads();
        if (STATES) {
            if (t0 % kDeltaChunk == 0)
                store_state<NP, R, VEC>(p.states + ((size_t)bh * p.nc + t0 / kDeltaChunk) * pn, p.P, p.N, row0, ln, S);
        } else {
            dot_tile<NP, R>(s);
            __syncthreads();
        }
        const int nt = min(kTile, len - t0);
#pragma unroll (R == 1 ? 4 : 1)
        for (int i = 0; i < kTile; ++i) {
            float2 k[NP / 16], q[NP / 16];
            read_row<NP>(s.k[i], ln, k);
            if (!STATES) read_row<NP>(s.q[i], ln, q);
            const float a = s.a[i], beta = s.beta[i];
            float v[R], out[R];
            read_rows<R>(&s.v[i][lrow], v);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float u = beta * fmaf(-a, sum8(dot_row<NP>(S[r], k)), v[r]);
                out[r] = STATES ? u : p.scale * fmaf(a, sum8(dot_row<NP>(S[r], q)), u * s.kq[i]);
#pragma unroll
                for (int m = 0; m < NP / 16; ++m) S[r][m] = __ffma2_rn(dup(u), k[m], __fmul2_rn(dup(a), S[r][m]));
            }
            if (ln == 0) write_rows<R>(&s.out[i][lrow], out);
        }
        __syncthreads();
        for (int e = tid; e < nt * (kRows / 4); e += kThreads) {
            const int t = t0 + e / (kRows / 4), c = (e % (kRows / 4)) * 4;
            if (p0 + c >= p.P) continue;
            const float4 f4 = *reinterpret_cast<const float4 *>(&s.out[t - t0][c]);
            const float f[4] = {f4.x, f4.y, f4.z, f4.w};
            if (STATES) store4_io<IO_F32, VEC>(p.u, ((long long)bh * p.nc * kDeltaChunk + t) * p.P + p0 + c, min(4, p.P - p0 - c), f);
            else store4_io<IO, VEC>(p.y, (((long long)b * p.L + t) * p.H + h) * p.P + p0 + c, min(4, p.P - p0 - c), f);
        }
    }
    if (STATES) return;
    if (p.final_state) store_state<NP, R, VEC>(p.final_state + bh * pn, p.P, p.N, row0, ln, S);
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    for (long long e = tid; e < (long long)(p.L - len) * (kRows / 4); e += kThreads) {
        const long long t = len + e / (kRows / 4);
        const int c = p0 + (e % (kRows / 4)) * 4;
        if (c < p.P) store4_io<IO, VEC>(p.y, ((b * (long long)p.L + t) * p.H + h) * p.P + c, min(4, p.P - c), zero);
    }
}

template <int IO, int NP, int R, bool VEC>
__device__ __forceinline__ void adjoint_rows(const DeltaParams &p, int block, Tile<NP, R> &s) {
    constexpr int kRows = 16 * R;
    const int tiles = (p.P + kRows - 1) / kRows, p0 = (block % tiles) * kRows;
    const int bh = block / tiles, h = bh % p.H, b = bh / p.H;
    const int tid = threadIdx.x, lane = tid & 31, ln = lane & 7, lrow = (tid >> 5) * 4 * R + (lane >> 3) * R, row0 = p0 + lrow;
    const int len = delta_length(p, b);
    const size_t pn = (size_t)p.P * p.N;
    const long long dys[2] = {(long long)p.L * p.H * p.P, (long long)p.H * p.P};
    float2 D[R][NP / 16];
    load_state<NP, R, VEC>(p.dfinal ? p.dfinal + bh * pn : nullptr, p.P, p.N, row0, ln, D);
    Staged<NP, R> next;
    const int last = len > 0 ? (len - 1) / kTile * kTile : -kTile;
    if (len > 0) load_tile<IO, NP, R, VEC>(p, p.dy, dys, b, h, p0, last, len, next);
    for (int t0 = last; t0 >= 0; t0 -= kTile) {
        __syncthreads();
        put_tile<IO, NP, R, VEC>(next, s);
        if (t0 > 0) load_tile<IO, NP, R, VEC>(p, p.dy, dys, b, h, p0, t0 - kTile, len, next);
        __syncthreads();
        dot_tile<NP, R>(s);
        __syncthreads();
        const int nt = min(kTile, len - t0);
        if ((t0 + kTile) % kDeltaChunk == 0 || t0 + nt == len)
            store_state<NP, R, VEC>(p.adj + ((size_t)bh * p.nc + t0 / kDeltaChunk) * pn, p.P, p.N, row0, ln, D);
#pragma unroll (R == 1 ? 4 : 1)
        for (int i = kTile - 1; i >= 0; --i) {
            float2 k[NP / 16], q[NP / 16];
            read_row<NP>(s.k[i], ln, k);
            read_row<NP>(s.q[i], ln, q);
            const float a = s.a[i], beta = s.beta[i], kq = s.kq[i];
            float d[R], out[R], dv[R];
            read_rows<R>(&s.v[i][lrow], d);
#pragma unroll
            for (int r = 0; r < R; ++r) d[r] *= p.scale;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                out[r] = fmaf(d[r], kq, sum8(dot_row<NP>(D[r], k)));
                const float2 wq = dup(a * d[r]), wk = dup(-a * beta * out[r]);
#pragma unroll
                for (int m = 0; m < NP / 16; ++m) D[r][m] = __ffma2_rn(wk, k[m], __ffma2_rn(wq, q[m], __fmul2_rn(dup(a), D[r][m])));
            }
#pragma unroll
            for (int r = 0; r < R; ++r) dv[r] = beta * out[r];
            if (ln == 0) {
                write_rows<R>(&s.out[i][lrow], out);
                write_rows<R>(&s.dv[i][lrow], dv);
            }
        }
        __syncthreads();
        for (int e = tid; e < nt * (kRows / 4); e += kThreads) {
            const int t = t0 + e / (kRows / 4), c = (e % (kRows / 4)) * 4, nv = min(4, p.P - p0 - c);
            if (nv <= 0) continue;
            const float4 r4 = *reinterpret_cast<const float4 *>(&s.out[t - t0][c]), v4 = *reinterpret_cast<const float4 *>(&s.dv[t - t0][c]);
            const float r[4] = {r4.x, r4.y, r4.z, r4.w}, v[4] = {v4.x, v4.y, v4.z, v4.w};
            store4_io<IO_F32, VEC>(p.dr, ((long long)bh * p.nc * kDeltaChunk + t) * p.P + p0 + c, nv, r);
            store4_io<IO, VEC>(p.dv, (((long long)b * p.L + t) * p.H + h) * p.P + p0 + c, nv, v);
        }
    }
    if (p.dh0) store_state<NP, R, VEC>(p.dh0 + bh * pn, p.P, p.N, row0, ln, D);
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    for (long long e = tid; e < (long long)(p.L - len) * (kRows / 4); e += kThreads) {
        const long long t = len + e / (kRows / 4);
        const int c = p0 + (e % (kRows / 4)) * 4;
        if (c < p.P) store4_io<IO, VEC>(p.dv, ((b * (long long)p.L + t) * p.H + h) * p.P + c, min(4, p.P - c), zero);
    }
}

template <int IO, int NP, int R, bool VEC>
__global__ void __launch_bounds__(kThreads)
delta_walk_kernel(const __grid_constant__ DeltaParams p) {
    __shared__ __align__(16) Tile<NP, R> s;
    walk_rows<IO, NP, R, VEC, false>(p, blockIdx.x, s);
}

// The gradients' two walks in one launch: they need nothing of one another, and few heads leave SMs for both.
template <int IO, int NP, int R, bool VEC>
__global__ void __launch_bounds__(kThreads)
delta_both_kernel(const __grid_constant__ DeltaParams p) {
    __shared__ __align__(16) Tile<NP, R> s;
    const int half = gridDim.x / 2;
    if ((int)blockIdx.x < half) adjoint_rows<IO, NP, R, VEC>(p, blockIdx.x, s);  // the longer ones first
    else walk_rows<IO, NP, R, VEC, true>(p, blockIdx.x - half, s);
}

// ---- one token of each of B sequences

// The same layout, R rows to a lane.  Bound by the state's bytes, read and written once: 256 sequences of 32 heads of 128 x 128
// 157 us, 6.9 TB/s (101 % of a plain copy's rate); one sequence of 16 heads 5.6 us, the launch.
template <int IO, int NP, int R, bool VEC>
__global__ void __launch_bounds__(kThreads)
delta_step_kernel(const __grid_constant__ DeltaStepParams p) {
    constexpr int kCtaRows = 16 * R;
    const int tiles = (p.P + kCtaRows - 1) / kCtaRows;
    const int bh = blockIdx.x / tiles, h = bh % p.H, b = bh / p.H;
    const int lane = threadIdx.x & 31, ln = lane & 7;
    const int row0 = (blockIdx.x % tiles) * kCtaRows + ((threadIdx.x >> 5) * 4 + (lane >> 3)) * R;
    const long long slot = p.slots ? __ldg(p.slots + b) : b;
    const bool live = slot >= 0 && slot < p.nslots;
    const long long at = (slot * p.H + h) * p.P * p.N, gn = (long long)(h / (p.H / p.G)) * p.N;
    Raw4 rs[R][NP / 32], rk[NP / 32], rq[NP / 32];
#pragma unroll
    for (int j = 0; j < NP / 32; ++j) {
        const int n = 32 * j + 4 * ln;
#pragma unroll
        for (int r = 0; r < R; ++r)
            rs[r][j] = load_raw4<IO_F32, VEC, false>(p.state, at + (long long)(row0 + r) * p.N + n, live && row0 + r < p.P && n < p.N, p.N - n);
        rk[j] = load_raw4<IO, VEC>(p.k, b * p.k_row + gn + n, n < p.N, p.N - n);
        rq[j] = load_raw4<IO, VEC>(p.q, b * p.q_row + gn + n, n < p.N, p.N - n);
    }
    float v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = load_one<IO>(p.v, b * p.v_row + (long long)h * p.P + row0 + r, row0 + r < p.P);
    const float a = expf(load_gate<IO>(p.g, b * p.g_row + h, p.g32, true)), beta = load_gate<IO>(p.beta, b * p.b_row + h, p.b32, true);
    float2 k[NP / 16], q[NP / 16], kq = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NP / 32; ++j) {
        float f[4];
        unpack4<IO, VEC>(rk[j], f);
        k[2 * j] = make_float2(f[0], f[1]), k[2 * j + 1] = make_float2(f[2], f[3]);
        unpack4<IO, VEC>(rq[j], f);
        q[2 * j] = make_float2(f[0], f[1]), q[2 * j + 1] = make_float2(f[2], f[3]);
        kq = __ffma2_rn(k[2 * j], q[2 * j], __ffma2_rn(k[2 * j + 1], q[2 * j + 1], kq));
    }
    const float dot = sum8(kq);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float2 S[NP / 16], sk = make_float2(0.f, 0.f), sq = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < NP / 32; ++j) {
            float f[4];
            unpack4<IO_F32, VEC>(rs[r][j], f);
            S[2 * j] = make_float2(f[0], f[1]), S[2 * j + 1] = make_float2(f[2], f[3]);
        }
#pragma unroll
        for (int m = 0; m < NP / 16; ++m) {
            sk = __ffma2_rn(S[m], k[m], sk);
            sq = __ffma2_rn(S[m], q[m], sq);
        }
        const float u = beta * fmaf(-a, sum8(sk), v[r]), y = p.scale * fmaf(a, sum8(sq), u * dot);
        if (row0 + r >= p.P) continue;
        if (ln == 0) st_io<IO>(p.y, ((size_t)b * p.H + h) * p.P + row0 + r, live ? y : 0.f);
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < NP / 32; ++j) {
            const int n = 32 * j + 4 * ln;
            const float2 x = __ffma2_rn(dup(a), S[2 * j], __fmul2_rn(dup(u), k[2 * j])),
                         z = __ffma2_rn(dup(a), S[2 * j + 1], __fmul2_rn(dup(u), k[2 * j + 1]));
            const float f[4] = {x.x, x.y, z.x, z.y};
            if (n < p.N) store4_io<IO_F32, VEC>(p.state_out, at + (long long)(row0 + r) * p.N + n, min(4, p.N - n), f);
        }
    }
}

// Whether a tensor's rows can be read by fours.
bool by_fours(const void *p, int io, long long s0, long long s1, int n) {
    return vec4_aligned(p, io) && s0 % 4 == 0 && s1 % 4 == 0 && n % 4 == 0;
}

template <int IO, int NP, int R, bool VEC>
cudaError_t launch_rows(const DeltaParams &p, bool both, cudaStream_t s) {
    const unsigned grid = (unsigned)(p.B * (long long)p.H * ((p.P + 16 * R - 1) / (16 * R)));
    if (both) delta_both_kernel<IO, NP, R, VEC><<<2 * grid, kThreads, 0, s>>>(p);
    else delta_walk_kernel<IO, NP, R, VEC><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <int IO, int NP, bool VEC>
cudaError_t walk_as(const DeltaParams &p, bool both, cudaStream_t s) {
    // A row to a lane until CTAs of 16 rows would give an SM more than four: above, the walks wait for issue slots, of which
    // four rows to a lane need fewer.
    const bool wide = p.B * (long long)p.H * ((p.P + 15) / 16) > 4LL * scan_sm_count();
    return wide ? launch_rows<IO, NP, 4, VEC>(p, both, s) : launch_rows<IO, NP, 1, VEC>(p, both, s);
}

template <int IO>
cudaError_t walk_io(const DeltaParams &p, bool both, cudaStream_t s) {
    const bool vec = by_fours(p.k, IO, p.ks[0], p.ks[1], p.N) && by_fours(p.q, IO, p.qs[0], p.qs[1], p.N) &&
                     by_fours(p.v, IO, p.vs[0], p.vs[1], p.P) && by_fours(p.h0, IO_F32, 0, 0, 4) && by_fours(p.y, IO, 0, 0, 4) &&
                     by_fours(p.final_state, IO_F32, 0, 0, 4) && by_fours(p.dy, IO, 0, 0, 4) && by_fours(p.dfinal, IO_F32, 0, 0, 4) &&
                     by_fours(p.dv, IO, 0, 0, 4) && by_fours(p.dh0, IO_F32, 0, 0, 4);
    if (p.N <= 64) return vec ? walk_as<IO, 64, true>(p, both, s) : walk_as<IO, 64, false>(p, both, s);
    return vec ? walk_as<IO, 128, true>(p, both, s) : walk_as<IO, 128, false>(p, both, s);
}

cudaError_t walk(const DeltaParams &p, int io, bool both, cudaStream_t s) {
    switch (io) {
        case IO_F32: return walk_io<IO_F32>(p, both, s);
        case IO_F16: return walk_io<IO_F16>(p, both, s);
        case IO_BF16: return walk_io<IO_BF16>(p, both, s);
        default: return cudaErrorInvalidValue;
    }
}

template <int IO, int NP, int R>
cudaError_t step_as(const DeltaStepParams &p, bool vec, cudaStream_t s) {
    const unsigned grid = (unsigned)(p.B * (long long)p.H * ((p.P + 16 * R - 1) / (16 * R)));
    if (vec) delta_step_kernel<IO, NP, R, true><<<grid, kThreads, 0, s>>>(p);
    else delta_step_kernel<IO, NP, R, false><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <int IO>
cudaError_t step_io(const DeltaStepParams &p, cudaStream_t s) {
    const bool vec = by_fours(p.k, IO, 0, p.k_row, p.N) && by_fours(p.q, IO, 0, p.q_row, p.N) && by_fours(p.state, IO_F32, 0, 0, 4) &&
                     by_fours(p.state_out, IO_F32, 0, 0, 4);
    // One row to a lane until the CTAs of 64 rows would give every SM four.
    const bool wide = (long long)p.B * p.H * ((p.P + 63) / 64) >= 4LL * scan_sm_count();
    if (p.N <= 64) return wide ? step_as<IO, 64, 4>(p, vec, s) : step_as<IO, 64, 1>(p, vec, s);
    return wide ? step_as<IO, 128, 4>(p, vec, s) : step_as<IO, 128, 1>(p, vec, s);
}

}  // namespace

cudaError_t launch_delta_walk(const DeltaParams &p, int io, cudaStream_t s) { return walk(p, io, false, s); }
cudaError_t launch_delta_walks(const DeltaParams &p, int io, cudaStream_t s) { return walk(p, io, true, s); }

cudaError_t launch_delta_step(const DeltaStepParams &p, int io, cudaStream_t s) {
    switch (io) {
        case IO_F32: return step_io<IO_F32>(p, s);
        case IO_F16: return step_io<IO_F16>(p, s);
        case IO_BF16: return step_io<IO_BF16>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace ssd

// conv_carry.cu -- the short causal convolution in front of the selective
// scan, over token-major prompts with a carried state, and its backward:
//
//   pre_t[c] = bias[c] + sum_k w[c,k] v_{t-(W-1)+k}[c],   y = silu(pre)
//   dp = dy silu'(pre);  dx_t = sum_k w[k] dp_{t+(W-1)-k};  dw[k] = sum_t dp_t v_{t-(W-1)+k}
//
// v is x, and the carried rows before it.  2 W + 4 operations per element
// against 4 bytes of 16-bit traffic: bound by HBM.  A thread owns four channels
// over a run of tokens and slides the window in registers, so each token is
// read once but for the W-1 before its run; a warp's 32 threads cover 128
// consecutive channels of a token.  Tokens are copied into the thread's own ring in
// shared memory, two blocks of eight ahead, so the loads run on beside the arithmetic
// and need neither registers nor a barrier.
// Measured in bf16 (the copy rate of the card is 6.8 TB/s): [2,8192,8192] with a carried
// state 86 us, 6.2 TB/s; backwards [4,2048,4096] 57 us, 3.5 TB/s: it reads x and dy once,
// but recomputes pre and its sigmoid and runs 128 registers a thread (8 to 12 bytes spilled), so of 16 warps per
// SM 12.3 are active on average and issue in 43 % of the cycles.  Rows that are not whole quads of four (8191 channels) go element by
// element: 160 us.
#include <math.h>

#include "scan_common.cuh"

namespace ssd {

namespace {

constexpr int kCx = 32, kCy = 4;   // threads: channel quads, runs
constexpr int kAhead = 8;
constexpr int kRun = 32;  // tokens per thread (backwards: ConvParams::run)
constexpr int kHalo(int W) { return W <= 4 ? 3 : 7; }  // KT - 1

template <bool V>
struct Flag {
    static constexpr bool value = V;
};

// v at token t as loaded: x inside the row, the carried rows before it, zeros elsewhere.
template <int IO, bool VEC>
__device__ __forceinline__ Raw4 conv_value(const ConvParams &p, int b, long long t, int len, int c, int nv) {
    const bool carried = t < 0;
    const void *base = carried ? p.h0 : p.x;
    const long long i = carried ? ((long long)b * (p.W - 1) + t + p.W - 1) * p.C + c : b * p.xs[0] + t * p.xs[1] + c;
    return load_raw4<IO, VEC>(base, i, carried ? p.h0 && t >= -(long long)(p.W - 1) : t < len, nv);
}

// Four channels as two pairs: the packed operations take one issue slot for both.
template <int IO, bool VEC>
__device__ __forceinline__ void unpack_pairs(const Raw4 &r, float2 (&v)[2]) {
    float f[4];
    unpack4<IO, VEC>(r, f);
    v[0] = make_float2(f[0], f[1]);
    v[1] = make_float2(f[2], f[3]);
}
template <int IO, bool VEC>
__device__ __forceinline__ void store_pairs(char *dst, int nv, const float2 (&v)[2]) {
    const float f[4] = {v[0].x, v[0].y, v[1].x, v[1].y};
    store4_io<IO, VEC>(dst, 0, nv, f);
}

// Taps sit right-aligned in KT slots (slot KT-1 is the current token), so every index is a constant.
template <int KT>
__device__ __forceinline__ void load_taps(const ConvParams &p, int c, int nv, float2 (&w)[KT][2], float2 (&bias)[2]) {
    const bool rows4 = KT == 4 && p.W == 4 && (reinterpret_cast<uintptr_t>(p.w) & 15) == 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (rows4) {  // a channel's taps in one load
            const Raw4 r = load_raw4<IO_F32, true>(p.w, (long long)(c + j) * 4, j < nv, 4);
#pragma unroll
            for (int s = 0; s < KT; ++s) {
                if (j & 1) w[s][j / 2].y = __uint_as_float(r.w[s & 3]);
                else w[s][j / 2].x = __uint_as_float(r.w[s & 3]);
            }
        } else {
#pragma unroll
            for (int s = 0; s < KT; ++s) {
                const int k = s - (KT - p.W);
                const float v = k >= 0 && j < nv ? __ldg(p.w + (long long)(c + j) * p.W + k) : 0.f;
                if (j & 1) w[s][j / 2].y = v;
                else w[s][j / 2].x = v;
            }
        }
        const float v = p.bias && j < nv ? __ldg(p.bias + c + j) : 0.f;
        if (j & 1) bias[j / 2].y = v;
        else bias[j / 2].x = v;
    }
}

template <int IO, int KT, bool VEC, bool SILU>
__global__ void __launch_bounds__(kCx * kCy, KT == 4 ? 8 : 1)
conv_carry_kernel(ConvParams p) {
    constexpr int kQ = IO == IO_F32 ? 16 : 8;  // bytes of four elements
    __shared__ __align__(16) char ring[2 * kAhead][kCx * kCy * kQ];
    const int c = (blockIdx.x * kCx + threadIdx.x) * 4;
    if (c >= p.C) return;
    const int nv = min(4, p.C - c), b = blockIdx.z;
    const int len = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.L) : p.L;
    if (blockIdx.y == gridDim.y - 1) {  // the last W-1 entries of v
        if (!p.final_state) return;
        for (int j = threadIdx.y; j < p.W - 1; j += kCy) {
            float v[4];
            unpack4<IO, VEC>(conv_value<IO, VEC>(p, b, (long long)len + j - (p.W - 1), len, c, nv), v);
            store4_io<IO, VEC>(p.final_state, ((long long)b * (p.W - 1) + j) * p.C + c, nv, v);
        }
        return;
    }
    constexpr int kEs = IO == IO_F32 ? 4 : 2;
    const int t0 = (blockIdx.y * kCy + threadIdx.y) * kRun, t1 = min(t0 + kRun, p.L);
    if (t0 >= t1) return;
    float2 w[KT][2], bias[2], win[KT][2];
    const char *px = static_cast<const char *>(p.x) + (b * p.xs[0] + t0 * p.xs[1] + c) * kEs;
    char *py = static_cast<char *>(p.y) + (((long long)b * p.L + t0) * p.C + c) * kEs;
    const long long sx = p.xs[1] * kEs, sy = (long long)p.C * kEs;
    const int live = min(t1, len);
    const int me = (threadIdx.y * kCx + threadIdx.x) * kQ;
    auto copy = [&](int t) {  // tokens t .. t + kAhead - 1
        const int slot = (t - t0) & kAhead;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            copy_quad<IO, VEC>(ring[slot + i] + me, px, t + i < live ? nv : 0);
            px += sx;
        }
        cp_commit();
    };
    copy(t0);
    copy(t0 + kAhead);
    load_taps<KT>(p, c, nv, w, bias);
#pragma unroll
    for (int s = 1; s < KT; ++s)  // slots 0..KT-2 of the first step are tokens t0-KT+1 .. t0-1
        unpack_pairs<IO, VEC>(conv_value<IO, VEC>(p, b, (long long)t0 - KT + s, len, c, nv), win[s]);
    // A block of kAhead tokens; EDGE: some of them are past the run's or the row's end.
    auto block = [&](int t, auto edge) {
        constexpr bool EDGE = decltype(edge)::value;
        const int slot = (t - t0) & kAhead;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
#pragma unroll
            for (int s = 0; s < KT - 1; ++s) win[s][0] = win[s + 1][0], win[s][1] = win[s + 1][1];
            read_quad<IO>(ring[slot + i] + me, win[KT - 1]);
            float2 o[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float2 a = bias[j];
#pragma unroll
                for (int s = 0; s < KT; ++s) a = __ffma2_rn(w[s][j], win[s][j], a);
                o[j] = SILU ? silu2(a) : a;
                if (EDGE && t + i >= live) o[j] = dup(0.f);
            }
            if (!EDGE || t + i < t1) store_pairs<IO, VEC>(py, nv, o);
            py += sy;
        }
    };
    for (int t = t0; t < t1; t += kAhead) {
        cp_wait<1>();
        if (t + kAhead <= live) block(t, Flag<false>{});
        else block(t, Flag<true>{});
        copy(t + 2 * kAhead);
    }
}

// A thread walks its run and the KT-1 tokens after it (dp of the first W-1
// reaches back into the run), recomputing pre from the window.  dw and dbias gather in
// registers over the run, then over the CTA's runs in shared memory in a fixed
// order, and leave as one row of partial sums per CTA.
template <int IO, int KT, bool VEC, bool SILU>
__global__ void __launch_bounds__(kCx * kCy, KT == 4 ? 4 : 1)
conv_bwd_kernel(ConvParams p) {
    tc::pdl_launch_dependents();
    constexpr int kQ = IO == IO_F32 ? 16 : 8;
    __shared__ __align__(16) float red[kCy][kCx * 4];
    extern __shared__ __align__(16) char ring[];  // [2 kAhead][2][kCx kCy] of four elements: x, dy
    const int c = (blockIdx.x * kCx + threadIdx.x) * 4;
    const int nv = min(4, p.C - c), b = blockIdx.z;
    const int len = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.L) : p.L;
    const int t0 = (blockIdx.y * kCy + threadIdx.y) * p.run, t1 = min(t0 + p.run, p.L);
    constexpr int kEs = IO == IO_F32 ? 4 : 2;
    float2 dw[KT][2], db[2] = {dup(0.f), dup(0.f)};
#pragma unroll
    for (int s = 0; s < KT; ++s) dw[s][0] = dw[s][1] = dup(0.f);
    if (c < p.C && t0 < t1) {
        float2 w[KT][2], bias[2], win[KT][2], dp[KT][2];  // dp[i]: of token t - i
#pragma unroll
        for (int s = 0; s < KT; ++s) dp[s][0] = dp[s][1] = dup(0.f);
        const char *px = static_cast<const char *>(p.x) + (b * p.xs[0] + t0 * p.xs[1] + c) * kEs;
        const long long o0 = ((long long)b * p.L + t0) * p.C + c;
        const char *pdy = static_cast<const char *>(p.dy) + o0 * kEs;
        char *pdx = static_cast<char *>(p.dx) + (o0 - (long long)(KT - 1) * p.C) * kEs;
        const long long sx = p.xs[1] * kEs, sy = (long long)p.C * kEs;
        const int tend = t1 + KT - 1, live = min(tend, len);
        constexpr int kLine = kCx * kCy * kQ;
        char *mine_ring = ring + (threadIdx.y * kCx + threadIdx.x) * kQ;
        auto copy = [&](int t) {  // tokens t .. t + kAhead - 1
            char *slot = mine_ring + ((t - t0) & kAhead) * 2 * kLine;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int n = t + i < live ? nv : 0;
                copy_quad<IO, VEC>(slot + 2 * i * kLine, px, n);
                copy_quad<IO, VEC>(slot + (2 * i + 1) * kLine, pdy, n);
                px += sx;
                pdy += sy;
            }
            cp_commit();
        };
        copy(t0);
        copy(t0 + kAhead);
        load_taps<KT>(p, c, nv, w, bias);
#pragma unroll
        for (int s = 1; s < KT; ++s)
            unpack_pairs<IO, VEC>(conv_value<IO, VEC>(p, b, (long long)t0 - KT + s, len, c, nv), win[s]);
        // A block of kAhead tokens; EDGE: some are past the run or the row, or complete entries of v outside them.
        auto block = [&](int t, auto edge) {
            constexpr bool EDGE = decltype(edge)::value;
            const char *slot = mine_ring + ((t - t0) & kAhead) * 2 * kLine;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int tt = t + i;
#pragma unroll
                for (int s = 0; s < KT - 1; ++s) win[s][0] = win[s + 1][0], win[s][1] = win[s + 1][1];
#pragma unroll
                for (int s = KT - 1; s > 0; --s) dp[s][0] = dp[s - 1][0], dp[s][1] = dp[s - 1][1];
                read_quad<IO>(slot + 2 * i * kLine, win[KT - 1]);
                float2 g[2], o[2];
                read_quad<IO>(slot + (2 * i + 1) * kLine, g);  // zeros past the row's tokens
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (SILU) {  // g silu'(a) = g s (1 + a (1 - s)), s = sigmoid(a)
                        float2 a = bias[j];
#pragma unroll
                        for (int s = 0; s < KT; ++s) a = __ffma2_rn(w[s][j], win[s][j], a);
                        const float2 sg = sigmoid2(a);
                        const float2 slope = __ffma2_rn(__fmul2_rn(a, sg), __ffma2_rn(sg, dup(-1.f), dup(1.f)), sg);
                        g[j] = __fmul2_rn(g[j], slope);
                        if (EDGE && tt >= live) g[j] = dup(0.f);
                    }
                    dp[0][j] = g[j];
                    const float2 mine = !EDGE || tt < t1 ? g[j] : dup(0.f);
                    db[j] = __fadd2_rn(db[j], mine);
#pragma unroll
                    for (int s = 0; s < KT; ++s) dw[s][j] = __ffma2_rn(mine, win[s][j], dw[s][j]);
                    float2 a = __fmul2_rn(w[0][j], dp[0][j]);  // the slot of tap k is its age past KT - W empty ones
#pragma unroll
                    for (int s = 1; s < KT; ++s) a = __ffma2_rn(w[s][j], dp[s][j], a);
                    o[j] = a;
                }
                const int tau = tt - (KT - 1);  // the entry of v this step completes
                if (!EDGE) {
                    store_pairs<IO, VEC>(pdx, nv, o);
                } else {
                    if (p.dfinal && tt < tend && tau >= len - (p.W - 1) && tau < len) {
                        float2 f[2];
                        unpack_pairs<IO, VEC>(load_raw4<IO, VEC>(p.dfinal, ((long long)b * (p.W - 1) + tau + p.W - 1 - len) * p.C + c, 1, nv), f);
                        o[0] = __fadd2_rn(o[0], f[0]);
                        o[1] = __fadd2_rn(o[1], f[1]);
                    }
                    if (tau < 0) {
                        if (t0 == 0 && p.dh0 && tau >= -(p.W - 1))
                            store_pairs<IO, VEC>(static_cast<char *>(p.dh0) + (((long long)b * (p.W - 1) + tau + p.W - 1) * p.C + c) * kEs, nv, o);
                    } else if (tau >= t0 && tau < t1) {
                        if (tau >= len) o[0] = o[1] = dup(0.f);
                        store_pairs<IO, VEC>(pdx, nv, o);
                    }
                }
                pdx += sy;
            }
        };
        for (int t = t0; t < tend; t += kAhead) {
            cp_wait<1>();
            if (t >= t0 + KT - 1 && t + kAhead <= min(t1, live) && t + kAhead - KT < len - (p.W - 1)) block(t, Flag<false>{});
            else block(t, Flag<true>{});
            copy(t + 2 * kAhead);
        }
    }
    const long long row = (long long)b * gridDim.y + blockIdx.y;
    const int cc = blockIdx.x * kCx * 4 + threadIdx.y * kCx + threadIdx.x;  // one channel per thread in the sums
#pragma unroll
    for (int s = 0; s <= KT; ++s) {
        const int k = s == KT ? p.W : s - (KT - p.W);  // dbias follows the taps
        if (k < 0) continue;
        const float2 *v = s == KT ? db : dw[s < KT ? s : 0];
        __syncthreads();
        *reinterpret_cast<float2 *>(&red[threadIdx.y][threadIdx.x * 4]) = v[0];
        *reinterpret_cast<float2 *>(&red[threadIdx.y][threadIdx.x * 4 + 2]) = v[1];
        __syncthreads();
        if (cc < p.C) {
            float a = 0.f;
#pragma unroll
            for (int y = 0; y < kCy; ++y) a += red[y][threadIdx.y * kCx + threadIdx.x];
            p.part[(row * (p.W + 1) + k) * p.C + cc] = a;
        }
    }
}

// dw[c,k] and dbias[c]: the partial rows summed in order, eight interleaved sums first.
__global__ void __launch_bounds__(256)
conv_bwd_sum_kernel(ConvParams p, int rows) {
    __shared__ float red[8][32];
    tc::pdl_wait();
    const int c = blockIdx.x * 32 + threadIdx.x, k = blockIdx.y;
    float a = 0.f;
    if (c < p.C) {
        const float *src = p.part + (long long)k * p.C + c;
        const long long step = (long long)(p.W + 1) * p.C;
        for (int r = threadIdx.y; r < rows; r += 32) {  // four rows' loads together
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = r + 8 * j < rows ? src[(r + 8 * j) * step] : 0.f;
            a += (v[0] + v[1]) + (v[2] + v[3]);
        }
    }
    red[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y != 0 || c >= p.C) return;
    for (int y = 1; y < 8; ++y) a += red[y][threadIdx.x];
    if (k < p.W) p.dw[(long long)c * p.W + k] = a;
    else if (p.dbias) p.dbias[c] = a;
}

// Whether every tensor moves in aligned groups of four channels (absent ones do).
bool conv_vec(const ConvParams &p, int io) {
    bool ok = p.C % 4 == 0 && vec4_strided(p.x, io, p.xs);
    for (const void *q : {p.h0, (const void *)p.y, (const void *)p.final_state, p.dy, p.dfinal, (const void *)p.dx,
                          (const void *)p.dh0})
        ok = ok && vec4_aligned(q, io);
    return ok;
}

template <int IO>
cudaError_t launch_conv_io(const ConvParams &p, cudaStream_t s) {
    const dim3 grid((p.C + 4 * kCx - 1) / (4 * kCx), (p.L + kCy * kRun - 1) / (kCy * kRun) + 1, p.B);
    static constexpr decltype(&conv_carry_kernel<IO, 4, true, true>) kernels[2][2][2] = {
        {{conv_carry_kernel<IO, 4, false, false>, conv_carry_kernel<IO, 4, false, true>},
         {conv_carry_kernel<IO, 4, true, false>, conv_carry_kernel<IO, 4, true, true>}},
        {{conv_carry_kernel<IO, 8, false, false>, conv_carry_kernel<IO, 8, false, true>},
         {conv_carry_kernel<IO, 8, true, false>, conv_carry_kernel<IO, 8, true, true>}}};
    auto *kernel = kernels[p.W > 4][conv_vec(p, IO)][p.silu != 0];
    kernel<<<grid, dim3(kCx, kCy), 0, s>>>(p);
    return cudaGetLastError();
}

template <int IO>
cudaError_t launch_conv_bwd_io(const ConvParams &p, cudaStream_t s) {
    const int rows = (int)(conv_bwd_part_rows(p) / p.B);
    const dim3 grid((p.C + 4 * kCx - 1) / (4 * kCx), rows, p.B);
    static constexpr decltype(&conv_bwd_kernel<IO, 4, true, true>) kernels[2][2][2] = {
        {{conv_bwd_kernel<IO, 4, false, false>, conv_bwd_kernel<IO, 4, false, true>},
         {conv_bwd_kernel<IO, 4, true, false>, conv_bwd_kernel<IO, 4, true, true>}},
        {{conv_bwd_kernel<IO, 8, false, false>, conv_bwd_kernel<IO, 8, false, true>},
         {conv_bwd_kernel<IO, 8, true, false>, conv_bwd_kernel<IO, 8, true, true>}}};
    auto *kernel = kernels[p.W > 4][conv_vec(p, IO)][p.silu != 0];
    constexpr int kBytes = 2 * kAhead * 2 * kCx * kCy * (IO == IO_F32 ? 16 : 8);
    cudaError_t e = allow_smem<kBytes>(kernel);
    if (e != cudaSuccess) return e;
    kernel<<<grid, dim3(kCx, kCy), kBytes, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_kernel(true, conv_bwd_sum_kernel, dim3((p.C + 31) / 32, p.W + 1), dim3(32, 8), 0, s, p, rows * p.B);
}

}  // namespace

// The run of a thread backwards: whole blocks of kAhead with the KT-1 tokens after
// it, as many as make the CTAs' waves (four CTAs per SM) cheapest; a CTA's start
// (taps, window) and end (sums) cost about two blocks.  The last CTAs, with the tokens a
// row has left, count in part where a wave has no others.  [4,2048,4096] in bf16 with runs
// of 2, 4, 8, 16, 17 and 20 blocks: 83, 68, 62, 58, 60 and 66 us; the rule takes 17 there.
int conv_bwd_run(const ConvParams &p) {
    const double slots = 4. * scan_sm_count();
    int best = 0;
    double least = 0.;
    for (int m = 2; m <= 24; ++m) {
        const int run = kAhead * m - kHalo(p.W);
        const long long x = (p.C + 4 * kCx - 1) / (4 * kCx), rows = (p.L + kCy * run - 1) / (kCy * run);
        const double ctas = (double)x * rows * p.B, waves = ceil(ctas / slots);
        const double part = ctas - (waves - 1) * slots <= x ? (double)p.L / (kCy * run) - (rows - 1) : 1.;
        const double cost = (waves - 1) * (m + 2) + part * m + 2;
        if (best == 0 || cost < least) best = run, least = cost;
    }
    return best;
}

long long conv_bwd_part_rows(const ConvParams &p) {
    const int tokens = kCy * p.run;
    return (long long)p.B * ((p.L + tokens - 1) / tokens);
}

cudaError_t launch_conv(const ConvParams &p, int io, cudaStream_t s) {
    switch (io) {
        case IO_F32: return launch_conv_io<IO_F32>(p, s);
        case IO_F16: return launch_conv_io<IO_F16>(p, s);
        case IO_BF16: return launch_conv_io<IO_BF16>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_conv_bwd(const ConvParams &p, int io, cudaStream_t s) {
    switch (io) {
        case IO_F32: return launch_conv_bwd_io<IO_F32>(p, s);
        case IO_F16: return launch_conv_bwd_io<IO_F16>(p, s);
        case IO_BF16: return launch_conv_bwd_io<IO_BF16>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace ssd

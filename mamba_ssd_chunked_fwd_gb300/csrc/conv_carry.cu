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
// consecutive channels of a token.  Eight tokens' loads go out together.
#include "scan_common.cuh"

namespace ssd {

namespace {

constexpr int kCx = 32, kCy = 4;   // threads: channel quads, runs
constexpr int kRun = 32;           // tokens per thread
constexpr int kCtaTokens = kCy * kRun;
constexpr int kAhead = 8;

// v at token t as loaded: x inside the row, the carried rows before it, zeros elsewhere.
template <int IO, bool VEC>
__device__ __forceinline__ Raw4 conv_value(const ConvParams &p, int b, long long t, int len, int c, int nv) {
    const bool carried = t < 0;
    const void *base = carried ? p.h0 : p.x;
    const long long i = carried ? ((long long)b * (p.W - 1) + t + p.W - 1) * p.C + c : b * p.xs[0] + t * p.xs[1] + c;
    return load_raw4<IO, VEC>(base, i, carried ? p.h0 && t >= -(long long)(p.W - 1) : t < len, nv);
}

// Taps sit right-aligned in KT slots (slot KT-1 is the current token), so every index is a constant.
template <int KT>
__device__ __forceinline__ void load_taps(const ConvParams &p, int c, int nv, float (&w)[KT][4], float (&bias)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int s = 0; s < KT; ++s) {
            const int k = s - (KT - p.W);
            w[s][j] = k >= 0 && j < nv ? __ldg(p.w + (long long)(c + j) * p.W + k) : 0.f;
        }
        bias[j] = p.bias && j < nv ? __ldg(p.bias + c + j) : 0.f;
    }
}

template <int IO, int KT, bool VEC>
__global__ void __launch_bounds__(kCx * kCy)
conv_carry_kernel(ConvParams p) {
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
    const int t0 = blockIdx.y * kCtaTokens + threadIdx.y * kRun, t1 = min(t0 + kRun, p.L);
    if (t0 >= t1) return;
    float w[KT][4], bias[4], win[KT][4];
    load_taps<KT>(p, c, nv, w, bias);
#pragma unroll
    for (int s = 1; s < KT; ++s)  // slots 0..KT-2 of the first step are tokens t0-KT+1 .. t0-1
        unpack4<IO, VEC>(conv_value<IO, VEC>(p, b, (long long)t0 - KT + s, len, c, nv), win[s]);
    for (int t = t0; t < t1; t += kAhead) {
        Raw4 r[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            r[i] = load_raw4<IO, VEC>(p.x, b * p.xs[0] + (t + i) * p.xs[1] + c, t + i < min(t1, len), nv);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (t + i >= t1) break;
            float o[4];
#pragma unroll
            for (int s = 0; s < KT - 1; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) win[s][j] = win[s + 1][j];
            unpack4<IO, VEC>(r[i], win[KT - 1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float a = bias[j];
#pragma unroll
                for (int s = 0; s < KT; ++s) a = fmaf(w[s][j], win[s][j], a);
                if (p.silu) a = silu_fast(a);
                o[j] = t + i < len ? a : 0.f;
            }
            store4_io<IO, VEC>(p.y, ((long long)b * p.L + t + i) * p.C + c, nv, o);
        }
    }
}

// A thread walks its run and the KT-1 tokens after it (dp of the first W-1
// reaches back into the run), recomputing pre from the window.  dw and dbias gather in
// registers over the run, then over the CTA's runs in shared memory in a fixed
// order, and leave as one row of partial sums per CTA.
template <int IO, int KT, bool VEC>
__global__ void __launch_bounds__(kCx * kCy)
conv_bwd_kernel(ConvParams p) {
    __shared__ float red[kCy][kCx * 4];
    const int c = (blockIdx.x * kCx + threadIdx.x) * 4;
    const int nv = min(4, p.C - c), b = blockIdx.z;
    const int len = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.L) : p.L;
    const int t0 = blockIdx.y * kCtaTokens + threadIdx.y * kRun, t1 = min(t0 + kRun, p.L);
    float dw[KT][4], db[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KT; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[s][j] = 0.f;
    if (c < p.C && t0 < t1) {
        float w[KT][4], bias[4], win[KT][4], dp[KT][4];  // dp[i]: of token t - i
        load_taps<KT>(p, c, nv, w, bias);
#pragma unroll
        for (int s = 1; s < KT; ++s)
            unpack4<IO, VEC>(conv_value<IO, VEC>(p, b, (long long)t0 - KT + s, len, c, nv), win[s]);
#pragma unroll
        for (int s = 0; s < KT; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) dp[s][j] = 0.f;
        const int tend = t1 + KT - 1;
        for (int t = t0; t < tend; t += kAhead) {
            Raw4 r[kAhead], rg[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const bool ok = t + i < min(tend, len);
                r[i] = load_raw4<IO, VEC>(p.x, b * p.xs[0] + (t + i) * p.xs[1] + c, ok, nv);
                rg[i] = load_raw4<IO, VEC>(p.dy, ((long long)b * p.L + t + i) * p.C + c, ok, nv);
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int tt = t + i;
                if (tt >= tend) break;
#pragma unroll
                for (int s = 0; s < KT - 1; ++s)
#pragma unroll
                    for (int j = 0; j < 4; ++j) win[s][j] = win[s + 1][j];
#pragma unroll
                for (int s = KT - 1; s > 0; --s)
#pragma unroll
                    for (int j = 0; j < 4; ++j) dp[s][j] = dp[s - 1][j];
                unpack4<IO, VEC>(r[i], win[KT - 1]);
                float g[4], o[4];
                unpack4<IO, VEC>(rg[i], g);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (p.silu) {
                        float a = bias[j];
#pragma unroll
                        for (int s = 0; s < KT; ++s) a = fmaf(w[s][j], win[s][j], a);
                        const float sg = sigmoid_f(a);
                        g[j] = tt < len ? g[j] * sg * fmaf(a, 1.f - sg, 1.f) : 0.f;  // silu'(a)
                    }
                    dp[0][j] = g[j];
                    if (tt < t1) {
                        db[j] += g[j];
#pragma unroll
                        for (int s = 0; s < KT; ++s) dw[s][j] = fmaf(g[j], win[s][j], dw[s][j]);
                    }
                    float a = 0.f;  // the slot of tap k is its age past KT - W empty ones
#pragma unroll
                    for (int s = 0; s < KT; ++s) a = fmaf(w[s][j], dp[s][j], a);
                    o[j] = a;
                }
                const int tau = tt - (KT - 1);  // the entry of v this step completes
                if (tau >= len - (p.W - 1) && tau < len && p.dfinal) {
                    float f[4];
                    unpack4<IO, VEC>(load_raw4<IO, VEC>(p.dfinal, ((long long)b * (p.W - 1) + tau + p.W - 1 - len) * p.C + c, true, nv), f);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] += f[j];
                }
                if (tau < 0) {
                    if (t0 == 0 && p.dh0 && tau >= -(p.W - 1))
                        store4_io<IO, VEC>(p.dh0, ((long long)b * (p.W - 1) + tau + p.W - 1) * p.C + c, nv, o);
                } else if (tau >= t0) {
                    if (tau >= len) o[0] = o[1] = o[2] = o[3] = 0.f;
                    store4_io<IO, VEC>(p.dx, ((long long)b * p.L + tau) * p.C + c, nv, o);
                }
            }
        }
    }
    const long long row = (long long)b * gridDim.y + blockIdx.y;
    const int cc = blockIdx.x * kCx * 4 + threadIdx.y * kCx + threadIdx.x;  // one channel per thread in the sums
#pragma unroll
    for (int s = 0; s <= KT; ++s) {
        const int k = s == KT ? p.W : s - (KT - p.W);  // dbias follows the taps
        if (k < 0) continue;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) red[threadIdx.y][threadIdx.x * 4 + j] = s == KT ? db[j] : dw[s < KT ? s : 0][j];
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
    const int c = blockIdx.x * 32 + threadIdx.x, k = blockIdx.y;
    float a = 0.f;
    if (c < p.C)
        for (int r = threadIdx.y; r < rows; r += 8) a += p.part[((long long)r * (p.W + 1) + k) * p.C + c];
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
    const dim3 grid((p.C + 4 * kCx - 1) / (4 * kCx), (p.L + kCtaTokens - 1) / kCtaTokens + 1, p.B);
    auto *kernel = conv_vec(p, IO) ? (p.W <= 4 ? conv_carry_kernel<IO, 4, true> : conv_carry_kernel<IO, 8, true>)
                                   : (p.W <= 4 ? conv_carry_kernel<IO, 4, false> : conv_carry_kernel<IO, 8, false>);
    kernel<<<grid, dim3(kCx, kCy), 0, s>>>(p);
    return cudaGetLastError();
}

template <int IO>
cudaError_t launch_conv_bwd_io(const ConvParams &p, cudaStream_t s) {
    const dim3 grid((p.C + 4 * kCx - 1) / (4 * kCx), (p.L + kCtaTokens - 1) / kCtaTokens, p.B);
    auto *kernel = conv_vec(p, IO) ? (p.W <= 4 ? conv_bwd_kernel<IO, 4, true> : conv_bwd_kernel<IO, 8, true>)
                                   : (p.W <= 4 ? conv_bwd_kernel<IO, 4, false> : conv_bwd_kernel<IO, 8, false>);
    kernel<<<grid, dim3(kCx, kCy), 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    conv_bwd_sum_kernel<<<dim3((p.C + 31) / 32, p.W + 1), dim3(32, 8), 0, s>>>(p, (int)conv_bwd_part_rows(p.B, p.L, p.C));
    return cudaGetLastError();
}

}  // namespace

long long conv_bwd_part_rows(int B, int L, int C) {
    (void)C;
    return (long long)B * ((L + kCtaTokens - 1) / kCtaTokens);
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

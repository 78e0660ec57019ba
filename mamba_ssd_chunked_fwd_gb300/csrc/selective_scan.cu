// selective_scan.cu -- the selective scan over prompts: the recurrence
//
//   h_t[n] = exp(d_t A[c,n]) h_{t-1}[n] + d_t x_t[c] B_t[n],   y_t[c] = h_t . C_t + Dskip[c] x_t[c]
//
// per channel c, with a decay per channel and state, so no product over tokens
// or channels is shared and the tensor cores have nothing to contract: the work
// is 16 (N) exponentials and 64 (4 N) fp32 operations per channel and token
// against 8 bytes of bf16 traffic, about level with the memory on this GPU
// (MUFU.EX2 32 and fp32 128 lanes per clock and SM, measured).
//
// Layout.  A lane holds 4 states (n) of 4 channels; LPC = N / 4 lanes hold a
// channel, so a load of B_t or C_t from shared memory (one 16-byte load, four
// clocks of the SM's 128-byte path) serves 16 state updates, and the packed fp32
// operations take two states per issue slot.  y is summed over the LPC lanes by
// halving exchanges.
// Roles.  A CTA is 4 walk warps (the recurrence) and 4 side warps: these load x,
// dt, B and C of the next tile, compute d and d x into shared memory, and
// finish the previous tile (Dskip x, the gate, the store), so memory latency, the
// softplus and the gate run beside the recurrence.  One barrier per tile; two
// buffers.  y of a tile overwrites its d x.
// Segments.  With few rows and channels the sequence is cut: a first walk gives
// each segment's state from zero and its sum of d, a fold over the segments
// gives every segment's entering state, then all segments are walked at once.
#include "scan_common.cuh"

namespace ssd {

namespace {

enum WalkMode {
    WALK_Y = 0,     // y and the final state
    WALK_SEG = 1,   // a segment's state from zero (segment 0: from h0) into slot seg + 1, its sum of d
    WALK_CKPT = 2,  // the state before every eighth token
    WALK_ADJ = 3    // backwards: a segment's adjoint from zero (the last: from dfinal) into slot seg - 1
};

constexpr int kWalkWarps = 4, kSideThreads = 128, kWalkThreads = kWalkWarps * 32 + kSideThreads;

template <int LPC>
struct WalkShape {
    static constexpr int kGroups = 32 / LPC;            // channel quads per warp
    static constexpr int kDc = kWalkWarps * kGroups * 4;  // channels per CTA
    static constexpr int kNp = LPC * 4;
    static constexpr int kT = LPC == 2 ? 8 : LPC == 8 ? 32 : 16;  // tokens per tile
    static constexpr int kQuads = kDc / 4;
    static constexpr int kUnits = (kT * kQuads + kSideThreads - 1) / kSideThreads;   // quads of a token per side thread
    static constexpr int kBcUnits = (kT * LPC + kSideThreads - 1) / kSideThreads;
};

// Sums v[0..3] (one per channel of the quad) over the LPC lanes of a group.
// While a lane holds several channels, each exchange halves them.  Returns
// the number of channels left in v[0..]; `first` is the first one's index.
template <int LPC>
__device__ __forceinline__ void reduce_quad(float (&v)[4], int lane) {
    if (LPC == 2) {
        const bool hi = lane & 1;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float keep = hi ? v[k + 2] : v[k], send = hi ? v[k] : v[k + 2];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, send, 1);
        }
        return;
    }
    {
        const bool hi = lane & 2;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float keep = hi ? v[k + 2] : v[k], send = hi ? v[k] : v[k + 2];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, send, 2);
        }
    }
    {
        const bool hi = lane & 1;
        const float keep = hi ? v[1] : v[0], send = hi ? v[0] : v[1];
        v[0] = keep + __shfl_xor_sync(0xffffffffu, send, 1);
    }
#pragma unroll
    for (int off = 4; off < LPC; off <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
}

template <int IO, int LPC, int MODE, bool VEC>
__global__ void __launch_bounds__(kWalkThreads, 2)
scan_walk_kernel(ScanParams p) {
    using S = WalkShape<LPC>;
    constexpr int kT = S::kT, kDc = S::kDc, kNp = S::kNp, kU = S::kUnits, kBu = S::kBcUnits;
    constexpr bool kY = MODE == WALK_Y, kRev = MODE == WALK_ADJ;
    __shared__ __align__(16) float s_d[2][kT * kDc];
    __shared__ __align__(16) float s_w[2][kT * kDc];  // d x (backwards: the gated dy); y in its place afterwards
    __shared__ __align__(16) float s_b[2][kT * kNp];  // B (backwards: C)
    __shared__ __align__(16) float s_c[kY ? 2 : 1][kY ? kT * kNp : 4];

    const int g = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles;
    const int seg = MODE == WALK_ADJ ? blockIdx.y + 1 : blockIdx.y, b = blockIdx.z;
    const int dg = p.D / p.G;
    const int c0 = g * dg + tile * kDc;
    const int nch = min(kDc, (g + 1) * dg - c0);
    const int len = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.L) : p.L;
    const int tb = seg * p.seg_len;
    const int ntok = max(0, min(len, tb + p.seg_len) - tb);
    const int nt = (ntok + kT - 1) / kT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp < kWalkWarps) {
        const int ln = lane % LPC, ch0 = (warp * S::kGroups + lane / LPC) * 4, n0 = ln * 4;
        float2 h[4][2], a2[4][2];
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        const float *start = nullptr;
        if (MODE == WALK_Y || MODE == WALK_CKPT)
            start = seg > 0 ? p.seg_states + ((long long)b * p.nseg + seg) * p.D * p.N
                            : (p.h0 ? p.h0 + (long long)b * p.D * p.N : nullptr);
        else if (MODE == WALK_SEG)
            start = seg == 0 && p.h0 ? p.h0 + (long long)b * p.D * p.N : nullptr;
        else
            start = seg == p.nseg - 1 && p.dfinal ? p.dfinal + (long long)b * p.D * p.N : nullptr;
        const bool va = aligned_n4(p.A, p.N), vs = aligned_n4(start, p.N);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a[4] = {0.f, 0.f, 0.f, 0.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
            if (ch0 + j < nch) {
                const long long i = (long long)(c0 + ch0 + j) * p.N + n0;
                load_n4(p.A, i, n0, p.N, va, a);
                if (start) load_n4(start, i, n0, p.N, vs, s);
            }
            // the decay as a power of two: exp(d A) = 2^(d A log2 e)
            a2[j][0] = make_float2(a[0] * kLog2e, a[1] * kLog2e);
            a2[j][1] = make_float2(a[2] * kLog2e, a[3] * kLog2e);
            h[j][0] = make_float2(s[0], s[1]);
            h[j][1] = make_float2(s[2], s[3]);
        }
        __syncthreads();  // tile 0 staged
        for (int k = 0; k < nt; ++k) {
            const int buf = k & 1;
            const float *sd = s_d[buf] + ch0, *sb = s_b[buf] + n0, *sc = s_c[kY ? buf : 0] + n0;
            float *sw = s_w[buf] + ch0;
            const int steps = min(kT, ntok - k * kT);  // rounded up to 4 below: the rest of a tile is staged as d = 0
#pragma unroll 1
            for (int t4 = 0; t4 < steps; t4 += 4) {
                if (MODE == WALK_CKPT && t4 % kCkpt == 0) {
                    const long long ck = (long long)b * ((p.L + kCkpt - 1) / kCkpt) + (tb + k * kT + t4) / kCkpt;
                    const bool vk = p.N % 4 == 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (ch0 + j < nch)
                            store_n4(p.ckpt, (ck * p.D + c0 + ch0 + j) * p.N + n0, n0, p.N, vk, h[j][0].x, h[j][0].y,
                                     h[j][1].x, h[j][1].y);
                }
#pragma unroll
                for (int tt = 0; tt < 4; ++tt) {
                    const int t = t4 + tt;
                    const float4 d4 = *reinterpret_cast<const float4 *>(sd + t * kDc);
                    const float4 w4 = *reinterpret_cast<const float4 *>(sw + t * kDc);
                    const float4 b4 = *reinterpret_cast<const float4 *>(sb + t * kNp);
                    const float2 b0 = make_float2(b4.x, b4.y), b1 = make_float2(b4.z, b4.w);
                    const float d[4] = {d4.x, d4.y, d4.z, d4.w}, w[4] = {w4.x, w4.y, w4.z, w4.w};
                    float v[4];
                    float2 cc0, cc1;
                    if (kY) {
                        const float4 c4 = *reinterpret_cast<const float4 *>(sc + t * kNp);
                        cc0 = make_float2(c4.x, c4.y);
                        cc1 = make_float2(c4.z, c4.w);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 dd = dup(d[j]), ww = dup(w[j]);
                        const float2 e0 = decay2(dd, a2[j][0]), e1 = decay2(dd, a2[j][1]);
                        if (kRev) {  // a_t (p + ds_t C_t)
                            h[j][0] = __fmul2_rn(e0, __ffma2_rn(ww, b0, h[j][0]));
                            h[j][1] = __fmul2_rn(e1, __ffma2_rn(ww, b1, h[j][1]));
                        } else {
                            h[j][0] = __ffma2_rn(e0, h[j][0], __fmul2_rn(ww, b0));
                            h[j][1] = __ffma2_rn(e1, h[j][1], __fmul2_rn(ww, b1));
                        }
                        if (kY) {
                            const float2 acc = __ffma2_rn(h[j][1], cc1, __fmul2_rn(h[j][0], cc0));
                            v[j] = acc.x + acc.y;
                        }
                        if (MODE == WALK_SEG) sum[j] += d[j];
                    }
                    if (kY) {
                        reduce_quad<LPC>(v, lane);
                        float *o = sw + t * kDc;
                        if (LPC == 2) *reinterpret_cast<float2 *>(o + 2 * (lane & 1)) = make_float2(v[0], v[1]);
                        else if (ln < 4) o[ln] = v[0];  // lane bits 1, 0 chose the channel
                    }
                }
            }
            __syncthreads();
        }
        float *out = nullptr;
        if (MODE == WALK_Y && seg == p.nseg - 1 && p.final_state) out = p.final_state + (long long)b * p.D * p.N;
        if (MODE == WALK_SEG) out = p.seg_states + ((long long)b * p.nseg + seg + 1) * p.D * p.N;
        if (MODE == WALK_ADJ) out = p.adj + ((long long)b * p.nseg + seg - 1) * p.D * p.N;
        if (out) {
            const bool vo = aligned_n4(out, p.N);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (ch0 + j < nch) {
                    store_n4(out, (long long)(c0 + ch0 + j) * p.N + n0, n0, p.N, vo, h[j][0].x, h[j][0].y, h[j][1].x,
                             h[j][1].y);
                    if (MODE == WALK_SEG && ln == 0)
                        p.seg_sum[((long long)b * p.nseg + seg) * p.D + c0 + ch0 + j] = sum[j];
                }
        }
        return;
    }

    // ---- side warps
    const int ta = threadIdx.x - kWalkWarps * 32;
    const int q = ta % S::kQuads;  // the thread's quad of channels is the same in every unit
    const int nv = min(4, nch - q * 4);
    const long long cq = c0 + q * 4;
    const void *xin = kRev ? p.dy : p.x;
    const void *bm = kRev ? p.Cm : p.Bm;
    const long long bb = kRev ? p.cs[0] : p.bs[0], bt = kRev ? p.cs[1] : p.bs[1];
    const long long xb = kRev ? (long long)p.L * p.D : p.xs[0], xt = kRev ? p.D : p.xs[1];
    const long long gn = (long long)g * p.N;
    float bias[4] = {0.f, 0.f, 0.f, 0.f}, skip[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < nv) {
            if (p.dt_bias) bias[j] = __ldg(p.dt_bias + cq + j);
            if (kY && p.Dskip) skip[j] = __ldg(p.Dskip + cq + j);
        }

    Raw4 rx[kU], rdt[kU], rz[kRev ? kU : 1], rb[kBu], rc[kY ? kBu : 1];
    // token of position i of the walk
    auto token = [&](int i) { return (long long)(kRev ? tb + ntok - 1 - i : tb + i); };
    auto load_tile = [&](int k) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int unit = ta + kSideThreads * u, i = k * kT + unit / S::kQuads;
            const bool ok = unit < kT * S::kQuads && i < ntok && nv > 0;
            const long long t = token(i);
            rx[u] = load_raw4<IO, VEC>(xin, b * xb + t * xt + cq, ok, nv);
            rdt[u] = load_raw4_dt<IO, VEC>(p.dt, b * p.dts[0] + t * p.dts[1] + cq, ok, nv, p.dt32);
            if (kRev) rz[kRev ? u : 0] = load_raw4<IO, VEC>(p.z, b * p.zs[0] + t * p.zs[1] + cq, ok && p.z, nv);
        }
#pragma unroll
        for (int u = 0; u < kBu; ++u) {
            const int unit = ta + kSideThreads * u, i = k * kT + unit / LPC, n = unit % LPC * 4;
            const bool ok = unit < kT * LPC && i < ntok && n < p.N;
            const long long t = token(i);
            rb[u] = load_raw4<IO, VEC>(bm, b * bb + t * bt + gn + n, ok, p.N - n);
            if (kY) rc[kY ? u : 0] = load_raw4<IO, VEC>(p.Cm, b * p.cs[0] + t * p.cs[1] + gn + n, ok, p.N - n);
        }
    };
    auto stage_tile = [&](int k) {
        const int buf = k & 1;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int unit = ta + kSideThreads * u, tl = unit / S::kQuads, i = k * kT + tl;
            if (unit >= kT * S::kQuads) continue;
            float d[4] = {0.f, 0.f, 0.f, 0.f}, w[4] = {0.f, 0.f, 0.f, 0.f};
            if (i < ntok && nv > 0) {
                float x[4], dt[4];
                unpack4<IO, VEC>(rx[u], x);
                unpack4_dt<IO, VEC>(rdt[u], dt, p.dt32);
                float z[4];
                if (kRev && p.z) unpack4<IO, VEC>(rz[kRev ? u : 0], z);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < nv) {
                        d[j] = step_of<false>(dt[j], bias[j], p.softplus, p.has_limit, p.dt_min, p.dt_max).d;
                        if (kRev) w[j] = p.z ? x[j] * silu_fast(z[j]) : x[j];
                        else w[j] = d[j] * x[j];
                    }
            }
            *reinterpret_cast<float4 *>(&s_d[buf][tl * kDc + q * 4]) = make_float4(d[0], d[1], d[2], d[3]);
            *reinterpret_cast<float4 *>(&s_w[buf][tl * kDc + q * 4]) = make_float4(w[0], w[1], w[2], w[3]);
        }
#pragma unroll
        for (int u = 0; u < kBu; ++u) {
            const int unit = ta + kSideThreads * u, tl = unit / LPC, n = unit % LPC * 4;
            if (unit >= kT * LPC) continue;
            const bool in = k * kT + tl < ntok && n < p.N;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (in) unpack4<IO, VEC>(rb[u], v);
            *reinterpret_cast<float4 *>(&s_b[buf][tl * kNp + n]) = make_float4(v[0], v[1], v[2], v[3]);
            if (kY) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                if (in) unpack4<IO, VEC>(rc[kY ? u : 0], c);
                *reinterpret_cast<float4 *>(&s_c[kY ? buf : 0][kY ? tl * kNp + n : 0]) = make_float4(c[0], c[1], c[2], c[3]);
            }
        }
    };
    // The epilogue of a tile; its x is read again (a tile or two after its first read, from L1 or L2).
    auto finish_tile = [&](int k) {
        Raw4 ex[kU], ez[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int unit = ta + kSideThreads * u, i = k * kT + unit / S::kQuads;
            const bool ok = unit < kT * S::kQuads && i < ntok && nv > 0;
            const long long t = token(i);
            ex[u] = load_raw4<IO, VEC>(p.x, b * p.xs[0] + t * p.xs[1] + cq, ok && p.Dskip, nv);
            ez[u] = load_raw4<IO, VEC>(p.z, b * p.zs[0] + t * p.zs[1] + cq, ok && p.z, nv);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int unit = ta + kSideThreads * u, tl = unit / S::kQuads, i = k * kT + tl;
            if (unit >= kT * S::kQuads || i >= ntok || nv <= 0) continue;
            const float4 y4 = *reinterpret_cast<const float4 *>(&s_w[k & 1][tl * kDc + q * 4]);
            float y[4] = {y4.x, y4.y, y4.z, y4.w};
            if (p.Dskip) {
                float x[4];
                unpack4<IO, VEC>(ex[u], x);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = fmaf(skip[j], x[j], y[j]);
            }
            if (p.z) {
                float z[4];
                unpack4<IO, VEC>(ez[u], z);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] *= silu_fast(z[j]);
            }
            store4_io<IO, VEC>(p.y, ((long long)b * p.L + tb + i) * p.D + cq, nv, y);
        }
    };

    if (nt > 0) {
        load_tile(0);
        stage_tile(0);
        if (nt > 1) load_tile(1);
    }
    __syncthreads();
    for (int k = 0; k < nt; ++k) {
        if (kY && k > 0) finish_tile(k - 1);
        if (k + 1 < nt) stage_tile(k + 1);
        if (k + 2 < nt) load_tile(k + 2);
        __syncthreads();
    }
    if (kY) {
        if (nt > 0) finish_tile(nt - 1);
        // padding of this segment: zeros
        const int pad0 = tb + ntok, pad1 = min(p.L, tb + p.seg_len);
        const long long n = (long long)max(0, pad1 - pad0) * nch;
        for (long long i = ta; i < n; i += kSideThreads)
            st_io<IO>(p.y, (size_t)(((long long)b * p.L + pad0 + i / nch) * p.D + c0 + i % nch), 0.f);
    }
}

// The state entering every segment, in place: slot s + 1 holds segment s's own
// state; S(s+1) = exp(A sum_s) S(s) + own(s), in order.
__global__ void __launch_bounds__(256)
scan_fold_kernel(ScanParams p) {
    const long long dn = (long long)p.D * p.N;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= dn) return;
    const int b = blockIdx.y;
    const float a2 = __ldg(p.A + i) * kLog2e;
    const long long c = i / p.N;
    float *st = p.seg_states + (long long)b * p.nseg * dn + i;
    const float *sm = p.seg_sum + (long long)b * p.nseg * p.D + c;
    float s = st[dn];
    for (int k = 1; k < p.nseg - 1; ++k) {
        s = fmaf(ex2(a2 * sm[(long long)k * p.D]), s, st[(k + 1) * dn]);
        st[(k + 1) * dn] = s;
    }
}

// The same for the adjoint, from the last segment down: slot s holds the adjoint after segment s.
__global__ void __launch_bounds__(256)
scan_fold_adj_kernel(ScanParams p) {
    const long long dn = (long long)p.D * p.N;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= dn) return;
    const int b = blockIdx.y;
    const float a2 = __ldg(p.A + i) * kLog2e;
    const long long c = i / p.N;
    float *st = p.adj + (long long)b * p.nseg * dn + i;
    const float *sm = p.seg_sum + (long long)b * p.nseg * p.D + c;
    float s = st[(p.nseg - 2) * dn];
    for (int k = p.nseg - 2; k > 0; --k) {
        s = fmaf(ex2(a2 * sm[(long long)k * p.D]), s, st[(k - 1) * dn]);
        st[(k - 1) * dn] = s;
    }
}

// Whether every tensor the side warps touch moves in aligned groups of four.
bool walk_vec(const ScanParams &p, int io, int mode) {
    const long long dense[2] = {(long long)p.L * p.D, p.D};
    const bool adj = mode == WALK_ADJ, y = mode == WALK_Y;
    return p.D / p.G % 4 == 0 && p.N % 4 == 0 && (adj || vec4_strided(p.x, io, p.xs)) &&
           vec4_strided(p.dt, p.dt32 ? (int)IO_F32 : io, p.dts) && (adj || vec4_strided(p.Bm, io, p.bs)) &&
           (!(adj || y) || (vec4_strided(p.Cm, io, p.cs) && (!p.z || vec4_strided(p.z, io, p.zs)))) &&
           (!y || vec4_strided(p.y, io, dense)) && (!adj || vec4_strided(p.dy, io, dense));
}

template <int IO, int LPC, int MODE>
cudaError_t launch_walk_as(ScanParams p, cudaStream_t s) {
    p.tiles = (p.D / p.G + WalkShape<LPC>::kDc - 1) / WalkShape<LPC>::kDc;
    const int segs = MODE == WALK_SEG || MODE == WALK_ADJ ? p.nseg - 1 : p.nseg;
    const dim3 grid(p.G * p.tiles, segs, p.B);
    if (walk_vec(p, IO, MODE)) scan_walk_kernel<IO, LPC, MODE, true><<<grid, kWalkThreads, 0, s>>>(p);
    else scan_walk_kernel<IO, LPC, MODE, false><<<grid, kWalkThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <int IO, int MODE>
cudaError_t launch_walk_io(const ScanParams &p, cudaStream_t s) {
    switch (scan_lanes(p.N)) {
        case 2: return launch_walk_as<IO, 2, MODE>(p, s);
        case 4: return launch_walk_as<IO, 4, MODE>(p, s);
        case 8: return launch_walk_as<IO, 8, MODE>(p, s);
        case 16: return launch_walk_as<IO, 16, MODE>(p, s);
        case 32: return launch_walk_as<IO, 32, MODE>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

template <int MODE>
cudaError_t launch_walk(const ScanParams &p, int io, cudaStream_t s) {
    switch (io) {
        case IO_F32: return launch_walk_io<IO_F32, MODE>(p, s);
        case IO_F16: return launch_walk_io<IO_F16, MODE>(p, s);
        case IO_BF16: return launch_walk_io<IO_BF16, MODE>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t segment_states(const ScanParams &p, int io, cudaStream_t s) {
    if (p.nseg == 1) return cudaSuccess;
    cudaError_t e = launch_walk<WALK_SEG>(p, io, s);
    if (e != cudaSuccess || p.nseg == 2) return e;
    const long long dn = (long long)p.D * p.N;
    scan_fold_kernel<<<dim3((unsigned)((dn + 255) / 256), p.B), 256, 0, s>>>(p);
    return cudaGetLastError();
}

int g_scan_sms[64] = {};

}  // namespace

int scan_sm_count() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return 1;
    }
    if (g_scan_sms[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) (void)cudaGetLastError();
        g_scan_sms[dev] = n > 0 ? n : 1;
    }
    return g_scan_sms[dev];
}

cudaError_t launch_scan(const ScanParams &p, int io, cudaStream_t s) {
    cudaError_t e = segment_states(p, io, s);
    if (e != cudaSuccess) return e;
    return launch_walk<WALK_Y>(p, io, s);
}

cudaError_t launch_scan_ckpt(const ScanParams &p, int io, cudaStream_t s) {
    cudaError_t e = segment_states(p, io, s);
    if (e != cudaSuccess) return e;
    return launch_walk<WALK_CKPT>(p, io, s);
}

cudaError_t launch_scan_adjoint(const ScanParams &p, int io, cudaStream_t s) {
    if (p.nseg == 1) return cudaSuccess;
    cudaError_t e = launch_walk<WALK_ADJ>(p, io, s);
    if (e != cudaSuccess || p.nseg == 2) return e;
    const long long dn = (long long)p.D * p.N;
    scan_fold_adj_kernel<<<dim3((unsigned)((dn + 255) / 256), p.B), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace ssd

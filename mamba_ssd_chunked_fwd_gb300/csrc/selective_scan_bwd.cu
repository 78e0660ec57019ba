// selective_scan_bwd.cu -- gradients of the selective scan.  With q_t = dL/dh_t
// (all the way from the tokens after t), ds the gradient of the ungated output,
// and a_t = exp(d_t A):
//
//   q_t = ds_t C_t + a_{t+1} q_{t+1}          (per channel and state)
//   dC_t = sum_c ds_t h_t,   dB_t = sum_c d_t x_t q_t
//   dx_t = d_t (q_t . B_t) + Dskip ds_t
//   dd_t = x_t (q_t . B_t) + sum_n A q_t a_t h_{t-1},   dA = sum_t d_t q_t a_t h_{t-1}
//
// The states are needed in reverse: a forward walk (selective_scan.cu) stores
// the state before every eighth token (4 N / 8 bytes per channel and token,
// beside 14 of bf16 tensors), and this kernel recomputes eight tokens at a time
// from it, keeping a_t h_{t-1} of the eight in registers: h_t is that plus
// d x B, so one value per token and state serves every term, and no state is
// ever recovered by dividing by a decay.  About 13 fp32 operations and two
// exponentials per state, channel and token: bound by the fp32 pipes.
//
// Layout as in the forward, two channels per lane (the eight tokens' 64 values
// leave no room for four): LPC lanes with four states each per channel; the
// three sums over states meet across those lanes, the sums over channels
// (dB, dC) across the others, then over the CTA's walk warps in shared memory
// and over the channel tiles in a second kernel, each in a fixed order.
// Walk and side warps as in the forward: the side warps stage d, d x, ds, B and
// C of the next tile and turn the previous tile's sums into dx, ddt and dz.
#include "scan_common.cuh"

namespace ssd {

namespace {

constexpr int kBw = 4, kBside = 128, kBthreads = kBw * 32 + kBside;

template <int LPC>
struct BwdShape {
    static constexpr int kGroups = 32 / LPC;
    static constexpr int kDc = kBw * kGroups * 2;
    static constexpr int kNp = LPC * 4;
    static constexpr int kT = LPC == 4 || LPC == 8 ? 16 : 8;
    static constexpr int kQuads = kDc / 4;
    static constexpr int kUnits = (kT * kQuads + kBside - 1) / kBside;
    static constexpr int kBcUnits = (kT * LPC + kBside - 1) / kBside;
    static constexpr int kTile = kT * kDc;
    // floats: d, dx, ds and three results, two buffers; B and C; dB and dC per warp
    static constexpr int kFloats = 2 * (6 * kTile + 2 * kT * kNp + kBw * kT * 2 * kNp);
};

// v[0..7] (dB then dC of the lane's four states) summed over the channel
// groups of the warp; while a lane holds several sums an exchange halves them.
// Returns the index of the first one left in v[0..kLeft).
template <int LPC>
struct GroupSum {
    static constexpr int kLeft = LPC >= 32 ? 8 : LPC == 16 ? 4 : LPC == 8 ? 2 : 1;
    static __device__ __forceinline__ int run(float (&v)[8], int lane) {
        int idx = 0, cnt = 8;
#pragma unroll
        for (int off = LPC; off < 32; off <<= 1) {
            if (cnt > 1) {
                const bool hi = lane & off;
                cnt >>= 1;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < cnt) {
                        const float keep = hi ? v[i + cnt] : v[i], send = hi ? v[i] : v[i + cnt];
                        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
                    }
                idx += hi ? cnt : 0;
            } else {
                v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
            }
        }
        return idx;
    }
};

template <int IO, int LPC, bool VEC>
__global__ void __launch_bounds__(kBthreads, 2)
scan_bwd_kernel(ScanParams p) {
    using S = BwdShape<LPC>;
    constexpr int kT = S::kT, kDc = S::kDc, kNp = S::kNp, kU = S::kUnits, kBu = S::kBcUnits, kTile = S::kTile;
    extern __shared__ __align__(16) float smem[];
    float *s_d = smem, *s_w = s_d + 2 * kTile, *s_g = s_w + 2 * kTile, *s_o = s_g + 2 * kTile;  // s_o[buf][3][kTile]
    float *s_b = s_o + 6 * kTile, *s_c = s_b + 2 * kT * kNp, *s_p = s_c + 2 * kT * kNp;         // s_p[buf][warp][kT][2 kNp]

    const int g = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles;
    const int seg = blockIdx.y, b = blockIdx.z;
    const int dg = p.D / p.G;
    const int c0 = g * dg + tile * kDc;
    const int nch = min(kDc, (g + 1) * dg - c0);
    const int len = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.L) : p.L;
    const int tb = seg * p.seg_len;
    const int ntok = max(0, min(len, tb + p.seg_len) - tb);
    const int nt = (ntok + kT - 1) / kT;  // iteration i handles tile nt - 1 - i
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long bseg = (long long)b * p.nseg + seg;

    if (warp < kBw) {
        const int ln = lane % LPC, ch0 = (warp * S::kGroups + lane / LPC) * 2, n0 = ln * 4;
        float2 a2[2][2], q[2][2], da[2][2];
        const float *start = seg < p.nseg - 1 ? p.adj + bseg * p.D * p.N
                                              : (p.dfinal ? p.dfinal + (long long)b * p.D * p.N : nullptr);
        const bool va = aligned_n4(p.A, p.N), vs = aligned_n4(start, p.N), vk = p.N % 4 == 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float a[4] = {0.f, 0.f, 0.f, 0.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
            if (ch0 + j < nch) {
                const long long i = (long long)(c0 + ch0 + j) * p.N + n0;
                load_n4(p.A, i, n0, p.N, va, a);
                if (start) load_n4(start, i, n0, p.N, vs, s);
            }
            a2[j][0] = make_float2(a[0] * kLog2e, a[1] * kLog2e);
            a2[j][1] = make_float2(a[2] * kLog2e, a[3] * kLog2e);
            q[j][0] = make_float2(s[0], s[1]);
            q[j][1] = make_float2(s[2], s[3]);
            da[j][0] = da[j][1] = make_float2(0.f, 0.f);
        }
        const long long nck = (p.L + kCkpt - 1) / kCkpt;
        auto load_state = [&](int t, float2 (&h)[2][2]) {  // before token t of the segment, t % 8 == 0
            const long long ck = (long long)b * nck + (tb + t) / kCkpt;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float v[4] = {0.f, 0.f, 0.f, 0.f};
                if (ch0 + j < nch) load_n4(p.ckpt, (ck * p.D + c0 + ch0 + j) * p.N + n0, n0, p.N, vk, v);
                h[j][0] = make_float2(v[0], v[1]);
                h[j][1] = make_float2(v[2], v[3]);
            }
        };
        float2 hn[2][2];
        if (nt > 0) load_state((ntok - 1) / kCkpt * kCkpt, hn);
        __syncthreads();  // the last tile staged
        for (int i = 0; i < nt; ++i) {
            const int buf = i & 1, k = nt - 1 - i;
            const float *sd = s_d + buf * kTile + ch0, *sw = s_w + buf * kTile + ch0, *sg = s_g + buf * kTile + ch0;
            const float *sb = s_b + buf * kT * kNp + n0, *sc = s_c + buf * kT * kNp + n0;
            float *so = s_o + buf * 3 * kTile, *sp = s_p + (buf * kBw + warp) * kT * 2 * kNp;
#pragma unroll 1
            for (int t8 = (min(kT, ntok - k * kT) - 1) / 8 * 8; t8 >= 0; t8 -= 8) {  // staged as d = 0 past the last token
                float2 h[2][2], ah[8][2][2], da8[2][2];  // da8: dA of these eight tokens, then added to the long sum
#pragma unroll
                for (int j = 0; j < 2; ++j) h[j][0] = hn[j][0], h[j][1] = hn[j][1];
                if (k * kT + t8 >= 8) load_state(k * kT + t8 - 8, hn);
#pragma unroll
                for (int tt = 0; tt < 8; ++tt) {
                    const int t = t8 + tt;
                    const float2 d2 = *reinterpret_cast<const float2 *>(sd + t * kDc);
                    const float2 w2 = *reinterpret_cast<const float2 *>(sw + t * kDc);
                    const float4 b4 = *reinterpret_cast<const float4 *>(sb + t * kNp);
                    const float2 b0 = make_float2(b4.x, b4.y), b1 = make_float2(b4.z, b4.w);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float2 dd = dup(j ? d2.y : d2.x), ww = dup(j ? w2.y : w2.x);
                        ah[tt][j][0] = __fmul2_rn(decay2(dd, a2[j][0]), h[j][0]);
                        ah[tt][j][1] = __fmul2_rn(decay2(dd, a2[j][1]), h[j][1]);
                        h[j][0] = __ffma2_rn(ww, b0, ah[tt][j][0]);
                        h[j][1] = __ffma2_rn(ww, b1, ah[tt][j][1]);
                    }
                }
#pragma unroll
                for (int tt = 7; tt >= 0; --tt) {
                    const int t = t8 + tt;
                    const float2 d2 = *reinterpret_cast<const float2 *>(sd + t * kDc);
                    const float2 w2 = *reinterpret_cast<const float2 *>(sw + t * kDc);
                    const float2 g2 = *reinterpret_cast<const float2 *>(sg + t * kDc);
                    const float4 b4 = *reinterpret_cast<const float4 *>(sb + t * kNp);
                    const float4 c4 = *reinterpret_cast<const float4 *>(sc + t * kNp);
                    const float2 b0 = make_float2(b4.x, b4.y), b1 = make_float2(b4.z, b4.w);
                    const float2 cc0 = make_float2(c4.x, c4.y), cc1 = make_float2(c4.z, c4.w);
                    float2 db0, db1, dc0, dc1;
                    float r[2][3];  // q . B, sum of A q a h (in units of log2 e), h . C
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float2 dd = dup(j ? d2.y : d2.x), ww = dup(j ? w2.y : w2.x), gg = dup(j ? g2.y : g2.x);
                        const float2 q0 = __ffma2_rn(gg, cc0, q[j][0]), q1 = __ffma2_rn(gg, cc1, q[j][1]);
                        const float2 h0 = __ffma2_rn(ww, b0, ah[tt][j][0]), h1 = __ffma2_rn(ww, b1, ah[tt][j][1]);
                        if (j == 0) {
                            dc0 = __fmul2_rn(gg, h0); dc1 = __fmul2_rn(gg, h1);
                            db0 = __fmul2_rn(ww, q0); db1 = __fmul2_rn(ww, q1);
                        } else {
                            dc0 = __ffma2_rn(gg, h0, dc0); dc1 = __ffma2_rn(gg, h1, dc1);
                            db0 = __ffma2_rn(ww, q0, db0); db1 = __ffma2_rn(ww, q1, db1);
                        }
                        const float2 x0 = __fmul2_rn(q0, ah[tt][j][0]), x1 = __fmul2_rn(q1, ah[tt][j][1]);
                        const float2 vb = __ffma2_rn(q1, b1, __fmul2_rn(q0, b0));
                        const float2 vr = __ffma2_rn(x1, a2[j][1], __fmul2_rn(x0, a2[j][0]));
                        const float2 vc = __ffma2_rn(h1, cc1, __fmul2_rn(h0, cc0));
                        da8[j][0] = tt == 7 ? __fmul2_rn(dd, x0) : __ffma2_rn(dd, x0, da8[j][0]);
                        da8[j][1] = tt == 7 ? __fmul2_rn(dd, x1) : __ffma2_rn(dd, x1, da8[j][1]);
                        q[j][0] = __fmul2_rn(decay2(dd, a2[j][0]), q0);
                        q[j][1] = __fmul2_rn(decay2(dd, a2[j][1]), q1);
                        r[j][0] = vb.x + vb.y;
                        r[j][1] = vr.x + vr.y;
                        r[j][2] = vc.x + vc.y;
                    }
                    // over the channel's lanes: the first exchange leaves one channel per lane parity
                    float s[3];
#pragma unroll
                    for (int e = 0; e < 3; ++e) {
                        const bool hi = lane & 1;
                        const float keep = hi ? r[1][e] : r[0][e], send = hi ? r[0][e] : r[1][e];
                        s[e] = keep + __shfl_xor_sync(0xffffffffu, send, 1);
#pragma unroll
                        for (int off = 2; off < LPC; off <<= 1) s[e] += __shfl_xor_sync(0xffffffffu, s[e], off);
                        if (ln < 2) so[e * kTile + t * kDc + ch0 + ln] = s[e];
                    }
                    float v[8] = {db0.x, db0.y, db1.x, db1.y, dc0.x, dc0.y, dc1.x, dc1.y};
                    const int idx = GroupSum<LPC>::run(v, lane);
                    if (LPC > 2 || !(lane & 16)) {
#pragma unroll
                        for (int e = 0; e < GroupSum<LPC>::kLeft; ++e) {
                            const int m = idx + e;
                            sp[t * 2 * kNp + (m >> 2) * kNp + n0 + (m & 3)] = v[e];
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    da[j][0] = __fadd2_rn(da[j][0], da8[j][0]);
                    da[j][1] = __fadd2_rn(da[j][1], da8[j][1]);
                }
            }
            __syncthreads();
        }
        float *pa = p.part_a + bseg * p.D * p.N;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (ch0 + j < nch) {
                const long long i = (long long)(c0 + ch0 + j) * p.N + n0;
                store_n4(pa, i, n0, p.N, vk, da[j][0].x, da[j][0].y, da[j][1].x, da[j][1].y);
                if (seg == 0 && p.dh0) {
                    float *o = p.dh0 + (long long)b * p.D * p.N;
                    store_n4(o, i, n0, p.N, aligned_n4(o, p.N), q[j][0].x, q[j][0].y, q[j][1].x, q[j][1].y);
                }
            }
        __syncthreads();  // the side warps' sums of dD and ddt_bias use the shared memory again
        return;
    }

    // ---- side warps
    const int ta = threadIdx.x - kBw * 32;
    const int qd = ta % S::kQuads;
    const int nv = min(4, nch - qd * 4);
    const long long cq = c0 + qd * 4;
    const long long dense[2] = {(long long)p.L * p.D, p.D};
    const long long gn = (long long)g * p.N;
    float bias[4] = {0.f, 0.f, 0.f, 0.f}, skip[4] = {0.f, 0.f, 0.f, 0.f};
    float acc_d[4] = {0.f, 0.f, 0.f, 0.f}, acc_b[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < nv) {
            if (p.dt_bias) bias[j] = __ldg(p.dt_bias + cq + j);
            if (p.Dskip) skip[j] = __ldg(p.Dskip + cq + j);
        }
    Raw4 rx[kU], rdt[kU], rdy[kU], rz[kU], rb[kBu], rc[kBu];
    auto load_unit = [&](long long t, bool ok, Raw4 &x, Raw4 &dt, Raw4 &dy, Raw4 &z) {
        x = load_raw4<IO, VEC>(p.x, b * p.xs[0] + t * p.xs[1] + cq, ok, nv);
        dt = load_raw4_dt<IO, VEC>(p.dt, b * p.dts[0] + t * p.dts[1] + cq, ok, nv, p.dt32);
        dy = load_raw4<IO, VEC>(p.dy, b * dense[0] + t * dense[1] + cq, ok, nv);
        z = load_raw4<IO, VEC>(p.z, b * p.zs[0] + t * p.zs[1] + cq, ok && p.z, nv);
    };
    auto load_tile = [&](int i) {
        const int k = nt - 1 - i;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int unit = ta + kBside * u, t = k * kT + unit / S::kQuads;
            load_unit(tb + t, unit < kT * S::kQuads && t < ntok && nv > 0, rx[u], rdt[u], rdy[u], rz[u]);
        }
#pragma unroll
        for (int u = 0; u < kBu; ++u) {
            const int unit = ta + kBside * u, t = k * kT + unit / LPC, n = unit % LPC * 4;
            const bool ok = unit < kT * LPC && t < ntok && n < p.N;
            rb[u] = load_raw4<IO, VEC>(p.Bm, b * p.bs[0] + (long long)(tb + t) * p.bs[1] + gn + n, ok, p.N - n);
            rc[u] = load_raw4<IO, VEC>(p.Cm, b * p.cs[0] + (long long)(tb + t) * p.cs[1] + gn + n, ok, p.N - n);
        }
    };
    auto stage_tile = [&](int i) {
        const int buf = i & 1, k = nt - 1 - i;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int unit = ta + kBside * u, tl = unit / S::kQuads;
            if (unit >= kT * S::kQuads) continue;
            float d[4] = {0.f, 0.f, 0.f, 0.f}, w[4] = {0.f, 0.f, 0.f, 0.f}, gg[4] = {0.f, 0.f, 0.f, 0.f};
            if (k * kT + tl < ntok && nv > 0) {
                float x[4], dt[4], dy[4], z[4];
                unpack4<IO, VEC>(rx[u], x);
                unpack4_dt<IO, VEC>(rdt[u], dt, p.dt32);
                unpack4<IO, VEC>(rdy[u], dy);
                if (p.z) unpack4<IO, VEC>(rz[u], z);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < nv) {
                        d[j] = step_of<false>(dt[j], bias[j], p.softplus, p.has_limit, p.dt_min, p.dt_max).d;
                        w[j] = d[j] * x[j];
                        gg[j] = p.z ? dy[j] * silu_fast(z[j]) : dy[j];
                    }
            }
            const int o = buf * kTile + tl * kDc + qd * 4;
            *reinterpret_cast<float4 *>(s_d + o) = make_float4(d[0], d[1], d[2], d[3]);
            *reinterpret_cast<float4 *>(s_w + o) = make_float4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<float4 *>(s_g + o) = make_float4(gg[0], gg[1], gg[2], gg[3]);
        }
#pragma unroll
        for (int u = 0; u < kBu; ++u) {
            const int unit = ta + kBside * u, tl = unit / LPC, n = unit % LPC * 4;
            if (unit >= kT * LPC) continue;
            float v[4] = {0.f, 0.f, 0.f, 0.f}, c[4] = {0.f, 0.f, 0.f, 0.f};
            if (k * kT + tl < ntok && n < p.N) {
                unpack4<IO, VEC>(rb[u], v);
                unpack4<IO, VEC>(rc[u], c);
            }
            *reinterpret_cast<float4 *>(s_b + (buf * kT + tl) * kNp + n) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(s_c + (buf * kT + tl) * kNp + n) = make_float4(c[0], c[1], c[2], c[3]);
        }
    };
    auto finish_tile = [&](int i) {
        const int buf = i & 1, k = nt - 1 - i;
        Raw4 ex[kU], edt[kU], edy[kU], ez[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int unit = ta + kBside * u, t = k * kT + unit / S::kQuads;
            load_unit(tb + t, unit < kT * S::kQuads && t < ntok && nv > 0, ex[u], edt[u], edy[u], ez[u]);
        }
        // dB and dC of the tile over the walk warps
        for (int e = ta; e < kT * 2 * kNp; e += kBside) {
            const int t = k * kT + e / (2 * kNp);
            if (t >= ntok) break;
            const float *sp = s_p + buf * kBw * kT * 2 * kNp + e;
            float v = sp[0];
#pragma unroll
            for (int w = 1; w < kBw; ++w) v += sp[w * kT * 2 * kNp];
            p.part_bc[(((long long)blockIdx.x * p.B + b) * p.L + tb + t) * 2 * kNp + e % (2 * kNp)] = v;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int unit = ta + kBside * u, tl = unit / S::kQuads, t = k * kT + tl;
            if (unit >= kT * S::kQuads || t >= ntok || nv <= 0) continue;
            const int o = tl * kDc + qd * 4;
            const float4 d4 = *reinterpret_cast<const float4 *>(s_d + buf * kTile + o);
            const float4 g4 = *reinterpret_cast<const float4 *>(s_g + buf * kTile + o);
            const float4 b4 = *reinterpret_cast<const float4 *>(s_o + (buf * 3 + 0) * kTile + o);
            const float4 r4 = *reinterpret_cast<const float4 *>(s_o + (buf * 3 + 1) * kTile + o);
            const float4 c4 = *reinterpret_cast<const float4 *>(s_o + (buf * 3 + 2) * kTile + o);
            const float d[4] = {d4.x, d4.y, d4.z, d4.w}, ds[4] = {g4.x, g4.y, g4.z, g4.w};
            const float qb[4] = {b4.x, b4.y, b4.z, b4.w}, qr[4] = {r4.x, r4.y, r4.z, r4.w};
            const float hc[4] = {c4.x, c4.y, c4.z, c4.w};
            float x[4], dt[4], dx[4], ddt[4];
            unpack4<IO, VEC>(ex[u], x);
            unpack4_dt<IO, VEC>(edt[u], dt, p.dt32);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float sig = p.softplus ? sigmoid_f(dt[j] + bias[j]) : 1.f;
                if (p.has_limit)
                    sig = step_of<true>(dt[j], bias[j], p.softplus, p.has_limit, p.dt_min, p.dt_max).sig;
                dx[j] = fmaf(d[j], qb[j], skip[j] * ds[j]);
                ddt[j] = fmaf(x[j], qb[j], kLn2 * qr[j]) * sig;
                if (j < nv) {
                    acc_d[j] = fmaf(ds[j], x[j], acc_d[j]);
                    acc_b[j] += ddt[j];
                }
            }
            const long long at = ((long long)b * p.L + tb + t) * p.D + cq;
            store4_io<IO, VEC>(p.dx, at, nv, dx);
            if (IO != IO_F32 && p.dt32) store4_io<IO_F32, VEC>(p.ddt, at, nv, ddt);
            else store4_io<IO, VEC>(p.ddt, at, nv, ddt);
            if (p.z) {
                float z[4], dy[4], dz[4];
                unpack4<IO, VEC>(ez[u], z);
                unpack4<IO, VEC>(edy[u], dy);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float sg = sigmoid_f(z[j]);
                    dz[j] = dy[j] * fmaf(skip[j], x[j], hc[j]) * (sg * fmaf(z[j], 1.f - sg, 1.f));
                }
                store4_io<IO, VEC>(p.dz, at, nv, dz);
            }
        }
    };

    if (nt > 0) {
        load_tile(0);
        stage_tile(0);
        if (nt > 1) load_tile(1);
    }
    __syncthreads();
    for (int i = 0; i < nt; ++i) {
        if (i > 0) finish_tile(i - 1);
        if (i + 1 < nt) stage_tile(i + 1);
        if (i + 2 < nt) load_tile(i + 2);
        __syncthreads();
    }
    if (nt > 0) finish_tile(nt - 1);
    {  // padding of this segment: zeros
        const int pad0 = tb + ntok, pad1 = min(p.L, tb + p.seg_len);
        const long long n = (long long)max(0, pad1 - pad0) * nch;
        for (long long i = ta; i < n; i += kBside) {
            const size_t at = (size_t)(((long long)b * p.L + pad0 + i / nch) * p.D + c0 + i % nch);
            st_io<IO>(p.dx, at, 0.f);
            if (IO != IO_F32 && p.dt32) st_io<IO_F32>(p.ddt, at, 0.f);
            else st_io<IO>(p.ddt, at, 0.f);
            if (p.z) st_io<IO>(p.dz, at, 0.f);
        }
    }
    // dD and ddt_bias over the threads of a quad, in order
    __syncthreads();
    float *red = s_p;  // [kBside][8]
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        red[ta * 8 + j] = acc_d[j];
        red[ta * 8 + 4 + j] = acc_b[j];
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kBside) : "memory");
    if (ta < S::kQuads && nv > 0) {
        float s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = 0.f;
        for (int y = ta; y < kBside; y += S::kQuads)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] += red[y * 8 + j];
        for (int j = 0; j < nv; ++j) {
            p.part_d[bseg * p.D + cq + j] = s[j];
            p.part_d[((long long)p.B * p.nseg + bseg) * p.D + cq + j] = s[4 + j];
        }
    }
}

// dA, dD and ddt_bias: the parts of every row and segment in order, four interleaved sums.
__global__ void __launch_bounds__(256)
scan_bwd_sum_kernel(const float *part, int rows, long long n, float *out) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    int r = 0;
    for (; r + 4 <= rows; r += 4)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] += __ldg(part + (long long)(r + j) * n + i);
    for (; r < rows; ++r) s[0] += __ldg(part + (long long)r * n + i);
    out[i] = (s[0] + s[1]) + (s[2] + s[3]);
}

// dB and dC of a token and group over the group's channel tiles, four interleaved sums.
template <int IO>
__global__ void __launch_bounds__(256)
scan_bwd_bc_kernel(ScanParams p, int np, void *dB, void *dC) {
    const long long per = (long long)p.B * p.L * 2 * np;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= per) return;
    const int g = blockIdx.y, e = (int)(i % (2 * np)), n = e % np;
    if (n >= p.N) return;
    const long long bt = i / (2 * np);
    const int b = (int)(bt / p.L), t = (int)(bt % p.L);
    const int len = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.L) : p.L;
    float v = 0.f;
    if (t < len) {
        const float *src = p.part_bc + (long long)g * p.tiles * per + i;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        int k = 0;
        for (; k + 4 <= p.tiles; k += 4)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] += __ldg(src + (k + j) * per);
        for (; k < p.tiles; ++k) s[0] += __ldg(src + k * per);
        v = (s[0] + s[1]) + (s[2] + s[3]);
    }
    st_io<IO>(e < np ? dB : dC, (size_t)((bt * p.G + g) * p.N + n), v);
}

bool bwd_vec(const ScanParams &p, int io) {
    const long long dense[2] = {(long long)p.L * p.D, p.D};
    const int dio = p.dt32 ? (int)IO_F32 : io;
    return p.D / p.G % 4 == 0 && p.N % 4 == 0 && vec4_strided(p.x, io, p.xs) && vec4_strided(p.dt, dio, p.dts) &&
           vec4_strided(p.Bm, io, p.bs) && vec4_strided(p.Cm, io, p.cs) && (!p.z || vec4_strided(p.z, io, p.zs)) &&
           vec4_strided(p.dy, io, dense) && vec4_strided(p.dx, io, dense) && vec4_strided(p.ddt, dio, dense) &&
           (!p.z || vec4_strided(p.dz, io, dense));
}

template <int IO, int LPC>
cudaError_t launch_bwd_as(ScanParams p, void *dB, void *dC, cudaStream_t s) {
    using S = BwdShape<LPC>;
    constexpr int kBytes = S::kFloats * (int)sizeof(float);
    p.tiles = scan_bwd_tiles(p);
    auto *kernel = bwd_vec(p, IO) ? scan_bwd_kernel<IO, LPC, true> : scan_bwd_kernel<IO, LPC, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    kernel<<<dim3(p.G * p.tiles, p.nseg, p.B), kBthreads, kBytes, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const long long per = (long long)p.B * p.L * 2 * S::kNp;
    scan_bwd_bc_kernel<IO><<<dim3((unsigned)((per + 255) / 256), p.G), 256, 0, s>>>(p, S::kNp, dB, dC);
    return cudaGetLastError();
}

template <int IO>
cudaError_t launch_bwd_io(const ScanParams &p, void *dB, void *dC, cudaStream_t s) {
    switch (scan_lanes(p.N)) {
        case 2: return launch_bwd_as<IO, 2>(p, dB, dC, s);
        case 4: return launch_bwd_as<IO, 4>(p, dB, dC, s);
        case 8: return launch_bwd_as<IO, 8>(p, dB, dC, s);
        case 16: return launch_bwd_as<IO, 16>(p, dB, dC, s);
        case 32: return launch_bwd_as<IO, 32>(p, dB, dC, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

int scan_bwd_tiles(const ScanParams &p) {
    const int dc = kBw * 32 / scan_lanes(p.N) * 2;
    return (p.D / p.G + dc - 1) / dc;
}

cudaError_t launch_scan_bwd(const ScanParams &p, int io, void *dB, void *dC, float *dA, float *dD, float *dbias,
                            cudaStream_t s) {
    cudaError_t e = launch_scan_ckpt(p, io, s);
    if (e != cudaSuccess) return e;
    if ((e = launch_scan_adjoint(p, io, s)) != cudaSuccess) return e;
    switch (io) {
        case IO_F32: e = launch_bwd_io<IO_F32>(p, dB, dC, s); break;
        case IO_F16: e = launch_bwd_io<IO_F16>(p, dB, dC, s); break;
        case IO_BF16: e = launch_bwd_io<IO_BF16>(p, dB, dC, s); break;
        default: return cudaErrorInvalidValue;
    }
    if (e != cudaSuccess) return e;
    const int rows = p.B * p.nseg;
    auto sum = [&](const float *part, long long n, float *out) {
        if (!out) return;
        scan_bwd_sum_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(part, rows, n, out);
    };
    sum(p.part_a, (long long)p.D * p.N, dA);
    sum(p.part_d, p.D, dD);
    sum(p.part_d + (long long)rows * p.D, p.D, dbias);
    return cudaGetLastError();
}

}  // namespace ssd

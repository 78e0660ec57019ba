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
// Measured: [4,2048,4096,16] in bf16 with the gate 823 us (41e9 channel-tokens/s; its bytes alone
// would take 70 us, its exponentials 115): the checkpoint walk 184, this kernel 621 (issue
// active in 65 % of the cycles with 12.9 warps per SM), the last sums 16. [4,2048,4096,8] 640 us,
// [4,2048,1024,64] 930 us; [2,333,328,8] in fp32, cut into segments, 30 us in five
// dependent launches (120 uncut).
#include "scan_common.cuh"

namespace ssd {

namespace {

constexpr int kBw = 4, kBside = 128, kBthreads = kBw * 32 + kBside;

template <int IO, int LPC>
struct BwdShape {
    static constexpr int kGroups = 32 / LPC;
    static constexpr int kDc = kBw * kGroups * 2;
    static constexpr int kNp = LPC * 4;
    static constexpr int kT = IO != IO_F32 && (LPC == 4 || LPC == 8) ? 16 : 8;
    static constexpr int kTile = kT * kDc;
    // side threads deal in chunks of 16 bytes, as in the forward
    static constexpr int kEs = IO == IO_F32 ? 4 : 2, kCh = 16 / kEs, kPairs = kCh / 2;
    static constexpr int kChunks = kDc / kCh;
    static constexpr int kUStep = kBside / kChunks < kT ? kBside / kChunks : kT;
    static constexpr int kUnits = kT / kUStep;
    static constexpr int kBcChunks = kNp / kCh;
    static constexpr int kBcStep = kBside / kBcChunks < kT ? kBside / kBcChunks : kT;
    static constexpr int kBcUnits = kT / kBcStep;
    static constexpr int kAhead = 1, kSlots = kAhead + 3;
    static constexpr int kRawTile = kTile * kEs, kRawBc = kT * kNp * kEs;
    static constexpr int slot(int wide) { return 3 * kRawTile + (wide ? kTile * 4 : kRawTile) + 2 * kRawBc; }  // x, dy, z, dt, B, C
    // floats: d, dx, ds and three results, two buffers; B and C; dB and dC per warp
    static constexpr int kFloats = 2 * (6 * kTile + 2 * kT * kNp + kBw * kT * 2 * kNp);
    static constexpr int bytes(int wide) { return kFloats * 4 + kSlots * slot(wide); }
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
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    using S = BwdShape<IO, LPC>;
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

    // Walk warps hold eight tokens' states and need the registers the side warps
    // do not: 144 and 112 of the 128 a thread is launched with (152 and 104, 160 and 96
    // measured 1% and 3% slower).
    if (warp < kBw) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
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
        const int again = p.L >> 31;
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
                // A token's values are loaded before the sums of the token after it are
                // stored: the stores may alias them, as far as the compiler knows.
                float2 dn, wn, gn;
                float4 bn, cn;
                // `again` is 0, which the compiler cannot know: the values read above are read
                // anew, since kept from there they would take 64 more registers.
                auto load_token = [&](int tok) {
                    const int t = tok + again;
                    dn = *reinterpret_cast<const float2 *>(sd + t * kDc);
                    wn = *reinterpret_cast<const float2 *>(sw + t * kDc);
                    gn = *reinterpret_cast<const float2 *>(sg + t * kDc);
                    bn = *reinterpret_cast<const float4 *>(sb + t * kNp);
                    cn = *reinterpret_cast<const float4 *>(sc + t * kNp);
                };
                load_token(t8 + 7);
#pragma unroll
                for (int tt = 7; tt >= 0; --tt) {
                    const int t = t8 + tt;
                    const float2 d2 = dn, w2 = wn, g2 = gn;
                    const float4 b4 = bn, c4 = cn;
                    if (tt > 0) load_token(t - 1);
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
    asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
    const int ta = threadIdx.x - kBw * 32;
    const int qd = ta % S::kChunks, tl0 = ta / S::kChunks;
    const int nv = min(S::kCh, nch - qd * S::kCh);
    const long long cq = c0 + (nv > 0 ? qd * S::kCh : 0);
    constexpr int kEs = S::kEs, kP = S::kPairs;
    const bool wide = IO != IO_F32 && p.dt32;
    const int dts = wide ? 4 : kEs;
    const long long dense0 = (long long)p.L * p.D, dense1 = p.D, gn = (long long)g * p.N;
    auto at = [](const void *base, long long bytes) { return static_cast<const char *>(base) + bytes; };
    // the thread's place in token tb + tl0 of every tensor; tiles come last first
    const long long first = tb + tl0;
    const char *px = at(p.x, (b * p.xs[0] + first * p.xs[1] + cq) * kEs), *pz = at(p.z, (b * p.zs[0] + first * p.zs[1] + cq) * kEs);
    const char *pdt = at(p.dt, (b * p.dts[0] + first * p.dts[1] + cq) * dts);
    const long long oy = b * dense0 + first * dense1 + cq;
    const char *pdy = at(p.dy, oy * kEs);
    const int nb = ta % S::kBcChunks * S::kCh, tlb = ta / S::kBcChunks, nbv = min(S::kCh, p.N - nb);
    const char *pb = at(p.Bm, (b * p.bs[0] + (long long)(tb + tlb) * p.bs[1] + gn + (nbv > 0 ? nb : 0)) * kEs);
    const char *pc = at(p.Cm, (b * p.cs[0] + (long long)(tb + tlb) * p.cs[1] + gn + (nbv > 0 ? nb : 0)) * kEs);
    char *ring = reinterpret_cast<char *>(smem + S::kFloats);
    const int slot = S::slot(wide);
    const int ox = (tl0 * kDc + qd * S::kCh) * kEs, ody = S::kRawTile + ox, oz = 2 * S::kRawTile + ox;
    const int odt = 3 * S::kRawTile + (tl0 * kDc + qd * S::kCh) * dts;
    const int ob = 3 * S::kRawTile + kTile * dts + (tlb * kNp + nb) * kEs;
    float *pbc = p.part_bc + (((long long)blockIdx.x * p.B + b) * p.L + tb) * 2 * kNp;  // the segment's partial dB and dC
    const bool flip = ta & 4;
    float2 bias[kP], skip[kP], acc_d[kP], acc_b[kP];
#pragma unroll
    for (int j = 0; j < kP; ++j) {
        const bool in0 = 2 * j < nv, in1 = 2 * j + 1 < nv;
        bias[j] = make_float2(in0 && p.dt_bias ? __ldg(p.dt_bias + cq + 2 * j) : 0.f,
                              in1 && p.dt_bias ? __ldg(p.dt_bias + cq + 2 * j + 1) : 0.f);
        skip[j] = make_float2(in0 && p.Dskip ? __ldg(p.Dskip + cq + 2 * j) : 0.f,
                              in1 && p.Dskip ? __ldg(p.Dskip + cq + 2 * j + 1) : 0.f);
        acc_d[j] = acc_b[j] = dup(0.f);
    }
    // Every pointer stands at the thread's first token of the tile to be copied next.
    {
        const long long t = (long long)(nt > 0 ? nt - 1 : 0) * kT;
        px += t * p.xs[1] * kEs, pz += t * p.zs[1] * kEs, pdt += t * p.dts[1] * dts, pdy += t * dense1 * kEs;
        pb += t * p.bs[1] * kEs, pc += t * p.cs[1] * kEs;
    }
    const long long tx = (long long)kT * p.xs[1] * kEs, tz = (long long)kT * p.zs[1] * kEs, tdt = (long long)kT * p.dts[1] * dts,
                    tdy = kT * dense1 * kEs, tB = (long long)kT * p.bs[1] * kEs, tC = (long long)kT * p.cs[1] * kEs;
    auto load_tile = [&](int i) {
        if (i < nt) {
            const int k = nt - 1 - i;
            char *s = ring + i % S::kSlots * slot;
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int t = u * S::kUStep;  // from the thread's first token of the tile
                const int n = k * kT + tl0 + t < ntok ? nv : 0;
                if (tl0 < kT) {
                    char *d = s + u * S::kUStep * kDc * kEs;
                    copy_chunk<IO, VEC>(d + ox, px + t * p.xs[1] * kEs, n);
                    copy_chunk<IO, VEC>(d + ody, pdy + t * dense1 * kEs, n);
                    if (p.z) copy_chunk<IO, VEC>(d + oz, pz + t * p.zs[1] * kEs, n);
                    char *sd = s + odt + u * S::kUStep * kDc * dts;
                    const char *src = pdt + t * p.dts[1] * dts;
                    if (wide) {
                        copy_chunk<IO_F32, VEC>(sd, src, n);
                        copy_chunk<IO_F32, VEC>(sd + 16, src + 16, n - 4);
                    } else {
                        copy_chunk<IO, VEC>(sd, src, n);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kBu; ++u) {
                const int t = u * S::kBcStep;
                const int n = k * kT + tlb + t < ntok ? nbv : 0;
                if (tlb < kT) {
                    copy_chunk<IO, VEC>(s + ob + u * S::kBcStep * kNp * kEs, pb + t * p.bs[1] * kEs, n);
                    copy_chunk<IO, VEC>(s + ob + S::kRawBc + u * S::kBcStep * kNp * kEs, pc + t * p.cs[1] * kEs, n);
                }
            }
            px -= tx, pz -= tz, pdt -= tdt, pdy -= tdy, pb -= tB, pc -= tC;
        }
        cp_commit();
    };
    auto stage_tile = [&](int i) {
        const int buf = i & 1, k = nt - 1 - i;
        const char *s = ring + i % S::kSlots * slot;
        if (tl0 < kT) {
            float2 d[kU * kP];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const char *sd = s + odt + u * S::kUStep * kDc * dts;
                if (wide) {
                    read_chunk<IO_F32>(sd, d + u * kP);
                    if (kP == 4) read_chunk<IO_F32>(sd + 16, d + u * kP + 2);
                } else {
                    read_chunk<IO>(sd, d + u * kP);
                }
#pragma unroll
                for (int j = 0; j < kP; ++j) d[u * kP + j] = __fadd2_rn(d[u * kP + j], bias[j]);
            }
            steps_of<kU * kP>(d, p.softplus, p.has_limit, p.dt_min, p.dt_max);
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int n = k * kT + tl0 + u * S::kUStep < ntok ? nv : 0;  // nothing past the last token or channel
                float2 v[kP];
                const char *c = s + u * S::kUStep * kDc * kEs;
                const int o = buf * kTile + (tl0 + u * S::kUStep) * kDc + qd * S::kCh;
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    if (2 * j >= n) d[u * kP + j].x = 0.f;
                    if (2 * j + 1 >= n) d[u * kP + j].y = 0.f;
                }
                spread<kP>(s_d + o, d + u * kP, flip);
                read_chunk<IO>(c + ox, v);  // zeros where nothing was loaded
#pragma unroll
                for (int j = 0; j < kP; ++j) v[j] = __fmul2_rn(v[j], d[u * kP + j]);
                spread<kP>(s_w + o, v, flip);
                read_chunk<IO>(c + ody, v);
                if (p.z) {
                    float2 z[kP];
                    read_chunk<IO>(c + oz, z);
#pragma unroll
                    for (int j = 0; j < kP; ++j) v[j] = __fmul2_rn(v[j], silu2(z[j]));
                }
                spread<kP>(s_g + o, v, flip);
            }
        }
        if (tlb < kT) {
#pragma unroll
            for (int u = 0; u < kBu; ++u) {
                float2 v[kP];
                const int o = buf * kT * kNp + (tlb + u * S::kBcStep) * kNp + nb;
                read_chunk<IO>(s + ob + u * S::kBcStep * kNp * kEs, v);
                spread<kP>(s_b + o, v, flip);
                read_chunk<IO>(s + ob + S::kRawBc + u * S::kBcStep * kNp * kEs, v);
                spread<kP>(s_c + o, v, flip);
            }
        }
    };
    // A tile's d and ds are taken before the next staging overwrites them.
    float2 td[kU * kP], tg[kU * kP];
    auto take_tile = [&](int i) {
        if (tl0 < kT)
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int o = (i & 1) * kTile + (tl0 + u * S::kUStep) * kDc + qd * S::kCh;
                gather<kP>(s_d + o, td + u * kP, flip);
                gather<kP>(s_g + o, tg + u * kP, flip);
            }
    };
    auto finish_tile = [&](int i) {
        const int buf = i & 1, k = nt - 1 - i;
        const char *s = ring + i % S::kSlots * slot;
        // dB and dC of the tile over the walk warps
#pragma unroll
        for (int e0 = 0; e0 < kT * 2 * kNp; e0 += kBside * 4) {
            const int e = e0 + ta * 4;
            if (e < kT * 2 * kNp && k * kT + e / (2 * kNp) < ntok) {
                const float *sp = s_p + buf * kBw * kT * 2 * kNp + e;
                float2 lo = dup(0.f), hi = dup(0.f);
#pragma unroll
                for (int w = 0; w < kBw; ++w) {
                    const float4 v = *reinterpret_cast<const float4 *>(sp + w * kT * 2 * kNp);
                    lo = __fadd2_rn(lo, make_float2(v.x, v.y));
                    hi = __fadd2_rn(hi, make_float2(v.z, v.w));
                }
                *reinterpret_cast<float4 *>(pbc + (long long)k * kT * 2 * kNp + e) = make_float4(lo.x, lo.y, hi.x, hi.y);
            }
        }
        if (tl0 >= kT) return;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int t = k * kT + u * S::kUStep;  // from the thread's first token
            const int n = tl0 + t < ntok ? nv : 0;
            const int o = (tl0 + u * S::kUStep) * kDc + qd * S::kCh;
            const char *c = s + u * S::kUStep * kDc * kEs;
            float2 x[kP], qb[kP], v[kP], sig[kP];
            read_chunk<IO>(c + ox, x);
            gather<kP>(s_o + (buf * 3 + 0) * kTile + o, qb, flip);
#pragma unroll
            for (int j = 0; j < kP; ++j) {
                const float2 g2 = tg[u * kP + j];
                v[j] = __ffma2_rn(td[u * kP + j], qb[j], __fmul2_rn(skip[j], g2));
                acc_d[j] = __ffma2_rn(g2, x[j], acc_d[j]);  // both zero past the last token
            }
            const long long row = oy + t * dense1;
            store_chunk<IO, VEC>(static_cast<char *>(p.dx) + row * kEs, n, v);
            const char *sd = s + odt + u * S::kUStep * kDc * dts;
            if (wide) {
                read_chunk<IO_F32>(sd, sig);
                if (kP == 4) read_chunk<IO_F32>(sd + 16, sig + 2);
            } else {
                read_chunk<IO>(sd, sig);
            }
            gather<kP>(s_o + (buf * 3 + 1) * kTile + o, v, flip);
            if (p.has_limit) {
#pragma unroll
                for (int j = 0; j < kP; ++j)
                    sig[j] = make_float2(step_of<true>(sig[j].x, bias[j].x, p.softplus, 1, p.dt_min, p.dt_max).sig,
                                         step_of<true>(sig[j].y, bias[j].y, p.softplus, 1, p.dt_min, p.dt_max).sig);
            } else {
#pragma unroll
                for (int j = 0; j < kP; ++j) sig[j] = p.softplus ? sigmoid2(__fadd2_rn(sig[j], bias[j])) : dup(1.f);
            }
#pragma unroll
            for (int j = 0; j < kP; ++j) {
                v[j] = __fmul2_rn(__ffma2_rn(x[j], qb[j], __fmul2_rn(dup(kLn2), v[j])), sig[j]);
                if (2 * j < n) acc_b[j].x += v[j].x;
                if (2 * j + 1 < n) acc_b[j].y += v[j].y;
            }
            if (wide) {
                char *dst = static_cast<char *>(p.ddt) + row * 4;
                store_chunk<IO_F32, VEC>(dst, n, v);
                if (kP == 4) store_chunk<IO_F32, VEC>(dst + 16, n - 4, v + 2);
            } else {
                store_chunk<IO, VEC>(static_cast<char *>(p.ddt) + row * kEs, n, v);
            }
            if (p.z) {
                float2 z[kP], dy[kP];
                read_chunk<IO>(c + oz, z);
                read_chunk<IO>(c + ody, dy);
                gather<kP>(s_o + (buf * 3 + 2) * kTile + o, v, flip);
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const float2 sg = sigmoid2(z[j]);
                    const float2 slope = __fmul2_rn(sg, __ffma2_rn(z[j], __fadd2_rn(dup(1.f), make_float2(-sg.x, -sg.y)), dup(1.f)));
                    v[j] = __fmul2_rn(__fmul2_rn(dy[j], __ffma2_rn(skip[j], x[j], v[j])), slope);
                }
                store_chunk<IO, VEC>(static_cast<char *>(p.dz) + row * kEs, n, v);
            }
        }
    };

    for (int i = 0; i <= S::kAhead; ++i) load_tile(i);
    cp_wait<S::kAhead>();
    if (nt > 0) stage_tile(0);
    __syncthreads();
    for (int i = 0; i < nt; ++i) {
        load_tile(i + 1 + S::kAhead);
        if (i > 0) take_tile(i - 1);
        cp_wait<S::kAhead>();
        if (i + 1 < nt) stage_tile(i + 1);
        if (i > 0) finish_tile(i - 1);
        __syncthreads();
    }
    if (nt > 0) take_tile(nt - 1), finish_tile(nt - 1);
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
    // dD and ddt_bias over the threads of a quad, in order; past this barrier the tiles' buffers are free
    static_assert(kBside * 2 * S::kCh <= S::kFloats, "the sums' rows must fit the tiles' buffers");
    __syncthreads();
    float *red = smem;  // [kBside][2 kCh]
#pragma unroll
    for (int j = 0; j < kP; ++j) {
        *reinterpret_cast<float2 *>(red + ta * 2 * S::kCh + 2 * j) = acc_d[j];
        *reinterpret_cast<float2 *>(red + ta * 2 * S::kCh + S::kCh + 2 * j) = acc_b[j];
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kBside) : "memory");
    if (ta < S::kChunks && nv > 0) {
        float s[2 * S::kCh];
#pragma unroll
        for (int j = 0; j < 2 * S::kCh; ++j) s[j] = 0.f;
        for (int y = ta; y < kBside; y += S::kChunks)
#pragma unroll
            for (int j = 0; j < 2 * S::kCh; ++j) s[j] += red[y * 2 * S::kCh + j];
#pragma unroll
        for (int j = 0; j < S::kCh; ++j)
            if (j < nv) {
                p.part_d[bseg * p.D + cq + j] = s[j];
                p.part_d[((long long)p.B * p.nseg + bseg) * p.D + cq + j] = s[S::kCh + j];
            }
    }
}

// n rows of partial sums, `stride` apart, in order: four interleaved sums.
__device__ __forceinline__ float sum_rows(const float *src, int n, long long stride) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    int k = 0;
    for (; k + 8 <= n; k += 8) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = src[(k + j) * stride];
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j & 3] += v[j];
    }
    for (; k < n; ++k) s[0] += src[k * stride];
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// The second kernel's sums, by blocks: first dA, dD and ddt_bias over the rows
// and segments, then dB and dC of a token and group over the group's channel tiles.
struct ScanSums {
    int np;
    long long blocks_a, blocks_d;
    float *dA, *dD, *dbias;
    void *dB, *dC;
};

template <int IO>
__global__ void __launch_bounds__(256)
scan_bwd_sums_kernel(ScanParams p, ScanSums o) {
    tc::pdl_wait();
    const int rows = p.B * p.nseg, np = o.np;
    long long blk = blockIdx.x;
    if (blk < o.blocks_a) {
        const long long n = (long long)p.D * p.N, i = blk * 256 + threadIdx.x;
        if (i < n) o.dA[i] = sum_rows(p.part_a + i, rows, n);
        return;
    }
    blk -= o.blocks_a;
    if (blk < o.blocks_d) {
        const long long i = blk * 256 + threadIdx.x, c = i % p.D;
        float *dst = i < p.D ? o.dD : o.dbias;
        if (i < 2 * p.D && dst) dst[c] = sum_rows(p.part_d + (i < p.D ? 0 : (long long)rows * p.D) + c, rows, p.D);
        return;
    }
    blk -= o.blocks_d;
    const long long per = (long long)p.B * p.L * 2 * np, i = blk * 256 + threadIdx.x;  // over groups, tokens, dB then dC
    if (i >= per * p.G) return;
    const int g = (int)(i / per), e = (int)(i % (2 * np)), n = e % np;
    if (n >= p.N) return;
    const long long bt = i % per / (2 * np);
    const int b = (int)(bt / p.L), t = (int)(bt % p.L);
    const int len = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.L) : p.L;
    const float v = t < len ? sum_rows(p.part_bc + (long long)g * p.tiles * per + i % per, p.tiles, per) : 0.f;
    st_io<IO>(e < np ? o.dB : o.dC, (size_t)((bt * p.G + g) * p.N + n), v);
}

bool bwd_vec(const ScanParams &p, int io) {
    const long long dense[2] = {(long long)p.L * p.D, p.D};
    const int ch = io == IO_F32 ? 4 : 8, dio = p.dt32 ? (int)IO_F32 : io;
    return p.D / p.G % ch == 0 && p.N % ch == 0 && chunk_strided(p.x, io, p.xs) && chunk_strided(p.dt, dio, p.dts) &&
           chunk_strided(p.Bm, io, p.bs) && chunk_strided(p.Cm, io, p.cs) && (!p.z || chunk_strided(p.z, io, p.zs)) &&
           chunk_strided(p.dy, io, dense) && chunk_strided(p.dx, io, dense) && chunk_strided(p.ddt, dio, dense) &&
           (!p.z || chunk_strided(p.dz, io, dense));
}

template <int IO, int LPC>
cudaError_t launch_bwd_as(ScanParams p, ScanSums o, cudaStream_t s) {
    using S = BwdShape<IO, LPC>;
    const int bytes = S::bytes(IO != IO_F32 && p.dt32);
    p.tiles = scan_bwd_tiles(p);
    auto *kernel = bwd_vec(p, IO) ? scan_bwd_kernel<IO, LPC, true> : scan_bwd_kernel<IO, LPC, false>;
    cudaError_t e = allow_smem<S::bytes(IO != IO_F32)>(kernel);  // bytes depend on dt's type
    if (e != cudaSuccess) return e;
    e = launch_kernel(true, kernel, dim3(p.G * p.tiles, p.nseg, p.B), kBthreads, bytes, s, p);
    if (e != cudaSuccess) return e;
    o.np = S::kNp;
    o.blocks_a = ((long long)p.D * p.N + 255) / 256;
    o.blocks_d = (2LL * p.D + 255) / 256;
    const long long blocks = o.blocks_a + o.blocks_d + ((long long)p.B * p.L * 2 * S::kNp * p.G + 255) / 256;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_kernel(true, scan_bwd_sums_kernel<IO>, dim3((unsigned)blocks), 256, 0, s, p, o);
}

template <int IO>
cudaError_t launch_bwd_io(const ScanParams &p, const ScanSums &o, cudaStream_t s) {
    switch (scan_lanes(p.N)) {
        case 2: return launch_bwd_as<IO, 2>(p, o, s);
        case 4: return launch_bwd_as<IO, 4>(p, o, s);
        case 8: return launch_bwd_as<IO, 8>(p, o, s);
        case 16: return launch_bwd_as<IO, 16>(p, o, s);
        case 32: return launch_bwd_as<IO, 32>(p, o, s);
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
    const ScanSums o = {0, 0, 0, dA, dD, dbias, dB, dC};
    switch (io) {
        case IO_F32: return launch_bwd_io<IO_F32>(p, o, s);
        case IO_F16: return launch_bwd_io<IO_F16>(p, o, s);
        case IO_BF16: return launch_bwd_io<IO_BF16>(p, o, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace ssd

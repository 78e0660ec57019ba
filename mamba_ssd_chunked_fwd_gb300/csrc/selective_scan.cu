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
// Roles.  A CTA is 4 walk warps (the recurrence; 2 where N <= 8) and 4 side warps: these load x,
// dt, B and C of the next tile, compute d and d x into shared memory, and
// finish the previous tile (Dskip x, the gate, the store), so memory latency, the
// softplus and the gate run beside the recurrence.  One barrier per tile; two
// buffers.  y of a tile overwrites its d x.
// Segments.  With few rows and channels the sequence is cut: a first walk gives
// each segment's state from zero and its sum of d, a fold over the segments
// gives every segment's entering state, then all segments are walked at once.
// Measured in bf16 with the gate: [8,4096,4096,16] 690 us, 194e9 channel-tokens/s (1.6 TB/s
// of tensors, 23 % of the copy rate; its exponentials alone take 230 us, with the packed
// multiply-adds and the sums of y about 410); 256 CTAs fill 84 % of the 304 places.
// [1,16384,2048,16] cut into segments 275 us (1571 uncut: 16 CTAs); three fp32 rows of
// 517 tokens and 202 channels 17 to 18 us called in turn (68 uncut). Issue is active in 63 % of the
// cycles of the first of these, with 12.4 warps per SM. N = 4 takes 812 us where N = 8 takes 529: its rows
// of B and C are not whole chunks, and then no tensor moves in whole chunks (walk_vec).
// Tried and slower at N = 16: 8 side warps, CTAs of one or two walk warps, eight states per lane.
#include "scan_common.cuh"

namespace ssd {

namespace {

enum WalkMode {
    WALK_Y = 0,     // y and the final state
    WALK_SEG = 1,   // a segment's state from zero (segment 0: from h0) into slot seg + 1, its sum of d
    WALK_CKPT = 2,  // the state before every eighth token
    WALK_ADJ = 3,   // backwards: a segment's adjoint from zero (the last: from dfinal) into slot seg - 1
    WALK_BOTH = 4   // WALK_SEG and WALK_ADJ of every segment that needs them, in one launch
};

constexpr int kSideThreads = 128;

// Four states of four channels per lane: LPC = N / 4 lanes hold a channel.
template <int IO, int LPC>
struct WalkShape {
    static constexpr int kGroups = 32 / LPC;              // channel quads per warp
    static constexpr int kWalkWarps = scan_walk_warps(LPC), kThreads = kWalkWarps * 32 + kSideThreads;
    static constexpr int kDc = kWalkWarps * kGroups * 4;  // channels per CTA
    static constexpr int kNp = LPC * 4;
    // tokens per tile: fp32 tiles are half as long, so that two CTAs' rings fit an SM
    static constexpr int kElems = IO == IO_F32 ? 1024 : 2048;
    static constexpr int kMost = kNp <= 16 ? 32 : kNp > 64 && IO == IO_F32 ? 8 : 16;
    static constexpr int kT = kElems / kDc < kMost ? kElems / kDc : kMost;
    // Side threads deal in chunks of 16 bytes of the tensors' type.  A thread's
    // chunk of channels is fixed and its tokens are kUStep apart (threads past
    // a tile's tokens idle); likewise B and C.
    static constexpr int kEs = IO == IO_F32 ? 4 : 2, kCh = 16 / kEs, kPairs = kCh / 2;
    static constexpr int kChunks = kDc / kCh;
    static constexpr int kUStep = kSideThreads / kChunks < kT ? kSideThreads / kChunks : kT;
    static constexpr int kUnits = kT / kUStep;
    static constexpr int kBcChunks = kNp / kCh;
    static constexpr int kBcStep = kSideThreads / kBcChunks < kT ? kSideThreads / kBcChunks : kT;
    static constexpr int kBcUnits = kT / kBcStep;
    // The ring of tiles as loaded: from the one being finished to kAhead past the one being staged.
    static constexpr int kAhead = 2, kSlots = kAhead + 3;
    static constexpr int kRawTile = kT * kDc * kEs, kRawBc = kT * kNp * kEs;
};

// Bytes of shared memory: d, d x, B (and C), two buffers each; the ring: x, dt, z, B, C.
template <int IO, int LPC, int MODE>
struct WalkSmem {
    using S = WalkShape<IO, LPC>;
    static constexpr bool kY = MODE == WALK_Y, kZ = MODE == WALK_Y || MODE == WALK_ADJ;
    static constexpr int kStage = (2 * 2 * S::kT * S::kDc + (kY ? 4 : 2) * S::kT * S::kNp) * 4;
    static constexpr int slot(int dt32) {  // dt may be wider than x
        return S::kRawTile * (1 + (kZ ? 1 : 0)) + (dt32 ? S::kT * S::kDc * 4 : S::kRawTile) + S::kRawBc * (kY ? 2 : 1);
    }
    static constexpr int bytes(int dt32) { return kStage + S::kSlots * slot(dt32); }
};

// Sums v[0..15] (four tokens of four channels, token-major) over the LPC lanes
// of a group.  While a lane holds several values, an exchange halves them: lane
// bit 0 chooses the pair of tokens, bit 1 the token, bit 2 the pair of channels
// and so on, so that 16 values take 12 exchanges over four lanes and each lane
// is left with one token's four channels.  Returns the index of v[0].
template <int LPC>
struct QuadSum {
    static constexpr int kLeft = LPC == 2 ? 8 : LPC == 4 ? 4 : LPC == 8 ? 2 : 1;
    static __device__ __forceinline__ int run(float (&v)[16], int lane) {
        int idx = 0, cnt = 16;
#pragma unroll
        for (int off = 1; off < LPC; off <<= 1) {
            if (cnt > 1) {
                const bool hi = lane & off;
                cnt >>= 1;
#pragma unroll
                for (int i = 0; i < 8; ++i)
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

template <int IO, int LPC, int MODE, bool VEC>
__device__ __forceinline__ void walk(const ScanParams &p, const int seg) {
    using S = WalkShape<IO, LPC>;
    constexpr int kT = S::kT, kDc = S::kDc, kNp = S::kNp, kU = S::kUnits, kBu = S::kBcUnits, kH = 2;
    constexpr bool kY = MODE == WALK_Y, kRev = MODE == WALK_ADJ, kZ = kY || kRev;
    extern __shared__ __align__(16) float smem[];
    float *s_d = smem;                            // [2][kT][kDc]
    float *s_w = s_d + 2 * kT * kDc;              // d x (backwards: the gated dy); y in its place afterwards
    float *s_b = s_w + 2 * kT * kDc;              // [2][kT][kNp] B (backwards: C)
    float *s_c = s_b + 2 * kT * kNp;              // only with y
    char *ring = reinterpret_cast<char *>(s_b + (kY ? 4 : 2) * kT * kNp);

    const int g = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles;
    const int b = blockIdx.z;
    const int dg = p.D / p.G;
    const int c0 = g * dg + tile * kDc;
    const int nch = min(kDc, (g + 1) * dg - c0);
    const int len = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.L) : p.L;
    const int tb = seg * p.seg_len;
    const int ntok = max(0, min(len, tb + p.seg_len) - tb);
    const int nt = (ntok + kT - 1) / kT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp < S::kWalkWarps) {
        const int ln = lane % LPC, ch0 = (warp * S::kGroups + lane / LPC) * 4, n0 = ln * 4;
        float2 h[4][kH], a2[4][kH];
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
        auto store_state = [&](float *base, long long row, bool vec) {  // row: of [*, N]
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (ch0 + j < nch)
                    store_n4(base, (row + j) * p.N + n0, n0, p.N, vec, h[j][0].x, h[j][0].y, h[j][1].x, h[j][1].y);
        };
        __syncthreads();  // tile 0 staged
        for (int k = 0; k < nt; ++k) {
            const int buf = k & 1;
            const float *sd = s_d + buf * kT * kDc + ch0, *sb = s_b + buf * kT * kNp + n0, *sc = s_c + buf * kT * kNp + n0;
            float *sw = s_w + buf * kT * kDc + ch0;
            const int steps = min(kT, ntok - k * kT);  // rounded up to 4 below: the rest of a tile is staged as d = 0
#pragma unroll 1
            for (int t4 = 0; t4 < steps; t4 += 4) {
                if (MODE == WALK_CKPT && (k * kT + t4) % kCkpt == 0)
                    store_state(p.ckpt, ((long long)b * ((p.L + kCkpt - 1) / kCkpt) + (tb + k * kT + t4) / kCkpt) * p.D +
                                            c0 + ch0, p.N % 4 == 0);
                // d and d x of the four tokens first: y is stored over d x below, and a load after such a
                // store would have to wait for it.
                float4 d4[4], w4[4];
#pragma unroll
                for (int tt = 0; tt < 4; ++tt) {
                    d4[tt] = *reinterpret_cast<const float4 *>(sd + (t4 + tt) * kDc);
                    w4[tt] = *reinterpret_cast<const float4 *>(sw + (t4 + tt) * kDc);
                }
                float v[16];
#pragma unroll
                for (int tt = 0; tt < 4; ++tt) {
                    const int t = t4 + tt;
                    const float d[4] = {d4[tt].x, d4[tt].y, d4[tt].z, d4[tt].w};
                    const float w[4] = {w4[tt].x, w4[tt].y, w4[tt].z, w4[tt].w};
                    const float4 b4 = *reinterpret_cast<const float4 *>(sb + t * kNp);
                    const float2 bb[kH] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
                    float2 cc[kH];
                    if (kY) {
                        const float4 c4 = *reinterpret_cast<const float4 *>(sc + t * kNp);
                        cc[0] = make_float2(c4.x, c4.y);
                        cc[1] = make_float2(c4.z, c4.w);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 dd = dup(d[j]), ww = dup(w[j]);
                        float2 acc;
#pragma unroll
                        for (int m = 0; m < kH; ++m) {
                            const float2 e = decay2(dd, a2[j][m]);
                            if (kRev) h[j][m] = __fmul2_rn(e, __ffma2_rn(ww, bb[m], h[j][m]));  // a_t (p + ds_t C_t)
                            else h[j][m] = __ffma2_rn(e, h[j][m], __fmul2_rn(ww, bb[m]));
                            if (kY) acc = m == 0 ? __fmul2_rn(h[j][m], cc[m]) : __ffma2_rn(h[j][m], cc[m], acc);
                        }
                        if (kY) v[tt * 4 + j] = acc.x + acc.y;
                        if (MODE == WALK_SEG) sum[j] += d[j];
                    }
                }
                if (kY) {
                    const int idx = QuadSum<LPC>::run(v, lane);
                    constexpr int kLeft = QuadSum<LPC>::kLeft;
                    float *o = sw + (t4 + (idx >> 2)) * kDc + (idx & 3);
                    if (kLeft >= 4) {
#pragma unroll
                        for (int i = 0; i < kLeft; i += 4)
                            *reinterpret_cast<float4 *>(o + i / 4 * kDc) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    } else if (kLeft == 2) {
                        *reinterpret_cast<float2 *>(o) = make_float2(v[0], v[1]);
                    } else if (ln < 16) {
                        *o = v[0];
                    }
                }
            }
            __syncthreads();
        }
        if (MODE == WALK_Y && seg == p.nseg - 1 && p.final_state)
            store_state(p.final_state, (long long)b * p.D + c0 + ch0, aligned_n4(p.final_state, p.N));
        if (MODE == WALK_SEG) {
            store_state(p.seg_states, ((long long)b * p.nseg + seg + 1) * p.D + c0 + ch0, p.N % 4 == 0);
            if (ln == 0)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (ch0 + j < nch) p.seg_sum[((long long)b * p.nseg + seg) * p.D + c0 + ch0 + j] = sum[j];
        }
        if (MODE == WALK_ADJ) store_state(p.adj, ((long long)b * p.nseg + seg - 1) * p.D + c0 + ch0, p.N % 4 == 0);
        return;
    }

    // ---- side warps.  Every chunk is copied, staged and finished by one thread,
    // so its copies need no barrier but the thread's own wait, and every tensor
    // is walked by one pointer and one stride.
    const int ta = threadIdx.x - S::kWalkWarps * 32;
    const int q = ta % S::kChunks, tl0 = ta / S::kChunks;
    const int nv = min(S::kCh, nch - q * S::kCh);
    const int mine = nv > 0 && tl0 < kT ? ntok : 0;  // tokens for this thread
    const long long cq = c0 + (nv > 0 ? q * S::kCh : 0);
    const long long first = kRev ? tb + ntok - 1 - tl0 : tb + tl0, dir = kRev ? -1 : 1;
    constexpr int kEs = S::kEs, kP = S::kPairs;
    const bool wide = IO != IO_F32 && p.dt32;  // dt in fp32 beside 16-bit tensors: two chunks
    const int dts = wide ? 4 : kEs;
    auto at = [](const void *base, long long bytes) { return static_cast<const char *>(base) + bytes; };
    const long long dense0 = (long long)p.L * p.D, dense1 = p.D;
    const void *xin = kRev ? p.dy : p.x;
    const long long xb = kRev ? dense0 : p.xs[0], xt = kRev ? dense1 : p.xs[1];
    const char *lx = at(xin, (b * xb + first * xt + cq) * kEs);
    const char *ldt = at(p.dt, (b * p.dts[0] + first * p.dts[1] + cq) * dts);
    const char *lz = at(p.z, (b * p.zs[0] + first * p.zs[1] + cq) * kEs);
    char *fy = static_cast<char *>(p.y) + (b * dense0 + first * dense1 + cq) * kEs;
    const long long sx = dir * S::kUStep * xt * kEs, sdt = dir * S::kUStep * p.dts[1] * dts,
                    sz = dir * S::kUStep * p.zs[1] * kEs, sy = S::kUStep * dense1 * kEs;
    const int nb = ta % S::kBcChunks * S::kCh, tlb = ta / S::kBcChunks;
    const int nbv = min(S::kCh, p.N - nb);
    const int bmine = nbv > 0 && tlb < kT ? ntok : 0;
    const long long firstb = kRev ? tb + ntok - 1 - tlb : tb + tlb, gn = (long long)g * p.N + (nbv > 0 ? nb : 0);
    const char *lb = kRev ? at(p.Cm, (b * p.cs[0] + firstb * p.cs[1] + gn) * kEs) : at(p.Bm, (b * p.bs[0] + firstb * p.bs[1] + gn) * kEs);
    const char *lc = at(p.Cm, (b * p.cs[0] + firstb * p.cs[1] + gn) * kEs);
    const long long sb = dir * S::kBcStep * (kRev ? p.cs[1] : p.bs[1]) * kEs, sc = (long long)S::kBcStep * p.cs[1] * kEs;
    // a thread's chunks in a ring slot: x, z, dt, B, C
    const int slot = WalkSmem<IO, LPC, MODE>::slot(wide);
    const int ox = (tl0 * kDc + q * S::kCh) * kEs, oz = S::kRawTile + ox;
    const int odt = S::kRawTile * (kZ ? 2 : 1) + (tl0 * kDc + q * S::kCh) * dts;
    const int ob = S::kRawTile * (kZ ? 2 : 1) + kT * kDc * dts + (tlb * kNp + nb) * kEs;

    float2 bias[kP], skip[kP];
#pragma unroll
    for (int j = 0; j < kP; ++j) {
        const bool in0 = 2 * j < nv, in1 = 2 * j + 1 < nv;
        bias[j] = make_float2(in0 && p.dt_bias ? __ldg(p.dt_bias + cq + 2 * j) : 0.f,
                              in1 && p.dt_bias ? __ldg(p.dt_bias + cq + 2 * j + 1) : 0.f);
        skip[j] = make_float2(kY && in0 && p.Dskip ? __ldg(p.Dskip + cq + 2 * j) : 0.f,
                              kY && in1 && p.Dskip ? __ldg(p.Dskip + cq + 2 * j + 1) : 0.f);
    }

    auto load_tile = [&](int k) {
        if (k < nt) {
            char *s = ring + k % S::kSlots * slot;
            int left = mine - k * kT - tl0;  // > 0: the unit's token exists
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int n = left > 0 ? nv : 0;
                if (tl0 < kT) {
                    copy_chunk<IO, VEC>(s + ox + u * S::kUStep * kDc * kEs, lx, n);
                    char *sd = s + odt + u * S::kUStep * kDc * dts;
                    if (wide) {
                        copy_chunk<IO_F32, VEC>(sd, ldt, n);
                        copy_chunk<IO_F32, VEC>(sd + 16, ldt + 16, n - 4);
                    } else {
                        copy_chunk<IO, VEC>(sd, ldt, n);
                    }
                    if (kZ && p.z) copy_chunk<IO, VEC>(s + oz + u * S::kUStep * kDc * kEs, lz, n);
                }
                left -= S::kUStep;
                lx += sx;
                ldt += sdt;
                lz += sz;
            }
            int leftb = bmine - k * kT - tlb;
#pragma unroll
            for (int u = 0; u < kBu; ++u) {
                const int n = leftb > 0 ? nbv : 0;
                if (tlb < kT) {
                    copy_chunk<IO, VEC>(s + ob + u * S::kBcStep * kNp * kEs, lb, n);
                    if (kY) copy_chunk<IO, VEC>(s + ob + S::kRawBc + u * S::kBcStep * kNp * kEs, lc, n);
                }
                leftb -= S::kBcStep;
                lb += sb;
                lc += sc;
            }
        }
        cp_commit();  // a group per tile, empty ones at the end
    };
    const bool flip = ta & 4;
    auto stage_tile = [&](int k) {
        const int buf = k & 1, left = mine - k * kT - tl0;
        const char *s = ring + k % S::kSlots * slot;
        if (tl0 < kT) {
            float2 d[kU * kP], w[kU * kP];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                read_chunk<IO>(s + ox + u * S::kUStep * kDc * kEs, w + u * kP);
                const char *sd = s + odt + u * S::kUStep * kDc * dts;
                if (wide) {
                    read_chunk<IO_F32>(sd, d + u * kP);
                    if (kP == 4) read_chunk<IO_F32>(sd + 16, d + u * kP + 2);
                } else {
                    read_chunk<IO>(sd, d + u * kP);
                }
#pragma unroll
                for (int i = 0; i < kP; ++i) d[u * kP + i] = __fadd2_rn(d[u * kP + i], bias[i]);
            }
            steps_of<kU * kP>(d, p.softplus, p.has_limit, p.dt_min, p.dt_max);
            if (!kRev) {
#pragma unroll
                for (int i = 0; i < kU * kP; ++i) w[i] = __fmul2_rn(w[i], d[i]);
            } else if (p.z) {
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    float2 z[kP];
                    read_chunk<IO>(s + oz + u * S::kUStep * kDc * kEs, z);
#pragma unroll
                    for (int i = 0; i < kP; ++i) w[u * kP + i] = __fmul2_rn(w[u * kP + i], silu2(z[i]));
                }
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                // no step past the last token or the group's last channel (x is zero there)
                const int n = left - u * S::kUStep > 0 ? nv : 0;
#pragma unroll
                for (int i = 0; i < kP; ++i) {
                    if (2 * i >= n) d[u * kP + i].x = 0.f, w[u * kP + i].x = 0.f;
                    if (2 * i + 1 >= n) d[u * kP + i].y = 0.f, w[u * kP + i].y = 0.f;
                }
                const int o = buf * kT * kDc + (tl0 + u * S::kUStep) * kDc + q * S::kCh;
                spread<kP>(s_d + o, d + u * kP, flip);
                spread<kP>(s_w + o, w + u * kP, flip);
            }
        }
        if (tlb < kT) {
#pragma unroll
            for (int u = 0; u < kBu; ++u) {  // zeros where nothing was loaded
                float2 v[kP];
                const int o = buf * kT * kNp + (tlb + u * S::kBcStep) * kNp + nb;
                read_chunk<IO>(s + ob + u * S::kBcStep * kNp * kEs, v);
                spread<kP>(s_b + o, v, flip);
                if (kY) {
                    read_chunk<IO>(s + ob + S::kRawBc + u * S::kBcStep * kNp * kEs, v);
                    spread<kP>(s_c + o, v, flip);
                }
            }
        }
    };
    // The epilogue of a tile, in two parts: the y that the next staging overwrites is taken first.
    float2 y[kY ? kU * kP : 1];
    auto take_tile = [&](int k) {
        if (tl0 < kT)
#pragma unroll
            for (int u = 0; u < (kY ? kU : 0); ++u)
                gather<kP>(s_w + (k & 1) * kT * kDc + (tl0 + u * S::kUStep) * kDc + q * S::kCh, y + u * kP, flip);
    };
    auto finish_tile = [&](int k) {
        const int left = mine - k * kT - tl0;
        const char *s = ring + k % S::kSlots * slot;
        if (tl0 < kT) {
            if (p.Dskip) {
#pragma unroll
                for (int u = 0; u < (kY ? kU : 0); ++u) {
                    float2 x[kP];
                    read_chunk<IO>(s + ox + u * S::kUStep * kDc * kEs, x);
#pragma unroll
                    for (int i = 0; i < kP; ++i) y[u * kP + i] = __ffma2_rn(skip[i], x[i], y[u * kP + i]);
                }
            }
            if (p.z) {
#pragma unroll
                for (int u = 0; u < (kY ? kU : 0); ++u) {
                    float2 z[kP];
                    read_chunk<IO>(s + oz + u * S::kUStep * kDc * kEs, z);
#pragma unroll
                    for (int i = 0; i < kP; ++i) y[u * kP + i] = __fmul2_rn(y[u * kP + i], silu2(z[i]));
                }
            }
        }
#pragma unroll
        for (int u = 0; u < (kY ? kU : 0); ++u) {
            store_chunk<IO, VEC>(fy, left - u * S::kUStep > 0 ? nv : 0, y + u * kP);
            fy += sy;
        }
    };

    // Groups committed at the start of iteration k: tiles 0 .. k + kAhead; tile k + 1 is needed.
    for (int k = 0; k <= S::kAhead; ++k) load_tile(k);
    cp_wait<S::kAhead>();
    if (nt > 0) stage_tile(0);
    __syncthreads();
    for (int k = 0; k < nt; ++k) {
        load_tile(k + 1 + S::kAhead);  // into the slot of tile k - 2, which is finished
        if (kY && k > 0) take_tile(k - 1);
        cp_wait<S::kAhead>();
        if (k + 1 < nt) stage_tile(k + 1);
        if (kY && k > 0) finish_tile(k - 1);
        __syncthreads();
    }
    if (kY) {
        if (nt > 0) take_tile(nt - 1), finish_tile(nt - 1);
        // padding of this segment: zeros
        const int pad0 = tb + ntok, pad1 = min(p.L, tb + p.seg_len);
        const long long n = (long long)max(0, pad1 - pad0) * nch;
        for (long long i = ta; i < n; i += kSideThreads)
            st_io<IO>(p.y, (size_t)(((long long)b * p.L + pad0 + i / nch) * p.D + c0 + i % nch), 0.f);
    }
}

template <int IO, int LPC, int MODE, bool VEC>
__global__ void __launch_bounds__((WalkShape<IO, LPC>::kThreads), 2)
scan_walk_kernel(ScanParams p) {
    if (MODE == WALK_Y || MODE == WALK_CKPT) tc::pdl_wait();
    if (MODE != WALK_Y) tc::pdl_launch_dependents();
    if (MODE != WALK_BOTH) {
        walk<IO, LPC, MODE == WALK_BOTH ? WALK_SEG : MODE, VEC>(p, blockIdx.y);
    } else if ((int)blockIdx.y < p.nseg - 1) {
        walk<IO, LPC, WALK_SEG, VEC>(p, blockIdx.y);
    } else {
        walk<IO, LPC, WALK_ADJ, VEC>(p, blockIdx.y - (p.nseg - 1) + 1);
    }
}

// The state entering every segment, in place: slot s + 1 holds segment s's own
// state; S(s+1) = exp(A sum_s) S(s) + own(s), in order.  blockIdx.z = 1: the same for
// the adjoint from the last segment down, slot s holding the adjoint after segment s.
// Eight segments' values are loaded together: the order of the sums is a chain of
// multiply-adds, not of memory latencies.
__global__ void __launch_bounds__(128)
scan_fold_kernel(ScanParams p) {
    constexpr int kStep = 8;
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    const bool adj = blockIdx.z;
    const long long dn = (long long)p.D * p.N;
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    if (i >= dn) return;
    const int b = blockIdx.y, n = p.nseg - 2;  // sums of n segments on top of the first slot
    const float a2 = __ldg(p.A + i) * kLog2e;
    float *st = (adj ? p.adj : p.seg_states) + (long long)b * p.nseg * dn + i;
    const float *sm = p.seg_sum + (long long)b * p.nseg * p.D + i / p.N;
    float s = st[(adj ? n : 1) * dn];
    for (int k0 = 0; k0 < n; k0 += kStep) {
        float own[kStep], sum[kStep];
#pragma unroll
        for (int j = 0; j < kStep; ++j) {
            const int k = adj ? n - (k0 + j) : k0 + j + 1;  // the segment passed through
            if (k0 + j < n) {
                own[j] = st[(adj ? k - 1 : k + 1) * dn];
                sum[j] = sm[(long long)k * p.D];
            }
        }
#pragma unroll
        for (int j = 0; j < kStep; ++j) {
            const int k = adj ? n - (k0 + j) : k0 + j + 1;
            if (k0 + j < n) {
                s = fmaf(ex2(a2 * sum[j]), s, own[j]);
                st[(adj ? k - 1 : k + 1) * dn] = s;
            }
        }
    }
}

// Whether every tensor the side warps touch moves in aligned, whole chunks of 16 bytes.
bool walk_vec(const ScanParams &p, int io, int mode) {
    const long long dense[2] = {(long long)p.L * p.D, p.D};
    const bool adj = mode == WALK_BOTH, y = mode == WALK_Y;
    const int ch = io == IO_F32 ? 4 : 8;
    return p.D / p.G % ch == 0 && p.N % ch == 0 && chunk_strided(p.x, io, p.xs) &&
           chunk_strided(p.dt, p.dt32 ? (int)IO_F32 : io, p.dts) && chunk_strided(p.Bm, io, p.bs) &&
           (!(adj || y) || (chunk_strided(p.Cm, io, p.cs) && (!p.z || chunk_strided(p.z, io, p.zs)))) &&
           (!y || chunk_strided(p.y, io, dense)) && (!adj || chunk_strided(p.dy, io, dense));
}

template <int IO, int LPC, int MODE>
cudaError_t launch_walk_as(ScanParams p, cudaStream_t s) {
    constexpr int kDc = WalkShape<IO, LPC>::kDc;
    p.tiles = (p.D / p.G + kDc - 1) / kDc;
    const int segs = MODE == WALK_SEG ? p.nseg - 1 : MODE == WALK_BOTH ? 2 * (p.nseg - 1) : p.nseg;
    constexpr int kMost = MODE == WALK_BOTH ? (int)WALK_ADJ : MODE;  // the mode that needs the most
    const int bytes = WalkSmem<IO, LPC, kMost>::bytes(IO != IO_F32 && p.dt32);
    auto *kernel = walk_vec(p, IO, MODE) ? scan_walk_kernel<IO, LPC, MODE, true> : scan_walk_kernel<IO, LPC, MODE, false>;
    cudaError_t e = allow_smem<WalkSmem<IO, LPC, kMost>::bytes(IO != IO_F32)>(kernel);  // bytes depend on dt's type
    if (e != cudaSuccess) return e;
    const bool after = (MODE == WALK_Y || MODE == WALK_CKPT) && p.nseg > 1;  // the cut's kernels
    return launch_kernel(after, kernel, dim3(p.G * p.tiles, segs, p.B), WalkShape<IO, LPC>::kThreads, bytes, s, p);
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

// What the segments start from: their states, and backwards their adjoints.
cudaError_t cut(const ScanParams &p, int io, bool backward, cudaStream_t s) {
    if (p.nseg == 1) return cudaSuccess;
    cudaError_t e = backward ? launch_walk<WALK_BOTH>(p, io, s) : launch_walk<WALK_SEG>(p, io, s);
    if (e != cudaSuccess || p.nseg == 2) return e;
    const long long dn = (long long)p.D * p.N;
    return launch_kernel(true, scan_fold_kernel, dim3((unsigned)((dn + 127) / 128), p.B, backward ? 2 : 1), 128, 0, s, p);
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
    cudaError_t e = cut(p, io, false, s);
    return e != cudaSuccess ? e : launch_walk<WALK_Y>(p, io, s);
}

cudaError_t launch_scan_ckpt(const ScanParams &p, int io, cudaStream_t s) {
    cudaError_t e = cut(p, io, true, s);
    return e != cudaSuccess ? e : launch_walk<WALK_CKPT>(p, io, s);
}

}  // namespace ssd

// delta_walk_tc.cuh -- the gated delta rule in chunks of 64 tokens on the tensor cores, for
// 16-bit tensors: the walk over the chunks.
//
// With G the running sum of g in a chunk, S the P x N state before it, and T and M of delta_prep.cu:
//
//     U = T diag(beta) (V - diag(exp G) K S^T)
//     Y = scale (diag(exp G) Q S^T + M U)
//     S <- exp(G_end) S + (diag(exp(G_end - G)) U)^T K
//
// A CTA walks the chunks of one head with up to 128 rows of its state, everything
// transposed: the state's rows are the 128 lanes of TMEM, and what the tokens'
// products with the state give (S K^T, U^T) lies along its columns, where the next
// product takes it as its A operand.  Only the chain S K^T -> U -> S is sequential,
// three products to a chunk; the rest runs beside it:
//
//   16 warps the chain: split S K^T, U and S into operands; the state's fp32 in registers
//   4 warps  y
//   1 warp   issues the products
//   3 warps  copy k, q, and v with a chunk's operands ahead
//
// Operands.  q, k and v are 16-bit as they come.  What is computed (S, S K^T, U, T, M) goes
// into a product as the sum of two 16-bit numbers, so that states keep 16 bits (bf16:
// relative error 4e-6 of a state, measured; one term would give 3e-3) and y is off by
// its own rounding alone.  In fp16 these terms hold values times powers of two (delta_tc.cuh), which the chain takes anew for
// every chunk, of a row of the state with its v: the state's largest over four threads, v's as the y warps have found it two
// chunks ahead, and v written back scaled while S k^T runs.  That and the state's columns leaving only once all are known make
// the walk 319 us for 213 in the case below (v's largest found by the chain's own warps: 344).
//
// Bound by the chain: 6300 cycles a chunk for three products and three round trips through registers, with the
// tensor pipe busy 41 % of them.  [4,4096] with 32 heads of 128 x 128, bf16: 213 us, 807 TFLOP/s of the products as formed.
//
// Every wait is bounded; once one gives up, what the CTA still writes is NaN.
#pragma once

#include "delta_tc.cuh"

namespace ssd {
namespace delta_walk {

constexpr int kChainWarps = 16, kOutWarps = 4, kOutWarp0 = kChainWarps, kMmaWarp = kOutWarp0 + kOutWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = (kLoadWarp + 3) * 32;
constexpr int kStages = 3;   // of k and q
constexpr int kVStages = 2;  // of v
constexpr int kOps = 2;      // of a chunk's operands
constexpr int kSlots = 4;    // of its gates

template <int NN>
struct Smem {
    static constexpr uint32_t KQ = 0, KQ_BYTES = 128 * NN * 2;  // rows 0-63 k, 64-127 q
    static constexpr uint32_t V = KQ + kStages * KQ_BYTES, V_BYTES = kC * 128 * 2;
    static constexpr uint32_t OP = V + kVStages * V_BYTES, GATES = OP + kOps * kOpGates, BYTES = GATES + kSlots * (uint32_t)sizeof(Gates);
};

enum Bar { kFullKQ = 0, kEmptyKQ = kFullKQ + kStages, kFullV = kEmptyKQ + kStages, kEmptyV = kFullV + kVStages, kFullOp = kEmptyV + kVStages,
           kEmptyOp = kFullOp + kOps, kD3 = kEmptyOp + kOps, kD3Read = kD3 + 2, kD4 = kD3Read + 2, kD4Read = kD4 + 2, kD1 = kD4Read + 2, kD2, kDS, kUOut, kS,
           kR = kS + 2, kU = kR + 4, kVUnit = kU + 4, kVMost, kDrain = kVMost + 2, kBars };

// TMEM columns.
template <int NN>
struct Tm {
    static constexpr uint32_t S = 0, X1 = NN, X2 = NN + 64, DS = NN + 128, O = 2 * NN + 128, COLS = 512;  // two of O
};

// What a CTA walks: tokens [t0, t1) of a head, from a state to a state.
struct Walk {
    int b, h, p0, t0, t1, chunks;
};

// What a walk gives: y and the last state; LOCAL: a segment's own state (the rows of v; from zero, the first segment from the
// initial state) and, but for the first, its transition (from the unit matrix, v = 0); STATES: for the gradients, the state before every chunk and U.
enum Mode { Y, LOCAL_STATE, STATES };
template <int IO, int NN, int MODE>
__device__ __forceinline__ void walk(const DeltaParams &p, int block) {
    constexpr bool BF16 = IO == IO_BF16, LOCAL = MODE == LOCAL_STATE;
    using SM = Smem<NN>;
    using TM = Tm<NN>;
    extern __shared__ __align__(1024) unsigned char sm[];
    __shared__ __align__(8) uint64_t bar_mem[kBars];
    __shared__ uint32_t tmem_slot;
    // fp16: the state, v and what follows from them are held times a power of two for each row (for the gradients, whose sums
    // run over the rows, one for the CTA): delta_tc.cuh
    constexpr bool UNITS = !BF16;
    __shared__ float most_mem[UNITS ? 4 * 128 : 1];
    __shared__ float2 vmost_mem[UNITS ? kSlots * 128 : 1], row_mem[UNITS ? kSlots * 128 : 1], gate_mem[UNITS ? kSlots : 1];
    const uint32_t sbase = tc::smem_addr(sm), bars = tc::smem_addr(bar_mem);
    Gates *gates = reinterpret_cast<Gates *>(sm + SM::GATES);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int ptiles = (p.P + 127) / 128, tiles = ptiles + (LOCAL ? 1 : 0);
    int at = block;
    const int tile = at % tiles;
    at /= tiles;
    const int nseg = LOCAL ? p.nseg - 1 : p.nseg, seg = at % nseg;
    at /= nseg;
    Walk w;
    w.h = at % p.H, w.b = at / p.H;
    const bool unit = LOCAL && tile == ptiles;  // the transition: rows are the state's columns
    if (unit && seg == 0) return;  // nothing enters it but the initial state
    w.p0 = unit ? 0 : tile * 128;
    const int len = delta_length(p, w.b);
    w.t0 = seg * p.seg_len;
    w.t1 = min(len, w.t0 + p.seg_len);
    w.chunks = max(0, (w.t1 - w.t0 + kC - 1) / kC);
    const int bh = w.b * p.H + w.h, grp = w.h / (p.H / p.G), rows = unit ? p.N : min(128, p.P - w.p0);
    const size_t pn = (size_t)p.P * p.N, nn = (size_t)p.N * p.N;

    if (tid == 0) {
        auto init = [&](int bar, int count, uint32_t arrivals) {
            for (int i = 0; i < count; ++i) tc::mbar_init(bars + 8 * (bar + i), arrivals);
        };
        init(kFullKQ, kStages, 64), init(kEmptyKQ, kStages, 1), init(kFullV, kVStages, 32), init(kEmptyV, kVStages, 1);
        init(kFullOp, kOps, 1), init(kEmptyOp, kOps, 1), init(kD3, 2, 1), init(kD3Read, 2, kOutWarps * 32);
        init(kD4, 2, 1), init(kD4Read, 2, kOutWarps * 32), init(kD1, 3, 1), init(kUOut, 1, kChainWarps * 32);
        init(kS, 2, kChainWarps * 32), init(kR, 8, kChainWarps * 8), init(kVUnit, 1, kChainWarps * 32), init(kVMost, 2, kOutWarps * 32), init(kDrain, 1, 1);
        tc::mbar_init_fence();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(tc::smem_addr(&tmem_slot), TM::COLS);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's, so they begin at column 0
    Waits wait{bars};

    if (warp < kChainWarps) {
        // ---- the chain: thread = row of the state, a quarter of its columns, 16 of the 64 tokens
        const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        constexpr int CW = NN / 4;
        float2 S[CW / 2];
        {
            const float *src = nullptr;
            if (!LOCAL && seg > 0) src = p.seg_states + ((size_t)bh * p.nseg + seg) * pn + (size_t)w.p0 * p.N;
            else if (seg == 0 && p.h0) src = p.h0 + bh * pn + (size_t)w.p0 * p.N;
#pragma unroll
            for (int j = 0; j < CW / 4; ++j) {
                const int n = part * CW + 4 * j;
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (src && row < rows && n < p.N) f = *reinterpret_cast<const float4 *>(src + (size_t)row * p.N + n);
                if (unit && row < p.N && (row & ~3) == n) f = make_float4(row == n, row == n + 1, row == n + 2, row == n + 3);
                S[2 * j] = make_float2(f.x, f.y), S[2 * j + 1] = make_float2(f.z, f.w);
            }
        }
        const uint32_t x1 = tl + TM::X1 + 16 * part, x2 = tl + TM::X2 + 16 * part;
        // v as this warp scales it: eight rows of its quarter, a lane to a token (and the one 32 on)
        const int group = 4 * quarter + part;
        unsigned char *vat = sm + SM::V + (lane >> 3) * 2048 + group * 128 + (lane & 7) * 16;
        float down = 1.f;
#pragma unroll 1
        for (int c = 0;; ++c) {
            const uint32_t par = c & 1;
            if (UNITS && c < w.chunks) wait.on(kVMost + par, (c >> 1) & 1);
            if (c > 0) {
                wait.on(kDS, par ^ 1);
                tc::fence_after_sync();
            }
            const float2 over = dup(c > 0 ? gates[(c - 1) % kSlots].over : 1.f);
            const float2 back = dup(down);
            auto send = [&](int j, float up) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) split2<BF16>(UNITS ? __fmul2_rn(dup(up), S[8 * j + i]) : S[8 * j + i], hi[i], lo[i]);
                tc::tmem_st8(tl + TM::S + part * CW + 8 * j, hi);
                tc::tmem_st8(tl + TM::S + part * CW + CW / 2 + 8 * j, lo);
                tc::tmem_wait_st();
                tc::fence_before_sync();
                tc::mbar_arrive(bars + 8 * (kS + j));
                if (MODE == STATES)
                    store_op(state_op<NN>(p.states, (size_t)bh * p.nc + c, ptiles, w.p0 + row) + (part * CW / 8 + 2 * j) * 128, hi, lo, NN * 16);
            };
            // the state after the chunk before, by 16 columns, and each of them as an operand: the product with k
            // begins with the first
#pragma unroll
            for (int j = 0; j < CW / 16; ++j) {
                if (c > 0) {
                    float v[16];
                    tc::tmem_ld16(tl + TM::DS + part * CW + 16 * j, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 ds = make_float2(v[2 * i], v[2 * i + 1]);
                        S[8 * j + i] = __ffma2_rn(over, S[8 * j + i], UNITS ? __fmul2_rn(back, ds) : ds);
                    }
                }
                if (!UNITS && c < w.chunks) send(j, 1.f);
            }
            if (c >= w.chunks) break;
            float s_up = 1.f, u_up = 1.f, ds_up = 1.f, b_unit = 1.f;  // what S, then v and U over beta, then U for the state are held times
            if constexpr (UNITS) {
                const Gates &gt = gates[c % kSlots];
                float2 v = vmost_mem[(c % kSlots) * 128 + row];
                const float2 g2 = gate_mem[c % kSlots];  // the largest beta's power of two; what S |k| counts times beside v
                b_unit = g2.x;
                float most = largest(S);
                if (MODE == STATES) {
                    most = warp_largest(most), v = make_float2(warp_largest(v.x), warp_largest(v.y));
                    if (lane == 0) most_mem[warp] = most, most_mem[16 + warp] = v.x, most_mem[32 + warp] = v.y;
                    __syncwarp();
                    tc::named_barrier(1, kChainWarps * 32);
                    const float *x = most_mem + (lane & 15);
                    most = warp_largest(x[0]), v = make_float2(warp_largest(x[16]), warp_largest(x[32]));
                } else {
                    most_mem[part * 128 + row] = most;
                    __syncwarp();
                    tc::named_barrier(1 + quarter, 128);
                    most = fmaxf(fmaxf(most_mem[row], most_mem[128 + row]), fmaxf(most_mem[256 + row], most_mem[384 + row]));
                }
                s_up = to_unit(most) * kUp;
                u_up = to_unit(fmaxf(finite_or_zero(most * g2.y), v.x)) * room(gt);
                ds_up = to_unit(fmaxf(finite_or_zero(v.y), finite_or_zero(most * gt.over * gt.k_len4))) * room(gt);
                down = inverse_power(ds_up);
                if (MODE == Y && part == 0)  // from S's scale to that of M U, and from there to y
                    row_mem[(c % kSlots) * 128 + row] = make_float2(u_up * inverse_power(s_up) * inverse_power(b_unit) * inverse_power(gt.m_unit),
                                                                    inverse_power(u_up) * b_unit * gt.m_unit);
                if (MODE == STATES && tid == 0)
                    *reinterpret_cast<float2 *>(p.units + (((size_t)bh * p.nc + c) * ptiles + tile) * 4) = make_float2(s_up, u_up);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < CW / 16; ++j) send(j, s_up);
                const uint4 vw[2] = {*reinterpret_cast<const uint4 *>(vat + (c % kVStages) * SM::V_BYTES),
                                     *reinterpret_cast<const uint4 *>(vat + (c % kVStages) * SM::V_BYTES + 4 * 2048)};
                uint32_t two[8] = {vw[0].x, vw[0].y, vw[0].z, vw[0].w, vw[1].x, vw[1].y, vw[1].z, vw[1].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // the units of rows 2 i and 2 i + 1 of the eight lie with the lanes that have these rows
                    const float2 by = MODE == STATES ? dup(u_up) : make_float2(__shfl_sync(0xffffffffu, u_up, 8 * part + 2 * i),
                                                                               __shfl_sync(0xffffffffu, u_up, 8 * part + 2 * i + 1));
#pragma unroll
                    for (int m = i; m < 8; m += 4) {
                        const float2 f = __fmul2_rn(by, unpack2<BF16>(two[m]));
                        two[m] = tcop::pack2(f.x, f.y, BF16);
                    }
                }
                *reinterpret_cast<uint4 *>(vat + (c % kVStages) * SM::V_BYTES) = make_uint4(two[0], two[1], two[2], two[3]);
                *reinterpret_cast<uint4 *>(vat + (c % kVStages) * SM::V_BYTES + 4 * 2048) = make_uint4(two[4], two[5], two[6], two[7]);
                tc::fence_smem_to_async();
                tc::mbar_arrive(bars + 8 * kVUnit);
            }
            const Gates &gt = gates[c % kSlots];
            wait.on(kFullOp + par, (c >> 1) & 1);  // the gates
            wait.on(kD1, par);
            tc::fence_after_sync();
            float v[16];
            tc::tmem_ld16(x1, v);
            split_scaled<BF16>(v, &gt.neg_into[16 * part], x1, UNITS ? u_up * inverse_power(s_up) : 1.f);  // -exp(G) S k^T
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(bars + 8 * (kR + part));
            wait.on(kD2, par);
            tc::fence_after_sync();
            tc::tmem_ld16(x2, v);
            if constexpr (UNITS) {
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] *= gt.t_unit;
            }
            split_scaled<BF16>(v, &gt.out[16 * part], x1, UNITS ? ds_up * inverse_power(u_up) * b_unit : 1.f);  // what U adds to the state
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(bars + 8 * (kU + part));
            if (MODE != LOCAL_STATE) {  // U itself, for y or the gradients
                const float bad = wait.dead() ? __int_as_float(0x7fffffff) : 0.f;
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) split2<BF16>(make_float2(v[2 * i] + bad, v[2 * i + 1] + bad), hi[i], lo[i]);
                if (MODE == STATES) {
                    store_op(token_op(p.u, (size_t)bh * p.nc + c, ptiles, w.p0 + row) + 2 * part * 128, hi, lo, 1024);
                    continue;
                }
                tc::tmem_st8(x2, hi);
                tc::tmem_st8(x2 + 8, lo);
                tc::tmem_wait_st();
                tc::fence_before_sync();
                tc::mbar_arrive(bars + 8 * kUOut);
            }
        }
        float *dst = nullptr;
        if (unit) dst = p.seg_trans + ((size_t)bh * nseg + seg) * nn;
        else if (LOCAL) dst = p.seg_states + ((size_t)bh * p.nseg + seg + 1) * pn + (size_t)w.p0 * p.N;
        else if (p.final_state && ((w.t0 < len && len <= w.t0 + p.seg_len) || (len == 0 && seg == 0)))
            dst = p.final_state + bh * pn + (size_t)w.p0 * p.N;
        if (dst && row < rows) {
            const float nan = __int_as_float(0x7fffffff);
#pragma unroll
            for (int j = 0; j < CW / 4; ++j) {
                const int n = part * CW + 4 * j;
                float4 f = make_float4(S[2 * j].x, S[2 * j].y, S[2 * j + 1].x, S[2 * j + 1].y);
                if (wait.dead()) f = make_float4(nan, nan, nan, nan);
                if (n < p.N) *reinterpret_cast<float4 *>(dst + (size_t)row * p.N + n) = f;
            }
        }
    } else if (warp < kMmaWarp) {
        // ---- y: thread = row of the state.  In fp16 also, two chunks ahead, the largest of v in every row
        auto look = [&](int c) {
            const Gates &gt = gates[c % kSlots];
            wait.on(kFullOp + (c & 1), (c >> 1) & 1);
            wait.on(kFullV + c % kVStages, (c / kVStages) & 1);
            const float fa = fabsf(gt.out[lane] * gt.beta[lane]), fb = fabsf(gt.out[lane + 32] * gt.beta[lane + 32]);
            const unsigned char *at = sm + SM::V + (c % kVStages) * SM::V_BYTES + (lane >> 3) * 2048 + (lane & 7) * 16;
#pragma unroll 1
            for (int group = 4 * (warp - kOutWarp0); group < 4 * (warp - kOutWarp0) + 4; ++group) {
                const float2 most = largest_of_rows(*reinterpret_cast<const uint4 *>(at + group * 128),
                                                    *reinterpret_cast<const uint4 *>(at + group * 128 + 4 * 2048), fa, fb, lane);
                if ((lane & 3) == 0) vmost_mem[(c % kSlots) * 128 + 8 * group + (lane >> 2)] = most;
                __syncwarp();
            }
            const float into = warp_largest(fmaxf(finite_or_zero(gt.into[lane]), finite_or_zero(gt.into[lane + 32]))), b_unit = beta_unit(gt, lane);
            if (warp == kOutWarp0 && lane == 0) gate_mem[c % kSlots] = make_float2(b_unit, gt.k_len4 * into);
            __syncwarp();
            if (!wait.dead()) tc::mbar_arrive(bars + 8 * (kVMost + (c & 1)));  // two: the chain may be two chunks behind
        };
        if constexpr (UNITS)
#pragma unroll 1
            for (int c = 0; c < (MODE == Y ? min(2, w.chunks) : w.chunks); ++c) look(c);
        if (MODE == Y) {
            const int quarter = warp - kOutWarp0, row = quarter * 32 + lane;
            const bool ok = row < rows;
            const size_t step = (size_t)p.H * p.P;
            const size_t base = ((size_t)w.b * p.L * p.H + w.h) * p.P + w.p0 + row;
            const int odd = lane & 1;
            uint16_t *y = static_cast<uint16_t *>(p.y) + base - odd + odd * step;  // of an odd lane: the token after, from the row before
#pragma unroll 1
            for (int c = 0; c < w.chunks; ++c) {
                const uint32_t par = (c >> 1) & 1, o = c & 1, tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + TM::O + 64 * o;
                const Gates &gt = gates[c % kSlots];
                wait.on(kD3 + o, par);
                tc::fence_after_sync();
                float up = 1.f;  // from S's scale to that of M U
                if (UNITS) up = row_mem[(c % kSlots) * 128 + row].x;
#pragma unroll 1
                for (int j = 0; j < kC; j += 16) {  // diag(exp G) Q S^T, onto which M U is summed
                    float v[16];
                    uint32_t r[16];
                    tc::tmem_ld16(tl + j, v);
#pragma unroll
                    for (int m = 0; m < 16; m += 4) {
                        float4 f = *reinterpret_cast<const float4 *>(&gt.into[j + m]);
                        if (UNITS) f.x *= up, f.y *= up, f.z *= up, f.w *= up;
                        r[m] = __float_as_uint(v[m] * f.x), r[m + 1] = __float_as_uint(v[m + 1] * f.y);
                        r[m + 2] = __float_as_uint(v[m + 2] * f.z), r[m + 3] = __float_as_uint(v[m + 3] * f.w);
                    }
                    tc::tmem_st16(tl + j, r);
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                tc::mbar_arrive(bars + 8 * (kD3Read + o));
                wait.on(kD4 + o, par);
                tc::fence_after_sync();
                const int tc0 = w.t0 + c * kC, n = min(kC, w.t1 - tc0);
                float scale = wait.dead() ? __int_as_float(0x7fffffff) : p.scale;
                if (UNITS) scale *= row_mem[(c % kSlots) * 128 + row].y;
                uint16_t *to = y + (size_t)tc0 * step;
#pragma unroll 1
                for (int j = 0; j < kC; j += 16) {
                    float v[16];
                    tc::tmem_ld16(tl + j, v);
                    // neighbouring lanes exchange: each then has two rows of every second token, a store of 4 bytes
#pragma unroll
                    for (int m = 0; m < 16; m += 2, to += 2 * step) {
                        const uint32_t two = exchange_rows<BF16>(scale * v[m], scale * v[m + 1], odd);
                        if (ok && j + m + odd < n) *reinterpret_cast<uint32_t *>(to) = two;
                    }
                }
                __syncwarp();
                tc::fence_before_sync();
                tc::mbar_arrive(bars + 8 * (kD4Read + o));
                if (UNITS && c + 2 < w.chunks) look(c + 2);
            }
            const int end = min(p.L, w.t0 + p.seg_len);
            if (ok)
                for (int t = max(w.t1, w.t0); t < end; ++t) st_io<IO>(p.y, base + (size_t)t * step, 0.f);
        }
    } else if (warp == kMmaWarp) {
        // ---- the products.  The warp stays together and one elected lane issues: the descriptors
        // are then the warp's, not a thread's, and a product costs a few instructions in place of
        // a dozen (measured beside busy warps: 16 products 540 to 2100 cycles, from a lane's branch 830 to 15000)
        const bool go = tc::elect_one();
        constexpr uint32_t ID = tc::idesc_f16(128, kC, BF16, false, false), ID_V = tc::idesc_f16(128, kC, BF16, true, false),
                           ID_DS = tc::idesc_f16(128, NN, BF16, false, true);
        constexpr int NK = NN / 16, J = NN / 64;  // steps of 16 along a state's columns; of a thread's part of them
        constexpr uint32_t K2 = 2 * 128 * 16 / 16;  // of a descriptor: from one step of 16 columns of k, q or v to the next
        constexpr uint32_t LO = kOpTerm / 16;       // to an operand's second terms
        auto s_term = [&](int k) { return tmem + TM::S + (k / J) * (NN / 4) + (k % J) * 8; };  // second term NN / 8 on
        auto x_term = [&](uint32_t x, int k) { return tmem + x + k * 16; };                     // second term 8 on
#pragma unroll 1
        for (int c = 0; c < w.chunks; ++c) {
            const uint32_t par = c & 1, par2 = (c >> 1) & 1, o = TM::O + 64 * par;
            const uint32_t kq = sbase + SM::KQ + (c % kStages) * SM::KQ_BYTES, op = sbase + SM::OP + par * kOpGates;
            const uint64_t kd = tc::desc(kq, 2048, 128), td = tc::desc(op + kOpT, 1024, 128);
            wait.on(kFullKQ + c % kStages, (c / kStages) & 1);
#pragma unroll
            for (int j = 0; j < J; ++j) {  // S k^T, as the state's columns come
                wait.on(kS + j, par);
                if (wait.dead()) goto given_up;
                tc::fence_after_sync();
                if (go) {
#pragma unroll
                    for (int k = j; k < NK; k += J) {
                        tc::mma_f16_ts(tmem + TM::X1, s_term(k), kd + k * K2, ID, k > 0);
                        tc::mma_f16_ts(tmem + TM::X1, s_term(k) + NN / 8, kd + k * K2, ID, 1);
                    }
                }
            }
            if (go) tc::commit(bars + 8 * kD1);
            wait.on(kFullOp + par, par2);
            if (UNITS) wait.on(kVUnit, par);
            else wait.on(kFullV + c % kVStages, (c / kVStages) & 1);
            if (wait.dead()) goto given_up;
            tc::fence_after_sync();
            if (go) {
                if (!unit) {
                    const uint64_t vd = tc::desc(sbase + SM::V + (c % kVStages) * SM::V_BYTES, 2048, 128);
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k) {  // v^T (T diag(beta))^T
                        tc::mma_f16(tmem + TM::X2, vd + k * K2, td + k * 128, ID_V, k > 0);
                        tc::mma_f16(tmem + TM::X2, vd + k * K2, td + LO + k * 128, ID_V, 1);
                    }
                }
                tc::commit(bars + 8 * (kEmptyV + c % kVStages));
            }
#pragma unroll
            for (int k = 0; k < kC / 16; ++k) {  // - (exp(G) S k^T) (T diag(beta))^T
                wait.on(kR + k, par);
                if (wait.dead()) goto given_up;
                tc::fence_after_sync();
                if (go) {
                    tc::mma_f16_ts(tmem + TM::X2, x_term(TM::X1, k), td + k * 128, ID, !unit || k > 0);
                    tc::mma_f16_ts(tmem + TM::X2, x_term(TM::X1, k), td + LO + k * 128, ID, 1);
                    tc::mma_f16_ts(tmem + TM::X2, x_term(TM::X1, k) + 8, td + k * 128, ID, 1);
                }
            }
            if (go) tc::commit(bars + 8 * kD2);
            if (MODE == Y) {  // while the chain splits U
                wait.on(kD4Read + par, par2 ^ 1);
                if (wait.dead()) goto given_up;
                tc::fence_after_sync();
                if (go) {
#pragma unroll
                    for (int k = 0; k < NK; ++k) {  // S q^T
                        tc::mma_f16_ts(tmem + o, s_term(k), kd + 64 + k * K2, ID, k > 0);
                        tc::mma_f16_ts(tmem + o, s_term(k) + NN / 8, kd + 64 + k * K2, ID, 1);
                    }
                    tc::commit(bars + 8 * (kD3 + par));
                }
            }
            const uint64_t kt = tc::desc(kq, 128, 2048);
#pragma unroll
            for (int k = 0; k < kC / 16; ++k) {  // the change of the state
                wait.on(kU + k, par);
                if (wait.dead()) goto given_up;
                tc::fence_after_sync();
                if (go) {
                    tc::mma_f16_ts(tmem + TM::DS, x_term(TM::X1, k), kt + k * 16, ID_DS, k > 0);
                    tc::mma_f16_ts(tmem + TM::DS, x_term(TM::X1, k) + 8, kt + k * 16, ID_DS, 1);
                }
            }
            if (go) {
                tc::commit(bars + 8 * kDS);
                tc::commit(bars + 8 * (kEmptyKQ + c % kStages));
            }
            if (MODE == Y) {
                wait.on(kUOut, par);
                wait.on(kD3Read + par, par2);
                if (wait.dead()) goto given_up;
                tc::fence_after_sync();
                if (go) {
                    const uint64_t md = tc::desc(op + kOpM, 1024, 128);
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k) {  // U^T M^T
                        tc::mma_f16_ts(tmem + o, x_term(TM::X2, k), md + k * 128, ID, 1);
                        tc::mma_f16_ts(tmem + o, x_term(TM::X2, k), md + LO + k * 128, ID, 1);
                        tc::mma_f16_ts(tmem + o, x_term(TM::X2, k) + 8, md + k * 128, ID, 1);
                    }
                    tc::commit(bars + 8 * (kD4 + par));
                }
            }
            if (go) tc::commit(bars + 8 * (kEmptyOp + par));
        }
    given_up:
        // the last products may still read shared memory: wait for them before the CTA ends
        if (go) tc::commit(bars + 8 * kDrain);
        Waits{bars}.on(kDrain, 0);
    } else {
        // ---- copies: lane = row of eight, 16-byte piece of four.  The first warp takes k, the second q, the third v and a chunk's operands
        const int r = lane & 7, piece = lane >> 3, which = warp - kLoadWarp;
        const void *src = which == 0 ? p.k : which == 1 ? p.q : p.v;
        const long long s0 = which == 0 ? p.ks[0] : which == 1 ? p.qs[0] : p.vs[0], s1 = which == 0 ? p.ks[1] : which == 1 ? p.qs[1] : p.vs[1];
        const char *from = static_cast<const char *>(src) + 2 * (w.b * s0 + (which < 2 ? (long long)grp * p.N : (long long)w.h * p.P + w.p0) + 8 * piece);
        // of a row of 16-byte pieces, those that exist from this lane's on; none of q in a walk without y, nor of v in a transition's
        const int width = (which == 1 && MODE != Y) || (which == 2 && unit) ? 0 : (which < 2 ? p.N : rows) - 8 * piece;
        const uint32_t to = sbase + (which < 2 ? SM::KQ + which * 1024 + piece * 2048 : SM::V + piece * 128) + r * 16;
        const uint32_t stage = which < 2 ? SM::KQ_BYTES : SM::V_BYTES, row_step = which < 2 ? 128 : 2048, col_step = which < 2 ? 8192 : 512;
        const int stages = which < 2 ? kStages : kVStages, empty = which < 2 ? kEmptyKQ : kEmptyV, full = which < 2 ? kFullKQ : kFullV;
        int at = 0, issued = 0;
        uint32_t parity = 1;
        const unsigned char *ops = p.ops + ((size_t)bh * p.nc + w.t0 / kC) * op_bytes(MODE == STATES);
#pragma unroll 1
        for (int c = 0; c < w.chunks; ++c) {
            if (which == 2) {  // with a place of T's, the gates four chunks back are done with too
                wait.on(kEmptyOp + (c & 1), ((c >> 1) & 1) ^ 1);
                if (wait.dead()) break;
                if (lane == 0) {
                    const uint32_t bar = bars + 8 * (kFullOp + (c & 1));
                    constexpr uint32_t bytes = MODE == Y ? kOpGates : kOpM;  // T and M, or T alone
                    const unsigned char *op = ops + (size_t)c * op_bytes(MODE == STATES);
                    tc::mbar_arrive_expect_tx(bar, bytes + (uint32_t)sizeof(Gates));
                    bulk_load(sbase + SM::OP + (c & 1) * kOpGates, op, bytes, bar);
                    bulk_load(sbase + SM::GATES + (c % kSlots) * (uint32_t)sizeof(Gates), op + kOpGates, (uint32_t)sizeof(Gates), bar);
                }
                __syncwarp();
                issued = c + 1;
            }
            wait.on(empty + at, parity);
            if (wait.dead()) break;
            const char *row = from + 2 * ((w.t0 + c * kC + r) * s1);
            uint32_t dst = to + at * stage;
#pragma unroll 1
            for (int rg = 0; rg < 8; ++rg, row += 16 * s1, dst += row_step) {
                const int live = w.t0 + c * kC + rg * 8 + r < w.t1 ? width : 0;
#pragma unroll
                for (int cg = 0; cg < 4; ++cg)
                    if (which == 2 || cg < NN / 32)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + cg * col_step),
                                     "l"(live > 32 * cg ? row + 64 * cg : nullptr), "r"(live > 32 * cg ? 16 : 0) : "memory");
            }
            cp_commit();
            cp_wait<0>();
            tc::fence_smem_to_async();
            tc::mbar_arrive(bars + 8 * (full + at));
            if (++at == stages) at = 0, parity ^= 1;
        }
        if (wait.dead())  // nobody may have waited for these
            for (int c = max(issued - kOps, 0); c < issued; ++c) Waits{bars}.on(kFullOp + (c & 1), (c >> 1) & 1);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem_slot, TM::COLS);
}

}  // namespace delta_walk
}  // namespace ssd

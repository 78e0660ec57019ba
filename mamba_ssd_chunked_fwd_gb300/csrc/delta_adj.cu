// delta_adj.cu -- the adjoint of the delta rule's state, chunk by chunk from the end, on the tensor
// cores, for 16-bit tensors: the backward counterpart of delta_walk_tc.cuh, with which
// it shares a launch.
//
// With D the adjoint of the state after a chunk, d = scale dy, and T, M and the gates of delta_prep.cu:
//
//     dU = M^T d + diag(exp(G_end - G)) K D^T
//     R  = T^T dU                                     (the gradient of v - S' k over beta)
//     D <- exp(G_end) D + (diag(exp G) d)^T Q - (diag(beta exp G) R)^T K
//
// and dv = beta R.  The layout is that of the forward walk (delta_walk_tc.cuh): rows of the state in TMEM's lanes, tokens
// along its columns, computed operands in two terms; the chain is D K^T -> dU -> R -> D:
//
//   16 warps the chain;  4 warps make an operand of d;  1 warp issues the products
//   3 warps  copy k, q, and dy with a chunk's operands ahead
//
// Bound by what it stores, 112 KB of D, R and dv to a chunk and SM, beside the chain: [4,2048] with 16 heads of 128 x 128, bf16,
// 193 us with the states' walk on the other SMs.  The stores of D, or of D and R, by the side warps from TMEM in place of
// the chain's took 7 and 14 us longer.  In fp16, with the powers of two of the operands (the largest D, d and M^T d of the
// CTA's rows by a barrier of the chain's warps, for which the side warps wait; the largest dU of a row over four threads), 269 us.
//
// It leaves D after every chunk and R as operands for delta_grad_tc.cu, and writes dv.
#include "delta_walk_tc.cuh"

namespace ssd {

namespace {

constexpr int kChainWarps = 16, kSideWarps = 4, kSideWarp0 = kChainWarps, kMmaWarp = kSideWarp0 + kSideWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = (kLoadWarp + 3) * 32;
constexpr int kStages = 3;   // of k and q
constexpr int kVStages = 2;  // of dy
constexpr int kOps = 2;      // of a chunk's operands
constexpr int kSlots = 4;    // of its gates

template <int NN>
struct Smem {
    static constexpr uint32_t KQ = 0, KQ_BYTES = 128 * NN * 2;  // rows 0-63 k, 64-127 q
    static constexpr uint32_t DY = KQ + kStages * KQ_BYTES, DY_BYTES = kC * 128 * 2;
    static constexpr uint32_t OP = DY + kVStages * DY_BYTES;  // M, T
    static constexpr uint32_t GATES = OP + kOps * 32768, BYTES = GATES + kSlots * (uint32_t)sizeof(Gates);
};

enum Bar { kFullKQ = 0, kEmptyKQ = kFullKQ + kStages, kFullV = kEmptyKQ + kStages, kEmptyV = kFullV + kVStages, kFullOp = kEmptyV + kVStages,
           kEmptyOp = kFullOp + kOps, kD1 = kEmptyOp + kOps, kD2, kDS, kDFree, kX2, kUnit, kDReady, kS, kR = kS + 2, kU = kR + 4, kDrain = kU + 4, kBars };

// TMEM columns: D's operand, D K^T and then the operands dU and R, M^T d, R, the change of D, d's operand.
template <int NN>
struct Tm {
    static constexpr uint32_t S = 0, X1 = NN, X2 = NN + 64, X3 = NN + 128, DS = NN + 192, XD = 2 * NN + 192, COLS = 512;
};

template <int IO, int NN>
__device__ __forceinline__ void adjoint(const DeltaParams &p, int block) {
    constexpr bool BF16 = IO == IO_BF16;
    using SM = Smem<NN>;
    using TM = Tm<NN>;
    extern __shared__ __align__(1024) unsigned char sm[];
    __shared__ __align__(8) uint64_t bar_mem[kBars];
    __shared__ uint32_t tmem_slot;
    // fp16: D, d and what follows from them are held times a power of two (delta_tc.cuh)
    constexpr bool UNITS = !BF16;
    __shared__ float most_mem[UNITS ? 3 * kChainWarps : 1], row_mem[UNITS ? 4 * 128 : 1], unit_mem[UNITS ? kSlots : 1];
    const uint32_t sbase = tc::smem_addr(sm), bars = tc::smem_addr(bar_mem);
    Gates *gates = reinterpret_cast<Gates *>(sm + SM::GATES);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tiles = (p.P + 127) / 128, p0 = (block % tiles) * 128, bh = block / tiles, h = bh % p.H, b = bh / p.H;
    const int len = delta_length(p, b), chunks = (len + kC - 1) / kC, grp = h / (p.H / p.G), rows = min(128, p.P - p0);
    const size_t pn = (size_t)p.P * p.N;

    if (tid == 0) {
        auto init = [&](int bar, int count, uint32_t arrivals) {
            for (int i = 0; i < count; ++i) tc::mbar_init(bars + 8 * (bar + i), arrivals);
        };
        init(kFullKQ, kStages, 64), init(kEmptyKQ, kStages, 1), init(kFullV, kVStages, 32), init(kEmptyV, kVStages, 1 + kSideWarps * 32);
        init(kFullOp, kOps, 1), init(kEmptyOp, kOps, 1), init(kD1, 6, 1), init(kDReady, 1, kSideWarps * 32);
        init(kS, 2, kChainWarps * 32), init(kR, 8, kChainWarps * 8), init(kDrain, 1, 1);
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

    // i counts the chunks as they are walked; the chunk is chunks - 1 - i
    if (warp < kChainWarps) {
        // ---- the chain: thread = row of the state, a quarter of its columns, 16 of the 64 tokens
        const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane, odd = lane & 1;
        const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        constexpr int CW = NN / 4;
        const bool ok = row < rows;
        float2 D[CW / 2];
#pragma unroll
        for (int j = 0; j < CW / 4; ++j) {
            const int n = part * CW + 4 * j;
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.dfinal && ok && n < p.N) f = *reinterpret_cast<const float4 *>(p.dfinal + bh * pn + (size_t)(p0 + row) * p.N + n);
            D[2 * j] = make_float2(f.x, f.y), D[2 * j + 1] = make_float2(f.z, f.w);
        }
        const uint32_t x1 = tl + TM::X1 + 16 * part, x2 = tl + TM::X2 + 16 * part, x3 = tl + TM::X3 + 16 * part;
        const size_t step = (size_t)p.H * p.P;
        uint16_t *dv = static_cast<uint16_t *>(p.dv) + ((size_t)b * p.L * p.H + h) * p.P + p0 + row - odd + odd * step;
        auto store_rows = [&](float *dst) {
            if (!ok) return;
            dst += (size_t)(p0 + row) * p.N + part * CW;
            const float bad = wait.dead() ? __int_as_float(0x7fffffff) : 0.f;
#pragma unroll
            for (int j = 0; j < CW / 4; ++j)
                if (part * CW + 4 * j < p.N)
                    *reinterpret_cast<float4 *>(dst + 4 * j) = make_float4(D[2 * j].x + bad, D[2 * j].y + bad, D[2 * j + 1].x + bad, D[2 * j + 1].y + bad);
        };
        float down = 1.f;
#pragma unroll 1
        for (int i = 0;; ++i) {
            const uint32_t par = i & 1;
            float dmost = 0.f;
            if constexpr (UNITS) {
                if (i < chunks) {  // the largest of exp(G) d, eight rows of two neighbouring tokens to a thread
                    const Gates &gt = gates[i % kSlots];
                    wait.on(kFullOp + par, (i >> 1) & 1);
                    wait.on(kFullV + i % kVStages, (i / kVStages) & 1);
                    const uint4 *at = reinterpret_cast<const uint4 *>(sm + SM::DY + (i % kVStages) * SM::DY_BYTES) + 2 * tid;
                    const uint4 a = at[0], e = at[1];
                    const uint32_t dw[8] = {a.x, a.y, a.z, a.w, e.x, e.y, e.z, e.w};
                    __half2 most[2] = {__float2half2_rn(0.f), __float2half2_rn(0.f)};
#pragma unroll
                    for (int m = 0; m < 8; ++m) most[m >> 2] = larger_of_halves(most[m >> 2], dw[m]);
                    const float2 into = *reinterpret_cast<const float2 *>(&gt.into[8 * (tid >> 6) + ((2 * tid) & 7)]);
                    dmost = finite_or_zero(fabsf(p.scale) * fmaxf(into.x * larger_half(most[0]), into.y * larger_half(most[1])));
                }
            }
            if (i > 0) {
                wait.on(kDS, par ^ 1);
                tc::fence_after_sync();
            }
            const float2 over = dup(i > 0 ? gates[(i - 1) % kSlots].over : 1.f);
            auto send = [&](int j, float up) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) split2<BF16>(UNITS ? __fmul2_rn(dup(up), D[8 * j + e]) : D[8 * j + e], hi[e], lo[e]);
                tc::tmem_st8(tl + TM::S + part * CW + 8 * j, hi);
                tc::tmem_st8(tl + TM::S + part * CW + CW / 2 + 8 * j, lo);
                tc::tmem_wait_st();
                tc::fence_before_sync();
                tc::mbar_arrive(bars + 8 * (kS + j));
                store_op(state_op<NN>(p.adj, (size_t)bh * p.nc + chunks - 1 - i, tiles, p0 + row) + (part * CW / 8 + 2 * j) * 128, hi, lo, NN * 16);
            };
#pragma unroll
            for (int j = 0; j < CW / 16; ++j) {
                if (i > 0) {
                    float v[16];
                    tc::tmem_ld16(tl + TM::DS + part * CW + 16 * j, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 ds = make_float2(v[2 * e], v[2 * e + 1]);
                        D[8 * j + e] = __ffma2_rn(over, D[8 * j + e], UNITS ? __fmul2_rn(dup(down), ds) : ds);
                    }
                }
                if (!UNITS && i < chunks) send(j, 1.f);
            }
            if (i >= chunks) break;
            const int c = chunks - 1 - i;
            const Gates &gt = gates[i % kSlots];
            wait.on(kFullOp + par, (i >> 1) & 1);  // the gates
            float r_up = 1.f, d_up = 1.f, ds_up = 1.f;  // what R, D, and what is summed onto D are held times
            if constexpr (UNITS) {
                float v[16], most = 0.f, wmost = 0.f, x = largest(D);
                wait.on(kX2, par);
                tc::fence_after_sync();
                tc::tmem_ld16(x2, v);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    most = fmaxf(most, fabsf(v[e]));
                    wmost = fmaxf(wmost, gt.into[16 * part + e] * fabsf(v[e]));
                }
                const float by = fabsf(p.scale) * gt.m_unit;
                most = warp_largest(fmaxf(finite_or_zero(most * by), finite_or_zero(x * gt.k_len4)));
                wmost = warp_largest(fmaxf(fmaxf(finite_or_zero(wmost * by), finite_or_zero(gt.over * x * gt.k_len4)), dmost));
                x = warp_largest(x);
                if (lane == 0) most_mem[warp] = most, most_mem[kChainWarps + warp] = wmost, most_mem[2 * kChainWarps + warp] = x;
                __syncwarp();
                tc::named_barrier(1, kChainWarps * 32);
                const float *at = most_mem + (lane & 15);
                r_up = to_unit(warp_largest(at[0])) * room(gt), ds_up = to_unit(warp_largest(at[kChainWarps])) * room(gt), d_up = to_unit(warp_largest(at[2 * kChainWarps])) * kUp;
                down = inverse_power(ds_up);
                if (tid == 0) {
                    unit_mem[i % kSlots] = ds_up;
                    *reinterpret_cast<float2 *>(p.units + (((size_t)bh * p.nc + c) * tiles + p0 / 128) * 4 + 2) = make_float2(d_up, r_up);
                    tc::mbar_arrive(bars + 8 * kUnit);
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < CW / 16; ++j) send(j, d_up);
            }
            wait.on(kD1, par);
            tc::fence_after_sync();
            float v[16], of_row = 1.f;  // (fp16) what of a row's R comes out of the product
            {
                float u[16];
                uint32_t hi[8], lo[8];
                tc::tmem_ld16x2(x1, x2, v, u);
                const float2 s2 = dup(UNITS ? p.scale * gt.m_unit : p.scale);
                const float d_down = UNITS ? inverse_power(d_up) : 1.f;
                float2 du[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float4 f = *reinterpret_cast<const float4 *>(&gt.out[16 * part + 4 * e]);
                    if (UNITS) f.x *= d_down, f.y *= d_down, f.z *= d_down, f.w *= d_down;
                    du[2 * e] = __ffma2_rn(s2, make_float2(u[4 * e], u[4 * e + 1]), __fmul2_rn(make_float2(v[4 * e], v[4 * e + 1]), make_float2(f.x, f.y)));
                    du[2 * e + 1] = __ffma2_rn(s2, make_float2(u[4 * e + 2], u[4 * e + 3]), __fmul2_rn(make_float2(v[4 * e + 2], v[4 * e + 3]), make_float2(f.z, f.w)));
                }
                float up = 1.f;
                if constexpr (UNITS) {
                    row_mem[part * 128 + row] = largest(du);
                    __syncwarp();
                    tc::named_barrier(2 + quarter, 128);
                    up = to_unit(fmaxf(fmaxf(row_mem[row], row_mem[128 + row]), fmaxf(row_mem[256 + row], row_mem[384 + row]))) * kUp;
                    of_row = inverse_power(up) * gt.t_unit;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) split2<BF16>(UNITS ? __fmul2_rn(dup(up), du[e]) : du[e], hi[e], lo[e]);
                tc::tmem_st8(x1, hi);
                tc::tmem_st8(x1 + 8, lo);
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(bars + 8 * (kR + part));
            wait.on(kD2, par);
            tc::fence_after_sync();
            tc::tmem_ld16(x3, v);
            {
                uint32_t hi[8], lo[8];
                const float by = UNITS ? ds_up * of_row : 1.f;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    float4 b4 = *reinterpret_cast<const float4 *>(&gt.beta[16 * part + e]);
                    if (UNITS) b4.x *= by, b4.y *= by, b4.z *= by, b4.w *= by;
                    const float4 n4 = *reinterpret_cast<const float4 *>(&gt.neg_into[16 * part + e]);
                    split2<BF16>(__fmul2_rn(make_float2(v[e], v[e + 1]), make_float2(b4.x * n4.x, b4.y * n4.y)), hi[e / 2], lo[e / 2]);
                    split2<BF16>(__fmul2_rn(make_float2(v[e + 2], v[e + 3]), make_float2(b4.z * n4.z, b4.w * n4.w)), hi[e / 2 + 1], lo[e / 2 + 1]);
                }
                tc::tmem_st8(x1, hi);
                tc::tmem_st8(x1 + 8, lo);
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(bars + 8 * (kU + part));
            {
                const float bad = wait.dead() ? __int_as_float(0x7fffffff) : 0.f;
                const int t = c * kC + 16 * part;
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = UNITS ? v[e] * of_row : v[e];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 r = make_float2(v[2 * e] + bad, v[2 * e + 1] + bad);
                    split2<BF16>(UNITS ? __fmul2_rn(dup(r_up), r) : r, hi[e], lo[e]);
                }
                store_op(token_op(p.dr, (size_t)bh * p.nc + c, tiles, p0 + row) + 2 * part * 128, hi, lo, 1024);
                uint16_t *to = dv + (size_t)t * step;
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float2 beta = *reinterpret_cast<const float2 *>(&gt.beta[16 * part + e]);
                    const uint32_t two = exchange_rows<BF16>(beta.x * v[e] + bad, beta.y * v[e + 1] + bad, odd);
                    if (ok && t + e + odd < len) *reinterpret_cast<uint32_t *>(to + e * step) = two;
                }
            }
        }
        if (p.dh0) store_rows(p.dh0 + bh * pn);
    } else if (warp < kMmaWarp) {
        // ---- exp(G) d as an operand: thread = row of the state
        const int quarter = warp - kSideWarp0, row = quarter * 32 + lane;
        const uint32_t xd = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + TM::XD;
#pragma unroll 1
        for (int i = 0; i < chunks; ++i) {
            const Gates &gt = gates[i % kSlots];
            wait.on(kFullOp + (i & 1), (i >> 1) & 1);
            wait.on(kFullV + i % kVStages, (i / kVStages) & 1);
            wait.on(kDFree, (i & 1) ^ 1);
            float scale = p.scale;
            if constexpr (UNITS) {
                wait.on(kUnit, i & 1);
                scale *= unit_mem[i % kSlots];
            }
            if (wait.dead()) break;
            tc::fence_after_sync();
            const unsigned char *dy = sm + SM::DY + (i % kVStages) * SM::DY_BYTES + (row >> 3) * 128 + (row & 7) * 2;
#pragma unroll 1
            for (int t = 0; t < kC; t += 16) {
                float f[16];
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 g4 = *reinterpret_cast<const float4 *>(&gt.into[t + e]);
                    f[e] = g4.x, f[e + 1] = g4.y, f[e + 2] = g4.z, f[e + 3] = g4.w;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {  // token t + e: row group (t + e) / 8, its row (t + e) % 8
                    const uint16_t raw = *reinterpret_cast<const uint16_t *>(dy + ((t + e) >> 3) * 2048 + (e & 7) * 16);
                    f[e] *= scale * (BF16 ? __uint_as_float((uint32_t)raw << 16) : __half2float(__ushort_as_half(raw)));
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) split2<BF16>(make_float2(f[2 * e], f[2 * e + 1]), hi[e], lo[e]);
                tc::tmem_st8(xd + t, hi);
                tc::tmem_st8(xd + t + 8, lo);
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(bars + 8 * kDReady);
            tc::mbar_arrive(bars + 8 * (kEmptyV + i % kVStages));
        }
        // behind the row's end: zeros
        const size_t step = (size_t)p.H * p.P;
        if (row < rows)
            for (int t = len; t < p.L; ++t) st_io<IO>(p.dv, ((size_t)b * p.L + t) * step + (size_t)h * p.P + p0 + row, 0.f);
    } else if (warp == kMmaWarp) {
        // ---- the products, by an elected lane (see delta_walk_tc.cuh)
        const bool go = tc::elect_one();
        constexpr uint32_t ID = tc::idesc_f16(128, kC, BF16, false, false), ID_B = tc::idesc_f16(128, kC, BF16, false, true),
                           ID_M = tc::idesc_f16(128, kC, BF16, true, true), ID_DS = tc::idesc_f16(128, NN, BF16, false, true);
        constexpr int NK = NN / 16, J = NN / 64;    // steps of 16 along a state's columns; of a thread's part of them
        constexpr uint32_t K2 = 2 * 128 * 16 / 16;  // of a descriptor: from one step of 16 columns of k, q or dy to the next
        constexpr uint32_t LO = kOpTerm / 16;       // to an operand's second terms
        auto s_term = [&](int k) { return tmem + TM::S + (k / J) * (NN / 4) + (k % J) * 8; };  // second term NN / 8 on
        auto x_term = [&](uint32_t x, int k) { return tmem + x + k * 16; };                     // second term 8 on
#pragma unroll 1
        for (int i = 0; i < chunks; ++i) {
            const uint32_t par = i & 1, par2 = (i >> 1) & 1;
            const uint32_t kq = sbase + SM::KQ + (i % kStages) * SM::KQ_BYTES, op = sbase + SM::OP + par * 32768;
            const uint64_t kd = tc::desc(kq, 2048, 128), md = tc::desc(op, 128, 1024), td = tc::desc(op + 16384, 128, 1024);
            wait.on(kFullOp + par, par2);
            wait.on(kFullV + i % kVStages, (i / kVStages) & 1);
            if (i > 0) {  // the M^T d before is read
                for (int k = 0; k < 4; ++k) wait.on(kR + k, par ^ 1);
            }
            if (wait.dead()) goto given_up;
            tc::fence_after_sync();
            if (go) {
                const uint64_t vd = tc::desc(sbase + SM::DY + (i % kVStages) * SM::DY_BYTES, 2048, 128);
#pragma unroll
                for (int k = 0; k < kC / 16; ++k) {  // dy^T M
                    tc::mma_f16(tmem + TM::X2, vd + k * K2, md + k * 16, ID_M, k > 0);
                    tc::mma_f16(tmem + TM::X2, vd + k * K2, md + LO + k * 16, ID_M, 1);
                }
                tc::commit(bars + 8 * (kEmptyV + i % kVStages));
                if (UNITS) tc::commit(bars + 8 * kX2);
            }
            wait.on(kFullKQ + i % kStages, (i / kStages) & 1);
#pragma unroll
            for (int j = 0; j < J; ++j) {  // D k^T, as the state's columns come
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
            const uint64_t kt = tc::desc(kq, 128, 2048);
            wait.on(kDReady, par);
            if (wait.dead()) goto given_up;
            tc::fence_after_sync();
            if (go) {
#pragma unroll
                for (int k = 0; k < kC / 16; ++k) {  // (exp(G) d)^T q
                    tc::mma_f16_ts(tmem + TM::DS, x_term(TM::XD, k), kt + 64 + k * 16, ID_DS, k > 0);
                    tc::mma_f16_ts(tmem + TM::DS, x_term(TM::XD, k) + 8, kt + 64 + k * 16, ID_DS, 1);
                }
                tc::commit(bars + 8 * kDFree);
            }
#pragma unroll
            for (int k = 0; k < kC / 16; ++k) {  // dU^T T
                wait.on(kR + k, par);
                if (wait.dead()) goto given_up;
                tc::fence_after_sync();
                if (go) {
                    tc::mma_f16_ts(tmem + TM::X3, x_term(TM::X1, k), td + k * 16, ID_B, k > 0);
                    tc::mma_f16_ts(tmem + TM::X3, x_term(TM::X1, k), td + LO + k * 16, ID_B, 1);
                    tc::mma_f16_ts(tmem + TM::X3, x_term(TM::X1, k) + 8, td + k * 16, ID_B, 1);
                }
            }
            if (go) {
                tc::commit(bars + 8 * kD2);
                tc::commit(bars + 8 * (kEmptyOp + par));
            }
#pragma unroll
            for (int k = 0; k < kC / 16; ++k) {  // - (beta exp(G) R)^T k
                wait.on(kU + k, par);
                if (wait.dead()) goto given_up;
                tc::fence_after_sync();
                if (go) {
                    tc::mma_f16_ts(tmem + TM::DS, x_term(TM::X1, k), kt + k * 16, ID_DS, 1);
                    tc::mma_f16_ts(tmem + TM::DS, x_term(TM::X1, k) + 8, kt + k * 16, ID_DS, 1);
                }
            }
            if (go) {
                tc::commit(bars + 8 * kDS);
                tc::commit(bars + 8 * (kEmptyKQ + i % kStages));
            }
        }
    given_up:
        // the last products may still read shared memory: wait for them before the CTA ends
        if (go) tc::commit(bars + 8 * kDrain);
        Waits{bars}.on(kDrain, 0);
    } else {
        // ---- copies: lane = row of eight, 16-byte piece of four.  The first warp takes k, the second q, the third dy and a chunk's operands
        const int r = lane & 7, piece = lane >> 3, which = warp - kLoadWarp;
        const void *src = which == 0 ? p.k : which == 1 ? p.q : p.dy;
        const long long s0 = which == 0 ? p.ks[0] : which == 1 ? p.qs[0] : (long long)p.L * p.H * p.P,
                        s1 = which == 0 ? p.ks[1] : which == 1 ? p.qs[1] : (long long)p.H * p.P;
        const char *from = static_cast<const char *>(src) + 2 * (b * s0 + (which < 2 ? (long long)grp * p.N : (long long)h * p.P + p0) + 8 * piece);
        const int width = (which < 2 ? p.N : rows) - 8 * piece;
        const uint32_t to = sbase + (which < 2 ? SM::KQ + which * 1024 + piece * 2048 : SM::DY + piece * 128) + r * 16;
        const uint32_t stage = which < 2 ? SM::KQ_BYTES : SM::DY_BYTES, row_step = which < 2 ? 128 : 2048, col_step = which < 2 ? 8192 : 512;
        const int stages = which < 2 ? kStages : kVStages, empty = which < 2 ? kEmptyKQ : kEmptyV, full = which < 2 ? kFullKQ : kFullV;
        int at = 0, issued = 0;
        uint32_t parity = 1;
        const unsigned char *ops = p.ops + (size_t)bh * p.nc * op_bytes(true);
#pragma unroll 1
        for (int i = 0; i < chunks; ++i) {
            const int c = chunks - 1 - i;
            if (which == 2) {  // with a place of T's, the gates four chunks back are done with too
                wait.on(kEmptyOp + (i & 1), ((i >> 1) & 1) ^ 1);
                if (wait.dead()) break;
                if (lane == 0) {
                    const uint32_t bar = bars + 8 * (kFullOp + (i & 1)), dst = sbase + SM::OP + (i & 1) * 32768;
                    const unsigned char *op = ops + (size_t)c * op_bytes(true);
                    tc::mbar_arrive_expect_tx(bar, 32768 + (uint32_t)sizeof(Gates));
                    bulk_load(dst, op + kOpM, 16384, bar);
                    bulk_load(dst + 16384, op + kOpPure, 16384, bar);
                    bulk_load(sbase + SM::GATES + (i % kSlots) * (uint32_t)sizeof(Gates), op + kOpGates, (uint32_t)sizeof(Gates), bar);
                }
                __syncwarp();
                issued = i + 1;
            }
            wait.on(empty + at, parity);
            if (wait.dead()) break;
            const char *row = from + 2 * ((c * kC + r) * s1);
            uint32_t dst = to + at * stage;
#pragma unroll 1
            for (int rg = 0; rg < 8; ++rg, row += 16 * s1, dst += row_step) {
                const int live = c * kC + rg * 8 + r < len ? width : 0;
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
            for (int i = max(issued - kOps, 0); i < issued; ++i) Waits{bars}.on(kFullOp + (i & 1), (i >> 1) & 1);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem_slot, TM::COLS);
}

// Both walks of the gradients in one launch: they need nothing of one another, and few heads leave SMs for both.
template <int IO, int NN>
__global__ void __launch_bounds__(kThreads, 1)
delta_both_kernel(const __grid_constant__ DeltaParams p) {
    const int half = gridDim.x / 2;
    if ((int)blockIdx.x < half) adjoint<IO, NN>(p, blockIdx.x);  // the longer ones first
    else delta_walk::walk<IO, NN, delta_walk::STATES>(p, blockIdx.x - half);
}

template <int IO, int NN>
cudaError_t both_as(const DeltaParams &p, cudaStream_t s) {
    auto *kernel = delta_both_kernel<IO, NN>;
    static_assert(kThreads == delta_walk::kThreads, "one launch");
    constexpr uint32_t bytes = Smem<NN>::BYTES > delta_walk::Smem<NN>::BYTES ? Smem<NN>::BYTES : delta_walk::Smem<NN>::BYTES;
    const cudaError_t e = allow_smem<bytes>(kernel);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(2LL * p.B * p.H * ((p.P + 127) / 128)), kThreads, bytes, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_tc_walks(const DeltaParams &p, int io, cudaStream_t s) {
    if (io == IO_BF16) return p.N <= 64 ? both_as<IO_BF16, 64>(p, s) : both_as<IO_BF16, 128>(p, s);
    return p.N <= 64 ? both_as<IO_F16, 64>(p, s) : both_as<IO_F16, 128>(p, s);
}

}  // namespace ssd

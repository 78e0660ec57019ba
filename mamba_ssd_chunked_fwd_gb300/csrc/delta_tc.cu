// delta_tc.cu -- the gated delta rule in chunks of 64 tokens on the tensor cores, for
// 16-bit tensors.
//
// With G the running sum of g in a chunk, W_ij = exp(G_i - G_j), S the P x N state before it:
//
//     A_ij = beta_i W_ij (k_i . k_j)  (j < i),    T = (I + A)^-1
//     U = T diag(beta) (V - diag(exp G) K S^T)
//     Y = scale (diag(exp G) Q S^T + M U),   M_ij = W_ij (q_i . k_j)  (j <= i)
//     S <- exp(G_end) S + (diag(exp(G_end - G)) U)^T K
//
// A CTA walks the chunks of one head with up to 128 rows of its state, everything
// transposed: the state's rows are the 128 lanes of TMEM, and what the tokens'
// products with the state give (S K^T, U^T) lies along its columns, where the next
// product takes it as its A operand.  Only the chain S K^T -> U -> S is sequential,
// three products to a chunk; the rest runs beside it:
//
//   8 warps  the chain: split S K^T, U and S into operands; the state's fp32 in registers
//   4 warps  A, T and M of the next chunk, and the gates
//   4 warps  y
//   1 warp   issues the products;  1 warp copies k, q and v, up to two chunks ahead
//
// Operands.  q, k and v are 16-bit as they come.  What is computed (S, S K^T, U, T, M) goes
// into a product as the sum of two 16-bit numbers, so that states keep 16 bits (bf16:
// relative error 4e-6 of a state, measured; one term would give 3e-3) and y is off by
// its own rounding alone.  With fp16 a state must stay below 65504.
//
// T.  The diagonal blocks of 16 are inverted by substitution in fp32, the blocks below by
// T_ij = -T_ii sum_k A_ik T_kj with mma.sync on split operands: blocks this small would leave
// tcgen05's 128 rows empty, and each needs the one before it.  No power of A is formed:
// with keys alike those would cancel.
//
// Every wait is bounded; one that gives up fills what its CTA still writes with NaN.
#include "delta.cuh"
#include "tc_operands.cuh"
#include "tc_ptx.cuh"

namespace ssd {

namespace {

constexpr int kC = kDeltaChunk;
constexpr int kChainWarps = 8, kPrepWarps = 4, kOutWarps = 4;
constexpr int kPrepWarp0 = kChainWarps, kOutWarp0 = kPrepWarp0 + kPrepWarps, kMmaWarp = kOutWarp0 + kOutWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = (kLoadWarp + 3) * 32;  // whole warpgroups: registers are dealt out by them
// Registers a thread, per warpgroup: 96 at launch; the chain 144 (its state is 64 of them), y 56, the last
// warpgroup 40.  2 * 144 + 96 + 56 + 40 = 5 * 96.
constexpr int kChainRegs = 144, kOutRegs = 56, kMmaRegs = 40;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kStages = 3;   // of k and q
constexpr int kVStages = 2;  // of v
constexpr int kSlots = 4;    // of a chunk's gates
constexpr int kAW = 68;      // floats between rows of A

struct alignas(16) Gates {
    float gh[kC], gl[kC], beta[kC], into[kC], neg_into[kC], out[kC];  // gh + gl: G in units of log2
    float over;
};

template <int NN>
struct Smem {
    static constexpr uint32_t KQ = 0, KQ_BYTES = 128 * NN * 2;  // rows 0-63 k, 64-127 q
    static constexpr uint32_t V = KQ + kStages * KQ_BYTES, V_BYTES = kC * 128 * 2;
    static constexpr uint32_t T = V + kVStages * V_BYTES, M = T + 2 * 16384;  // two of (8 KB first terms, 8 KB second)
    static constexpr uint32_t A = M + 2 * 16384, GATES = A + kC * kAW * 4, BYTES = GATES + kSlots * (uint32_t)sizeof(Gates) + 128;
};

enum Bar { kFullKQ = 0, kEmptyKQ = 3, kFullV = 6, kEmptyV = 8, kFullT = 10, kEmptyT = 12, kKQDone = 14, kKQRead, kD1, kR, kD2, kU, kDS, kS, kD3, kD3Read,
           kD4, kD4Read, kBars };

// TMEM columns.
template <int NN>
struct Tm {
    static constexpr uint32_t S = 0, X1 = NN, X2 = NN + 64, DS = NN + 128, O = 2 * NN + 128, KQ = 2 * NN + 192, COLS = 512;
};

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
// Two numbers as sums of two 16-bit numbers each.
template <bool BF16>
__device__ __forceinline__ void split2(float2 v, uint32_t &hi, uint32_t &lo) {
    hi = tcop::pack2(v.x, v.y, BF16);
    const float2 h = unpack2<BF16>(hi), d = __fadd2_rn(v, make_float2(-h.x, -h.y));
    lo = tcop::pack2(d.x, d.y, BF16);
}

// ex2 that stays where it is: moved into a branch on whether its result is wanted, each would wait for the one before
// (measured: 68 cycles an element in place of 20).
__device__ __forceinline__ float ex2_now(float v) {
    float r;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// D (16 x 8) += A (16 x 16) B (16 x 8), fp32 sums.
template <bool BF16>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    if (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// A 16 x 16 block as the A operand of a product, in two terms.
struct Frag {
    uint32_t hi[4], lo[4];
};
// Of an accumulated block, acc[half][4]: columns 8 half + ..
template <bool BF16>
__device__ __forceinline__ Frag to_frag(const float (&acc)[2][4]) {
    Frag f;
#pragma unroll
    for (int i = 0; i < 4; ++i) split2<BF16>(make_float2(acc[i >> 1][2 * (i & 1)], acc[i >> 1][2 * (i & 1) + 1]), f.hi[i], f.lo[i]);
    return f;
}
// acc += a X^T with X a 16 x 16 block of `x`, rows kAW apart.
template <bool BF16>
__device__ __forceinline__ void times_transposed(float (&acc)[2][4], const Frag &a, const float *x, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const float *row = x + (8 * half + g) * kAW + 2 * t;
        uint32_t hi[2], lo[2];
        split2<BF16>(*reinterpret_cast<const float2 *>(row), hi[0], lo[0]);
        split2<BF16>(*reinterpret_cast<const float2 *>(row + 8), hi[1], lo[1]);
        mma_16x8x16<BF16>(acc[half], a.lo, hi);
        mma_16x8x16<BF16>(acc[half], a.hi, lo);
        mma_16x8x16<BF16>(acc[half], a.hi, hi);
    }
}

__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

template <int N, bool MORE>
__device__ __forceinline__ void set_registers() {
    if (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A thread's waits: once one has given up, the rest return at once.
struct Waits {
    uint32_t bars;
    bool dead = false;
    __device__ __forceinline__ void on(int bar, uint32_t parity) {
        if (!dead && !tc::mbar_wait(bars + 8 * bar, parity, kWaitNs)) dead = true;
    }
};

// What a CTA walks: tokens [t0, t1) of a head, from a state to a state.
struct Walk {
    int b, h, p0, t0, t1, chunks;
};

// LOCAL: a segment's own state (from zero, the rows of v) and its transition (from the unit matrix, v = 0), no y.
template <int IO, int NN, bool LOCAL>
__global__ void __launch_bounds__(kThreads, 1)
delta_tc_kernel(const __grid_constant__ DeltaParams p) {
    constexpr bool BF16 = IO == IO_BF16;
    using SM = Smem<NN>;
    using TM = Tm<NN>;
    extern __shared__ __align__(1024) unsigned char sm[];
    __shared__ __align__(8) uint64_t bar_mem[kBars];
    __shared__ uint32_t tmem_slot;
    const uint32_t sbase = tc::smem_addr(sm), bars = tc::smem_addr(bar_mem);
    Gates *gates = reinterpret_cast<Gates *>(sm + SM::GATES);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int ptiles = (p.P + 127) / 128, tiles = ptiles + (LOCAL ? 1 : 0);
    int at = blockIdx.x;
    const int tile = at % tiles;
    at /= tiles;
    const int nseg = LOCAL ? p.nseg - 1 : p.nseg, seg = at % nseg;
    at /= nseg;
    Walk w;
    w.h = at % p.H, w.b = at / p.H;
    const bool unit = LOCAL && tile == ptiles;  // the transition: rows are the state's columns
    w.p0 = unit ? 0 : tile * 128;
    const int len = delta_length(p, w.b);
    w.t0 = seg * p.seg_len;
    w.t1 = min(len, w.t0 + p.seg_len);
    w.chunks = max(0, (w.t1 - w.t0 + kC - 1) / kC);
    const int bh = w.b * p.H + w.h, grp = w.h / (p.H / p.G), rows = unit ? p.N : min(128, p.P - w.p0);
    const size_t pn = (size_t)p.P * p.N, nn = (size_t)p.N * p.N;

    if (tid == 0) {
        auto init = [&](int bar, uint32_t count) { tc::mbar_init(bars + 8 * bar, count); };
        for (int i = 0; i < kStages; ++i) init(kFullKQ + i, 32), init(kEmptyKQ + i, 1);
        for (int i = 0; i < 2; ++i) init(kFullV + i, 32), init(kEmptyV + i, 1), init(kFullT + i, kPrepWarps * 32), init(kEmptyT + i, 1);
        for (int b : {(int)kKQDone, (int)kD1, (int)kD2, (int)kDS, (int)kD3, (int)kD4}) init(b, 1);
        init(kKQRead, kPrepWarps * 32);
        for (int b : {(int)kR, (int)kU, (int)kS}) init(b, kChainWarps * 32);
        init(kD3Read, kOutWarps * 32), init(kD4Read, kOutWarps * 32);
        tc::mbar_init_fence();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(tc::smem_addr(&tmem_slot), TM::COLS);
        tc::tmem_relinquish();
    }
    // the blocks of T and M above their diagonals stay zero
    for (int e = tid; e < 4 * 16384 / 16; e += kThreads) tcop::st_shared_v4(sbase + SM::T + 16 * e, 0u, 0u, 0u, 0u);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's, so they begin at column 0
    Waits wait{bars};

    if (warp < kChainWarps) {
        // ---- the chain: thread = row of the state, half of the columns
        set_registers<kChainRegs, true>();
        const int quarter = warp & 3, half = warp >> 2, row = quarter * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        constexpr int NH = NN / 2;
        float2 S[NH / 2];
        auto load_row = [&](const float *src) {
            const bool ok = src && row < rows;
#pragma unroll
            for (int j = 0; j < NH / 4; ++j) {
                const int n = half * NH + 4 * j;
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (ok && n < p.N) f = *reinterpret_cast<const float4 *>(src + (size_t)row * p.N + n);
                S[2 * j] = make_float2(f.x, f.y), S[2 * j + 1] = make_float2(f.z, f.w);
            }
        };
        if (unit) {
#pragma unroll
            for (int j = 0; j < NH / 2; ++j)
                S[j] = make_float2(row == half * NH + 2 * j && row < p.N ? 1.f : 0.f, row == half * NH + 2 * j + 1 && row < p.N ? 1.f : 0.f);
        } else if (LOCAL) {
            load_row(nullptr);
        } else if (seg > 0) {
            load_row(p.seg_states + ((size_t)bh * p.nseg + seg) * pn + (size_t)w.p0 * p.N);
        } else {
            load_row(p.h0 ? p.h0 + bh * pn + (size_t)w.p0 * p.N : nullptr);
        }
        auto publish = [&]() {  // the state as an operand: terms of 16 columns side by side
#pragma unroll
            for (int j = 0; j < NH / 16; ++j) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) split2<BF16>(S[8 * j + i], hi[i], lo[i]);
                tc::tmem_st8(tl + TM::S + half * NH + 8 * j, hi);
                tc::tmem_st8(tl + TM::S + half * NH + NH / 2 + 8 * j, lo);
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(bars + 8 * kS);
        };
        if (w.chunks > 0) publish();
        for (int c = 0; c < w.chunks; ++c) {
            const uint32_t par = c & 1;
            const Gates &gt = gates[c % kSlots];
            wait.on(kFullT + par, (c >> 1) & 1);  // the gates
            wait.on(kD1, par);
            tc::fence_after_sync();
            const uint32_t x1 = tl + TM::X1 + 32 * half, x2 = tl + TM::X2 + 32 * half;
            {
                float a[16], b[16];
                tc::tmem_ld16x2(x1, x1 + 16, a, b);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const float(&v)[16] = s ? b : a;
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 f = *reinterpret_cast<const float4 *>(&gt.neg_into[32 * half + 16 * s + 4 * i]);
                        split2<BF16>(__fmul2_rn(make_float2(v[4 * i], v[4 * i + 1]), make_float2(f.x, f.y)), hi[2 * i], lo[2 * i]);
                        split2<BF16>(__fmul2_rn(make_float2(v[4 * i + 2], v[4 * i + 3]), make_float2(f.z, f.w)), hi[2 * i + 1], lo[2 * i + 1]);
                    }
                    tc::tmem_st8(x1 + 8 * s, hi);
                    tc::tmem_st8(x1 + 16 + 8 * s, lo);
                }
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(bars + 8 * kR);

            wait.on(kD2, par);
            tc::fence_after_sync();
            {
                float a[16], b[16];
                tc::tmem_ld16x2(x2, x2 + 16, a, b);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const float(&v)[16] = s ? b : a;
                    uint32_t hi[8], lo[8];
                    if (!LOCAL) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) split2<BF16>(make_float2(v[2 * i], v[2 * i + 1]), hi[i], lo[i]);
                        tc::tmem_st8(x2 + 8 * s, hi);
                        tc::tmem_st8(x2 + 16 + 8 * s, lo);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 f = *reinterpret_cast<const float4 *>(&gt.out[32 * half + 16 * s + 4 * i]);
                        split2<BF16>(__fmul2_rn(make_float2(v[4 * i], v[4 * i + 1]), make_float2(f.x, f.y)), hi[2 * i], lo[2 * i]);
                        split2<BF16>(__fmul2_rn(make_float2(v[4 * i + 2], v[4 * i + 3]), make_float2(f.z, f.w)), hi[2 * i + 1], lo[2 * i + 1]);
                    }
                    tc::tmem_st8(x1 + 8 * s, hi);
                    tc::tmem_st8(x1 + 16 + 8 * s, lo);
                }
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(bars + 8 * kU);

            const float2 over = dup(gt.over);
            wait.on(kDS, par);
            tc::fence_after_sync();
#pragma unroll
            for (int j = 0; j < NH / 32; ++j) {
                float a[16], b[16];
                tc::tmem_ld16x2(tl + TM::DS + half * NH + 32 * j, tl + TM::DS + half * NH + 32 * j + 16, a, b);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    S[16 * j + i] = __ffma2_rn(over, S[16 * j + i], make_float2(a[2 * i], a[2 * i + 1]));
                    S[16 * j + 8 + i] = __ffma2_rn(over, S[16 * j + 8 + i], make_float2(b[2 * i], b[2 * i + 1]));
                }
            }
            if (c + 1 < w.chunks) publish();
        }
        float *dst = nullptr;
        if (unit) dst = p.seg_trans + ((size_t)bh * nseg + seg) * nn;
        else if (LOCAL) dst = p.seg_states + ((size_t)bh * p.nseg + seg + 1) * pn + (size_t)w.p0 * p.N;
        else if (p.final_state && ((w.t0 < len && len <= w.t0 + p.seg_len) || (len == 0 && seg == 0)))
            dst = p.final_state + bh * pn + (size_t)w.p0 * p.N;
        if (dst && row < rows) {
            const float nan = __int_as_float(0x7fffffff);
#pragma unroll
            for (int j = 0; j < NH / 4; ++j) {
                const int n = half * NH + 4 * j;
                float4 f = make_float4(S[2 * j].x, S[2 * j].y, S[2 * j + 1].x, S[2 * j + 1].y);
                if (wait.dead) f = make_float4(nan, nan, nan, nan);
                if (n < p.N) *reinterpret_cast<float4 *>(dst + (size_t)row * p.N + n) = f;
            }
        }
    } else if (warp < kOutWarp0) {
        // ---- T and M of each chunk
        const int pw = warp - kPrepWarp0, ptid = pw * 32 + lane, i = ptid & 63;
        const uint32_t tl = tmem + (static_cast<uint32_t>(pw * 32) << 16);
        float *A = reinterpret_cast<float *>(sm + SM::A);
        float graw[2] = {0.f, 0.f}, braw[2] = {0.f, 0.f};
        auto fetch = [&](int c) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int t = w.t0 + c * kC + 2 * lane + m;
                graw[m] = load_gate<IO>(p.g, w.b * p.gs[0] + t * p.gs[1] + w.h, p.g32, t < w.t1);
                braw[m] = load_gate<IO>(p.beta, w.b * p.bs[0] + t * p.bs[1] + w.h, p.b32, t < w.t1);
            }
        };
        if (pw == 0 && w.chunks > 0) fetch(0);
        for (int c = 0; c < w.chunks; ++c) {
            const uint32_t par = c & 1, half_par = (c >> 1) & 1;
            Gates &gt = gates[c % kSlots];
            if (pw == 0) {  // the running sum of g as the sum of two floats, so that differences keep their precision
                auto add = [](float &h0, float &l0, float h1, float l1) {
                    const float sum = h0 + h1, t = sum - h0, err = (h0 - (sum - t)) + (h1 - t) + l0 + l1;
                    h0 = sum + err;
                    l0 = err - (h0 - sum);
                };
                float hi[2], lo[2];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float g = graw[m];
                    asm("max.NaN.f32 %0, %0, %1;" : "+f"(g) : "f"(-200.f));  // exp(-200) is 0, and sums stay finite
                    hi[m] = g * kLog2e;
                    lo[m] = fmaf(g, kLog2e, -hi[m]) + g * 1.92596299e-8f;  // log2(e) - fl(log2(e))
                    gt.beta[2 * lane + m] = braw[m];
                }
                if (c + 1 < w.chunks) fetch(c + 1);
                add(hi[1], lo[1], hi[0], lo[0]);
                float th = hi[1], tl2 = lo[1];
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const float oh = __shfl_up_sync(0xffffffffu, th, m), ol = __shfl_up_sync(0xffffffffu, tl2, m);
                    if (lane >= m) add(th, tl2, oh, ol);
                }
                const float ph = __shfl_up_sync(0xffffffffu, th, 1), pl = __shfl_up_sync(0xffffffffu, tl2, 1);
                if (lane > 0) add(hi[0], lo[0], ph, pl);
                hi[1] = th, lo[1] = tl2;
                const float eh = __shfl_sync(0xffffffffu, th, 31), el = __shfl_sync(0xffffffffu, tl2, 31);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int t = 2 * lane + m;
                    const float in = exp2f(hi[m] + lo[m]);
                    gt.gh[t] = hi[m], gt.gl[t] = lo[m], gt.into[t] = in, gt.neg_into[t] = -in;
                    gt.out[t] = exp2f((eh - hi[m]) + (el - lo[m]));
                }
                if (lane == 0) gt.over = exp2f(eh + el);
            }
            tc::named_barrier(1, kPrepWarps * 32);  // the gates; and A of the chunk before is done with
            wait.on(kKQDone, par);
            wait.on(kEmptyT + par, half_par ^ 1);
            tc::fence_after_sync();
            const float gh = gt.gh[i], gl = gt.gl[i], factor = pw < 2 ? gt.beta[i] : 1.f;
            const int limit = pw < 2 ? i : i + 1;
            const int last = (i | 31);  // of the warp's rows
#pragma unroll 1
            for (int j0 = 0; j0 <= last; j0 += 16) {
                float v[16];
                tc::tmem_ld16(tl + TM::KQ + j0, v);
#pragma unroll
                for (int m = 0; m < 16; m += 4) {
                    const int j = j0 + m;
                    const float4 h4 = *reinterpret_cast<const float4 *>(&gt.gh[j]), l4 = *reinterpret_cast<const float4 *>(&gt.gl[j]);
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float2 d = __fadd2_rn(__fadd2_rn(dup(gh), e ? make_float2(-h4.z, -h4.w) : make_float2(-h4.x, -h4.y)),
                                                    __fadd2_rn(dup(gl), e ? make_float2(-l4.z, -l4.w) : make_float2(-l4.x, -l4.y)));
                        const float2 x = __fmul2_rn(__fmul2_rn(make_float2(ex2_now(d.x), ex2_now(d.y)), dup(factor)), make_float2(v[m + e], v[m + e + 1]));
                        v[m + e] = j + e < limit ? x.x : 0.f;
                        v[m + e + 1] = j + e + 1 < limit ? x.y : 0.f;
                    }
                }
                if (pw < 2) {
#pragma unroll
                    for (int m = 0; m < 16; m += 4) *reinterpret_cast<float4 *>(A + i * kAW + j0 + m) = make_float4(v[m], v[m + 1], v[m + 2], v[m + 3]);
                } else if (!LOCAL) {
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int m = 0; m < 8; ++m) split2<BF16>(make_float2(v[2 * m], v[2 * m + 1]), hi[m], lo[m]);
                    const uint32_t dst = sbase + SM::M + par * 16384 + ((j0 >> 3) * 8 + (i >> 3)) * 128 + (i & 7) * 16;
                    tcop::st_shared_v4(dst, hi[0], hi[1], hi[2], hi[3]);
                    tcop::st_shared_v4(dst + 1024, hi[4], hi[5], hi[6], hi[7]);
                    tcop::st_shared_v4(dst + 8192, lo[0], lo[1], lo[2], lo[3]);
                    tcop::st_shared_v4(dst + 8192 + 1024, lo[4], lo[5], lo[6], lo[7]);
                }
            }
            tc::fence_before_sync();
            tc::mbar_arrive(bars + 8 * kKQRead);
            tc::named_barrier(1, kPrepWarps * 32);
            // the diagonal block pw: lane = column, both halves of the warp alike; the inverse takes its place
            float *D = A + 16 * pw * kAW + 16 * pw;
            {
                const int col = lane & 15;
                float x[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float s0 = r == col ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
                    for (int k = 0; k < r; k += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(D + r * kAW + k);
                        s0 = fmaf(-f.x, x[k], s0);
                        if (k + 1 < r) s1 = fmaf(-f.y, x[k + 1 < 16 ? k + 1 : 0], s1);
                        if (k + 2 < r) s0 = fmaf(-f.z, x[k + 2 < 16 ? k + 2 : 0], s0);
                        if (k + 3 < r) s1 = fmaf(-f.w, x[k + 3 < 16 ? k + 3 : 0], s1);
                    }
                    x[r] = s0 + s1;
                }
                __syncwarp();
                if (lane < 16) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) D[r * kAW + col] = x[r];
                }
            }
            tc::named_barrier(1, kPrepWarps * 32);
            // column pw of blocks, transposed: element (c, r) of a block is T[r][c]
            {
                const int g = lane >> 2, t = lane & 3;
                const float b0 = gt.beta[16 * pw + g], b1 = gt.beta[16 * pw + g + 8];
                const uint32_t to = sbase + SM::T + par * 16384 + ((2 * pw + ((lane >> 3) & 1)) * 8 + (lane >> 4)) * 128 + (lane & 7) * 16;
                auto store = [&](const float(&acc)[2][4], int bi) {  // T diag(beta) in two terms
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const float b = m & 1 ? b1 : b0;
                        split2<BF16>(make_float2(b * acc[m >> 1][2 * (m & 1)], b * acc[m >> 1][2 * (m & 1) + 1]), hi[m], lo[m]);
                    }
                    stmatrix_x4_trans(to + bi * 256, hi);
                    stmatrix_x4_trans(to + bi * 256 + 8192, lo);
                };
                Frag T[3];
                float acc[2][4];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[m][e] = D[(8 * m + 2 * t + (e & 1)) * kAW + g + 8 * (e >> 1)];
                store(acc, pw);
                T[0] = to_frag<BF16>(acc);
#pragma unroll
                for (int s = 1; s < 4; ++s) {
                    const int bi = pw + s;
                    if (bi < 4) {
                        float sum[2][4] = {};
#pragma unroll
                        for (int k = 0; k < s; ++k) times_transposed<BF16>(sum, T[k], A + 16 * bi * kAW + 16 * (pw + k), lane);
                        float res[2][4] = {};
                        times_transposed<BF16>(res, to_frag<BF16>(sum), A + 16 * bi * kAW + 16 * bi, lane);
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int e = 0; e < 4; ++e) res[m][e] = -res[m][e];
                        store(res, bi);
                        if (s < 3) T[s < 3 ? s : 0] = to_frag<BF16>(res);
                    }
                }
            }
            tc::fence_smem_to_async();
            tc::mbar_arrive(bars + 8 * (kFullT + par));
        }
    } else if (warp < kMmaWarp) {
        // ---- y: thread = row of the state
        set_registers<kOutRegs, false>();
        if (!LOCAL) {
            const int quarter = warp - kOutWarp0, row = quarter * 32 + lane;
            const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + TM::O;
            const bool ok = row < rows;
            const size_t step = (size_t)p.H * p.P;
            const size_t base = ((size_t)w.b * p.L * p.H + w.h) * p.P + w.p0 + row;
            const int odd = lane & 1;
            uint16_t *y = static_cast<uint16_t *>(p.y) + base - odd + odd * step;  // of an odd lane: the token after, from the row before
            for (int c = 0; c < w.chunks; ++c) {
                const uint32_t par = c & 1;
                const Gates &gt = gates[c % kSlots];
                wait.on(kFullT + par, (c >> 1) & 1);
                wait.on(kD3, par);
                tc::fence_after_sync();
#pragma unroll 1
                for (int j = 0; j < kC; j += 16) {  // diag(exp G) Q S^T, onto which M U is summed
                    float v[16];
                    uint32_t r[16];
                    tc::tmem_ld16(tl + j, v);
#pragma unroll
                    for (int m = 0; m < 16; m += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(&gt.into[j + m]);
                        r[m] = __float_as_uint(v[m] * f.x), r[m + 1] = __float_as_uint(v[m + 1] * f.y);
                        r[m + 2] = __float_as_uint(v[m + 2] * f.z), r[m + 3] = __float_as_uint(v[m + 3] * f.w);
                    }
                    tc::tmem_st16(tl + j, r);
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                tc::mbar_arrive(bars + 8 * kD3Read);
                wait.on(kD4, par);
                tc::fence_after_sync();
                const int tc0 = w.t0 + c * kC, n = min(kC, w.t1 - tc0);
                const float scale = wait.dead ? __int_as_float(0x7fffffff) : p.scale;
                uint16_t *to = y + (size_t)tc0 * step;
#pragma unroll 1
                for (int j = 0; j < kC; j += 16, to += 16 * step) {
                    float v[16];
                    tc::tmem_ld16(tl + j, v);
                    // neighbouring lanes exchange: each then has two rows of every second token, a store of 4 bytes
#pragma unroll
                    for (int m = 0; m < 16; m += 2) {
                        const uint32_t own = tcop::pack2(scale * v[m], scale * v[m + 1], BF16), other = __shfl_xor_sync(0xffffffffu, own, 1);
                        const uint32_t two = __byte_perm(own, other, odd ? 0x3276 : 0x5410);
                        if (ok && j + m + odd < n) *reinterpret_cast<uint32_t *>(to + m * step) = two;
                    }
                }
                tc::fence_before_sync();
                tc::mbar_arrive(bars + 8 * kD4Read);
            }
            const int end = min(p.L, w.t0 + p.seg_len);
            if (ok)
                for (int t = max(w.t1, w.t0); t < end; ++t) st_io<IO>(p.y, base + (size_t)t * step, 0.f);
        }
    } else if (set_registers<kMmaRegs, false>(); warp == kMmaWarp) {
        // ---- the products.  The warp stays together and one elected lane issues: the descriptors
        // are then the warp's, not a thread's, and a product costs a few instructions in place of
        // a dozen (measured beside busy warps: 16 products 540 to 2100 cycles, from a lane's branch 830 to 15000)
        const bool go = tc::elect_one();
        constexpr uint32_t ID = tc::idesc_f16(128, kC, BF16, false, false), ID_V = tc::idesc_f16(128, kC, BF16, true, false),
                           ID_DS = tc::idesc_f16(128, NN, BF16, false, true);
        constexpr int NK = NN / 16;  // steps of 16 along a state's columns
        auto s_term = [&](int k, int term) {  // 16 columns of the state's operand: first or second term
            return tmem + TM::S + (k / (NK / 2)) * (NN / 2) + term * (NN / 4) + (k % (NK / 2)) * 8;
        };
        auto x_term = [&](uint32_t x, int k, int term) { return tmem + x + (k >> 1) * 32 + term * 16 + (k & 1) * 8; };
        auto kq_product = [&](int c) {  // [k; q] k^T
            const uint32_t kq = sbase + SM::KQ + (c % kStages) * SM::KQ_BYTES;
            wait.on(kFullKQ + c % kStages, (c / kStages) & 1);
            wait.on(kKQRead, (c & 1) ^ 1);
            tc::fence_after_sync();
            if (go) {
#pragma unroll
                for (int k = 0; k < NK; ++k)
                    tc::mma_f16(tmem + TM::KQ, tc::desc(kq + k * 4096, 2048, 128), tc::desc(kq + k * 4096, 2048, 128), ID, k > 0);
                tc::commit(bars + 8 * kKQDone);
            }
        };
        if (w.chunks > 0) kq_product(0);
        for (int c = 0; c < w.chunks; ++c) {
            const uint32_t par = c & 1, kq = sbase + SM::KQ + (c % kStages) * SM::KQ_BYTES, v = sbase + SM::V + (c % kVStages) * SM::V_BYTES;
            const uint32_t T = sbase + SM::T + par * 16384, M = sbase + SM::M + par * 16384;
            wait.on(kS, par);
            tc::fence_after_sync();
            if (go) {
#pragma unroll
                for (int k = 0; k < NK; ++k) {  // S k^T
                    const uint64_t b = tc::desc(kq + k * 4096, 2048, 128);
                    tc::mma_f16_ts(tmem + TM::X1, s_term(k, 0), b, ID, k > 0);
                    tc::mma_f16_ts(tmem + TM::X1, s_term(k, 1), b, ID, 1);
                }
                tc::commit(bars + 8 * kD1);
            }
            if (c + 1 < w.chunks) kq_product(c + 1);
            wait.on(kFullT + par, (c >> 1) & 1);
            wait.on(kFullV + c % kVStages, (c / kVStages) & 1);
            tc::fence_after_sync();
            if (go) {
                if (!unit) {
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k) {  // v^T (T diag(beta))^T
                        const uint64_t a = tc::desc(v + k * 4096, 2048, 128);
                        tc::mma_f16(tmem + TM::X2, a, tc::desc(T + k * 2048, 1024, 128), ID_V, k > 0);
                        tc::mma_f16(tmem + TM::X2, a, tc::desc(T + 8192 + k * 2048, 1024, 128), ID_V, 1);
                    }
                }
                tc::commit(bars + 8 * (kEmptyV + c % kVStages));
            }
            wait.on(kR, par);
            tc::fence_after_sync();
            if (go) {
#pragma unroll
                for (int k = 0; k < kC / 16; ++k) {  // - (exp(G) S k^T) (T diag(beta))^T
                    const uint64_t hi = tc::desc(T + k * 2048, 1024, 128), lo = tc::desc(T + 8192 + k * 2048, 1024, 128);
                    tc::mma_f16_ts(tmem + TM::X2, x_term(TM::X1, k, 0), hi, ID, !unit || k > 0);
                    tc::mma_f16_ts(tmem + TM::X2, x_term(TM::X1, k, 0), lo, ID, 1);
                    tc::mma_f16_ts(tmem + TM::X2, x_term(TM::X1, k, 1), hi, ID, 1);
                }
                tc::commit(bars + 8 * kD2);
            }
            if (!LOCAL) {  // while the chain splits U
                wait.on(kD4Read, par ^ 1);
                tc::fence_after_sync();
                if (go) {
#pragma unroll
                    for (int k = 0; k < NK; ++k) {  // S q^T
                        const uint64_t b = tc::desc(kq + 1024 + k * 4096, 2048, 128);
                        tc::mma_f16_ts(tmem + TM::O, s_term(k, 0), b, ID, k > 0);
                        tc::mma_f16_ts(tmem + TM::O, s_term(k, 1), b, ID, 1);
                    }
                    tc::commit(bars + 8 * kD3);
                }
            }
            wait.on(kU, par);
            tc::fence_after_sync();
            if (go) {
#pragma unroll
                for (int k = 0; k < kC / 16; ++k) {  // the change of the state
                    const uint64_t b = tc::desc(kq + k * 256, 128, 2048);
                    tc::mma_f16_ts(tmem + TM::DS, x_term(TM::X1, k, 0), b, ID_DS, k > 0);
                    tc::mma_f16_ts(tmem + TM::DS, x_term(TM::X1, k, 1), b, ID_DS, 1);
                }
                tc::commit(bars + 8 * kDS);
                tc::commit(bars + 8 * (kEmptyKQ + c % kStages));
            }
            if (!LOCAL) {
                wait.on(kD3Read, par);
                tc::fence_after_sync();
                if (go) {
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k) {  // U^T M^T
                        const uint64_t hi = tc::desc(M + k * 2048, 1024, 128), lo = tc::desc(M + 8192 + k * 2048, 1024, 128);
                        tc::mma_f16_ts(tmem + TM::O, x_term(TM::X2, k, 0), hi, ID, 1);
                        tc::mma_f16_ts(tmem + TM::O, x_term(TM::X2, k, 0), lo, ID, 1);
                        tc::mma_f16_ts(tmem + TM::O, x_term(TM::X2, k, 1), hi, ID, 1);
                    }
                    tc::commit(bars + 8 * kD4);
                }
            }
            if (go) tc::commit(bars + 8 * (kEmptyT + par));
        }
        // the last products may still read shared memory: wait for them before the CTA ends
        if (w.chunks > 0) wait.on(kEmptyT + ((w.chunks - 1) & 1), ((w.chunks - 1) >> 1) & 1);
        __syncwarp();
    } else if (warp == kLoadWarp) {
        // ---- copies: lane = row of eight, 16-byte piece of four
        const int r = lane & 7, piece = lane >> 3;
        const char *kb = static_cast<const char *>(p.k) + 2 * (w.b * p.ks[0] + (long long)grp * p.N);
        const char *qb = static_cast<const char *>(p.q) + 2 * (w.b * p.qs[0] + (long long)grp * p.N);
        const char *vb = static_cast<const char *>(p.v) + 2 * (w.b * p.vs[0] + (long long)w.h * p.P + w.p0);
        auto copy = [&](uint32_t dst, const char *src, bool ok) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(ok ? src : nullptr), "r"(ok ? 16 : 0) : "memory");
        };
        for (int i = 0; i < w.chunks + 2; ++i) {
            if (i < w.chunks) {
                wait.on(kEmptyKQ + i % kStages, ((i / kStages) & 1) ^ 1);
                const uint32_t kq = sbase + SM::KQ + (i % kStages) * SM::KQ_BYTES;
#pragma unroll 2
                for (int rg = 0; rg < 8; ++rg) {
                    const int t = w.t0 + i * kC + rg * 8 + r;
                    const bool live = t < w.t1;
                    const char *ks = kb + 2 * (t * p.ks[1]), *qs = qb + 2 * (t * p.qs[1]);
#pragma unroll
                    for (int cg = 0; cg < NN / 32; ++cg) {
                        const int col = cg * 4 + piece;
                        const uint32_t dst = kq + (col * 16 + rg) * 128 + r * 16;
                        const bool ok = live && col * 8 < p.N;
                        copy(dst, ks + 16 * col, ok);
                        if (!LOCAL) copy(dst + 1024, qs + 16 * col, ok);
                    }
                }
            }
            cp_commit();
            if (i >= 1 && i - 1 < w.chunks) {
                const int c = i - 1;
                wait.on(kEmptyV + c % kVStages, ((c / kVStages) & 1) ^ 1);
                const uint32_t v = sbase + SM::V + (c % kVStages) * SM::V_BYTES;
                if (!unit) {
#pragma unroll 2
                    for (int rg = 0; rg < 8; ++rg) {
                        const int t = w.t0 + c * kC + rg * 8 + r;
                        const char *vs = vb + 2 * (t * p.vs[1]);
#pragma unroll
                        for (int cg = 0; cg < 4; ++cg) {
                            const int col = cg * 4 + piece;
                            copy(v + (rg * 16 + col) * 128 + r * 16, vs + 16 * col, t < w.t1 && col * 8 < rows);
                        }
                    }
                }
            }
            cp_commit();
            cp_wait<2>();  // all but this round's two groups
            tc::fence_smem_to_async();
            if (i >= 1 && i - 1 < w.chunks) tc::mbar_arrive(bars + 8 * (kFullKQ + (i - 1) % kStages));
            if (i >= 2) tc::mbar_arrive(bars + 8 * (kFullV + (i - 2) % kVStages));
        }
        cp_wait<0>();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem_slot, TM::COLS);
}

template <int IO, int NN>
cudaError_t tc_as(const DeltaParams &p, bool local, cudaStream_t s) {
    const long long tiles = (p.P + 127) / 128;
    if (local) {
        auto *kernel = delta_tc_kernel<IO, NN, true>;
        const cudaError_t e = allow_smem<Smem<NN>::BYTES>(kernel);
        if (e != cudaSuccess) return e;
        kernel<<<(unsigned)((long long)p.B * p.H * (p.nseg - 1) * (tiles + 1)), kThreads, Smem<NN>::BYTES, s>>>(p);
    } else {
        auto *kernel = delta_tc_kernel<IO, NN, false>;
        const cudaError_t e = allow_smem<Smem<NN>::BYTES>(kernel);
        if (e != cudaSuccess) return e;
        kernel<<<(unsigned)((long long)p.B * p.H * p.nseg * tiles), kThreads, Smem<NN>::BYTES, s>>>(p);
    }
    return cudaGetLastError();
}

template <int IO>
cudaError_t tc_io(const DeltaParams &p, cudaStream_t s) {
    return p.N <= 64 ? tc_as<IO, 64>(p, false, s) : tc_as<IO, 128>(p, false, s);
}

bool by_eights(const void *p, long long s0, long long s1) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && s0 % 8 == 0 && s1 % 8 == 0;
}

}  // namespace

// 16-byte pieces of k, q and v, and float4 of the states.
bool delta_tc_takes(const DeltaParams &p, int io) {
    return io != IO_F32 && p.N % 8 == 0 && p.P % 8 == 0 && by_eights(p.k, p.ks[0], p.ks[1]) && by_eights(p.q, p.qs[0], p.qs[1]) &&
           by_eights(p.v, p.vs[0], p.vs[1]) && by_eights(p.y, 0, 0) && by_eights(p.h0, 0, 0) && by_eights(p.final_state, 0, 0);
}

cudaError_t launch_delta_tc(const DeltaParams &p, int io, cudaStream_t s) {
    return io == IO_BF16 ? tc_io<IO_BF16>(p, s) : tc_io<IO_F16>(p, s);
}

}  // namespace ssd

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
//   16 warps the chain: split S K^T, U and S into operands; the state's fp32 in registers
//   4 warps  A and T of the next chunk
//   4 warps  y, and M of the next chunk
//   1 warp   issues the products
//   3 warps  copy k, q and v ahead; the third works out the gates
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
constexpr int kChainWarps = 16, kPrepWarps = 4, kOutWarps = 4;
constexpr int kPrepWarp0 = kChainWarps, kOutWarp0 = kPrepWarp0 + kPrepWarps, kMmaWarp = kOutWarp0 + kOutWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = (kLoadWarp + 3) * 32;  // three warps copy: k, q, and v with the gates
// Registers a thread, per warpgroup: 72 at launch; the chain's four 80 (the state is 32 of them), T 88, y 48, the last
// 48.  4 * 80 + 88 + 48 + 48 = 7 * 72.
constexpr int kChainRegs = 80, kPrepRegs = 88, kOutRegs = 48, kMmaRegs = 48;
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

enum Bar { kFullKQ = 0, kEmptyKQ = 3, kFullV = 6, kEmptyV = 8, kFullT = 10, kEmptyT = 12, kFullM = 14, kFullG = 16, kKQDone = 20, kKQRead, kD1, kD2, kDS,
           kD3, kD3Read, kD4, kD4Read, kUOut, kS, kR = kS + 2, kU = kR + 4, kBars = kU + 4 };

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
    const float2 d = __ffma2_rn(unpack2<BF16>(hi), make_float2(-1.f, -1.f), v);
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

// A chunk's gates by one warp, two tokens to a lane: the running sum of g as the sum of two floats, so that
// differences keep their precision.
__device__ __forceinline__ void make_gates(Gates &gt, const float (&graw)[2], const float (&beta)[2], int lane) {
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
        gt.beta[2 * lane + m] = beta[m];
    }
    add(hi[1], lo[1], hi[0], lo[0]);
    float th = hi[1], tl = lo[1];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const float oh = __shfl_up_sync(0xffffffffu, th, m), ol = __shfl_up_sync(0xffffffffu, tl, m);
        if (lane >= m) add(th, tl, oh, ol);
    }
    const float ph = __shfl_up_sync(0xffffffffu, th, 1), pl = __shfl_up_sync(0xffffffffu, tl, 1);
    if (lane > 0) add(hi[0], lo[0], ph, pl);
    hi[1] = th, lo[1] = tl;
    const float eh = __shfl_sync(0xffffffffu, th, 31), el = __shfl_sync(0xffffffffu, tl, 31);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int t = 2 * lane + m;
        const float in = exp2f(hi[m] + lo[m]);
        gt.gh[t] = hi[m], gt.gl[t] = lo[m], gt.into[t] = in, gt.neg_into[t] = -in;
        gt.out[t] = exp2f((eh - hi[m]) + (el - lo[m]));
    }
    if (lane == 0) gt.over = exp2f(eh + el);
}

// 16 columns from j0 on of a row of products, each times its decay and the row's factor; zero from column `limit` on.
__device__ __forceinline__ void decayed(float (&v)[16], const Gates &gt, int j0, float gh, float gl, float factor, int limit) {
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
// Of a block in shared memory, rows kAW apart.
template <bool BF16>
__device__ __forceinline__ Frag load_frag(const float *x, int lane) {
    const float *at = x + (lane >> 2) * kAW + 2 * (lane & 3);
    Frag f;
#pragma unroll
    for (int i = 0; i < 4; ++i) split2<BF16>(*reinterpret_cast<const float2 *>(at + (i & 1) * 8 * kAW + (i >> 1) * 8), f.hi[i], f.lo[i]);
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

// 16 tokens' values, each times its factor, as an operand: first terms at `to`, second ones 8 columns on.
template <bool BF16>
__device__ __forceinline__ void split_scaled(const float (&x)[16], const float *f16, uint32_t to) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 f = *reinterpret_cast<const float4 *>(f16 + 4 * i);
        split2<BF16>(__fmul2_rn(make_float2(x[4 * i], x[4 * i + 1]), make_float2(f.x, f.y)), hi[2 * i], lo[2 * i]);
        split2<BF16>(__fmul2_rn(make_float2(x[4 * i + 2], x[4 * i + 3]), make_float2(f.z, f.w)), hi[2 * i + 1], lo[2 * i + 1]);
    }
    tc::tmem_st8(to, hi);
    tc::tmem_st8(to + 8, lo);
}

template <int N, bool MORE>
__device__ __forceinline__ void set_registers() {
    if (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A thread's waits: each lasts 2000 tries of up to a millisecond; once one has given up, the rest return
// at once.  Short code: five kinds of warps run side by side, and what they run has to stay in the
// instruction cache (with unrolled loops and longer waits every second cycle went to fetching).
struct Waits {
    uint32_t bars;
    uint32_t tries = 2000;
    __device__ __forceinline__ bool dead() const { return tries == 0; }
    __device__ __forceinline__ void on(int bar, uint32_t parity) {
        uint32_t done = 0;
#pragma unroll 1
        for (uint32_t i = 0; i < tries && !done; ++i)
            asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000000;\n\tselp.u32 %0, 1, 0, p;\n}\n"
                         : "=r"(done) : "r"(bars + 8 * bar), "r"(parity) : "memory");
        tries = done ? tries : 0u;
        asm volatile("" : "+r"(tries));  // or the code after it is laid out twice, for a thread that waits and one that does not
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
        for (int i = 0; i < kStages; ++i) init(kFullKQ + i, 64), init(kEmptyKQ + i, 1);
        for (int i = 0; i < 2; ++i) init(kFullV + i, 32), init(kEmptyV + i, 1), init(kFullT + i, kPrepWarps * 32), init(kEmptyT + i, 1), init(kFullM + i, 64);
        for (int i = 0; i < kSlots; ++i) init(kFullG + i, 32);
        for (int b : {(int)kKQDone, (int)kD1, (int)kD2, (int)kDS, (int)kD3, (int)kD4}) init(b, 1);
        init(kKQRead, 128);
        for (int b = kS; b < kR; ++b) init(b, kChainWarps * 32);
        for (int b = kR; b < kBars; ++b) init(b, kChainWarps * 8);
        init(kUOut, kChainWarps * 32), init(kD3Read, kOutWarps * 32), init(kD4Read, kOutWarps * 32);
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
        // ---- the chain: thread = row of the state, a quarter of its columns, 16 of the 64 tokens
        set_registers<kChainRegs, true>();
        const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        constexpr int CW = NN / 4;
        float2 S[CW / 2];
        {
            const float *src = nullptr;
            if (!LOCAL && seg > 0) src = p.seg_states + ((size_t)bh * p.nseg + seg) * pn + (size_t)w.p0 * p.N;
            else if (!LOCAL && p.h0) src = p.h0 + bh * pn + (size_t)w.p0 * p.N;
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
#pragma unroll 1
        for (int c = 0;; ++c) {
            const uint32_t par = c & 1;
            if (c > 0) {
                wait.on(kDS, par ^ 1);
                tc::fence_after_sync();
            }
            const float2 over = dup(c > 0 ? gates[(c - 1) % kSlots].over : 1.f);
            // the state after the chunk before, by 16 columns, and each of them as an operand: the product with k
            // begins with the first
#pragma unroll
            for (int j = 0; j < CW / 16; ++j) {
                if (c > 0) {
                    float v[16];
                    tc::tmem_ld16(tl + TM::DS + part * CW + 16 * j, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) S[8 * j + i] = __ffma2_rn(over, S[8 * j + i], make_float2(v[2 * i], v[2 * i + 1]));
                }
                if (c < w.chunks) {
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) split2<BF16>(S[8 * j + i], hi[i], lo[i]);
                    tc::tmem_st8(tl + TM::S + part * CW + 8 * j, hi);
                    tc::tmem_st8(tl + TM::S + part * CW + CW / 2 + 8 * j, lo);
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    tc::mbar_arrive(bars + 8 * (kS + j));
                }
            }
            if (c >= w.chunks) break;
            const Gates &gt = gates[c % kSlots];
            wait.on(kFullG + c % kSlots, (c / kSlots) & 1);
            wait.on(kD1, par);
            tc::fence_after_sync();
            float v[16];
            tc::tmem_ld16(x1, v);
            split_scaled<BF16>(v, &gt.neg_into[16 * part], x1);  // -exp(G) S k^T
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(bars + 8 * (kR + part));
            wait.on(kD2, par);
            tc::fence_after_sync();
            tc::tmem_ld16(x2, v);
            split_scaled<BF16>(v, &gt.out[16 * part], x1);  // what U adds to the state
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(bars + 8 * (kU + part));
            if (!LOCAL) {  // U itself, for y
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) split2<BF16>(make_float2(v[2 * i], v[2 * i + 1]), hi[i], lo[i]);
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
    } else if (warp < kOutWarp0) {
        // ---- T of each chunk
        set_registers<kPrepRegs, true>();
        const int pw = warp - kPrepWarp0, ptid = pw * 32 + lane, i = ptid & 63;
        const uint32_t tl = tmem + (static_cast<uint32_t>(pw * 32) << 16);
        float *A = reinterpret_cast<float *>(sm + SM::A);
        for (int c = 0; c < w.chunks; ++c) {
            const uint32_t par = c & 1, half_par = (c >> 1) & 1;
            const Gates &gt = gates[c % kSlots];
            tc::named_barrier(1, kPrepWarps * 32);  // A of the chunk before is done with
            wait.on(kFullG + c % kSlots, (c / kSlots) & 1);
            if (pw < 2) {
                wait.on(kKQDone, par);
                tc::fence_after_sync();
                const float gh = gt.gh[i], gl = gt.gl[i], beta = gt.beta[i];
                const int last = i | 31;  // of the warp's rows
#pragma unroll 1
                for (int j0 = 0; j0 <= last; j0 += 16) {
                    float v[16];
                    tc::tmem_ld16(tl + TM::KQ + j0, v);
                    decayed(v, gt, j0, gh, gl, beta, i);
#pragma unroll
                    for (int m = 0; m < 16; m += 4) *reinterpret_cast<float4 *>(A + i * kAW + j0 + m) = make_float4(v[m], v[m + 1], v[m + 2], v[m + 3]);
                }
                tc::fence_before_sync();
                tc::mbar_arrive(bars + 8 * kKQRead);
            }
            wait.on(kEmptyT + par, half_par ^ 1);
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
                // element (c, r) of block (pw, k) of the buffer, above its diagonal, will be T[r][c] of T's block (k, pw)
                float *mine = A + 16 * pw * kAW;
                float acc[2][4];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[m][e] = D[(8 * m + 2 * t + (e & 1)) * kAW + g + 8 * (e >> 1)];
                store(acc, pw);
                const Frag first = to_frag<BF16>(acc);
#pragma unroll 1
                for (int bi = pw + 1; bi < 4; ++bi) {
                    float sum[2][4] = {};
                    times_transposed<BF16>(sum, first, A + 16 * bi * kAW + 16 * pw, lane);
#pragma unroll 1
                    for (int k = pw + 1; k < bi; ++k) times_transposed<BF16>(sum, load_frag<BF16>(mine + 16 * k, lane), A + 16 * bi * kAW + 16 * k, lane);
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum[m][e] = -sum[m][e], acc[m][e] = 0.f;
                    times_transposed<BF16>(acc, to_frag<BF16>(sum), A + 16 * bi * kAW + 16 * bi, lane);
                    store(acc, bi);
                    if (bi < 3) {
#pragma unroll
                        for (int m = 0; m < 4; ++m)
                            *reinterpret_cast<float2 *>(mine + 16 * bi + (g + 8 * (m & 1)) * kAW + 2 * t + 8 * (m >> 1)) =
                                make_float2(acc[m >> 1][2 * (m & 1)], acc[m >> 1][2 * (m & 1) + 1]);
                        __syncwarp();
                    }
                }
            }
            tc::fence_smem_to_async();
            tc::mbar_arrive(bars + 8 * (kFullT + par));
        }
    } else if (warp < kMmaWarp) {
        // ---- y: thread = row of the state
        set_registers<kOutRegs, false>();
        if (LOCAL) {  // no y, no M: what the other half of a product's lanes would be read for
            if (warp - kOutWarp0 >= 2)
                for (int c = 0; c < w.chunks; ++c) {
                    wait.on(kKQDone, c & 1);
                    tc::mbar_arrive(bars + 8 * kKQRead);
                }
        } else {
            const int quarter = warp - kOutWarp0, row = quarter * 32 + lane;
            const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + TM::O;
            const bool ok = row < rows;
            const size_t step = (size_t)p.H * p.P;
            // M: q's rows of the product with k lie in lanes 64 to 127
            auto make_m = [&](int c) {
                if (quarter < 2) return;
                const Gates &gt = gates[c % kSlots];
                const int i = row - 64, last = i | 31;
                const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + TM::KQ, to = sbase + SM::M + (c & 1) * 16384 + (i >> 3) * 128 + (i & 7) * 16;
                wait.on(kFullG + c % kSlots, (c / kSlots) & 1);
                wait.on(kKQDone, c & 1);
                tc::fence_after_sync();
                const float gh = gt.gh[i], gl = gt.gl[i];
#pragma unroll 1
                for (int j0 = 0; j0 <= last; j0 += 16) {
                    float v[16];
                    uint32_t hi[8], lo[8];
                    tc::tmem_ld16(from + j0, v);
                    decayed(v, gt, j0, gh, gl, 1.f, i + 1);
#pragma unroll
                    for (int m = 0; m < 8; ++m) split2<BF16>(make_float2(v[2 * m], v[2 * m + 1]), hi[m], lo[m]);
                    const uint32_t dst = to + (j0 >> 3) * 1024;
                    tcop::st_shared_v4(dst, hi[0], hi[1], hi[2], hi[3]);
                    tcop::st_shared_v4(dst + 1024, hi[4], hi[5], hi[6], hi[7]);
                    tcop::st_shared_v4(dst + 8192, lo[0], lo[1], lo[2], lo[3]);
                    tcop::st_shared_v4(dst + 8192 + 1024, lo[4], lo[5], lo[6], lo[7]);
                }
                tc::fence_before_sync();
                tc::mbar_arrive(bars + 8 * kKQRead);
                tc::fence_smem_to_async();
                tc::mbar_arrive(bars + 8 * (kFullM + (c & 1)));
            };
            const size_t base = ((size_t)w.b * p.L * p.H + w.h) * p.P + w.p0 + row;
            const int odd = lane & 1;
            uint16_t *y = static_cast<uint16_t *>(p.y) + base - odd + odd * step;  // of an odd lane: the token after, from the row before
#pragma unroll 1
            for (int c = 0; c <= w.chunks; ++c) {  // the y of chunk c - 1; in between M of chunk c, whose buffer's last product the y before waited for
                const uint32_t par = (c & 1) ^ 1;
                if (c > 0) {
                    const Gates &gt = gates[(c - 1) % kSlots];
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
                }
                if (c < w.chunks) make_m(c);
                if (c == 0) continue;
                wait.on(kD4, par);
                tc::fence_after_sync();
                const int tc0 = w.t0 + (c - 1) * kC, n = min(kC, w.t1 - tc0);
                const float scale = wait.dead() ? __int_as_float(0x7fffffff) : p.scale;
                uint16_t *to = y + (size_t)tc0 * step;
#pragma unroll 1
                for (int j = 0; j < kC; j += 16) {
                    float v[16];
                    tc::tmem_ld16(tl + j, v);
                    // neighbouring lanes exchange: each then has two rows of every second token, a store of 4 bytes
#pragma unroll
                    for (int m = 0; m < 16; m += 2, to += 2 * step) {
                        const uint32_t own = tcop::pack2(scale * v[m], scale * v[m + 1], BF16), other = __shfl_xor_sync(0xffffffffu, own, 1);
                        const uint32_t two = __byte_perm(own, other, odd ? 0x3276 : 0x5410);
                        if (ok && j + m + odd < n) *reinterpret_cast<uint32_t *>(to) = two;
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
        constexpr int NK = NN / 16, J = NN / 64;  // steps of 16 along a state's columns; of a thread's part of them
        constexpr uint32_t K2 = 2 * 128 * 16 / 16;  // of a descriptor: from one step of 16 columns of k, q or v to the next
        auto s_term = [&](int k) { return tmem + TM::S + (k / J) * (NN / 4) + (k % J) * 8; };  // second term NN / 8 on
        auto x_term = [&](uint32_t x, int k) { return tmem + x + k * 16; };                     // second term 8 on
        auto kq_product = [&](int c) {  // [k; q] k^T
            wait.on(kFullKQ + c % kStages, (c / kStages) & 1);
            wait.on(kKQRead, (c & 1) ^ 1);
            tc::fence_after_sync();
            if (go) {
                const uint64_t d = tc::desc(sbase + SM::KQ + (c % kStages) * SM::KQ_BYTES, 2048, 128);
#pragma unroll
                for (int k = 0; k < NK; ++k) tc::mma_f16(tmem + TM::KQ, d + k * K2, d + k * K2, ID, k > 0);
                tc::commit(bars + 8 * kKQDone);
            }
        };
        if (w.chunks > 0) kq_product(0);
#pragma unroll 1
        for (int c = 0; c < w.chunks; ++c) {
            const uint32_t par = c & 1, kq = sbase + SM::KQ + (c % kStages) * SM::KQ_BYTES;
            const uint64_t kd = tc::desc(kq, 2048, 128), td = tc::desc(sbase + SM::T + par * 16384, 1024, 128);
#pragma unroll
            for (int j = 0; j < J; ++j) {  // S k^T, as the state's columns come
                wait.on(kS + j, par);
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
            if (c + 1 < w.chunks) kq_product(c + 1);
            wait.on(kFullT + par, (c >> 1) & 1);
            wait.on(kFullV + c % kVStages, (c / kVStages) & 1);
            tc::fence_after_sync();
            if (go) {
                if (!unit) {
                    const uint64_t vd = tc::desc(sbase + SM::V + (c % kVStages) * SM::V_BYTES, 2048, 128);
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k) {  // v^T (T diag(beta))^T
                        tc::mma_f16(tmem + TM::X2, vd + k * K2, td + k * 128, ID_V, k > 0);
                        tc::mma_f16(tmem + TM::X2, vd + k * K2, td + 512 + k * 128, ID_V, 1);
                    }
                }
                tc::commit(bars + 8 * (kEmptyV + c % kVStages));
            }
#pragma unroll
            for (int k = 0; k < kC / 16; ++k) {  // - (exp(G) S k^T) (T diag(beta))^T
                wait.on(kR + k, par);
                tc::fence_after_sync();
                if (go) {
                    tc::mma_f16_ts(tmem + TM::X2, x_term(TM::X1, k), td + k * 128, ID, !unit || k > 0);
                    tc::mma_f16_ts(tmem + TM::X2, x_term(TM::X1, k), td + 512 + k * 128, ID, 1);
                    tc::mma_f16_ts(tmem + TM::X2, x_term(TM::X1, k) + 8, td + k * 128, ID, 1);
                }
            }
            if (go) tc::commit(bars + 8 * kD2);
            if (!LOCAL) {  // while the chain splits U
                wait.on(kD4Read, par ^ 1);
                tc::fence_after_sync();
                if (go) {
#pragma unroll
                    for (int k = 0; k < NK; ++k) {  // S q^T
                        tc::mma_f16_ts(tmem + TM::O, s_term(k), kd + 64 + k * K2, ID, k > 0);
                        tc::mma_f16_ts(tmem + TM::O, s_term(k) + NN / 8, kd + 64 + k * K2, ID, 1);
                    }
                    tc::commit(bars + 8 * kD3);
                }
            }
            const uint64_t kt = tc::desc(kq, 128, 2048);
#pragma unroll
            for (int k = 0; k < kC / 16; ++k) {  // the change of the state
                wait.on(kU + k, par);
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
            if (!LOCAL) {
                wait.on(kFullM + par, (c >> 1) & 1);
                wait.on(kUOut, par);
                wait.on(kD3Read, par);
                tc::fence_after_sync();
                if (go) {
                    const uint64_t md = tc::desc(sbase + SM::M + par * 16384, 1024, 128);
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k) {  // U^T M^T
                        tc::mma_f16_ts(tmem + TM::O, x_term(TM::X2, k), md + k * 128, ID, 1);
                        tc::mma_f16_ts(tmem + TM::O, x_term(TM::X2, k), md + 512 + k * 128, ID, 1);
                        tc::mma_f16_ts(tmem + TM::O, x_term(TM::X2, k) + 8, md + k * 128, ID, 1);
                    }
                    tc::commit(bars + 8 * kD4);
                }
            }
            if (go) tc::commit(bars + 8 * (kEmptyT + par));
        }
        // the last products may still read shared memory: wait for them before the CTA ends
        if (w.chunks > 0) wait.on(kEmptyT + ((w.chunks - 1) & 1), ((w.chunks - 1) >> 1) & 1);
        __syncwarp();
    } else {
        // ---- copies: lane = row of eight, 16-byte piece of four.  The first warp takes k, the second q, the third v and the gates
        const int r = lane & 7, piece = lane >> 3, which = warp - kLoadWarp;
        const void *src = which == 0 ? p.k : which == 1 ? p.q : p.v;
        const long long s0 = which == 0 ? p.ks[0] : which == 1 ? p.qs[0] : p.vs[0], s1 = which == 0 ? p.ks[1] : which == 1 ? p.qs[1] : p.vs[1];
        const char *from = static_cast<const char *>(src) + 2 * (w.b * s0 + (which < 2 ? (long long)grp * p.N : (long long)w.h * p.P + w.p0) + 8 * piece);
        // of a row of 16-byte pieces, those that exist from this lane's on; none of q in a pass without y, nor of v in a transition's
        const int width = (which == 1 && LOCAL) || (which == 2 && unit) ? 0 : (which < 2 ? p.N : rows) - 8 * piece;
        const uint32_t to = sbase + (which < 2 ? SM::KQ + which * 1024 + piece * 2048 : SM::V + piece * 128) + r * 16;
        const uint32_t stage = which < 2 ? SM::KQ_BYTES : SM::V_BYTES, row_step = which < 2 ? 128 : 2048, col_step = which < 2 ? 8192 : 512;
        const int stages = which < 2 ? kStages : kVStages, empty = which < 2 ? kEmptyKQ : kEmptyV, full = which < 2 ? kFullKQ : kFullV;
        int at = 0;
        uint32_t parity = 1;
        float graw[2] = {0.f, 0.f}, braw[2] = {0.f, 0.f};
#pragma unroll 1
        for (int c = -1; c < w.chunks; ++c) {
            if (c >= 0) {
                wait.on(empty + at, parity);  // with a place of v's, the gates four chunks back are done with too
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
            }
            if (which == 2) {
                if (c >= 0) {
                    make_gates(gates[c % kSlots], graw, braw, lane);
                    tc::mbar_arrive(bars + 8 * (kFullG + c % kSlots));
                }
#pragma unroll
                for (int m = 0; m < 2; ++m) {  // of the next chunk
                    const int t = w.t0 + (c + 1) * kC + 2 * lane + m;
                    graw[m] = load_gate<IO>(p.g, w.b * p.gs[0] + t * p.gs[1] + w.h, p.g32, t < w.t1);
                    braw[m] = load_gate<IO>(p.beta, w.b * p.bs[0] + t * p.bs[1] + w.h, p.b32, t < w.t1);
                }
            }
            if (c < 0) continue;
            cp_wait<0>();
            tc::fence_smem_to_async();
            tc::mbar_arrive(bars + 8 * (full + at));
            if (++at == stages) at = 0, parity ^= 1;
        }
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

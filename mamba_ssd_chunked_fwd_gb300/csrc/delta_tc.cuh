// delta_tc.cuh -- what the delta rule's tensor-core kernels share: a chunk's operands in
// global memory, numbers as two 16-bit terms, bounded waits.
#pragma once

#include "delta.cuh"
#include "tc_operands.cuh"
#include "tc_ptx.cuh"

namespace ssd {

constexpr int kC = kDeltaChunk;

// A chunk's gates.  With G the running sum of g: gh + gl = G log2(e), into = exp(G), out = exp(G_end - G),
// over = exp(G_end).  For fp16: the powers of two that T and M were divided by; four times the longest key.
struct alignas(16) Gates {
    float gh[kC], gl[kC], beta[kC], into[kC], neg_into[kC], out[kC];
    float over, t_unit, m_unit, k_len4;
};

// What delta_prep.cu leaves of every chunk of every head: T diag(beta) and M, both 64 x 64 in blocks of 8 rows x 16
// bytes (block (column / 8, row / 8) at (column / 8) * 1024 + (row / 8) * 128), as first terms, then second ones; the gates.
// For the gradients T itself follows.
constexpr uint32_t kOpT = 0, kOpM = 16384, kOpTerm = 8192, kOpGates = 32768, kOpPure = kOpGates + (uint32_t)sizeof(Gates);
__host__ __device__ constexpr uint32_t op_bytes(bool pure) { return kOpPure + (pure ? 16384u : 0u); }

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

// Two terms of bf16 have fp32's range; two of fp16 hold a value to 2^-22 of itself only between 2^-3 and 2^16, below that to
// 2^-25 whatever its size.  So in fp16 every operand that is computed is first multiplied by a power of two that
// comes from the largest magnitude around it, which is taken out again where the product's fp32 sums are read.  `Row`: taken of a row
// of the state (for the gradients, whose sums run over the rows, of a CTA's); `chunk`: of all of it.
//
//     S            its largest to [2^13, 2^14)                                              row
//     v, exp(G) S k^T, U over beta       the larger of v and exp(G) S |k| to [2^6, 2^7)                     row
//     exp(G_end - G) U                   the larger of exp(G_end - G) beta v and exp(G_end) S |k| to [2^6, 2^7)   row
//     D            its largest to [2^13, 2^14)                                              the CTA's rows
//     dU           its largest to [2^13, 2^14)                                              always a row
//     exp(G) d, beta exp(G) R            the largest of exp(G) d, exp(G) M^T d and exp(G_end) D |k| to [2^6, 2^7)   the CTA's rows
//     R            the larger of M^T d and D |k| to [2^6, 2^7)                             the CTA's rows
//     T, T diag(beta)                    by 2^13 (or, of expanding steps, its largest to [2^13, 2^14)), and beta by its largest   chunk
//     M            its largest to [2^13, 2^14), never down                                  chunk
//     Y, Z         their largest to [2^12, 2^13)                                            chunk
//
// with |k| four times the longest key.  Those to [2^6, 2^7) are bounds of single terms: 2^9 is left for what T makes of 64 of them (each
// at most beta |k_i| |k_j| while steps do not expand; less of it is used by as much as T is beyond 8).  What is far smaller than the
// largest keeps 2^-31 of that bound, and 2^-38 where the largest itself is known.
constexpr float kUp = 4096.f, kT = 8192.f;
__device__ __forceinline__ float inverse_power(float v) { return __uint_as_float(0x7f000000u - __float_as_uint(v)); }
// The power of two that takes a magnitude to [2, 4), 2^100 at most.
__device__ __forceinline__ float to_unit(float most) { return __uint_as_float((255u - min(max(__float_as_uint(most) >> 23, 30u), 252u)) << 23); }
// A magnitude for the largest: what is not finite poisons its own row and says nothing about the others.
__device__ __forceinline__ float finite_or_zero(float v) { return v <= 3.402823466e38f ? v : 0.f; }
template <int W>
__device__ __forceinline__ float largest(const float2 (&v)[W]) {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) most = fmaxf(most, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
    return finite_or_zero(most);
}
// The larger of both, of each half; infinities (0 * inf is NaN) and NaN drop out.
__device__ __forceinline__ __half2 larger_of_halves(__half2 most, uint32_t w) {
    const __half2 h = *reinterpret_cast<const __half2 *>(&w);
    return __hmax2(most, __hfma2(h, __float2half2_rn(0.f), __habs2(h)));
}
// Of eight rows, two tokens of them to a lane with the factors fa and fb: the largest of row lane / 4 over the warp's tokens, and
// with the factors.
__device__ __forceinline__ float2 largest_of_rows(const uint4 &a, const uint4 &b, float fa, float fb, int lane) {
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
    float2 v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = __half22float2(larger_of_halves(__float2half2_rn(0.f), aw[i])), y = __half22float2(larger_of_halves(__float2half2_rn(0.f), bw[i]));
        v[2 * i] = make_float2(fmaxf(x.x, y.x), fmaxf(fa * x.x, fb * y.x));
        v[2 * i + 1] = make_float2(fmaxf(x.y, y.y), fmaxf(fa * x.y, fb * y.y));
    }
    auto larger = [&](float2 p, float2 q, int bit) {
        return make_float2(fmaxf(p.x, __shfl_xor_sync(0xffffffffu, q.x, bit)), fmaxf(p.y, __shfl_xor_sync(0xffffffffu, q.y, bit)));
    };
#pragma unroll
    for (int half = 4, bit = 16; half >= 1; half >>= 1, bit >>= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int m = 0; m < half; ++m) v[m] = larger(up ? v[m + half] : v[m], up ? v[m] : v[m + half], bit);
    }
    v[0] = larger(v[0], v[0], 2);
    return larger(v[0], v[0], 1);
}
__device__ __forceinline__ float larger_half(__half2 v) { return fmaxf(__low2float(v), __high2float(v)); }
__device__ __forceinline__ float warp_largest(float v) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v))); }
// The power of two that a chunk's beta are divided by, the largest one's; by a warp.
__device__ __forceinline__ float beta_unit(const Gates &gt, int lane) {
    const float most = warp_largest(fmaxf(finite_or_zero(fabsf(gt.beta[lane])), finite_or_zero(fabsf(gt.beta[lane + 32]))));
    return __uint_as_float(min(max(__float_as_uint(most) >> 23, 67u), 187u) << 23);  // 2^-60 .. 2^60
}

// What a bound in [2, 4) is multiplied by: 2^5, less where T is beyond 8.
__device__ __forceinline__ float room(const Gates &gt) { return inverse_power(gt.t_unit) * (32.f / kT); }

// A thread's waits: each lasts 2000 tries of up to a millisecond; once one has given up, the rest return
// at once.  Short code: five kinds of warps run side by side, and what they run has to stay in the
// instruction cache (with unrolled loops and longer waits every second cycle went to fetching).
// Every lane of a warp calls it, and the warp goes on together: tcgen05.ld and .st and the named barriers want that, and a
// store by some of the lanes before them leaves the compiler free to run the rest apart.
// A wait that gives up: what its warp would store is NaN from then on, and a warp that only hands on (products, copies, side
// operands) hands on nothing more, so that those behind it give up too.
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
        tries = __all_sync(0xffffffffu, done) ? tries : 0u;
        asm volatile("" : "+r"(tries));  // or the code after it is laid out twice, for a thread that waits and one that does not
    }
};

// A chunk's gates where its preparation has given up: every factor of every walk's results is NaN.  By one warp.
__device__ __forceinline__ void poison(Gates &gt, int lane) {
    float *f = reinterpret_cast<float *>(&gt);
    for (int i = lane; i < (int)(sizeof(Gates) / sizeof(float)); i += 32) f[i] = __int_as_float(0x7fffffff);
}

// ex2 that stays where it is: moved into a branch on whether its result is wanted, each would wait for the one before
// (measured: 68 cycles an element in place of 20).
__device__ __forceinline__ float ex2_now(float v) {
    float r;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Global to shared memory, completing on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// 16 tokens' values, each times its factor (in fp16 and `by`), as an operand: first terms at `to`, second ones 8 columns on.
template <bool BF16>
__device__ __forceinline__ void split_scaled(const float (&x)[16], const float *f16, uint32_t to, float by = 1.f) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float4 f = *reinterpret_cast<const float4 *>(f16 + 4 * i);
        if (!BF16) f.x *= by, f.y *= by, f.z *= by, f.w *= by;
        split2<BF16>(__fmul2_rn(make_float2(x[4 * i], x[4 * i + 1]), make_float2(f.x, f.y)), hi[2 * i], lo[2 * i]);
        split2<BF16>(__fmul2_rn(make_float2(x[4 * i + 2], x[4 * i + 3]), make_float2(f.z, f.w)), hi[2 * i + 1], lo[2 * i + 1]);
    }
    tc::tmem_st8(to, hi);
    tc::tmem_st8(to + 8, lo);
}

// A pair of neighbouring tokens' values of neighbouring lanes' rows exchanged: an even lane gets its row and the next of the
// first token, an odd lane the row before and its own of the second.
template <bool BF16>
__device__ __forceinline__ uint32_t exchange_rows(float first, float second, int odd) {
    const uint32_t own = tcop::pack2(first, second, BF16), other = __shfl_xor_sync(0xffffffffu, own, 1);
    return __byte_perm(own, other, odd ? 0x3276 : 0x5410);
}

// What the walks leave of a chunk for the gradients of keys and gates, as operands in two terms: S and D by 32 rows of P,
// blocks of 8 rows x 8 columns (row group: first terms of its columns, then second ones); U and R by 32 rows of
// P, blocks of 8 rows x 8 tokens.  `unit`: chunk of a head; `row` of ptiles * 128.
template <int NN>
__device__ __forceinline__ unsigned char *state_op(float *base, size_t unit, int ptiles, int row) {
    return reinterpret_cast<unsigned char *>(base) + ((unit * ptiles * 4 + (row >> 5)) * 4 + ((row >> 3) & 3)) * (2 * NN * 16) + (row & 7) * 16;
}
__device__ __forceinline__ unsigned char *token_op(float *base, size_t unit, int ptiles, int row) {
    return reinterpret_cast<unsigned char *>(base) + ((unit * ptiles * 4 + (row >> 5)) * 4 + ((row >> 3) & 3)) * 2048 + (row & 7) * 16;
}
// 16 neighbours (two blocks) of a row; the second terms lie `lo_at` bytes on.
__device__ __forceinline__ void store_op(unsigned char *to, const uint32_t (&hi)[8], const uint32_t (&lo)[8], uint32_t lo_at) {
    *reinterpret_cast<uint4 *>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4 *>(to + 128) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
    *reinterpret_cast<uint4 *>(to + lo_at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4 *>(to + lo_at + 128) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
}

}  // namespace ssd

// delta_prep.cu -- per chunk of 64 tokens and head, what the chunked delta rule's walks
// (delta_walk_tc.cuh) read beside k, q and v, for 16-bit tensors.  With G the running sum of g in the
// chunk and W_ij = exp(G_i - G_j):
//
//     A_ij = beta_i W_ij (k_i . k_j)  (j < i),   T = (I + A)^-1,   M_ij = W_ij (q_i . k_j)  (j <= i)
//
// The products of k and q with k are one product of 128 rows on the tensor cores.  The diagonal
// blocks of 16 of T are inverted by substitution in fp32, the blocks below by
// T_ij = -T_ii sum_k A_ik T_kj with mma.sync on operands of two terms (bf16, or tf32 for fp16 tensors, whose range does not hold
// decays): blocks this small would leave
// tcgen05's 128 rows empty, and each needs the one before it.  No power of A is formed:
// with keys alike those would cancel.
//
// A kernel of its own, not warps of the walk, for rows that are cut and for the gradients: chunks are independent, eight CTAs
// share an SM, and the walks of segments and of the gradients read its results again (one row of 16384
// tokens 1058 us with it inside the walk, 877 with it apart).  Where heads fill the SMs, it costs: prompts of [4,4096,32,128,128]
// took 278 us as one kernel and take 347 as two, though the walk alone went from 278 to 213 (a third less code
// for the instruction cache).  Both forms side by side are not built.
//
// [4,4096] with 32 heads of 128 x 128, bf16 (8192 chunks): 132 us (fp16, M looked at twice and T's blocks in tf32, 150), with T for the gradients 42 us for 2048 of them.  No pipe is
// above 25 %; bound by latency (barriers, the loads, the blocks of T's first column one after another).  With k and q
// whole and T in shared memory, six CTAs to an SM: 140 and 50 us.
#include "delta_tc.cuh"

namespace ssd {

namespace {

constexpr int kThreads = 128;
constexpr int kAW = 68;  // floats between rows of A

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

// A chunk's gates by one warp, two tokens to a lane.  The running sum of g log2(e) is taken in whole
// numbers of 2^-40, exactly, and handed on as the sum of two floats: differences of far larger sums then keep
// their precision.  To and from whole numbers in halves of 32 bits: through fp64, or with floats added
// in pairs, this took 5600 of the kernel's 23000 cycles.
__device__ __forceinline__ void make_gates(Gates &gt, const float (&graw)[2], const float (&beta)[2], int lane) {
    long long sum[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        // Sums of 64 tokens stay below 2^17.  exp(1400) is infinite.  A gate that empties the state counts as -200: no growth that
        // leaves every factor of the chunk finite (a sum of 88 between any two of its tokens) brings exp(-200) back above 0
        // in fp32, and more of it makes factors that span it infinite, and what they enter infinite or NaN.
        const float g = fminf(fmaxf(graw[m], -200.f), 1400.f), hi = g * kLog2e;
        const float lo = fmaf(g, kLog2e, -hi) + g * 1.92596299e-8f;  // log2(e) - fl(log2(e))
        const float big = rintf(hi * 16384.f);
        sum[m] = ((long long)(int)big << 26) + __float2int_rn((hi * 16384.f - big) * 67108864.f + lo * 1099511627776.f);
        gt.beta[2 * lane + m] = beta[m];
    }
    const uint32_t nan0 = __ballot_sync(0xffffffffu, isnan(graw[0])), nan1 = __ballot_sync(0xffffffffu, isnan(graw[1]));
    sum[1] += sum[0];
    long long pair = sum[1];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, pair, m);
        if (lane >= m) pair += o;
    }
    sum[0] += pair - sum[1];
    sum[1] = pair;
    const long long end = __shfl_sync(0xffffffffu, pair, 31);
    auto parts = [](long long v) {  // v 2^-40 as two floats
        const int a = (int)(v >> 26), b = (int)(v & 0x3ffffff);
        const float fa = (float)a;
        return make_float2(fa * 6.103515625e-5f, fmaf((float)(a - (int)fa), 6.103515625e-5f, (float)b * 9.094947017729282e-13f));
    };
    const uint32_t before = (1u << lane) - 1u, upto = before | (1u << lane);
    const float nan = __int_as_float(0x7fffffff);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int t = 2 * lane + m;
        const float2 v = parts(sum[m]), rest = parts(end - sum[m]);
        const bool bad = (nan0 & upto) || (nan1 & (m ? upto : before));
        const float in = bad ? nan : ex2(v.x + v.y);
        gt.gh[t] = bad ? nan : v.x, gt.gl[t] = v.y, gt.into[t] = in, gt.neg_into[t] = -in;
        gt.out[t] = nan0 | nan1 ? nan : ex2(rest.x + rest.y);
    }
    const float2 all = parts(end);
    if (lane == 0) gt.over = nan0 | nan1 ? nan : ex2(all.x + all.y), gt.t_unit = gt.m_unit = gt.k_len4 = 1.f;
}

// 16 columns from j0 on of a row of products, each times its decay and the row's factor; zero from column `limit` on.
__device__ __forceinline__ void decayed(float (&v)[16], const Gates &gt, int j0, float gh, float gl, float factor, int limit) {
#pragma unroll
    for (int m = 0; m < 16; m += 4) {
        const int j = j0 + m;
        const float4 h4 = *reinterpret_cast<const float4 *>(&gt.gh[j]), l4 = *reinterpret_cast<const float4 *>(&gt.gl[j]);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const float2 minus = make_float2(-1.f, -1.f);
            const float2 d = __fadd2_rn(__ffma2_rn(e ? make_float2(h4.z, h4.w) : make_float2(h4.x, h4.y), minus, dup(gh)),
                                        __ffma2_rn(e ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y), minus, dup(gl)));
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

// The same in fp16's preparation, with two tf32 terms: A and T hold decays, which fp16 loses.  Slot t of the eight columns stands for
// column 2 t, slot t + 4 for 2 t + 1, in both operands, so that an accumulated block is an operand as it lies.
__device__ __forceinline__ uint32_t tf32_of(float v) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ void mma_16x8x8(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// acc += a X^T; `a` as it is accumulated: a[half][..], columns 8 half + 2 t + (0, 1) of rows g (0, 1) and g + 8 (2, 3).
__device__ __forceinline__ void times_transposed(float (&acc)[2][4], const float (&a)[2][4], const float *x, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t ah[4], al[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float v = a[k][(e & 1) * 2 + (e >> 1)];
            ah[e] = tf32_of(v), al[e] = tf32_of(v - __uint_as_float(ah[e]));
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float2 b = *reinterpret_cast<const float2 *>(x + (8 * half + g) * kAW + 2 * t + 8 * k);
            const uint32_t bh[2] = {tf32_of(b.x), tf32_of(b.y)};
            const uint32_t bl[2] = {tf32_of(b.x - __uint_as_float(bh[0])), tf32_of(b.y - __uint_as_float(bh[1]))};
            mma_16x8x8(acc[half], al, bh);
            mma_16x8x8(acc[half], ah, bl);
            mma_16x8x8(acc[half], ah, bh);
        }
    }
}
// A block in shared memory as an accumulated one.
__device__ __forceinline__ void load_block(float (&a)[2][4], const float *x, int lane) {
    const float *at = x + (lane >> 2) * kAW + 2 * (lane & 3);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const float2 v = *reinterpret_cast<const float2 *>(at + (m & 1) * 8 * kAW + (m >> 1) * 8);
        a[m >> 1][2 * (m & 1)] = v.x, a[m >> 1][2 * (m & 1) + 1] = v.y;
    }
}

// An 8 x 8 block of a product's result, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

// 64 columns of k (rows 0-63) and q at a time; once multiplied, A takes their place.
constexpr uint32_t kKQ = 0, kA = 0, kGates = kA + kC * kAW * 4, kSmem = 26624;  // eight CTAs to an SM, whose TMEM has places for eight
static_assert(kGates % 16 == 0 && 128 * 64 * 2 <= kGates && kGates + sizeof(Gates) <= kSmem, "shared memory");

// PURE: T itself as well, for the gradients.
template <int IO, int NN, bool PURE>
__global__ void __launch_bounds__(kThreads, 8)
delta_prep_kernel(const __grid_constant__ DeltaParams p) {
    constexpr bool BF16 = IO == IO_BF16;
    extern __shared__ __align__(1024) unsigned char sm[];
    __shared__ __align__(8) uint64_t bar_mem;
    __shared__ uint32_t tmem_slot;
    __shared__ float m_most[2], k_most[2], t_most[4];  // (fp16) the largest of M, of a key's length squared, of T, by warps
    const uint32_t sbase = tc::smem_addr(sm);
    Gates &gt = *reinterpret_cast<Gates *>(sm + kGates);
    float *A = reinterpret_cast<float *>(sm + kA);
    const int tid = threadIdx.x, pw = tid >> 5, lane = tid & 31;
    const int c = blockIdx.x % p.nc, bh = blockIdx.x / p.nc, h = bh % p.H, b = bh / p.H, grp = h / (p.H / p.G);
    const int t0 = c * kC, len = delta_length(p, b);
    if (t0 >= len) return;  // no walk comes here

    if (tid == 0) {
        tc::mbar_init(tc::smem_addr(&bar_mem), 1);
        tc::mbar_init_fence();
    }
    if (pw == 1) {
        tc::tmem_alloc(tc::smem_addr(&tmem_slot), 64);
        tc::tmem_relinquish();
    }
    float graw[2] = {0.f, 0.f}, braw[2] = {0.f, 0.f};
    if (pw == 0) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int t = t0 + 2 * lane + m;
            graw[m] = load_gate<IO>(p.g, b * p.gs[0] + t * p.gs[1] + h, p.g32, t < len);
            braw[m] = load_gate<IO>(p.beta, b * p.bs[0] + t * p.bs[1] + h, p.b32, t < len);
        }
    }
    auto load = [&](int half) {
        const int r = lane & 7, piece = lane >> 3;
#pragma unroll
        for (int rg = pw; rg < 16; rg += 4) {  // row groups of k, then of q
            const int t = t0 + (rg & 7) * 8 + r, col = 64 * half + 8 * piece;
            const char *row = static_cast<const char *>(rg < 8 ? p.k : p.q) +
                              2 * (b * (rg < 8 ? p.ks[0] : p.qs[0]) + t * (rg < 8 ? p.ks[1] : p.qs[1]) + (long long)grp * p.N + col);
            const int live = t < len ? p.N - col : 0;
#pragma unroll
            for (int cg = 0; cg < 2; ++cg)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sbase + kKQ + ((cg * 4 + piece) * 16 + rg) * 128 + r * 16),
                             "l"(live > 32 * cg ? row + 64 * cg : nullptr), "r"(live > 32 * cg ? 16 : 0) : "memory");
        }
        cp_commit();
    };
    load(0);
    if (pw == 0) make_gates(gt, graw, braw, lane);
    Waits wait{tc::smem_addr(&bar_mem)};
    uint32_t tmem = 0;
#pragma unroll 1
    for (int half = 0; half < NN / 64; ++half) {
        if (half > 0) load(half);
        cp_wait<0>();
        tc::fence_smem_to_async();
        tc::fence_before_sync();
        __syncthreads();
        tc::fence_after_sync();
        tmem = tmem_slot;
        if (tid == 0) {
            constexpr uint32_t ID = tc::idesc_f16(128, kC, BF16, false, false);
            uint64_t d = tc::desc(sbase + kKQ, 2048, 128);
#pragma unroll 1
            for (int k = 0; k < 4; ++k, d += 256) tc::mma_f16(tmem, d, d, ID, half + k > 0);
            tc::commit(tc::smem_addr(&bar_mem));
        }
        __syncwarp();
        wait.on(0, half);
        tc::fence_after_sync();
    }
    unsigned char *dst = p.ops + (size_t)blockIdx.x * op_bytes(PURE);
    {
        const uint32_t tl = tmem + (static_cast<uint32_t>(pw * 32) << 16);
        const int i = tid & 63, last = i | 31;  // of the warp's rows
        const float gh = gt.gh[i], gl = gt.gl[i], factor = pw < 2 ? gt.beta[i] : 1.f;
        const int limit = pw < 2 ? i : i + 1;
        float up = 1.f, length = 0.f;
        if constexpr (!BF16) {
            if (pw >= 2) {  // the largest of M first
                float most = 0.f;
#pragma unroll 1
                for (int j0 = 0; j0 <= last; j0 += 16) {
                    float v[16];
                    tc::tmem_ld16(tl + j0, v);
                    decayed(v, gt, j0, gh, gl, 1.f, limit);
#pragma unroll
                    for (int m = 0; m < 16; ++m) most = fmaxf(most, finite_or_zero(fabsf(v[m])));
                }
                most = warp_largest(most);
                if (lane == 0) m_most[pw - 2] = most;
                __syncwarp();
                tc::named_barrier(1, 64);
                // never down: what decays that grow push past fp16 ends as infinity, not as zeros beside it
                up = __uint_as_float((267u - min(max(__float_as_uint(fmaxf(m_most[0], m_most[1])) >> 23, 100u), 140u)) << 23);
                if (tid == 64) gt.m_unit = inverse_power(up);
                __syncwarp();
            }
        }
#pragma unroll 1
        for (int j0 = 0; j0 < kC; j0 += 16) {
            float v[16];
            uint4 *to = reinterpret_cast<uint4 *>(dst + kOpM + ((j0 >> 3) * 8 + (i >> 3)) * 128 + (i & 7) * 16);
            if (j0 > last) {  // above the diagonal: of A nothing is read, M is zero
                if (pw < 2) break;
                to[0] = to[64] = to[kOpTerm / 16] = to[kOpTerm / 16 + 64] = make_uint4(0, 0, 0, 0);
                continue;
            }
            tc::tmem_ld16(tl + j0, v);
            if constexpr (!BF16) {
#pragma unroll
                for (int m = 0; m < 16; ++m) length = j0 + m == i ? v[m] : length;
            }
            decayed(v, gt, j0, gh, gl, BF16 || pw < 2 ? factor : up, limit);
            if (pw < 2) {
#pragma unroll
                for (int m = 0; m < 16; m += 4) *reinterpret_cast<float4 *>(A + i * kAW + j0 + m) = make_float4(v[m], v[m + 1], v[m + 2], v[m + 3]);
            } else {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int m = 0; m < 8; ++m) split2<BF16>(make_float2(v[2 * m], v[2 * m + 1]), hi[m], lo[m]);
                to[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                to[64] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
                to[kOpTerm / 16] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                to[kOpTerm / 16 + 64] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
            }
        }
        if constexpr (!BF16) {
            __syncwarp();
            length = warp_largest(finite_or_zero(length));
            if (pw < 2 && lane == 0) k_most[pw] = length;
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (pw == 1) tc::tmem_dealloc(tmem, 64);
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
    __syncthreads();
    // column pw of blocks, transposed: element (c, r) of a block is T[r][c]
    {
        const int g = lane >> 2, t = lane & 3;
        const float unit = BF16 ? 1.f : inverse_power(beta_unit(gt, lane)), b0 = unit * gt.beta[16 * pw + g], b1 = unit * gt.beta[16 * pw + g + 8];
        float up = BF16 ? 1.f : kT, most = 0.f;
        // of a 16 x 16 block of T four blocks of 8 x 8, one after another along its columns, 128 bytes a warp
        auto put = [&](uint32_t op, int bi, const uint32_t(&v)[4]) {
#pragma unroll
            for (int m = 0; m < 4; ++m) *reinterpret_cast<uint32_t *>(dst + op + ((2 * pw + (m & 1)) * 8 + (m >> 1) + 2 * bi) * 128 + 4 * lane) = transposed(v[m]);
        };
        auto store = [&](float(&acc)[2][4], int bi) {  // T diag(beta) in two terms
            uint32_t hi[4], lo[4];
            if constexpr (!BF16) {
#pragma unroll
                for (int m = 0; m < 8; ++m) most = fmaxf(most, fabsf(acc[m >> 2][m & 3]));
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float b = BF16 ? (m & 1 ? b1 : b0) : up * (m & 1 ? b1 : b0);
                split2<BF16>(make_float2(b * acc[m >> 1][2 * (m & 1)], b * acc[m >> 1][2 * (m & 1) + 1]), hi[m], lo[m]);
            }
            put(kOpT, bi, hi);
            put(kOpT + kOpTerm, bi, lo);
            if (PURE) {
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float2 v = make_float2(acc[m >> 1][2 * (m & 1)], acc[m >> 1][2 * (m & 1) + 1]);
                    split2<BF16>(BF16 ? v : __fmul2_rn(dup(up), v), hi[m], lo[m]);
                }
                put(kOpPure, bi, hi);
                put(kOpPure + kOpTerm, bi, lo);
            }
        };
        // element (c, r) of block (pw, k) of the buffer, above its diagonal, will be T[r][c] of T's block (k, pw)
        float *mine = A + 16 * pw * kAW;
#pragma unroll 1
        for (int bi = 0; bi < pw; ++bi) {  // above the diagonal
            const uint32_t none[4] = {0, 0, 0, 0};
            put(kOpT, bi, none), put(kOpT + kOpTerm, bi, none);
            if (PURE) put(kOpPure, bi, none), put(kOpPure + kOpTerm, bi, none);
        }
#pragma unroll 1
        for (;;) {
            float acc[2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][e] = D[(8 * m + 2 * t + (e & 1)) * kAW + g + 8 * (e >> 1)];
            store(acc, pw);
            float first[2][4];
            Frag first_frag;
            if constexpr (BF16) first_frag = to_frag<BF16>(acc);
            else
#pragma unroll
                for (int m = 0; m < 8; ++m) first[m >> 2][m & 3] = acc[m >> 2][m & 3];
#pragma unroll 1
            for (int bi = pw + 1; bi < 4; ++bi) {
                float sum[2][4] = {};
                if constexpr (BF16) {
                    times_transposed<BF16>(sum, first_frag, A + 16 * bi * kAW + 16 * pw, lane);
#pragma unroll 1
                    for (int k = pw + 1; k < bi; ++k) times_transposed<BF16>(sum, load_frag<BF16>(mine + 16 * k, lane), A + 16 * bi * kAW + 16 * k, lane);
                } else {
                    times_transposed(sum, first, A + 16 * bi * kAW + 16 * pw, lane);
#pragma unroll 1
                    for (int k = pw + 1; k < bi; ++k) {
                        float block[2][4];
                        load_block(block, mine + 16 * k, lane);
                        times_transposed(sum, block, A + 16 * bi * kAW + 16 * k, lane);
                    }
                }
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[m][e] = -sum[m][e], acc[m][e] = 0.f;
                if constexpr (BF16) times_transposed<BF16>(acc, to_frag<BF16>(sum), A + 16 * bi * kAW + 16 * bi, lane);
                else times_transposed(acc, sum, A + 16 * bi * kAW + 16 * bi, lane);
                store(acc, bi);
                if (bi < 3) {
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        *reinterpret_cast<float2 *>(mine + 16 * bi + (g + 8 * (m & 1)) * kAW + 2 * t + 8 * (m >> 1)) =
                            make_float2(acc[m >> 1][2 * (m & 1)], acc[m >> 1][2 * (m & 1) + 1]);
                    __syncwarp();
                }
            }
            if constexpr (BF16) break;
            // steps that expand (beta |k|^2 > 2) may leave T above 8: once more, by its largest
            most = warp_largest(most);
            if (lane == 0) t_most[pw] = most;
            __syncthreads();
            most = fmaxf(fmaxf(t_most[0], t_most[1]), fmaxf(t_most[2], t_most[3]));
            if (!(most * up > 65504.f) || most > 3e38f || up < kT) break;
            up = to_unit(most) * kUp;
            __syncthreads();
        }
        if constexpr (!BF16) {
            if (tid == 0) {
                gt.t_unit = inverse_power(up);
                gt.k_len4 = 4.f * sqrtf(fmaxf(k_most[0], k_most[1]));
            }
        }
    }
    if (wait.dead()) poison(gt, lane);
    tc::fence_smem_to_async();
    __syncthreads();
    if (tid == 0) {
        bulk_store(dst + kOpGates, sbase + kGates, (uint32_t)sizeof(Gates));
        tc::bulk_commit();
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // shared memory is read; the grid's end covers the rest
    }
}

template <int IO, int NN, bool PURE>
cudaError_t prep_as(const DeltaParams &p, cudaStream_t s) {
    auto *kernel = delta_prep_kernel<IO, NN, PURE>;
    const cudaError_t e = allow_smem<kSmem>(kernel);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)((long long)p.B * p.H * p.nc), kThreads, kSmem, s>>>(p);
    return cudaGetLastError();
}

template <int IO>
cudaError_t prep_io(const DeltaParams &p, bool pure, cudaStream_t s) {
    if (pure) return p.N <= 64 ? prep_as<IO, 64, true>(p, s) : prep_as<IO, 128, true>(p, s);
    return p.N <= 64 ? prep_as<IO, 64, false>(p, s) : prep_as<IO, 128, false>(p, s);
}

}  // namespace

size_t delta_op_bytes(bool pure) { return op_bytes(pure); }

cudaError_t launch_delta_prep(const DeltaParams &p, int io, bool pure, cudaStream_t s) {
    return io == IO_BF16 ? prep_io<IO_BF16>(p, pure, s) : prep_io<IO_F16>(p, pure, s);
}

}  // namespace ssd

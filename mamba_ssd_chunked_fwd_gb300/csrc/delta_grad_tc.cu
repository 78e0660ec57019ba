// delta_grad_tc.cu -- delta_grad.cu's gradients on the tensor cores, for 16-bit tensors: from the
// state S before a chunk, the adjoint D after it, U and R, which delta_tc.cu and delta_adj.cu leave as
// operands (two 16-bit terms each, in blocks of 8 rows x 16 bytes).  The formulas stand there.
//
// Everything is transposed, so that a head's N columns are the 128 lanes of TMEM (or, of the products
// between tokens, the 64 tokens j), and the tokens i its columns:
//
//     P1 = S^T d^T,  P2 = S^T R^T,  P3 = D^T U^T          [N x 64], over P
//     X4 = U d^T,    X5 = U R^T,    X6 = V R^T (its diagonal)   [64 x 64], over P
//     KK = K K^T,    KQ = K Q^T                            [64 x 64], over N
//     Y[j][i] = scale W_ij X4[j][i],  Z[j][i] = beta_i W_ij X5[j][i]
//     dq^T = scale exp(G_i) P1 + K^T Y
//     dk^T = -beta_i exp(G_i) P2 + exp(G_end - G_i) P3 - K^T (Z + Z^T) + Q^T Y^T
//
// [4,2048] with 16 heads of 128 x 128, bf16 (2048 chunks): 183 us, 2.9 TB/s of operands read.  A chunk's 22000 cycles are products
// 7000 (both operands from shared memory: 56 cycles each), waits for S and D 3000, Y and Z 3000, sums over N 2600, second
// products and stores 3500; with 16 warps in place of 8 the same.  In fp16, Y and Z made twice, once for their largest, 203 us.  TMEM is full, so that two chunks do not overlap.
//
// Y and Z lie in shared memory once: read along j they are an operand, read along i its transpose.
// A CTA takes one chunk of one head after another; while its warps finish one, the next one's tiles are copied:
//
//   8 warps  Y, Z, the sums over N and the stores: thread = lane, half of the tokens
//   1 warp   issues the products;  3 warps copy (k and q; S, D, U, R, dy and v by 32 of the P rows, a warp to
//            a stage: with one for both, a stage's copies began when the other's had landed)
#include <math.h>

#include "delta_tc.cuh"

namespace ssd {

namespace {

constexpr int kMathWarps = 8, kMmaWarp = kMathWarps, kCopyWarp = kMmaWarp + 1;
constexpr int kStages = 2, kRowsP = 32;  // rows of P in a stage
constexpr int kThreads = (kCopyWarp + 1 + kStages) * 32;

template <int NN>
struct Smem {
    // a stage: S and D (32 rows x NN, two terms), U and R (32 rows x 64, two terms), dy and v (64 rows x 32)
    static constexpr uint32_t ST = kRowsP * NN * 2 * 2, UT = kRowsP * kC * 2 * 2, VT = kRowsP * kC * 2;
    static constexpr uint32_t S = 0, D = ST, U = 2 * ST, R = U + UT, DY = R + UT, V = DY + VT, STAGE = V + VT;
    static constexpr uint32_t KQ = kStages * STAGE, KQ_BYTES = 128 * NN * 2;
    static constexpr uint32_t YZ = KQ + 2 * KQ_BYTES;  // Y, -Z: two terms of 8 KB each
    static constexpr uint32_t GATES = YZ + 32768, SUMS = GATES + 2 * (uint32_t)sizeof(Gates), BYTES = SUMS + 4096 + 2048;
};

enum Bar { kFull = 0, kEmpty = kFull + kStages, kFullKQ = kEmpty + kStages, kEmptyKQ = kFullKQ + 2, kX = kEmptyKQ + 2, kYZ, kIn, kOut, kDone, kScaled, kDrain = kScaled + kStages, kBars };

template <int NN>
struct Tm {  // columns
    static constexpr uint32_t P1 = 0, P2 = 64, P3 = 128, X4 = 192, X5 = 256, X6 = 320, KK = 384;  // KK and KQ: 128
};

// Sums over a warp's lanes of 16 numbers each: lane l ends with that of number l >> 1.
__device__ __forceinline__ float sum_columns(float (&v)[16], int lane) {
#pragma unroll
    for (int half = 8, bit = 16; half >= 1; half >>= 1, bit >>= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int m = 0; m < half; ++m) {
            const float keep = up ? v[m + half] : v[m], send = up ? v[m] : v[m + half];
            v[m] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

template <int IO, int NN>
__global__ void __launch_bounds__(kThreads, 1)
delta_grad_tc_kernel(const __grid_constant__ DeltaParams p) {
    constexpr bool BF16 = IO == IO_BF16;
    using SM = Smem<NN>;
    using TM = Tm<NN>;
    extern __shared__ __align__(1024) unsigned char sm[];
    __shared__ __align__(8) uint64_t bar_mem[kBars];
    __shared__ uint32_t tmem_slot;
    const uint32_t sbase = tc::smem_addr(sm), bars = tc::smem_addr(bar_mem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ptiles = (p.P + 127) / 128, steps = ptiles * 4, units = p.B * p.H * p.nc;
    // fp16: the operands come times powers of two, of each 128 rows of P (delta_tc.cuh).  Where those of several differ, what has
    // the larger one is brought down in place
    constexpr bool UNITS = !BF16;
    const bool level = UNITS && ptiles > 1;

    if (tid == 0) {
        auto init = [&](int bar, int count, uint32_t arrivals) {
            for (int i = 0; i < count; ++i) tc::mbar_init(bars + 8 * (bar + i), arrivals);
        };
        init(kFull, kStages, 33), init(kEmpty, kStages, 1 + kMathWarps * 32), init(kFullKQ, 2, 33), init(kEmptyKQ, 2, 1 + kMathWarps * 32);
        init(kX, 1, 1), init(kYZ, 1, 128), init(kIn, 1, kMathWarps * 32), init(kOut, 1, 1), init(kDone, 1, kMathWarps * 32);
        init(kScaled, kStages, kMathWarps * 32), init(kDrain, 1, 1);
        tc::mbar_init_fence();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(tc::smem_addr(&tmem_slot), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's, so they begin at column 0
    Waits wait{bars};
    // units in turn; those behind their row's end have nothing but zeros to store
    auto tokens_of = [&](int unit) {
        const int c = unit % p.nc, b = unit / p.nc / p.H;
        return min(max(delta_length(p, b) - c * kC, 0), kC);
    };

    if (warp < kMathWarps) {
        const int quarter = warp & 3, half = warp >> 2, row = quarter * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + 32 * half;
        float *part = reinterpret_cast<float *>(sm + SM::SUMS);  // [5][4 quarters][64]: sums over lanes
        float *once = part + 5 * 4 * kC;                         // [3][64]: a thread's sums of its columns, by halves; r . v
        float *sds = once + 3 * kC;                              // [8]: shares of <S, D>; two sums over 32 tokens; [8]: the largest of Y and Z
        const bool shared_keys = p.H > p.G;
        int n_unit = 0, stage_count = 0;
#pragma unroll 1
        for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
            const int n = tokens_of(unit), c = unit % p.nc, bh = unit / p.nc, h = bh % p.H, b = bh / p.H, grp = h / (p.H / p.G);
            const int t0 = c * kC, tokens = min(kC, p.L - t0);
            if (n == 0) {
                for (int e = tid; e < tokens * p.N; e += kMathWarps * 32) {
                    const long long t = (long long)b * p.L + t0 + e / p.N;
                    const int col = e % p.N;
                    if (shared_keys) p.dqh[(t * p.H + h) * p.N + col] = p.dkh[(t * p.H + h) * p.N + col] = 0.f;
                    else st_io<IO>(p.dq, (t * p.G + grp) * p.N + col, 0.f), st_io<IO>(p.dk, (t * p.G + grp) * p.N + col, 0.f);
                }
                if (tid < tokens) {
                    store_gate<IO>(p.dg, ((long long)b * p.L + t0 + tid) * p.H + h, p.g32, 0.f);
                    store_gate<IO>(p.dbeta, ((long long)b * p.L + t0 + tid) * p.H + h, p.b32, 0.f);
                }
                continue;
            }
            const uint32_t par = n_unit & 1;
            const unsigned char *kq = sm + SM::KQ + (n_unit & 1) * SM::KQ_BYTES;
            const Gates &gt = *reinterpret_cast<const Gates *>(sm + SM::GATES + (n_unit & 1) * sizeof(Gates));
            float4 held = make_float4(1.f, 1.f, 1.f, 1.f);  // what S, U, D and R are held times
            if constexpr (UNITS) {
                held = __ldg(reinterpret_cast<const float4 *>(p.units) + (size_t)unit * ptiles);
                for (int m = 1; m < ptiles; ++m) {
                    const float4 x = __ldg(reinterpret_cast<const float4 *>(p.units) + (size_t)unit * ptiles + m);
                    held = make_float4(fminf(held.x, x.x), fminf(held.y, x.y), fminf(held.z, x.z), fminf(held.w, x.w));
                }
            }
            // <S, D>, as the tiles pass
            float sd = 0.f;
#pragma unroll 1
            for (int s = 0; s < steps; ++s, ++stage_count) {
                const int at = stage_count % kStages;
                wait.on(kFull + at, (stage_count / kStages) & 1);
                unsigned char *st = sm + at * SM::STAGE;
                if constexpr (UNITS) {
                    if (level) {
                        const float4 own = __ldg(reinterpret_cast<const float4 *>(p.units) + (size_t)unit * ptiles + s / 4);
                        auto bring = [&](uint32_t from, uint32_t bytes, float to, float was) {
                            const __half2 f = __float2half2_rn(to * inverse_power(was));
                            for (uint32_t e = 16 * tid; e < bytes; e += 16 * kMathWarps * 32) {
                                uint4 v = *reinterpret_cast<const uint4 *>(st + from + e);
                                uint32_t *x = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                                for (int m = 0; m < 4; ++m) {
                                    const __half2 h = __hmul2(*reinterpret_cast<const __half2 *>(&x[m]), f);
                                    x[m] = *reinterpret_cast<const uint32_t *>(&h);
                                }
                                *reinterpret_cast<uint4 *>(st + from + e) = v;
                            }
                        };
                        bring(SM::S, SM::ST, held.x, own.x), bring(SM::U, SM::UT, held.y, own.y);
                        bring(SM::D, SM::ST, held.z, own.z), bring(SM::R, SM::UT, held.w, own.w);
                        tc::fence_smem_to_async();
                        tc::mbar_arrive(bars + 8 * (kScaled + at));
                        __syncwarp();
                        tc::named_barrier(1, kMathWarps * 32);  // the rows that another thread brought down
                    }
                }
#pragma unroll 1
                for (int e = tid; e < kRowsP * NN / 8; e += kMathWarps * 32) {  // 16 bytes: row group, then columns' group and row
                    const uint32_t off = (e / NN) * (2 * NN * 16) + (e % NN) * 16;
                    const uint4 a = *reinterpret_cast<const uint4 *>(st + SM::S + off), al = *reinterpret_cast<const uint4 *>(st + SM::S + off + NN * 16),
                                d = *reinterpret_cast<const uint4 *>(st + SM::D + off), dl = *reinterpret_cast<const uint4 *>(st + SM::D + off + NN * 16);
                    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, alw[4] = {al.x, al.y, al.z, al.w}, dw[4] = {d.x, d.y, d.z, d.w}, dlw[4] = {dl.x, dl.y, dl.z, dl.w};
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const float2 x = __fadd2_rn(unpack2<BF16>(aw[m]), unpack2<BF16>(alw[m])), y = __fadd2_rn(unpack2<BF16>(dw[m]), unpack2<BF16>(dlw[m]));
                        sd = fmaf(x.x, y.x, fmaf(x.y, y.y, sd));
                    }
                }
                tc::fence_smem_to_async();  // or a load still under way reads what the next copy writes
                tc::mbar_arrive(bars + 8 * (kEmpty + at));
            }
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) sd += __shfl_xor_sync(0xffffffffu, sd, m);
            if (lane == 0) sds[warp] = wait.dead() ? __int_as_float(0x7fffffff) : sd;
            wait.on(kFullKQ + (n_unit & 1), (n_unit >> 1) & 1);  // the gates
            wait.on(kX, par);
            tc::fence_after_sync();
            // what the sums over P carry: of S, U (over the largest beta), R, D
            const float of_s = inverse_power(held.x), of_u = UNITS ? inverse_power(held.y) * beta_unit(gt, lane) : 1.f, of_d = inverse_power(held.z),
                        of_r = inverse_power(held.w);
            // 16 tokens i of row j of Y and Z, and what dbeta takes off before beta and k . k
            auto make_yz = [&](int j, int i, float gh, float gl, float(&y)[16], float(&z)[16], float(&wx)[16]) {
#pragma unroll
                for (int m = 0; m < 16; ++m) {
                    const float w = ex2_now((gt.gh[i + m] - gh) + (gt.gl[i + m] - gl));
                    const float x4 = UNITS ? of_u * y[m] : y[m], x5 = UNITS ? of_u * of_r * z[m] : z[m];
                    y[m] = i + m >= j ? p.scale * w * x4 : 0.f, wx[m] = i + m > j ? w * x5 : 0.f, z[m] = gt.beta[i + m] * wx[m];
                }
            };
            float up = 1.f;
            if constexpr (UNITS) {
                if (quarter < 2) {
                    float most = 0.f;
#pragma unroll 1
                    for (int i0 = 0; i0 < 32; i0 += 16) {
                        float y[16], z[16], wx[16];
                        tc::tmem_ld16x2(tl + TM::X4 + i0, tl + TM::X5 + i0, y, z);
                        make_yz(row, 32 * half + i0, gt.gh[row], gt.gl[row], y, z, wx);
#pragma unroll
                        for (int m = 0; m < 16; ++m) most = fmaxf(most, fmaxf(finite_or_zero(fabsf(y[m])), finite_or_zero(fabsf(z[m]))));
                    }
                    most = warp_largest(most);
                    if (lane == 0) sds[kMathWarps + 2 + warp] = most;
                }
                __syncwarp();
                tc::named_barrier(1, kMathWarps * 32);
                const float *most = sds + kMathWarps + 2;  // warps 0, 1, 4 and 5
                up = fminf(to_unit(fmaxf(fmaxf(most[0], most[1]), fmaxf(most[4], most[5]))), 1.152921504606847e18f) * (kUp / 2.f);
            }
            if (quarter < 2) {  // lanes 0-63: Y and Z, thread = token j, columns = tokens i of this half
                const int j = row;
                const float gh = gt.gh[j], gl = gt.gl[j];
                float col_e = 0.f;
#pragma unroll 1
                for (int i0 = 0; i0 < 32; i0 += 16) {
                    const int i = 32 * half + i0;
                    float x4[16], x5[16], wx[16], kk[16], kqv[16];
                    tc::tmem_ld16x2(tl + TM::X4 + i0, tl + TM::X5 + i0, x4, x5);
                    tc::tmem_ld16x2(tl + TM::KK + i0, tl + TM::KK + 64 + i0, kk, kqv);
                    uint32_t yh[8], yl[8], zh[8], zl[8];
                    make_yz(j, i, gh, gl, x4, x5, wx);
#pragma unroll
                    for (int m = 0; m < 16; ++m) {
                        const float e = i + m > j ? x4[m] * kqv[m] - x5[m] * kk[m] : 0.f;
                        kk[m] = wx[m] * kk[m];  // what dbeta takes off
                        kqv[m] = e;
                        col_e += e;
                    }
#pragma unroll
                    for (int m = 0; m < 8; ++m) {
                        const float2 y = make_float2(x4[2 * m], x4[2 * m + 1]), z = make_float2(-x5[2 * m], -x5[2 * m + 1]);
                        split2<BF16>(UNITS ? __fmul2_rn(dup(up), y) : y, yh[m], yl[m]);
                        split2<BF16>(UNITS ? __fmul2_rn(dup(up), z) : z, zh[m], zl[m]);
                    }
                    const uint32_t to = sbase + SM::YZ + (i >> 3) * 1024 + (j >> 3) * 128 + (j & 7) * 16;
                    tcop::st_shared_v4(to, yh[0], yh[1], yh[2], yh[3]);
                    tcop::st_shared_v4(to + 1024, yh[4], yh[5], yh[6], yh[7]);
                    tcop::st_shared_v4(to + 8192, yl[0], yl[1], yl[2], yl[3]);
                    tcop::st_shared_v4(to + 8192 + 1024, yl[4], yl[5], yl[6], yl[7]);
                    tcop::st_shared_v4(to + 16384, zh[0], zh[1], zh[2], zh[3]);
                    tcop::st_shared_v4(to + 16384 + 1024, zh[4], zh[5], zh[6], zh[7]);
                    tcop::st_shared_v4(to + 24576, zl[0], zl[1], zl[2], zl[3]);
                    tcop::st_shared_v4(to + 24576 + 1024, zl[4], zl[5], zl[6], zl[7]);
                    const float se = sum_columns(kqv, lane), sp = sum_columns(kk, lane);
                    if (!(lane & 1)) part[(3 * 4 + quarter) * kC + i + (lane >> 1)] = se, part[(4 * 4 + quarter) * kC + i + (lane >> 1)] = sp;
                    __syncwarp();
                    // r . v: the diagonal
                    tc::tmem_ld16(tl + TM::X6 + i0, x4);
                    float rv = 0.f;
#pragma unroll
                    for (int m = 0; m < 16; ++m) rv = i + m == j ? x4[m] : rv;
                    if (j >= i && j < i + 16) once[2 * kC + j] = UNITS ? of_r * rv : rv;
                    __syncwarp();
                }
                once[half * kC + j] = col_e;
                tc::fence_smem_to_async();
                tc::fence_before_sync();
                tc::mbar_arrive(bars + 8 * kYZ);
            }
            // P1, P2, P3: their sums with q and k over N, and what they give to dq and dk
            const unsigned char *kp = kq + (row >> 3) * 2048 + (row & 7) * 2;  // column `row` of k
            const bool col_ok = row < NN;
#pragma unroll 1
            for (int i0 = 0; i0 < 32; i0 += 16) {
                const int i = 32 * half + i0;
                float p1[16], p2[16], p3[16], t1[16], t2[16], t3[16];
                tc::tmem_ld16x2(tl + TM::P1 + i0, tl + TM::P2 + i0, p1, p2);
                tc::tmem_ld16(tl + TM::P3 + i0, p3);
                uint32_t r1[16], r2[16];
#pragma unroll
                for (int m = 0; m < 16; ++m) {
                    uint16_t kraw = 0, qraw = 0;
                    if (col_ok) {
                        kraw = *reinterpret_cast<const uint16_t *>(kp + ((i + m) >> 3) * 128 + ((i + m) & 7) * 16);
                        qraw = *reinterpret_cast<const uint16_t *>(kp + 1024 + ((i + m) >> 3) * 128 + ((i + m) & 7) * 16);
                    }
                    const float k = BF16 ? __uint_as_float((uint32_t)kraw << 16) : __half2float(__ushort_as_half(kraw));
                    const float q = BF16 ? __uint_as_float((uint32_t)qraw << 16) : __half2float(__ushort_as_half(qraw));
                    const float into = gt.into[i + m], f1 = p.scale * into, f2 = -gt.beta[i + m] * into, f3 = gt.out[i + m];
                    if (UNITS) p1[m] *= of_s, p2[m] *= of_s * of_r, p3[m] *= of_d * of_u;
                    t1[m] = col_ok ? f1 * q * p1[m] + f2 * k * p2[m] : 0.f;
                    t2[m] = col_ok ? into * k * p2[m] : 0.f;
                    t3[m] = col_ok ? f3 * k * p3[m] : 0.f;
                    r1[m] = __float_as_uint(UNITS ? up * (f1 * p1[m]) : f1 * p1[m]);
                    const float dk = fmaf(f3, p3[m], f2 * p2[m]);
                    r2[m] = __float_as_uint(UNITS ? up * dk : dk);
                }
                tc::tmem_st16(tl + TM::P1 + i0, r1);
                tc::tmem_st16(tl + TM::P2 + i0, r2);
                const float s1 = sum_columns(t1, lane), s2 = sum_columns(t2, lane), s3 = sum_columns(t3, lane);
                if (!(lane & 1)) {
                    const int at = i + (lane >> 1);
                    part[quarter * kC + at] = s1, part[(4 + quarter) * kC + at] = s2, part[(8 + quarter) * kC + at] = s3;
                }
                __syncwarp();
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(bars + 8 * kIn);
            tc::named_barrier(1, kMathWarps * 32);  // the sums
            if (tid < kC) {
                auto lanes = [&](int which, int at) {
                    const float *x = part + which * 4 * kC + at;
                    return (x[0] + x[kC]) + (x[2 * kC] + x[3 * kC]);
                };
                auto tokens2 = [&](int which, int at) { return part[which * 4 * kC + at] + part[(which * 4 + 1) * kC + at]; };
                const float dbeta = once[2 * kC + tid] - lanes(1, tid) - tokens2(4, tid);
                float total = 0.f;
#pragma unroll
                for (int m = 0; m < kMathWarps; ++m) total += sds[m];
                if (UNITS) total *= of_s * of_d;
                // sums over the tokens before, and from this one on: over a warp, then over both
                float w = lanes(2, tid), x = lanes(0, tid) + (tokens2(3, tid) - (once[tid] + once[kC + tid]));
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const float down = __shfl_up_sync(0xffffffffu, w, m), up = __shfl_down_sync(0xffffffffu, x, m);
                    if (lane >= m) w += down;
                    if (lane + m < 32) x += up;
                }
                float *over = sds + kMathWarps;
                if (tid == 31) over[0] = w;
                if (tid == 32) over[1] = x;
                __syncwarp();
                tc::named_barrier(2, kC);
                const float left = __shfl_up_sync(0xffffffffu, w, 1);
                const float before = (lane > 0 ? left : 0.f) + (tid >= 32 ? over[0] : 0.f), after = x + (tid < 32 ? over[1] : 0.f);
                if (tid < tokens) {
                    const long long at = ((long long)b * p.L + t0 + tid) * p.H + h;
                    const float bad = wait.dead() ? __int_as_float(0x7fffffff) : 0.f;
                    store_gate<IO>(p.dg, at, p.g32, tid < n ? gt.over * total + before + after + bad : 0.f);
                    store_gate<IO>(p.dbeta, at, p.b32, tid < n ? dbeta + bad : 0.f);
                }
            }
            // dq and dk
            wait.on(kOut, par);
            tc::fence_after_sync();
            const int odd = lane & 1;
            const float bad = wait.dead() ? __int_as_float(0x7fffffff) : 0.f;
            const long long t = (long long)b * p.L + t0 + 32 * half;
            const size_t step = (size_t)(shared_keys ? p.H : p.G) * p.N;
#pragma unroll 1
            for (int which = 0; which < 2; ++which) {
                float *share = (which ? p.dkh : p.dqh) + t * step + (size_t)h * p.N + row;
                uint16_t *out = static_cast<uint16_t *>(which ? p.dk : p.dq) + (t + odd) * step + (size_t)grp * p.N + row - odd;
#pragma unroll 1
                for (int i0 = 0; i0 < 32; i0 += 16) {
                    float v[16];
                    tc::tmem_ld16(tl + (which ? TM::P2 : TM::P1) + i0, v);
                    const int i = 32 * half + i0, left = row < p.N ? tokens - i : 0;
                    if (UNITS) {
#pragma unroll
                        for (int m = 0; m < 16; ++m) v[m] *= inverse_power(up);
                    }
                    if (i + 16 > n) {
#pragma unroll
                        for (int m = 0; m < 16; ++m) v[m] = i + m < n ? v[m] : 0.f;
                    }
#pragma unroll
                    for (int m = 0; m < 16; m += 2) {
                        if (shared_keys) {
                            if (m < left) share[0] = v[m] + bad;
                            if (m + 1 < left) share[step] = v[m + 1] + bad;
                            share += 2 * step;
                        } else {
                            const uint32_t two = exchange_rows<BF16>(v[m] + bad, v[m + 1] + bad, odd);
                            if (m + odd < left) *reinterpret_cast<uint32_t *>(out) = two;
                            out += 2 * step;
                        }
                    }
                }
            }
            __syncwarp();
            tc::fence_before_sync();
            tc::mbar_arrive(bars + 8 * (kEmptyKQ + (n_unit & 1)));
            tc::mbar_arrive(bars + 8 * kDone);
            tc::named_barrier(1, kMathWarps * 32);  // the sums' places are free
            ++n_unit;
        }
    } else if (warp == kMmaWarp) {
        const bool go = tc::elect_one();
        // transposed operands: A and B along their rows (MN-major) unless said otherwise
        constexpr uint32_t I_AB = tc::idesc_f16(128, kC, BF16, true, true), I_A = tc::idesc_f16(128, kC, BF16, true, false),
                           I_B = tc::idesc_f16(128, kC, BF16, false, true), I_KQ = tc::idesc_f16(128, 128, BF16, false, false);
        constexpr uint32_t SL = NN * 16 / 16, UL = 1024 / 16;  // second terms of S and D; of U and R
        int n_unit = 0, stage_count = 0;
#pragma unroll 1
        for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
            if (tokens_of(unit) == 0) continue;
            const uint32_t par = n_unit & 1, kq = sbase + SM::KQ + par * SM::KQ_BYTES;
            wait.on(kFullKQ + par, (n_unit >> 1) & 1);
            wait.on(kDone, par ^ 1);  // the unit before has been read
            if (wait.dead()) goto given_up;
            tc::fence_after_sync();
            if (go) {
                const uint64_t d = tc::desc(kq, 2048, 128);
#pragma unroll 1
                for (int k = 0; k < NN / 16; ++k) tc::mma_f16(tmem + TM::KK, d + k * 256, d + k * 256, I_KQ, k > 0);
            }
#pragma unroll 1
            for (int s = 0; s < steps; ++s, ++stage_count) {
                const int at = stage_count % kStages;
                const uint32_t st = sbase + at * SM::STAGE;
                wait.on(kFull + at, (stage_count / kStages) & 1);
                if (level) wait.on(kScaled + at, (stage_count / kStages) & 1);
                if (wait.dead()) goto given_up;
                tc::fence_after_sync();
                if (go) {
                    const uint64_t sd = tc::desc(st + SM::S, 2 * NN * 16, 128), dd = tc::desc(st + SM::D, 2 * NN * 16, 128);
                    const uint64_t ud = tc::desc(st + SM::U, 2048, 128), rd = tc::desc(st + SM::R, 2048, 128);
                    const uint64_t yd = tc::desc(st + SM::DY, 1024, 128), vd = tc::desc(st + SM::V, 1024, 128);
#pragma unroll 1
                    for (int k = 0; k < kRowsP / 16; ++k) {  // 16 rows of P: two groups of 8
                        const uint32_t on = s + k > 0, ks = k * 2 * 2 * NN, ku = k * 2 * 128, kv = k * 2 * 64;
                        tc::mma_f16(tmem + TM::P1, sd + ks, yd + kv, I_A, on);
                        tc::mma_f16(tmem + TM::P1, sd + ks + SL, yd + kv, I_A, 1);
                        tc::mma_f16(tmem + TM::P2, sd + ks, rd + ku, I_AB, on);
                        tc::mma_f16(tmem + TM::P2, sd + ks, rd + ku + UL, I_AB, 1);
                        tc::mma_f16(tmem + TM::P2, sd + ks + SL, rd + ku, I_AB, 1);
                        tc::mma_f16(tmem + TM::P3, dd + ks, ud + ku, I_AB, on);
                        tc::mma_f16(tmem + TM::P3, dd + ks, ud + ku + UL, I_AB, 1);
                        tc::mma_f16(tmem + TM::P3, dd + ks + SL, ud + ku, I_AB, 1);
                        // rows 64-127 of these operands are what lies behind the 64 tokens; nothing reads those lanes
                        tc::mma_f16(tmem + TM::X4, ud + ku, yd + kv, I_A, on);
                        tc::mma_f16(tmem + TM::X4, ud + ku + UL, yd + kv, I_A, 1);
                        tc::mma_f16(tmem + TM::X5, ud + ku, rd + ku, I_AB, on);
                        tc::mma_f16(tmem + TM::X5, ud + ku, rd + ku + UL, I_AB, 1);
                        tc::mma_f16(tmem + TM::X5, ud + ku + UL, rd + ku, I_AB, 1);
                        tc::mma_f16(tmem + TM::X6, vd + kv, rd + ku, I_B, on);
                        tc::mma_f16(tmem + TM::X6, vd + kv, rd + ku + UL, I_B, 1);
                    }
                    tc::commit(bars + 8 * (kEmpty + at));
                }
            }
            if (go) tc::commit(bars + 8 * kX);
            wait.on(kYZ, par);
            wait.on(kIn, par);
            if (wait.dead()) goto given_up;
            tc::fence_after_sync();
            if (go) {
                const uint64_t kt = tc::desc(kq, 128, 2048), qt = kt + 64;  // k^T, q^T as first operands: 16 tokens are 256 bytes
                const uint64_t along_i = tc::desc(sbase + SM::YZ, 128, 1024), along_j = tc::desc(sbase + SM::YZ, 1024, 128);
                constexpr uint32_t LO = 8192 / 16, Z = 16384 / 16;
#pragma unroll 1
                for (int k = 0; k < kC / 16; ++k) {
                    const uint64_t ka = kt + k * 16, qa = qt + k * 16, bi = along_i + k * 16, bj = along_j + k * 128;
                    tc::mma_f16(tmem + TM::P1, ka, bi, I_AB, 1);
                    tc::mma_f16(tmem + TM::P1, ka, bi + LO, I_AB, 1);
                    tc::mma_f16(tmem + TM::P2, ka, bi + Z, I_AB, 1);
                    tc::mma_f16(tmem + TM::P2, ka, bi + Z + LO, I_AB, 1);
                    tc::mma_f16(tmem + TM::P2, ka, bj + Z, I_A, 1);
                    tc::mma_f16(tmem + TM::P2, ka, bj + Z + LO, I_A, 1);
                    tc::mma_f16(tmem + TM::P2, qa, bj, I_A, 1);
                    tc::mma_f16(tmem + TM::P2, qa, bj + LO, I_A, 1);
                }
                tc::commit(bars + 8 * kOut);
                tc::commit(bars + 8 * (kEmptyKQ + par));
            }
            ++n_unit;
        }
    given_up:
        // the last products may still read shared memory: wait for them before the CTA ends
        if (go) tc::commit(bars + 8 * kDrain);
        Waits{bars}.on(kDrain, 0);
    } else if (warp == kCopyWarp) {
        // ---- k, q and the gates
        const int r = lane & 7, piece = lane >> 3;
        int n_unit = 0;
#pragma unroll 1
        for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
            const int n = tokens_of(unit), c = unit % p.nc, bh = unit / p.nc, h = bh % p.H, b = bh / p.H, grp = h / (p.H / p.G);
            if (n == 0) continue;
            const uint32_t at = n_unit & 1, bar = bars + 8 * (kFullKQ + at);
            wait.on(kEmptyKQ + at, ((n_unit >> 1) & 1) ^ 1);
            if (wait.dead()) break;
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(bar, (uint32_t)sizeof(Gates));
                bulk_load(sbase + SM::GATES + at * (uint32_t)sizeof(Gates), p.ops + (size_t)unit * op_bytes(true) + kOpGates, (uint32_t)sizeof(Gates), bar);
            }
            __syncwarp();
#pragma unroll 1
            for (int rg = 0; rg < 16; ++rg) {  // row groups of k, then of q
                const int i = (rg & 7) * 8 + r, t = c * kC + i;
                const char *src = static_cast<const char *>(rg < 8 ? p.k : p.q) +
                                  2 * (b * (rg < 8 ? p.ks[0] : p.qs[0]) + t * (rg < 8 ? p.ks[1] : p.qs[1]) + (long long)grp * p.N + 8 * piece);
                const int live = i < n ? p.N - 8 * piece : 0;
#pragma unroll
                for (int cg = 0; cg < NN / 32; ++cg)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sbase + SM::KQ + at * SM::KQ_BYTES + ((cg * 4 + piece) * 16 + rg) * 128 + r * 16),
                                 "l"(live > 32 * cg ? src + 64 * cg : nullptr), "r"(live > 32 * cg ? 16 : 0) : "memory");
            }
            cp_commit();
            cp_wait<0>();
            tc::fence_smem_to_async();
            tc::mbar_arrive(bar);
            ++n_unit;
        }
        if (wait.dead())  // nobody may have waited for these
            for (int n = max(n_unit - 2, 0); n < n_unit; ++n) Waits{bars}.on(kFullKQ + (n & 1), (n >> 1) & 1);
    } else {
        // ---- 32 rows of P at a time: S, D, U and R as they lie, dy and v (lane = token of eight, 16-byte piece of the 32 rows)
        const int r = lane & 7, piece = lane >> 3, at = warp - kCopyWarp - 1;
        int stage_count = 0, issued = 0;  // of this stage
#pragma unroll 1
        for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
            const int n = tokens_of(unit), c = unit % p.nc, bh = unit / p.nc, h = bh % p.H, b = bh / p.H;
            if (n == 0) continue;
            const long long dys = (long long)p.H * p.P;
            const char *dy = static_cast<const char *>(p.dy) + 2 * (((long long)b * p.L + c * kC + r) * dys + (long long)h * p.P + 8 * piece);
            const char *v = static_cast<const char *>(p.v) + 2 * (b * p.vs[0] + (c * kC + r) * p.vs[1] + (long long)h * p.P + 8 * piece);
#pragma unroll 1
            for (int s = 0; s < steps; ++s, ++stage_count) {
                if (stage_count % kStages != at) continue;
                const uint32_t st = sbase + at * SM::STAGE, bar = bars + 8 * (kFull + at);
                wait.on(kEmpty + at, ((stage_count / kStages) & 1) ^ 1);
                if (wait.dead()) break;
                if (lane == 0) {
                    const size_t from = (size_t)unit * steps + s;
                    tc::mbar_arrive_expect_tx(bar, 2 * SM::ST + 2 * SM::UT);
                    bulk_load(st + SM::S, reinterpret_cast<const char *>(p.states) + from * SM::ST, SM::ST, bar);
                    bulk_load(st + SM::D, reinterpret_cast<const char *>(p.adj) + from * SM::ST, SM::ST, bar);
                    bulk_load(st + SM::U, reinterpret_cast<const char *>(p.u) + from * SM::UT, SM::UT, bar);
                    bulk_load(st + SM::R, reinterpret_cast<const char *>(p.dr) + from * SM::UT, SM::UT, bar);
                }
                __syncwarp();
#pragma unroll 2
                for (int rg = 0; rg < 8; ++rg) {
                    const bool ok = rg * 8 + r < n && s * kRowsP + 8 * piece < p.P;
                    const uint32_t dst = st + piece * 1024 + rg * 128 + r * 16;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + SM::DY), "l"(ok ? dy + 16 * rg * dys + 2 * s * kRowsP : nullptr), "r"(ok ? 16 : 0) : "memory");
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + SM::V), "l"(ok ? v + 16 * rg * p.vs[1] + 2 * s * kRowsP : nullptr), "r"(ok ? 16 : 0) : "memory");
                }
                cp_commit();
                cp_wait<0>();
                tc::fence_smem_to_async();
                tc::mbar_arrive(bar);
                ++issued;
            }
        }
        if (wait.dead() && issued > 0) Waits{bars}.on(kFull + at, (issued - 1) & 1);  // nobody may have waited for it
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem_slot, 512);
}

template <int IO, int NN>
cudaError_t grad_as(const DeltaParams &p, cudaStream_t s) {
    auto *kernel = delta_grad_tc_kernel<IO, NN>;
    const cudaError_t e = allow_smem<Smem<NN>::BYTES>(kernel);
    if (e != cudaSuccess) return e;
    const long long units = (long long)p.B * p.H * p.nc, sms = scan_sm_count();
    kernel<<<(unsigned)(units < sms ? units : sms), kThreads, Smem<NN>::BYTES, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_grad_tc(const DeltaParams &p, int io, cudaStream_t s) {
    if (io == IO_BF16) return p.N <= 64 ? grad_as<IO_BF16, 64>(p, s) : grad_as<IO_BF16, 128>(p, s);
    return p.N <= 64 ? grad_as<IO_F16, 64>(p, s) : grad_as<IO_F16, 128>(p, s);
}

}  // namespace ssd

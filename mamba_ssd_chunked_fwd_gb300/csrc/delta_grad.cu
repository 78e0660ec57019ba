// delta_grad.cu -- the gated delta rule's gradients that sum over the state's
// rows, a chunk of 64 tokens per CTA, in fp32.  Given, of a chunk, the state S before it, the
// adjoint D after it, u and r (delta_walk.cu), with G the running sum of g in
// the chunk, W_ij = exp(G_i - G_j) and d = scale dy:
//
//     Y_ij = W_ij (d_i . u_j)  (j <= i),   Z_ij = beta_i W_ij (r_i . u_j)  (j < i)
//     dq_i = exp(G_i) S^T d_i + sum_j Y_ij k_j
//     dk_i = -beta_i exp(G_i) S^T r_i - sum_j Z_ij k_j                         (as the key that is read)
//            + exp(G_end - G_i) D^T u_i + sum_m (Y_mi q_m - Z_mi k_m)         (as the key that is written)
//     dbeta_i = r_i . (v_i - exp(G_i) S k_i - sum_{j<i} W_ij (k_i . k_j) u_j)
//     dg_t = exp(G_end) <S, D> + sum_{j<t} k_j . exp(G_end - G_j) D^T u_j
//            + sum_{i>=t} (exp(G_i) q_i . S^T d_i - beta_i exp(G_i) k_i . S^T r_i) + sum_{i>=t>j} E_ij,
//     E_ij = Y_ij (q_i . k_j) - Z_ij (k_i . k_j)
//
// dg is the sum over every decay that contains g_t.  It is taken from these pieces,
// not from q . dq and k . dk: those hold terms without a decay, which cancel, and with
// strong decays little more than their rounding is left.
//
// [2,333] with 6 heads of 64 x 64: 42 us on 72 CTAs, a chunk and head each; issue 39 %, the rest of the SMs idle.
#include "delta.cuh"

namespace ssd {

namespace {

constexpr int kC = kDeltaChunk, kThreads = 256, kPT = 32;

template <int NP>
struct GradSmem {
    static constexpr int W = NP + 4, U = kPT + 4, Y = kC + 4;
    float k[kC * W], q[kC * W];
    union {
        struct {
            float u[kC * U], d[kC * U], r[kC * U], s[kPT * W], a[kPT * W];
        } t;
        struct {
            float y[kC * Y], z[kC * Y], e[kC * Y];
        } m;
    } x;
    float gh[kC], gl[kC], beta[kC], into[kC], out[kC];
    float state_in[kC], key_read[kC], written[kC], row_e[kC], bdot[kC], prior[kC], over[2];
    float warp_sum[kThreads / 32];
};

__device__ __forceinline__ float sum16(float v) {  // over the 16 threads of a row
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// acc[4][4] (rows ty + 16 i, columns tx + 16 j) += A B^T over n columns of rows `w` apart.
template <int N4>
__device__ __forceinline__ void dots(const float *A, const float *B, int w, int ty, int tx, float (&acc)[4][4]) {
#pragma unroll 2
    for (int m = 0; m < N4; ++m) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = *reinterpret_cast<const float4 *>(A + (ty + 16 * i) * w + 4 * m);
            b[i] = *reinterpret_cast<const float4 *>(B + (tx + 16 * i) * w + 4 * m);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, acc[i][j]))));
    }
}

template <int IO, int NP>
__global__ void __launch_bounds__(kThreads)
delta_grad_kernel(const __grid_constant__ DeltaParams p) {
    using SM = GradSmem<NP>;
    constexpr int W = SM::W, U = SM::U, YW = SM::Y, NJ = NP / 64;  // four columns 4 tx + 64 j for each j
    extern __shared__ __align__(16) unsigned char raw[];
    SM &s = *reinterpret_cast<SM *>(raw);
    const int c = blockIdx.x % p.nc, bh = blockIdx.x / p.nc, h = bh % p.H, b = bh / p.H;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, t0 = c * kC, grp = h / (p.H / p.G);
    const int left = delta_length(p, b) - t0, n = min(max(left, 0), kC);
    const bool shared_keys = p.H > p.G;
    const size_t pn = (size_t)p.P * p.N;
    if (n == 0) {  // behind the row's end: zeros
        const int rows = min(kC, p.L - t0);
        for (int e = tid; e < rows * p.N; e += kThreads) {
            const long long t = (long long)b * p.L + t0 + e / p.N;
            const int col = e % p.N;
            if (shared_keys) {
                p.dqh[(t * p.H + h) * p.N + col] = 0.f;
                p.dkh[(t * p.H + h) * p.N + col] = 0.f;
            } else {
                st_io<IO>(p.dq, (t * p.G + grp) * p.N + col, 0.f);
                st_io<IO>(p.dk, (t * p.G + grp) * p.N + col, 0.f);
            }
        }
        if (tid < rows) {
            store_gate<IO>(p.dg, ((long long)b * p.L + t0 + tid) * p.H + h, p.g32, 0.f);
            store_gate<IO>(p.dbeta, ((long long)b * p.L + t0 + tid) * p.H + h, p.b32, 0.f);
        }
        return;
    }
    for (int e = tid; e < kC * NP; e += kThreads) {
        const int i = e / NP, col = e % NP;
        const bool ok = i < n && col < p.N;
        s.k[i * W + col] = load_one<IO>(p.k, b * p.ks[0] + (t0 + i) * p.ks[1] + grp * p.N + col, ok);
        s.q[i * W + col] = load_one<IO>(p.q, b * p.qs[0] + (t0 + i) * p.qs[1] + grp * p.N + col, ok);
    }
    if (tid < 32) {  // the running sum of g as the sum of two floats, so that differences keep their precision
        float hi[2], lo[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int i = 2 * tid + m;
            float g = load_gate<IO>(p.g, b * p.gs[0] + (t0 + i) * p.gs[1] + h, p.g32, i < n);
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(g) : "f"(-200.f));  // sums stay finite; on growth beside it see delta_prep.cu
            hi[m] = g, lo[m] = 0.f;
            s.beta[i] = load_gate<IO>(p.beta, b * p.bs[0] + (t0 + i) * p.bs[1] + h, p.b32, i < n);
        }
        auto add = [](float &h0, float &l0, float h1, float l1) {
            const float sum = h0 + h1, t = sum - h0, err = (h0 - (sum - t)) + (h1 - t) + l0 + l1;
            h0 = sum + err;
            l0 = err - (h0 - sum);
        };
        add(hi[1], lo[1], hi[0], lo[0]);
        float th = hi[1], tl = lo[1];
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const float oh = __shfl_up_sync(0xffffffffu, th, m), ol = __shfl_up_sync(0xffffffffu, tl, m);
            if (tid >= m) add(th, tl, oh, ol);
        }
        const float ph = __shfl_up_sync(0xffffffffu, th, 1), pl = __shfl_up_sync(0xffffffffu, tl, 1);
        if (tid > 0) add(hi[0], lo[0], ph, pl);
        hi[1] = th, lo[1] = tl;
        const float eh = __shfl_sync(0xffffffffu, th, 31), el = __shfl_sync(0xffffffffu, tl, 31);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int i = 2 * tid + m;
            s.gh[i] = hi[m], s.gl[i] = lo[m];
            s.into[i] = expf(hi[m]);
            s.out[i] = expf((eh - hi[m]) + (el - lo[m]));
        }
    }
    __syncthreads();
    float kk[4][4] = {}, qk[4][4] = {};
    dots<NP / 4>(s.k, s.k, W, ty, tx, kk);
    dots<NP / 4>(s.q, s.k, W, ty, tx, qk);

    float du[4][4] = {}, ru[4][4] = {};
    float dS[4][NJ][4] = {}, rS[4][NJ][4] = {}, uD[4][NJ][4] = {};
    float rv = 0.f, sd = 0.f;  // r . v of row tid / 4, a share of <S, D>
    const float *S = p.states + ((size_t)bh * p.nc + c) * pn, *D = p.adj + ((size_t)bh * p.nc + c) * pn;
    for (int p0 = 0; p0 < p.P; p0 += kPT) {
        __syncthreads();
#pragma unroll
        for (int m = 0; m < kPT / 4; ++m) {
            const int i = tid >> 2, col = (tid & 3) + 4 * m;
            const bool ok = i < n && p0 + col < p.P;
            const long long at = ((long long)bh * p.nc * kC + t0 + i) * p.P + p0 + col;
            const float u = load_one<IO_F32>(p.u, at, ok), r = load_one<IO_F32>(p.dr, at, ok);
            s.x.t.u[i * U + col] = u;
            s.x.t.r[i * U + col] = r;
            s.x.t.d[i * U + col] = load_one<IO>(p.dy, (((long long)b * p.L + t0 + i) * p.H + h) * p.P + p0 + col, ok);
            rv = fmaf(r, load_one<IO>(p.v, b * p.vs[0] + (t0 + i) * p.vs[1] + (long long)h * p.P + p0 + col, ok), rv);
        }
        for (int e = tid; e < kPT * NP; e += kThreads) {
            const int row = e / NP, col = e % NP;
            const bool ok = p0 + row < p.P && col < p.N;
            const long long at = (long long)(p0 + row) * p.N + col;
            const float x = load_one<IO_F32>(S, at, ok), y = load_one<IO_F32>(D, at, ok);
            s.x.t.s[row * W + col] = x;
            s.x.t.a[row * W + col] = y;
            sd = fmaf(x, y, sd);
        }
        __syncthreads();
        dots<kPT / 4>(s.x.t.d, s.x.t.u, U, ty, tx, du);
        dots<kPT / 4>(s.x.t.r, s.x.t.u, U, ty, tx, ru);
#pragma unroll 2
        for (int m = 0; m < kPT; ++m) {
            float4 x[NJ], y[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                x[j] = *reinterpret_cast<const float4 *>(&s.x.t.s[m * W + 4 * tx + 64 * j]);
                y[j] = *reinterpret_cast<const float4 *>(&s.x.t.a[m * W + 4 * tx + 64 * j]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = (ty + 16 * i) * U + m;
                const float d = s.x.t.d[row], r = s.x.t.r[row], u = s.x.t.u[row];
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const float xs[4] = {x[j].x, x[j].y, x[j].z, x[j].w}, ys[4] = {y[j].x, y[j].y, y[j].z, y[j].w};
#pragma unroll
                    for (int l = 0; l < 4; ++l) {
                        dS[i][j][l] = fmaf(d, xs[l], dS[i][j][l]);
                        rS[i][j][l] = fmaf(r, xs[l], rS[i][j][l]);
                        uD[i][j][l] = fmaf(u, ys[l], uD[i][j][l]);
                    }
                }
            }
        }
    }
    rv += __shfl_xor_sync(0xffffffffu, rv, 1);
    rv += __shfl_xor_sync(0xffffffffu, rv, 2);
    if ((tid & 3) == 0) s.bdot[tid >> 2] = rv;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) sd += __shfl_xor_sync(0xffffffffu, sd, m);
    if ((tid & 31) == 0) s.warp_sum[tid >> 5] = sd;
    __syncthreads();
    // Y, Z and E over the tiles of u, d, r, S and D
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = ty + 16 * i;
        const float into = s.into[row], beta = s.beta[row];
        float row_e = 0.f, prior = 0.f, q_in = 0.f, k_in = 0.f, wr = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = tx + 16 * j;
            const float w = col <= row ? expf((s.gh[row] - s.gh[col]) + (s.gl[row] - s.gl[col])) : 0.f;
            const float y = col <= row ? p.scale * w * du[i][j] : 0.f, z = col < row ? beta * w * ru[i][j] : 0.f;
            const float e = col < row ? y * qk[i][j] - z * kk[i][j] : 0.f;
            s.x.m.y[row * YW + col] = y;
            s.x.m.z[row * YW + col] = z;
            s.x.m.e[row * YW + col] = e;
            row_e += e;
            if (col < row) prior = fmaf(w * kk[i][j], ru[i][j], prior);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int l = 0; l < 4; ++l) {
                const int at = row * W + 4 * tx + 64 * j + l;
                q_in = fmaf(s.q[at], dS[i][j][l], q_in);
                k_in = fmaf(s.k[at], rS[i][j][l], k_in);
                wr = fmaf(s.k[at], uD[i][j][l], wr);
            }
        row_e = sum16(row_e), prior = sum16(prior), q_in = sum16(q_in), k_in = sum16(k_in), wr = sum16(wr);
        if (tx == 0) {
            s.row_e[row] = row_e;
            s.prior[row] = prior;
            s.state_in[row] = p.scale * into * q_in - beta * into * k_in;
            s.key_read[row] = into * k_in;
            s.written[row] = s.out[row] * wr;
        }
    }
    __syncthreads();
    // dq, dk
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = ty + 16 * i;
        const float fq = p.scale * s.into[row], fr = -s.beta[row] * s.into[row], fu = s.out[row];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int l = 0; l < 4; ++l) {
                dS[i][j][l] *= fq;
                rS[i][j][l] = fmaf(fu, uD[i][j][l], fr * rS[i][j][l]);
            }
    }
    for (int m = 0; m < kC; ++m) {
        float4 k[NJ], q[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            k[j] = *reinterpret_cast<const float4 *>(&s.k[m * W + 4 * tx + 64 * j]);
            q[j] = *reinterpret_cast<const float4 *>(&s.q[m * W + 4 * tx + 64 * j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = ty + 16 * i;
            const float y = s.x.m.y[row * YW + m], z = -(s.x.m.z[row * YW + m] + s.x.m.z[m * YW + row]), yt = s.x.m.y[m * YW + row];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const float ks[4] = {k[j].x, k[j].y, k[j].z, k[j].w}, qs[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
                for (int l = 0; l < 4; ++l) {
                    dS[i][j][l] = fmaf(y, ks[l], dS[i][j][l]);
                    rS[i][j][l] = fmaf(yt, qs[l], fmaf(z, ks[l], rS[i][j][l]));
                }
            }
        }
    }
    const int rows = min(kC, p.L - t0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = ty + 16 * i;
        if (row >= rows) continue;
        const long long t = (long long)b * p.L + t0 + row;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int l = 0; l < 4; ++l) {
                const int col = 4 * tx + 64 * j + l;
                const float x = row < n ? dS[i][j][l] : 0.f, y = row < n ? rS[i][j][l] : 0.f;
                if (col >= p.N) continue;
                if (shared_keys) {
                    p.dqh[(t * p.H + h) * p.N + col] = x;
                    p.dkh[(t * p.H + h) * p.N + col] = y;
                } else {
                    st_io<IO>(p.dq, (t * p.G + grp) * p.N + col, x);
                    st_io<IO>(p.dk, (t * p.G + grp) * p.N + col, y);
                }
            }
    }
    // dbeta, dg: thread t for its token.  Sums over the tokens before, and from this one on: over a warp, then over both
    float own = 0.f;
    if (tid < kC)
#pragma unroll 8
        for (int i = tid + 1; i < kC; ++i) own += s.x.m.e[i * YW + tid];  // its column of E
    float w = tid < kC ? s.written[tid] : 0.f, x = tid < kC ? s.state_in[tid] + (s.row_e[tid] - own) : 0.f;
    const int lane = tid & 31;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const float down = __shfl_up_sync(0xffffffffu, w, m), up = __shfl_down_sync(0xffffffffu, x, m);
        if (lane >= m) w += down;
        if (lane + m < 32) x += up;
    }
    if (tid == 31) s.over[0] = w;
    if (tid == 32) s.over[1] = x;
    const float before = __shfl_up_sync(0xffffffffu, w, 1);
    __syncthreads();
    if (tid < rows) {
        float total = 0.f;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) total += s.warp_sum[i];
        const float g = s.into[kC - 1] * total + ((lane > 0 ? before : 0.f) + (tid >= 32 ? s.over[0] : 0.f)) + (x + (tid < 32 ? s.over[1] : 0.f));
        const long long at = ((long long)b * p.L + t0 + tid) * p.H + h;
        store_gate<IO>(p.dg, at, p.g32, tid < n ? g : 0.f);
        store_gate<IO>(p.dbeta, at, p.b32, tid < n ? s.bdot[tid] - s.key_read[tid] - s.prior[tid] : 0.f);
    }
}

// dq, dk of a group: the sums over its heads, in their order.
template <int IO>
__global__ void __launch_bounds__(256)
delta_heads_kernel(const __grid_constant__ DeltaParams p) {
    const long long count = (long long)p.B * p.L * p.G * p.N, e = blockIdx.x * 256LL + threadIdx.x;
    if (e >= count) return;
    const int hpg = p.H / p.G;
    const long long col = e % p.N, tg = e / p.N, src = tg * hpg * p.N + col;
    float q = 0.f, k = 0.f;
    for (int i = 0; i < hpg; ++i) {
        q += __ldg(p.dqh + src + (long long)i * p.N);
        k += __ldg(p.dkh + src + (long long)i * p.N);
    }
    st_io<IO>(p.dq, e, q);
    st_io<IO>(p.dk, e, k);
}

template <int IO, int NP>
cudaError_t grad_as(const DeltaParams &p, cudaStream_t s) {
    const cudaError_t e = allow_smem<sizeof(GradSmem<NP>)>(delta_grad_kernel<IO, NP>);
    if (e != cudaSuccess) return e;
    delta_grad_kernel<IO, NP><<<(unsigned)((long long)p.B * p.H * p.nc), kThreads, sizeof(GradSmem<NP>), s>>>(p);
    return cudaGetLastError();
}

template <int IO>
cudaError_t grad_io(const DeltaParams &p, cudaStream_t s) {
    return p.N <= 64 ? grad_as<IO, 64>(p, s) : grad_as<IO, 128>(p, s);
}

cudaError_t launch_delta_heads(const DeltaParams &p, int io, cudaStream_t s) {
    const long long count = (long long)p.B * p.L * p.G * p.N;
    const unsigned grid = (unsigned)((count + 255) / 256);
    if (io == IO_F32) delta_heads_kernel<IO_F32><<<grid, 256, 0, s>>>(p);
    else if (io == IO_F16) delta_heads_kernel<IO_F16><<<grid, 256, 0, s>>>(p);
    else delta_heads_kernel<IO_BF16><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_grad(const DeltaParams &p, int io, cudaStream_t s) {
    switch (io) {
        case IO_F32: return grad_io<IO_F32>(p, s);
        case IO_F16: return grad_io<IO_F16>(p, s);
        case IO_BF16: return grad_io<IO_BF16>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_delta_bwd(const DeltaParams &p, int io, cudaStream_t s) {
    cudaError_t e;
    if (p.chunked) {
        if ((e = launch_delta_prep(p, io, true, s)) != cudaSuccess) return e;
        if ((e = launch_delta_tc_walks(p, io, s)) != cudaSuccess) return e;
        if ((e = launch_delta_grad_tc(p, io, s)) != cudaSuccess) return e;
    } else {
        if ((e = launch_delta_walks(p, io, s)) != cudaSuccess) return e;
        if ((e = launch_delta_grad(p, io, s)) != cudaSuccess) return e;
    }
    return p.H > p.G ? launch_delta_heads(p, io, s) : cudaSuccess;
}

}  // namespace ssd

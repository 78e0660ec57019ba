// block_norm.cu -- the end of one block and the norm before the next:
//
//   p = o / rms(o) * w_post,  r' = r + scale gate p,  n = r' / rms(r') * w_pre
//
// and its backward.  With a = d o / rms(o) (the normalised rows hat_o, hat_r):
//   dr     = dr_out + (v - hat_r mean(v hat_r)) / rms(r'),       v = dn w_pre
//   d_o    = (u - hat_o mean(u hat_o)) / rms(o),                 u = dr scale gate w_post
//   dgate  = dr scale w_post hat_o,   dw_pre = sum dn hat_r,
//   dscale = w_post s,  dw_post = scale s,                       s = sum dr gate hat_o
//
// About 11 (backward 30) operations per element against 8 to 16 bytes: bound by
// HBM.  A row stays in the registers of its threads, K runs of four elements
// each, between the two reductions, so every tensor moves once; the threads
// walk rows with the weights (and, backwards, the column sums) in registers.
// 16-bit rows are kept as loaded and unpacked at each use.
#include "scan_common.cuh"

namespace ssd {

namespace {

// Sums of v over the row's TPR threads (blockDim.x), for every one of them.  One
// barrier: consecutive calls must use different `slot`s.
template <int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float (*slot)[32]) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return;  // rows of one warp are independent of each other
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < NV; ++i) slot[i][w] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        v[i] = lane < nw ? slot[i][lane] : 0.f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    }
}

template <int SIO>
__device__ __forceinline__ float round_io(float v) {
    return IoTraits<SIO>::to_f(IoTraits<SIO>::from_f(v));
}

template <int IO, int SIO, int K, bool VEC>
__global__ void __launch_bounds__(K <= 2 ? 256 : 512)
block_norm_kernel(BlockNormParams p) {
    __shared__ float red[2][1][32];
    const int tpr = blockDim.x;
    float wp[K][4], ws[K][4];  // w_pre; scale w_post
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = (threadIdx.x + tpr * k) * 4 + j;
            const bool in = c < p.D;
            wp[k][j] = in ? __ldg(p.w_pre + c) : 0.f;
            ws[k][j] = in ? (p.w_post ? __ldg(p.w_post + c) : 1.f) * (p.scale ? __ldg(p.scale + c) : 1.f) : 0.f;
        }
    const float inv_d = 1.f / (float)p.D;
    for (long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y; row < p.rows;
         row += (long long)gridDim.x * blockDim.y) {
        const long long base = row * p.D, gbase = p.gate ? row / p.rows_per_gate * p.D : 0;
        Raw4 ro[K], rr[K], rg[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (threadIdx.x + tpr * k) * 4, nv = min(4, p.D - c);
            rr[k] = load_raw4<SIO, VEC, false>(p.r, base + c, nv > 0, nv);
            ro[k] = load_raw4<IO, VEC>(p.o, base + c, nv > 0 && p.o, nv);
            rg[k] = load_raw4<IO, VEC>(p.gate, gbase + c, nv > 0 && p.gate, nv);
        }
        float inv = 1.f;
        if (p.o && p.w_post) {
            float ss[1] = {0.f};
#pragma unroll
            for (int k = 0; k < K; ++k)
                if ((threadIdx.x + tpr * k) * 4 < p.D) {
                    float o[4];
                    unpack4<IO, VEC>(ro[k], o);
#pragma unroll
                    for (int j = 0; j < 4; ++j) ss[0] = fmaf(o[j], o[j], ss[0]);
                }
            row_sum(ss, red[0]);
            inv = rsqrtf(ss[0] * inv_d + p.eps);
        }
        float r[K][4], ss[1] = {0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (threadIdx.x + tpr * k) * 4, nv = min(4, p.D - c);
            if (nv <= 0) continue;
            unpack4<SIO, VEC>(rr[k], r[k]);
            if (p.o) {
                float o[4], g[4] = {1.f, 1.f, 1.f, 1.f};
                unpack4<IO, VEC>(ro[k], o);
                if (p.gate) unpack4<IO, VEC>(rg[k], g);
#pragma unroll
                for (int j = 0; j < 4; ++j) r[k][j] = round_io<SIO>(fmaf(g[j] * ws[k][j], o[j] * inv, r[k][j]));
                store4_io<SIO, VEC>(p.r_out, base + c, nv, r[k]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) ss[0] = j < nv ? fmaf(r[k][j], r[k][j], ss[0]) : ss[0];
        }
        row_sum(ss, red[1]);
        const float inv2 = rsqrtf(ss[0] * inv_d + p.eps);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (threadIdx.x + tpr * k) * 4, nv = min(4, p.D - c);
            if (nv <= 0) continue;
            float n[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) n[j] = r[k][j] * inv2 * wp[k][j];
            store4_io<IO, VEC>(p.n, base + c, nv, n);
        }
        if (!(p.o && p.w_post) && blockDim.x > 32) __syncthreads();  // one reduction per row only: its slot is free again
    }
}

template <int IO, int SIO, int K, bool VEC>
__global__ void __launch_bounds__(512, 1)
block_norm_bwd_kernel(BlockNormParams p) {
    __shared__ float red[2][3][32];
    const int tpr = blockDim.x;
    const long long chunk = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    if (chunk >= p.chunks) return;  // blockDim.y > 1 only for rows of one warp
    const bool seq_gate = p.gate && p.rows_per_gate > 1;
    long long r0, r1;
    if (seq_gate) {
        const long long per = (p.rows_per_gate + p.chunk_rows - 1) / p.chunk_rows, gi = chunk / per;
        r0 = gi * p.rows_per_gate + chunk % per * p.chunk_rows;
        r1 = min((gi + 1) * p.rows_per_gate, r0 + p.chunk_rows);
    } else {
        r0 = chunk * p.chunk_rows;
        r1 = min(p.rows, r0 + p.chunk_rows);
    }
    float wp[K][4], ws[K][4], acc1[K][4], acc2[K][4];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = (threadIdx.x + tpr * k) * 4 + j;
            const bool in = c < p.D;
            wp[k][j] = in ? __ldg(p.w_pre + c) : 0.f;
            ws[k][j] = in ? (p.w_post ? __ldg(p.w_post + c) : 1.f) * (p.scale ? __ldg(p.scale + c) : 1.f) : 0.f;
            acc1[k][j] = acc2[k][j] = 0.f;
        }
    const float inv_d = 1.f / (float)p.D;
    for (long long row = r0; row < r1; ++row) {
        const long long base = row * p.D, gbase = p.gate ? row / p.rows_per_gate * p.D : 0;
        Raw4 ro[K], rr[K], rg[K], rn[K], rd[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (threadIdx.x + tpr * k) * 4, nv = min(4, p.D - c);
            rr[k] = load_raw4<SIO, VEC>(p.r_out, base + c, nv > 0, nv);
            rn[k] = load_raw4<IO, VEC>(p.dn, base + c, nv > 0, nv);
            rd[k] = load_raw4<SIO, VEC>(p.dr_out, base + c, nv > 0 && p.dr_out, nv);
            ro[k] = load_raw4<IO, VEC>(p.o, base + c, nv > 0 && p.o, nv);
            rg[k] = load_raw4<IO, VEC>(p.gate, gbase + c, nv > 0 && p.gate, nv);
        }
        float s[3] = {0.f, 0.f, 0.f};  // |r'|^2, dn w_pre . r', |o|^2
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float r[4], n[4], o[4];
            unpack4<SIO, VEC>(rr[k], r);
            unpack4<IO, VEC>(rn[k], n);
            unpack4<IO, VEC>(ro[k], o);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[0] = fmaf(r[j], r[j], s[0]);
                s[1] = fmaf(n[j] * wp[k][j], r[j], s[1]);
                s[2] = fmaf(o[j], o[j], s[2]);
            }
        }
        row_sum(s, red[0]);
        const float inv2 = rsqrtf(s[0] * inv_d + p.eps), m2 = s[1] * inv_d * inv2 * inv2;
        const float inv = p.w_post ? rsqrtf(s[2] * inv_d + p.eps) : 1.f;
        // dr of four elements: (v - r' inv2^2 mean(v r')) inv2 + dr_out
        auto dr_of = [&](int k, float (&dr)[4]) {
            float r[4], n[4];
            unpack4<SIO, VEC>(rr[k], r);
            unpack4<IO, VEC>(rn[k], n);
            unpack4<SIO, VEC>(rd[k], dr);
#pragma unroll
            for (int j = 0; j < 4; ++j) dr[j] = fmaf(fmaf(-r[j], m2, n[j] * wp[k][j]), inv2, dr[j]);
        };
        float t[1] = {0.f};  // u . o
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (threadIdx.x + tpr * k) * 4, nv = min(4, p.D - c);
            if (nv <= 0) continue;
            float dr[4], r[4], n[4];
            dr_of(k, dr);
            unpack4<SIO, VEC>(rr[k], r);
            unpack4<IO, VEC>(rn[k], n);
            store4_io<SIO, VEC>(p.dr, base + c, nv, dr);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc2[k][j] = fmaf(n[j], r[j] * inv2, acc2[k][j]);
            if (!p.o) continue;
            float o[4], g[4] = {1.f, 1.f, 1.f, 1.f}, dg[4];
            unpack4<IO, VEC>(ro[k], o);
            if (p.gate) unpack4<IO, VEC>(rg[k], g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float dh = dr[j] * (o[j] * inv);  // dr hat_o
                dg[j] = dh * ws[k][j];
                t[0] = fmaf(g[j] * dr[j] * ws[k][j], o[j], t[0]);
                acc1[k][j] += seq_gate ? dh : dh * g[j];
            }
            if (p.gate && !seq_gate) store4_io<IO, VEC>(p.dgate, base + c, nv, dg);
        }
        if (!p.o) {
            if (blockDim.x > 32) __syncthreads();  // the slot is free again
            continue;
        }
        row_sum(t, red[1]);
        const float m = p.w_post ? t[0] * inv_d * inv * inv : 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (threadIdx.x + tpr * k) * 4, nv = min(4, p.D - c);
            if (nv <= 0) continue;
            float dr[4], o[4], g[4] = {1.f, 1.f, 1.f, 1.f};
            dr_of(k, dr);
            unpack4<IO, VEC>(ro[k], o);
            if (p.gate) unpack4<IO, VEC>(rg[k], g);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = fmaf(-o[j], m, g[j] * dr[j] * ws[k][j]) * inv;
            store4_io<IO, VEC>(p.d_o, base + c, nv, o);
        }
    }
    float *part = p.part + chunk * 2 * p.D;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = (threadIdx.x + tpr * k) * 4 + j;
            if (c < p.D) {
                part[c] = acc1[k][j];
                part[p.D + c] = acc2[k][j];
            }
        }
}

// The column sums over the chunks, in a fixed order: 32 interleaved sums per column, then those in turn.
template <int IO>
__global__ void __launch_bounds__(1024)
block_norm_sum_kernel(BlockNormParams p) {
    __shared__ float red[2][32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    const bool seq_gate = p.gate && p.rows_per_gate > 1, in = c < p.D;
    const float wpost = in && p.w_post ? __ldg(p.w_post + c) : 1.f, scale = in && p.scale ? __ldg(p.scale + c) : 1.f;
    float s1 = 0.f, s2 = 0.f;
    if (in) {
        if (seq_gate) {
            const long long per = (p.rows_per_gate + p.chunk_rows - 1) / p.chunk_rows, gates = p.rows / p.rows_per_gate;
            for (long long gi = threadIdx.y; gi < gates; gi += 32) {
                float s = 0.f;
                for (long long q = gi * per; q < (gi + 1) * per; ++q) {
                    s += p.part[q * 2 * p.D + c];
                    s2 += p.part[(q * 2 + 1) * p.D + c];
                }
                st_io<IO>(p.dgate, (size_t)(gi * p.D + c), s * (wpost * scale));
                s1 = fmaf(ld_io<IO>(p.gate, (size_t)(gi * p.D + c)), s, s1);
            }
        } else {
            for (long long q = threadIdx.y; q < p.chunks; q += 32) {
                s1 += p.part[q * 2 * p.D + c];
                s2 += p.part[(q * 2 + 1) * p.D + c];
            }
        }
    }
    red[0][threadIdx.y][threadIdx.x] = s1;
    red[1][threadIdx.y][threadIdx.x] = s2;
    __syncthreads();
    if (threadIdx.y != 0 || !in) return;
    for (int y = 1; y < 32; ++y) {
        s1 += red[0][y][threadIdx.x];
        s2 += red[1][y][threadIdx.x];
    }
    p.dw_pre[c] = s2;
    if (p.dw_post) p.dw_post[c] = scale * s1;
    if (p.dscale) p.dscale[c] = wpost * s1;
}

// Threads of a row and rows of a CTA for K runs of four elements per thread.
dim3 row_block(int D, int K) {
    const int tpr = ((D + 4 * K - 1) / (4 * K) + 31) / 32 * 32;
    return dim3(tpr, tpr == 32 ? 4 : 1);
}

bool norm_vec(const BlockNormParams &p, int io, int sio) {
    auto ok = [](const void *q, int t) { return reinterpret_cast<uintptr_t>(q) % (t == IO_F32 ? 16 : 8) == 0; };
    return p.D % 4 == 0 && ok(p.o, io) && ok(p.r, sio) && ok(p.gate, io) && ok(p.n, io) && ok(p.r_out, sio) &&
           ok(p.dn, io) && ok(p.dr_out, sio) && ok(p.d_o, io) && ok(p.dr, sio) && ok(p.dgate, io);
}

template <int IO, int SIO, int K>
cudaError_t launch_norm_as(const BlockNormParams &p, cudaStream_t s) {
    const dim3 block = row_block(p.D, K);
    auto *kernel = norm_vec(p, IO, SIO) ? block_norm_kernel<IO, SIO, K, true> : block_norm_kernel<IO, SIO, K, false>;
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, block.x * block.y, 0) !=
            cudaSuccess || per_sm < 1) {
        (void)cudaGetLastError();
        per_sm = 1;
    }
    const long long need = (p.rows + block.y - 1) / block.y, most = (long long)scan_sm_count() * per_sm;
    kernel<<<(unsigned)(need < most ? need : most), block, 0, s>>>(p);
    return cudaGetLastError();
}

template <int IO, int SIO>
cudaError_t launch_norm_io(const BlockNormParams &p, cudaStream_t s) {
    if (p.D <= 128) return launch_norm_as<IO, SIO, 1>(p, s);
    if (p.D <= 2048) return launch_norm_as<IO, SIO, 2>(p, s);
    if (p.D <= 8192) return launch_norm_as<IO, SIO, 4>(p, s);
    return launch_norm_as<IO, SIO, 8>(p, s);
}

template <int IO, int SIO, int K>
cudaError_t launch_norm_bwd_as(const BlockNormParams &p, cudaStream_t s) {
    const dim3 block = row_block(p.D, K);
    auto *kernel = norm_vec(p, IO, SIO) ? block_norm_bwd_kernel<IO, SIO, K, true> : block_norm_bwd_kernel<IO, SIO, K, false>;
    kernel<<<(unsigned)((p.chunks + block.y - 1) / block.y), block, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    block_norm_sum_kernel<IO><<<(p.D + 31) / 32, dim3(32, 32), 0, s>>>(p);
    return cudaGetLastError();
}

template <int IO, int SIO>
cudaError_t launch_norm_bwd_io(const BlockNormParams &p, cudaStream_t s) {
    if (p.D <= 128) return launch_norm_bwd_as<IO, SIO, 1>(p, s);
    if (p.D <= 4096) return launch_norm_bwd_as<IO, SIO, 2>(p, s);
    if (p.D <= 8192) return launch_norm_bwd_as<IO, SIO, 4>(p, s);
    return launch_norm_bwd_as<IO, SIO, 8>(p, s);
}

}  // namespace

// About four chunks of rows per SM; a chunk never spans two gates of several rows.
void block_norm_chunks(BlockNormParams &p) {
    const long long target = 4LL * scan_sm_count();
    const bool seq_gate = p.gate && p.rows_per_gate > 1;
    const long long span = seq_gate ? p.rows_per_gate : p.rows, spans = p.rows / span;
    long long per = (target + spans - 1) / spans;  // chunks per span
    if (per > span) per = span;
    p.chunk_rows = (span + per - 1) / per;
    p.chunks = spans * ((span + p.chunk_rows - 1) / p.chunk_rows);
}

#define SSD_NORM_DISPATCH(FN)                                                     \
    if (io == IO_F32 && sio == IO_F32) return FN<IO_F32, IO_F32>(p, s);  \
    if (io == IO_F16 && sio == IO_F16) return FN<IO_F16, IO_F16>(p, s);  \
    if (io == IO_F16 && sio == IO_F32) return FN<IO_F16, IO_F32>(p, s);  \
    if (io == IO_BF16 && sio == IO_BF16) return FN<IO_BF16, IO_BF16>(p, s); \
    if (io == IO_BF16 && sio == IO_F32) return FN<IO_BF16, IO_F32>(p, s); \
    return cudaErrorInvalidValue;

cudaError_t launch_block_norm(const BlockNormParams &p, int io, int sio, cudaStream_t s) {
    SSD_NORM_DISPATCH(launch_norm_io)
}

cudaError_t launch_block_norm_bwd(const BlockNormParams &p, int io, int sio, cudaStream_t s) {
    SSD_NORM_DISPATCH(launch_norm_bwd_io)
}

}  // namespace ssd

// scan_common.cuh -- what the selective-scan kernels share: the parameter
// block, loads of four channels at a time, the step d_t and packed fp32 math.
#pragma once

#include "ssd_internal.cuh"
#include "tc_ptx.cuh"

namespace ssd {

struct ScanParams {
    int B, L, D, N, G;
    const void *x, *dt, *Bm, *Cm, *z;
    const float *A, *Dskip, *dt_bias, *h0;
    const int32_t *lengths;
    void *y;
    float *final_state;
    long long xs[2], dts[2], zs[2], bs[2], cs[2];  // strides (batch, token) in elements
    int dt32;                                      // dt is fp32
    int softplus, has_limit;
    float dt_min, dt_max;
    // segments: tokens [s seg_len, (s+1) seg_len) of every row; seg_len a multiple of 16
    int nseg, seg_len;
    float *seg_states;  // [B,nseg,D,N] state entering a segment (slot 0 unused)
    float *seg_sum;     // [B,nseg,D]   sum of d over a segment
    int tiles;          // channel tiles per group
    // backward
    const void *dy;
    const float *dfinal;
    float *ckpt;        // [B,ceil(L/8),D,N] state before every eighth token
    float *adj;         // [B,nseg,D,N] adjoint state after a segment (last slot unused)
    void *dx, *ddt, *dz;
    float *dh0;
    float *part_bc;     // [G*tiles,B,L,2*NP] per-tile dB and dC
    float *part_a;      // [B*nseg,D,N]
    float *part_d;      // [2,B*nseg,D] dD, ddt_bias
};

// One token per sequence (scan_step.cu).
struct ScanStepParams {
    int B, D, N, G;
    long long nslots;
    const void *x, *dt, *Bm, *Cm, *z;
    const float *A, *Dskip, *dt_bias, *state;
    float *state_out;
    const int32_t *slots;
    void *y;
    long long x_row, dt_row, z_row, b_row, c_row;
    int dt32, softplus, has_limit;
    float dt_min, dt_max;
};
cudaError_t launch_scan_step(const ScanStepParams &p, int io, cudaStream_t s);

struct ConvStepParams {
    int B, C, W;
    long long nslots, x_row;
    const void *x;
    const float *w, *bias;
    const void *state;
    void *state_out;
    const int32_t *slots;
    void *y;
    int silu;
};
cudaError_t launch_conv_step(const ConvStepParams &p, int io, cudaStream_t s);

// The convolution over prompts and its backward (conv_carry.cu).
struct ConvParams {
    int B, L, C, W;
    const void *x;
    long long xs[2];
    const float *w, *bias;
    const void *h0;
    const int32_t *lengths;
    void *y, *final_state;
    int silu;
    // backward
    const void *dy, *dfinal;
    void *dx, *dh0;
    float *dw, *dbias;
    float *part;  // [rows, W + 1, C] sums of dw (first W) and dbias
    int run;      // tokens per thread, conv_bwd_run()
};
cudaError_t launch_conv(const ConvParams &p, int io, cudaStream_t s);
cudaError_t launch_conv_bwd(const ConvParams &p, int io, cudaStream_t s);
int conv_bwd_run(const ConvParams &p);
long long conv_bwd_part_rows(const ConvParams &p);

// The block norm and its backward (block_norm.cu).
struct BlockNormParams {
    long long rows, rows_per_gate;
    int D;
    const void *o, *r, *gate;
    const float *w_post, *w_pre, *scale;
    void *n, *r_out;
    float eps;
    // backward
    const void *dn, *dr_out;
    void *d_o, *dr, *dgate;
    float *dw_post, *dw_pre, *dscale;
    float *part;          // [chunks, 2, D]
    long long chunk_rows;  // rows per chunk; a chunk lies within one gate's rows
    long long chunks;
};
cudaError_t launch_block_norm(const BlockNormParams &p, int io, int sio, cudaStream_t s);
cudaError_t launch_block_norm_bwd(const BlockNormParams &p, int io, int sio, cudaStream_t s);
void block_norm_chunks(BlockNormParams &p);

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kCkpt = 8;  // tokens between stored states (backward)

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Two fp32 numbers in one register pair; a packed operation takes one issue
// slot for both.
__device__ __forceinline__ float2 dup(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 ex2_2(float2 v) { return make_float2(ex2(v.x), ex2(v.y)); }

// exp(d A) from A log2(e): ex2.approx is low by 0.5 to 3e-8 on average for the
// exponents of a slow decay (measured over [-0.5, -1e-5]), and a state that
// remembers a thousand tokens multiplies that.  2.4e-8 added to the exponent
// centres the result (mean error within 1.2e-8 there, the conversion's own
// rounding being 3e-8); d = 0 still gives exactly 1.
constexpr float kDecayCentre = 2.4e-8f;
__device__ __forceinline__ float2 decay2(float2 d, float2 a2) {
    const float2 v = __ffma2_rn(d, a2, make_float2(kDecayCentre, kDecayCentre));
    return make_float2(ex2(v.x), ex2(v.y));
}

// Four consecutive elements as loaded, 8 bytes (16-bit types) or 16.
struct Raw4 {
    uint32_t w[4];
};

// Predicated loads (where `ok` > 0): a branch around a load (or a choice between two) would make
// the compiler wait for its data where the paths meet again, one latency per
// load; a predicated load leaves them all in flight.  What is not loaded stays as it was.
__device__ __forceinline__ void ldg_v4(uint32_t (&w)[4], const void *p, int ok) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.gt.s32 q, %5, 0;\n\t@q ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "+r"(w[0]), "+r"(w[1]), "+r"(w[2]), "+r"(w[3]) : "l"(p), "r"(ok));
}
__device__ __forceinline__ void ldg_v2(uint32_t (&w)[4], const void *p, int ok) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.gt.s32 q, %3, 0;\n\t@q ld.global.nc.v2.u32 {%0, %1}, [%2];\n\t}"
                 : "+r"(w[0]), "+r"(w[1]) : "l"(p), "r"(ok));
}
// Without the read-only path: tensors that the same thread writes later (updates in place).
__device__ __forceinline__ void ld_v4(uint32_t (&w)[4], const void *p, int ok) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.gt.s32 q, %5, 0;\n\t@q ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "+r"(w[0]), "+r"(w[1]), "+r"(w[2]), "+r"(w[3]) : "l"(p), "r"(ok) : "memory");
}
__device__ __forceinline__ void ld_v2(uint32_t (&w)[4], const void *p, int ok) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.gt.s32 q, %3, 0;\n\t@q ld.global.v2.u32 {%0, %1}, [%2];\n\t}"
                 : "+r"(w[0]), "+r"(w[1]) : "l"(p), "r"(ok) : "memory");
}
__device__ __forceinline__ void ld_u32(uint32_t &w, const void *p, int ok) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.gt.s32 q, %2, 0;\n\t@q ld.global.u32 %0, [%1];\n\t}"
                 : "+r"(w) : "l"(p), "r"(ok) : "memory");
}
__device__ __forceinline__ void ld_u16(uint16_t &w, const void *p, int ok) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.gt.s32 q, %2, 0;\n\t@q ld.global.u16 %0, [%1];\n\t}"
                 : "+h"(w) : "l"(p), "r"(ok) : "memory");
}
__device__ __forceinline__ void ldg_u32(uint32_t &w, const void *p, int ok) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.gt.s32 q, %2, 0;\n\t@q ld.global.nc.u32 %0, [%1];\n\t}"
                 : "+r"(w) : "l"(p), "r"(ok));
}
__device__ __forceinline__ void ldg_u16(uint16_t &w, const void *p, int ok) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.gt.s32 q, %2, 0;\n\t@q ld.global.nc.u16 %0, [%1];\n\t}"
                 : "+h"(w) : "l"(p), "r"(ok));
}

// Elements i .. i+3, where `ok`; zeros otherwise.  VEC: the address is aligned to
// four elements and all four exist; else the first nv of them, one by one.
// RO: through the read-only path.
template <int IO, bool VEC, bool RO = true>
__device__ __forceinline__ Raw4 load_raw4(const void *base, long long i, int ok, int nv) {
    Raw4 r = {{0u, 0u, 0u, 0u}};
    if (IO == IO_F32) {
        const uint32_t *p = static_cast<const uint32_t *>(base) + i;
        if (VEC) {
            if (RO) ldg_v4(r.w, p, ok);
            else ld_v4(r.w, p, ok);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (RO) ldg_u32(r.w[j], p + j, j < nv ? ok : 0);
                else ld_u32(r.w[j], p + j, j < nv ? ok : 0);
            }
        }
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(base) + i;
        if (VEC) {
            if (RO) ldg_v2(r.w, p, ok);
            else ld_v2(r.w, p, ok);
        } else {  // one to a word; unpack4 reads them there
            uint16_t e[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (RO) ldg_u16(e[j], p + j, j < nv ? ok : 0);
                else ld_u16(e[j], p + j, j < nv ? ok : 0);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) r.w[j] = e[j];
        }
    }
    return r;
}

template <int IO, bool VEC>
__device__ __forceinline__ void unpack4(const Raw4 &r, float (&v)[4]) {
    if (IO == IO_F32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(r.w[j]);
    } else if (!VEC) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = IO == IO_BF16 ? __uint_as_float(r.w[j] << 16) : __half2float(__ushort_as_half((unsigned short)r.w[j]));
    } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (IO == IO_BF16) {
                v[2 * q] = __uint_as_float(r.w[q] << 16);
                v[2 * q + 1] = __uint_as_float(r.w[q] & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r.w[q]));
                v[2 * q] = f.x; v[2 * q + 1] = f.y;
            }
        }
    }
}

// Copies from global to shared memory that run on while the thread goes on
// (cp.async); the thread that issued them waits with cp_wait.  What is not read is filled with zeros.
__device__ __forceinline__ void cp_async16(void *dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(void *dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4_if(bool ok, void *dst, const void *src, int bytes) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.s32 q, %3, 0;\n\t@q cp.async.ca.shared.global [%0], [%1], 4, %2;\n\t}" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(bytes), "r"((int)ok) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// A pair of floats as 16-bit elements.
template <int IO>
__device__ __forceinline__ uint32_t pack16(float2 v) {
    if (IO == IO_BF16) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y);
        return *reinterpret_cast<const uint32_t *>(&a);
    }
    const __half2 a = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&a);
}

// Eight 16-bit elements at any address, of which the first n exist, into shared memory:
// pairs from a 4-byte boundary are copied asynchronously; off it there is no
// asynchronous form, and the first element, the pairs after it and the last element
// are loaded, all at once, and stored.  Predicates, no branch: the loads of several calls overlap.
// The scan of [8,4096,D,16] at D = 4094 and 4095: 958 and 1338 us (1380 both with eight loads
// of an element each; 692 with whole chunks at D = 4096); gradients of [4,2048,D,16]: 1082
// and 1205 (1171 both; 822).
__device__ __forceinline__ void copy_any16(void *dst, const char *src, int n) {
    const bool even = (reinterpret_cast<size_t>(src) & 3) == 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int bytes = min(max(2 * (n - 2 * j), 0), 4);
        cp_async4_if(even, static_cast<char *>(dst) + 4 * j, bytes > 0 ? src + 4 * j : nullptr, bytes);
    }
    const int m = even ? 0 : n;
    uint16_t first = 0, last = 0;
    uint32_t pair[5] = {0, 0, 0, 0, 0};  // pair[j]: elements 2 j - 1 and 2 j
    ldg_u16(first, src, m > 0);
    ldg_u16(last, src + 2 * (m - 1), m > 0 && !(m & 1));
#pragma unroll
    for (int j = 1; j < 4; ++j) ldg_u32(pair[j], src + 4 * j - 2, m > 2 * j);
    pair[0] = (uint32_t)first << 16;
#pragma unroll
    for (int j = 1; j <= 4; ++j)
        if (m == 2 * j) pair[j] = last;
    if (!even)
        *static_cast<uint4 *>(dst) = make_uint4(__byte_perm(pair[0], pair[1], 0x5432), __byte_perm(pair[1], pair[2], 0x5432),
                                                __byte_perm(pair[2], pair[3], 0x5432), __byte_perm(pair[3], pair[4], 0x5432));
}
// The same elements, in pairs of floats, to any address.
template <int IO>
__device__ __forceinline__ void store_any16(char *dst, int n, const float2 *v) {
    uint32_t w[5];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack16<IO>(v[j]);
    w[4] = 0;
    if ((reinterpret_cast<size_t>(dst) & 3) == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (2 * j + 1 < n) *reinterpret_cast<uint32_t *>(dst + 4 * j) = w[j];
            else if (2 * j < n) *reinterpret_cast<uint16_t *>(dst + 4 * j) = (uint16_t)w[j];
        }
    } else {
        if (n > 0) *reinterpret_cast<uint16_t *>(dst) = (uint16_t)w[0];
#pragma unroll
        for (int j = 1; j <= 4; ++j) {
            if (2 * j < n) *reinterpret_cast<uint32_t *>(dst + 4 * j - 2) = __byte_perm(w[j - 1], w[j], 0x5432);
            else if (2 * j - 1 < n) *reinterpret_cast<uint16_t *>(dst + 4 * j - 2) = (uint16_t)(w[j - 1] >> 16);
        }
    }
}

// One 16-byte chunk of a row (8 or 4 elements, of which the first n exist) into
// shared memory.  VEC: the chunk is aligned and whole (n is all or none).  fp32
// of any alignment goes element by element, still asynchronously.
template <int IO, bool VEC>
__device__ __forceinline__ void copy_chunk(void *dst, const char *src, int n) {
    if (VEC) {
        cp_async16(dst, n > 0 ? src : nullptr, n > 0 ? 16 : 0);
    } else if (IO == IO_F32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) cp_async4(static_cast<float *>(dst) + j, j < n ? src + 4 * j : nullptr, j < n ? 4 : 0);
    } else {
        copy_any16(dst, src, n);
    }
}

// Four elements of a row, of which the first n exist, in the same way (8 or 16 bytes).
template <int IO, bool VEC>
__device__ __forceinline__ void copy_quad(void *dst, const char *src, int n) {
    if (IO == IO_F32) {
        copy_chunk<IO_F32, VEC>(dst, src, n);
    } else if (VEC) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
                     "l"(n > 0 ? src : nullptr), "r"(n > 0 ? 8 : 0) : "memory");
    } else {
        uint16_t e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            e[j] = 0;
            ldg_u16(e[j], src + 2 * j, j < n);
        }
        *static_cast<uint2 *>(dst) = make_uint2(e[0] | ((uint32_t)e[1] << 16), e[2] | ((uint32_t)e[3] << 16));
    }
}
template <int IO>
__device__ __forceinline__ void read_quad(const void *src, float2 (&v)[2]) {
    if (IO == IO_F32) {
        const float4 f = *static_cast<const float4 *>(src);
        v[0] = make_float2(f.x, f.y);
        v[1] = make_float2(f.z, f.w);
    } else {
        const uint2 u = *static_cast<const uint2 *>(src);
        const uint32_t w[2] = {u.x, u.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (IO == IO_BF16) v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
            else v[i] = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        }
    }
}

// A chunk from shared memory as pairs of floats.
template <int IO>
__device__ __forceinline__ void read_chunk(const void *src, float2 *v) {
    const uint4 u = *static_cast<const uint4 *>(src);
    if (IO == IO_F32) {
        v[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
        v[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (IO == IO_BF16) v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
            else v[i] = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        }
    }
}

// A chunk's values to global memory, the first n of them (VEC: all, aligned).
template <int IO, bool VEC>
__device__ __forceinline__ void store_chunk(char *dst, int n, const float2 *v) {
    if (n <= 0) return;
    if (VEC) {
        uint4 u;
        uint32_t *w = &u.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (IO == IO_F32) {
                w[i] = __float_as_uint(i & 1 ? v[i / 2].y : v[i / 2].x);
            } else if (IO == IO_BF16) {
                const __nv_bfloat162 a = __floats2bfloat162_rn(v[i].x, v[i].y);
                w[i] = *reinterpret_cast<const uint32_t *>(&a);
            } else {
                const __half2 a = __floats2half2_rn(v[i].x, v[i].y);
                w[i] = *reinterpret_cast<const uint32_t *>(&a);
            }
        }
        *reinterpret_cast<uint4 *>(dst) = u;
    } else if (IO != IO_F32) {
        store_any16<IO>(dst, n, v);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (2 * i < n) st_io<IO>(dst, 2 * i, v[i].x);
            if (2 * i + 1 < n) st_io<IO>(dst, 2 * i + 1, v[i].y);
        }
    }
}

// Pairs of a chunk into or out of fp32 shared memory.  `flip` (threads of odd
// groups of four): the halves of an 8-element chunk go in the other order, since
// threads 32 bytes apart would meet in a bank.
template <int KP>
__device__ __forceinline__ void spread(float *dst, const float2 *v, bool flip) {
    const float4 a = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    if (KP == 2) {
        *reinterpret_cast<float4 *>(dst) = a;
        return;
    }
    const float4 c = make_float4(v[KP - 2].x, v[KP - 2].y, v[KP - 1].x, v[KP - 1].y);
    *reinterpret_cast<float4 *>(dst + (flip ? 4 : 0)) = flip ? c : a;
    *reinterpret_cast<float4 *>(dst + (flip ? 0 : 4)) = flip ? a : c;
}
template <int KP>
__device__ __forceinline__ void gather(const float *src, float2 *v, bool flip) {
    float4 a = *reinterpret_cast<const float4 *>(src + (KP == 4 && flip ? 4 : 0));
    if (KP == 4) {
        const float4 c = *reinterpret_cast<const float4 *>(src + (flip ? 0 : 4)), lo = flip ? c : a, hi = flip ? a : c;
        v[KP - 2] = make_float2(hi.x, hi.y);
        v[KP - 1] = make_float2(hi.z, hi.w);
        a = lo;
    }
    v[0] = make_float2(a.x, a.y);
    v[1] = make_float2(a.z, a.w);
}

// One element, where `ok`.
template <int IO>
__device__ __forceinline__ float load_one(const void *base, long long i, bool ok) {
    if (IO == IO_F32) {
        uint32_t w = 0;
        ldg_u32(w, static_cast<const uint32_t *>(base) + i, ok);
        return __uint_as_float(w);
    }
    uint16_t h = 0;
    ldg_u16(h, static_cast<const uint16_t *>(base) + i, ok);
    return IO == IO_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}

template <int IO, bool VEC>
__device__ __forceinline__ void store4_io(void *base, long long i, int nv, const float (&v)[4]) {
    if (!VEC) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < nv) st_io<IO>(base, (size_t)(i + j), v[j]);
        return;
    }
    if (IO == IO_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(base) + i) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        uint2 u;
        if (IO == IO_BF16) {
            __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
            u.x = *reinterpret_cast<uint32_t *>(&a); u.y = *reinterpret_cast<uint32_t *>(&b);
        } else {
            __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
            u.x = *reinterpret_cast<uint32_t *>(&a); u.y = *reinterpret_cast<uint32_t *>(&b);
        }
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(base) + i) = u;
    }
}

// The shared memory of a CTA: 227 KB, less a little for a kernel's static arrays.
constexpr int kSmemMost = 227 * 1024 - 1024;

// Lets a kernel be launched with up to BYTES of dynamic shared memory.  The limit belongs to the
// function, not to the launch, and another host thread may set it between this one's
// setting and its launch: so BYTES is a constant of the kernel, the most that any call of it takes.
template <int BYTES, class K>
cudaError_t allow_smem(K *kernel) {
    static_assert(BYTES <= kSmemMost, "more shared memory than a CTA may hold");
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
}

// A launch that may start while the kernel before it on the stream still runs (`after`):
// that one has let it with pdl_launch_dependents, and this one's threads all begin with
// pdl_wait, so nothing is read or written early; what is saved is the gap between the two.
// What the kernel before wrote is read by plain or L2 loads, never by read-only ones.
template <class... P, class... A>
cudaError_t launch_kernel(bool after, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = after ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...), last = cudaGetLastError();
    return e != cudaSuccess ? e : last;
}

// Four fp32 values of a [*,N] row from column n on; zeros past N.
__device__ __forceinline__ void load_n4(const float *base, long long i, int n, int N, bool vec, float (&v)[4]) {
    if (vec && n + 4 <= N) {
        const float4 f = *reinterpret_cast<const float4 *>(base + i);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = n + j < N ? base[i + j] : 0.f;
    }
}

__device__ __forceinline__ void store_n4(float *base, long long i, int n, int N, bool vec, float a, float b, float c,
                                         float d) {
    if (vec && n + 4 <= N) {
        *reinterpret_cast<float4 *>(base + i) = make_float4(a, b, c, d);
    } else {
        const float v[4] = {a, b, c, d};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < N) base[i + j] = v[j];
    }
}

__device__ __forceinline__ bool aligned_n4(const float *p, int N) {
    return N % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

// Whether groups of four elements of a [B,L,...] tensor sit on boundaries of four elements (host).
inline bool chunk_aligned(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
inline bool chunk_strided(const void *p, int io, const long long (&st)[2]) {
    const int n = io == IO_F32 ? 4 : 8;
    return chunk_aligned(p) && st[0] % n == 0 && st[1] % n == 0;
}
inline bool vec4_aligned(const void *p, int io) { return reinterpret_cast<uintptr_t>(p) % (io == IO_F32 ? 16 : 8) == 0; }
inline bool vec4_strided(const void *p, int io, const long long (&st)[2]) {
    return vec4_aligned(p, io) && st[0] % 4 == 0 && st[1] % 4 == 0;
}

// The clamp of a step.  NaN stays NaN: fminf and fmaxf would return the limit instead.
__device__ __forceinline__ float clamp_step(float v, float lo, float hi) {
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(v), "f"(lo));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(v), "f"(hi));
    return v;
}

// d_t of one raw step.  softplus(v) = max(v, 0) + log1p(w), w = exp(-|v|) in
// (0, 1]: log1p(w) = w P(w) with P of degree 8 fitted for the smallest
// relative error on [0, 1] (1.6e-7 with fp32 evaluation), which keeps the full
// relative precision of small steps, where log(1 + w) loses it.  w is exp2 of
// the rounded product |v| log2(e) corrected to first order by the product's
// rounding error.  sig = d softplus / dv = 1 / (1 + exp(-v)), zero where the clamp is active.
struct StepOut {
    float d, sig;
};

template <bool SIG>
__device__ __forceinline__ StepOut step_of(float raw, float bias, int softplus, int has_limit, float dmin, float dmax) {
    StepOut o;
    const float v = raw + bias;
    o.sig = 1.f;
    if (softplus) {
        const float av = -fminf(fabsf(v), 100.f);  // exp(-100) is 0 in fp32's normal range
        const float t = av * kLog2e;
        const float e = fmaf(av, 1.92596299e-8f, fmaf(av, kLog2e, -t));  // log2(e) - fl(log2(e))
        const float w0 = ex2(t);
        const float w = fmaf(w0, e * kLn2, w0);
        float p = 0.005232690833508968f;
        p = fmaf(p, w, -0.029505228623747826f);
        p = fmaf(p, w, 0.07822594791650772f);
        p = fmaf(p, w, -0.13663245737552643f);
        p = fmaf(p, w, 0.19106008112430573f);
        p = fmaf(p, w, -0.2484298199415207f);
        p = fmaf(p, w, 0.3331909775733948f);
        p = fmaf(p, w, -0.4999949336051941f);
        p = fmaf(p, w, 0.9999999403953552f);
        float m;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(v), "f"(0.f));
        o.d = fmaf(w, p, m);
        if (SIG) o.sig = __fdividef(v >= 0.f ? 1.f : w, 1.f + w);
    } else {
        o.d = v;
    }
    if (has_limit) {
        if (SIG && (o.d < dmin || o.d > dmax)) o.sig = 0.f;
        o.d = clamp_step(o.d, dmin, dmax);
    }
    return o;
}

// step_of for 2 K channels at once, d only: v holds raw + bias.  The options are
// tested once around all of them, so that the K chains of operations interleave.
template <int K>
__device__ __forceinline__ void steps_of(float2 (&v)[K], int softplus, int has_limit, float dmin, float dmax) {
    if (softplus) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const float2 av = make_float2(-fminf(fabsf(v[i].x), 100.f), -fminf(fabsf(v[i].y), 100.f));
            const float2 t = __fmul2_rn(av, dup(kLog2e));
            const float2 e = __ffma2_rn(av, dup(1.92596299e-8f), __ffma2_rn(av, dup(kLog2e), make_float2(-t.x, -t.y)));
            const float2 w0 = ex2_2(t);
            const float2 w = __ffma2_rn(w0, __fmul2_rn(e, dup(kLn2)), w0);
            float2 p = dup(0.005232690833508968f);
            p = __ffma2_rn(p, w, dup(-0.029505228623747826f));
            p = __ffma2_rn(p, w, dup(0.07822594791650772f));
            p = __ffma2_rn(p, w, dup(-0.13663245737552643f));
            p = __ffma2_rn(p, w, dup(0.19106008112430573f));
            p = __ffma2_rn(p, w, dup(-0.2484298199415207f));
            p = __ffma2_rn(p, w, dup(0.3331909775733948f));
            p = __ffma2_rn(p, w, dup(-0.4999949336051941f));
            p = __ffma2_rn(p, w, dup(0.9999999403953552f));
            float2 m;
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(m.x) : "f"(v[i].x), "f"(0.f));
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(m.y) : "f"(v[i].y), "f"(0.f));
            v[i] = __ffma2_rn(w, p, m);
        }
    }
    if (has_limit) {
#pragma unroll
        for (int i = 0; i < K; ++i)
            v[i] = make_float2(clamp_step(v[i].x, dmin, dmax), clamp_step(v[i].y, dmin, dmax));
    }
}

__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// sigmoid and silu of two numbers; 1 + exp(-v) = inf gives 0, the limit.
__device__ __forceinline__ float2 sigmoid2(float2 v) {
    const float2 e = __fadd2_rn(ex2_2(__fmul2_rn(v, dup(-kLog2e))), dup(1.f));
    return make_float2(rcp_approx(e.x), rcp_approx(e.y));
}
__device__ __forceinline__ float2 silu2(float2 v) { return __fmul2_rn(v, sigmoid2(v)); }

cudaError_t launch_scan(const ScanParams &p, int io, cudaStream_t s);
cudaError_t launch_scan_ckpt(const ScanParams &p, int io, cudaStream_t s);  // and the adjoint after every segment
cudaError_t launch_scan_bwd(const ScanParams &p, int io, void *dB, void *dC, float *dA, float *dD, float *dbias,
                            cudaStream_t s);
int scan_bwd_tiles(const ScanParams &p);
int scan_sm_count();

// n-columns are dealt four to a lane: lanes per channel for N states.
inline int scan_lanes(int64_t N) {
    int l = 2;
    while (l * 4 < N) l *= 2;
    return l;
}
// Warps of a CTA of the forward's walk.  With two lanes per channel, two: four would hand
// the four side warps 128 channels, and those would be what the walk waits for ([8,4096,4096,N] in
// bf16 at N = 8 and 4: 529 and 812 us with two, 668 and 1166 with four).
constexpr int scan_walk_warps(int lanes) { return lanes == 2 ? 2 : 4; }

}  // namespace ssd

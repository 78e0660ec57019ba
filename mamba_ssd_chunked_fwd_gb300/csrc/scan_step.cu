// scan_step.cu -- one token of the selective scan and of its convolution for
// each of B sequences, from carried states in a pool of slots.
//
//   scan:  h' = exp(d A[c,:]) h + d x[c] B,  y[c] = (h' . C + Dskip[c] x[c]) silu(z[c])
//   conv:  y[c] = silu(bias[c] + sum_k w[c,k] v[k]),  v = (state rows, x);  state' = v[1:]
//
// Both read and write their state once and are bound by it: 8 N bytes per
// channel for the scan, 4 (W-1) bytes for a 16-bit convolution.
#include "scan_common.cuh"

namespace ssd {

namespace {

// LPC lanes hold a channel's states, four to a lane, so a warp reads and
// writes 512 consecutive bytes of the state; the LPC lanes' parts of y meet in
// xor exchanges.  Each lane repeats its channel's softplus: about 30 operations
// beside 32 bytes of state.  CPT channels per lane, their loads issued
// together; B and C are loaded once for them.
constexpr int kStepThreads = 128;

template <int IO, int LPC, int CPT, bool VEC>
__global__ void __launch_bounds__(kStepThreads)
scan_step_kernel(ScanStepParams p) {
    constexpr int kCh = kStepThreads / LPC;  // channels per CTA and round
    const int b = blockIdx.y;
    const int ln = threadIdx.x % LPC, n0 = ln * 4;
    const int cb = blockIdx.x * (kCh * CPT) + threadIdx.x / LPC;
    const long long slot = p.slots ? __ldg(p.slots + b) : b;
    const bool live = slot >= 0 && slot < p.nslots;
    const long long s0 = slot * p.D * p.N;
    const int dg = p.D / p.G, nn = p.N - n0;
    Raw4 rs[CPT], ra[CPT], rb[CPT], rc[CPT];
    float x[CPT], raw[CPT], z[CPT], bias[CPT], skip[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {  // every load first
        const int c = cb + k * kCh;
        const bool ok = live && c < p.D, okn = ok && nn > 0;
        const long long i = (long long)c * p.N + n0, gn = (long long)(c / dg) * p.N + n0;
        rs[k] = load_raw4<IO_F32, VEC, false>(p.state, s0 + i, okn, nn);
        ra[k] = load_raw4<IO_F32, VEC>(p.A, i, okn, nn);
        rb[k] = load_raw4<IO, VEC>(p.Bm, b * p.b_row + gn, okn, nn);
        rc[k] = load_raw4<IO, VEC>(p.Cm, b * p.c_row + gn, okn, nn);
        x[k] = load_one<IO>(p.x, b * p.x_row + c, ok);
        raw[k] = load_one<IO>(p.dt, b * p.dt_row + c, ok && (IO == IO_F32 || !p.dt32));
        if (IO != IO_F32) raw[k] += load_one<IO_F32>(p.dt, b * p.dt_row + c, ok && p.dt32);  // one of the two is 0
        z[k] = load_one<IO>(p.z, b * p.z_row + c, ok && p.z);
        bias[k] = load_one<IO_F32>(p.dt_bias, c, ok && p.dt_bias);
        skip[k] = load_one<IO_F32>(p.Dskip, c, ok && p.Dskip);
    }
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int c = cb + k * kCh;
        const bool in = live && c < p.D;
        float acc = 0.f;
        if (in) {
            const float d = step_of<false>(raw[k], bias[k], p.softplus, p.has_limit, p.dt_min, p.dt_max).d;
            const float dx = d * x[k];
            float o[4], s[4], a[4], bv[4], cv[4];
            unpack4<IO_F32, VEC>(rs[k], s);
            unpack4<IO_F32, VEC>(ra[k], a);
            unpack4<IO, VEC>(rb[k], bv);
            unpack4<IO, VEC>(rc[k], cv);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                o[j] = fmaf(ex2(fmaf(d, a[j] * kLog2e, kDecayCentre)), s[j], dx * bv[j]);
                acc = fmaf(o[j], cv[j], acc);
            }
            store_n4(p.state_out + s0, (long long)c * p.N + n0, n0, p.N, VEC, o[0], o[1], o[2], o[3]);
        }
#pragma unroll
        for (int off = LPC / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
        if (ln == 0 && c < p.D) {
            float y = 0.f;
            if (live) {
                y = p.Dskip ? fmaf(skip[k], x[k], acc) : acc;
                if (p.z) y *= silu_fast(z[k]);
            }
            st_io<IO>(p.y, (size_t)b * p.D + c, y);
        }
    }
}

template <int IO, int LPC>
cudaError_t launch_step_as(const ScanStepParams &p, cudaStream_t s) {
    constexpr int kCh = kStepThreads / LPC;
    // Four channels per lane once that still gives every SM eight CTAs: more bytes in flight per lane;
    // below that one channel per lane spreads the few channels over more SMs.
    const long long ctas4 = (long long)p.B * ((p.D + 4 * kCh - 1) / (4 * kCh));
    const bool vec = p.N % 4 == 0 && vec4_aligned(p.state, IO_F32) && vec4_aligned(p.state_out, IO_F32) &&
                     vec4_aligned(p.A, IO_F32) && vec4_aligned(p.Bm, IO) && vec4_aligned(p.Cm, IO) &&
                     p.b_row % 4 == 0 && p.c_row % 4 == 0;
    const bool many = ctas4 >= 8LL * scan_sm_count();
    const dim3 grid(many ? (p.D + 4 * kCh - 1) / (4 * kCh) : (p.D + kCh - 1) / kCh, p.B);
    auto *kernel = many ? (vec ? scan_step_kernel<IO, LPC, 4, true> : scan_step_kernel<IO, LPC, 4, false>)
                        : (vec ? scan_step_kernel<IO, LPC, 1, true> : scan_step_kernel<IO, LPC, 1, false>);
    kernel<<<grid, kStepThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <int IO>
cudaError_t launch_step_io(const ScanStepParams &p, cudaStream_t s) {
    switch (scan_lanes(p.N)) {
        case 2: return launch_step_as<IO, 2>(p, s);
        case 4: return launch_step_as<IO, 4>(p, s);
        case 8: return launch_step_as<IO, 8>(p, s);
        case 16: return launch_step_as<IO, 16>(p, s);
        case 32: return launch_step_as<IO, 32>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

// One thread per channel; the W-1 state rows of a sequence are dense, so a
// warp's accesses are consecutive.
template <int IO>
__global__ void __launch_bounds__(256)
conv_step_kernel(ConvStepParams p) {
    const int b = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
    if (c >= p.C) return;
    const long long slot = p.slots ? __ldg(p.slots + b) : b;
    if (slot < 0 || slot >= p.nslots) {
        st_io<IO>(p.y, (size_t)b * p.C + c, 0.f);
        return;
    }
    using T = typename IoTraits<IO>::T;
    const long long s0 = slot * (p.W - 1) * p.C + c;
    const T *in = static_cast<const T *>(p.state) + s0;
    T *out = static_cast<T *>(p.state_out) + s0;
    T v[8];
#pragma unroll
    for (int k = 0; k < 7; ++k)
        if (k < p.W - 1) v[k] = in[(long long)k * p.C];
    const T x = static_cast<const T *>(p.x)[b * p.x_row + c];
    float acc = p.bias ? __ldg(p.bias + c) : 0.f;
#pragma unroll
    for (int k = 0; k < 7; ++k)
        if (k < p.W - 1) {
            acc = fmaf(__ldg(p.w + (long long)c * p.W + k), IoTraits<IO>::to_f(v[k]), acc);
            if (k > 0) out[(long long)(k - 1) * p.C] = v[k];
        }
    acc = fmaf(__ldg(p.w + (long long)c * p.W + p.W - 1), IoTraits<IO>::to_f(x), acc);
    if (p.W > 1) out[(long long)(p.W - 2) * p.C] = x;
    st_io<IO>(p.y, (size_t)b * p.C + c, p.silu ? silu_fast(acc) : acc);
}

}  // namespace

cudaError_t launch_scan_step(const ScanStepParams &p, int io, cudaStream_t s) {
    switch (io) {
        case IO_F32: return launch_step_io<IO_F32>(p, s);
        case IO_F16: return launch_step_io<IO_F16>(p, s);
        case IO_BF16: return launch_step_io<IO_BF16>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_conv_step(const ConvStepParams &p, int io, cudaStream_t s) {
    const dim3 grid((p.C + 255) / 256, p.B);
    switch (io) {
        case IO_F32: conv_step_kernel<IO_F32><<<grid, 256, 0, s>>>(p); break;
        case IO_F16: conv_step_kernel<IO_F16><<<grid, 256, 0, s>>>(p); break;
        case IO_BF16: conv_step_kernel<IO_BF16><<<grid, 256, 0, s>>>(p); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

}  // namespace ssd

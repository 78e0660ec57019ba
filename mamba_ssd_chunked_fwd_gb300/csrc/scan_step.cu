// scan_step.cu -- one token of the selective scan and of its convolution for
// each of B sequences, from carried states in a pool of slots.
//
//   scan:  h' = exp(d A[c,:]) h + d x[c] B,  y[c] = (h' . C + Dskip[c] x[c]) silu(z[c])
//   conv:  y[c] = silu(bias[c] + sum_k w[c,k] v[k]),  v = (state rows, x);  state' = v[1:]
//
// Both read and write their state once and are bound by it: 8 N bytes per
// channel for the scan, 4 (W-1) bytes for a 16-bit convolution.  Measured: 256 sequences
// of 8192 channels, N = 16, in fp16 49 us (5.8 TB/s, 85 % of the copy rate); one sequence
// of 2048 channels 5.5 to 7.9 us called in turn, the host's part; the convolution of 64 sequences 6.2 to 8.5 us.
#include "scan_common.cuh"

namespace ssd {

namespace {

// LPC lanes hold a channel's states, four to a lane, so a warp reads and
// writes 512 consecutive bytes of the state.  A lane takes the same channel of
// NB sequences: A is loaded once for them, and with NB = 4 lane j of a group
// works out the step of sequence j (the softplus, about 25 operations) and
// hands it to the others, then ends up with sequence j's sum over the lanes
// (halving exchanges), its gate and its store.
constexpr int kStepThreads = 128;

template <int IO, int LPC, int NB, bool VEC>
__global__ void __launch_bounds__(kStepThreads)
scan_step_kernel(ScanStepParams p) {
    static_assert(NB == 1 || (NB == 4 && LPC >= 4), "one lane of the group per sequence");
    constexpr int kCh = kStepThreads / LPC;  // channels per CTA
    const int lane = threadIdx.x & 31, ln = threadIdx.x % LPC, n0 = ln * 4, nn = p.N - n0;
    const int c = blockIdx.x * kCh + threadIdx.x / LPC;
    const int b0 = blockIdx.y * NB;
    const bool ch = c < p.D;
    const int dg = p.D / p.G;
    const long long i = (long long)c * p.N + n0, gn = (long long)(c / dg) * p.N + n0;
    long long s0[NB];
    bool live[NB];
    Raw4 rs[NB], rb[NB], rc[NB], ra;
#pragma unroll
    for (int k = 0; k < NB; ++k) {  // every load first
        const int b = b0 + k;
        long long slot = -1;
        if (b < p.B) slot = p.slots ? __ldg(p.slots + b) : b;
        live[k] = slot >= 0 && slot < p.nslots;
        s0[k] = slot * p.D * p.N;
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
        const int b = b0 + k;
        const bool ok = live[k] && ch && nn > 0;
        rs[k] = load_raw4<IO_F32, VEC, false>(p.state, s0[k] + i, ok, nn);
        rb[k] = load_raw4<IO, VEC>(p.Bm, b * p.b_row + gn, ok, nn);
        rc[k] = load_raw4<IO, VEC>(p.Cm, b * p.c_row + gn, ok, nn);
    }
    ra = load_raw4<IO_F32, VEC>(p.A, i, ch && nn > 0, nn);
    const int mine = NB == 1 ? 0 : ln & 3, bm = b0 + mine;  // the sequence whose step is this lane's
    const bool okm = ch && (NB == 1 ? live[0] : mine == 0 ? live[0] : mine == 1 ? live[NB > 1] : mine == 2 ? live[NB > 2 ? 2 : 0] : live[NB > 3 ? 3 : 0]);
    const float x = load_one<IO>(p.x, bm * p.x_row + c, okm);
    float raw = load_one<IO>(p.dt, bm * p.dt_row + c, okm && (IO == IO_F32 || !p.dt32));
    if (IO != IO_F32) raw += load_one<IO_F32>(p.dt, bm * p.dt_row + c, okm && p.dt32);  // one of the two is 0
    const float z = load_one<IO>(p.z, bm * p.z_row + c, okm && p.z);
    const float bias = load_one<IO_F32>(p.dt_bias, c, ch && p.dt_bias), skip = load_one<IO_F32>(p.Dskip, c, ch && p.Dskip);
    const float d = step_of<false>(raw, bias, p.softplus, p.has_limit, p.dt_min, p.dt_max).d, dx = d * x;
    float a[4], acc[NB];
    unpack4<IO_F32, VEC>(ra, a);
    const float2 a0 = make_float2(a[0] * kLog2e, a[1] * kLog2e), a1 = make_float2(a[2] * kLog2e, a[3] * kLog2e);
#pragma unroll
    for (int k = 0; k < NB; ++k) {
        const int src = (lane & ~(LPC - 1)) | k;
        const float2 dk = dup(NB == 1 ? d : __shfl_sync(0xffffffffu, d, src));
        const float2 wk = dup(NB == 1 ? dx : __shfl_sync(0xffffffffu, dx, src));
        float s[4], bv[4], cv[4];
        unpack4<IO_F32, VEC>(rs[k], s);
        unpack4<IO, VEC>(rb[k], bv);
        unpack4<IO, VEC>(rc[k], cv);
        const float2 h0 = __ffma2_rn(decay2(dk, a0), make_float2(s[0], s[1]), __fmul2_rn(wk, make_float2(bv[0], bv[1])));
        const float2 h1 = __ffma2_rn(decay2(dk, a1), make_float2(s[2], s[3]), __fmul2_rn(wk, make_float2(bv[2], bv[3])));
        const float2 v = __ffma2_rn(h1, make_float2(cv[2], cv[3]), __fmul2_rn(h0, make_float2(cv[0], cv[1])));
        acc[k] = v.x + v.y;
        if (live[k] && ch) store_n4(p.state_out + s0[k], i, n0, p.N, VEC, h0.x, h0.y, h1.x, h1.y);
    }
    float y;
    if (NB == 1) {
        y = acc[0];
#pragma unroll
        for (int off = LPC / 2; off > 0; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
    } else {  // lane bit 1, then bit 0, choose the sequence a lane is left with: its own
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const bool hi = lane & 2;
            const float keep = hi ? acc[NB > 1 ? k + 2 : 0] : acc[NB > 1 ? k : 0], send = hi ? acc[NB > 1 ? k : 0] : acc[NB > 1 ? k + 2 : 0];
            acc[NB > 1 ? k : 0] = keep + __shfl_xor_sync(0xffffffffu, send, 2);
        }
        const bool hi = lane & 1;
        const float keep = hi ? acc[NB > 1] : acc[0], send = hi ? acc[0] : acc[NB > 1];
        y = keep + __shfl_xor_sync(0xffffffffu, send, 1);
#pragma unroll
        for (int off = 4; off < LPC; off <<= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
    }
    if (ln < NB && ch && bm < p.B) {
        y = p.Dskip ? fmaf(skip, x, y) : y;
        if (p.z) y *= silu_fast(z);
        st_io<IO>(p.y, (size_t)bm * p.D + c, okm ? y : 0.f);
    }
}

template <int IO, int LPC>
cudaError_t launch_step_as(const ScanStepParams &p, cudaStream_t s) {
    constexpr int kCh = kStepThreads / LPC;
    const bool vec = p.N % 4 == 0 && vec4_aligned(p.state, IO_F32) && vec4_aligned(p.state_out, IO_F32) &&
                     vec4_aligned(p.A, IO_F32) && vec4_aligned(p.Bm, IO) && vec4_aligned(p.Cm, IO) &&
                     p.b_row % 4 == 0 && p.c_row % 4 == 0;
    const int tiles = (p.D + kCh - 1) / kCh;
    // Four sequences per lane once that leaves every SM four CTAs; below, one, so
    // that the few channels reach more SMs.  Two lanes per channel take one.  256
    // sequences of 8192 channels: 50 us by fours, 78 by one; 64 and 16 of 2048: level, 10.9 and 8.8 (with events around).
    if constexpr (LPC >= 4) {
        if ((long long)tiles * (p.B / 4) >= 4LL * scan_sm_count()) {
            auto *kernel = vec ? scan_step_kernel<IO, LPC, 4, true> : scan_step_kernel<IO, LPC, 4, false>;
            kernel<<<dim3(tiles, (p.B + 3) / 4), kStepThreads, 0, s>>>(p);
            return cudaGetLastError();
        }
    }
    auto *kernel = vec ? scan_step_kernel<IO, LPC, 1, true> : scan_step_kernel<IO, LPC, 1, false>;
    kernel<<<dim3(tiles, p.B), kStepThreads, 0, s>>>(p);
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

// Four channels per thread; the W-1 state rows of a sequence are dense, so a
// warp's accesses are consecutive.  A row's taps come in one load when W is 4.
template <int IO, bool VEC>
__global__ void __launch_bounds__(128)
conv_step_kernel(ConvStepParams p) {
    const int b = blockIdx.y, c = (blockIdx.x * 128 + threadIdx.x) * 4;
    if (c >= p.C) return;
    const int nv = min(4, p.C - c), W1 = p.W - 1;
    const long long slot = p.slots ? __ldg(p.slots + b) : b;
    const long long out = (long long)b * p.C + c;
    if (slot < 0 || slot >= p.nslots) {
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        store4_io<IO, VEC>(p.y, out, nv, zero);
        return;
    }
    const long long s0 = slot * W1 * p.C + c;
    Raw4 r[8];
    float w[4][8];
#pragma unroll
    for (int k = 0; k < 7; ++k) r[k] = load_raw4<IO, VEC, false>(p.state, s0 + (long long)k * p.C, k < W1, nv);
    const Raw4 rx = load_raw4<IO, VEC>(p.x, b * p.x_row + c, 1, nv);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const long long at = (long long)(c + j) * p.W;
        if (VEC && p.W == 4) {
            const Raw4 t = load_raw4<IO_F32, true>(p.w, at, 1, 4);
#pragma unroll
            for (int k = 0; k < 8; ++k) w[j][k] = k < 4 ? __uint_as_float(t.w[k & 3]) : 0.f;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) w[j][k] = load_one<IO_F32>(p.w, at + k, k < p.W && j < nv);
        }
    }
    float acc[4], v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = load_one<IO_F32>(p.bias, c + j, p.bias && j < nv);
#pragma unroll
    for (int k = 0; k < 8; ++k) {  // the W entries in order: the state's, then x
        if (k < W1) unpack4<IO, VEC>(r[k < 7 ? k : 0], v);
        else unpack4<IO, VEC>(rx, v);
        if (k < p.W) {
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = fmaf(w[j][k], v[j], acc[j]);
            if (k > 0) store4_io<IO, VEC>(p.state_out, s0 + (long long)(k - 1) * p.C, nv, v);
        }
    }
    if (p.silu) {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = silu_fast(acc[j]);
    }
    store4_io<IO, VEC>(p.y, out, nv, acc);
}

template <int IO>
cudaError_t launch_conv_step_io(const ConvStepParams &p, cudaStream_t s) {
    const bool vec = p.C % 4 == 0 && p.x_row % 4 == 0 && vec4_aligned(p.x, IO) && vec4_aligned(p.state, IO) &&
                     vec4_aligned(p.state_out, IO) && vec4_aligned(p.y, IO) && vec4_aligned(p.w, IO_F32);
    auto *kernel = vec ? conv_step_kernel<IO, true> : conv_step_kernel<IO, false>;
    kernel<<<dim3((p.C + 511) / 512, p.B), 128, 0, s>>>(p);
    return cudaGetLastError();
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
    switch (io) {
        case IO_F32: return launch_conv_step_io<IO_F32>(p, s);
        case IO_F16: return launch_conv_step_io<IO_F16>(p, s);
        case IO_BF16: return launch_conv_step_io<IO_BF16>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace ssd

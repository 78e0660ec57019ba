// scan_api.cu -- C entries of the selective scan, its convolution and the
// block norm: validation, segments, workspace layout, launches.  Host code only.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <initializer_list>

#include "scan_common.cuh"

namespace {

ssd_status fail(ssd_status st, const char *fmt, ...) {
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return ssd::report_error(st, msg);
}

ssd_status ok() { return ssd::report_error(SSD_OK, ""); }

ssd_status cuda_fail(cudaError_t e, const char *where) {
    return fail(SSD_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

constexpr int64_t kMaxDim = 0x7fffffffLL - 65536;  // sums of an index and a tile stay in 32 bits
size_t align_up(size_t v) { return (v + 255) / 256 * 256; }
bool known_dtype(int32_t d) { return d == SSD_F32 || d == SSD_F16 || d == SSD_BF16; }
bool aligned256(const void *p) { return reinterpret_cast<uintptr_t>(p) % 256 == 0; }

// Strides of a [B,L,...] tensor whose tokens are `width` wide; both zero: dense.
bool strides_of(const int64_t (&in)[2], int64_t L, int64_t width, long long (&out)[2]) {
    out[0] = in[0];
    out[1] = in[1];
    if (in[0] == 0 && in[1] == 0) {
        out[0] = L * width;
        out[1] = width;
    }
    return in[0] >= 0 && in[1] >= 0;
}

size_t element(int32_t dtype) { return dtype == SSD_F32 ? 4 : 2; }

// Whether two ranges of memory share bytes (an absent or empty one shares none).
bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x && y && na && nb && x < y + nb && y < x + na;
}

// A tensor's range of memory, under the name that an error gives it.
struct Span {
    const void *p;
    size_t bytes;
    const char *what;
};

// An output must lie apart from tensors that other threads read while it is written, and from other outputs.
ssd_status apart(const Span &out, std::initializer_list<Span> others) {
    for (const Span &o : others)
        if (overlap(out.p, out.bytes, o.p, o.bytes)) return fail(SSD_ERR_INVALID_ARG, "%s must not overlap %s", out.what, o.what);
    return SSD_OK;
}

// What a [B,L,...] tensor reaches over through its strides; `st` as strides_of gives them.
Span strided(const void *p, int64_t B, int64_t L, int64_t width, const long long (&st)[2], size_t es, const char *what) {
    return {p, ((size_t)(B - 1) * st[0] + (size_t)(L - 1) * st[1] + width) * es, what};
}

// The same for a tensor of y's shape that y may replace: where it is dense, of y's type and
// at y's address, an element is read by the thread that writes it, before it does, and nothing is left to compare.
Span replaced(const void *y, int32_t y_dtype, const void *p, int32_t dtype, int64_t B, int64_t L, int64_t width,
              const long long (&st)[2], const char *what) {
    const bool dense = (B == 1 || st[0] == L * width) && (L == 1 || st[1] == width);
    if (p == y && dtype == y_dtype && dense) return {nullptr, 0, what};
    return strided(p, B, L, width, st, element(dtype), what);
}

ssd_status check_limit(float dt_min, float dt_max) {
    if (isnan(dt_min) || isnan(dt_max) || !(dt_min <= dt_max))
        return fail(SSD_ERR_INVALID_ARG, "dt_limit must satisfy dt_min <= dt_max");
    return SSD_OK;
}

bool limited(float dt_min, float dt_max) { return !(dt_min == 0.f && isinf(dt_max) && dt_max > 0.f); }

ssd_status check_scan_shape(const ssd_scan_args *a) {
    if (!a) return fail(SSD_ERR_INVALID_ARG, "args is NULL");
    if (a->B <= 0 || a->L <= 0 || a->D <= 0 || a->N <= 0 || a->G <= 0)
        return fail(SSD_ERR_INVALID_ARG, "every dim must be > 0 (B=%lld L=%lld D=%lld N=%lld G=%lld)", (long long)a->B,
                    (long long)a->L, (long long)a->D, (long long)a->N, (long long)a->G);
    if (a->D % a->G != 0)
        return fail(SSD_ERR_INVALID_ARG, "D (%lld) must be a multiple of G (%lld)", (long long)a->D, (long long)a->G);
    if (a->N > 128) return fail(SSD_ERR_UNSUPPORTED, "N must be <= 128 (got %lld)", (long long)a->N);
    if (a->B > 65535 || a->L > kMaxDim || a->D > (1 << 24))
        return fail(SSD_ERR_UNSUPPORTED, "B <= 65535, L < 2^31 - 65536 and D <= 2^24 required");
    if (!known_dtype(a->x_dtype)) return fail(SSD_ERR_INVALID_ARG, "unknown dtype code %d", a->x_dtype);
    if (!known_dtype(a->dt_dtype)) return fail(SSD_ERR_INVALID_ARG, "unknown dtype code %d", a->dt_dtype);
    if (a->dt_dtype != a->x_dtype && a->dt_dtype != SSD_F32)
        return fail(SSD_ERR_UNSUPPORTED, "dt must have the dtype of x or fp32");
    return check_limit(a->dt_min, a->dt_max);
}

// The cut of the sequences into n segments.  A CTA of the forward's walk advances a
// token in about 0.096 us alone on its SM, two that share one in 0.165 us, so a walk
// by few CTAs is cut until there are CTAs for the SMs.  The cut costs a first walk
// (each segment's state from zero, 0.65 of the forward's time; backwards as many CTAs
// again walk for the adjoint), a fold over the segments, whose states move four times, and
// two launches.  Unit: the token of a CTA alone.  Uncut and cut by this rule: [1,16384,2048,16]
// 1571 and 278 us, gradients of [2,333,328,8] 121 and 32; where the SMs are full, nothing is cut.
void choose_segments(ssd::ScanParams &p, bool backward) {
    const int lanes = ssd::scan_lanes(p.N);
    // Backwards the model was fitted with CTAs of four walk warps, and keeps that count where N <= 8 takes two: with
    // two it cuts less, [4,2048,4096,8] 977 us instead of 640 ([6,8923,648,8] 1127 instead of 1166).
    const int dc = (backward ? 4 : ssd::scan_walk_warps(lanes)) * (32 / lanes) * 4;
    const double sms = ssd::scan_sm_count(), pair = 1.72;
    const double ctas = (double)p.B * p.G * ((p.D / p.G + dc - 1) / dc), state = (double)p.B * p.D * p.N;
    auto waves = [&](double k) {
        const double full = floor(k / (2 * sms)), rest = k - full * 2 * sms;
        return full * pair + (rest == 0. ? 0. : rest <= sms ? 1. : pair);
    };
    auto cost = [&](long long m) {
        const long long len = ((p.L + m - 1) / m + 15) / 16 * 16, n = (p.L + len - 1) / len;
        const double walk = waves(ctas * n), first = waves((backward ? 2. : 1.) * ctas * (n - 1));
        const double cut = n > 1 ? 0.65 * first * len + 1.5 * n + (backward ? 5e-5 : 2.5e-5) * state * n + 90. : 0.;
        return (backward ? 0.8 * walk + 1.7 * waves(2 * ctas * n) : walk) * len + cut;
    };
    long long best = 1;
    for (long long n = 2; n <= 1024 && (p.L + n - 1) / n >= 16; n = n < 8 ? n + 1 : n + n / 4)
        if (cost(n) < cost(best)) best = n;
    p.seg_len = (int)(((p.L + best - 1) / best + 15) / 16 * 16);
    p.nseg = (int)((p.L + p.seg_len - 1) / p.seg_len);
}

ssd_status make_scan(const ssd_scan_args *a, ssd::ScanParams &p) {
    p = ssd::ScanParams{};
    p.B = (int)a->B; p.L = (int)a->L; p.D = (int)a->D; p.N = (int)a->N; p.G = (int)a->G;
    p.x = a->x; p.dt = a->dt; p.A = a->A; p.Bm = a->Bm; p.Cm = a->Cm; p.Dskip = a->Dskip; p.z = a->z;
    p.dt_bias = a->dt_bias; p.h0 = a->initial_state; p.lengths = a->lengths; p.y = a->y;
    p.final_state = a->final_state;
    if (!strides_of(a->x_stride, a->L, a->D, p.xs) || !strides_of(a->dt_stride, a->L, a->D, p.dts) ||
        !strides_of(a->z_stride, a->L, a->D, p.zs) || !strides_of(a->b_stride, a->L, a->G * a->N, p.bs) ||
        !strides_of(a->c_stride, a->L, a->G * a->N, p.cs))
        return fail(SSD_ERR_INVALID_ARG, "strides must be >= 0");
    p.dt32 = a->dt_dtype == SSD_F32;
    p.softplus = a->dt_softplus ? 1 : 0;
    p.has_limit = limited(a->dt_min, a->dt_max);
    p.dt_min = a->dt_min; p.dt_max = a->dt_max;
    return SSD_OK;
}

ssd_status check_scan_inputs(const ssd_scan_args *a) {
    if (!a->x || !a->dt || !a->A || !a->Bm || !a->Cm)
        return fail(SSD_ERR_INVALID_ARG, "x, dt, A, B and C are required");
    return SSD_OK;
}

struct ScanLayout {
    size_t states, sums, total;
};

ScanLayout scan_layout(const ssd::ScanParams &p) {
    ScanLayout l = {0, 0, 0};
    if (p.nseg == 1) return l;
    l.sums = align_up((size_t)p.B * p.nseg * p.D * p.N * sizeof(float));
    l.total = l.sums + align_up((size_t)p.B * p.nseg * p.D * sizeof(float));
    return l;
}

ssd_status check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return SSD_OK;
    if (!ws || have < need)
        return fail(SSD_ERR_WORKSPACE, "workspace of %zu bytes required (got %zu)", need, ws ? have : (size_t)0);
    if (!aligned256(ws)) return fail(SSD_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    return SSD_OK;
}

struct ScanBwdLayout {
    size_t states, sums, adj, ckpt, bc, part_a, part_d, total;
};

ScanBwdLayout scan_bwd_layout(const ssd::ScanParams &p) {
    const size_t f = sizeof(float), dn = (size_t)p.D * p.N;
    ScanBwdLayout l;
    const ScanLayout s = scan_layout(p);
    l.states = s.states;
    l.sums = s.sums;
    l.adj = s.total;
    l.ckpt = l.adj + (p.nseg > 1 ? align_up((size_t)p.B * p.nseg * dn * f) : 0);
    l.bc = l.ckpt + align_up((size_t)p.B * ((p.L + ssd::kCkpt - 1) / ssd::kCkpt) * dn * f);
    l.part_a = l.bc + align_up((size_t)p.G * ssd::scan_bwd_tiles(p) * p.B * p.L * 2 * 4 * ssd::scan_lanes(p.N) * f);
    l.part_d = l.part_a + align_up((size_t)p.B * p.nseg * dn * f);
    l.total = l.part_d + align_up((size_t)2 * p.B * p.nseg * p.D * f);
    return l;
}

ssd_status check_conv(const ssd_conv_args *a, ssd::ConvParams &p) {
    if (!a) return fail(SSD_ERR_INVALID_ARG, "args is NULL");
    if (a->B <= 0 || a->L <= 0 || a->C <= 0 || a->W <= 0)
        return fail(SSD_ERR_INVALID_ARG, "every dim must be > 0 (B=%lld L=%lld C=%lld W=%lld)", (long long)a->B,
                    (long long)a->L, (long long)a->C, (long long)a->W);
    if (a->W > 8) return fail(SSD_ERR_UNSUPPORTED, "W must be <= 8 (got %lld)", (long long)a->W);
    if (a->B > 65535 || a->L > 8000000 || a->C > (1 << 24))
        return fail(SSD_ERR_UNSUPPORTED, "B <= 65535, L <= 8000000 and C <= 2^24 required");
    if (!known_dtype(a->dtype)) return fail(SSD_ERR_INVALID_ARG, "unknown dtype code %d", a->dtype);
    p = ssd::ConvParams{};
    p.B = (int)a->B; p.L = (int)a->L; p.C = (int)a->C; p.W = (int)a->W;
    p.x = a->x; p.w = a->w; p.bias = a->bias; p.h0 = a->initial_state; p.lengths = a->lengths;
    p.y = a->y; p.final_state = a->final_state; p.silu = a->silu ? 1 : 0;
    if (!strides_of(a->x_stride, a->L, a->C, p.xs)) return fail(SSD_ERR_INVALID_ARG, "strides must be >= 0");
    p.run = ssd::conv_bwd_run(p);
    return SSD_OK;
}

size_t conv_bwd_bytes(const ssd::ConvParams &p) {
    return align_up((size_t)ssd::conv_bwd_part_rows(p) * (p.W + 1) * p.C * sizeof(float));
}

ssd_status check_norm(const ssd_block_norm_args *a, ssd::BlockNormParams &p) {
    if (!a) return fail(SSD_ERR_INVALID_ARG, "args is NULL");
    if (a->rows <= 0 || a->D <= 0)
        return fail(SSD_ERR_INVALID_ARG, "rows and D must be > 0 (rows=%lld D=%lld)", (long long)a->rows, (long long)a->D);
    if (a->D > 16384) return fail(SSD_ERR_UNSUPPORTED, "D must be <= 16384 (got %lld)", (long long)a->D);
    if (a->rows > 0x7fffffffLL) return fail(SSD_ERR_UNSUPPORTED, "rows must be < 2^31");
    if (!known_dtype(a->dtype) || !known_dtype(a->stream_dtype))
        return fail(SSD_ERR_INVALID_ARG, "unknown dtype code %d", known_dtype(a->dtype) ? a->stream_dtype : a->dtype);
    if (a->stream_dtype != a->dtype && a->stream_dtype != SSD_F32)
        return fail(SSD_ERR_UNSUPPORTED, "the stream must have the dtype of o or fp32");
    if (!(a->eps >= 0.f && a->eps < INFINITY)) return fail(SSD_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (a->gate && (a->rows_per_gate <= 0 || a->rows % a->rows_per_gate != 0))
        return fail(SSD_ERR_INVALID_ARG, "rows (%lld) must be a multiple of rows_per_gate (%lld)", (long long)a->rows,
                    (long long)a->rows_per_gate);
    if (!a->o && (a->gate || a->w_post || a->scale))
        return fail(SSD_ERR_INVALID_ARG, "gate, w_post and scale need o");
    if (!a->w_pre) return fail(SSD_ERR_INVALID_ARG, "w_pre is required");
    p = ssd::BlockNormParams{};
    p.rows = a->rows; p.rows_per_gate = a->gate ? a->rows_per_gate : 1; p.D = (int)a->D;
    p.o = a->o; p.r = a->r; p.gate = a->gate; p.w_post = a->w_post; p.w_pre = a->w_pre; p.scale = a->scale;
    p.n = a->n; p.r_out = a->r_out; p.eps = a->eps;
    return SSD_OK;
}

size_t norm_bwd_bytes(ssd::BlockNormParams &p) {
    ssd::block_norm_chunks(p);
    return align_up((size_t)p.chunks * 2 * p.D * sizeof(float));
}

}  // namespace

extern "C" {

ssd_status ssd_selective_scan_workspace_size(const ssd_scan_args *a, size_t *bytes) {
    ssd_status st = check_scan_shape(a);
    if (st != SSD_OK) return st;
    if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
    ssd::ScanParams p = {};
    if ((st = make_scan(a, p)) != SSD_OK) return st;
    choose_segments(p, false);
    *bytes = scan_layout(p).total;
    return ok();
}

ssd_status ssd_selective_scan(const ssd_scan_args *a, void *stream) {
    ssd_status st = check_scan_shape(a);
    if (st != SSD_OK) return st;
    if ((st = check_scan_inputs(a)) != SSD_OK) return st;
    if (!a->y) return fail(SSD_ERR_INVALID_ARG, "y is required");
    ssd::ScanParams p = {};
    if ((st = make_scan(a, p)) != SSD_OK) return st;
    const size_t f = sizeof(float), es = element(a->x_dtype), state = (size_t)a->B * a->D * a->N * f, gn = a->G * a->N;
    const Span y = {a->y, (size_t)a->B * a->L * a->D * es, "y"}, fin = {a->final_state, state, "final_state"};
    const Span B = strided(a->Bm, a->B, a->L, gn, p.bs, es, "B"), C = strided(a->Cm, a->B, a->L, gn, p.cs, es, "C"),
               A = {a->A, (size_t)a->D * a->N * f, "A"}, Dskip = {a->Dskip, a->D * f, "Dskip"},
               bias = {a->dt_bias, a->D * f, "dt_bias"}, h0 = {a->initial_state, state, "initial_state"},
               len = {a->lengths, a->B * sizeof(int32_t), "lengths"};
    st = apart(y, {replaced(a->y, a->x_dtype, a->x, a->x_dtype, a->B, a->L, a->D, p.xs, "x"),
                   replaced(a->y, a->x_dtype, a->dt, a->dt_dtype, a->B, a->L, a->D, p.dts, "dt"),
                   replaced(a->y, a->x_dtype, a->z, a->x_dtype, a->B, a->L, a->D, p.zs, "z"), B, C, A, Dskip, bias, h0, len, fin});
    if (st != SSD_OK) return st;
    st = apart(fin, {strided(a->x, a->B, a->L, a->D, p.xs, es, "x"),
                     strided(a->dt, a->B, a->L, a->D, p.dts, element(a->dt_dtype), "dt"),
                     strided(a->z, a->B, a->L, a->D, p.zs, es, "z"), B, C, A, Dskip, bias, h0, len});
    if (st != SSD_OK) return st;
    choose_segments(p, false);
    const ScanLayout l = scan_layout(p);
    if ((st = check_workspace(a->workspace, a->workspace_bytes, l.total)) != SSD_OK) return st;
    char *ws = static_cast<char *>(a->workspace);
    p.seg_states = reinterpret_cast<float *>(ws + l.states);
    p.seg_sum = reinterpret_cast<float *>(ws + l.sums);
    cudaError_t e = ssd::launch_scan(p, a->x_dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "selective_scan");
    return ok();
}

ssd_status ssd_selective_scan_bwd_workspace_size(const ssd_scan_bwd_args *b, size_t *bytes) {
    ssd_status st = check_scan_shape(b ? &b->fwd : nullptr);
    if (st != SSD_OK) return st;
    if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
    ssd::ScanParams p = {};
    if ((st = make_scan(&b->fwd, p)) != SSD_OK) return st;
    choose_segments(p, true);
    *bytes = scan_bwd_layout(p).total;
    return ok();
}

ssd_status ssd_selective_scan_bwd(const ssd_scan_bwd_args *b, void *stream) {
    ssd_status st = check_scan_shape(b ? &b->fwd : nullptr);
    if (st != SSD_OK) return st;
    const ssd_scan_args *a = &b->fwd;
    if ((st = check_scan_inputs(a)) != SSD_OK) return st;
    if (!b->dy || !b->dx || !b->ddt || !b->dA || !b->dB || !b->dC)
        return fail(SSD_ERR_INVALID_ARG, "dy, dx, ddt, dA, dB and dC are required");
    if (a->Dskip && !b->dD) return fail(SSD_ERR_INVALID_ARG, "dD is required with Dskip");
    if (a->z && !b->dz) return fail(SSD_ERR_INVALID_ARG, "dz is required with z");
    if (a->dt_bias && !b->ddt_bias) return fail(SSD_ERR_INVALID_ARG, "ddt_bias is required with dt_bias");
    ssd::ScanParams p = {};
    if ((st = make_scan(a, p)) != SSD_OK) return st;
    choose_segments(p, true);
    const ScanBwdLayout l = scan_bwd_layout(p);
    if ((st = check_workspace(b->workspace, b->workspace_bytes, l.total)) != SSD_OK) return st;
    char *ws = static_cast<char *>(b->workspace);
    p.seg_states = reinterpret_cast<float *>(ws + l.states);
    p.seg_sum = reinterpret_cast<float *>(ws + l.sums);
    p.adj = reinterpret_cast<float *>(ws + l.adj);
    p.ckpt = reinterpret_cast<float *>(ws + l.ckpt);
    p.part_bc = reinterpret_cast<float *>(ws + l.bc);
    p.part_a = reinterpret_cast<float *>(ws + l.part_a);
    p.part_d = reinterpret_cast<float *>(ws + l.part_d);
    p.dy = b->dy; p.dfinal = b->dfinal; p.dx = b->dx; p.ddt = b->ddt; p.dz = b->dz; p.dh0 = b->dh0;
    p.y = nullptr; p.final_state = nullptr;
    cudaError_t e = ssd::launch_scan_bwd(p, a->x_dtype, b->dB, b->dC, b->dA, a->Dskip ? b->dD : nullptr,
                                         a->dt_bias ? b->ddt_bias : nullptr, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "selective_scan_bwd");
    return ok();
}

ssd_status ssd_selective_scan_step(const ssd_scan_step_args *a, void *stream) {
    if (!a) return fail(SSD_ERR_INVALID_ARG, "args is NULL");
    if (a->B <= 0 || a->D <= 0 || a->N <= 0 || a->G <= 0 || a->nslots <= 0)
        return fail(SSD_ERR_INVALID_ARG, "every dim must be > 0 (B=%lld D=%lld N=%lld G=%lld nslots=%lld)", (long long)a->B,
                    (long long)a->D, (long long)a->N, (long long)a->G, (long long)a->nslots);
    if (a->D % a->G != 0)
        return fail(SSD_ERR_INVALID_ARG, "D (%lld) must be a multiple of G (%lld)", (long long)a->D, (long long)a->G);
    if (a->N > 128) return fail(SSD_ERR_UNSUPPORTED, "N must be <= 128 (got %lld)", (long long)a->N);
    if (a->B > 65535 || a->D > (1 << 24)) return fail(SSD_ERR_UNSUPPORTED, "B <= 65535 and D <= 2^24 required");
    if (!known_dtype(a->x_dtype)) return fail(SSD_ERR_INVALID_ARG, "unknown dtype code %d", a->x_dtype);
    if (!known_dtype(a->dt_dtype)) return fail(SSD_ERR_INVALID_ARG, "unknown dtype code %d", a->dt_dtype);
    if (a->dt_dtype != a->x_dtype && a->dt_dtype != SSD_F32)
        return fail(SSD_ERR_UNSUPPORTED, "dt must have the dtype of x or fp32");
    ssd_status st = check_limit(a->dt_min, a->dt_max);
    if (st != SSD_OK) return st;
    if (!a->x || !a->dt || !a->A || !a->Bm || !a->Cm || !a->state || !a->state_out || !a->y)
        return fail(SSD_ERR_INVALID_ARG, "x, dt, A, B, C, state, state_out and y are required");
    if (!a->slots && a->nslots < a->B)
        return fail(SSD_ERR_INVALID_ARG, "without slots nslots (%lld) must be at least B (%lld)", (long long)a->nslots,
                    (long long)a->B);
    for (int64_t r : {a->x_row, a->dt_row, a->z_row, a->b_row, a->c_row})
        if (r < 0) return fail(SSD_ERR_INVALID_ARG, "row strides must be >= 0");
    ssd::ScanStepParams p = {};
    p.B = (int)a->B; p.D = (int)a->D; p.N = (int)a->N; p.G = (int)a->G; p.nslots = a->nslots;
    p.x = a->x; p.dt = a->dt; p.A = a->A; p.Bm = a->Bm; p.Cm = a->Cm; p.z = a->z; p.Dskip = a->Dskip;
    p.dt_bias = a->dt_bias; p.state = a->state; p.state_out = a->state_out; p.slots = a->slots; p.y = a->y;
    const int64_t gn = a->G * a->N;
    p.x_row = a->x_row ? a->x_row : a->D; p.dt_row = a->dt_row ? a->dt_row : a->D;
    p.z_row = a->z_row ? a->z_row : a->D; p.b_row = a->b_row ? a->b_row : gn; p.c_row = a->c_row ? a->c_row : gn;
    p.dt32 = a->dt_dtype == SSD_F32;
    p.softplus = a->dt_softplus ? 1 : 0;
    p.has_limit = limited(a->dt_min, a->dt_max);
    p.dt_min = a->dt_min; p.dt_max = a->dt_max;
    const size_t f = sizeof(float), es = element(a->x_dtype), pool = (size_t)a->nslots * a->D * a->N * f;
    const long long xr[2] = {0, p.x_row}, dtr[2] = {0, p.dt_row}, zr[2] = {0, p.z_row}, br[2] = {0, p.b_row}, cr[2] = {0, p.c_row};
    const Span y = {a->y, (size_t)a->B * a->D * es, "y"}, to = {a->state_out, pool, "state_out"};
    const Span B = strided(a->Bm, 1, a->B, gn, br, es, "B"), C = strided(a->Cm, 1, a->B, gn, cr, es, "C"),
               A = {a->A, (size_t)a->D * a->N * f, "A"}, Dskip = {a->Dskip, a->D * f, "Dskip"},
               bias = {a->dt_bias, a->D * f, "dt_bias"}, slots = {a->slots, a->B * sizeof(int32_t), "slots"},
               from = {a->state == a->state_out ? nullptr : a->state, pool, "state"};
    st = apart(y, {replaced(a->y, a->x_dtype, a->x, a->x_dtype, 1, a->B, a->D, xr, "x"),
                   replaced(a->y, a->x_dtype, a->dt, a->dt_dtype, 1, a->B, a->D, dtr, "dt"),
                   replaced(a->y, a->x_dtype, a->z, a->x_dtype, 1, a->B, a->D, zr, "z"), B, C, A, Dskip, bias, slots, from, to});
    if (st != SSD_OK) return st;
    st = apart(to, {strided(a->x, 1, a->B, a->D, xr, es, "x"), strided(a->dt, 1, a->B, a->D, dtr, element(a->dt_dtype), "dt"),
                    strided(a->z, 1, a->B, a->D, zr, es, "z"), B, C, A, Dskip, bias, slots, from});
    if (st != SSD_OK) return st;
    cudaError_t e = ssd::launch_scan_step(p, a->x_dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "selective_scan_step");
    return ok();
}

ssd_status ssd_causal_conv_carry(const ssd_conv_args *a, void *stream) {
    ssd::ConvParams p = {};
    ssd_status st = check_conv(a, p);
    if (st != SSD_OK) return st;
    if (!a->x || !a->w || !a->y) return fail(SSD_ERR_INVALID_ARG, "x, w and y are required");
    // a thread reads the tokens before its run, which another one writes
    const size_t f = sizeof(float), es = element(a->dtype), state = (size_t)a->B * (a->W - 1) * a->C * es;
    const Span y = {a->y, (size_t)a->B * a->L * a->C * es, "y"}, fin = {a->final_state, state, "final_state"};
    const Span x = strided(a->x, a->B, a->L, a->C, p.xs, es, "x"), w = {a->w, (size_t)a->C * a->W * f, "w"},
               bias = {a->bias, a->C * f, "bias"}, h0 = {a->initial_state, state, "initial_state"},
               len = {a->lengths, a->B * sizeof(int32_t), "lengths"};
    if ((st = apart(y, {x, w, bias, h0, len, fin})) != SSD_OK) return st;
    if ((st = apart(fin, {x, w, bias, h0, len})) != SSD_OK) return st;
    cudaError_t e = ssd::launch_conv(p, a->dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "causal_conv_carry");
    return ok();
}

ssd_status ssd_causal_conv_bwd_workspace_size(const ssd_conv_bwd_args *b, size_t *bytes) {
    ssd::ConvParams p = {};
    ssd_status st = check_conv(b ? &b->fwd : nullptr, p);
    if (st != SSD_OK) return st;
    if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = conv_bwd_bytes(p);
    return ok();
}

ssd_status ssd_causal_conv_bwd(const ssd_conv_bwd_args *b, void *stream) {
    ssd::ConvParams p = {};
    ssd_status st = check_conv(b ? &b->fwd : nullptr, p);
    if (st != SSD_OK) return st;
    if (!p.x || !p.w || !b->dy || !b->dx || !b->dw)
        return fail(SSD_ERR_INVALID_ARG, "x, w, dy, dx and dw are required");
    if (p.bias && !b->dbias) return fail(SSD_ERR_INVALID_ARG, "dbias is required with bias");
    if ((st = check_workspace(b->workspace, b->workspace_bytes, conv_bwd_bytes(p))) != SSD_OK) return st;
    p.dy = b->dy; p.dfinal = b->dfinal; p.dx = b->dx; p.dw = b->dw; p.dbias = p.bias ? b->dbias : nullptr;
    p.dh0 = b->dh0; p.part = static_cast<float *>(b->workspace);
    cudaError_t e = ssd::launch_conv_bwd(p, b->fwd.dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "causal_conv_bwd");
    return ok();
}

ssd_status ssd_causal_conv_step(const ssd_conv_step_args *a, void *stream) {
    if (!a) return fail(SSD_ERR_INVALID_ARG, "args is NULL");
    if (a->B <= 0 || a->C <= 0 || a->W <= 0 || a->nslots <= 0)
        return fail(SSD_ERR_INVALID_ARG, "every dim must be > 0 (B=%lld C=%lld W=%lld nslots=%lld)", (long long)a->B,
                    (long long)a->C, (long long)a->W, (long long)a->nslots);
    if (a->W > 8) return fail(SSD_ERR_UNSUPPORTED, "W must be <= 8 (got %lld)", (long long)a->W);
    if (a->B > 65535 || a->C > (1 << 24)) return fail(SSD_ERR_UNSUPPORTED, "B <= 65535 and C <= 2^24 required");
    if (!known_dtype(a->dtype)) return fail(SSD_ERR_INVALID_ARG, "unknown dtype code %d", a->dtype);
    if (!a->x || !a->w || !a->y) return fail(SSD_ERR_INVALID_ARG, "x, w and y are required");
    if (a->W > 1 && (!a->state || !a->state_out))
        return fail(SSD_ERR_INVALID_ARG, "state and state_out are required");
    if (!a->slots && a->nslots < a->B)
        return fail(SSD_ERR_INVALID_ARG, "without slots nslots (%lld) must be at least B (%lld)", (long long)a->nslots,
                    (long long)a->B);
    if (a->x_row < 0) return fail(SSD_ERR_INVALID_ARG, "row strides must be >= 0");
    ssd::ConvStepParams p = {};
    p.B = (int)a->B; p.C = (int)a->C; p.W = (int)a->W; p.nslots = a->nslots;
    p.x_row = a->x_row ? a->x_row : a->C;
    p.x = a->x; p.w = a->w; p.bias = a->bias; p.state = a->state; p.state_out = a->state_out; p.slots = a->slots;
    p.y = a->y; p.silu = a->silu ? 1 : 0;
    const size_t f = sizeof(float), es = element(a->dtype), pool = (size_t)a->nslots * (a->W - 1) * a->C * es;
    const long long xr[2] = {0, p.x_row};
    const Span y = {a->y, (size_t)a->B * a->C * es, "y"}, to = {a->state_out, pool, "state_out"};
    const Span w = {a->w, (size_t)a->C * a->W * f, "w"}, bias = {a->bias, a->C * f, "bias"},
               slots = {a->slots, a->B * sizeof(int32_t), "slots"},
               from = {a->state == a->state_out ? nullptr : a->state, pool, "state"};
    ssd_status st = apart(y, {replaced(a->y, a->dtype, a->x, a->dtype, 1, a->B, a->C, xr, "x"), w, bias, slots, from, to});
    if (st != SSD_OK) return st;
    if ((st = apart(to, {strided(a->x, 1, a->B, a->C, xr, es, "x"), w, bias, slots, from})) != SSD_OK) return st;
    cudaError_t e = ssd::launch_conv_step(p, a->dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "causal_conv_step");
    return ok();
}

ssd_status ssd_block_norm(const ssd_block_norm_args *a, void *stream) {
    ssd::BlockNormParams p = {};
    ssd_status st = check_norm(a, p);
    if (st != SSD_OK) return st;
    if (!a->r || !a->n) return fail(SSD_ERR_INVALID_ARG, "r and n are required");
    if (a->o && !a->r_out) return fail(SSD_ERR_INVALID_ARG, "r_out is required with o");
    const long long dense[2] = {0, a->D};
    const size_t f = sizeof(float), nd = (size_t)a->rows * a->D;
    const int64_t gates = a->gate ? a->rows / a->rows_per_gate : 0;
    const Span w_pre = {a->w_pre, a->D * f, "w_pre"}, w_post = {a->w_post, a->D * f, "w_post"}, scale = {a->scale, a->D * f, "scale"};
    auto clear = [&](const void *out, int32_t type, const char *what) {  // o, r and a gate per token may be written over in place
        auto in = [&](const void *p, int32_t t, int64_t rows, const char *name) {
            return rows == a->rows ? replaced(out, type, p, t, 1, rows, a->D, dense, name)
                                   : Span{p, (size_t)rows * a->D * element(t), name};
        };
        return apart({out, nd * element(type), what}, {in(a->o, a->dtype, a->rows, "o"), in(a->r, a->stream_dtype, a->rows, "r"),
                                                       in(a->gate, a->dtype, gates, "gate"), w_pre, w_post, scale});
    };
    const void *r_out = a->o ? a->r_out : nullptr;
    if ((st = clear(a->n, a->dtype, "n")) != SSD_OK || (st = clear(r_out, a->stream_dtype, "r_out")) != SSD_OK) return st;
    st = apart({a->n, nd * element(a->dtype), "n"}, {{r_out, nd * element(a->stream_dtype), "r_out"}});
    if (st != SSD_OK) return st;
    cudaError_t e = ssd::launch_block_norm(p, a->dtype, a->stream_dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "block_norm");
    return ok();
}

ssd_status ssd_block_norm_bwd_workspace_size(const ssd_block_norm_bwd_args *b, size_t *bytes) {
    ssd::BlockNormParams p = {};
    ssd_status st = check_norm(b ? &b->fwd : nullptr, p);
    if (st != SSD_OK) return st;
    if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = norm_bwd_bytes(p);
    return ok();
}

ssd_status ssd_block_norm_bwd(const ssd_block_norm_bwd_args *b, void *stream) {
    ssd::BlockNormParams p = {};
    ssd_status st = check_norm(b ? &b->fwd : nullptr, p);
    if (st != SSD_OK) return st;
    if (!p.r_out || !b->dn || !b->dr || !b->dw_pre)
        return fail(SSD_ERR_INVALID_ARG, "r_out, dn, dr and dw_pre are required");
    if (p.o && !b->d_o) return fail(SSD_ERR_INVALID_ARG, "d_o is required with o");
    if (p.gate && !b->dgate) return fail(SSD_ERR_INVALID_ARG, "dgate is required with gate");
    if (p.w_post && !b->dw_post) return fail(SSD_ERR_INVALID_ARG, "dw_post is required with w_post");
    if (p.scale && !b->dscale) return fail(SSD_ERR_INVALID_ARG, "dscale is required with scale");
    if ((st = check_workspace(b->workspace, b->workspace_bytes, norm_bwd_bytes(p))) != SSD_OK) return st;
    p.r = nullptr; p.n = nullptr;
    p.dn = b->dn; p.dr_out = b->dr_out; p.d_o = b->d_o; p.dr = b->dr; p.dgate = b->dgate;
    p.dw_post = p.w_post ? b->dw_post : nullptr; p.dw_pre = b->dw_pre; p.dscale = p.scale ? b->dscale : nullptr;
    p.part = static_cast<float *>(b->workspace);
    cudaError_t e = ssd::launch_block_norm_bwd(p, b->fwd.dtype, b->fwd.stream_dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "block_norm_bwd");
    return ok();
}

}  // extern "C"

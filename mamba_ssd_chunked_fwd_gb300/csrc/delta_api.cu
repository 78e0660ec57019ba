// delta_api.cu -- C entries of the gated delta rule and of the norm of queries and
// keys: validation, workspace layout, launches.  Host code only.
#include <math.h>

#include "api_checks.cuh"
#include "delta.cuh"
#include "qk_norm.cuh"

using namespace ssd::api;

namespace {

ssd_status check_gate_type(int32_t dtype, int32_t io, const char *what) {
    if (!known_dtype(dtype)) return fail(SSD_ERR_INVALID_ARG, "unknown dtype code %d", dtype);
    if (dtype != io && dtype != SSD_F32) return fail(SSD_ERR_UNSUPPORTED, "%s must have the dtype of q or fp32", what);
    return SSD_OK;
}

ssd_status check_delta_dims(int64_t B, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P) {
    if (B <= 0 || L <= 0 || H <= 0 || G <= 0 || N <= 0 || P <= 0)
        return fail(SSD_ERR_INVALID_ARG, "every dim must be > 0 (B=%lld L=%lld H=%lld G=%lld N=%lld P=%lld)", (long long)B, (long long)L,
                    (long long)H, (long long)G, (long long)N, (long long)P);
    if (H % G != 0) return fail(SSD_ERR_INVALID_ARG, "H (%lld) must be a multiple of G (%lld)", (long long)H, (long long)G);
    if (N > 128) return fail(SSD_ERR_UNSUPPORTED, "N must be <= 128 (got %lld)", (long long)N);
    if (P > 1024 || H > 65536 || B > 65536 || L > kMaxDim || B * H > (1 << 20))
        return fail(SSD_ERR_UNSUPPORTED, "P <= 1024, B and H <= 65536, B H <= 2^20 and L < 2^31 - 65536 required");
    if (B * H * ((L + 63) / 64) > 0x7fffffffLL) return fail(SSD_ERR_UNSUPPORTED, "B H L / 64 must be < 2^31");
    return SSD_OK;
}

ssd_status check_delta(const ssd_delta_args *a, ssd::DeltaParams &p) {
    if (!a) return fail(SSD_ERR_INVALID_ARG, "args is NULL");
    ssd_status st = check_delta_dims(a->B, a->L, a->H, a->G, a->N, a->P);
    if (st != SSD_OK) return st;
    if (!known_dtype(a->dtype)) return fail(SSD_ERR_INVALID_ARG, "unknown dtype code %d", a->dtype);
    if ((st = check_gate_type(a->g_dtype, a->dtype, "g")) != SSD_OK || (st = check_gate_type(a->beta_dtype, a->dtype, "beta")) != SSD_OK)
        return st;
    if (!isfinite(a->scale)) return fail(SSD_ERR_INVALID_ARG, "scale must be finite");
    p = ssd::DeltaParams{};
    p.B = (int)a->B; p.L = (int)a->L; p.H = (int)a->H; p.G = (int)a->G; p.N = (int)a->N; p.P = (int)a->P;
    p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->g; p.beta = a->beta; p.h0 = a->initial_state; p.lengths = a->lengths;
    p.y = a->y; p.final_state = a->final_state;
    const int64_t gn = a->G * a->N, hp = a->H * a->P;
    if (!strides_of(a->q_stride, a->L, gn, p.qs) || !strides_of(a->k_stride, a->L, gn, p.ks) || !strides_of(a->v_stride, a->L, hp, p.vs) ||
        !strides_of(a->g_stride, a->L, a->H, p.gs) || !strides_of(a->beta_stride, a->L, a->H, p.bs))
        return fail(SSD_ERR_INVALID_ARG, "strides must be >= 0");
    p.g32 = a->g_dtype == SSD_F32;
    p.b32 = a->beta_dtype == SSD_F32;
    p.scale = a->scale;
    p.nc = (int)((a->L + ssd::kDeltaChunk - 1) / ssd::kDeltaChunk);
    return SSD_OK;
}

ssd_status check_delta_inputs(const ssd_delta_args *a) {
    if (!a->q || !a->k || !a->v || !a->g || !a->beta) return fail(SSD_ERR_INVALID_ARG, "q, k, v, g and beta are required");
    return SSD_OK;
}

struct DeltaLayout {
    size_t ops, states, trans, total;
};

// And by which kernels: in chunks, maybe of segments, or token by token.
DeltaLayout delta_layout(ssd::DeltaParams &p, int32_t dtype) {
    p.chunked = ssd::delta_tc_takes(p, dtype);
    DeltaLayout l = {0, 0, 0, 0};
    if (!p.chunked) return l;
    ssd::delta_segments(p);
    const size_t f = sizeof(float), heads = (size_t)p.B * p.H;
    l.states = align_up(heads * p.nc * ssd::delta_op_bytes(false));
    l.trans = l.states + (p.nseg > 1 ? align_up(heads * p.nseg * p.P * p.N * f) : 0);
    l.total = l.trans + (p.nseg > 1 ? align_up(heads * (p.nseg - 1) * p.N * p.N * f) : 0);
    return l;
}

struct DeltaBwdLayout {
    size_t states, adj, u, dr, dqh, dkh, ops, units, total;
};

DeltaBwdLayout delta_bwd_layout(ssd::DeltaParams &p, int32_t dtype) {
    p.chunked = ssd::delta_tc_takes(p, dtype);
    p.nseg = 1;
    p.seg_len = p.nc * ssd::kDeltaChunk;
    const size_t f = sizeof(float), chunks = (size_t)p.B * p.H * p.nc;
    // as operands, whole tiles of rows and columns
    const size_t P = p.chunked ? (p.P + 127) / 128 * 128 : p.P, N = p.chunked ? (p.N <= 64 ? 64 : 128) : p.N;
    DeltaBwdLayout l;
    l.states = 0;
    l.adj = l.states + align_up(chunks * P * N * f);
    l.u = l.adj + align_up(chunks * P * N * f);
    l.dr = l.u + align_up(chunks * ssd::kDeltaChunk * P * f);
    l.dqh = l.dr + align_up(chunks * ssd::kDeltaChunk * P * f);
    const size_t share = p.H > p.G ? align_up((size_t)p.B * p.L * p.H * p.N * f) : 0;
    l.dkh = l.dqh + share;
    l.ops = l.dkh + share;
    l.units = l.ops + (p.chunked ? align_up(chunks * ssd::delta_op_bytes(true)) : 0);
    l.total = l.units + (p.chunked && dtype == SSD_F16 ? align_up(chunks * (P / 128) * 4 * f) : 0);
    return l;
}

void delta_bwd_params(const ssd_delta_bwd_args *b, ssd::DeltaParams &p) {
    p.y = nullptr; p.final_state = nullptr;
    p.dy = b->dy; p.dfinal = b->dfinal; p.dq = b->dq; p.dk = b->dk; p.dv = b->dv; p.dg = b->dg; p.dbeta = b->dbeta; p.dh0 = b->dh0;
}

ssd_status check_qk_norm(const ssd_qk_norm_args *a, ssd::QkNormParams &p) {
    if (!a) return fail(SSD_ERR_INVALID_ARG, "args is NULL");
    if (a->B <= 0 || a->L <= 0 || a->H <= 0 || a->G <= 0 || a->N <= 0)
        return fail(SSD_ERR_INVALID_ARG, "every dim must be > 0 (B=%lld L=%lld H=%lld G=%lld N=%lld)", (long long)a->B, (long long)a->L,
                    (long long)a->H, (long long)a->G, (long long)a->N);
    if (a->N > 256) return fail(SSD_ERR_UNSUPPORTED, "N must be <= 256 (got %lld)", (long long)a->N);
    if (a->B > 0x7fffffffLL || a->L > kMaxDim || a->H > 65536 || a->G > 65536)
        return fail(SSD_ERR_UNSUPPORTED, "H and G <= 65536, B < 2^31 and L < 2^31 - 65536 required");
    if (!known_dtype(a->dtype)) return fail(SSD_ERR_INVALID_ARG, "unknown dtype code %d", a->dtype);
    if (a->kind != SSD_NORM_RMS && a->kind != SSD_NORM_L2) return fail(SSD_ERR_INVALID_ARG, "unknown norm %d", a->kind);
    if (!(a->eps >= 0.f && a->eps < INFINITY)) return fail(SSD_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (a->nfreq < 0 || 2 * a->nfreq > a->N)
        return fail(SSD_ERR_INVALID_ARG, "%lld frequencies for vectors of %lld", (long long)a->nfreq, (long long)a->N);
    if (a->nfreq > 0 && !a->freqs) return fail(SSD_ERR_INVALID_ARG, "freqs is required with nfreq > 0");
    p = ssd::QkNormParams{};
    p.B = (int)a->B; p.L = (int)a->L; p.H = (int)a->H; p.G = (int)a->G; p.N = (int)a->N; p.half = (int)a->nfreq;
    p.q = a->q; p.k = a->k; p.w_q = a->w_q; p.w_k = a->w_k; p.freqs = a->freqs; p.positions = a->positions;
    p.q_out = a->q_out; p.k_out = a->k_out;
    if (!strides_of(a->q_stride, a->L, a->H * a->N, p.qs) || !strides_of(a->k_stride, a->L, a->G * a->N, p.ks))
        return fail(SSD_ERR_INVALID_ARG, "strides must be >= 0");
    p.l2 = a->kind == SSD_NORM_L2;
    p.interleaved = a->interleaved ? 1 : 0;
    p.eps = a->eps;
    return SSD_OK;
}

size_t qk_norm_bwd_bytes(const ssd::QkNormParams &p) {
    return p.w_q || p.w_k ? align_up((size_t)ssd::qk_norm_parts(p) * p.N * sizeof(float)) : 0;
}

}  // namespace

extern "C" {

ssd_status ssd_delta_rule_workspace_size(const ssd_delta_args *a, size_t *bytes) {
    ssd::DeltaParams p;
    ssd_status st = check_delta(a, p);
    if (st != SSD_OK) return st;
    if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = delta_layout(p, a->dtype).total;
    return ok();
}

ssd_status ssd_delta_rule(const ssd_delta_args *a, void *stream) {
    ssd::DeltaParams p;
    ssd_status st = check_delta(a, p);
    if (st != SSD_OK) return st;
    if ((st = check_delta_inputs(a)) != SSD_OK) return st;
    if (!a->y) return fail(SSD_ERR_INVALID_ARG, "y is required");
    const size_t f = sizeof(float), es = element(a->dtype), state = (size_t)a->B * a->H * a->P * a->N * f;
    const int64_t gn = a->G * a->N, hp = a->H * a->P;
    const Span y = {a->y, (size_t)a->B * a->L * hp * es, "y"}, fin = {a->final_state, state, "final_state"};
    const Span q = strided(a->q, a->B, a->L, gn, p.qs, es, "q"), k = strided(a->k, a->B, a->L, gn, p.ks, es, "k"),
               v = strided(a->v, a->B, a->L, hp, p.vs, es, "v"), g = strided(a->g, a->B, a->L, a->H, p.gs, element(a->g_dtype), "g"),
               beta = strided(a->beta, a->B, a->L, a->H, p.bs, element(a->beta_dtype), "beta"), h0 = {a->initial_state, state, "initial_state"},
               len = {a->lengths, a->B * sizeof(int32_t), "lengths"};
    if ((st = apart(y, {q, k, v, g, beta, h0, len, fin})) != SSD_OK) return st;
    if ((st = apart(fin, {q, k, v, g, beta, h0, len})) != SSD_OK) return st;
    const DeltaLayout l = delta_layout(p, a->dtype);
    if ((st = check_workspace(a->workspace, a->workspace_bytes, l.total)) != SSD_OK) return st;
    unsigned char *ws = static_cast<unsigned char *>(a->workspace);
    p.ops = ws + l.ops;
    p.seg_states = reinterpret_cast<float *>(ws + l.states);
    p.seg_trans = reinterpret_cast<float *>(ws + l.trans);
    cudaError_t e = p.chunked ? ssd::launch_delta_tc(p, a->dtype, static_cast<cudaStream_t>(stream))
                              : ssd::launch_delta_walk(p, a->dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "delta_rule");
    return ok();
}

ssd_status ssd_delta_rule_bwd_workspace_size(const ssd_delta_bwd_args *b, size_t *bytes) {
    ssd::DeltaParams p;
    ssd_status st = check_delta(b ? &b->fwd : nullptr, p);
    if (st != SSD_OK) return st;
    if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
    delta_bwd_params(b, p);
    *bytes = delta_bwd_layout(p, b->fwd.dtype).total;
    return ok();
}

ssd_status ssd_delta_rule_bwd(const ssd_delta_bwd_args *b, void *stream) {
    ssd::DeltaParams p;
    ssd_status st = check_delta(b ? &b->fwd : nullptr, p);
    if (st != SSD_OK) return st;
    if ((st = check_delta_inputs(&b->fwd)) != SSD_OK) return st;
    if (!b->dy || !b->dq || !b->dk || !b->dv || !b->dg || !b->dbeta)
        return fail(SSD_ERR_INVALID_ARG, "dy, dq, dk, dv, dg and dbeta are required");
    delta_bwd_params(b, p);
    const DeltaBwdLayout l = delta_bwd_layout(p, b->fwd.dtype);
    if ((st = check_workspace(b->workspace, b->workspace_bytes, l.total)) != SSD_OK) return st;
    unsigned char *ws = static_cast<unsigned char *>(b->workspace);
    p.ops = ws + l.ops;
    p.states = reinterpret_cast<float *>(ws + l.states);
    p.adj = reinterpret_cast<float *>(ws + l.adj);
    p.u = reinterpret_cast<float *>(ws + l.u);
    p.dr = reinterpret_cast<float *>(ws + l.dr);
    p.dqh = reinterpret_cast<float *>(ws + l.dqh);
    p.dkh = reinterpret_cast<float *>(ws + l.dkh);
    p.units = reinterpret_cast<float *>(ws + l.units);
    cudaError_t e = ssd::launch_delta_bwd(p, b->fwd.dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "delta_rule_bwd");
    return ok();
}

ssd_status ssd_delta_rule_step(const ssd_delta_step_args *a, void *stream) {
    if (!a) return fail(SSD_ERR_INVALID_ARG, "args is NULL");
    ssd_status st = check_delta_dims(a->B, 1, a->H, a->G, a->N, a->P);
    if (st != SSD_OK) return st;
    if (a->nslots <= 0) return fail(SSD_ERR_INVALID_ARG, "nslots must be > 0");
    if (!known_dtype(a->dtype)) return fail(SSD_ERR_INVALID_ARG, "unknown dtype code %d", a->dtype);
    if ((st = check_gate_type(a->g_dtype, a->dtype, "g")) != SSD_OK || (st = check_gate_type(a->beta_dtype, a->dtype, "beta")) != SSD_OK)
        return st;
    if (!isfinite(a->scale)) return fail(SSD_ERR_INVALID_ARG, "scale must be finite");
    if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->state || !a->state_out || !a->y)
        return fail(SSD_ERR_INVALID_ARG, "q, k, v, g, beta, state, state_out and y are required");
    if (!a->slots && a->nslots < a->B)
        return fail(SSD_ERR_INVALID_ARG, "without slots nslots (%lld) must be at least B (%lld)", (long long)a->nslots, (long long)a->B);
    for (int64_t r : {a->q_row, a->k_row, a->v_row, a->g_row, a->beta_row})
        if (r < 0) return fail(SSD_ERR_INVALID_ARG, "row strides must be >= 0");
    ssd::DeltaStepParams p = {};
    p.B = (int)a->B; p.H = (int)a->H; p.G = (int)a->G; p.N = (int)a->N; p.P = (int)a->P; p.nslots = a->nslots;
    p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->g; p.beta = a->beta; p.state = a->state; p.state_out = a->state_out;
    p.slots = a->slots; p.y = a->y;
    const int64_t gn = a->G * a->N, hp = a->H * a->P;
    p.q_row = a->q_row ? a->q_row : gn; p.k_row = a->k_row ? a->k_row : gn; p.v_row = a->v_row ? a->v_row : hp;
    p.g_row = a->g_row ? a->g_row : a->H; p.b_row = a->beta_row ? a->beta_row : a->H;
    p.g32 = a->g_dtype == SSD_F32;
    p.b32 = a->beta_dtype == SSD_F32;
    p.scale = a->scale;
    const size_t es = element(a->dtype), pool = (size_t)a->nslots * hp * a->N * sizeof(float);
    const long long qr[2] = {0, p.q_row}, kr[2] = {0, p.k_row}, vr[2] = {0, p.v_row}, gr[2] = {0, p.g_row}, br[2] = {0, p.b_row};
    const Span y = {a->y, (size_t)a->B * hp * es, "y"}, to = {a->state_out, pool, "state_out"};
    const Span q = strided(a->q, 1, a->B, gn, qr, es, "q"), k = strided(a->k, 1, a->B, gn, kr, es, "k"), v = strided(a->v, 1, a->B, hp, vr, es, "v"),
               g = strided(a->g, 1, a->B, a->H, gr, element(a->g_dtype), "g"), beta = strided(a->beta, 1, a->B, a->H, br, element(a->beta_dtype), "beta"),
               slots = {a->slots, a->B * sizeof(int32_t), "slots"}, from = {a->state == a->state_out ? nullptr : a->state, pool, "state"};
    if ((st = apart(y, {q, k, v, g, beta, slots, from, to})) != SSD_OK) return st;
    if ((st = apart(to, {q, k, v, g, beta, slots, from})) != SSD_OK) return st;
    cudaError_t e = ssd::launch_delta_step(p, a->dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "delta_rule_step");
    return ok();
}

ssd_status ssd_qk_norm(const ssd_qk_norm_args *a, void *stream) {
    ssd::QkNormParams p;
    ssd_status st = check_qk_norm(a, p);
    if (st != SSD_OK) return st;
    if (!a->q || !a->k || !a->q_out || !a->k_out) return fail(SSD_ERR_INVALID_ARG, "q, k, q_out and k_out are required");
    const size_t f = sizeof(float), es = element(a->dtype);
    const int64_t hn = a->H * a->N, gn = a->G * a->N;
    const Span q = strided(a->q, a->B, a->L, hn, p.qs, es, "q"), k = strided(a->k, a->B, a->L, gn, p.ks, es, "k"),
               w_q = {a->w_q, a->N * f, "w_q"}, w_k = {a->w_k, a->N * f, "w_k"}, freqs = {a->freqs, a->nfreq * f, "freqs"},
               pos = {a->positions, (size_t)a->B * a->L * sizeof(int32_t), "positions"};
    const Span qo = {a->q_out, (size_t)a->B * a->L * hn * es, "q_out"}, ko = {a->k_out, (size_t)a->B * a->L * gn * es, "k_out"};
    // a vector is read by the lanes that write it, before they do: an output may take its own input's place
    st = apart(qo, {replaced(a->q_out, a->dtype, a->q, a->dtype, a->B, a->L, hn, p.qs, "q"), k, w_q, w_k, freqs, pos, ko});
    if (st != SSD_OK) return st;
    st = apart(ko, {replaced(a->k_out, a->dtype, a->k, a->dtype, a->B, a->L, gn, p.ks, "k"), q, w_q, w_k, freqs, pos});
    if (st != SSD_OK) return st;
    cudaError_t e = ssd::launch_qk_norm(p, a->dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "qk_norm");
    return ok();
}

ssd_status ssd_qk_norm_bwd_workspace_size(const ssd_qk_norm_bwd_args *b, size_t *bytes) {
    ssd::QkNormParams p;
    ssd_status st = check_qk_norm(b ? &b->fwd : nullptr, p);
    if (st != SSD_OK) return st;
    if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = qk_norm_bwd_bytes(p);
    return ok();
}

ssd_status ssd_qk_norm_bwd(const ssd_qk_norm_bwd_args *b, void *stream) {
    ssd::QkNormParams p;
    ssd_status st = check_qk_norm(b ? &b->fwd : nullptr, p);
    if (st != SSD_OK) return st;
    if (!p.q || !p.k || !b->dq_out || !b->dk_out || !b->dq || !b->dk)
        return fail(SSD_ERR_INVALID_ARG, "q, k, dq_out, dk_out, dq and dk are required");
    if (p.w_q && !b->dw_q) return fail(SSD_ERR_INVALID_ARG, "dw_q is required with w_q");
    if (p.w_k && !b->dw_k) return fail(SSD_ERR_INVALID_ARG, "dw_k is required with w_k");
    if ((st = check_workspace(b->workspace, b->workspace_bytes, qk_norm_bwd_bytes(p))) != SSD_OK) return st;
    p.q_out = p.k_out = nullptr;
    p.dq_out = b->dq_out; p.dk_out = b->dk_out; p.dq = b->dq; p.dk = b->dk;
    p.dw_q = p.w_q ? b->dw_q : nullptr; p.dw_k = p.w_k ? b->dw_k : nullptr;
    p.part = static_cast<float *>(b->workspace);
    cudaError_t e = ssd::launch_qk_norm_bwd(p, b->fwd.dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "qk_norm_bwd");
    return ok();
}

}  // extern "C"

// api_checks.cuh -- what the C entries of the selective scan, its neighbours and
// the delta rule share: error reports, strides and ranges of memory.  Host code only.
#pragma once

#include <stdarg.h>
#include <stdio.h>

#include <initializer_list>

#include "ssd_internal.cuh"

namespace ssd {
namespace api {

inline ssd_status fail(ssd_status st, const char *fmt, ...) {
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return ssd::report_error(st, msg);
}

inline ssd_status ok() { return ssd::report_error(SSD_OK, ""); }

inline ssd_status cuda_fail(cudaError_t e, const char *where) {
    return fail(SSD_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

constexpr int64_t kMaxDim = 0x7fffffffLL - 65536;  // sums of an index and a tile stay in 32 bits
inline size_t align_up(size_t v) { return (v + 255) / 256 * 256; }
inline bool known_dtype(int32_t d) { return d == SSD_F32 || d == SSD_F16 || d == SSD_BF16; }
inline bool aligned256(const void *p) { return reinterpret_cast<uintptr_t>(p) % 256 == 0; }

// Strides of a [B,L,...] tensor whose tokens are `width` wide; both zero: dense.
inline bool strides_of(const int64_t (&in)[2], int64_t L, int64_t width, long long (&out)[2]) {
    out[0] = in[0];
    out[1] = in[1];
    if (in[0] == 0 && in[1] == 0) {
        out[0] = L * width;
        out[1] = width;
    }
    return in[0] >= 0 && in[1] >= 0;
}

inline size_t element(int32_t dtype) { return dtype == SSD_F32 ? 4 : 2; }

// Whether two ranges of memory share bytes (an absent or empty one shares none).
inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
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
inline ssd_status apart(const Span &out, std::initializer_list<Span> others) {
    for (const Span &o : others)
        if (overlap(out.p, out.bytes, o.p, o.bytes)) return fail(SSD_ERR_INVALID_ARG, "%s must not overlap %s", out.what, o.what);
    return SSD_OK;
}

// What a [B,L,...] tensor reaches over through its strides; `st` as strides_of gives them.
inline Span strided(const void *p, int64_t B, int64_t L, int64_t width, const long long (&st)[2], size_t es, const char *what) {
    return {p, ((size_t)(B - 1) * st[0] + (size_t)(L - 1) * st[1] + width) * es, what};
}

// The same for a tensor of y's shape that y may replace: where it is dense, of y's type and
// at y's address, an element is read by the thread that writes it, before it does, and nothing is left to compare.
inline Span replaced(const void *y, int32_t y_dtype, const void *p, int32_t dtype, int64_t B, int64_t L, int64_t width,
              const long long (&st)[2], const char *what) {
    const bool dense = (B == 1 || st[0] == L * width) && (L == 1 || st[1] == width);
    if (p == y && dtype == y_dtype && dense) return {nullptr, 0, what};
    return strided(p, B, L, width, st, element(dtype), what);
}

inline ssd_status check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return SSD_OK;
    if (!ws || have < need)
        return fail(SSD_ERR_WORKSPACE, "workspace of %zu bytes required (got %zu)", need, ws ? have : (size_t)0);
    if (!aligned256(ws)) return fail(SSD_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    return SSD_OK;
}

}  // namespace api
}  // namespace ssd

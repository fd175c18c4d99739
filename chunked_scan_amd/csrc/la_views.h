// la_views.h -- argument checks shared by the entry points of the recurrent layers: sizes, limits, strided views and their
// overlap, traces, workspaces.  Host code only.
#pragma once
#include <stdint.h>

#include "la_chunk.h"
#include "la_internal.h"

namespace la {
namespace api {

// The limits keep every launch below 2^32 threads in each dimension and every byte offset far below 2^63.
constexpr int64_t kMaxB = 1 << 20, kMaxTokens = 1 << 24, kMaxChannels = 1 << 25, kMaxElems = (int64_t)1 << 35;
constexpr int64_t kMaxNormRows = 1 << 25, kMaxNormElems = (int64_t)1 << 34, kMaxSpan = (int64_t)1 << 42;

// a * b of non-negative sizes, or a value over every limit.
inline int64_t mul(int64_t a, int64_t b) {
    if (a == 0 || b == 0) return 0;
    return a > ((int64_t)1 << 60) / b ? (int64_t)1 << 61 : a * b;
}

inline size_t esize(int dtype) { return dtype == LA_BF16 ? 2 : 4; }
inline bool dtype_ok(int dtype) { return dtype == LA_F32 || dtype == LA_BF16; }
inline la_status from_hip(hipError_t e) { return e == hipSuccess ? LA_OK : LA_ERR_LAUNCH; }

// A [n0, n1, w] view: n0 blocks s0 bytes apart of n1 rows s1 bytes apart of w bytes each.
struct View {
    const void* p;
    int64_t n0, n1, s0, s1, w;
    int64_t span() const { return p && n0 > 0 && n1 > 0 && w > 0 ? (n0 - 1) * s0 + (n1 - 1) * s1 + w : 0; }
};
inline View flat(const void* p, int64_t bytes) { return {p, 1, 1, 0, 0, bytes}; }

// Whether two views may share memory.  Spans that meet still do not where both step through one row
// pitch and their columns are apart (two slices of one wide buffer).
inline bool overlap(const View& a, const View& b) {
    const int64_t na = a.span(), nb = b.span();
    if (na == 0 || nb == 0) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    if (!(x < y + nb && y < x + na)) return false;
    // the row pitch: the inner stride, or the outer one where there is one row per block
    const int64_t pa = a.n1 > 1 ? a.s1 : a.s0, pb = b.n1 > 1 ? b.s1 : b.s0;
    if (pa != pb || pa <= 0) return true;
    if ((a.n0 > 1 && a.s0 % pa) || (b.n0 > 1 && b.s0 % pa)) return true;
    const int64_t off = y >= x ? (int64_t)((y - x) % (uintptr_t)pa) : (pa - (int64_t)((x - y) % (uintptr_t)pa)) % pa;
    return !(off >= a.w && off + b.w <= pa);
}
// Whether rows of an output view overlap each other.
inline bool self_overlap(const View& v) {
    if (v.span() == 0) return false;
    if (v.n1 > 1 && v.s1 < v.w) return true;
    if (v.n0 > 1) {
        if (v.n1 <= 1) return v.s0 < v.w;
        if (v.s0 >= (v.n1 - 1) * v.s1 + v.w) return false;
        // blocks interleaved in the rows' gaps: [B, L, D] seen through [L, B, D] memory
        return !(v.s0 >= v.w && (v.n0 - 1) * v.s0 + v.w <= v.s1);
    }
    return false;
}
// No output may overlap an input, itself or another output.
template <int NI, int NO>
bool clash(const View (&in)[NI], const View (&out)[NO]) {
    for (int o = 0; o < NO; o++) {
        if (self_overlap(out[o])) return true;
        for (int i = 0; i < NI; i++)
            if (overlap(out[o], in[i])) return true;
        for (int k = 0; k < o; k++)
            if (overlap(out[o], out[k])) return true;
    }
    return false;
}

template <typename S>
bool rows_ok(const S* s, const la_rows& r, int64_t L) {
    return r.batch >= 0 && r.token >= 0 && r.batch <= kMaxSpan && r.token <= kMaxSpan &&
           mul(s->B, r.batch) <= kMaxSpan && mul(L, r.token) <= kMaxSpan;
}
// The sizes that the convolution's and the scan's shapes share.
template <typename S>
la_status sizes_ok(const S* s, int64_t L) {
    if (s->B < 0 || s->D < 0 || L < 0) return LA_ERR_SHAPE;
    if (s->B > kMaxB || mul(s->B, L) > kMaxTokens || L > kMaxTokens || s->D > kMaxChannels ||
        mul(s->B, s->D) > kMaxChannels || mul(mul(s->B, L), s->D) > kMaxElems)
        return LA_ERR_UNSUPPORTED;
    return LA_OK;
}
inline la_rows resolve(const la_rows& r, int64_t L, int64_t w) {
    return r.batch == 0 && r.token == 0 ? la_rows{L * w, w} : r;
}
inline View rows(const void* p, const la_rows& r, int64_t B, int64_t L, int64_t w, size_t es) {
    return {p, B, L, r.batch * (int64_t)es, r.token * (int64_t)es, w * (int64_t)es};
}

inline la_status check_trace(la_trace* t) {
    if (!t) return LA_OK;
    if (t->capacity < 0 || t->capacity > LA_TRACE_MAX_KERNELS) return LA_ERR_SHAPE;
    for (int i = 0; i < t->capacity; i++)
        if (!t->start[i] || !t->stop[i]) return LA_ERR_NULL;
    return LA_OK;
}
inline la::Tracer make_tracer(la_trace* t, void* stream) {
    la::Tracer tr;
    tr.t = t;
    tr.s = (hipStream_t)stream;
    if (t) t->count = 0;
    return tr;
}
inline bool ws_bad(const void* ws, uint64_t have, size_t need) {
    return need > 0 && (!ws || (uintptr_t)ws % 16 != 0 || have < need);
}

inline View mat(const void* p, int64_t M, int64_t stride, int64_t D, size_t es) {
    return {p, M, 1, stride * (int64_t)es, D * (int64_t)es, D * (int64_t)es};
}
// `out` written in place over `in`: the same rows.  Otherwise they may not overlap.
inline bool clash_inplace(const View& out, const View& in) { return !(out.p == in.p && out.s0 == in.s0) && overlap(out, in); }

}  // namespace api
}  // namespace la

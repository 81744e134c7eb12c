// Host checks of the layer operators: what a call writes shares no byte with what
// else it writes or reads.
#pragma once

#include "token_internal.cuh"

namespace tbe {

// Rows of bytes, `stride` apart.
struct Span {
    uintptr_t from, row, stride, rows;
};
inline Span span_of(const tbe_matrix *m) {
    if (m == nullptr || m->rows < 1) return Span{0, 0, 0, 0};
    const uintptr_t e = dtype_bytes(m->dtype);
    return Span{(uintptr_t)m->data, m->cols * e, m->stride * e, (uintptr_t)m->rows};
}
// A vector, a scalar or a workspace of so many bytes; none: nothing.
inline Span span_of(const void *p, uintptr_t bytes) { return Span{(uintptr_t)p, bytes, bytes, p != nullptr && bytes > 0}; }
// All that lies between the first and the last element counts.
inline Span span_of(const tbe_experts *w) {
    const uintptr_t e = dtype_bytes(w->dtype);
    const uintptr_t bytes = ((w->experts - 1) * w->expert_stride + (w->rows - 1) * w->stride + w->cols) * e;
    return Span{(uintptr_t)w->data, bytes, bytes, 1};
}
// Whether two may share a byte: where they lie apart, or their rows, with one
// stride, in between one another, they do not.
inline bool share(Span a, Span b) {
    if (a.rows == 0 || b.rows == 0) return false;
    if (a.rows == 1) a.stride = b.stride;
    if (b.rows == 1) b.stride = a.stride;
    if (a.from >= b.from + (b.rows - 1) * b.stride + b.row || b.from >= a.from + (a.rows - 1) * a.stride + a.row) return false;
    if (a.stride != b.stride || a.stride == 0) return true;
    const uintptr_t gap = a.from > b.from ? (a.stride - (a.from - b.from) % a.stride) % a.stride : (b.from - a.from) % a.stride;
    return gap < a.row || a.stride - gap < b.row;
}
template <typename... Others> inline bool share(const Span &a, const Span &b, const Others &...others) {
    return share(a, b) || share(a, others...);
}

}  // namespace tbe

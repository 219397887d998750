// gdna_checks.cuh -- host checks of arguments that the attention-layer and decoder-block entry
// points share.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gdna_internal.cuh"

namespace gdna {
namespace checks {

// One operand: `rows` rows of `len` elements, `stride` apart.  An operand without
// elements may be NULL.
struct Operand {
    const void *p;
    int64_t rows, len, stride, elem;
};

struct Span {
    uintptr_t lo, hi;
};

constexpr int64_t kMostElems = INT64_MAX / 16;             // of an array: its bytes are an int64, with room to add

// Elements from the first to the last of `heads` heads of d, `stride` apart; more than kMostElems counts as one more.
inline int64_t heads_len(int64_t heads, int64_t stride, int64_t d)
{
    if (heads <= 0) return 0;
    if (heads > 1 && stride > (kMostElems - d) / (heads - 1)) return kMostElems + 1;
    return (heads > 1 ? (heads - 1) * stride : 0) + d;
}

inline bool overlap(const Span &a, const Span &b) { return a.lo < b.hi && b.lo < a.hi; }
inline bool aligned(const void *p, int64_t a) { return (uintptr_t)p % (uintptr_t)a == 0; }

inline int check_operand(const Operand &o, Span *span)
{
    *span = Span{0, 0};
    if (o.rows <= 0 || o.len <= 0) return GDN_OK;
    if (o.p == nullptr) return GDN_ERR_ARG;
    if (o.rows > 1 && o.stride < o.len) return GDN_ERR_ARG;
    if (!aligned(o.p, o.elem)) return GDN_ERR_ALIGN;
    if (o.len > kMostElems || (o.rows > 1 && o.rows - 1 > (kMostElems - o.len) / o.stride)) return GDN_ERR_ARG;
    const int64_t elems = (o.rows > 1 ? (o.rows - 1) * o.stride : 0) + o.len;
    span->lo = (uintptr_t)o.p;
    span->hi = span->lo + (uintptr_t)elems * (uintptr_t)o.elem;
    return span->hi > span->lo ? GDN_OK : GDN_ERR_ARG;
}

// Rows that lie side by side in wider rows (q, k and v of one projection, say): same stride, and neither's columns
// reach into the other's.
inline bool side_by_side(const Operand &a, const Operand &b)
{
    const uint64_t stride = (uint64_t)a.stride * (uint64_t)a.elem;
    if (a.rows <= 1 || b.rows <= 1 || stride == 0 || stride != (uint64_t)b.stride * (uint64_t)b.elem) return false;
    const uint64_t la = (uint64_t)a.len * (uint64_t)a.elem, lb = (uint64_t)b.len * (uint64_t)b.elem;
    const uint64_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
    const uint64_t off = pb >= pa ? (pb - pa) % stride : (stride - (pa - pb) % stride) % stride;   // of b's columns in a's rows
    return off >= la && off + lb <= stride;
}

// Every operand is sound; outputs (the first n_out) overlap nothing else, except
// the pair (may_a, may_b) if it is given.
inline int check_operands(const Operand *ops, int n, int n_out, int may_a = -1, int may_b = -1)
{
    Span spans[24];
    for (int i = 0; i < n; ++i) {
        const int st = check_operand(ops[i], &spans[i]);
        if (st != GDN_OK) return st;
    }
    for (int i = 0; i < n_out; ++i)
        for (int j = 0; j < n; ++j)
            if (j != i && !((i == may_a && j == may_b) || (i == may_b && j == may_a)) && overlap(spans[i], spans[j]) &&
                !side_by_side(ops[i], ops[j]))
                return GDN_ERR_ALIAS;
    return GDN_OK;
}

inline int64_t elem_size(int dtype) { return dtype == GDNA_F32 ? 4 : dtype == GDNA_E4M3 ? 1 : 2; }
inline bool plain_type(int dtype) { return dtype == GDNA_F32 || dtype == GDNA_F16 || dtype == GDNA_BF16; }
inline bool cache_type(int dtype) { return dtype == GDNA_F16 || dtype == GDNA_BF16 || dtype == GDNA_E4M3; }
inline bool sound_scale(float x) { return std::isfinite(x) && x > 0.f; }

// An attention item is (key head, tile of 8 query rows or more); the rows of a sequence and all its items are int32.
inline bool countable(int batch, int q_len, int nq)
{
    return (int64_t)q_len * nq <= (1 << 24) && batch <= (1 << 20) && (int64_t)batch * q_len <= INT32_MAX;
}

// The cache's strides keep its (page, token, head) vectors apart, and K's from V's
// where the two share a buffer.  `span` is the elements of one array.
inline int check_cache(const void *k, const void *v, int dtype, const CacheLayout &c, int nkv, int d, Operand *ok, Operand *ov)
{
    if (c.pages <= 0 || c.page_size <= 0) return GDN_ERR_ARG;
    if (c.pages > INT32_MAX) return GDN_ERR_UNSUPPORTED;   // page numbers are int32
    const int64_t elem = elem_size(dtype);
    struct Dim { int64_t stride, count; } dims[4] = {
        {c.page_stride, c.pages}, {c.token_stride, c.page_size}, {c.head_stride, nkv}, {0, 1}};
    auto apart = [&](int n, int64_t *extent) {
        std::sort(dims, dims + n, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
        *extent = d;
        for (int i = 0; i < n; ++i) {
            if (dims[i].count <= 1) continue;
            if (dims[i].stride < *extent) return false;
            if (dims[i].count - 1 > (kMostElems - *extent) / dims[i].stride) return false;
            *extent += (dims[i].count - 1) * dims[i].stride;
        }
        return true;
    };
    int64_t extent = 0;
    if (c.page_stride < 0 || c.token_stride < 0 || c.head_stride < 0 || !apart(3, &extent)) return GDN_ERR_ARG;
    *ok = Operand{k, 1, extent, extent, elem};
    *ov = Operand{v, 1, extent, extent, elem};
    Span a, b;
    int st = check_operand(*ok, &a);
    if (st == GDN_OK) st = check_operand(*ov, &b);
    if (st != GDN_OK) return st;
    if (overlap(a, b)) {
        const uintptr_t apart_bytes = a.lo > b.lo ? a.lo - b.lo : b.lo - a.lo;
        dims[3] = Dim{(int64_t)(apart_bytes / (uintptr_t)elem), 2};
        if (apart_bytes % (uintptr_t)elem != 0 || !apart(4, &extent)) return GDN_ERR_ALIAS;
    }
    return GDN_OK;
}

// Every vector of an array starts on an `align`-byte boundary.
inline bool rows_aligned(const void *p, int64_t elem, int64_t align, std::initializer_list<int64_t> strides)
{
    if (!aligned(p, align)) return false;
    for (int64_t s : strides)
        if (s * elem % align != 0) return false;
    return true;
}

}  // namespace checks
}  // namespace gdna

// gdna_abi.cu -- the extern "C" entry points of the attention-layer operators
// (declared in include/gdna.h): argument checks on the host, then the launches.
// Every check runs before any CUDA call.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gdna_internal.cuh"

namespace gdna {
namespace {

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
int64_t heads_len(int64_t heads, int64_t stride, int64_t d)
{
    if (heads <= 0) return 0;
    if (heads > 1 && stride > (kMostElems - d) / (heads - 1)) return kMostElems + 1;
    return (heads > 1 ? (heads - 1) * stride : 0) + d;
}

bool overlap(const Span &a, const Span &b) { return a.lo < b.hi && b.lo < a.hi; }
bool aligned(const void *p, int64_t a) { return (uintptr_t)p % (uintptr_t)a == 0; }

int check_operand(const Operand &o, Span *span)
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
bool side_by_side(const Operand &a, const Operand &b)
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
int check_operands(const Operand *ops, int n, int n_out, int may_a = -1, int may_b = -1)
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

int64_t elem_size(int dtype) { return dtype == GDNA_F32 ? 4 : dtype == GDNA_E4M3 ? 1 : 2; }
bool plain_type(int dtype) { return dtype == GDNA_F32 || dtype == GDNA_F16 || dtype == GDNA_BF16; }
bool cache_type(int dtype) { return dtype == GDNA_F16 || dtype == GDNA_BF16 || dtype == GDNA_E4M3; }
bool sound_scale(float x) { return std::isfinite(x) && x > 0.f; }

// An attention item is (key head, tile of 8 query rows or more); the rows of a sequence and all its items are int32.
bool countable(int batch, int q_len, int nq)
{
    return (int64_t)q_len * nq <= (1 << 24) && batch <= (1 << 20) && (int64_t)batch * q_len <= INT32_MAX;
}

// The cache's strides keep its (page, token, head) vectors apart, and K's from V's
// where the two share a buffer.  `span` is the elements of one array.
int check_cache(const void *k, const void *v, int dtype, const CacheLayout &c, int nkv, int d, Operand *ok, Operand *ov)
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
bool rows_aligned(const void *p, int64_t elem, int64_t align, std::initializer_list<int64_t> strides)
{
    if (!aligned(p, align)) return false;
    for (int64_t s : strides)
        if (s * elem % align != 0) return false;
    return true;
}

}  // namespace
}  // namespace gdna

using namespace gdna;

extern "C" {

GDN_API int gdna_page_assign(const int32_t *cached, const int32_t *fresh, int32_t *table, int64_t table_stride,
                             const int32_t *free_pages, int64_t n_free, const int32_t *free_head,
                             int32_t *kv_len, int32_t *row_start, int64_t *slots, int32_t *positions,
                             int32_t *free_head_out, int32_t *unserved,
                             int batch, int64_t rows, int page_size, int max_pages, void *stream)
{
    if (batch < 0 || rows < 0 || page_size < 1 || max_pages < 1 || n_free < 0) return GDN_ERR_ARG;
    if (batch > (1 << 20) || rows >= INT32_MAX - 4096 || n_free > INT32_MAX) return GDN_ERR_UNSUPPORTED;
    if (batch == 0) return GDN_OK;
    const Operand ops[] = {
        {table, batch, max_pages, table_stride, 4}, {kv_len, 1, batch, batch, 4},
        {row_start, 1, (int64_t)batch + 1, (int64_t)batch + 1, 4}, {slots, 1, rows, rows, 8},
        {positions, 1, rows, rows, 4}, {free_head_out, 1, 1, 1, 4}, {unserved, 1, 1, 1, 4},
        {cached, 1, batch, batch, 4}, {fresh, 1, batch, batch, 4}, {free_pages, 1, n_free, n_free, 4},
        {free_head, 1, 1, 1, 4}};
    const int st = check_operands(ops, 11, 7);
    if (st != GDN_OK) return st;
    PageParams p{};
    p.cached = cached; p.fresh = fresh; p.table = table; p.table_stride = table_stride;
    p.free_pages = free_pages; p.n_free = n_free; p.free_head = free_head;
    p.kv_len = kv_len; p.row_start = row_start; p.slots = slots; p.positions = positions;
    p.free_head_out = free_head_out; p.unserved = unserved;
    p.rows = rows; p.batch = batch; p.page_size = page_size; p.max_pages = max_pages;
    return gdn::report_cuda_error(launch_page_assign(p, (cudaStream_t)stream));
}

GDN_API int gdna_qk_norm_rope(const void *q, const void *k, const void *v, gdna_dtype dtype,
                              const float *qn, const float *kn, float eps,
                              const float *cos_sin, int64_t n_pos, int rot, int interleaved,
                              const int32_t *positions, const int64_t *slots,
                              void *q_out, void *k_out, void *k_cache, void *v_cache, gdna_dtype cache_dtype,
                              float k_scale, float v_scale,
                              int64_t rows, int nq, int nkv, int d, int64_t pages, int page_size,
                              int64_t q_stride, int64_t q_head_stride, int64_t k_stride, int64_t v_stride,
                              int64_t q_out_stride, int64_t k_out_stride,
                              int64_t page_stride, int64_t token_stride, int64_t head_stride, void *stream)
{
    if (rows < 0 || nq < 0 || nkv < 0 || nq + (int64_t)nkv == 0 || d <= 0) return GDN_ERR_ARG;
    if (rot < 0 || rot % 2 != 0 || rot > d || (rot > 0 && n_pos <= 0)) return GDN_ERR_ARG;
    if (!plain_type(dtype) || d > 256) return GDN_ERR_UNSUPPORTED;
    if ((int64_t)nq + 2 * (int64_t)nkv > (1 << 20) || rows > INT32_MAX) return GDN_ERR_UNSUPPORTED;
    if ((qn != nullptr || kn != nullptr) && !(eps >= 0.f && std::isfinite(eps))) return GDN_ERR_ARG;
    const bool caching = k_cache != nullptr;
    if (nkv > 0 && !caching && k_out == nullptr) return GDN_ERR_ARG;     // the keys would go nowhere
    if ((v != nullptr) != (v_cache != nullptr)) return GDN_ERR_ARG;
    if ((v_cache != nullptr && !caching) || (nkv == 0 && (caching || k_out != nullptr))) return GDN_ERR_ARG;
    if (nq > 0 && q_head_stride < d) return GDN_ERR_ARG;
    if (caching && !cache_type(cache_dtype)) return GDN_ERR_UNSUPPORTED;
    if (caching && !(sound_scale(k_scale) && sound_scale(v_scale))) return GDN_ERR_ARG;
    if (rows == 0) return GDN_OK;
    const int64_t e = elem_size(dtype), hk = (int64_t)nkv * d, hq = (int64_t)nq * d;
    RopeParams p{};
    p.cache = CacheLayout{page_stride, token_stride, head_stride, pages, page_size};
    Operand ops[16];
    int n = 0;
    ops[n++] = {q_out, rows, hq, q_out_stride, e};
    int at_k = -1, at_v = -1;
    if (k_out != nullptr) ops[n++] = {k_out, rows, hk, k_out_stride, e};
    if (caching) {
        Operand ok, ov;
        const int st = check_cache(k_cache, v_cache != nullptr ? v_cache : k_cache, cache_dtype, p.cache, nkv, d, &ok, &ov);
        // without a V cache the K cache stands in for it: the same array "overlaps" itself
        if (st != GDN_OK && !(v_cache == nullptr && st == GDN_ERR_ALIAS)) return st;
        ops[at_k = n++] = ok;
        if (v_cache != nullptr) ops[at_v = n++] = ov;
    }
    const int n_out = n;
    // q_out on top of q, row for row and head for head, is the in-place call
    const bool in_place = q_out == q && q_head_stride == d && (q_out_stride == q_stride || rows == 1);
    const int64_t q_len = heads_len(nq, q_head_stride, d);
    if (in_place) {
        if (rows > 1 && q_stride < hq) return GDN_ERR_ARG;
    } else {
        ops[n++] = {q, rows, q_len, q_stride, e};
    }
    ops[n++] = {k, rows, hk, k_stride, e};
    if (v != nullptr) ops[n++] = {v, rows, hk, v_stride, e};
    if (qn != nullptr) ops[n++] = {qn, 1, d, d, 4};
    if (kn != nullptr) ops[n++] = {kn, 1, d, d, 4};
    if (rot > 0) {
        ops[n++] = {cos_sin, n_pos, rot, rot, 4};
        ops[n++] = {positions, 1, rows, rows, 4};
    }
    if (caching) ops[n++] = {slots, 1, rows, rows, 8};
    const int st = check_operands(ops, n, n_out, at_k, at_v);
    if (st != GDN_OK) return st;

    p.q = q; p.k = k; p.v = v; p.qn = qn; p.kn = kn; p.cos_sin = cos_sin;
    p.positions = positions; p.slots = slots; p.q_out = q_out; p.k_out = k_out;
    p.k_cache = k_cache; p.v_cache = v_cache;
    p.rows = rows; p.n_pos = n_pos;
    p.q_stride = q_stride; p.q_head_stride = q_head_stride; p.k_stride = k_stride; p.v_stride = v_stride;
    p.q_out_stride = q_out_stride; p.k_out_stride = k_out_stride;
    p.dtype = dtype; p.cache_dtype = cache_dtype; p.nq = nq; p.nkv = nkv; p.d = d; p.rot = rot;
    p.interleaved = interleaved != 0;
    p.eps = eps; p.k_scale = k_scale; p.v_scale = v_scale;
    // the vector kernel moves four elements at a time, eight a lane with the rotated ones in whole lanes
    const int64_t c = elem_size(cache_dtype);
    const bool fast = (d == 64 || d == 128 || d == 256) && rot % 8 == 0 &&
                      rows_aligned(q, e, 4 * e, {q_stride, q_head_stride}) && rows_aligned(k, e, 4 * e, {k_stride}) &&
                      rows_aligned(v, e, 4 * e, {v_stride}) && rows_aligned(q_out, e, 4 * e, {q_out_stride}) &&
                      rows_aligned(k_out, e, 4 * e, {k_out_stride}) && aligned(qn, 16) && aligned(kn, 16) && aligned(cos_sin, 16) &&
                      (!caching || (rows_aligned(k_cache, c, 4 * c, {page_stride, token_stride, head_stride}) && aligned(v_cache, 4 * c)));
    // the general kernel's blocks of eight heads are counted in 31 bits
    if (!fast && rows * (nq + (v != nullptr ? 2 : 1) * (int64_t)nkv) > 8 * (int64_t)INT32_MAX) return GDN_ERR_UNSUPPORTED;
    return gdn::report_cuda_error(launch_qk_norm_rope(p, fast, (cudaStream_t)stream));
}

GDN_API int64_t gdna_attn_workspace(int batch, int q_len, int nq, int nkv, int d)
{
    if (batch < 0 || q_len < 0 || nq <= 0 || nkv <= 0 || nq % nkv != 0 || d <= 0 || d > 256 ||
        !countable(batch, q_len, nq))
        return 0;
    return attn_workspace_bytes((int64_t)q_len * (nq / nkv), d);
}

GDN_API int gdna_attn_decode(const void *q, gdna_dtype dtype, const void *gate,
                             const void *k_cache, const void *v_cache, gdna_dtype cache_dtype,
                             float k_scale, float v_scale,
                             const int32_t *table, int64_t table_stride, const int32_t *kv_len, float scale,
                             void *out, gdna_dtype out_dtype, float *lse,
                             void *workspace, int64_t workspace_bytes,
                             int batch, int q_len, int nq, int nkv, int d,
                             int64_t pages, int page_size, int max_pages,
                             int64_t q_stride, int64_t gate_stride, int64_t gate_head_stride, int64_t out_stride,
                             int64_t page_stride, int64_t token_stride, int64_t head_stride, void *stream)
{
    if (batch < 0 || q_len < 0 || nq <= 0 || nkv <= 0 || d <= 0 || max_pages < 1) return GDN_ERR_ARG;
    if (!plain_type(dtype) || !plain_type(out_dtype) || !cache_type(cache_dtype)) return GDN_ERR_UNSUPPORTED;
    if (d > 256 || nq % nkv != 0) return GDN_ERR_UNSUPPORTED;
    if (!sound_scale(scale) || !sound_scale(k_scale) || !sound_scale(v_scale)) return GDN_ERR_ARG;
    const float scale2 = (float)((double)scale * k_scale * 1.4426950408889634);
    if (!sound_scale(scale2)) return GDN_ERR_ARG;
    const int64_t rows = (int64_t)batch * q_len, hq = (int64_t)nq * d;
    if (!countable(batch, q_len, nq)) return GDN_ERR_UNSUPPORTED;
    if (gate != nullptr && gate_head_stride < d) return GDN_ERR_ARG;
    if (rows == 0) return GDN_OK;
    // the row of all units of work (16 keys at least each, and what an item costs beside them) is counted in 64 bits
    const double most = ((double)max_pages * (page_size > 0 ? page_size : 0) / 16 + 64) * batch * nkv *
                        ((double)q_len * (nq / nkv) / 8 + 1);
    if (most > 4e18) return GDN_ERR_UNSUPPORTED;
    AttnParams p{};
    p.cache = CacheLayout{page_stride, token_stride, head_stride, pages, page_size};
    Operand ops[10];
    int n = 0;
    const int64_t need = attn_workspace_bytes((int64_t)q_len * (nq / nkv), d);
    ops[n++] = {out, rows, hq, out_stride, elem_size(out_dtype)};
    ops[n++] = {workspace, 1, need, need, 1};
    if (lse != nullptr) ops[n++] = {lse, 1, rows * nq, rows * nq, 4};
    const int n_out = n;
    if (k_cache == nullptr || v_cache == nullptr) return GDN_ERR_ARG;
    // K and V are only read here: they may be one array
    int st = check_cache(k_cache, v_cache, cache_dtype, p.cache, nkv, d, &ops[n], &ops[n + 1]);
    if (st != GDN_OK && st != GDN_ERR_ALIAS) return st;
    n += 2;
    ops[n++] = {q, rows, hq, q_stride, elem_size(dtype)};
    ops[n++] = {table, batch, max_pages, table_stride, 4};
    ops[n++] = {kv_len, 1, batch, batch, 4};
    if (gate != nullptr)
        ops[n++] = {gate, rows, heads_len(nq, gate_head_stride, d), gate_stride, elem_size(dtype)};
    st = check_operands(ops, n, n_out);
    if (st != GDN_OK) return st;
    if (workspace_bytes < need) return GDN_ERR_ARG;
    if (!aligned(workspace, 16)) return GDN_ERR_ALIGN;

    p.q = q; p.gate = gate; p.k = k_cache; p.v = v_cache; p.table = table; p.kv_len = kv_len;
    p.out = out; p.lse = lse; p.workspace = workspace;
    p.table_stride = table_stride; p.q_stride = q_stride; p.gate_stride = gate_stride;
    p.gate_head_stride = gate_head_stride; p.out_stride = out_stride;
    p.dtype = dtype; p.cache_dtype = cache_dtype; p.out_dtype = out_dtype;
    p.batch = batch; p.q_len = q_len; p.nq = nq; p.nkv = nkv; p.group = nq / nkv; p.d = d; p.max_pages = max_pages;
    p.scale = scale2; p.v_scale = v_scale;
    p.q_vec = rows_aligned(q, elem_size(dtype), 4 * elem_size(dtype), {q_stride, d});
    p.gate_vec = rows_aligned(gate, elem_size(dtype), 4 * elem_size(dtype), {gate_stride, gate_head_stride});
    p.out_vec = rows_aligned(out, elem_size(out_dtype), 4 * elem_size(out_dtype), {out_stride, d});
    // the tensor-core kernel copies a key's head in 16-byte pieces
    const int64_t e = elem_size(cache_dtype);
    const bool fast = d * e % 16 == 0 && rows_aligned(k_cache, e, 16, {page_stride, token_stride, head_stride}) && aligned(v_cache, 16);
    return gdn::report_cuda_error(launch_attn_decode(p, fast, (cudaStream_t)stream));
}

}  // extern "C"

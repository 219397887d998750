// gdnb_abi.cu -- the extern "C" entry points of the decoder-block operators
// (declared in include/gdnb.h): argument checks on the host, then the launches.
// Every check runs before any CUDA call.
#include "gdna_checks.cuh"
#include "gdnb_internal.cuh"

using namespace gdna;
using namespace gdna::checks;

namespace {

constexpr int64_t kMostRows = INT32_MAX - 4095;
constexpr int kMostSegments = 65536, kMostGroup = 128;

int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

bool heads_ok(int nq, int nkv, int d) { return nq > 0 && nkv > 0 && d > 0 && d <= 256 && nq % nkv == 0 && nq / nkv <= kMostGroup && nq <= (1 << 20); }

// How the cache's rows come in, and the vector flags: bases and strides are known to be sound.
void set_paths(gdnb::FlashParams &p, int64_t page_stride, int64_t token_stride, int64_t head_stride)
{
    const int64_t e = elem_size(p.cache_dtype), qe = elem_size(p.dtype);
    const bool pieces = p.d * e % 16 == 0 && rows_aligned(p.k, e, 16, {page_stride, token_stride, head_stride}) && aligned(p.v, 16);
    const int size = p.table != nullptr ? p.cache.page_size & -p.cache.page_size : 128;
    p.copy_keys = size < 128 ? size : 128;
    // (32 copies a stage at most, and eight rows of a swizzle together)
    p.copy_mode = !pieces ? gdnb::kElements : p.copy_keys >= (p.cache_dtype == GDNA_E4M3 ? 4 : 8) ? gdnb::kTensorCopies : gdnb::kPieces16;
    p.q_vec = p.d % 8 == 0 && rows_aligned(p.q, qe, 16, {p.q_stride, p.d});
    p.gate_vec = p.d % 8 == 0 && rows_aligned(p.gate, qe, 16, {p.gate_stride, p.gate_head_stride});
    p.out_vec = p.d % 8 == 0 && rows_aligned(p.out, 2, 16, {p.out_stride, p.d});
}

// Scratch of a shared call: the own attention's, its output and log-sums, the prefix's partial results.
struct SharedSpace {
    int64_t decode, own, lse, parts;       // bytes
    bool together;                         // own keys by the prefix's kernel
    int64_t all() const { return decode + own + lse + parts; }
};
// Requests whose own keys go through the prefix's kernel with the prefix: as many as make about a tile for each SM.  That saves two
// launches and their latencies, and a tile of a few rows costs as much as a full one.  Both ways, us: 24/4 heads of 256, own keys to
// 100 and to 3000, 16 tiles 28 and 32 against 42 and 44, 152 tiles 36 and 59 against 49 and 68, 304 tiles 49 and 83 against 56 and
// 92; 48/8 of 128 at 304 tiles, own keys to 3000, 66 against 62; over E4M3 at 200 tiles, own keys to 900, 106 against 89; 768 tiles of
// 128, own keys to 2500, 260 against 227.
constexpr int64_t kTogether = 152;
SharedSpace shared_space(int batch, int groups, int q_len, int nq, int nkv, int d)
{
    const int64_t rows = (int64_t)batch * q_len, own_tiles = gdnb::flash_tiles(q_len, batch, nq / nkv, nkv, d);
    if (own_tiles <= kTogether) return SharedSpace{0, 0, 0, gdnb::flash_parts_bytes(rows, groups, nq / nkv, nkv, d, true, own_tiles), true};
    return SharedSpace{round256(attn_workspace_bytes((int64_t)q_len * (nq / nkv), d)), round256(rows * nq * d * 4), round256(rows * nq * 4),
                       gdnb::flash_parts_bytes(rows, groups, nq / nkv, nkv, d, true), false};
}
// What a caller has to bring: never less for more requests, groups or tokens, so that scratch for a server's largest step serves the
// smaller ones.  A step whose own keys go with the prefix needs a partial result for each of their tiles, more than a somewhat larger
// step by the other way, so the largest such steps within this one count too: of so many tiles a request, all tokens that those
// hold, and as many requests as go together.
int64_t shared_bytes(int batch, int groups, int q_len, int nq, int nkv, int d)
{
    int64_t most = shared_space(batch, groups, q_len, nq, nkv, d).all();
    const int64_t tile = gdnb::flash_tile_tokens(nq / nkv, d);
    for (int64_t each = 1; each * nkv <= kTogether && (each - 1) * tile < q_len; ++each) {
        const int64_t tokens = std::min<int64_t>(q_len, each * tile), requests = std::min<int64_t>(batch, kTogether / (each * nkv));
        most = std::max(most, shared_space((int)requests, groups, (int)tokens, nq, nkv, d).all());
    }
    return most;
}

}  // namespace

extern "C" {

GDN_API int gdnb_residual_norm(const void *x, gdna_dtype x_dtype, const void *y, gdna_dtype y_dtype,
                               const void *gate, const float *post, const float *pre, float scale, float eps,
                               void *x_out, void *h, gdna_dtype h_dtype, int64_t rows, int c,
                               int64_t x_stride, int64_t y_stride, int64_t gate_stride,
                               int64_t x_out_stride, int64_t h_stride, void *stream)
{
    if (rows < 0 || c <= 0) return GDN_ERR_ARG;
    if (!plain_type(x_dtype) || (y != nullptr && !plain_type(y_dtype)) || (h != nullptr && !plain_type(h_dtype))) return GDN_ERR_UNSUPPORTED;
    if (c > 16384) return GDN_ERR_UNSUPPORTED;
    if (!std::isfinite(scale) || !(eps >= 0.f && std::isfinite(eps))) return GDN_ERR_ARG;
    if (rows == 0) return GDN_OK;
    if (x_out == nullptr && h == nullptr) return GDN_ERR_ARG;
    if (y == nullptr && (gate != nullptr || post != nullptr)) return GDN_ERR_ARG;
    if (gate_stride < 0) return GDN_ERR_ARG;
    const int64_t xe = elem_size(x_dtype), ye = elem_size(y_dtype), he = elem_size(h_dtype);
    Operand ops[8];
    int n = 0;
    if (x_out != nullptr) ops[n++] = {x_out, rows, c, x_out_stride, xe};
    if (h != nullptr) ops[n++] = {h, rows, c, h_stride, he};
    const int n_out = n;
    // an output in its input's place, row for row
    const bool x_here = x_out != nullptr && x_out == x && (x_out_stride == x_stride || rows == 1);
    const bool y_here = h != nullptr && y != nullptr && h == y && h_dtype == y_dtype && (h_stride == y_stride || rows == 1);
    if (!x_here) ops[n++] = {x, rows, c, x_stride, xe};
    if (y != nullptr && !y_here) ops[n++] = {y, rows, c, y_stride, ye};
    if (gate != nullptr) ops[n++] = {gate, gate_stride == 0 ? 1 : rows, c, gate_stride, ye};
    if (post != nullptr) ops[n++] = {post, 1, c, c, 4};
    if (pre != nullptr) ops[n++] = {pre, 1, c, c, 4};
    const int st = check_operands(ops, n, n_out);
    if (st != GDN_OK) return st;
    gdnb::NormParams p{};
    p.x = x; p.y = y; p.gate = gate; p.post = post; p.pre = pre; p.x_out = x_out; p.h = h;
    p.rows = rows; p.x_stride = x_stride; p.y_stride = y_stride; p.gate_stride = gate_stride;
    p.x_out_stride = x_out_stride; p.h_stride = h_stride;
    p.x_dtype = x_dtype; p.y_dtype = y != nullptr ? y_dtype : x_dtype; p.h_dtype = h_dtype; p.c = c;
    p.scale = scale; p.eps = eps;
    const bool vec = c % 8 == 0 && rows_aligned(x, xe, 16, {x_stride}) && rows_aligned(y, ye, 16, {y != nullptr ? y_stride : 0}) &&
                     rows_aligned(gate, ye, 16, {gate != nullptr ? gate_stride : 0}) &&
                     rows_aligned(x_out, xe, 16, {x_out != nullptr ? x_out_stride : 0}) &&
                     rows_aligned(h, he, 16, {h != nullptr ? h_stride : 0}) && aligned(post, 16) && aligned(pre, 16);
    return gdn::report_cuda_error(gdnb::launch_residual_norm(p, vec, (cudaStream_t)stream));
}

GDN_API int64_t gdnb_attn_prompt_workspace(int64_t rows, int batch, int nq, int nkv, int d)
{
    if (rows < 0 || rows > kMostRows || batch < 0 || batch > kMostSegments || !heads_ok(nq, nkv, d)) return 0;
    return gdnb::flash_parts_bytes(rows, batch, nq / nkv, nkv, d, false);
}

GDN_API int gdnb_attn_prompt(const void *q, gdna_dtype dtype, const void *gate,
                             const void *k_cache, const void *v_cache, gdna_dtype cache_dtype,
                             float k_scale, float v_scale,
                             const int32_t *table, int64_t table_stride,
                             const int32_t *row_start, const int32_t *kv_len, float scale,
                             void *out, gdna_dtype out_dtype, void *workspace, int64_t workspace_bytes,
                             int64_t rows, int batch, int nq, int nkv, int d,
                             int64_t pages, int page_size, int max_pages,
                             int64_t q_stride, int64_t gate_stride, int64_t gate_head_stride, int64_t out_stride,
                             int64_t page_stride, int64_t token_stride, int64_t head_stride, void *stream)
{
    const bool paged = table != nullptr;
    if (batch < 0 || rows < 0 || nq <= 0 || nkv <= 0 || d <= 0 || (paged && max_pages < 1)) return GDN_ERR_ARG;
    if (!plain_type(dtype) || !cache_type(cache_dtype) || !(out_dtype == GDNA_F16 || out_dtype == GDNA_BF16)) return GDN_ERR_UNSUPPORTED;
    if (!paged && cache_dtype == GDNA_E4M3) return GDN_ERR_UNSUPPORTED;
    if (!heads_ok(nq, nkv, d) || rows > kMostRows || batch > kMostSegments) return GDN_ERR_UNSUPPORTED;
    if (!sound_scale(scale) || !sound_scale(k_scale) || !sound_scale(v_scale)) return GDN_ERR_ARG;
    const float scale2 = (float)((double)scale * k_scale * 1.4426950408889634);
    if (!sound_scale(scale2)) return GDN_ERR_ARG;
    if (gate != nullptr && gate_head_stride < d) return GDN_ERR_ARG;
    if (rows == 0 || batch == 0) return GDN_OK;
    if (row_start == nullptr || k_cache == nullptr || v_cache == nullptr || (paged && kv_len == nullptr)) return GDN_ERR_ARG;
    gdnb::FlashParams p{};
    p.cache = paged ? CacheLayout{page_stride, token_stride, head_stride, pages, page_size}
                    : CacheLayout{0, token_stride, head_stride, 1, (int)rows};
    Operand ops[12];
    int n = 0;
    const int64_t hq = (int64_t)nq * d, need = gdnb::flash_parts_bytes(rows, batch, nq / nkv, nkv, d, false);
    ops[n++] = {out, rows, hq, out_stride, 2};
    ops[n++] = {workspace, 1, need, need, 1};
    const int n_out = n;
    if (paged) {
        // K and V are only read here: they may be one array
        const int st = check_cache(k_cache, v_cache, cache_dtype, p.cache, nkv, d, &ops[n], &ops[n + 1]);
        if (st != GDN_OK && st != GDN_ERR_ALIAS) return st;
        n += 2;
        ops[n++] = {table, batch, max_pages, table_stride, 4};
    } else {
        if (head_stride < 0 || (nkv > 1 && head_stride < d)) return GDN_ERR_ARG;
        const int64_t len = heads_len(nkv, head_stride, d);
        ops[n++] = {k_cache, rows, len, token_stride, 2};
        ops[n++] = {v_cache, rows, len, token_stride, 2};
    }
    ops[n++] = {q, rows, hq, q_stride, elem_size(dtype)};
    ops[n++] = {row_start, 1, (int64_t)batch + 1, (int64_t)batch + 1, 4};
    if (kv_len != nullptr) ops[n++] = {kv_len, 1, batch, batch, 4};
    if (gate != nullptr) ops[n++] = {gate, rows, heads_len(nq, gate_head_stride, d), gate_stride, elem_size(dtype)};
    const int st = check_operands(ops, n, n_out);
    if (st != GDN_OK) return st;
    if (workspace_bytes < need) return GDN_ERR_ARG;
    if (!aligned(workspace, 16)) return GDN_ERR_ALIGN;

    p.q = q; p.gate = gate; p.k = k_cache; p.v = v_cache; p.table = table; p.row_start = row_start; p.kv_len = kv_len;
    p.out = out; p.workspace = workspace;
    p.rows = rows; p.table_stride = table_stride; p.q_stride = q_stride; p.gate_stride = gate_stride;
    p.gate_head_stride = gate_head_stride; p.out_stride = out_stride;
    p.dtype = dtype; p.cache_dtype = cache_dtype; p.out_dtype = out_dtype;
    p.segs = batch; p.row_mult = 1; p.nq = nq; p.nkv = nkv; p.group = nq / nkv; p.d = d; p.max_pages = max_pages;
    p.causal = 1; p.scale2 = scale2; p.v_scale = v_scale;
    set_paths(p, paged ? page_stride : 0, token_stride, head_stride);
    return gdn::report_cuda_error(gdnb::launch_flash(p, (cudaStream_t)stream));
}

GDN_API int64_t gdnb_attn_shared_workspace(int batch, int groups, int q_len, int nq, int nkv, int d)
{
    if (batch < 0 || q_len < 0 || groups < 1 || groups > kMostSegments || !heads_ok(nq, nkv, d) || !countable(batch, q_len, nq) ||
        (int64_t)batch * q_len > kMostRows)
        return 0;
    return shared_bytes(batch, groups, q_len, nq, nkv, d);
}

GDN_API int gdnb_attn_shared(const void *q, gdna_dtype dtype, const void *gate,
                             const void *k_cache, const void *v_cache, gdna_dtype cache_dtype,
                             float k_scale, float v_scale,
                             const int32_t *group_start, int groups,
                             const int32_t *shared_table, int64_t shared_stride, const int32_t *shared_len,
                             const int32_t *table, int64_t table_stride, const int32_t *kv_len, float scale,
                             void *out, gdna_dtype out_dtype, void *workspace, int64_t workspace_bytes,
                             int batch, int q_len, int nq, int nkv, int d,
                             int64_t pages, int page_size, int max_shared_pages, int max_pages,
                             int64_t q_stride, int64_t gate_stride, int64_t gate_head_stride, int64_t out_stride,
                             int64_t page_stride, int64_t token_stride, int64_t head_stride, void *stream)
{
    if (batch < 0 || q_len < 0 || groups < 1 || nq <= 0 || nkv <= 0 || d <= 0 || max_pages < 1 || max_shared_pages < 1) return GDN_ERR_ARG;
    if (group_start == nullptr && groups != 1) return GDN_ERR_ARG;
    if (!plain_type(dtype) || !cache_type(cache_dtype) || !(out_dtype == GDNA_F16 || out_dtype == GDNA_BF16)) return GDN_ERR_UNSUPPORTED;
    const int64_t rows = (int64_t)batch * q_len, hq = (int64_t)nq * d;
    if (!heads_ok(nq, nkv, d) || groups > kMostSegments || !countable(batch, q_len, nq) || rows > kMostRows) return GDN_ERR_UNSUPPORTED;
    if (!sound_scale(scale) || !sound_scale(k_scale) || !sound_scale(v_scale)) return GDN_ERR_ARG;
    const float scale2 = (float)((double)scale * k_scale * 1.4426950408889634);
    if (!sound_scale(scale2)) return GDN_ERR_ARG;
    if (gate != nullptr && gate_head_stride < d) return GDN_ERR_ARG;
    if (rows == 0) return GDN_OK;
    // (as gdna_attn_decode counts its own keys' work)
    const double most = ((double)max_pages * (page_size > 0 ? page_size : 0) / 16 + 64) * batch * nkv * ((double)q_len * (nq / nkv) / 8 + 1);
    if (most > 4e18) return GDN_ERR_UNSUPPORTED;
    if (k_cache == nullptr || v_cache == nullptr || shared_table == nullptr || shared_len == nullptr) return GDN_ERR_ARG;
    const SharedSpace space = shared_space(batch, groups, q_len, nq, nkv, d);
    const int64_t need = shared_bytes(batch, groups, q_len, nq, nkv, d);
    const CacheLayout cache{page_stride, token_stride, head_stride, pages, page_size};
    Operand ops[12];
    int n = 0;
    ops[n++] = {out, rows, hq, out_stride, 2};
    ops[n++] = {workspace, 1, need, need, 1};
    const int n_out = n;
    int st = check_cache(k_cache, v_cache, cache_dtype, cache, nkv, d, &ops[n], &ops[n + 1]);
    if (st != GDN_OK && st != GDN_ERR_ALIAS) return st;
    n += 2;
    ops[n++] = {q, rows, hq, q_stride, elem_size(dtype)};
    ops[n++] = {shared_table, groups, max_shared_pages, shared_stride, 4};
    ops[n++] = {shared_len, 1, groups, groups, 4};
    ops[n++] = {table, batch, max_pages, table_stride, 4};
    ops[n++] = {kv_len, 1, batch, batch, 4};
    if (group_start != nullptr) ops[n++] = {group_start, 1, (int64_t)groups + 1, (int64_t)groups + 1, 4};
    if (gate != nullptr) ops[n++] = {gate, rows, heads_len(nq, gate_head_stride, d), gate_stride, elem_size(dtype)};
    st = check_operands(ops, n, n_out);
    if (st != GDN_OK) return st;
    if (workspace_bytes < need) return GDN_ERR_ARG;
    if (!aligned(workspace, 16)) return GDN_ERR_ALIGN;

    uint8_t *at = static_cast<uint8_t *>(workspace);
    float *own = reinterpret_cast<float *>(at + space.decode), *own_lse = reinterpret_cast<float *>(at + space.decode + space.own);
    if (!space.together) {
        // each request's own keys
        AttnParams a{};
        a.cache = cache;
        a.q = q; a.k = k_cache; a.v = v_cache; a.table = table; a.kv_len = kv_len;
        a.out = own; a.lse = own_lse; a.workspace = workspace;
        a.table_stride = table_stride; a.q_stride = q_stride; a.gate_stride = hq; a.gate_head_stride = d; a.out_stride = hq;
        a.dtype = dtype; a.cache_dtype = cache_dtype; a.out_dtype = GDNA_F32;
        a.batch = batch; a.q_len = q_len; a.nq = nq; a.nkv = nkv; a.group = nq / nkv; a.d = d; a.max_pages = max_pages;
        a.scale = scale2; a.v_scale = v_scale;
        a.q_vec = rows_aligned(q, elem_size(dtype), 4 * elem_size(dtype), {q_stride, d});
        a.out_vec = d % 4 == 0 && aligned(own, 16);
        const int64_t e = elem_size(cache_dtype);
        const bool fast = d * e % 16 == 0 && rows_aligned(k_cache, e, 16, {page_stride, token_stride, head_stride}) && aligned(v_cache, 16);
        st = gdn::report_cuda_error(launch_attn_decode(a, fast, (cudaStream_t)stream));
        if (st != GDN_OK) return st;
    }
    // the prefix, and both joined
    gdnb::FlashParams p{};
    p.cache = cache;
    p.q = q; p.gate = gate; p.k = k_cache; p.v = v_cache; p.table = shared_table; p.row_start = group_start; p.kv_len = shared_len;
    p.out = out; p.workspace = at + space.decode + space.own + space.lse;
    p.rows = rows; p.table_stride = shared_stride; p.q_stride = q_stride; p.gate_stride = gate_stride;
    p.gate_head_stride = gate_head_stride; p.out_stride = out_stride;
    p.dtype = dtype; p.cache_dtype = cache_dtype; p.out_dtype = out_dtype;
    p.segs = groups; p.row_mult = q_len; p.nq = nq; p.nkv = nkv; p.group = nq / nkv; p.d = d; p.max_pages = max_shared_pages;
    p.all_parts = 1; p.scale2 = scale2; p.v_scale = v_scale;
    if (space.together) {
        p.segs += batch;
        p.own_segs = batch; p.own_table = table; p.own_table_stride = table_stride; p.own_kv_len = kv_len; p.own_max_pages = max_pages;
    } else {
        p.own = own; p.own_lse = own_lse;
    }
    set_paths(p, page_stride, token_stride, head_stride);
    return gdn::report_cuda_error(gdnb::launch_flash(p, (cudaStream_t)stream));
}

}  // extern "C"

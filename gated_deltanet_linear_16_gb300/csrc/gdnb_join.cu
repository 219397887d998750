// gdnb_join.cu -- partial results of split tiles added up (gdnb_flash.cuh has how they come about), and
// the prefix's joined with the requests' own attention; the launches.
//
//     o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i        M the largest m_i, in units of log2
//
// and with a request's own keys (o', lse') the two are weighted by 2^(lse2 - largest).  A block is 32 rows of a
// tile: a lane a row, a warp every eighth four of columns, as the partial results lie; through shared memory the
// output's lanes take pieces that lie side by side.  All it reads has just been written, most of it is in the L2.
#include "gdnb_flash.cuh"

namespace gdnb {
namespace flash {
namespace {

constexpr int kJoinWarps = 8;
constexpr int kJoinCols = 64;              // columns of a block

__device__ __forceinline__ bool sound(const FlashParams &p, const Record &x)
{
    return x.parts > 0 && x.parts <= kMaxGrid && x.first_slot >= 0 && x.first_slot + x.parts <= p.slots && x.row0 >= 0 && x.n > 0 &&
           x.row0 + x.n <= p.rows && x.token0 >= 0 && x.token0 < x.n && x.head >= 0 && x.head < p.nkv;
}

template <int D, bool LIFTED>
__global__ void __launch_bounds__(32 * kJoinWarps) join_parts(const FlashParams p)
{
    constexpr int kRows = D <= 128 ? 256 : 128;
    constexpr int64_t kPart = (int64_t)kRows * (D + 2);
    constexpr int kMine = kJoinCols / 4 / kJoinWarps;          // a warp's fours of columns
    __shared__ __align__(16) float sums[32][kJoinCols + 4];
    __shared__ float own_weight[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, col0 = blockIdx.z * kJoinCols;
    gdn::early_start<true>(nullptr, 0);
    const int64_t tiles = *record_count(p);
    for (int64_t tile = blockIdx.x; tile < tiles && tile < p.most_tiles; tile += gridDim.x) {
        const Record item = records(p)[tile];
        // (a record is whole unless its block gave up: then it may be anything)
        if (!sound(p, item)) continue;
        const int rows = min(p.tile_tokens, item.n - item.token0) * p.group;
        for (int r0 = blockIdx.y * 32; r0 < rows; r0 += gridDim.y * 32) {
            const int r = r0 + lane, t = r / p.group;
            const bool real = r < rows;
            // the row's partial results: of its tile, and of its request's own
            struct Parts {
                const float *first;
                int n, row;
            } lists[2] = {{p.parts + item.first_slot * kPart, real ? item.parts : 0, r}, {nullptr, 0, 0}};
            if (p.own_segs > 0 && real) {
                const int64_t row = item.row0 + item.token0 + t, request = row / p.row_mult;
                const int token = (int)(row - request * p.row_mult), tau = token / p.tile_tokens;
                const int each = (p.row_mult + p.tile_tokens - 1) / p.tile_tokens;
                const int64_t at = tiles + (request * p.nkv + item.head) * each + tau;
                if (request < p.own_segs && at < p.most_tiles) {
                    const Record own = records(p)[at];
                    if (sound(p, own))
                        lists[1] = {p.parts + own.first_slot * kPart, own.parts, (token - tau * p.tile_tokens) * p.group + (r - t * p.group)};
                }
            }
            auto ml = [&](const Parts &x, int i) { return *reinterpret_cast<const float2 *>(x.first + i * kPart + kRows * D + 2 * x.row); };
            // every warp has all rows' maxima and sums for itself
            float top = kNegInf;
#pragma unroll
            for (int which = 0; which < 2; ++which)
#pragma unroll 8
                for (int i = 0; i < lists[which].n; ++i) top = fmaxf(top, ml(lists[which], i).x);
            const float from = top == kNegInf ? 0.f : top;
            float l = 0.f;
            float4 o[kMine];
#pragma unroll
            for (int k = 0; k < kMine; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                const Parts x = lists[which];
#pragma unroll 4
                for (int i = 0; i < x.n; ++i) {
                    const float2 y = ml(x, i);
                    const float w = ex2(y.x - from);
                    l = fmaf(w, y.y, l);
#pragma unroll
                    for (int k = 0; k < kMine; ++k) {
                        const float4 u = *reinterpret_cast<const float4 *>(x.first + i * kPart + ((int64_t)(col0 / 4 + warp + kJoinWarps * k) * kRows + x.row) * 4);
                        o[k].x = fmaf(w, u.x, o[k].x); o[k].y = fmaf(w, u.y, o[k].y);
                        o[k].z = fmaf(w, u.z, o[k].z); o[k].w = fmaf(w, u.w, o[k].w);
                    }
                }
            }
            float norm = l == 0.f ? 0.f : p.v_scale / l, w_own = 0.f;
            if (p.own != nullptr && real) {
                const float mine = l == 0.f ? kNegInf : top + log2f(l) - (LIFTED ? 7.f : 0.f);
                const float other = p.own_lse[(item.row0 + item.token0 + t) * p.nq + (int64_t)item.head * p.group + (r - t * p.group)] * 1.4426950408889634f;
                const float big = fmaxf(mine, other), w = big == kNegInf ? 0.f : ex2(mine - big);
                w_own = big == kNegInf ? 0.f : ex2(other - big);
                const float sum = w + w_own;
                norm = sum == 0.f ? 0.f : norm * (w / sum);
                w_own = sum == 0.f ? 0.f : w_own / sum;
            }
            if (warp == 0) own_weight[lane] = w_own;
#pragma unroll
            for (int k = 0; k < kMine; ++k)
                *reinterpret_cast<float4 *>(&sums[lane][4 * (warp + kJoinWarps * k)]) =
                    make_float4(o[k].x * norm, o[k].y * norm, o[k].z * norm, o[k].w * norm);
            __syncthreads();
            for (int x = tid; x < 32 * (kJoinCols / 4); x += 32 * kJoinWarps) {
                const int row_in = x / (kJoinCols / 4), in_cols = 4 * (x % (kJoinCols / 4)), col = col0 + in_cols, rr = r0 + row_in;
                if (rr >= rows || col >= p.d) continue;
                const int tt = rr / p.group;
                const int64_t row = item.row0 + item.token0 + tt, head = (int64_t)item.head * p.group + (rr - tt * p.group);
                const float4 y = *reinterpret_cast<const float4 *>(&sums[row_in][in_cols]);
                float a[4] = {y.x, y.y, y.z, y.w}, g[4] = {0.f, 0.f, 0.f, 0.f};
                const int64_t g_at = row * p.gate_stride + head * p.gate_head_stride + col;
                const int64_t own_at = (row * p.nq + head) * p.d + col;
                if (p.gate != nullptr) {
                    if (p.gate_vec) {
                        const float4 u = gdna::got4(gdna::ask4(p.gate, g_at, p.dtype, true), p.dtype, true);
                        g[0] = u.x; g[1] = u.y; g[2] = u.z; g[3] = u.w;
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) g[e] = col + e < p.d ? gdna::load_elem(p.gate, g_at + e, p.dtype) : 0.f;
                    }
                }
                const float w = p.own != nullptr ? own_weight[row_in] : 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (w != 0.f && col + e < p.d) a[e] = fmaf(w, p.own[own_at + e], a[e]);
                    if (p.gate != nullptr) a[e] = a[e] / (1.f + expf(-g[e]));
                }
                const int64_t to = row * p.out_stride + head * p.d + col;
                if (p.out_vec) {
                    gdna::store4(p.out, to, p.out_dtype, true, make_float4(a[0], a[1], a[2], a[3]));
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (col + e < p.d) gdna::store_elem(p.out, to + e, p.out_dtype, a[e]);
                }
            }
            __syncthreads();
        }
    }
}

template <int D> cudaError_t launch_join(const FlashParams &p, int64_t tiles, cudaStream_t s)
{
    const int64_t rows = p.rows * p.group < p.tile_rows ? p.rows * p.group : p.tile_rows;  // of a tile
    // eight blocks an SM, which take tile after tile: often nothing is split, and what is launched only ends
    const int64_t each = (rows + 31) / 32 * (D / kJoinCols), most = (8 * (int64_t)p.grid + each - 1) / each;
    const dim3 grid((unsigned)(tiles < most ? tiles : most), (unsigned)((rows + 31) / 32), D / kJoinCols);
    if (p.cache_dtype == GDNA_BF16) return gdn::launch_early(join_parts<D, false>, grid, 32 * kJoinWarps, 0, s, true, p);
    return gdn::launch_early(join_parts<D, true>, grid, 32 * kJoinWarps, 0, s, true, p);
}

int width_of(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
int rows_of(int d) { return d <= 128 ? 256 : 128; }

// Tiles that `rows` rows in `segs` segments make, at most.
int64_t most_tiles(int64_t rows, int segs, int group, int nkv, int d)
{
    return (rows / (rows_of(d) / group) + (rows < segs ? rows : segs)) * nkv;
}

}  // namespace
}  // namespace flash

using namespace flash;

// Tiles that may be split, and the bytes of their records (with the header).
static int64_t split_tiles(int64_t most, bool all_parts) { return !all_parts && most > 2 * kMaxGrid ? 2 * kMaxGrid : most; }
static int64_t record_bytes(int64_t tiles) { return (64 + tiles * (int64_t)sizeof(Record) + 255) / 256 * 256; }

int flash_tile_tokens(int group, int d) { return rows_of(d) / group; }
int64_t flash_tiles(int tokens, int segs, int group, int nkv, int d)
{
    const int tile = flash_tile_tokens(group, d);
    return (int64_t)segs * ((tokens + tile - 1) / tile) * nkv;
}

int64_t flash_parts_bytes(int64_t rows, int segs, int group, int nkv, int d, bool all_parts, int64_t own_tiles)
{
    const int64_t tiles = split_tiles(most_tiles(rows, segs, group, nkv, d) + own_tiles, all_parts);
    return record_bytes(tiles) + (tiles + kMaxGrid) * rows_of(d) * (width_of(d) + 2) * (int64_t)sizeof(float);
}

cudaError_t launch_flash(FlashParams p, cudaStream_t s)
{
    const int sms = gdn::sm_count();
    p.grid = sms < kMaxGrid ? sms : kMaxGrid;
    p.tile_tokens = flash_tile_tokens(p.group, p.d);
    p.tile_rows = p.tile_tokens * p.group;
    p.group_div = Divisor::of((unsigned)p.group);
    p.page_div = Divisor::of((unsigned)(p.table != nullptr ? p.cache.page_size : 1));
    p.own_tiles = flash_tiles(p.row_mult, p.own_segs, p.group, p.nkv, p.d);
    const int64_t joined = most_tiles(p.rows, p.segs - p.own_segs, p.group, p.nkv, p.d);
    p.most_tiles = joined + p.own_tiles;
    const int64_t tiles = split_tiles(p.most_tiles, p.all_parts != 0);
    p.slots = tiles + kMaxGrid;
    const int64_t to_join = joined < tiles ? joined : tiles;   // (a request's own tiles are joined with its prefix's)
    p.records = p.workspace;
    p.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(p.workspace) + record_bytes(tiles));
    const bool bf16 = p.cache_dtype == GDNA_BF16;
    const cudaError_t e = p.d <= 64    ? (bf16 ? launch_flash_64_bf16(p, s) : launch_flash_64_f16(p, s))
                          : p.d <= 128 ? (bf16 ? launch_flash_128_bf16(p, s) : launch_flash_128_f16(p, s))
                                       : (bf16 ? launch_flash_256_bf16(p, s) : launch_flash_256_f16(p, s));
    if (e != cudaSuccess) return e;
    const int64_t keys = p.table != nullptr ? (int64_t)p.max_pages * p.cache.page_size : p.rows;
    if (never_split(p, keys)) return cudaSuccess;
    return p.d <= 64 ? launch_join<64>(p, to_join, s) : p.d <= 128 ? launch_join<128>(p, to_join, s) : launch_join<256>(p, to_join, s);
}

cudaError_t flash_wait_timeouts(unsigned *count)
{
    cudaError_t (*const units[])(unsigned *) = {flash_timeouts_64_f16, flash_timeouts_64_bf16, flash_timeouts_128_f16,
                                                flash_timeouts_128_bf16, flash_timeouts_256_f16, flash_timeouts_256_bf16};
    *count = 0;
    for (const auto unit : units) {
        unsigned n = 0;
        const cudaError_t e = unit(&n);
        if (e != cudaSuccess) return e;
        *count += n;
    }
    return cudaSuccess;
}

}  // namespace gdnb

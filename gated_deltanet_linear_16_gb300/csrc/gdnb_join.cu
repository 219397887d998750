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

template <int D, bool LIFTED>
__global__ void __launch_bounds__(32 * kJoinWarps) join_parts(const FlashParams p)
{
    constexpr int kRows = D <= 128 ? 256 : 128;
    constexpr int64_t kPart = (int64_t)kRows * (D + 2);
    constexpr int kMine = D / 4 / kJoinWarps;                  // a warp's fours of columns
    __shared__ __align__(16) float sums[32][D + 4];
    __shared__ float own_weight[32];
    __shared__ int64_t red[kJoinWarps][2];
    __shared__ int64_t first_slot;
    __shared__ Item item;
    __shared__ int parts, has[kMaxGrid];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Totals all = totals(p, red);
    if (whole_tiles(p, all)) return;
    for (int64_t tile = blockIdx.x; tile < all.tiles; tile += gridDim.x) {
        __syncthreads();
        if (warp == 0) {
            const Place at = find<false>(p, 0, 0, 0, tile);
            const int64_t idx = tile - at.tiles;
            const int head = (int)(idx / at.t.count);
            const int64_t tau = idx - head * at.t.count;
            const int64_t begin = at.cost + head * at.t.cost + cost_before(at.t, tau), end = begin + cost_of(p, at.t, tau);
            const int blocks = (int)(((int64_t)keys_of(p, at.t, tau) + kKeys - 1) / kKeys);
            const int64_t run = run_of(p, all), c0 = begin / run, c1 = (end - 1) / run;
            int full = 0;
            for (int c = (int)c0 + lane; c <= (int)c1; c += 32) {
                const int b0 = c * run > begin ? blocks_before(c * run - begin, blocks) : 0;
                const int b1 = (c + 1) * run < end ? blocks_before((c + 1) * run - begin, blocks) : blocks;
                has[c - c0] = b0 < b1 || (blocks == 0 && c == c0);
                full |= b0 == 0 && b1 == blocks && has[c - c0];
            }
            full = __any_sync(kFull, full);
            if (lane == 0) {
                const Segment s = segment(p, at.seg);
                item.row0 = s.row0;
                item.n = s.n;
                item.head = head;
                item.token0 = (int)(tau * p.tile_tokens);
                first_slot = tile + c0;
                parts = full && !p.all_parts ? 0 : (int)(c1 - c0 + 1);         // 0: the result is final
            }
        }
        __syncthreads();
        const int n = parts;
        if (n == 0) continue;
        const int rows = min(p.tile_tokens, item.n - item.token0) * p.group;
        for (int r0 = blockIdx.y * 32; r0 < rows; r0 += gridDim.y * 32) {
            const int r = r0 + lane;
            const bool real = r < rows;
            auto part = [&](int i) { return p.parts + (first_slot + i) * kPart; };
            auto ml = [&](int i) { return *reinterpret_cast<const float2 *>(part(i) + kRows * D + 2 * r); };
            // every warp has all rows' maxima and sums for itself
            float top = kNegInf;
            if (real)
                for (int i = 0; i < n; ++i)
                    if (has[i]) top = fmaxf(top, ml(i).x);
            const float from = top == kNegInf ? 0.f : top;
            float l = 0.f;
            float4 o[kMine];
#pragma unroll
            for (int k = 0; k < kMine; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (real)
#pragma unroll 2
                for (int i = 0; i < n; ++i) {
                    if (!has[i]) continue;
                    const float2 x = ml(i);
                    const float w = ex2(x.x - from);
                    l = fmaf(w, x.y, l);
#pragma unroll
                    for (int k = 0; k < kMine; ++k) {
                        const float4 u = *reinterpret_cast<const float4 *>(part(i) + ((int64_t)(warp + kJoinWarps * k) * kRows + r) * 4);
                        o[k].x = fmaf(w, u.x, o[k].x); o[k].y = fmaf(w, u.y, o[k].y);
                        o[k].z = fmaf(w, u.z, o[k].z); o[k].w = fmaf(w, u.w, o[k].w);
                    }
                }
            const int t = r / p.group;
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
            for (int x = tid; x < 32 * (D / 4); x += 32 * kJoinWarps) {
                const int row_in = x / (D / 4), col = 4 * (x % (D / 4)), rr = r0 + row_in;
                if (rr >= rows || col >= p.d) continue;
                const int tt = rr / p.group;
                const int64_t row = item.row0 + item.token0 + tt, head = (int64_t)item.head * p.group + (rr - tt * p.group);
                const float4 y = *reinterpret_cast<const float4 *>(&sums[row_in][col]);
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

template <int D> cudaError_t launch_join(const FlashParams &p, unsigned tiles, cudaStream_t s)
{
    // 32 rows a block at once; a split tile's rows over as many blocks
    const dim3 grid(tiles, (unsigned)((p.tile_rows < (D <= 128 ? 256 : 128) ? p.tile_rows : (D <= 128 ? 256 : 128)) + 31) / 32);
    if (p.cache_dtype == GDNA_BF16) join_parts<D, false><<<grid, 32 * kJoinWarps, 0, s>>>(p);
    else join_parts<D, true><<<grid, 32 * kJoinWarps, 0, s>>>(p);
    return cudaGetLastError();
}

int width_of(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
int rows_of(int d) { return d <= 128 ? 256 : 128; }

// Tiles that `rows` rows in `segs` segments make, at most.
int64_t most_tiles(int64_t rows, int segs, int group, int nkv, int d)
{
    const int64_t tokens = rows_of(d) / group;
    return (rows / tokens + (rows < segs ? rows : segs)) * nkv;
}

}  // namespace
}  // namespace flash

using namespace flash;

int64_t flash_parts_bytes(int64_t rows, int segs, int group, int nkv, int d, bool all_parts)
{
    int64_t tiles = most_tiles(rows, segs, group, nkv, d);
    if (!all_parts && tiles > 2 * kMaxGrid) tiles = 2 * kMaxGrid;      // (more are not split)
    return (tiles + kMaxGrid) * rows_of(d) * (width_of(d) + 2) * (int64_t)sizeof(float);
}

cudaError_t launch_flash(FlashParams p, cudaStream_t s)
{
    const int sms = gdn::sm_count();
    p.grid = sms < kMaxGrid ? sms : kMaxGrid;
    p.tile_tokens = rows_of(p.d) / p.group;
    p.tile_rows = p.tile_tokens * p.group;
    p.group_div = Divisor::of((unsigned)p.group);
    p.page_div = Divisor::of((unsigned)(p.table != nullptr ? p.cache.page_size : 1));
    p.most_tiles = most_tiles(p.rows, p.segs, p.group, p.nkv, p.d);
    cudaError_t e = p.d <= 64 ? launch_flash_64(p, s) : p.d <= 128 ? launch_flash_128(p, s) : launch_flash_256(p, s);
    if (e != cudaSuccess) return e;
    int64_t tiles = p.most_tiles;
    if (!p.all_parts && tiles > 2 * p.grid) tiles = 2 * p.grid;
    if (tiles > 65536) tiles = 65536;
    if (p.rows < p.tile_tokens) p.tile_rows = (int)p.rows * p.group;   // (rows of a tile, for the join's grid)
    return p.d <= 64 ? launch_join<64>(p, (unsigned)tiles, s) : p.d <= 128 ? launch_join<128>(p, (unsigned)tiles, s)
                                                                           : launch_join<256>(p, (unsigned)tiles, s);
}

cudaError_t flash_wait_timeouts(unsigned *count)
{
    unsigned n[3] = {0, 0, 0};
    cudaError_t e = flash_timeouts_64(&n[0]);
    if (e == cudaSuccess) e = flash_timeouts_128(&n[1]);
    if (e == cudaSuccess) e = flash_timeouts_256(&n[2]);
    *count = n[0] + n[1] + n[2];
    return e;
}

}  // namespace gdnb

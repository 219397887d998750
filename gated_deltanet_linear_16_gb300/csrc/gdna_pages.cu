// gdna_pages.cu -- block tables, slots and positions of a step's new tokens from
// the sequences' lengths (gdna_page_assign).
//
// With c tokens cached, f fresh ones and pages of P: a sequence holds
// have = ceil(c/P) pages and takes need = ceil((c+f)/P) - have more, its first
// one `sum of need before it` past the free list's head; its token rows start at
// `sum of f before it`.  Both are prefix sums over the batch.
//
// One launch.  A block owns kTile consecutive token rows and recomputes the
// prefix sums up to them itself: 8 bytes a sequence from L2, against a second
// launch or a wait between blocks.  Sequences whose rows meet the tile go to a
// list in shared memory, and every row finds its own by bisection there.  No
// block reads what another writes: of the table only entries below `have` are
// read and only entries from `have` on are written.
#include "gdna_internal.cuh"

namespace gdna {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 1024;                // token rows of a block
constexpr int kWarps = kThreads / 32;

struct Entry {                             // a sequence with rows in the tile
    int start;                             // its first row, relative to the tile (negative: before it)
    int cached, have, seq;
    int64_t first;                         // index into free_pages of its first new page; -1: not served
};

__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane)
{
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, x, off);
        if (lane >= off) x += y;
    }
    return x;
}

__global__ void __launch_bounds__(kThreads)
page_assign(const PageParams p)
{
    __shared__ Entry list[kTile];
    __shared__ int64_t warp_rows[kWarps], warp_pages[kWarps];
    __shared__ int warp_count[kWarps];
    __shared__ unsigned long long top;     // largest free-list index past a served sequence's pages
    __shared__ int refused;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t lo = (int64_t)blockIdx.x * kTile, hi = min(lo + kTile, p.rows);
    const bool last = blockIdx.x == gridDim.x - 1;
    gdn::early_start<true>(nullptr, 0);
    const int64_t head = *p.free_head, P = p.page_size;
    if (tid == 0) { top = 0; refused = 0; }

    int64_t rows_before = 0, pages_before = 0;         // sums over the sequences of earlier passes
    int listed = 0;
    for (int base = 0; base < p.batch; base += kThreads) {
        // the last block sees every sequence (totals); the others stop once their rows are covered
        if (!last && rows_before >= hi) break;
        const int b = base + tid;
        int64_t c = 0, f = 0;
        if (b < p.batch) {
            c = max(p.cached[b], 0);
            f = max(p.fresh[b], 0);
        }
        auto pages_of = [&](int64_t n) { return n > 0 ? (int64_t)p.page_div.quotient((unsigned)(n - 1)) + 1 : 0; };
        const int64_t have = pages_of(c), want = c + f <= INT32_MAX ? pages_of(c + f) : INT32_MAX;
        const bool fits = f == 0 || (want <= p.max_pages && c + f <= INT32_MAX);
        const int64_t need = fits ? want - have : 0;

        int64_t row_end = warp_scan(f, lane), page_end = warp_scan(need, lane);
        if (lane == 31) { warp_rows[warp] = row_end; warp_pages[warp] = page_end; }
        __syncthreads();
        int64_t row_total = 0, page_total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) { row_end += warp_rows[w]; page_end += warp_pages[w]; }
            row_total += warp_rows[w];
            page_total += warp_pages[w];
        }
        row_end += rows_before;
        page_end += pages_before;
        const int64_t start = row_end - f, first = head + page_end - need;
        const bool served = fits && (need == 0 || (head >= 0 && head + page_end <= p.n_free)) &&
                            (f == 0 || row_end <= p.rows);

        // per-sequence outputs: by the block whose tile holds the first row
        if (b < p.batch && start >= lo && (start < hi || last)) {
            p.kv_len[b] = (int32_t)(served ? c + f : c);
            p.row_start[b] = (int32_t)min(start, p.rows);
        }
        if (last && b < p.batch) {
            if (b == p.batch - 1) p.row_start[p.batch] = (int32_t)min(row_end, p.rows);
            if (served && need > 0) atomicMax(&top, (unsigned long long)page_end);
            if (!served && f > 0) atomicAdd(&refused, 1);
        }

        // the sequences with rows in the tile, in order
        const bool in = f > 0 && start < hi && row_end > lo;
        const unsigned votes = __ballot_sync(kFull, in);
        if (lane == 0) warp_count[warp] = __popc(votes);
        __syncthreads();
        int at = listed + __popc(votes & ((1u << lane) - 1));
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += warp_count[w];
            listed += warp_count[w];
        }
        if (in) {                          // at most kTile sequences have a row in the tile
            Entry e;
            e.start = (int)max(start - lo, (int64_t)INT32_MIN);
            e.cached = (int)c;
            e.have = (int)have;
            e.seq = b;
            e.first = served ? first : -1;
            list[at] = e;
        }
        rows_before += row_total;
        pages_before += page_total;
        __syncthreads();                   // the warp sums are free again; the list is visible
    }
    if (last && tid == 0) {
        *p.free_head_out = (int32_t)(head + (int64_t)top);
        *p.unserved = refused;
    }
    __syncthreads();

    for (int64_t row = lo + tid; row < hi; row += kThreads) {
        const int r = (int)(row - lo);
        int64_t slot = -1;
        int pos = 0;
        if (row < rows_before && listed > 0) {
            int a = 0, z = listed - 1;     // the last sequence that starts at or before the row
            while (a < z) {
                const int m = (a + z + 1) >> 1;
                if (list[m].start <= r) a = m; else z = m - 1;
            }
            const Entry e = list[a];
            const int64_t at = e.cached + ((int64_t)r - e.start);
            pos = (int)min(at, (int64_t)INT32_MAX);
            if (e.first >= 0) {
                const int64_t pg = p.page_div.quotient((unsigned)pos), in_page = pos - pg * P;
                int32_t *entry = p.table + e.seq * p.table_stride + pg;
                int64_t page;
                if (pg < e.have) {
                    page = *entry;
                } else {
                    page = p.free_pages[e.first + (pg - e.have)];
                    if (in_page == 0) *entry = (int32_t)page;    // the page's first token places it
                }
                if (page >= 0) slot = page * P + in_page;
            }
        }
        p.slots[row] = slot;
        p.positions[row] = pos;
    }
}

}  // namespace

cudaError_t launch_page_assign(PageParams p, cudaStream_t s)
{
    const int64_t tiles = (p.rows + kTile - 1) / kTile;
    p.page_div = Divisor::of((unsigned)p.page_size);
    return gdn::launch_early(page_assign, (unsigned)(tiles > 0 ? tiles : 1), kThreads, 0, s, true, p);
}

}  // namespace gdna

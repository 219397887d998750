// gdnb_flash.cuh -- attention of many query rows over one list of keys each, on the
// fifth-generation tensor cores: the kernel behind gdnb_attn_prompt (a segment is a
// sequence, causal) and behind the prefix of gdnb_attn_shared (a segment is a group
// of requests, every row sees every key).
//
// Mathematics.  A tile is 128 or 256 rows (token, head of the group) of a segment that read
// the same key head.  One pass over its keys, 128 at a time:
//     S = Q K^T,  m' = max(m, rowmax S),  P = exp2(scale2 S - scale2 m'),  l += rowsum P,  O += P V
// with O rescaled by exp2(scale2 (m - m')) only where a row's maximum has grown by more than
// kSlack (in log2): until then P may exceed 1, which costs nothing while it fits its type.  A row of S is one
// thread's (tensor memory gives a thread its lane), so maximum and sum need no shuffles.
//
// Where things are.  S of a block is 128 columns of tensor memory, and P takes the first 64 of
// them as the A operand of the second product; O stays in tensor memory for the whole tile.  D <= 128:
// two row tiles of 128 with an S each: one tile's softmax runs under the other's products.
// D = 256: O takes half of tensor memory, so one row tile, and two S that alternate: S of the next
// block is computed before P V of this one.  Q stays in shared memory; K and V come through one ring
// of stages of 128 keys x 128 columns (32 KB; 64 columns for D = 64), rows in panels of 128
// bytes with the 128-byte swizzle: K-major for the first product, and read along the other
// direction (N-major) for the second.
//
// Who does what (512 threads, one block an SM, persistent).  Warps 0-7: softmax, rescale, output, and the
// queries' way into shared memory.  Warps 8 and 9 issue the products of a row tile each, warp 10 deals out work, warps 12-15 fill
// the ring, a stage each in turn, by tensor copies or by loads (E4M3, odd pages and layouts), and warp 11 looks at the values that
// not every row sees.
//
// Work.  With many tiles a block takes every grid-th one, longest first within a sequence and in alternating
// direction, so that neighbours read the same keys at the same time and loads even out.  With
// fewer than two tiles a block, the tiles' costs (keys, and a lead for what a tile costs beside them) stand in one row
// and every block takes an equal run of it: a tile that lies in several blocks leaves partial
// results that join_parts adds up.  No host knowledge of lengths is needed for either.
//
// Rounding.  Products are of 16-bit operands with fp32 sums: keys and values exactly (E4M3 widens to fp16), queries in
// `PARTS` parts (x = hi + lo), for fp16 products scaled by a power of two a row where their type has a
// wider range.  A weight enters in one part: 2^-8 (2^-11 in fp16) of itself, of the order of
// the 16-bit output's own rounding.  For fp16 products weights are lifted by 2^kLift, so that one far below
// its row's largest keeps its bits (fp16's steps end at 2^-24).  m, l, S and O are fp32.
//
// What a row does not see.  Masked scores are replaced.  In blocks where some row does not see all
// keys, values that are not finite are taken out of V (0 x NaN) and the first such key of each column is noted: the rows
// that see it come out NaN in that column, the others clean.  Keys past the end count as zeros.
//
// What bounds it (GB300, device time).  Long lists of keys: 512 rows over 60000 keys of 8 heads of 128 take 335 us, 1510 TFLOP/s or
// 0.79 of the measured rate (360 from call to call with cold keys, 1400); there shared memory is full: Q and K of the first product take
// its 128 bytes a cycle by themselves, and the copies come on top.  Prompts: eight of 4096, 24/4 heads of 256, 1580 us (1044 TFLOP/s; two
// of 16384 1305): what a tile costs beside its 16 blocks, gates and output (without gates 1431); the next one's queries and first scores
// come meanwhile.  A packed batch at 128 1519 us (1113): what a tile costs beside its keys, queries, first scores and output.  Heads of
// 64: 220 us (400 TFLOP/s), the softmax warps' issue slots, and tiles dealt unevenly: the busiest block has 1.2 times the mean.  E4M3, fp32 queries in two parts: 362 us for 107 GFLOP, a ring of
// three stages (a query in one part: 217, five stages), the widening (a conversion of two codes takes a quarter of the schedulers' time),
// and tiles dealt unevenly (1.4).  Short calls: 23 us for one prompt of 180 tokens: 2 us until sums of lengths are there, 3 until the first item is
// dealt, then a chain of copies, products, softmax, output, in code that no cache holds yet.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_tc.cuh"
#include "gdnb_internal.cuh"

namespace gdnb {
namespace flash {

using gdn::kFull;
namespace tc = gdn::tc;

constexpr int kKeys = 128;                 // keys of a block
constexpr int kThreads = 512;
constexpr int kMaxGrid = 160;              // blocks that share the work, at most
constexpr int kItems = 4;                  // slots of the work queue
constexpr int kCopyWarps = 4;
constexpr int kLead = 256;                 // what a tile costs beside its keys, in keys: queries, first products, output
constexpr int kLeastChunk = 768;           // a block's run of the row of costs, at least; tiles that cost less stay whole
constexpr int kLongItem = 32;               // blocks from which on the order of an item's keys is chosen
static_assert(kLeastChunk >= kKeys, "every block between a tile's first and last has keys of it");
constexpr int kLeastPart = 256;            // the same where every result is a partial one: a block of keys or two (four requests, one
                                           // prefix of 3000: 43 us against 49)
constexpr int kMostKeys = INT32_MAX - 4095;
constexpr float kNegInf = -__builtin_huge_valf();

// ------------------------------------------------------------------ work

struct Segment {
    int64_t row0;
    int n, kv;                             // tokens, keys
    bool causal;                           // the t-th of n tokens sees n - 1 - t keys less than the last; else all see all
    const int32_t *pages;                  // its row of the block table
};

__device__ __forceinline__ Segment segment(const FlashParams &p, int b)
{
    Segment s;
    int64_t r0 = 0, r1 = p.rows, most;
    const int32_t *len = p.kv_len;
    int at = b;
    if (b >= p.segs - p.own_segs) {        // a request's own keys
        at = b - (p.segs - p.own_segs);
        r0 = (int64_t)at * p.row_mult;
        r1 = r0 + p.row_mult;
        len = p.own_kv_len;
        most = (int64_t)p.own_max_pages * p.cache.page_size;
        s.causal = true;
        s.pages = p.own_table + at * p.own_table_stride;
    } else {
        if (p.row_start != nullptr) {
            r0 = min(max((int64_t)p.row_start[b] * p.row_mult, (int64_t)0), p.rows);
            r1 = min(max((int64_t)p.row_start[b + 1] * p.row_mult, r0), p.rows);
        }
        most = p.table == nullptr ? r1 - r0 : (int64_t)p.max_pages * p.cache.page_size;
        s.causal = p.causal != 0;
        s.pages = p.table == nullptr ? nullptr : p.table + b * p.table_stride;
    }
    s.row0 = r0;
    s.n = (int)(r1 - r0);
    if (most > kMostKeys) most = kMostKeys;
    s.kv = len == nullptr ? (int)most : (int)min((int64_t)max(len[at], 0), most);
    return s;
}

// Tiles of a segment for one head, and where their costs begin.
struct Tiles {
    int64_t count;                         // tiles
    int64_t base;                          // cost of a tile beside its own tokens
    int64_t cost;                          // of all
    int step;                              // tokens a tile adds (0: every tile costs the same)
    int n, kv;
    bool causal;
};
__device__ __forceinline__ Tiles tiles_of(const FlashParams &p, const Segment &s)
{
    Tiles t;
    t.n = s.n;
    t.kv = s.kv;
    t.causal = s.causal;
    t.count = ((int64_t)s.n + p.tile_tokens - 1) / p.tile_tokens;
    // Of more tokens than keys the first see none, and all tiles cost what the last does: no tile's cost may pass kLead and its
    // segment's keys, which is what the launcher goes by (never_split).
    t.step = s.causal && s.n <= s.kv ? p.tile_tokens : 0;
    t.base = kLead + (t.step != 0 ? s.kv - s.n : s.kv);
    t.cost = t.count * t.base;
    if (t.step != 0 && t.count > 0) t.cost += (int64_t)t.step * (t.count * (t.count - 1) / 2) + s.n;
    return t;
}
__device__ __forceinline__ int64_t cost_before(const Tiles &t, int64_t tau)       // of tiles [0, tau), tau < count
{
    return tau * t.base + (int64_t)t.step * (tau * (tau + 1) / 2);
}
__device__ __forceinline__ int64_t cost_of(const FlashParams &p, const Tiles &t, int64_t tau)
{
    return t.base + (t.step != 0 ? min((tau + 1) * t.step, (int64_t)t.n) : 0);
}
// Keys that tile tau's last token sees, and its blocks.
__device__ __forceinline__ int keys_of(const FlashParams &p, const Tiles &t, int64_t tau)
{
    if (!t.causal) return t.kv;
    const int64_t k = t.kv - (int64_t)t.n + min((tau + 1) * (int64_t)p.tile_tokens, (int64_t)t.n);
    return k < 0 ? 0 : (int)k;
}
// Blocks of a tile that stand before place `x` of its cost.
__device__ __forceinline__ int blocks_before(int64_t x, int blocks)
{
    if (x <= kLead) return 0;
    const int64_t b = (x - kLead) / kKeys;
    return b < blocks ? (int)b : blocks;
}
// a / b of what is not negative: most of it has 32 bits, whose division is a fifth of the 64-bit one.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// The tile in which place `y` of a head's costs lies.
__device__ __forceinline__ int64_t tile_at(const Tiles &t, int64_t y)
{
    int64_t tau;
    if (t.step == 0) {
        tau = quotient(y, t.base);
    } else {                               // tau (base + step/2) + step/2 tau^2 <= y: near enough in fp32, then step by step
        const float h = 0.5f * (float)t.step, b = (float)t.base + h;
        tau = (int64_t)(2.f * (float)y / (sqrtf(b * b + 4.f * h * (float)y) + b));
    }
    if (tau < 0) tau = 0;
    if (tau > t.count - 1) tau = t.count - 1;
    while (tau > 0 && cost_before(t, tau) > y) --tau;
    while (tau + 1 < t.count && cost_before(t, tau + 1) <= y) ++tau;
    return tau;
}

// Sums over all segments, by all threads of the block.
struct Totals {
    int64_t cost, tiles;
};
__device__ __forceinline__ Totals totals(const FlashParams &p, int64_t (*red)[2])
{
    int64_t cost = 0, tiles = 0;
    for (int b = threadIdx.x; b < p.segs; b += blockDim.x) {
        const Tiles t = tiles_of(p, segment(p, b));
        cost += t.cost;
        tiles += t.count;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        cost += __shfl_xor_sync(kFull, cost, off);
        tiles += __shfl_xor_sync(kFull, tiles, off);
    }
    if ((threadIdx.x & 31) == 0) { red[threadIdx.x >> 5][0] = cost; red[threadIdx.x >> 5][1] = tiles; }
    __syncthreads();
    Totals all{0, 0};
    for (int w = 0; w < (int)blockDim.x / 32; ++w) { all.cost += red[w][0]; all.tiles += red[w][1]; }
    all.cost *= p.nkv;
    all.tiles *= p.nkv;
    // starts that go back, so that segments overlap: there may be more tiles than partial results have room
    if (p.all_parts && all.tiles > p.most_tiles) all = Totals{0, 0};
    return all;
}
__device__ __forceinline__ bool whole_tiles(const FlashParams &p, const Totals &all)
{
    return !p.all_parts && (all.tiles >= 2 * (int64_t)p.grid || all.tiles > p.most_tiles || all.cost <= all.tiles * kLeastChunk);
}
// Whether whole_tiles() is sure to hold, whatever the lengths, where no segment has more than `keys` keys: then nothing is to be joined.
inline bool never_split(const FlashParams &p, int64_t keys) { return !p.all_parts && keys + kLead <= kLeastChunk; }
// Cost of a block's run.
__device__ __forceinline__ int64_t run_of(const FlashParams &p, const Totals &all)
{
    const int64_t even = (all.cost + p.grid - 1) / p.grid;
    const int64_t least = p.all_parts ? kLeastPart : kLeastChunk;
    return even < least ? least : even;
}

// 32 segments in the lanes of a warp, with the costs and tiles up to and with each (over all heads).
struct Window {
    int first;                             // segment of lane 0
    Segment s;
    Tiles t;
    int64_t cost, tiles;
    __device__ __forceinline__ void load(const FlashParams &p, int seg, int64_t cost0, int64_t tiles0)
    {
        const int lane = threadIdx.x & 31;
        first = seg;
        s = Segment{};
        t = Tiles{};
        if (seg + lane < p.segs) {
            s = segment(p, seg + lane);
            t = tiles_of(p, s);
        }
        cost = t.cost * p.nkv;
        tiles = t.count * p.nkv;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t u = __shfl_up_sync(kFull, cost, off), v = __shfl_up_sync(kFull, tiles, off);
            if (lane >= off) { cost += u; tiles += v; }
        }
        cost += cost0;
        tiles += tiles0;
    }
    // The lane whose segment has place x of the costs (BY_COST; else tile x), windows further on if need be; -1: none.
    template <bool BY_COST> __device__ __forceinline__ int find(const FlashParams &p, int64_t x)
    {
        for (;;) {
            const unsigned hit = __ballot_sync(kFull, (BY_COST ? cost : tiles) > x);
            if (hit) return __ffs(hit) - 1;
            if (first + 32 >= p.segs) return -1;
            load(p, first + 32, __shfl_sync(kFull, cost, 31), __shfl_sync(kFull, tiles, 31));
        }
    }
};

// Where a split tile's partial results are, for the join: a header with the number of tiles, then a record each.
struct Record {
    int64_t row0, first_slot;
    int n, head, token0;
    int parts;                             // 0: the result is final already
};
__device__ __forceinline__ int64_t *record_count(const FlashParams &p) { return reinterpret_cast<int64_t *>(p.records); }
__device__ __forceinline__ Record *records(const FlashParams &p) { return reinterpret_cast<Record *>(static_cast<uint8_t *>(p.records) + 64); }

// A block's piece of work: some key blocks of a tile.
struct Item {
    int64_t row0;                          // first row of the segment
    int n, kv, head, token0;               // token0: first token of the tile
    int first, last;                       // key blocks [first, last)
    int turned, by;                        // of which [first, turned), which all rows see, come from first + by on, then from first on
    int whole;                             // all of the tile's: the result is final
    int causal;
    int clear;                             // keys that its first token sees: a value from there on may be out of some row's sight
    const int32_t *pages;
    int64_t slot;                          // of the partial result
    int valid;
};
// The block that is copied as the j-th (`turned` and `by` matter to the copies alone: rows see all of any block before `turned`).
__device__ __forceinline__ int block_at(const Item &it, int j)
{
    if (j >= it.turned) return j;
    j += it.by;
    return j < it.turned ? j : j - (it.turned - it.first);
}

// ------------------------------------------------------------------ tensor core pieces (16-bit operands)

template <bool BF16> __host__ __device__ constexpr uint32_t idesc16(int m, int n, bool b_n_major)
{
    return (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | ((b_n_major ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// A shared-memory descriptor's halves.  Low: the address in 16-byte units, and (N-major: B read along its rows) the distance
// of the panels of 64 columns.  High: eight rows (one swizzle atom) 1024 bytes apart, descriptor version, 128-byte swizzle.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t panel) { return ((addr & 0x3FFFFu) >> 4) | ((panel >> 4) << 16); }
__device__ __forceinline__ void mma16_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kDescHigh) : "memory");
}
__device__ __forceinline__ void mma16_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kDescHigh) : "memory");
}
// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void arrive_expect(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap *map, int x, int token, int head, int page, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4, %5}], [%6];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(token), "r"(head), "r"(page), "r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void lds16(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Place of 16-byte piece c of row r in panels of 128 rows x 128 bytes.
__device__ __forceinline__ uint32_t piece_at(int r, int c)
{
    return (uint32_t)((c >> 3) * (kKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

template <bool BF16> __device__ __forceinline__ uint32_t pack16(float a, float b)
{
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
template <bool BF16> __device__ __forceinline__ float2 unpack16(uint32_t u)
{
    if constexpr (BF16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}
// Waits on the kernel's barriers that ran out on this device (each instance's unit has its own).
static __device__ unsigned g_wait_timeouts;

// ------------------------------------------------------------------ shapes

template <int D> struct Shared {                               // beside queries and ring
    uint64_t full[8], empty[8], landed[8];
    uint64_t q_full[2], q_over[2], s_full[2][2], p_full[2], o_full[2], o_free, drain;
    uint64_t item_full[kItems], item_empty[kItems];
    Item item[kItems];
    int64_t red[kThreads / 32][2];
    uint32_t tmem;
    int dead, turn;                                            // turn: a product warp issues, the other waits
    uint8_t landed_turn[8];                                    // parity of a stage's next copy that lands before it is looked at
    uint8_t flying[kCopyWarps][2];                             // a copying warp's last two tensor copies: 128, 16: landed, 8: parity, stage
    int poisoned[kItems];
    uint32_t poison[kItems][D / 2];                            // 16 bits a column: which rows see a value that is not finite
};

template <int D, int PARTS, int COPY> struct Shape {
    static constexpr int kTiles = D <= 128 ? 2 : 1;            // row tiles of 128
    static constexpr int kRows = 128 * kTiles;
    static constexpr int kCols = D < 128 ? D : 128;            // columns of a stage
    static constexpr int kHalves = D / kCols;                  // stages of a block of K, or V
    static constexpr int kPanelBytes = kKeys * 128;
    static constexpr int kStage = kKeys * kCols * 2;
    static constexpr int kQTile = 128 * D * 2;                 // a row tile's queries, a part
    static constexpr int kQBytes = kTiles * PARTS * kQTile;
    // The softmax warps' room for 32 rows x 64 columns of output each, where a ring of four stages is left beside it; else
    // they use their queries' place.  (E4M3 codes would have a warp less to widen them: 326 us against 311.)
    static constexpr int kOutWarp = 32 * 128;
    static constexpr bool kOutRoom = kTiles == 2 && COPY != kCodeCopies && 224 * 1024 - kQBytes - 8 * kOutWarp >= 4 * kStage;
    static constexpr int kOutBytes = kOutRoom ? 8 * kOutWarp : 0;
    static constexpr int kRoom = 224 * 1024 - kQBytes - kOutBytes;
    static constexpr int kStages = kRoom / kStage < 8 ? kRoom / kStage : 8;
    static_assert(kStages >= 3, "K of a block and V of the one before, in part");
    // Warps that fill the ring, in turn.  A warp that passes on from fill f knows that f - kStages is released; its next fill
    // waits for f + kFillers - kStages, whose barrier tells that phase from the one before it only if f + kFillers - 2 kStages is.
    static constexpr int kFillers = kStages < kCopyWarps ? kStages : kCopyWarps;
    // (E4M3 codes come by tensor copies to the last panel of their stage and are widened there; a warp asks for its next stage's
    // before it widens this one's where that stage is free already, and else after.)
    static constexpr int kSmem = kQBytes + kOutBytes + kStages * kStage + (int)sizeof(Shared<D>);
    static_assert(kSmem <= 227 * 1024, "a block's shared memory");
    static constexpr int64_t kPart = (int64_t)kRows * (D + 2); // floats of a partial result: O by fours of columns, row after row, then m and l of each row
};

// A bounded wait; false (and from then on everywhere in the block) where the bound runs out.
struct Wait {
    volatile int *dead;
    uint32_t limit;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const
    {
        const uint32_t s = smem_addr(bar);
        for (uint32_t i = 0; i < limit; ++i) {
            uint32_t done;
            asm volatile("{\n\t.reg .pred p;\n\t"
                         "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                         "selp.u32 %0, 1, 0, p;\n\t}"
                         : "=r"(done) : "r"(s), "r"(parity) : "memory");
            if (done) return true;
            if (*dead) return false;
        }
        if (atomicExch(const_cast<int *>(dead), 1) == 0) atomicAdd(&g_wait_timeouts, 1u);
        return false;
    }
};
// Whether it is over already.
__device__ __forceinline__ bool test(uint64_t *bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(smem_addr(bar)), "r"(parity) : "memory");
    return done != 0;
}
// The same on the way out, whatever the others found: copies and products in flight end by themselves.
__device__ __forceinline__ void wait_out(uint64_t *bar, uint32_t parity)
{
    for (uint32_t i = 0; i < (1u << 22); ++i)
        if (test(bar, parity)) return;
}

// ------------------------------------------------------------------ values that some rows do not see

// A stage of V's block in shared memory, columns from col0 on, taken over by a warp.  Its first `keys` keys are real; every row of the
// tile sees those before `clear` (counted from the block's first).  Keys past the end become zeros; values from `clear` on that are
// not finite do too, and which rows see them is noted: those `rel` or more tokens behind the tile's first.
template <int D, bool BF16, int COLS>
__device__ __forceinline__ void sanitize(Shared<D> &sh, int slot, uint32_t stage, int keys, int clear, int col0, int lane)
{
    constexpr int kPieces = COLS / 8;
    const int from = max(clear, 0);
    // x * 0 + .. is a NaN from the first value on that is not finite: four instructions for eight values
    uint32_t odd = 0;
    auto add = [&](uint32_t x) {
        if constexpr (BF16) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(odd) : "r"(x), "r"(0u));
        else asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(odd) : "r"(x), "r"(0u));
    };
#pragma unroll 8
    for (int i = from * kPieces + lane; i < keys * kPieces; i += 32) {
        uint32_t u[4];
        lds16(u, stage + piece_at(i / kPieces, i % kPieces));
        add(u[0]); add(u[1]); add(u[2]); add(u[3]);
    }
#pragma unroll 4
    for (int i = keys * kPieces + lane; i < kKeys * kPieces; i += 32) sts16(stage + piece_at(i / kPieces, i % kPieces), 0u, 0u, 0u, 0u);
    if (!__any_sync(kFull, (odd & 0x7fff7fffu) != 0)) return;
#pragma unroll 1
    for (int i = from * kPieces + lane; i < keys * kPieces; i += 32) {
        const int row = i / kPieces, rel = min(row - clear + 1, 0xfffe);
        const uint32_t piece = stage + piece_at(row, i % kPieces);
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {
            constexpr uint32_t x = BF16 ? 0x7f80u : 0x7c00u;
            uint32_t half;
            asm volatile("{\n\t.reg .b16 h;\n\tld.shared.b16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(half) : "r"(piece + 2 * e) : "memory");
            if ((half & x) != x) continue;
            asm volatile("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tst.shared.b16 [%0], h;\n\t}" ::"r"(piece + 2 * e), "r"(0u) : "memory");
            const int col = col0 + 8 * (i % kPieces) + e;
            uint32_t *at = &sh.poison[slot][col >> 1];
            const unsigned shift = (col & 1) * 16;
            uint32_t old = *reinterpret_cast<volatile uint32_t *>(at);
            while (((old >> shift) & 0xffffu) > (uint32_t)rel) {
                const uint32_t got = atomicCAS(at, old, (old & ~(0xffffu << shift)) | ((uint32_t)rel << shift));
                if (got == old) break;
                old = got;
            }
            *(volatile int *)&sh.poisoned[slot] = 1;
        }
    }
}

// ------------------------------------------------------------------ softmax warps

// Queries of a warp's 32 rows into shared memory, eight elements a lane, in PARTS 16-bit parts; returns what
// the scores of this lane's row are to be multiplied by (fp16 products of a type with a wider range: the row's largest
// element is brought to 2^14 .. 2^15).
template <int D, bool BF16, int PARTS> __device__ __forceinline__ bool as_they_lie(const FlashParams &p)
{
    return PARTS == 1 && p.q_vec && p.dtype == (BF16 ? GDNA_BF16 : GDNA_F16);
}
template <int D, bool BF16, int PARTS, int COPY>
__device__ __forceinline__ float load_queries(const FlashParams &p, const Item &it, int rows, int row0, uint32_t q_smem, int lane)
{
    using S = Shape<D, PARTS, COPY>;
    constexpr int kLanes = D / 8, kPer = 32 / kLanes, kPasses = 32 / kPer;     // lanes of a row, rows of a pass
    constexpr int kGo = 8;                                     // passes asked for at once
    const int col = (lane % kLanes) * 8;
    const bool scaled = !BF16 && p.dtype != GDNA_F16;
    float mine = 1.f;
    // lane l has the place of the warp's row l
    const int t_mine = (int)p.group_div.quotient((unsigned)(row0 + lane));
    const int64_t place = (it.row0 + it.token0 + t_mine) * p.q_stride + ((int64_t)it.head * p.group + (row0 + lane - t_mine * p.group)) * p.d;
    // queries of the products' type go as they lie, and are on their way on return
    if (as_they_lie<D, BF16, PARTS>(p)) {
#pragma unroll 4
        for (int pass = 0; pass < kPasses; ++pass) {
            const int in_warp = pass * kPer + lane / kLanes;
            const int64_t from = __shfl_sync(kFull, place, in_warp) + col;
            const bool in = row0 + in_warp < rows && col < p.d;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                         ::"r"(q_smem + piece_at((row0 & 127) + in_warp, lane % kLanes)),
                           "l"(static_cast<const uint16_t *>(p.q) + (in ? from : 0)), "r"(in ? 16 : 0) : "memory");
        }
        return mine;
    }
#pragma unroll 1
    for (int pass = 0; pass < kPasses; pass += kGo) {
        uint4 raw[kGo][2];
#pragma unroll
        for (int k = 0; k < kGo; ++k) {
            const int in_warp = (pass + k) * kPer + lane / kLanes;
            const int64_t from = __shfl_sync(kFull, place, in_warp) + col;
            raw[k][0] = raw[k][1] = make_uint4(0u, 0u, 0u, 0u);
            if (row0 + in_warp >= rows || col >= p.d) continue;
            if (p.q_vec) {
                if (p.dtype == GDNA_F32) {
                    const uint4 *at = reinterpret_cast<const uint4 *>(static_cast<const float *>(p.q) + from);
                    raw[k][0] = at[0];
                    raw[k][1] = at[1];
                } else {
                    raw[k][0] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + from);
                }
            } else {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = col + j < p.d ? gdna::load_elem(p.q, from + j, p.dtype) : 0.f;
                raw[k][0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
                raw[k][1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
            }
        }
#pragma unroll
        for (int k = 0; k < kGo; ++k) {
            const int in_warp = (pass + k) * kPer + lane / kLanes;
            float x[8];
            if (!p.q_vec || p.dtype == GDNA_F32) {
                x[0] = __uint_as_float(raw[k][0].x); x[1] = __uint_as_float(raw[k][0].y);
                x[2] = __uint_as_float(raw[k][0].z); x[3] = __uint_as_float(raw[k][0].w);
                x[4] = __uint_as_float(raw[k][1].x); x[5] = __uint_as_float(raw[k][1].y);
                x[6] = __uint_as_float(raw[k][1].z); x[7] = __uint_as_float(raw[k][1].w);
            } else {
                const uint32_t u[4] = {raw[k][0].x, raw[k][0].y, raw[k][0].z, raw[k][0].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = p.dtype == GDNA_BF16 ? unpack16<true>(u[j]) : unpack16<false>(u[j]);
                    x[2 * j] = f.x;
                    x[2 * j + 1] = f.y;
                }
            }
            if (scaled) {                              // (for the whole warp)
                float top = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
#pragma unroll
                for (int off = kLanes / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
                int e = (int)(__float_as_uint(top) >> 23) - 127;
                e = top > 0.f && e < 128 ? max(e, -100) : 14;
                const float up = __uint_as_float((unsigned)(127 + 14 - e) << 23);
                const float back = __uint_as_float((unsigned)(127 - 14 + e) << 23);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= up;
                const int which = lane - (pass + k) * kPer;            // this lane's row among the pass's
                const float got = __shfl_sync(kFull, back, (which & (kPer - 1)) * kLanes);
                if (which >= 0 && which < kPer) mine = got;
            }
            const uint32_t at = q_smem + piece_at((row0 & 127) + in_warp, lane % kLanes);
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
                uint32_t u[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u[j] = pack16<BF16>(x[2 * j], x[2 * j + 1]);
                    const float2 f = unpack16<BF16>(u[j]);
                    x[2 * j] -= f.x;
                    x[2 * j + 1] -= f.y;
                }
                sts16(at + part * S::kQTile, u[0], u[1], u[2], u[3]);
            }
        }
    }
    return mine;
}

// 1 / (1 + e^-x): both steps to two units in the last place, far below a 16-bit output's rounding.
__device__ __forceinline__ float sigmoid(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.f + ex2(x * -1.4426950408889634f)));
    return y;
}
__device__ __forceinline__ void fma2(float &a, float &b, float s, float c)        // a = a s + c, b = b s + c
{
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}" : "+f"(a), "+f"(b) : "f"(s), "f"(c));
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// 16 columns of this thread's lane.
__device__ __forceinline__ void st16(uint32_t at, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                   "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}
__device__ __forceinline__ void add2(float &a, float &b, float c, float d)        // a += c, b += d
{
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}" : "+f"(a), "+f"(b) : "f"(c), "f"(d));
}

// ------------------------------------------------------------------ the kernel

// COPY: how keys come in.  (A template argument, for the registers of the warps that fill the ring.)
template <int D, bool BF16, int PARTS, int COPY>
__global__ void __launch_bounds__(kThreads, 1)
flash_rows(const FlashParams p, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
           const uint32_t polls)
{
    using S = Shape<D, PARTS, COPY>;
    constexpr int TILES = S::kTiles;
    // how far P may exceed 1 before O is rescaled (log2), and what fp16 weights are lifted by (log2): 2^(8 + 7) fits fp16.
    // (Slack 4 and lift 11: some row of 32 grew that far every few blocks, and a packed batch took 2070 us instead of 1735.)
    constexpr float kSlack = 8.f, kLift = BF16 ? 0.f : 7.f;
    extern __shared__ __align__(1024) uint8_t raw[];
    const uint32_t base = smem_addr(raw);
    const uint32_t q_smem = base, out_smem = base + S::kQBytes, ring = out_smem + S::kOutBytes;
    Shared<D> &sh = *reinterpret_cast<Shared<D> *>(raw + S::kQBytes + S::kOutBytes + S::kStages * S::kStage);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            tc::mbar_init(&sh.full[i], 1);
            tc::mbar_init(&sh.empty[i], TILES);
            tc::mbar_init(&sh.landed[i], 1);
            sh.landed_turn[i] = 0;
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh.q_full[i], 4);
            tc::mbar_init(&sh.q_over[i], 4);
            tc::mbar_init(&sh.s_full[i][0], 1);
            tc::mbar_init(&sh.s_full[i][1], 1);
            tc::mbar_init(&sh.p_full[i], 4);
            tc::mbar_init(&sh.o_full[i], 1);
        }
        tc::mbar_init(&sh.o_free, 4);
        tc::mbar_init(&sh.drain, TILES);
        for (int i = 0; i < kItems; ++i) {
            tc::mbar_init(&sh.item_full[i], 1);
            tc::mbar_init(&sh.item_empty[i], TILES + 1 + kCopyWarps + 8);
        }
        sh.turn = 0;
        for (int i = 0; i < kCopyWarps; ++i) sh.flying[i][0] = sh.flying[i][1] = 0;
        sh.dead = (base & 1023u) != 0;                 // (dynamic shared memory starts where the swizzle can)
        if (sh.dead) atomicAdd(&g_wait_timeouts, 1u);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) tc::tmem_alloc(&sh.tmem, 512);
    if (COPY != kLoads && tid == 32 * 12) {            // (the first copies would wait for them)
        asm volatile("prefetch.tensormap [%0];" ::"l"(&k_map) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&v_map) : "memory");
    }
    gdn::early_start<true>(nullptr, 0);                // (nothing of other kernels' is read or written before)
    const Totals all = totals(p, sh.red);              // (a barrier)
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem;
    const Wait wait{&sh.dead, sh.dead ? 0u : polls};
    auto wait_warp = [&](uint64_t *bar, uint32_t parity) { return (bool)__all_sync(kFull, wait(bar, parity)); };
    // for the end of another's item, which may have a million keys: 256 times the bound (a wait that runs out elsewhere ends these too)
    const Wait patient{&sh.dead, wait.limit < (1u << 24) ? wait.limit << 8 : 0xffffffffu};
    auto wait_long = [&](uint64_t *bar, uint32_t parity) { return (bool)__all_sync(kFull, patient(bar, parity)); };
    auto s_col = [&](int i) { return tmem + 128 * i; };                            // of S, and P
    auto o_col = [&](int t) { return tmem + 256 + (TILES == 2 ? t * D : 0); };
    auto rows_in = [&](const Item &it) {               // rows of a tile that are real
        return min(p.tile_tokens, it.n - it.token0) * p.group;
    };

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ---------------------------------------------------------------- softmax and output: a thread a row
        const int wg = warp >> 2, quarter = warp & 3;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        uint32_t items = 0, blocks_all = 0, s_count[2] = {0, 0}, o_count = 0;
        // this warp's queries of an item on their way into shared memory, and the products told once they are there
        auto ask_queries = [&](const Item &it) {
            return load_queries<D, BF16, PARTS, COPY>(p, it, rows_in(it), (TILES == 2 ? wg * 128 : 0) + quarter * 32,
                                                q_smem + (TILES == 2 ? wg * PARTS * S::kQTile : 0), lane);
        };
        auto tell_queries = [&]() {
            asm volatile("cp.async.wait_all;" ::: "memory");
            tc::fence_smem_async();
            __syncwarp();
            if (lane == 0) arrive(&sh.q_full[wg]);
        };
        float ahead = 0.f;                             // the next item's queries are in already, with this scale
        for (;; ++items) {
            const int slot = items % kItems;
            if (!wait_long(&sh.item_full[slot], (items / kItems) & 1)) break;
            const Item it = sh.item[slot];
            if (!it.valid) break;
            const int blocks = it.last - it.first, rows = rows_in(it);
            const int row0 = (TILES == 2 ? wg * 128 : 0) + quarter * 32, r = row0 + lane;
            const bool mine = TILES == 2 ? rows > wg * 128 : (items & 1) == (uint32_t)wg;
            if (!mine) {
                __syncwarp();
                if (lane == 0) arrive(&sh.item_empty[slot]);
                blocks_all += blocks;
                continue;
            }
            const int t = (int)p.group_div.quotient((unsigned)r);
            const bool real = r < rows;
            int limit = it.causal ? it.clear + t : it.clear;       // keys that the row sees
            if (!real || limit < 0) limit = 0;
            float m = kNegInf, l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f, scale = p.scale2;
            // (every phase of a barrier is waited for, in order: one that was skipped would be taken for the one after it)
            if (TILES == 1 && items > 0 && !wait_long(&sh.q_over[(items - 1) & 1], ((items - 1) >> 1) & 1)) break;
            if (blocks > 0) {
                if (ahead == 0.f) {
                    ahead = ask_queries(it);
                    tell_queries();
                }
                scale *= ahead;
                ahead = 0.f;
            }
            bool ok = true;
            for (int j = 0; j < blocks; ++j) {
                const int b = TILES == 2 ? 0 : (int)((blocks_all + j) & 1);
                const int col = TILES == 2 ? wg : b;   // which S
                ok = wait_long(&sh.s_full[wg][b], s_count[b]++ & 1);   // (the first of a second row tile: while another item is without one)
                if (!ok) break;
                tc::fence_after_sync();
                if (TILES == 1 && j + 1 == blocks && lane == 0) arrive(&sh.q_over[wg]);    // nothing reads these queries any more
                const uint32_t s_at = s_col(col) + lanes;
                const int seen = limit - (it.first + j) * kKeys;
                const bool masked = __any_sync(kFull, seen < kKeys);
                float s[4][32];
                auto scores = [&]() {
#pragma unroll
                    for (int x = 0; x < 4; ++x) tc::tmem_ld32(s_at + 32 * x, s[x]);
                    tc::ld_wait();
                    if (masked) {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (32 * x + i >= seen) s[x][i] = kNegInf;
                    }
                };
                auto largest = [&](int x, float top) { // of 32 columns, and top
                    float a = max3(top, s[x][0], s[x][1]), b = max3(s[x][2], s[x][3], s[x][4]);
#pragma unroll
                    for (int i = 5; i < 29; i += 4) { a = max3(a, s[x][i], s[x][i + 1]); b = max3(b, s[x][i + 2], s[x][i + 3]); }
                    return max3(max3(a, s[x][29], s[x][30]), b, s[x][31]);
                };
                // The weights by the maximum so far, with the block's maximum beside them: only where that is more than kSlack
                // above (in the first blocks, as a rule) they are taken again.
                bool behind = TILES == 1 && j > 0;     // the last block's products are still to be waited for
                uint32_t u[4][16];
                float t0, t1, t2, t3;
                for (bool fresh = j == 0;; fresh = false) {
                    scores();
                    if (fresh) {
                        float top[2] = {kNegInf, kNegInf};
#pragma unroll
                        for (int x = 0; x < 4; ++x) top[x & 1] = largest(x, top[x & 1]);
                        m = fmaxf(top[0], top[1]);
                    }
                    const float from = m == kNegInf ? 0.f : kLift - m * scale;
                    float top[2] = {m, kNegInf};
                    t0 = t1 = t2 = t3 = 0.f;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        top[x & 1] = largest(x, top[x & 1]);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) fma2(s[x][i], s[x][i + 1], scale, from);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float a = ex2(s[x][i]), c = ex2(s[x][i + 1]);
                            u[x][i / 2] = pack16<BF16>(a, c);
                            if (i & 2) add2(t2, t3, a, c);
                            else add2(t0, t1, a, c);
                        }
                    }
                    const float m_new = fmaxf(top[0], top[1]);
                    if (!__any_sync(kFull, (m_new - m) * scale > kSlack)) break;
                    const float f = ex2((m - m_new) * scale);
                    if (j > 0) {
                        // (two row tiles: the scores were asked for after the last block's products, so those are done)
                        if (behind) {
                            ok = wait_warp(&sh.o_full[wg], (o_count + j - 1) & 1);
                            if (!ok) break;
                            tc::fence_after_sync();
                            behind = false;
                        }
                        const float keep = m_new == m ? 1.f : f;
#pragma unroll 1
                        for (int x = 0; x < D; x += 32) {
                            float o[32];
                            tc::tmem_ld32(o_col(TILES == 2 ? wg : 0) + lanes + x, o);
                            tc::ld_wait();
                            uint32_t v[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(o[i] * keep);
                            tc::tmem_st32(o_col(TILES == 2 ? wg : 0) + lanes + x, v);
                        }
                        l0 *= keep; l1 *= keep; l2 *= keep; l3 *= keep;
                    }
                    m = m_new;
                }
                if (!ok) break;
#pragma unroll
                for (int x = 0; x < 4; ++x) st16(s_at + 16 * x, u[x]);
                add2(l0, l1, t0, t1);
                add2(l2, l3, t2, t3);
                tc::st_wait();
                if (behind) ok = wait_warp(&sh.o_full[wg], (o_count + j - 1) & 1);
                if (!ok) break;
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive(&sh.p_full[col]);
            }
            if (!ok) break;
            if (TILES == 1 && blocks == 0) {
                __syncwarp();
                if (lane == 0) arrive(&sh.q_over[wg]);
            }
            // with room for the output: the next item's queries first, so that its products run while this one's output is written (the
            // scores of the last block are here, so nothing reads the old ones any more)
            if (S::kOutRoom && blocks > 0) {
                const int after = (items + 1) % kItems;
                if (!wait_long(&sh.item_full[after], ((items + 1) / kItems) & 1)) break;
                const Item &then = sh.item[after];
                if (as_they_lie<D, BF16, PARTS>(p) && then.valid && then.first < then.last && rows_in(then) > wg * 128) ahead = ask_queries(then);
            }
            // ---- the output: a row's 64 columns at a time out of its thread's lane, through shared memory, where lanes then
            // take pieces of 16 bytes that lie side by side; gates the other way
            const bool final_rows = it.whole && !p.all_parts;
            const uint32_t stage = S::kOutRoom ? out_smem + warp * S::kOutWarp
                                               : q_smem + (TILES == 2 ? wg * PARTS * S::kQTile : 0) + quarter * 32 * 128;
            constexpr int kNext = S::kOutRoom ? 0 : S::kPanelBytes;    // from one panel of columns to the next
            const bool gated = p.gate != nullptr && final_rows, gate_pieces = gated && p.gate_vec && p.dtype != GDNA_F32;
            // lane l has the places of the warp's row l in the output and the gates; lanes take pieces of four rows at a time
            const int64_t token_row = it.row0 + it.token0 + t, head_row = (int64_t)it.head * p.group + (r - t * p.group);
            const int64_t out_row = token_row * p.out_stride + head_row * p.d;
            const int64_t gate_row = token_row * p.gate_stride + head_row * p.gate_head_stride;
            const unsigned reals = __ballot_sync(kFull, real);
            auto place = [&](int row) { return (uint32_t)(row * 128 + (((lane & 7) ^ (row & 7)) << 4)); };
            auto ask_gates = [&](int c) {
                const int col = 64 * c + 8 * (lane & 7);
#pragma unroll 2
                for (int i = 0; i < 8; ++i) {
                    const int from = 4 * i + (lane >> 3);
                    const int64_t at = __shfl_sync(kFull, gate_row, from) + col;
                    const bool in = (reals >> from & 1) && col < p.d;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                                 ::"r"(stage + c * kNext + place(from)), "l"(static_cast<const uint16_t *>(p.gate) + (in ? at : 0)), "r"(in ? 16 : 0) : "memory");
                }
            };
            // eight columns of this thread's row, scaled, gated, rounded and put into their place; `plain`: gates and output
            // are of the products' type, which the compiler then knows
            const bool plain = p.out_dtype == (BF16 ? GDNA_BF16 : GDNA_F16) && (!gated || (gate_pieces && p.dtype == (BF16 ? GDNA_BF16 : GDNA_F16)));
            if (TILES == 2 && gate_pieces)
#pragma unroll 1
                for (int c = 0; c < (S::kOutRoom ? 1 : D / 64); ++c) ask_gates(c);
            // (a single row tile: a lane writes its own row)
            const uint4 *gate_at = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.gate) + gate_row);
            uint4 ahead_g[8];
            auto ask_row = [&](int x) {                // 64 columns of the row's gates
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ahead_g[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (real && x + 8 * i < p.d) ahead_g[i] = gate_at[x / 8 + i];
                }
            };
            const bool wide = plain && p.out_vec;
            if (TILES == 1 && wide && gated) ask_row(0);
            if (blocks > 0) {
                const uint32_t last = TILES == 2 ? o_count++ : (o_count += blocks) - 1;
                if (!wait_warp(&sh.o_full[wg], last & 1)) break;
                tc::fence_after_sync();
                if (ahead != 0.f) tell_queries();
            }
            const float l = (l0 + l2) + (l1 + l3);
            const float norm = final_rows ? (l == 0.f ? 0.f : p.v_scale / l) : 1.f;
            const bool poisoned = blocks > 0 && *(volatile int *)&sh.poisoned[slot];
            float *part = p.parts + it.slot * S::kPart;
            if (!final_rows && real)
                *reinterpret_cast<float2 *>(part + S::kRows * D + 2 * r) = make_float2(m == kNegInf ? kNegInf : m * scale, l);
            if constexpr (TILES == 1) {
#pragma unroll 1
                for (int x = 0; x < (wide || !final_rows ? D : 0); x += 64) {
                    float o[2][32];
                    if (blocks > 0) {
                        tc::tmem_ld32(o_col(0) + lanes + x, o[0]);
                        tc::tmem_ld32(o_col(0) + lanes + x + 32, o[1]);
                        tc::ld_wait();
                    } else {
#pragma unroll
                        for (int i = 0; i < 64; ++i) o[i / 32][i % 32] = 0.f;
                    }
                    if (poisoned) {
                        const uint16_t *poison = reinterpret_cast<const uint16_t *>(sh.poison[slot]);
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (poison[x + i] <= (it.causal ? t : 0)) o[i / 32][i % 32] = __int_as_float(0x7fffffff);
                    }
                    if (!final_rows) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (real)
                                *reinterpret_cast<float4 *>(part + ((int64_t)(x / 4 + i) * S::kRows + r) * 4) =
                                    make_float4(o[i / 8][4 * i % 32], o[i / 8][4 * i % 32 + 1], o[i / 8][4 * i % 32 + 2], o[i / 8][4 * i % 32 + 3]);
                        continue;
                    }
                    if (gated) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t u[4] = {ahead_g[i].x, ahead_g[i].y, ahead_g[i].z, ahead_g[i].w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 g = unpack16<BF16>(u[e]);
                                o[i / 4][8 * i % 32 + 2 * e] *= sigmoid(g.x);
                                o[i / 4][8 * i % 32 + 2 * e + 1] *= sigmoid(g.y);
                            }
                        }
                        if (x + 64 < D) ask_row(x + 64);
                    }
                    uint4 *out_at = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + out_row + x);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float *y = &o[i / 4][8 * i % 32];
                        if (real && x + 8 * i < p.d)
                            out_at[i] = make_uint4(pack16<BF16>(y[0] * norm, y[1] * norm), pack16<BF16>(y[2] * norm, y[3] * norm),
                                                   pack16<BF16>(y[4] * norm, y[5] * norm), pack16<BF16>(y[6] * norm, y[7] * norm));
                    }
                }
                // other types, and rows that do not begin at 16 bytes
#pragma unroll 1
                for (int x = 0; x < (wide || !final_rows ? 0 : p.d); x += 8) {
                    float o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = 0.f;
                    if (blocks > 0) {
                        tc::tmem_ld8(o_col(0) + lanes + x, o);
                        tc::ld_wait();
                    }
                    float g[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] = 0.f;
                    if (gated && p.gate_vec && real) {
                        const uint4 u = gdna::ask4(p.gate, gate_row + x, p.dtype, true), v = gdna::ask4(p.gate, gate_row + x + 4, p.dtype, true);
                        const float4 a = gdna::got4(u, p.dtype, true), b = gdna::got4(v, p.dtype, true);
                        g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w; g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
                    } else if (gated && real) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (x + i < p.d) g[i] = gdna::load_elem(p.gate, gate_row + x + i, p.dtype);
                    }
                    const uint16_t *poison = reinterpret_cast<const uint16_t *>(sh.poison[slot]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (poisoned && poison[x + i] <= (it.causal ? t : 0)) o[i] = __int_as_float(0x7fffffff);
                        o[i] *= norm * (gated ? sigmoid(g[i]) : 1.f);
                    }
                    if (p.out_vec && real) {
                        gdna::store4(p.out, out_row + x, p.out_dtype, true, make_float4(o[0], o[1], o[2], o[3]));
                        gdna::store4(p.out, out_row + x + 4, p.out_dtype, true, make_float4(o[4], o[5], o[6], o[7]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (real && x + i < p.d) gdna::store_elem(p.out, out_row + x + i, p.out_dtype, o[i]);
                    }
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < D / 64; ++c) {
                    const uint32_t here = stage + c * kNext;
                    if (gate_pieces) {
                        if (S::kOutRoom && c > 0) ask_gates(c);
                        if (S::kOutRoom || c == 0) asm volatile("cp.async.wait_all;" ::: "memory");
                        __syncwarp();
                    }
                    // (rolled up: this code runs once an item, out of a cold instruction cache; unrolled it took longer)
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        const int x = 64 * c + 32 * half;
                        float o[32];
                        if (blocks > 0) {
                            tc::tmem_ld32(o_col(wg) + lanes + x, o);
                            tc::ld_wait();
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = 0.f;
                        }
                        if (poisoned) {
                            const uint16_t *poison = reinterpret_cast<const uint16_t *>(sh.poison[slot]);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (poison[x + i] <= (it.causal ? t : 0)) o[i] = __int_as_float(0x7fffffff);
                        }
                        if (!final_rows) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (real)
                                    *reinterpret_cast<float4 *>(part + ((int64_t)(x / 4 + i) * S::kRows + r) * 4) =
                                        make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                            continue;
                        }
                        const uint32_t at0 = here + lane * 128;
                        if (plain) {
                            uint32_t u[4][4];              // (all gates first, so that the four chains of latencies run side by side)
                            if (gated) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) lds16(u[i], at0 + (((4 * half + i) ^ (lane & 7)) << 4));
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const float2 g = unpack16<BF16>(u[i / 4][i % 4]);
                                    o[2 * i] *= sigmoid(g.x);
                                    o[2 * i + 1] *= sigmoid(g.y);
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i) u[i / 4][i % 4] = pack16<BF16>(o[2 * i] * norm, o[2 * i + 1] * norm);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                sts16(at0 + (((4 * half + i) ^ (lane & 7)) << 4), u[i][0], u[i][1], u[i][2], u[i][3]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t at = at0 + (((4 * half + i) ^ (lane & 7)) << 4);
                                float g[8];
                                if (gate_pieces) {
                                    uint32_t u[4];
                                    lds16(u, at);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const float2 f = p.dtype == GDNA_BF16 ? unpack16<true>(u[e]) : unpack16<false>(u[e]);
                                        g[2 * e] = f.x;
                                        g[2 * e + 1] = f.y;
                                    }
                                } else if (gated && p.gate_vec) {          // (fp32)
                                    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
                                    if (real && x + 8 * i < p.d) {
                                        const float4 *from = reinterpret_cast<const float4 *>(static_cast<const float *>(p.gate) + gate_row + x + 8 * i);
                                        a = from[0];
                                        b = from[1];
                                    }
                                    g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w; g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
                                } else if (gated) {
#pragma unroll
                                    for (int e = 0; e < 8; ++e)
                                        g[e] = real && x + 8 * i + e < p.d ? gdna::load_elem(p.gate, gate_row + x + 8 * i + e, p.dtype) : 0.f;
                                }
                                float y[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) y[e] = o[8 * i + e] * norm * (gated ? sigmoid(g[e]) : 1.f);
                                uint32_t u[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    u[e] = p.out_dtype == GDNA_BF16 ? pack16<true>(y[2 * e], y[2 * e + 1]) : pack16<false>(y[2 * e], y[2 * e + 1]);
                                sts16(at, u[0], u[1], u[2], u[3]);
                            }
                        }
                    }
                    if (!final_rows) continue;
                    __syncwarp();
                    const int col = 64 * c + 8 * (lane & 7);
#pragma unroll 1
                    for (int i0 = 0; i0 < 8; i0 += 4) {
                        uint16_t *at[4];
                        uint32_t u[4][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int from = 4 * (i0 + i) + (lane >> 3);
                            at[i] = static_cast<uint16_t *>(p.out) + (__shfl_sync(kFull, out_row, from) + col);
                            lds16(u[i], here + place(from));
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int from = 4 * (i0 + i) + (lane >> 3);
                            if (!(reals >> from & 1) || col >= p.d) continue;
                            if (p.out_vec) {
                                *reinterpret_cast<uint4 *>(at[i]) = make_uint4(u[i][0], u[i][1], u[i][2], u[i][3]);
                            } else {                       // element by element
#pragma unroll 1
                                for (int e = 0; e < 8 && col + e < p.d; ++e) {
                                    uint16_t x;
                                    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(x) : "r"(here + place(from) + 2 * e) : "memory");
                                    at[i][e] = x;
                                }
                            }
                        }
                    }
                    __syncwarp();
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                // (an item without blocks has no O: its arrival would stand for one of a warp that is not done with the item before)
                if (TILES == 1 && blocks > 0) arrive(&sh.o_free);
                arrive(&sh.item_empty[slot]);
            }
            blocks_all += blocks;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 10) {
            // ------------------------------------------------------------ work
            // Each lane has a segment; the one whose turn it is works out the item and writes it.
            uint32_t n = 0;
            auto room = [&]() -> bool {                // for the next item, with nothing noted against it
                const int slot = n % kItems;
                if (!wait_long(&sh.item_empty[slot], ((n / kItems) & 1) ^ 1)) return false;
                for (int i = lane; i < D / 2; i += 32) sh.poison[slot][i] = 0xffffffffu;
                if (lane == 0) sh.poisoned[slot] = 0;
                return true;
            };
            auto tell = [&]() {
                __syncwarp();
                if (lane == 0) arrive(&sh.item_full[n % kItems]);
                ++n;
            };
            Window win;
            win.load(p, 0, 0, 0);
            auto write = [&](int head, int64_t tau, int first, int last, bool whole, int64_t slot, int turned, int by) {
                Item &it = sh.item[n % kItems];
                const int token0 = (int)(tau * p.tile_tokens);
                it.row0 = win.s.row0;
                it.n = win.s.n;
                it.kv = win.s.kv;
                it.head = head;
                it.token0 = token0;
                it.first = first;
                it.last = last;
                it.turned = turned;
                it.by = by;
                it.whole = whole;
                it.causal = win.s.causal;
                it.clear = win.s.causal ? win.s.kv - win.s.n + token0 + 1 : win.s.kv;
                it.pages = win.s.pages;
                it.slot = slot;
                it.valid = 1;
            };
            const int g = p.grid, c = blockIdx.x;
            bool ok = true;
            const bool whole = whole_tiles(p, all);
            // (a request's own keys are joined with its prefix's: their records stand behind the others)
            if (c == 0 && lane == 0) *record_count(p) = whole || all.tiles == 0 ? 0 : all.tiles - p.own_tiles;
            if (whole) {
                for (int64_t k = 0; ok; ++k) {
                    const int64_t i = k * g + ((k & 1) ? g - 1 - c : c);
                    if (i >= all.tiles) break;         // (and so is every later turn)
                    const int at = win.find<false>(p, i);
                    if (at < 0) break;
                    ok = room();
                    if (ok && lane == at) {
                        const int64_t idx = i - (win.tiles - win.t.count * p.nkv), row = quotient(idx, p.nkv), tau = win.t.count - 1 - row;
                        write((int)(idx - row * p.nkv), tau, 0, (int)(((int64_t)keys_of(p, win.t, tau) + kKeys - 1) / kKeys), true, 0, 0, 0);
                    }
                    if (ok) tell();
                }
            } else {
                const int64_t run = run_of(p, all), x0 = c * run;
                const int64_t x1 = x0 + run < all.cost ? x0 + run : all.cost;
                for (int64_t x = x0; ok && x < x1;) {
                    const int at = win.find<true>(p, x);
                    if (at < 0) break;
                    int64_t end = 0, tile = 0, tau = 0;
                    int head = 0, first = 0, last = 0, blocks = 0, some = 0;
                    if (lane == at) {
                        const int64_t before = win.cost - win.t.cost * p.nkv;
                        head = (int)quotient(x - before, win.t.cost);
                        const int64_t y = x - before - head * win.t.cost;
                        tau = tile_at(win.t, y);
                        const int64_t begin = x - y + cost_before(win.t, tau);
                        end = begin + cost_of(p, win.t, tau);
                        blocks = (int)(((int64_t)keys_of(p, win.t, tau) + kKeys - 1) / kKeys);
                        first = x0 > begin ? blocks_before(x0 - begin, blocks) : 0;
                        last = x1 < end ? blocks_before(x1 - begin, blocks) : blocks;
                        tile = win.tiles - win.t.count * p.nkv + head * win.t.count + tau;
                        // a tile without keys is the block's in which it begins
                        some = first < last || (blocks == 0 && begin >= x0);
                        // and that block tells which have a part of the tile: from the one in whose run the first keys end to that in
                        // whose run the last ones begin (a run is longer than a block of keys, so those between all have some)
                        if (begin >= x0) {
                            int64_t b0 = quotient(begin + kLead + kKeys + run - 1, run) - 1, b1 = quotient(begin + kLead + (int64_t)kKeys * blocks - 1, run);
                            const int64_t most = quotient(end - 1, run);
                            if (b0 < c) b0 = c;
                            if (b0 > most) b0 = most;
                            if (b1 > most) b1 = most;
                            if (blocks == 0) b0 = b1 = c;
                            const bool one = b0 == b1 && !p.all_parts;
                            records(p)[tile] = Record{win.s.row0, tile + b0, win.s.n, head, (int)(tau * p.tile_tokens), one ? 0 : (int)(b1 - b0 + 1)};
                        }
                    }
                    if (__shfl_sync(kFull, some, at)) {
                        ok = room();
                        if (ok && lane == at) {
                            // Runs of one head's tiles begin at different keys, and what one block has read the others would
                            // read again long after.  So a long item's keys are taken in an order by which all blocks are at
                            // equal keys, modulo a run, at equal times: 512 rows over 60000 keys 375 -> 334 us, heads of 256 895 -> 589.
                            int turned = 0, by = 0;
                            if (last - first >= kLongItem) {
                                const int64_t period = run / kKeys, late = ((x - x0) / kKeys - first) % period;
                                const int clear = win.s.causal ? win.s.kv - win.s.n + (int)(tau * p.tile_tokens) + 1 : win.s.kv;
                                turned = min(last, clear / kKeys);
                                by = (int)(late < 0 ? late + period : late);
                                if (first + by >= turned) turned = by = 0;
                            }
                            write(head, tau, first, last, first == 0 && last == blocks, tile + c, turned, by);
                        }
                        if (ok) tell();
                    }
                    x = __shfl_sync(kFull, end, at);
                }
            }
            if (ok && room()) {
                if (lane == 0) sh.item[n % kItems].valid = 0;
                tell();
            }
        } else if (warp < 8 + TILES) {
            // ------------------------------------------------------------ products: a warp for each row tile
            // The whole warp walks along, with values that are the same in all lanes (from shuffles and votes), so that
            // descriptors stay in uniform registers; one lane issues.  (One thread by itself: 120 cycles a product.)  Two
            // warps, so that one's waits pass under the other's products.
            const int tile = warp - 8;
            constexpr uint32_t kQK = idesc16<BF16>(128, kKeys, false), kPV = idesc16<BF16>(128, S::kCols, true);
            constexpr int kSteps = S::kCols / 16;      // of a stage's columns
            const uint32_t t_base = __shfl_sync(kFull, tmem, 0), q_low = desc_low(__shfl_sync(kFull, q_smem, 0), 16);
            const uint32_t ring_k = desc_low(__shfl_sync(kFull, ring, 0), 16), ring_v = desc_low(__shfl_sync(kFull, ring, 0), S::kPanelBytes);
            const bool leader = elect();
            uint32_t items = 0, blocks = 0, q_count = 0, p_count = 0;  // (parities, of two barriers where there are two S)
            uint32_t o_turn = 0;                       // items that had blocks
            // the ring's next stage, and its phase
            uint32_t next = 0, phase = 0;
            struct Stages {
                uint32_t at[S::kHalves];
            };
            bool ok = true;
            auto take = [&]() {                        // the stages of the next block of K, or V, once they are full
                Stages x;
#pragma unroll
                for (int h = 0; h < S::kHalves; ++h) {
                    ok = ok && wait_warp(&sh.full[next], phase);
                    x.at[h] = next;
                    if (++next == (uint32_t)S::kStages) { next = 0; phase ^= 1; }
                }
                return x;
            };
            // (in the ring's order, which the copying warps count on: K of the next block before V of this one)
            auto release = [&](const Stages &x) {
                if (leader)
#pragma unroll
                    for (int h = 0; h < S::kHalves; ++h) tc::mma_commit(&sh.empty[x.at[h]]);
            };
            const uint32_t q_tile = q_low + ((tile * PARTS * S::kQTile) >> 4), o_tile = t_base + 256 + tile * D;
            auto qk = [&](uint32_t s, const Stages &x, uint64_t *bar) {            // S s = Q . K^T
                const uint32_t d = t_base + 128 * s;
                tc::fence_after_sync();
                if (leader) {
#pragma unroll
                    for (int i = 0; i < PARTS * S::kHalves; ++i) {
                        const int part = i / S::kHalves, h = i % S::kHalves;
                        const uint32_t a = q_tile + ((part * S::kQTile + h * S::kStage) >> 4);
                        const uint32_t b = ring_k + x.at[h] * (S::kStage >> 4);
#pragma unroll
                        for (int k = 0; k < kSteps; ++k) {             // (16 columns are 32 bytes of a panel)
                            const uint32_t off = (k >> 2) * (S::kPanelBytes >> 4) + (k & 3) * 2;
                            mma16_ss(d, a + off, b + off, kQK, i + k > 0);
                        }
                    }
                    tc::mma_commit(bar);
                }
                __syncwarp();
            };
            // A tile's P V and Q K go to the tensor core in one piece: with the two tiles' products between one another, both tiles'
            // scores were ready at once, and no softmax ran under products (period of a block 4700 cycles against 3500).  (Heads
            // of 64: the products are bound by their issue, which two warps do side by side: 283 us against 236.)
            constexpr bool kTurns = TILES == 2 && D == 128;
            auto mine_now = [&]() {
                if (!kTurns) return;
                if (leader)
                    for (uint32_t i = 0; i < (1u << 20); ++i)          // (the other holds it while it issues, and waits for nothing)
                        if (atomicCAS(&sh.turn, 0, 1) == 0) break;
                __syncwarp();
            };
            auto yours = [&]() {
                if (kTurns && leader) atomicExch(&sh.turn, 0);
            };
            auto pv = [&](uint32_t s, const Stages &x, uint32_t acc) {             // O += P . V
                const uint32_t a = t_base + 128 * s;
                ok = ok && wait_warp(&sh.p_full[s], (p_count >> s) & 1);
                p_count ^= 1u << s;
                if (!ok) return;
                mine_now();
                tc::fence_after_sync();
                if (leader)
#pragma unroll
                    for (int h = 0; h < S::kHalves; ++h) {
                        const uint32_t b = ring_v + x.at[h] * (S::kStage >> 4);
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k)           // (16 keys are 2048 bytes)
                            mma16_ts(o_tile + h * S::kCols, a + 8 * k, b + k * (2048 >> 4), kPV, k > 0 ? 1u : acc);
                    }
                __syncwarp();
            };
            for (; ok; ++items) {
                const int slot = items % kItems;
                if (!wait_long(&sh.item_full[slot], (items / kItems) & 1)) break;
                const Item *it = &sh.item[slot];
                if (!__shfl_sync(kFull, it->valid, 0)) break;
                const int first_block = __shfl_sync(kFull, it->first, 0), last_block = __shfl_sync(kFull, it->last, 0);
                const bool rows_here = __shfl_sync(kFull, rows_in(*it), 0) > 128 * tile;
                const uint32_t owner = items & 1;      // of a single row tile: the softmax warps take turns
                __syncwarp();
                if (leader) arrive(&sh.item_empty[slot]);
                if (!rows_here) {                      // the other tile's keys pass by
                    for (int j = 2 * first_block; ok && j < 2 * last_block; ++j) {
                        const Stages x = take();
                        if (ok && leader)
#pragma unroll
                            for (int h = 0; h < S::kHalves; ++h) arrive(&sh.empty[x.at[h]]);
                        __syncwarp();
                    }
                    continue;
                }
                auto s_full = [&](uint32_t block) { return TILES == 2 ? &sh.s_full[tile][0] : &sh.s_full[owner][block & 1]; };
                auto s_of = [&](uint32_t block) { return TILES == 2 ? (uint32_t)tile : block & 1; };
                if (first_block >= last_block) continue;
                const int q = TILES == 2 ? tile : (int)owner;
                Stages k_at = take();
                ok = ok && wait_warp(&sh.q_full[q], (q_count >> q) & 1);
                q_count ^= 1u << q;
                if (!ok) break;
                qk(s_of(blocks), k_at, s_full(blocks));
                release(k_at);
                for (int j = first_block; j < last_block; ++j, ++blocks) {
                    const bool more = j + 1 < last_block;
                    const uint32_t acc = j > first_block;
                    if (more) k_at = take();
                    if (!ok) break;
                    if constexpr (TILES == 1) {
                        if (more) {
                            qk(s_of(blocks + 1), k_at, s_full(blocks + 1));
                            release(k_at);
                        }
                        if (acc == 0 && o_turn++ > 0) ok = wait_warp(&sh.o_free, o_turn & 1);      // (of the last item with blocks)
                    }
                    const Stages v_at = take();
                    pv(s_of(blocks), v_at, acc);
                    if (!ok) break;
                    if constexpr (TILES == 1) {
                        if (leader) tc::mma_commit(&sh.o_full[owner]);
                    } else if (more) {
                        qk(tile, k_at, &sh.s_full[tile][0]);
                        yours();
                        release(k_at);
                    } else {
                        yours();
                        if (leader) tc::mma_commit(&sh.o_full[tile]);
                    }
                    release(v_at);
                    __syncwarp();
                }
            }
            // products in flight end before tensor memory is given back
            __syncwarp();
            if (leader) tc::mma_commit(&sh.drain);
            wait_out(&sh.drain, 0);
            __syncwarp();
        } else if (warp == 11) {
            // ------------------------------------------------------------ values that some rows do not see
            uint32_t items = 0, fills = 0, turns = 0;  // (turns: a parity for each stage)
            for (bool ok = true; ok; ++items) {
                const int slot = items % kItems;
                if (!wait_long(&sh.item_full[slot], (items / kItems) & 1)) break;
                const Item it = sh.item[slot];
                if (!it.valid) break;
                for (int j = it.first; ok && j < it.last; ++j) {
                    // (the ring's order: K of the first block, then K of the next and V of this one)
                    fills += (j == it.first ? S::kHalves : 0) + (j + 1 < it.last ? S::kHalves : 0);
                    const int key0 = j * kKeys, clear = it.clear - key0;
                    if (COPY == kTensorCopies && clear < kKeys)
                        for (int h = 0; ok && h < S::kHalves; ++h) {
                            const int st = (fills + h) % S::kStages;
                            const uint32_t turn = (turns >> st) & 1;
                            turns ^= 1u << st;
                            ok = wait_long(&sh.landed[st], turn);  // (the first: while all other blocks pass)
                            if (!ok) break;
                            sanitize<D, BF16, S::kCols>(sh, slot, ring + st * S::kStage, min(kKeys, it.kv - key0), clear, h * S::kCols, lane);
                            tc::fence_smem_async();
                            __syncwarp();
                            if (lane == 0) arrive(&sh.full[st]);
                        }
                    fills += S::kHalves;
                }
                __syncwarp();
                if (ok && lane == 0) arrive(&sh.item_empty[slot]);
            }
        } else if (warp >= 12) {
            // ------------------------------------------------------------ the ring
            constexpr int kPanels = S::kCols / 64, kPieces = S::kCols / 8;
            const int me = warp - 12;
            uint32_t items = 0, fills = 0;

            const bool codes = COPY == kCodeCopies || (COPY == kLoads && p.cache_dtype == GDNA_E4M3);
            constexpr bool ahead = COPY == kCodeCopies;
            constexpr uint32_t fillers = S::kFillers;

            // E4M3 codes of a stage, a row's where its last panel begins, to fp16: the lanes that read a row's write the row
            auto widen_stage = [&](uint32_t dst) {
                constexpr int kLanes = S::kCols / 16, kPer = 32 / kLanes, kGo = 4;
                const int q = lane % kLanes;
#pragma unroll 1
                for (int row0 = lane / kLanes; row0 < kKeys; row0 += kGo * kPer) {
                    uint32_t u[kGo][4];
#pragma unroll
                    for (int k = 0; k < kGo; ++k) lds16(u[k], dst + (kPanels - 1) * S::kPanelBytes + (row0 + k * kPer) * 128 + q * 16);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < kGo; ++k) {
                        uint32_t a[4], b[4];
                        auto widen = [](uint32_t x, uint32_t &lo, uint32_t &hi) {
                            asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
                                "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(lo), "=r"(hi) : "r"(x));
                        };
                        widen(u[k][0], a[0], a[1]); widen(u[k][1], a[2], a[3]);
                        widen(u[k][2], b[0], b[1]); widen(u[k][3], b[2], b[3]);
                        sts16(dst + piece_at(row0 + k * kPer, 2 * q), a[0], a[1], a[2], a[3]);
                        sts16(dst + piece_at(row0 + k * kPer, 2 * q + 1), b[0], b[1], b[2], b[3]);
                    }
                }
            };
            // a stage filled by this warp's own hand goes to the products
            auto hand_over = [&](int slot, int st, bool masked, int keys, int clear, int h) {
                __syncwarp();
                if (masked) sanitize<D, BF16, S::kCols>(sh, slot, ring + st * S::kStage, keys, clear, h * S::kCols, lane);
                tc::fence_smem_async();
                __syncwarp();
                if (lane == 0) arrive(&sh.full[st]);
            };
            // the stage whose codes are on their way
            int w_slot = 0, w_fill = -1, w_keys = 0, w_clear = 0, w_h = 0;
            auto widen_last = [&]() -> bool {
                if (w_fill < 0) return true;
                const int st = w_fill % S::kStages;
                const uint32_t parity = (uint32_t)(w_fill / S::kStages) & 1;
                const bool masked = w_clear < kKeys;
                w_fill = -1;
                if (!wait_warp(&sh.landed[st], parity)) {
                    wait_out(&sh.landed[st], parity);
                    return false;
                }
                widen_stage(ring + st * S::kStage);
                hand_over(w_slot, st, masked, w_keys, w_clear, w_h);
                return true;
            };

            // Fill f: the keys of block j, columns from h * kCols on, of K or V.
            auto fill = [&](const Item &it, int slot, int j, int h, bool is_v) -> bool {
                const uint32_t f = fills++;
                if (f % fillers != (uint32_t)me) return true;
                const int st = f % S::kStages;
                const uint32_t dst = ring + st * S::kStage, phase = ((f / S::kStages) & 1) ^ 1;
                const int key0 = block_at(it, j) * kKeys, keys = min(kKeys, it.kv - key0);       // (at least one)
                const int clear = is_v ? it.clear - key0 : kKeys;
                const bool masked = clear < kKeys;
                auto page_of = [&](int key, int &token) -> int {       // (key < kv)
                    if (it.pages == nullptr) {
                        token = (int)it.row0 + key;
                        return 0;
                    }
                    const unsigned q = p.page_div.quotient((unsigned)key);
                    token = key - (int)q * p.cache.page_size;
                    return it.pages[q];
                };

                if constexpr (COPY != kLoads) {
                    const int per = p.copy_keys, count = (keys + per - 1) / per;   // keys of a copy; copies of a panel (32 at most)
                    int page = 0, token = 0;
                    if (lane < count) page = page_of(key0 + lane * per, token);    // before the stage is waited for
                    if (ahead && !__all_sync(kFull, test(&sh.empty[st], phase)) && !widen_last()) return false;
                    if (!wait_warp(&sh.empty[st], phase)) return false;
                    if constexpr (ahead) {
                        if (lane == 0) arrive_expect(&sh.landed[st], (uint32_t)(count * per * 128));
                        __syncwarp();
                        if (lane < count)
                            copy_box(dst + (kPanels - 1) * S::kPanelBytes + lane * per * 128, is_v ? &v_map : &k_map, h * S::kCols, token, it.head,
                                     page, &sh.landed[st]);
                        const bool good = widen_last();
                        w_slot = slot; w_fill = (int)f; w_keys = keys; w_clear = clear; w_h = h;
                        return good;
                    }
                    // (a masked stage goes on to the warp that looks at its values)
                    uint64_t *bar = masked ? &sh.landed[st] : &sh.full[st];
                    uint32_t parity = phase ^ 1;
                    if (masked) {
                        parity = *(volatile uint8_t *)&sh.landed_turn[st];
                        __syncwarp();
                        if (lane == 0) *(volatile uint8_t *)&sh.landed_turn[st] = (uint8_t)(parity ^ 1);
                    }
                    if (lane == 0) sh.flying[me][f / fillers & 1] = (uint8_t)(128u | (masked ? 16u : 0u) | parity << 3 | st);
                    if (lane == 0) arrive_expect(bar, (uint32_t)(count * kPanels * per * 128));
                    __syncwarp();
                    if (lane < count)
#pragma unroll
                        for (int x = 0; x < kPanels; ++x)
                            copy_box(dst + x * S::kPanelBytes + lane * per * 128, is_v ? &v_map : &k_map, h * S::kCols + 64 * x, token,
                                     it.head, page, bar);
                    return true;
                } else {

                // by loads: lane l has the places of keys l, l + 32, ..
                int64_t place[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    place[i] = -1;
                    const int row = lane + 32 * i;
                    if (row < keys) {
                        int token;
                        const int page = page_of(key0 + row, token);
                        if (page >= 0 && page < p.cache.pages)
                            place[i] = (int64_t)page * p.cache.page_stride + (int64_t)token * p.cache.token_stride + (int64_t)it.head * p.cache.head_stride;
                    }
                }
                if (!wait_warp(&sh.empty[st], phase)) return false;
                const void *from = is_v ? p.v : p.k;
                if (p.copy_mode == kPieces16) {
                    // 16 bytes at a time, as they lie: E4M3 codes to the row's place in the last panel, to be widened there
                    const int elem = codes ? 1 : 2, each = 16 / elem, across = S::kCols / each;    // elements, pieces of a row
                    const int shift = 31 - __clz(across);
#pragma unroll 1
                    for (int i = 0; i < 4; ++i)
#pragma unroll 4
                        for (int x = 0; x < across; ++x) {
                            const int row = (x * 32 + lane) >> shift, piece = lane & (across - 1);
                            const int64_t at = __shfl_sync(kFull, i == 0 ? place[0] : i == 1 ? place[1] : i == 2 ? place[2] : place[3], row);
                            const int col = h * S::kCols + piece * each;
                            const bool in = at >= 0 && col < p.d;
                            const uint32_t to = dst + (codes ? (kPanels - 1) * S::kPanelBytes + (32 * i + row) * 128 + piece * 16
                                                             : piece_at(32 * i + row, piece));
                            const void *src = in ? static_cast<const uint8_t *>(from) + (at + col) * elem : from;
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(in ? 16 : 0) : "memory");
                        }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    __syncwarp();
                    if (codes) widen_stage(dst);
                } else {
                    // element by element: any alignment, any head size
#pragma unroll 1
                    for (int i = 0; i < 4; ++i)
#pragma unroll 1
                        for (int x = 0; x < kPieces; ++x) {
                            const int row = (x * 32 + lane) / kPieces, piece = lane % kPieces;
                            const int64_t at = __shfl_sync(kFull, i == 0 ? place[0] : i == 1 ? place[1] : i == 2 ? place[2] : place[3], row);
                            const int col = h * S::kCols + piece * 8;
                            float e[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) e[k] = at >= 0 && col + k < p.d ? gdna::load_elem(from, at + col + k, p.cache_dtype) : 0.f;
                            uint32_t u[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) u[k] = pack16<BF16>(e[2 * k], e[2 * k + 1]);
                            sts16(dst + piece_at(32 * i + row, piece), u[0], u[1], u[2], u[3]);
                        }
                }
                hand_over(slot, st, masked, keys, clear, h);
                return true;
                }
            };
            for (bool ok = true; ok; ++items) {
                const int slot = items % kItems;
                if (!wait_long(&sh.item_full[slot], (items / kItems) & 1)) break;
                const Item it = sh.item[slot];
                if (!it.valid) break;
                auto block = [&](int j, bool is_v) {
                    for (int h = 0; ok && h < S::kHalves; ++h) ok = fill(it, slot, j, h, is_v);
                };
                // in the products' order: K of the first block, then K of the next and V of this one
                if (it.first < it.last) block(it.first, false);
                for (int j = it.first; ok && j < it.last; ++j) {
                    if (j + 1 < it.last) block(j + 1, false);
                    block(j, true);
                }
                if (ahead && ok) ok = widen_last();    // (what it notes goes by the item's slot)
                __syncwarp();
                if (ok && lane == 0) arrive(&sh.item_empty[slot]);
            }
            __syncwarp();
            if (ahead && w_fill >= 0) wait_out(&sh.landed[w_fill % S::kStages], (uint32_t)(w_fill / S::kStages) & 1);
        }
    }
    __syncthreads();
    if (warp == 8) tc::tmem_dealloc(tmem, 512);
    // Where a wait ran out, anywhere in the block: copies in flight land before their memory is another block's.  (Asked here, as
    // the warp whose copies they are may have had nothing to wait for.  Two a warp: its third is asked for only after its first has
    // been used.)
    if (*(volatile int *)&sh.dead == 0) return;
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (COPY == kTensorCopies && warp >= 12)
        for (int i = 0; i < 2; ++i) {
            const unsigned x = *(volatile uint8_t *)&sh.flying[warp - 12][i];
            if (x != 0) wait_out(x & 16 ? &sh.landed[x & 7] : &sh.full[x & 7], x >> 3 & 1);
        }
}

// ------------------------------------------------------------------ launch

// The map of K's or V's rows: element, token, head, page; box: 128 bytes (a panel's 64 elements, or E4M3 codes) x `copy_keys` tokens.  What
// lies past a head, and in pages that are none, comes as zeros.  False where the encoder refuses the layout.
inline bool rows_map(const FlashParams &p, const void *base, CUtensorMap *map)
{
    const auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(gdn::tensor_map_encoder());
    if (encode == nullptr) return false;
    const bool codes = p.cache_dtype == GDNA_E4M3;
    const cuuint64_t size[4] = {(cuuint64_t)p.d, (cuuint64_t)(p.table != nullptr ? p.cache.page_size : p.rows), (cuuint64_t)p.nkv,
                                (cuuint64_t)(p.table != nullptr ? p.cache.pages : 1)};
    const int64_t strides[3] = {p.cache.token_stride, p.cache.head_stride, p.table != nullptr ? p.cache.page_stride : 64};
    cuuint64_t stride[3];
    for (int i = 0; i < 3; ++i) {
        int64_t bytes = strides[i] * (codes ? 1 : 2);
        if (size[i + 1] == 1 && bytes <= 0) bytes = 16;        // (a dimension of one)
        if (bytes <= 0 || bytes >= (int64_t{1} << 40)) return false;
        stride[i] = (cuuint64_t)bytes;
    }
    const cuuint32_t box[4] = {codes ? 128u : 64u, (cuuint32_t)p.copy_keys, 1, 1}, step[4] = {1, 1, 1, 1};
    return encode(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void *>(base), size, stride, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, codes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF16, int PARTS, int COPY>
cudaError_t launch_copy(const FlashParams &p, const CUtensorMap &k_map, const CUtensorMap &v_map, cudaStream_t s)
{
    using S = Shape<D, PARTS, COPY>;
    const cudaError_t e = gdn::allow_dynamic_smem<&flash_rows<D, BF16, PARTS, COPY>>(S::kSmem);
    if (e != cudaSuccess) return e;
    return gdn::launch_early(flash_rows<D, BF16, PARTS, COPY>, dim3(p.grid), kThreads, S::kSmem, s, true, p, k_map, v_map, gdn::tc_copy_wait_polls());
}

template <int D, bool BF16, int PARTS> cudaError_t launch(FlashParams p, cudaStream_t s)
{
    CUtensorMap k_map{}, v_map{};
    const bool codes = p.cache_dtype == GDNA_E4M3;
    // (heads of up to 64 codes do not fill a row of a stage: by loads)
    if (p.copy_mode == kTensorCopies && ((codes && !(D >= 128)) || !(rows_map(p, p.k, &k_map) && rows_map(p, p.v, &v_map))))
        p.copy_mode = kPieces16;
    if (p.copy_mode != kTensorCopies) return launch_copy<D, BF16, PARTS, kLoads>(p, k_map, v_map, s);
    if constexpr (!BF16 && (D >= 128))
        if (codes) return launch_copy<D, BF16, PARTS, kCodeCopies>(p, k_map, v_map, s);
    return launch_copy<D, BF16, PARTS, kTensorCopies>(p, k_map, v_map, s);
}

// 16-bit parts of a query: one where the products' type holds its type (fp16 holds a row of bf16's once that is scaled), else two.  (One
// for an F32 query in fp16 products and a bf16 output would halve the first product, but a score is off by what the query
// leaves out times the score itself: with 11 bits scores of a hundred by up to 0.05, weights by 5 %, which no output's type hides.)
template <int D, bool BF16> cudaError_t launch_by_type(const FlashParams &p, cudaStream_t s)
{
    const bool one = p.dtype == GDNA_BF16 || (!BF16 && p.dtype == GDNA_F16);
    return one ? launch<D, BF16, 1>(p, s) : launch<D, BF16, 2>(p, s);
}

// (each unit's own: internal linkage, as the counter has)
static inline cudaError_t wait_timeouts(unsigned *count) { return cudaMemcpyFromSymbol(count, g_wait_timeouts, sizeof(unsigned)); }

}  // namespace flash

// One unit each (gdnb_flash_64_f16.cu ...).
cudaError_t launch_flash_64_f16(const FlashParams &p, cudaStream_t s);
cudaError_t flash_timeouts_64_f16(unsigned *count);
cudaError_t launch_flash_64_bf16(const FlashParams &p, cudaStream_t s);
cudaError_t flash_timeouts_64_bf16(unsigned *count);
cudaError_t launch_flash_128_f16(const FlashParams &p, cudaStream_t s);
cudaError_t flash_timeouts_128_f16(unsigned *count);
cudaError_t launch_flash_128_bf16(const FlashParams &p, cudaStream_t s);
cudaError_t flash_timeouts_128_bf16(unsigned *count);
cudaError_t launch_flash_256_f16(const FlashParams &p, cudaStream_t s);
cudaError_t flash_timeouts_256_f16(unsigned *count);
cudaError_t launch_flash_256_bf16(const FlashParams &p, cudaStream_t s);
cudaError_t flash_timeouts_256_bf16(unsigned *count);

}  // namespace gdnb

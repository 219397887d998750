// gdna_attn_tc.cuh -- paged decode attention on the tensor cores (head sizes 64,
// 128 and 256, and those in between): the kernel's template.  gdna_attn.cuh has the deal of the work and
// the partial results.
//
// Mathematics.  With few query rows (8 to 64: the tokens and the group's heads) and
// many keys, the keys take the side of the product that is 16 wide and the query
// rows the side that is 8 wide:
//
//     S^T [16 keys x 8 rows]  = K [16 x D] . Q^T          D/16 products a row tile
//     O^T [D x 8 rows]       += V^T [D x 16] . P^T        D/16 products a row tile
//
// so a row tile of 8 costs what it holds.  A warp takes 16 keys at a time with a
// running maximum m and sum l for each row: S^T's columns are rows, so the maximum
// over keys is three shuffles for each row, and the rescale of O^T is by its own columns.  P^T
// needs the transpose of what the first product leaves; an 8 x 8 register transpose
// (movmatrix) does it, nothing passes through shared memory.
//
// Rounding.  K and V are exact in the products (E4M3 widens to fp16 exactly).  The
// queries enter in as many 16-bit parts as their type needs (`q_parts`: x = hi + lo
// [+ lower]), scaled by a power of two per row for fp16 products, so that no query
// over- or underflows.  The weights exp2(s - m) <= 1 enter in two
// parts, three where bf16 products give an fp32 output: one part's 2^-9 (2^-12 in fp16), relative to the largest
// values, would show where sums cancel.  For fp16 products they are lifted by 2^15, and with them l and O, until a part is
// added up: fp16's steps end at 2^-24, and one key far ahead of the others (a first token that all attend to) whose value is
// near zero leaves the output to weights that small.  Lifted, a weight is held to 2^-40 of the row's largest, or to 2^-22 of
// itself (500 keys, f16, the first 16 nats ahead and its value zero: 6e-6 of the output's norm, 1e-1 without).
// m, l, S and O are fp32.
//
// What a row does not see.  Masked scores are replaced, not added to.  Keys past the
// sequence's end are not loaded (zeros stand for them).  The keys that some tokens see
// and others do not (the last q_len - 1) may hold Inf or NaN values, and 0 * NaN would
// carry them into rows that do not see them: there a tile with a non-finite V adds its
// rows key by key instead.
//
// Data.  A block is some producer warps and W consumer warps.  A
// producer walks the block's parts on its own and keeps its rings full: it is already
// copying the next item's keys while the consumers finish the last one's rows.  Each
// consumer warp (or the R warps that share keys, each with its own rows) has a ring of
// stages in shared memory, a step's K and V each, with a full and an empty mbarrier a
// stage.  Rows lie in panels of 128 bytes with the 128-byte swizzle (64 with the 64-byte
// one), so eight rows of an ldmatrix start in eight different bank groups.
//   A tensor copy brings as many keys as surely lie in one page, 16 or a smaller power of two
// that divides the page size, one lane a copy; 16 keys come with all panels of a head at once
// (a producer pays some 40 ns a copy, one after the other).  Where that makes more than 32
// copies (short pages), for heads that end within their only panel, and for layouts that the
// encoder refuses, the producer's lanes copy 16 bytes at a time (cp.async) to the same places.
// Head sizes in between run padded to the next of the three: a copy fills what lies past a
// head with zeros.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "gdna_attn.cuh"
#include "gdn_tc.cuh"

namespace gdna {
namespace tc {

constexpr int kKeys = 16;                  // keys of a block: one side of a product
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kSmemOne = 224 * 1024, kSmemTwo = 111 * 1024;      // of a block beside its static arrays: one, two an SM
constexpr int kMaxStages = 6;              // of a ring
// Slots of the parts in hand.  The producer tells part n + 1 before it waits for the release of step n - stages.  With one
// step a part, step n - 1 - stages is then known to be released, but its part may still be added up: stages + 3 parts, from
// that one to n + 1, need a slot each.
constexpr int kQueue = kMaxStages + 3;

__device__ __forceinline__ unsigned smem_addr(const void *p) { return (unsigned)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void ldsm4(unsigned (&r)[4], unsigned addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(unsigned (&r)[4], unsigned addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// The transpose of an 8 x 8 matrix of 16-bit elements, one row of two a lane.
__device__ __forceinline__ unsigned transpose8(unsigned x)
{
    unsigned y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void lds16(unsigned (&r)[4], unsigned addr)
{
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void cp_async16(unsigned dst, const void *src, bool real)
{
    const int n = real ? 16 : 0;           // 0: sixteen zero bytes, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// Some keys of a head, from element x on; the map's other dimension is the panel.
// Keys that are read once are the first to leave the L2 (`policy`), which has the program's code, block table and
// activations to keep (two-token verify: 74.6 us against 80.9).
__device__ __forceinline__ void copy_keys(unsigned dst, const CUtensorMap *map, int x, int token, int head, int page, unsigned bar,
                                          uint64_t policy)
{
    asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
                 "[%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;"
                 ::"r"(dst), "l"(map), "r"(x), "r"(token), "r"(0), "r"(head), "r"(page), "r"(bar), "l"(policy) : "memory");
}
__device__ __forceinline__ uint64_t keep_policy(bool once)
{
    uint64_t policy;
    if (once) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
    return policy;
}
// A hint only: nothing is read.
__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void arrive_expect(uint64_t *bar, unsigned bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
// One arrival once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void arrive_copies(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// Waits on the kernel's barriers that ran out on this device (each cache type's kernels have their own).
static __device__ unsigned g_wait_timeouts;

// 16-bit operand type of the products: bf16 for a bf16 cache, else fp16.  kLift: what weights are multiplied by for it.
template <int CACHE> struct Op {
    static constexpr float kLift = 32768.f;
    __device__ static unsigned pack(float a, float b)
    {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<unsigned *>(&h);
    }
    __device__ static float2 unpack(unsigned u) { return __half22float2(*reinterpret_cast<__half2 *>(&u)); }
    __device__ static void mma(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1)
    {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
template <> struct Op<GDNA_BF16> {
    static constexpr float kLift = 1.f;
    __device__ static unsigned pack(float a, float b)
    {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<unsigned *>(&h);
    }
    __device__ static float2 unpack(unsigned u)
    {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    __device__ static void mma(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1)
    {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// Four E4M3 values of a word to four fp16, exactly: the low two, the high two.
__device__ __forceinline__ void widen4(unsigned x, unsigned &lo, unsigned &hi)
{
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(x));
}

template <int CACHE, int D, int NT, int R> struct Shape {
    static constexpr int kElem = CACHE == GDNA_E4M3 ? 1 : 2;
    static constexpr int kRowBytes = D * kElem;                // 64, 128, 256 or 512
    static constexpr int kPanel = kRowBytes < 128 ? kRowBytes : 128;           // bytes of a row in a panel
    static constexpr int kPanels = kRowBytes / kPanel;
    static constexpr int kPanelBytes = kKeys * kPanel;
    static constexpr int kBlockBytes = kKeys * kRowBytes;      // K, or V, of a block
    // Blocks of 16 keys a step.  Two where three stages of them fit a ring: the maximum's shuffles, the
    // barriers and the loop are then paid once for 32 keys (256 requests over an E4M3 cache: 158 us against
    // 212; 32 rows, bf16, D 128: 88 against 106).
    static constexpr int kBlocks = kRowBytes <= 128 || (kRowBytes == 256 && R >= 2) || R >= 4 ? 2 : 1;
    static constexpr int kStep = kKeys * kBlocks;
    static constexpr int kStage = 2 * kBlocks * kBlockBytes;   // K's blocks, then V's
    // Blocks on an SM.  Rows up to 256 bytes: two, so that one reads on while the other goes from an item to the
    // next (256 requests over an E4M3 cache, D 128: 104 us against 119 with one block of eight consumers; 32 requests
    // over a bf16 cache, D 128: 100.9 against 102.5).  Longer rows: one, whose rings hold more (262144 keys, D 256:
    // 167 us against 177 with two).
    static constexpr int kPerSm = kRowBytes <= 256 && R <= 4 ? 2 : 1;
    // Consumers on an SM: eight, with 168 registers each; four (255 registers) where eight rings of such long rows
    // would hold one stage.
    static constexpr int kWarps = kPerSm == 2 || (kRowBytes == 512 && R == 1) ? 4 : 8;
    static constexpr int kKeyWarps = kWarps / R;
    static constexpr int kRows = 8 * NT * R;
    // Producers, each for its own rings: at most as many warps as leave the consumers their registers.
    static constexpr int kProducers = kKeyWarps < (kPerSm == 2 ? 2 : 4) ? kKeyWarps : kPerSm == 2 ? 2 : 4;
    static constexpr int kThreads = 32 * (kWarps + kProducers);
    static constexpr int kCopies = 2 * kBlocks;                // blocks of K and V of a stage
    static constexpr int kQPitch = 2 * D + 16;
    // the consumers' sums are added up some columns at a time: 64 where three stages fit beside them
    static constexpr int kSmem = kPerSm == 2 ? kSmemTwo : kSmemOne;
    static constexpr int kColumns = 1024 + 3 * kKeyWarps * kStage + 2 * kRows * kQPitch + kKeyWarps * kRows * 68 * 4 <= kSmem ? 64 : 32;
    static constexpr int kSumPitch = kColumns + 4;             // floats
    static constexpr int kSumBytes = kKeyWarps * kRows * kSumPitch * 4;
    static_assert(kKeyWarps * kCopies <= 32, "a lane for each block of a step");

    // Swizzled place of byte `b` of row `r` in a block.
    __device__ __forceinline__ static unsigned place(unsigned r, unsigned b)
    {
        if constexpr (kPanel == 128) return b / 128 * kPanelBytes + r * 128 + ((b % 128) ^ ((r & 7) << 4));
        else return r * 64 + (b ^ (((r >> 1) & 3) << 4));
    }
    // From the place of (row, byte 0 or 16) to that of 32 x cols further on.
    __device__ __forceinline__ static unsigned across(unsigned at, int x)
    {
        return (at ^ (unsigned)(32 * x % kPanel)) + 32 * x / kPanel * kPanelBytes;
    }
};

// The query rows of an item, eight elements a lane: `fetch` brings the rows of some passes
// into registers, `put` leaves them in shared memory in 16-bit parts.  For E4M3 the elements
// stand in the order in which K's come: a 32-bit word of four becomes two operand registers,
// slots 2q, 2q+1 and 8+2q, 8+2q+1 of the 16 that a product contracts.
template <int CACHE, int D, int NT, int R> struct Queries {
    using S = Shape<CACHE, D, NT, R>;
    using O = Op<CACHE>;
    static constexpr int kRows = S::kRows, kLanes = D / 8, kPerWarp = 32 / kLanes;        // lanes of a row, rows of a warp
    static constexpr int kPasses = (kRows + S::kWarps * kPerWarp - 1) / (S::kWarps * kPerWarp);
    static constexpr int kGo = kPasses < 4 ? kPasses : 4;      // passes at once
    uint4 raw[kGo][2];

    __device__ __forceinline__ void fetch(const AttnParams &p, const Part &part, int pass)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int head = part.item / p.row_tiles, row0 = (part.item - head * p.row_tiles) * kRows;
#pragma unroll
        for (int k = 0; k < kGo; ++k) {
            const int r = ((pass + k) * S::kWarps + warp) * kPerWarp + lane / kLanes, row = row0 + r;
            raw[k][0] = raw[k][1] = make_uint4(0u, 0u, 0u, 0u);
            if (r < kRows && row < p.q_len * p.group && (lane % kLanes) * 8 < p.d) {
                const int token = row / p.group;
                const int64_t from = ((int64_t)part.seq * p.q_len + token) * p.q_stride +
                                     ((int64_t)head * p.group + (row - token * p.group)) * p.d + (lane % kLanes) * 8;
                raw[k][0] = ask4(p.q, from, p.dtype, p.q_vec);
                raw[k][1] = ask4(p.q, from + 4, p.dtype, p.q_vec);
            }
        }
    }

    __device__ __forceinline__ void put(const AttnParams &p, int pass, int q_parts, uint8_t *qs, float *row_scale)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = (lane % kLanes) * 8;
#pragma unroll
        for (int k = 0; k < kGo; ++k) {
            const int r = ((pass + k) * S::kWarps + warp) * kPerWarp + lane / kLanes;
            float back = 1.f, x[8];
            const float4 a = got4(raw[k][0], p.dtype, p.q_vec), b = got4(raw[k][1], p.dtype, p.q_vec);
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
            if constexpr (CACHE != GDNA_BF16) {                // fp16: the row's largest element to 2^14 .. 2^15
                float top = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
#pragma unroll
                for (int off = kLanes / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
                int e = (int)(__float_as_uint(top) >> 23) - 127;
                e = top > 0.f && e < 128 ? max(e, -100) : 14;
                const float up = __uint_as_float((unsigned)(127 + 14 - e) << 23);
                back = __uint_as_float((unsigned)(127 - 14 + e) << 23);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= up;
            }
            if (r < kRows) {
                for (int part = 0; part < q_parts; ++part) {
                    unsigned u[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        u[j] = O::pack(x[2 * j], x[2 * j + 1]);
                        const float2 f = O::unpack(u[j]);
                        x[2 * j] -= f.x;
                        x[2 * j + 1] -= f.y;
                    }
                    uint8_t *to = qs + (part * kRows + r) * S::kQPitch;
                    if constexpr (CACHE == GDNA_E4M3) {
                        const int slot = (at & ~15) + (at & 8) / 2;
                        *reinterpret_cast<uint2 *>(to + slot * 2) = make_uint2(u[0], u[2]);
                        *reinterpret_cast<uint2 *>(to + (slot + 8) * 2) = make_uint2(u[1], u[3]);
                    } else {
                        *reinterpret_cast<uint4 *>(to + at * 2) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
                if (at == 0) row_scale[r] = p.scale * back;
            }
        }
    }
};

// The tensor copies: how many keys one brings (those that lie in one page wherever pages begin: 16, or a smaller power
// of two that divides the page size; 0: no tensor copies), and in how many pieces a head comes.
struct Copies {
    int keys, pieces;
};

// What a producer leaves behind: the next stage, the parity of its empty barrier's next wait, and how many of
// the stages before it were filled (at most all).
struct Ring {
    int slot, filled;
    unsigned phase;
    bool ok;                               // every wait was in time
};

// Producer warp `who` of P: fills the rings of consumers who, who + P, .., part after part.  The first one tells
// the consumers the parts after the first, in `queue`, as it comes to them; a part of no sequence ends them.
template <int CACHE, int D, int NT, int R>
__device__ __forceinline__ Ring produce(const AttnParams &p, Run run, int c, int who, int P, const CUtensorMap &k_map, const CUtensorMap &v_map,
                                        const Copies copies, int stages, unsigned polls, uint8_t *smem,
                                        uint64_t (*full)[Shape<CACHE, D, NT, R>::kKeyWarps],
                                        uint64_t (*empty)[Shape<CACHE, D, NT, R>::kKeyWarps], Part *queue, uint64_t *told)
{
    using S = Shape<CACHE, D, NT, R>;
    constexpr int TW = S::kKeyWarps, KB = S::kBlocks;
    const int lane = threadIdx.x & 31;
    const unsigned page_size = (unsigned)p.cache.page_size, ring = smem_addr(smem);
    int slot = 0, filled = 0, entered = 0;
    unsigned phase = 1;                    // the first round finds all stages empty
    bool ok = true;

    // The steps of the block's parts in order.  Pages are looked up a step before they are needed, also from
    // one part to the next: a load's latency there would leave the rings dry.  What a stage's refill waits for
    // is short for the same reason.  The table is read by plain loads: the call before this one may still write it when
    // this kernel becomes resident, so it is not read-only for the kernel's life.
    // lane: a copy of a unit, some keys of a block of K or V for consumer y (or, without tensor copies, a key of each)
    const int per = copies.keys != 0 ? S::kCopies * (kKeys / copies.keys) : 32;
    const int y = who + lane / per * P, copy = lane % per, block = copy % KB, values = copy / KB % 2, row = copy / S::kCopies * copies.keys;
    const unsigned first = copies.keys != 0 ? y * S::kStep + block * kKeys + row : who * S::kStep + lane % S::kStep;     // its key of a unit
    int left = 0, head = 0;                // steps of the part that are not looked up; its key head
    unsigned key = 0, keys = 0;            // the key to look up next, the sequence's keys
    const int32_t *table = nullptr;
    Part part = {};
    bool more = true, fresh = false;       // a step is left; a part was entered just now
    auto enter = [&]() {                   // the next part
        more = fresh = next_part(p, run, c, part);
        if (!more) part.seq = -1;
        if (who == 0 && lane == 0 && entered > 0) {
            queue[entered % kQueue] = part;
            arrive(&told[entered % kQueue]);
        }
        ++entered;
        if (!more) return;
        left = (int)(part.u1 - part.u0);
        key = (unsigned)(part.u0 * TW) * S::kStep + first;
        keys = (unsigned)part.keys;
        table = p.table + part.seq * p.table_stride;
        head = part.item / p.row_tiles;
    };
    auto warm = [&]() {                    // its query and gate rows on their way to the L2, before they are asked for
        fresh = false;
        if (who != P - 1) return;
        const int elem = p.dtype == GDNA_F32 ? 4 : 2;
        const int row0 = (part.item - head * p.row_tiles) * S::kRows, rows = min(S::kRows, p.q_len * p.group - row0);
        for (int r = lane >> 2; r < rows; r += 8) {            // four lanes a row, a line of 128 bytes each at a time
            const int row = row0 + r, token = row / p.group;
            const int64_t n = (int64_t)part.seq * p.q_len + token, h = (int64_t)head * p.group + (row - token * p.group);
            for (int at = (lane & 3) * 128; at < p.d * elem; at += 512) {
                prefetch_l2(static_cast<const uint8_t *>(p.q) + (n * p.q_stride + h * p.d) * elem + at);
                if (p.gate != nullptr)
                    prefetch_l2(static_cast<const uint8_t *>(p.gate) + (n * p.gate_stride + h * p.gate_head_stride) * elem + at);
            }
        }
    };
    enter();

    if (copies.keys != 0) {
        const bool mine = y < TW;
        const uint64_t policy = keep_policy(p.row_tiles == 1);
        const unsigned dst = ring + (mine ? y : 0) * stages * S::kStage + (values * KB + block) * S::kBlockBytes + row * S::kPanel;
        const CUtensorMap *map = values ? &v_map : &k_map;
        int page = 0, token = 0;
        auto look_up = [&]() {             // past the cache (zeros) if there is no such page
            page = -1;
            token = 0;
            if (mine && key < keys) {
                const unsigned n = p.page_div.quotient(key);
                token = (int)(key - n * page_size);
                page = table[n];
            }
        };
        if (more) look_up();
        while (more) {
            const int at = (unsigned)page < (unsigned)p.cache.pages ? page : (int)p.cache.pages, from = token, of = head;
            key += TW * S::kStep;
            if (--left == 0) enter();
            if (more) look_up();
            ok = __all_sync(kFull, !mine || gdn::tc::mbar_wait(&empty[slot][mine ? y : 0], phase, polls));
            if (!ok) break;
            if (mine && copy == 0) arrive_expect(&full[slot][y], S::kStage);
            __syncwarp();
            if (mine)
                for (int z = 0; z < copies.pieces; ++z)
                    copy_keys(dst + slot * S::kStage + z * S::kPanelBytes, map, z * (S::kPanel / S::kElem), from, of, at,
                              smem_addr(&full[slot][y]), policy);
            filled = min(filled + 1, stages);
            if (++slot == stages) { slot = 0; phase ^= 1; }
            if (fresh) warm();
        }
    } else {
        const int64_t page_bytes = p.cache.page_stride * S::kElem, token_bytes = p.cache.token_stride * S::kElem;
        constexpr int kPieces = S::kRowBytes / 16, kAtOnce = 32 / kPieces;     // 16-byte pieces of a row, rows at once
        const int sub = lane / kPieces, piece = lane % kPieces * 16;
        int page = -1;
        unsigned place = 0;                // of the looked-up key in its page
        auto look_up = [&]() {             // lane j: key j of a consumer's step
            page = -1;
            if (key < keys) {
                const unsigned n = p.page_div.quotient(key);
                place = key - n * page_size;
                page = table[n];
            }
        };
        if (more) look_up();
        while (more && ok) {
            const int64_t base = (int64_t)head * p.cache.head_stride * S::kElem;
            const uint8_t *kb = static_cast<const uint8_t *>(p.k) + base, *vb = static_cast<const uint8_t *>(p.v) + base;
            for (int z = who; z < TW && ok; z += P) {
                const int64_t at = (unsigned)page < (unsigned)p.cache.pages ? page * page_bytes + place * token_bytes : -1;
                const bool last = z + P >= TW;
                key += (last ? TW - (z - who) : P) * S::kStep;
                if (last && --left == 0) enter();
                if (more) look_up();
                ok = __all_sync(kFull, gdn::tc::mbar_wait(&empty[slot][z], phase, polls));
                if (!ok) break;
                const unsigned to = ring + (z * stages + slot) * S::kStage;
#pragma unroll 4
                for (int r = 0; r < S::kStep; r += kAtOnce) {
                    const int row = r + sub;
                    const int64_t from = __shfl_sync(kFull, at, row);
                    const bool on = from >= 0 && piece < p.d * S::kElem;
                    const unsigned dst = to + row / kKeys * S::kBlockBytes + S::place(row % kKeys, piece);
                    cp_async16(dst, kb + (on ? from + piece : 0), on);
                    cp_async16(dst + KB * S::kBlockBytes, vb + (on ? from + piece : 0), on);
                }
                arrive_copies(&full[slot][z]);
            }
            if (++slot == stages) { slot = 0; phase ^= 1; }
            if (fresh) warm();
        }
        gdn::cp_async_wait<0>();
    }
    return Ring{slot, filled, phase, ok};
}

// A wait gave up: NaN for every row of the block's parts.
static __device__ __noinline__ void fill_nan(const AttnParams &p, Run run, int c, int rows)
{
    const float nan = __int_as_float(0x7fc00000);
    Join join = {0, 0, 0, 0};
    Part part;
    while (next_part(p, run, c, part)) {
        const int head = part.item / p.row_tiles, row0 = (part.item - head * p.row_tiles) * rows;
        float *to = part_of(p, 2 * c + (part.begins ? 1 : 0));
        for (int i = threadIdx.x; i < rows * p.d; i += blockDim.x) {
            const int r = i / p.d, x = i - r * p.d;
            if (row0 + r >= p.q_len * p.group) break;
            if (part.begins && part.ends) {
                write_out(p, part.seq, head, row0 + r, x, nan);
                if (x == 0) write_lse(p, part.seq, head, row0 + r, nan, nan);
            } else {
                to[r * p.d + x] = nan;
                if (x == 0) to[rows * p.d + 2 * r] = to[rows * p.d + 2 * r + 1] = nan;
            }
        }
        if (part.begins && !part.ends) join = Join{part.seq, part.item, part.blocks, 0};
    }
    if (threadIdx.x == 0) joins_of(p)[c] = join;
}

template <int CACHE, int D, int NT, int R>
__global__ void __launch_bounds__(Shape<CACHE, D, NT, R>::kThreads, Shape<CACHE, D, NT, R>::kPerSm)
attn_tc(const AttnParams p, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
        const Copies copies, const int stages, const int q_parts, const int w_parts, const unsigned polls)
{
    using S = Shape<CACHE, D, NT, R>;
    using O = Op<CACHE>;
    constexpr bool kF8 = CACHE == GDNA_E4M3;
    constexpr int W = S::kWarps, TW = S::kKeyWarps, ROWS = S::kRows, KB = S::kBlocks;
    constexpr int kParts = 2;              // of the weights; a third follows in a pass of its own
    extern __shared__ uint8_t smem_raw[];
    __shared__ int64_t scratch[S::kThreads / 32 + 3];
    __shared__ float row_scale[ROWS], warp_m[TW][ROWS], warp_l[TW][ROWS];
    __shared__ uint64_t full[kMaxStages][TW], empty[kMaxStages][TW];
    __shared__ int gave_up;
    __shared__ Part queue[kQueue];         // the part in hand and those after it
    __shared__ uint64_t told[kQueue];
    __shared__ Run whole_run;
    __shared__ Join join;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
    uint8_t *smem = smem_raw + (-smem_addr(smem_raw) & 1023u);                 // the swizzle's period
    uint8_t *qs = smem + TW * stages * S::kStage;
    float *sums = reinterpret_cast<float *>(qs + q_parts * ROWS * S::kQPitch); // [TW][ROWS][kSumPitch]
    const bool tensor_copies = copies.keys != 0;

    if (tid == 0) {
        for (int i = 0; i < stages; ++i)
            for (int y = 0; y < TW; ++y) {
                gdn::tc::mbar_init(&full[i][y], tensor_copies ? 1 : 32);
                gdn::tc::mbar_init(&empty[i][y], R);
            }
        for (int i = 0; i < kQueue; ++i) gdn::tc::mbar_init(&told[i], 1);
        gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    gdn::early_start<true>(nullptr, 0);
    Run run = find_run(p, c, scratch);     // (synchronises: the barriers are set up)

    if (warp >= W) {
        const Ring left = produce<CACHE, D, NT, R>(p, run, c, warp - W, blockDim.x / 32 - W, k_map, v_map, copies, stages, polls, smem, full, empty, queue, told);
        if (!left.ok && lane == 0) gave_up = 1;
        __syncthreads();
        if (gave_up) {
            // No copy is left in flight when the block's memory is freed: consumers that kept up have waited for
            // every stage; else what was issued is waited for (again bounded).
            const int mine = warp - W + lane * (blockDim.x / 32 - W), y = mine < TW ? mine : warp - W;
            for (int i = 0; i < left.filled; ++i) {
                // a stage's last fill completes its full barrier's phase with the parity of the next empty wait
                const int at = left.slot - 1 - i;
                gdn::tc::mbar_wait(&full[at < 0 ? at + stages : at][y], at < 0 ? left.phase : left.phase ^ 1,
                                   GDN_DEFAULT_WAIT_POLLS);
            }
            if (warp == W && lane == 0) atomicAdd(&g_wait_timeouts, 1u);
            fill_nan(p, run, c, ROWS);
        }
        return;
    }

    const int tw = warp / R, rg = warp % R;                    // the keys it takes, the rows it takes
    const int l4 = lane >> 2, c4 = lane & 3;
    const unsigned ring = smem_addr(smem) + tw * stages * S::kStage;
    const int group_rows = p.q_len * p.group;
    int slot = 0;
    unsigned phase = 0;
    bool ok = true;                        // every wait so far was in time
    auto all_consumers = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(32 * W) : "memory"); };
    auto all_agree = [&](bool x) {         // the same, and whether x holds for all
        int y;
        asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.s32 a, %1, 0;\n\tbar.red.and.pred b, 1, %2, a;\n\tselp.s32 %0, 1, 0, b;\n\t}"
                     : "=r"(y) : "r"((int)x), "n"(32 * W) : "memory");
        return y != 0;
    };
    Queries<CACHE, D, NT, R> queries;
    {
        Run r = run;
        Part first;
        if (!next_part(p, r, c, first)) first.seq = -1;
        if (tid == 0) {
            queue[0] = first;
            whole_run = run;
            join = Join{0, 0, 0, 0};
        }
    }
    all_consumers();

    for (int turn = 0; queue[turn % kQueue].seq >= 0; ++turn) {
        const Part &part = queue[turn % kQueue];
        const int steps = (int)(part.u1 - part.u0), keys = part.keys;
        for (int pass = 0; pass < queries.kPasses; pass += queries.kGo) {
            queries.fetch(p, part, pass);
            queries.put(p, pass, q_parts, qs, row_scale);
        }
        all_consumers();                   // (and the last part is done with)
        const int row0 = part.item % p.row_tiles * ROWS;

        // this lane's rows: rg * 8 NT + 8 t + 2 c4 + j
        float m[NT][2], l[NT][2], rs[NT][2], o[D / 16][NT][4];
        int seen[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = rg * 8 * NT + 8 * t + 2 * c4 + j;
                m[t][j] = kNegInf;
                l[t][j] = 0.f;
                rs[t][j] = row_scale[r];
                seen[t][j] = keys_seen(p, keys, row0 + r);
            }
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[x][t][j] = 0.f;
        const int all_see = keys - (p.q_len - 1);         // keys that every row sees
        const unsigned q_at = smem_addr(qs + (rg * 8 * NT + (lane & 7)) * S::kQPitch + (lane >> 3) * 16);

        int key0 = (int)((part.u0 * TW + tw) * S::kStep);
#pragma unroll 1
        for (int i = 0; i < steps; ++i) {
            ok = ok && __all_sync(kFull, gdn::tc::mbar_wait(&full[slot][tw], phase, polls));
            const unsigned ks = ring + slot * S::kStage;
            if (ok && key0 < keys) {
                if (key0 + S::kStep > keys) {
                    // past the sequence's end a page holds what it held before: 0 * NaN must not come of it
                    for (int x = lane; x < S::kStep * (S::kRowBytes / 16); x += 32) {
                        const int r = x / (S::kRowBytes / 16), b = x % (S::kRowBytes / 16) * 16;
                        if (key0 + r >= keys)
                            *reinterpret_cast<uint4 *>(smem + (ks - smem_addr(smem)) + (KB + r / kKeys) * S::kBlockBytes +
                                                       S::place(r % kKeys, b)) = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                const unsigned k_at = ks + S::place(lane & 15, (lane >> 4) * 16);

                // S^T: two chains of products a row tile and block
                float s2[KB][2][NT][4];
#pragma unroll
                for (int y = 0; y < KB; ++y)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int j = 0; j < 4; ++j) s2[y][h][t][j] = 0.f;
#pragma unroll 1
                for (int part_i = 0; part_i < q_parts; ++part_i) {
                    const unsigned q_now = q_at + part_i * ROWS * S::kQPitch;
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) {
                        unsigned b[NT][4];
#pragma unroll
                        for (int t = 0; t < NT; ++t) ldsm4(b[t], q_now + 8 * t * S::kQPitch + x * 64);
#pragma unroll
                        for (int y = 0; y < KB; ++y) {
                            unsigned a[2][4];
                            if constexpr (kF8) {
                                unsigned w[4];
                                ldsm4(w, S::across(k_at, x) + y * S::kBlockBytes);
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    widen4(w[2 * h], a[h][0], a[h][2]);
                                    widen4(w[2 * h + 1], a[h][1], a[h][3]);
                                }
                            } else {
                                ldsm4(a[0], S::across(k_at, 2 * x) + y * S::kBlockBytes);
                                ldsm4(a[1], S::across(k_at, 2 * x + 1) + y * S::kBlockBytes);
                            }
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                O::mma(s2[y][0][t], a[0], b[t][0], b[t][1]);
                                O::mma(s2[y][1][t], a[1], b[t][2], b[t][3]);
                            }
                        }
                    }
                }
                // scores in units of log2, what a row does not see replaced
                float w[KB][NT][4];
#pragma unroll
                for (int y = 0; y < KB; ++y)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[y][t][j] = (s2[y][0][t][j] + s2[y][1][t][j]) * rs[t][j & 1];
                const bool edge = key0 + S::kStep > all_see;
                if (edge) {
#pragma unroll
                    for (int y = 0; y < KB; ++y)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (key0 + y * kKeys + l4 + (j >> 1) * 8 >= seen[t][j & 1]) w[y][t][j] = kNegInf;
                }
                bool moved = false;
                float top[NT][2];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float x = fmaxf(w[0][t][j], w[0][t][j + 2]);
#pragma unroll
                        for (int y = 1; y < KB; ++y) x = fmaxf(x, fmaxf(w[y][t][j], w[y][t][j + 2]));
                        x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
                        top[t][j] = fmaxf(x, m[t][j]);
                        moved |= top[t][j] != m[t][j];
                    }
                if (__any_sync(kFull, moved)) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float down[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            down[j] = weight_of(m[t][j], top[t][j]);
                            m[t][j] = top[t][j];
                            l[t][j] *= down[j];
                        }
#pragma unroll
                        for (int x = 0; x < D / 16; ++x)
#pragma unroll
                            for (int j = 0; j < 4; ++j) o[x][t][j] *= down[j & 1];
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float from = m[t][j] == kNegInf ? 0.f : m[t][j];
#pragma unroll
                        for (int y = 0; y < KB; ++y) {
                            w[y][t][j] = O::kLift * ex2(w[y][t][j] - from);
                            w[y][t][j + 2] = O::kLift * ex2(w[y][t][j + 2] - from);
                            l[t][j] += w[y][t][j] + w[y][t][j + 2];
                        }
                    }

                bool plain = true;
                if (edge && p.q_len > 1) { // keys that some rows do not see: is every value finite?
                    bool odd = false;
                    for (int x = lane; x < S::kStep * (S::kRowBytes / 16); x += 32) {
                        unsigned words[4];
                        lds16(words, ks + KB * S::kBlockBytes + x * 16);
                        // an element's all-ones exponent (E4M3: its one NaN) carries into its clear top bit
                        constexpr unsigned kMask = kF8 ? 0x7f7f7f7fu : CACHE == GDNA_F16 ? 0x7c007c00u : 0x7f807f80u;
                        constexpr unsigned kOne = kF8 ? 0x01010101u : CACHE == GDNA_F16 ? 0x04000400u : 0x00800080u;
                        constexpr unsigned kTop = kF8 ? 0x80808080u : 0x80008000u;
#pragma unroll
                        for (int y = 0; y < 4; ++y) odd |= (((words[y] & kMask) + kOne) & kTop) != 0;
                    }
                    plain = !__any_sync(kFull, odd);
                }
                if (plain) {
#pragma unroll
                    for (int y = 0; y < KB; ++y) {
                        const unsigned v_at = ks + (KB + y) * S::kBlockBytes +
                                              (kF8 ? S::place(lane & 15, (lane >> 4) * 16)
                                                   : S::place((lane & 7) + (lane >> 4) * 8, ((lane >> 3) & 1) * 16));
                        float rest[NT][4];
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int j = 0; j < 4; ++j) rest[t][j] = w[y][t][j];
                        auto next_part_of_weights = [&](unsigned (&b)[NT][2]) {
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const unsigned u = O::pack(rest[t][2 * h], rest[t][2 * h + 1]);
                                    const float2 f = O::unpack(u);
                                    rest[t][2 * h] -= f.x;
                                    rest[t][2 * h + 1] -= f.y;
                                    b[t][h] = transpose8(u);
                                }
                        };
                        unsigned b[kParts][NT][2];
#pragma unroll
                        for (int z = 0; z < kParts; ++z) next_part_of_weights(b[z]);
                        // the 16 x 16 blocks of V^T a few at a time: the first part's products of all, then the next's
                        constexpr int kGo = D * NT > 256 ? 2 : 4;              // (registers)
                        auto values = [&](unsigned (&a)[kGo][4], int x0) {
                            if constexpr (kF8) {
#pragma unroll
                                for (int x = 0; x < kGo / 2; ++x) {
                                    unsigned u[4];
                                    ldsm4_trans(u, S::across(v_at, x0 / 2 + x));
#pragma unroll
                                    for (int h = 0; h < 2; ++h) {
                                        // bytes of a word: keys 2c4, 2c4+1 of elements 2 l4, 2 l4 + 1
                                        widen4(__byte_perm(u[2 * h], 0, 0x3120), a[2 * x + h][0], a[2 * x + h][1]);
                                        widen4(__byte_perm(u[2 * h + 1], 0, 0x3120), a[2 * x + h][2], a[2 * x + h][3]);
                                    }
                                }
                            } else {
#pragma unroll
                                for (int x = 0; x < kGo; ++x) ldsm4_trans(a[x], S::across(v_at, x0 + x));
                            }
                        };
#pragma unroll
                        for (int x0 = 0; x0 < D / 16; x0 += kGo) {
                            unsigned a[kGo][4];
                            values(a, x0);
#pragma unroll
                            for (int z = 0; z < kParts; ++z)
#pragma unroll
                                for (int x = 0; x < kGo; ++x)
#pragma unroll
                                    for (int t = 0; t < NT; ++t) O::mma(o[x0 + x][t], a[x], b[z][t][0], b[z][t][1]);
                        }
#pragma unroll 1
                        for (int z = kParts; z < w_parts; ++z) {
                            next_part_of_weights(b[0]);
#pragma unroll
                            for (int x0 = 0; x0 < D / 16; x0 += kGo) {
                                unsigned a[kGo][4];
                                values(a, x0);
#pragma unroll
                                for (int x = 0; x < kGo; ++x)
#pragma unroll
                                    for (int t = 0; t < NT; ++t) O::mma(o[x0 + x][t], a[x], b[0][t][0], b[0][t][1]);
                            }
                        }
                    }
                } else {
                    const uint8_t *vs = smem + (ks - smem_addr(smem)) + KB * S::kBlockBytes;
#pragma unroll
                    for (int y = 0; y < KB; ++y)
#pragma unroll 1
                        for (int k = 0; k < kKeys; ++k) {
                            float wk[NT][2];
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int j = 0; j < 2; ++j)
                                    wk[t][j] = __shfl_sync(kFull, k < 8 ? w[y][t][j] : w[y][t][j + 2], (k & 7) * 4 + c4);
#pragma unroll
                            for (int x = 0; x < D / 16; ++x)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const int e = 16 * x + (kF8 ? 2 * l4 + h : l4 + 8 * h);
                                    const float v = load_elem(vs + y * S::kBlockBytes + S::place(k, e * S::kElem), 0, CACHE);
#pragma unroll
                                    for (int t = 0; t < NT; ++t)
#pragma unroll
                                        for (int j = 0; j < 2; ++j)
                                            if (key0 + y * kKeys + k < seen[t][j])
                                                o[x][t][2 * h + j] = fmaf(wk[t][j], v, o[x][t][2 * h + j]);
                                }
                        }
                }
            }
            key0 += TW * S::kStep;
            __syncwarp();
            if (ok && lane == 0) arrive(&empty[slot][tw]);     // (after a failed wait nothing more may be copied)
            if (++slot == stages) { slot = 0; phase ^= 1; }
        }
        // the part after this one was told (a barrier of `told` completes for every kQueue-th part; the first is not told)
        const int after = (turn + 1) % kQueue;
        ok = ok && __all_sync(kFull, gdn::tc::mbar_wait(&told[after], ((turn + 1) / kQueue - (after == 0)) & 1, polls));

        // add up the key warps' rows, some columns at a time: a task is four columns of a row
        const bool whole = part.begins && part.ends;
        const int head = part.item / p.row_tiles;
        float *to = part_of(p, 2 * c + (part.begins ? 1 : 0));
        constexpr int kQuads = S::kColumns / 4, kAll = ROWS * kQuads, kTasks = (kAll + W * 32 - 1) / (W * 32);
        float share[kTasks][TW], norm[kTasks];
        int64_t out_at[kTasks], gate_at[kTasks];
        bool real[kTasks];
#pragma unroll
        for (int k = 0; k < kTasks; ++k) {
            const int task = tid + k * W * 32, r = task / kQuads, row = row0 + r, token = row / p.group;
            const int64_t r_at = (int64_t)part.seq * p.q_len + token, h_at = (int64_t)head * p.group + (row - token * p.group);
            real[k] = task < kAll && row < group_rows;
            out_at[k] = whole ? r_at * p.out_stride + h_at * p.d + 4 * (task % kQuads) : r * p.d + 4 * (task % kQuads);
            gate_at[k] = r_at * p.gate_stride + h_at * p.gate_head_stride + 4 * (task % kQuads);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float x = l[t][j];
                x += __shfl_xor_sync(kFull, x, 4);
                x += __shfl_xor_sync(kFull, x, 8);
                x += __shfl_xor_sync(kFull, x, 16);
                const int r = rg * 8 * NT + 8 * t + 2 * c4 + j;
                if (l4 == 0) { warp_m[tw][r] = m[t][j]; warp_l[tw][r] = x; }
            }
        // The gates of all columns are asked for at once where they are few registers, so that their latency is paid
        // once an item (111 requests of 5-139 keys, 10/5 heads of 256: 26.4 us against 27.5); else some columns at a time.
        constexpr int kChunks = D / S::kColumns;
        constexpr bool kAtOnce = kTasks * kChunks <= 4;
        uint4 gate[kAtOnce ? kChunks : 1][kTasks];
        auto ask_gates = [&](uint4 (&to)[kTasks], int x0) {
#pragma unroll
            for (int k = 0; k < kTasks; ++k) {
                to[k] = make_uint4(0u, 0u, 0u, 0u);
                if (whole && p.gate != nullptr && real[k] && x0 + 4 * ((tid + k * W * 32) % kQuads) < p.d)
                    to[k] = ask4(p.gate, gate_at[k] + x0, p.dtype, p.gate_vec);
            }
        };
        if constexpr (kAtOnce)
#pragma unroll
            for (int y = 0; y < kChunks; ++y) ask_gates(gate[y], y * S::kColumns);
#pragma unroll
        for (int x0 = 0; x0 < D; x0 += S::kColumns) {
            if (x0 >= p.d) break;
            const int gx = kAtOnce ? x0 / S::kColumns : 0;
            if constexpr (!kAtOnce) ask_gates(gate[0], x0);
            if (x0 > 0) all_consumers();   // the last columns are added up
#pragma unroll
            for (int y = x0 / 16; y < (x0 + S::kColumns) / 16; ++y)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            sums[(tw * ROWS + rg * 8 * NT + 8 * t + 2 * c4 + j) * S::kSumPitch + 16 * y - x0 +
                                 (kF8 ? 2 * l4 + h : l4 + 8 * h)] = o[y][t][2 * h + j];
            if (x0 > 0) all_consumers();
            else ok = all_agree(ok);
            if (!ok) break;
#pragma unroll
            for (int k = 0; k < kTasks; ++k) {
                const int task = tid + k * W * 32, r = task / kQuads;
                if (!real[k]) continue;
                if (x0 == 0) {             // each warp's share of a row
                    float top = kNegInf, total = 0.f;
#pragma unroll
                    for (int y = 0; y < TW; ++y) top = fmaxf(top, warp_m[y][r]);
                    const float from = top == kNegInf ? 0.f : top;
#pragma unroll
                    for (int y = 0; y < TW; ++y) {
                        share[k][y] = weight_of(warp_m[y][r], from) * (1.f / O::kLift);
                        total = fmaf(share[k][y], warp_l[y][r], total);
                    }
                    norm[k] = total == 0.f ? 0.f : p.v_scale / total;
                    if (task % kQuads == 0) {
                        if (!whole) { to[ROWS * p.d + 2 * r] = top; to[ROWS * p.d + 2 * r + 1] = total; }
                        else if (p.lse != nullptr) write_lse(p, part.seq, head, row0 + r, top, total);
                    }
                }
                if (x0 + 4 * (task % kQuads) >= p.d) continue;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int y = 0; y < TW; ++y) {
                    const float4 v = *reinterpret_cast<const float4 *>(sums + (y * ROWS + r) * S::kSumPitch + 4 * (task % kQuads));
                    a.x = fmaf(share[k][y], v.x, a.x);
                    a.y = fmaf(share[k][y], v.y, a.y);
                    a.z = fmaf(share[k][y], v.z, a.z);
                    a.w = fmaf(share[k][y], v.w, a.w);
                }
                if (whole) {
                    finish4(p, a, norm[k], got4(gate[gx][k], p.dtype, p.gate_vec));
                    store4(p.out, out_at[k] + x0, p.out_dtype, p.out_vec, a);
                } else {
                    *reinterpret_cast<float4 *>(to + out_at[k] + x0) = a;
                }
            }
        }
        if (!ok) break;                    // (for all consumers alike)
        if (tid == 0 && part.begins && !part.ends) join = Join{part.seq, part.item, part.blocks, 0};
    }
    if (!ok && tid == 0) gave_up = 1;
    __syncthreads();
    if (gave_up) fill_nan(p, whole_run, c, ROWS);
    else if (tid == 0) joins_of(p)[c] = join;
}

// The map of the cache's K or V: elements of a panel, token, panel, head, page; box: `keys` tokens x all panels of a
// head, which is how they lie in a stage.  Fewer than 16 keys, and a head of several panels that ends within one, come
// panel by panel, the head's elements the first dimension and the panel none: what lies past the head is filled with
// zeros.  False where the encoder refuses the layout.
template <int CACHE, int D, int NT, int R>
bool cache_map(const AttnParams &p, const void *base, const Copies &copies, CUtensorMap *map)
{
    using S = Shape<CACHE, D, NT, R>;
    const auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(gdn::tensor_map_encoder());
    if (encode == nullptr) return false;
    constexpr int kPanelElems = S::kPanel / S::kElem;
    const bool whole = copies.pieces == 1;                     // (its panels are full: `launch`)
    const int64_t strides[4] = {p.cache.token_stride, kPanelElems, p.cache.head_stride, p.cache.page_stride};
    const cuuint64_t size[5] = {(cuuint64_t)(whole ? kPanelElems : p.d), (cuuint64_t)p.cache.page_size,
                                (cuuint64_t)(whole ? p.d / kPanelElems : 1), (cuuint64_t)p.nkv, (cuuint64_t)p.cache.pages};
    const cuuint32_t box[5] = {(cuuint32_t)kPanelElems, (cuuint32_t)copies.keys, (cuuint32_t)(whole ? S::kPanels : 1), 1, 1};
    const cuuint32_t step[5] = {1, 1, 1, 1, 1};
    cuuint64_t stride[4];
    for (int i = 0; i < 4; ++i) {
        const int64_t bytes = strides[i] * S::kElem;
        if (bytes <= 0 || bytes >= (int64_t{1} << 40)) return false;
        stride[i] = (cuuint64_t)bytes;
    }
    return encode(map, S::kElem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 5,
                  const_cast<void *>(base), size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  S::kPanel == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  S::kRowBytes >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CACHE, int D, int NT, int R>
cudaError_t launch(AttnParams p, cudaStream_t s)
{
    using S = Shape<CACHE, D, NT, R>;
    const bool bf16 = CACHE == GDNA_BF16;
    // 16-bit parts of a query: what its type holds (bf16 products have 8 bits a part, fp16 products 11).  An fp32 query over
    // a bf16 cache needs three; two, where nothing but a bf16 output shows it: its scores are then off by up to 2^-17 of
    // sum |q_i k_i| * scale, which moves a weight less than the keys' own 2^-9 did when they were stored.  32 requests, two
    // against three parts: 8 rows of 128 99 against 101 us, 16 rows 61 against 70, 12 rows of 256 74 against 86.
    const bool coarse = p.out_dtype == GDNA_BF16 && p.lse == nullptr;
    const int q_parts = p.dtype == GDNA_BF16 ? 1 : p.dtype == GDNA_F16 ? (bf16 ? 2 : 1) : (bf16 && !coarse ? 3 : 2);
    // and weights: two fp16 parts hold 22 bits (down to 2^-40 of the row's largest), two bf16 parts 16, three 24 for an fp32
    // output
    const int w_parts = bf16 && p.out_dtype == GDNA_F32 ? 3 : 2;
    constexpr int kFixed = 1024 + S::kSumBytes;                // alignment of the ring; the sums
    constexpr int kSmem = S::kSmem;
    static_assert((kSmem - kFixed - 3 * S::kRows * S::kQPitch) / (S::kKeyWarps * S::kStage) >= 2,
                  "two stages whatever the queries' type");
    const int fixed = kFixed + q_parts * S::kRows * S::kQPitch;
    const int room = (kSmem - fixed) / (S::kKeyWarps * S::kStage);
    const int stages = room < kMaxStages ? room : kMaxStages;
    p.unit = S::kStep * S::kKeyWarps;
    // what an item costs beside its keys (queries, adding up, output), in bytes of keys that the block could read
    // meanwhile: measured best at 64 KB for 8 rows of 128, 256 KB for 16 rows of 256
    const int cost = S::kRows * D < 4096 ? S::kRows * D * 64 : 256 * 1024;
    p.lead = cost / (S::kKeyWarps * S::kStage);
    p.page_div = Divisor::of((unsigned)p.cache.page_size);
    p.tile_rows = S::kRows;
    p.row_tiles = (int)(((int64_t)p.q_len * p.group + S::kRows - 1) / S::kRows);
    const int blocks = gdn::sm_count() * S::kPerSm;
    p.grid = blocks < kMaxGrid ? blocks : kMaxGrid;
    CUtensorMap k_map{}, v_map{};
    Copies copies{p.cache.page_size & -p.cache.page_size, S::kPanels};
    if (copies.keys >= kKeys) copies = Copies{kKeys, p.d * S::kElem % S::kPanel == 0 ? 1 : S::kPanels};
    // Producers by the copies of a unit.  D 256, 262144 keys: with 8 copies 165 us by one warp, 167 by two; 64 (pages
    // of a multiple of 8) 278 by one, 172 by two, 173 by four; 128 (of 4) 277 by two, 171 by four.  D 128, 32 requests:
    // with 8 copies 101 by one, 102 by two; 32 107 and 102; cp.async 159 and 105.
    const int lanes = S::kKeyWarps * S::kCopies * (kKeys / copies.keys);
    int producers = lanes * copies.pieces <= 16 ? 1 : lanes * copies.pieces <= 64 ? 2 : 4;
    if (producers > S::kProducers) producers = S::kProducers;
    // a lane for each copy's key (all its pieces); else cp.async.  A head that ends within its only panel as well: tensor
    // copies that fill the rest took 71 us against 67 for 32 requests of bf16 heads of 48, 137 against 133 and 136 against
    // 127 for 256 requests of E4M3 heads of 96 and 80 (and 48 against 54 for bf16 heads of 32, not taken apart).
    if ((S::kPanels == 1 && p.d * S::kElem % S::kPanel != 0) || (S::kKeyWarps + producers - 1) / producers * S::kCopies * (kKeys / copies.keys) > 32 ||
        !cache_map<CACHE, D, NT, R>(p, p.k, copies, &k_map) || !cache_map<CACHE, D, NT, R>(p, p.v, copies, &v_map)) {
        copies = Copies{0, 0};
        producers = S::kPerSm == 2 && S::kProducers == 2 ? 2 : 1;
    }
    cudaError_t e = gdn::allow_dynamic_smem<&attn_tc<CACHE, D, NT, R>>(kSmem);
    if (e != cudaSuccess) return e;
    e = gdn::launch_early(attn_tc<CACHE, D, NT, R>, (unsigned)p.grid, 32 * (S::kWarps + producers), (size_t)(fixed + stages * S::kKeyWarps * S::kStage),
                          s, true, p, k_map, v_map, copies, stages, q_parts, w_parts, gdn::tc_copy_wait_polls());
    return e != cudaSuccess ? e : launch_join(p, s);
}

template <int CACHE, int D>
cudaError_t by_rows(const AttnParams &p, cudaStream_t s)
{
    // Eight rows a warp and as many warps to a ring as the rows need: the kernel is bound by each warp's chain of
    // latencies, and more warps hide it (32 rows of 16 heads on one key head, bf16, D 128: 88 us against 127 with 16 rows
    // a warp).  Sixteen where every warp of a ring would widen the same E4M3 keys again (256 requests, 16 rows, D 128:
    // 153 us against 181), and for more than 32 rows of D <= 128: every warp reads all its ring's keys from shared
    // memory, which eight of them could not do fast enough.
    const int64_t rows = (int64_t)p.q_len * p.group;
    if (rows <= 8) return launch<CACHE, D, 1, 1>(p, s);
    if constexpr (CACHE == GDNA_E4M3 && D <= 128) {
        if (rows <= 16) return launch<CACHE, D, 2, 1>(p, s);
        if (rows <= 32) return launch<CACHE, D, 2, 2>(p, s);
    } else {
        if (rows <= 16) return launch<CACHE, D, 1, 2>(p, s);
        if (rows <= 32) return launch<CACHE, D, 1, 4>(p, s);
    }
    if constexpr (D == 256) return launch<CACHE, D, 1, 8>(p, s);
    else return launch<CACHE, D, 2, 4>(p, s);
}

}  // namespace tc

template <int CACHE> cudaError_t attn_wait_timeouts(unsigned *count)
{
    return cudaMemcpyFromSymbol(count, tc::g_wait_timeouts, sizeof(unsigned));
}

template <int CACHE> cudaError_t launch_attn_tc(const AttnParams &p, cudaStream_t s)
{
    return p.d <= 64 ? tc::by_rows<CACHE, 64>(p, s) : p.d <= 128 ? tc::by_rows<CACHE, 128>(p, s) : tc::by_rows<CACHE, 256>(p, s);
}

}  // namespace gdna

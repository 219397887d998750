// gdna_attn_tc.cuh -- paged decode attention on the tensor cores (head sizes 64,
// 128 and 256): the kernel's template.  gdna_attn.cuh has the deal of the work and
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
// over- or underflows.  The weights exp2(s - m) <= 1 enter in as many parts as put
// their rounding well below the output's (`w_parts`): bf16 products take two (one part's 2^-9
// would be as large as a bf16 output's own), three for an fp32 output; fp16 products one
// (2^-12), two for fp16 and fp32 outputs.  m, l, S and O are fp32.
//
// What a row does not see.  Masked scores are replaced, not added to.  Keys past the
// sequence's end are not loaded (zeros stand for them).  The keys that some tokens see
// and others do not (the last q_len - 1) may hold Inf or NaN values, and 0 * NaN would
// carry them into rows that do not see them: there a tile with a non-finite V adds its
// rows key by key instead.
//
// Data.  A block is one producer warp and W consumer warps, one block an SM.  The
// producer walks the block's parts on its own and keeps the rings full: it is already
// copying the next item's keys while the consumers finish the last one's rows.  Each
// consumer warp (or the R warps that share keys, each with its own rows) has a ring of
// stages in shared memory, a step's K and V each, with a full and an empty mbarrier a
// stage.  Rows lie in panels of 128 bytes with the 128-byte swizzle (64 with the 64-byte
// one), so eight rows of an ldmatrix start in eight different bank groups.
//   Where pages hold a multiple of 16 keys, a block of 16 keys lies in one page and a tensor
// copy brings a panel of it: the (copy, consumer) pairs of a step are one lane each.
// Otherwise the producer's lanes copy 16 bytes at a time (cp.async) to the same layout.
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
// A panel of 16 keys: {x, c1, c2, c3} are the map's coordinates.
__device__ __forceinline__ void copy_panel(unsigned dst, const CUtensorMap *map, int x, int c1, int c2, int c3, unsigned bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4, %5}], [%6];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(c1), "r"(c2), "r"(c3), "r"(bar) : "memory");
}
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

// 16-bit operand type of the products: bf16 for a bf16 cache, else fp16.
template <int CACHE> struct Op {
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

// Two E4M3 values (16 bits) to two fp16, exactly.
__device__ __forceinline__ unsigned widen2(unsigned short x)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(x, __NV_E4M3);
    return (unsigned)h.x | ((unsigned)h.y << 16);
}

template <int CACHE, int D, int NT, int R> struct Shape {
    static constexpr int kElem = CACHE == GDNA_E4M3 ? 1 : 2;
    static constexpr int kRowBytes = D * kElem;                // 64, 128, 256 or 512
    static constexpr int kPanel = kRowBytes < 128 ? kRowBytes : 128;           // bytes of a row in a panel
    static constexpr int kPanels = kRowBytes / kPanel;
    static constexpr int kPanelBytes = kKeys * kPanel;
    static constexpr int kBlockBytes = kKeys * kRowBytes;      // K, or V, of a block
    // Blocks of 16 keys a step.  Short rows take two: the maximum's shuffles, the barriers and the
    // loop are then paid once for 32 keys.
    static constexpr int kBlocks = kRowBytes <= 128 ? 2 : 1;
    static constexpr int kStep = kKeys * kBlocks;
    static constexpr int kStage = 2 * kBlocks * kBlockBytes;   // K's blocks, then V's
    // Consumers: eight, with 168 registers each; four (255 registers) where two row tiles of a large
    // head need them, or where eight rings of such long rows would hold one stage.
    static constexpr int kWarps = (kRowBytes == 512 && R == 1) || (NT == 2 && D >= 128) ? 4 : 8;
    static constexpr int kKeyWarps = kWarps / R;
    static constexpr int kRows = 8 * NT * R;
    static constexpr int kThreads = 32 * (kWarps + 1);
    static constexpr int kCopies = 2 * kBlocks * kPanels;      // tensor copies of a stage
    static constexpr int kQPitch = 2 * D + 16;
    // the consumers' sums are added up some columns at a time
    static constexpr int kColumns = kKeyWarps * kRows <= 64 ? 64 : 32;
    static constexpr int kSumPitch = kColumns + 4;             // floats
    static constexpr int kSumBytes = kKeyWarps * kRows * kSumPitch * 4;
    static constexpr int kMaxStages = 6;
    static_assert(kKeyWarps * kCopies <= 32, "a lane for each copy of a step");

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

// The query rows of an item into shared memory, in 16-bit parts.  Eight elements a lane,
// several rows in flight.  For E4M3 the elements stand in the order in which K's come:
// a 32-bit word of four becomes two operand registers, slots 2q, 2q+1 and 8+2q, 8+2q+1 of
// the 16 that a product contracts.
template <int CACHE, int D, int NT, int R>
__device__ __forceinline__ void load_queries(const AttnParams &p, int seq, int head, int row0, int q_parts, uint8_t *qs,
                                             float *row_scale)
{
    using S = Shape<CACHE, D, NT, R>;
    using O = Op<CACHE>;
    constexpr int ROWS = S::kRows, kLanes = D / 8, kPerWarp = 32 / kLanes;       // lanes of a row, rows of a warp
    constexpr int kPasses = (ROWS + S::kWarps * kPerWarp - 1) / (S::kWarps * kPerWarp), kGo = kPasses < 4 ? kPasses : 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group_rows = p.q_len * p.group;
    const int at = (lane % kLanes) * 8;
#pragma unroll 1
    for (int pass = 0; pass < kPasses; pass += kGo) {
        float x[kGo][8];
#pragma unroll
        for (int k = 0; k < kGo; ++k) {
            const int r = ((pass + k) * S::kWarps + warp) * kPerWarp + lane / kLanes, row = row0 + r;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[k][j] = 0.f;
            if (r < ROWS && row < group_rows) {
                const int token = row / p.group;
                const int64_t from = ((int64_t)seq * p.q_len + token) * p.q_stride +
                                     ((int64_t)head * p.group + (row - token * p.group)) * D + at;
                const float4 a = load4(p.q, from, p.dtype, p.q_vec), b = load4(p.q, from + 4, p.dtype, p.q_vec);
                x[k][0] = a.x; x[k][1] = a.y; x[k][2] = a.z; x[k][3] = a.w;
                x[k][4] = b.x; x[k][5] = b.y; x[k][6] = b.z; x[k][7] = b.w;
            }
        }
#pragma unroll
        for (int k = 0; k < kGo; ++k) {
            const int r = ((pass + k) * S::kWarps + warp) * kPerWarp + lane / kLanes;
            float back = 1.f;
            if constexpr (CACHE != GDNA_BF16) {                // fp16: the row's largest element to 2^14 .. 2^15
                float top = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[k][j]));
#pragma unroll
                for (int off = kLanes / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
                int e = (int)(__float_as_uint(top) >> 23) - 127;
                e = top > 0.f && e < 128 ? max(e, -100) : 14;
                const float up = __uint_as_float((unsigned)(127 + 14 - e) << 23);
                back = __uint_as_float((unsigned)(127 - 14 + e) << 23);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[k][j] *= up;
            }
            if (r < ROWS) {
                for (int part = 0; part < q_parts; ++part) {
                    unsigned u[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        u[j] = O::pack(x[k][2 * j], x[k][2 * j + 1]);
                        const float2 f = O::unpack(u[j]);
                        x[k][2 * j] -= f.x;
                        x[k][2 * j + 1] -= f.y;
                    }
                    uint8_t *to = qs + (part * ROWS + r) * S::kQPitch;
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
}

// How the tensor maps number the cache's dimensions after the elements of a head.
struct MapDims {
    int token, head, page;                 // 1 .. 3
};

// The producer warp: fills the consumers' rings, part after part.
template <int CACHE, int D, int NT, int R>
__device__ __forceinline__ void produce(const AttnParams &p, Run run, int c, const CUtensorMap &k_map, const CUtensorMap &v_map,
                                        const MapDims dims, int stages, unsigned polls, uint8_t *smem,
                                        uint64_t (*full)[Shape<CACHE, D, NT, R>::kKeyWarps],
                                        uint64_t (*empty)[Shape<CACHE, D, NT, R>::kKeyWarps], int *gave_up)
{
    using S = Shape<CACHE, D, NT, R>;
    constexpr int TW = S::kKeyWarps, KB = S::kBlocks;
    const int lane = threadIdx.x & 31;
    const unsigned page_size = (unsigned)p.cache.page_size, ring = smem_addr(smem);
    int slot = 0, filled = 0;              // the next stage; stages filled so far, at most `stages`
    unsigned phase = 1;                    // of its empty barrier: the first round finds all of them empty
    bool ok = true;

    if (dims.page != 0) {
        // lane: the consumer it copies for, and which panel of which block of K or V
        const int y = lane / S::kCopies, copy = lane % S::kCopies;
        const bool mine = y < TW;
        const int panel = copy % S::kPanels, block = copy / S::kPanels % KB, values = copy / (S::kPanels * KB);
        const unsigned dst = ring + (mine ? y : 0) * stages * S::kStage + (values * KB + block) * S::kBlockBytes +
                             panel * S::kPanelBytes;
        const CUtensorMap *map = values ? &v_map : &k_map;
        while (ok && run.at < run.end) {
            const Part part = next_part(p, run, c);
            const int head = part.item / p.row_tiles, steps = (int)(part.u1 - part.u0);
            const int32_t *table = p.table + part.seq * p.table_stride;
            unsigned key = (unsigned)((part.u0 * TW + y) * S::kStep + block * kKeys);
            auto look_up = [&](int i) {    // the page of this lane's block; past the cache (zeros) if there is none
                int page = i < steps && mine && key < (unsigned)part.keys ? __ldg(table + p.page_div.quotient(key)) : -1;
                return (unsigned)page < (unsigned)p.cache.pages ? page : (int)p.cache.pages;
            };
            int page = look_up(0);
            for (int i = 0; i < steps; ++i) {
                const int token = (int)(key - p.page_div.quotient(min(key, 0x7fffffffu)) * page_size), at = page;
                key += TW * S::kStep;
                page = look_up(i + 1);
                ok = __all_sync(kFull, !mine || gdn::tc::mbar_wait(&empty[slot][mine ? y : 0], phase, polls));
                if (!ok) break;
                if (mine && copy == 0) arrive_expect(&full[slot][y], S::kStage);
                __syncwarp();
                if (mine) {
                    const int c1 = dims.token == 1 ? token : dims.head == 1 ? head : at;
                    const int c2 = dims.token == 2 ? token : dims.head == 2 ? head : at;
                    const int c3 = dims.token == 3 ? token : dims.head == 3 ? head : at;
                    copy_panel(dst + slot * S::kStage, map, panel * (S::kPanel / S::kElem), c1, c2, c3, smem_addr(&full[slot][y]));
                }
                filled = min(filled + 1, stages);
                if (++slot == stages) { slot = 0; phase ^= 1; }
            }
        }
    } else {
        const int64_t page_bytes = p.cache.page_stride * S::kElem, token_bytes = p.cache.token_stride * S::kElem;
        constexpr int kPieces = S::kRowBytes / 16, kAtOnce = 32 / kPieces;     // 16-byte pieces of a row, rows at once
        const int sub = lane / kPieces, piece = lane % kPieces * 16;
        while (ok && run.at < run.end) {
            const Part part = next_part(p, run, c);
            const int head = part.item / p.row_tiles, steps = (int)(part.u1 - part.u0);
            const int32_t *table = p.table + part.seq * p.table_stride;
            const uint8_t *kb = static_cast<const uint8_t *>(p.k) + head * p.cache.head_stride * S::kElem;
            const uint8_t *vb = static_cast<const uint8_t *>(p.v) + head * p.cache.head_stride * S::kElem;
            unsigned key = (unsigned)(part.u0 * TW) * S::kStep + lane % S::kStep;      // the one this lane looks up
            auto look_up = [&](int i) {
                return i < steps && key < (unsigned)part.keys ? __ldg(table + p.page_div.quotient(key)) : -1;
            };
            int page = look_up(0);
            for (int i = 0; i < steps; ++i) {
                for (int y = 0; y < TW && ok; ++y) {
                    int64_t at = -1;
                    if ((unsigned)page < (unsigned)p.cache.pages)
                        at = page * page_bytes + (int64_t)(key - p.page_div.quotient(key) * page_size) * token_bytes;
                    key += S::kStep;
                    page = look_up(y + 1 < TW ? i : i + 1);
                    ok = __all_sync(kFull, gdn::tc::mbar_wait(&empty[slot][y], phase, polls));
                    if (!ok) break;
                    const unsigned to = ring + (y * stages + slot) * S::kStage;
#pragma unroll 4
                    for (int r = 0; r < S::kStep; r += kAtOnce) {
                        const int row = r + sub;
                        const int64_t from = __shfl_sync(kFull, at, row);
                        const unsigned dst = to + row / kKeys * S::kBlockBytes + S::place(row % kKeys, piece);
                        cp_async16(dst, kb + (from >= 0 ? from + piece : 0), from >= 0);
                        cp_async16(dst + KB * S::kBlockBytes, vb + (from >= 0 ? from + piece : 0), from >= 0);
                    }
                    arrive_copies(&full[slot][y]);
                }
                if (!ok) break;
                if (++slot == stages) { slot = 0; phase ^= 1; }
            }
        }
        gdn::cp_async_wait<0>();
    }
    // No copy is left in flight when the block's memory is freed: consumers that kept up have waited for
    // every stage; where a wait gave up, here or there, what was issued is waited for (again bounded).
    __syncthreads();
    if (!ok || *(volatile int *)gave_up != 0) {
        const int y = lane < TW ? lane : 0;
        for (int i = 0; i < filled; ++i) {
            // a stage's last fill completes its full barrier's phase with the parity of the next empty wait
            const int at = slot - 1 - i;
            gdn::tc::mbar_wait(&full[at < 0 ? at + stages : at][y], at < 0 ? phase : phase ^ 1, GDN_DEFAULT_WAIT_POLLS);
        }
        if (lane == 0) atomicAdd(&g_wait_timeouts, 1u);
    }
}

template <int CACHE, int D, int NT, int R>
__global__ void __launch_bounds__(Shape<CACHE, D, NT, R>::kThreads, 1)
attn_tc(const AttnParams p, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
        const MapDims dims, const int stages, const int q_parts, const int w_parts, const unsigned polls)
{
    using S = Shape<CACHE, D, NT, R>;
    using O = Op<CACHE>;
    constexpr bool kF8 = CACHE == GDNA_E4M3;
    constexpr int W = S::kWarps, TW = S::kKeyWarps, ROWS = S::kRows, KB = S::kBlocks;
    // weight parts of the products proper; more follow in passes of their own
    constexpr int kParts = kF8 ? 1 : 2;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int64_t scratch[W + 3];
    __shared__ float row_scale[ROWS], warp_m[TW][ROWS], warp_l[TW][ROWS];
    __shared__ uint64_t full[S::kMaxStages][TW], empty[S::kMaxStages][TW];
    __shared__ int gave_up;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
    uint8_t *smem = smem_raw + (-smem_addr(smem_raw) & 1023u);                 // the swizzle's period
    uint8_t *qs = smem + TW * stages * S::kStage;
    float *sums = reinterpret_cast<float *>(qs + q_parts * ROWS * S::kQPitch); // [TW][ROWS][kSumPitch]
    const bool tensor_copies = dims.page != 0;

    if (tid == 0) {
        for (int i = 0; i < stages; ++i)
            for (int y = 0; y < TW; ++y) {
                gdn::tc::mbar_init(&full[i][y], tensor_copies ? 1 : 32);
                gdn::tc::mbar_init(&empty[i][y], R);
            }
        gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    gdn::early_start<true>(nullptr, 0);
    Run run = find_run(p, c, scratch);     // (synchronises: the barriers are set up)

    if (warp == W) {
        produce<CACHE, D, NT, R>(p, run, c, k_map, v_map, dims, stages, polls, smem, full, empty, &gave_up);
        return;
    }

    const int tw = warp / R, rg = warp % R;                    // the keys it takes, the rows it takes
    const int l4 = lane >> 2, c4 = lane & 3;
    const unsigned ring = smem_addr(smem) + tw * stages * S::kStage;
    const int group_rows = p.q_len * p.group;
    int slot = 0;
    unsigned phase = 0;
    bool ok = true;                        // every wait so far was in time
    Join join = {0, 0, 0, 0};
    auto all_consumers = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(32 * W) : "memory"); };

    while (run.at < run.end) {
        const Part part = next_part(p, run, c);
        const int head = part.item / p.row_tiles, row0 = (part.item % p.row_tiles) * ROWS;
        const int steps = (int)(part.u1 - part.u0);
        load_queries<CACHE, D, NT, R>(p, part.seq, head, row0, q_parts, qs, row_scale);
        all_consumers();

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
                seen[t][j] = keys_seen(p, part.keys, row0 + r);
            }
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[x][t][j] = 0.f;
        const int all_see = part.keys - (p.q_len - 1);         // keys that every row sees
        const unsigned q_at = smem_addr(qs + (rg * 8 * NT + (lane & 7)) * S::kQPitch + (lane >> 3) * 16);

        int key0 = (int)((part.u0 * TW + tw) * S::kStep);
#pragma unroll 1
        for (int i = 0; i < steps; ++i) {
            ok = ok && __all_sync(kFull, gdn::tc::mbar_wait(&full[slot][tw], phase, polls));
            const unsigned ks = ring + slot * S::kStage;
            if (ok && key0 < part.keys) {
                if (key0 + S::kStep > part.keys) {
                    // past the sequence's end a page holds what it held before: 0 * NaN must not come of it
                    for (int x = lane; x < S::kStep * (S::kRowBytes / 16); x += 32) {
                        const int r = x / (S::kRowBytes / 16), b = x % (S::kRowBytes / 16) * 16;
                        if (key0 + r >= part.keys)
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
                                    a[h][0] = widen2((unsigned short)w[2 * h]);
                                    a[h][1] = widen2((unsigned short)w[2 * h + 1]);
                                    a[h][2] = widen2((unsigned short)(w[2 * h] >> 16));
                                    a[h][3] = widen2((unsigned short)(w[2 * h + 1] >> 16));
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
                            w[y][t][j] = ex2(w[y][t][j] - from);
                            w[y][t][j + 2] = ex2(w[y][t][j + 2] - from);
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
                                        const unsigned e0 = __byte_perm(u[2 * h], 0, 0x3120), e1 = __byte_perm(u[2 * h + 1], 0, 0x3120);
                                        a[2 * x + h][0] = widen2((unsigned short)e0);
                                        a[2 * x + h][1] = widen2((unsigned short)(e0 >> 16));
                                        a[2 * x + h][2] = widen2((unsigned short)e1);
                                        a[2 * x + h][3] = widen2((unsigned short)(e1 >> 16));
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
        if (!ok) {                         // copies that never came: the rows come out NaN
#pragma unroll
            for (int t = 0; t < NT; ++t) l[t][0] = l[t][1] = __int_as_float(0x7fc00000);
            if (lane == 0) atomicExch(&gave_up, 1);
        }

        // add up the key warps' rows, some columns at a time
        const bool whole = part.begins && part.ends;
        float *to = part_of(p, 2 * c + (part.begins ? 1 : 0));
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
        constexpr int kQuads = S::kColumns / 4, kAll = ROWS * kQuads, kTasks = (kAll + W * 32 - 1) / (W * 32);
        float4 gate[kTasks];
        auto load_gates = [&](int x0) {
#pragma unroll
            for (int k = 0; k < kTasks; ++k) {
                const int task = tid + k * W * 32, row = row0 + task / kQuads;
                if (whole && p.gate != nullptr && task < kAll && row < group_rows) {
                    const int token = row / p.group;
                    gate[k] = load4(p.gate, ((int64_t)part.seq * p.q_len + token) * p.gate_stride +
                                                ((int64_t)head * p.group + (row - token * p.group)) * p.gate_head_stride +
                                                x0 + 4 * (task % kQuads), p.dtype, p.gate_vec);
                }
            }
        };
        load_gates(0);
#pragma unroll
        for (int x0 = 0; x0 < D; x0 += S::kColumns) {
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
            all_consumers();
#pragma unroll
            for (int k = 0; k < kTasks; ++k) {
                const int task = tid + k * W * 32, r = task / kQuads, x = 4 * (task % kQuads);
                if (task >= kAll || row0 + r >= group_rows) continue;
                float top = kNegInf, total = 0.f;
#pragma unroll
                for (int y = 0; y < TW; ++y) top = fmaxf(top, warp_m[y][r]);
                const float mm = top;
                if (top == kNegInf) top = 0.f;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int y = 0; y < TW; ++y) {
                    const float share = weight_of(warp_m[y][r], top);
                    total = fmaf(share, warp_l[y][r], total);
                    const float4 v = *reinterpret_cast<const float4 *>(sums + (y * ROWS + r) * S::kSumPitch + x);
                    a.x = fmaf(share, v.x, a.x);
                    a.y = fmaf(share, v.y, a.y);
                    a.z = fmaf(share, v.z, a.z);
                    a.w = fmaf(share, v.w, a.w);
                }
                if (whole) {
                    const int token = (row0 + r) / p.group;
                    const int64_t r_at = (int64_t)part.seq * p.q_len + token;
                    const int64_t h_at = (int64_t)head * p.group + (row0 + r - token * p.group);
                    finish4(p, a, total, gate[k]);
                    store4(p.out, r_at * p.out_stride + h_at * D + x0 + x, p.out_dtype, p.out_vec, a);
                    if (x0 + x == 0 && p.lse != nullptr) p.lse[r_at * p.nq + h_at] = lse_of(mm, total);
                } else {
                    *reinterpret_cast<float4 *>(to + r * D + x0 + x) = a;
                    if (x0 + x == 0) { to[ROWS * D + 2 * r] = mm; to[ROWS * D + 2 * r + 1] = total; }
                }
            }
            if (x0 + S::kColumns < D) load_gates(x0 + S::kColumns);
            all_consumers();
        }
        if (part.begins && !part.ends) join = Join{part.seq, part.item, part.blocks, 0};
    }
    if (tid == 0) joins_of(p)[c] = join;
    __syncthreads();                       // (the producer looks whether all waits were in time)
}

constexpr int kSmemBytes = 224 * 1024;     // of a block, beside its static arrays

// The 4-D map of the cache's K or V: the elements of a head, then (token, head, page) in the order of
// their strides; box: 16 tokens x a panel.  False where the layout does not allow it.
template <int CACHE, int D, int NT, int R>
bool cache_map(const AttnParams &p, const void *base, CUtensorMap *map, MapDims *dims)
{
    using S = Shape<CACHE, D, NT, R>;
    const auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(gdn::tensor_map_encoder());
    if (encode == nullptr) return false;
    struct Dim { int64_t stride, count; int box, *number; } d[3] = {
        {p.cache.token_stride, p.cache.page_size, kKeys, &dims->token},
        {p.cache.head_stride, p.nkv, 1, &dims->head},
        {p.cache.page_stride, p.cache.pages, 1, &dims->page}};
    std::sort(d, d + 3, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
    cuuint64_t size[4] = {(cuuint64_t)D}, stride[3];
    cuuint32_t box[4] = {(cuuint32_t)(S::kPanel / S::kElem)};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    for (int i = 0; i < 3; ++i) {
        const int64_t bytes = d[i].stride * S::kElem;
        if (bytes <= 0 || bytes >= (int64_t{1} << 40)) return false;
        size[i + 1] = (cuuint64_t)d[i].count;
        stride[i] = (cuuint64_t)bytes;
        box[i + 1] = (cuuint32_t)d[i].box;
        *d[i].number = i + 1;
    }
    return encode(map, S::kElem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4,
                  const_cast<void *>(base), size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  S::kPanel == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CACHE, int D, int NT, int R>
cudaError_t launch(AttnParams p, cudaStream_t s)
{
    using S = Shape<CACHE, D, NT, R>;
    const bool bf16 = CACHE == GDNA_BF16;
    // 16-bit parts that hold a query of its type: bf16 products have 8 bits a part, fp16 products 11
    const int q_parts = p.dtype == GDNA_BF16 ? 1 : p.dtype == GDNA_F16 ? (bf16 ? 2 : 1) : (bf16 ? 3 : 2);
    // and weights: to well below the output's rounding
    const int w_parts = (bf16 ? 2 : 1) + (p.out_dtype == GDNA_F32 || (CACHE != GDNA_BF16 && p.out_dtype == GDNA_F16));
    constexpr int kFixed = 1024 + S::kSumBytes;                // alignment of the ring; the sums
    static_assert((kSmemBytes - kFixed - 3 * S::kRows * S::kQPitch) / (S::kKeyWarps * S::kStage) >= 2,
                  "two stages whatever the queries' type");
    const int fixed = kFixed + q_parts * S::kRows * S::kQPitch;
    const int room = (kSmemBytes - fixed) / (S::kKeyWarps * S::kStage);
    const int stages = room < S::kMaxStages ? room : S::kMaxStages;
    p.unit = S::kStep * S::kKeyWarps;
    p.page_div = Divisor::of((unsigned)p.cache.page_size);
    p.tile_rows = S::kRows;
    p.row_tiles = (int)(((int64_t)p.q_len * p.group + S::kRows - 1) / S::kRows);
    const int sms = gdn::sm_count();
    p.grid = sms < kMaxGrid ? sms : kMaxGrid;
    CUtensorMap k_map{}, v_map{};
    MapDims dims{};
    if (p.cache.page_size % kKeys != 0 || !cache_map<CACHE, D, NT, R>(p, p.k, &k_map, &dims) ||
        !cache_map<CACHE, D, NT, R>(p, p.v, &v_map, &dims))
        dims = MapDims{0, 0, 0};
    cudaError_t e = gdn::allow_dynamic_smem<&attn_tc<CACHE, D, NT, R>>(kSmemBytes);
    if (e != cudaSuccess) return e;
    e = gdn::launch_early(attn_tc<CACHE, D, NT, R>, (unsigned)p.grid, S::kThreads, (size_t)(fixed + stages * S::kKeyWarps * S::kStage),
                          s, true, p, k_map, v_map, dims, stages, q_parts, w_parts, gdn::tc_copy_wait_polls());
    return e != cudaSuccess ? e : launch_join(p, s);
}

template <int CACHE, int D>
cudaError_t by_rows(const AttnParams &p, cudaStream_t s)
{
    const int64_t rows = (int64_t)p.q_len * p.group;
    if (rows <= 8) return launch<CACHE, D, 1, 1>(p, s);
    if (rows <= 16) return launch<CACHE, D, 1, 2>(p, s);
    if (rows <= 32) return launch<CACHE, D, 2, 2>(p, s);
    return launch<CACHE, D, 2, 4>(p, s);
}

}  // namespace tc

template <int CACHE> cudaError_t attn_wait_timeouts(unsigned *count)
{
    return cudaMemcpyFromSymbol(count, tc::g_wait_timeouts, sizeof(unsigned));
}

template <int CACHE> cudaError_t launch_attn_tc(const AttnParams &p, cudaStream_t s)
{
    return p.d == 64 ? tc::by_rows<CACHE, 64>(p, s) : p.d == 128 ? tc::by_rows<CACHE, 128>(p, s) : tc::by_rows<CACHE, 256>(p, s);
}

}  // namespace gdna

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
// Data.  A warp (or the R warps that share keys, each with its own rows) has its own
// ring of stages in shared memory, 16 keys of K and V each, filled by cp.async in
// 16-byte pieces (a key's head is D contiguous elements; keys lie anywhere) and drained
// without any barrier over the block.  Rows are padded by 16 bytes: eight rows of an
// ldmatrix then start in eight different bank groups.
#pragma once

#include "gdna_attn.cuh"

namespace gdna {
namespace tc {

constexpr int kKeys = 16;                  // keys of a block: one side of a product
constexpr int kMaxStages = 8;
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
// All but the newest `stages - 2` copy groups have landed.
__device__ __forceinline__ void wait_stage(int stages)
{
    switch (stages) {
    case 2: gdn::cp_async_wait<0>(); break;
    case 3: gdn::cp_async_wait<1>(); break;
    case 4: gdn::cp_async_wait<2>(); break;
    case 5: gdn::cp_async_wait<3>(); break;
    case 6: gdn::cp_async_wait<4>(); break;
    case 7: gdn::cp_async_wait<5>(); break;
    default: gdn::cp_async_wait<6>(); break;
    }
}

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
    static constexpr int kRowBytes = D * kElem;
    static constexpr int kPitch = kRowBytes + 16;
    // Blocks of 16 keys a step.  Short rows take two: the maximum's shuffles, the barrier and the
    // addresses are then paid once for 32 keys.
    static constexpr int kBlocks = kRowBytes <= 128 ? 2 : 1;
    static constexpr int kStep = kKeys * kBlocks;
    static constexpr int kStage = 2 * kStep * kPitch;          // K, then V
    static constexpr int kWarps = (kRowBytes == 512 && R == 1) ? 2 : 4;
    static constexpr int kKeyWarps = kWarps / R;
    static constexpr int kRows = 8 * NT * R;
    static constexpr int kQPitch = 2 * D + 16;
    static constexpr int kSumPitch = D + 4;                    // floats
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

template <int CACHE, int D, int NT, int R>
__global__ void __launch_bounds__(Shape<CACHE, D, NT, R>::kWarps * 32, 2)
attn_tc(const AttnParams p, const int stages, const int q_parts, const int w_parts)
{
    using S = Shape<CACHE, D, NT, R>;
    using O = Op<CACHE>;
    constexpr bool kF8 = CACHE == GDNA_E4M3;
    constexpr int W = S::kWarps, TW = S::kKeyWarps, ROWS = S::kRows, KB = S::kBlocks;
    // weight parts of the products proper; more follow in passes of their own
    constexpr int kParts = kF8 ? 1 : 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t scratch[W + 2];
    __shared__ float row_scale[ROWS], warp_m[TW][ROWS], warp_l[TW][ROWS];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
    const int tw = warp / R, rg = warp % R;                    // the keys it takes, the rows it takes
    const int l4 = lane >> 2, c4 = lane & 3;
    const unsigned ring = smem_addr(smem) + tw * stages * S::kStage, ring_end = ring + stages * S::kStage;
    uint8_t *qs = smem + TW * stages * S::kStage;
    float *sums = reinterpret_cast<float *>(smem);             // after the keys: [TW][ROWS][kSumPitch]
    const int group_rows = p.q_len * p.group;
    const unsigned page_size = (unsigned)p.cache.page_size;
    const bool in_page = page_size % kKeys == 0;               // a block of keys lies in one page
    const int64_t page_bytes = p.cache.page_stride * S::kElem, token_bytes = p.cache.token_stride * S::kElem;

    gdn::early_start<true>(nullptr, 0);
    Run run = find_run(p, c, scratch);
    Join join = {0, 0, 0, 0};

    while (run.at < run.end) {
        const Part part = next_part(p, run, c);
        const int head = part.item / p.row_tiles, row0 = (part.item % p.row_tiles) * ROWS;
        const int steps = (int)(part.u1 - part.u0);
        const unsigned keys = (unsigned)part.keys;
        const int32_t *table = p.table + part.seq * p.table_stride;
        const uint8_t *kb = static_cast<const uint8_t *>(p.k) + head * p.cache.head_stride * S::kElem;
        const uint8_t *vb = static_cast<const uint8_t *>(p.v) + head * p.cache.head_stride * S::kElem;
        __syncthreads();                   // the last part's sums and queries are used up

        // Lane j looks up the page of key j of a step, a step before it is needed; -1: none.
        const unsigned start = (unsigned)(part.u0 * TW + tw) * S::kStep;       // this warp's first key
        unsigned look = start + lane % S::kStep;                               // the key to look up next
        int ahead = 0;                                                         // its step
        auto next_page = [&]() {
            const int page = ahead < steps && look < keys ? __ldg(table + p.page_div.quotient(look)) : -1;
            ++ahead;
            look += TW * S::kStep;
            return page;
        };
        unsigned fill = start, fill_at = ring;                                 // the next step to copy: key, stage
        auto issue = [&](int page) {
            constexpr int kPieces = S::kRowBytes / 16;         // 16-byte pieces of a row: 4 .. 32
            constexpr int kAtOnce = 32 / kPieces;              // rows of one instruction
            constexpr int kMine = S::kStep / R;                // rows this warp copies
            static_assert(kAtOnce <= kMine && (kMine % kKeys == 0 || kKeys % kMine == 0), "whole instructions");
            const int sub = lane / kPieces, piece = (lane % kPieces) * 16;
            const unsigned dst = fill_at + (rg * kMine + sub) * S::kPitch + piece;
            const unsigned mine = fill + lane % S::kStep;
            const unsigned place = mine - p.page_div.quotient(mine) * page_size;          // in its page
            const int64_t at = (unsigned)page < (unsigned)p.cache.pages
                                   ? page * page_bytes + (int64_t)place * token_bytes : -1;
            if (in_page) {
#pragma unroll
                for (int r0 = 0; r0 < kMine; r0 += kKeys) {    // a block: one address, then equal steps
                    const int first = (rg * kMine + r0) / kKeys * kKeys, off = (rg * kMine + r0) % kKeys + sub;
                    const int64_t block = __shfl_sync(kFull, at, first);
                    int64_t from = block + off * token_bytes + piece;
                    const int left = block >= 0 ? (int)(keys - fill) - first - off : 0;
#pragma unroll
                    for (int r = 0; r < kKeys && r < kMine; r += kAtOnce) {
                        const bool on = r < left;
                        cp_async16(dst + (r0 + r) * S::kPitch, kb + (on ? from : 0), on);
                        cp_async16(dst + (S::kStep + r0 + r) * S::kPitch, vb + (on ? from : 0), on);
                        from += kAtOnce * token_bytes;
                    }
                }
            } else {
#pragma unroll
                for (int r = 0; r < kMine; r += kAtOnce) {
                    const int64_t from = __shfl_sync(kFull, at, rg * kMine + r + sub);
                    const bool on = from >= 0;
                    cp_async16(dst + r * S::kPitch, kb + (on ? from + piece : 0), on);
                    cp_async16(dst + (S::kStep + r) * S::kPitch, vb + (on ? from + piece : 0), on);
                }
            }
            fill += TW * S::kStep;
            fill_at += S::kStage;
            if (fill_at == ring_end) fill_at = ring;
        };
        int page = next_page();
        for (int i = 0; i < stages - 1; ++i) {
            const int next = next_page();
            if (i < steps) issue(page);
            gdn::cp_async_commit();
            page = next;
        }
        load_queries<CACHE, D, NT, R>(p, part.seq, head, row0, q_parts, qs, row_scale);
        __syncthreads();

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

        unsigned ks = ring;                                    // the step's stage
        int key0 = (int)start;
#pragma unroll 1
        for (int i = 0; i < steps; ++i) {
            wait_stage(stages);
            if constexpr (R == 1) __syncwarp();
            else asm volatile("bar.sync %0, %1;" ::"r"(1 + tw), "n"(32 * R) : "memory");
            // the stage that was used up a step ago takes the keys of stages - 1 steps ahead
            {
                const int next = next_page();
                if (i + stages - 1 < steps) issue(page);
                gdn::cp_async_commit();
                page = next;
            }
            if (key0 < part.keys) {
                const unsigned k_at = ks + (lane & 15) * S::kPitch + (lane >> 4) * 16;

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
                                ldsm4(w, k_at + y * kKeys * S::kPitch + x * 32);
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    a[h][0] = widen2((unsigned short)w[2 * h]);
                                    a[h][1] = widen2((unsigned short)w[2 * h + 1]);
                                    a[h][2] = widen2((unsigned short)(w[2 * h] >> 16));
                                    a[h][3] = widen2((unsigned short)(w[2 * h + 1] >> 16));
                                }
                            } else {
                                ldsm4(a[0], k_at + y * kKeys * S::kPitch + x * 64);
                                ldsm4(a[1], k_at + y * kKeys * S::kPitch + x * 64 + 32);
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
                    constexpr int kPieces = S::kRowBytes / 16;
                    bool odd = false;
                    for (int x = lane; x < S::kStep * kPieces; x += 32) {
                        unsigned words[4];
                        lds16(words, ks + (S::kStep + x / kPieces) * S::kPitch + x % kPieces * 16);
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
                        const unsigned vs = ks + (S::kStep + y * kKeys) * S::kPitch;
                        const unsigned v_at = kF8 ? vs + (lane & 15) * S::kPitch + (lane >> 4) * 16
                                                  : vs + ((lane & 7) + (lane >> 4) * 8) * S::kPitch + ((lane >> 3) & 1) * 16;
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
                                    ldsm4_trans(u, v_at + (x0 / 2 + x) * 32);
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
                                for (int x = 0; x < kGo; ++x) ldsm4_trans(a[x], v_at + (x0 + x) * 32);
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
                    const uint8_t *vs = smem + (ks - smem_addr(smem)) + S::kStep * S::kPitch;
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
                                    const float v = load_elem(vs + (y * kKeys + k) * S::kPitch, e, CACHE);
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
            ks += S::kStage;
            if (ks == ring_end) ks = ring;
        }

        // join the key warps' rows in shared memory, over the ring
        gdn::cp_async_wait<0>();
        __syncthreads();
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
#pragma unroll
                for (int y = 0; y < D / 16; ++y)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        sums[(tw * ROWS + r) * S::kSumPitch + 16 * y + (kF8 ? 2 * l4 + h : l4 + 8 * h)] = o[y][t][2 * h + j];
            }
        __syncthreads();
        const bool whole = part.begins && part.ends;
        float *to = part_of(p, 2 * c + (part.begins ? 1 : 0));
        constexpr int kQuads = D / 4, kTasks = ROWS * kQuads / (W * 32), kGo = kTasks < 4 ? kTasks : 4;
#pragma unroll 1
        for (int k0 = 0; k0 < kTasks; k0 += kGo) {
            float4 gate[kGo];
            int64_t r_at[kGo], h_at[kGo];
#pragma unroll
            for (int k = 0; k < kGo; ++k) {                    // every gate in flight
                const int task = tid + (k0 + k) * W * 32, row = row0 + task / kQuads;
                const int token = row / p.group;
                r_at[k] = (int64_t)part.seq * p.q_len + token;
                h_at[k] = (int64_t)head * p.group + (row - token * p.group);
                gate[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (whole && p.gate != nullptr && row < group_rows)
                    gate[k] = load4(p.gate, r_at[k] * p.gate_stride + h_at[k] * p.gate_head_stride + 4 * (task % kQuads),
                                    p.dtype, p.gate_vec);
            }
#pragma unroll
            for (int k = 0; k < kGo; ++k) {
                const int task = tid + (k0 + k) * W * 32, r = task / kQuads, x = 4 * (task % kQuads);
                if (row0 + r >= group_rows) continue;
                float top = kNegInf, total = 0.f, share[TW];
#pragma unroll
                for (int y = 0; y < TW; ++y) top = fmaxf(top, warp_m[y][r]);
                const float mm = top;
                if (top == kNegInf) top = 0.f;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int y = 0; y < TW; ++y) {
                    share[y] = weight_of(warp_m[y][r], top);
                    total = fmaf(share[y], warp_l[y][r], total);
                    const float4 v = *reinterpret_cast<const float4 *>(sums + (y * ROWS + r) * S::kSumPitch + x);
                    a.x = fmaf(share[y], v.x, a.x);
                    a.y = fmaf(share[y], v.y, a.y);
                    a.z = fmaf(share[y], v.z, a.z);
                    a.w = fmaf(share[y], v.w, a.w);
                }
                if (whole) {
                    finish4(p, a, total, gate[k]);
                    store4(p.out, r_at[k] * p.out_stride + h_at[k] * D + x, p.out_dtype, p.out_vec, a);
                    if (x == 0 && p.lse != nullptr) p.lse[r_at[k] * p.nq + h_at[k]] = lse_of(mm, total);
                } else {
                    *reinterpret_cast<float4 *>(to + r * D + x) = a;
                    if (x == 0) { to[ROWS * D + 2 * r] = mm; to[ROWS * D + 2 * r + 1] = total; }
                }
            }
        }
        if (part.begins && !part.ends) join = Join{part.seq, part.item, part.blocks, 0};
    }
    if (tid == 0) joins_of(p)[c] = join;
}

constexpr int kTwoPerSm = 111 * 1024;      // shared memory of a block of which two fit an SM
constexpr int kOnePerSm = 224 * 1024;

template <int CACHE, int D, int NT, int R>
cudaError_t launch(AttnParams p, cudaStream_t s)
{
    using S = Shape<CACHE, D, NT, R>;
    const bool bf16 = CACHE == GDNA_BF16;
    // 16-bit parts that hold a query of its type: bf16 products have 8 bits a part, fp16 products 11
    const int q_parts = p.dtype == GDNA_BF16 ? 1 : p.dtype == GDNA_F16 ? (bf16 ? 2 : 1) : (bf16 ? 3 : 2);
    // and weights: to well below the output's rounding
    const int w_parts = (bf16 ? 2 : 1) + (p.out_dtype == GDNA_F32 || (CACHE != GDNA_BF16 && p.out_dtype == GDNA_F16));
    const int q_bytes = q_parts * S::kRows * S::kQPitch;
    const int least = (S::kRows * S::kSumPitch * 4 + S::kStage - 1) / S::kStage;     // the sums lie over the ring
    int stages = (kTwoPerSm - q_bytes) / (S::kKeyWarps * S::kStage);
    if (stages < 3 || stages < least) stages = (kOnePerSm - q_bytes) / (S::kKeyWarps * S::kStage);
    stages = stages > kMaxStages ? kMaxStages : stages;
    static_assert(kOnePerSm - 3 * S::kRows * S::kQPitch >= S::kKeyWarps * S::kStage * 3 &&
                  kOnePerSm - 3 * S::kRows * S::kQPitch >= S::kKeyWarps * S::kRows * S::kSumPitch * 4 + S::kKeyWarps * S::kStage,
                  "three stages, and room for the sums, whatever the queries' type");
    static_assert(kMaxStages * S::kStage >= S::kRows * S::kSumPitch * 4, "the sums lie over the ring");
    const int bytes = S::kKeyWarps * stages * S::kStage + q_bytes;
    p.unit = S::kStep * S::kKeyWarps;
    p.page_div = Divisor::of((unsigned)p.cache.page_size);
    p.tile_rows = S::kRows;
    p.row_tiles = (int)(((int64_t)p.q_len * p.group + S::kRows - 1) / S::kRows);
    const int grid = gdn::sm_count() * (bytes <= kTwoPerSm ? 2 : 1);
    p.grid = grid < kMaxGrid ? grid : kMaxGrid;
    cudaError_t e = gdn::allow_dynamic_smem<&attn_tc<CACHE, D, NT, R>>(kOnePerSm);
    if (e != cudaSuccess) return e;
    e = gdn::launch_early(attn_tc<CACHE, D, NT, R>, (unsigned)p.grid, S::kWarps * 32, bytes, s, true, p, stages, q_parts, w_parts);
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

template <int CACHE> cudaError_t launch_attn_tc(const AttnParams &p, cudaStream_t s)
{
    return p.d == 64 ? tc::by_rows<CACHE, 64>(p, s) : p.d == 128 ? tc::by_rows<CACHE, 128>(p, s) : tc::by_rows<CACHE, 256>(p, s);
}

}  // namespace gdna

// gdna_attn.cuh -- what the attention kernels share: how the work is dealt out,
// and where partial results lie (gdna_attn_decode).
//
// Work.  An item is one (sequence, key head, tile of query rows); its keys are cut
// into units of `unit` keys (a sequence without keys has one empty unit, which
// writes its zeros).  All units of all items stand in one row, item after item,
// and every block takes an equal run of them: long and short sequences, few and
// many heads balance without the host knowing a length.  Before its units an item
// has `lead` places that stand for what an item costs beside its keys (queries,
// adding up, output).  A block finds its run from kv_len alone (a prefix sum over
// the batch that every block repeats).
//
// Results.  An item that lies within one block's run is finished there.  One that
// crosses blocks leaves in each a partial: rows x D fp32 sums and each row's
// running maximum and sum.  A block has at most two of them, its first item
// (slot 2c) and its last (slot 2c + 1; an item that begins in the block is always
// its last), so the workspace is two slots a block however long the sequences.
// Block c also leaves a Join: the item that begins in it and continues, and in
// how many blocks.  attn_join adds those up in the blocks' order, so the result
// does not depend on timing.
#pragma once

#include "gdna_internal.cuh"

namespace gdna {

constexpr int kMaxKeys = INT32_MAX - 4095; // so that a step past a sequence's end is an int
constexpr int kMaxGrid = 608;              // blocks at most: workspace for two partials each

struct Join {
    int seq, item;                         // item within the sequence: key head * row_tiles + row tile
    int parts;                             // blocks the item lies in; 0: nothing to join here
    int pad;
};

__host__ __device__ __forceinline__ int part_width(int d) { return (d + 3) & ~3; }
// floats of one partial: rows x D sums, then rows x (maximum, sum)
__host__ __device__ __forceinline__ int64_t part_floats(int rows, int d) { return (int64_t)rows * (part_width(d) + 2); }

__device__ __forceinline__ Join *joins_of(const AttnParams &p) { return static_cast<Join *>(p.workspace); }
__device__ __forceinline__ float *part_of(const AttnParams &p, int slot)
{
    return reinterpret_cast<float *>(static_cast<Join *>(p.workspace) + kMaxGrid) +
           slot * part_floats(p.tile_rows, p.d);
}

// Keys of sequence b in its cache.
__device__ __forceinline__ int keys_of(const AttnParams &p, int b)
{
    const int64_t most = min((int64_t)p.max_pages * p.cache.page_size, (int64_t)kMaxKeys);
    return (int)min((int64_t)max(p.kv_len[b], 0), most);
}
// Places of an item in the row: its units behind its lead.
__device__ __forceinline__ int64_t places_of(const AttnParams &p, int keys)
{
    return p.lead + (keys > 0 ? ((unsigned)keys + (unsigned)p.unit - 1) / (unsigned)p.unit : 1u);
}

// a / b, in 32 bits where both fit (64-bit division is some hundred instructions).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b)
{
    return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((unsigned)a / (unsigned)b) : a / b;
}

// A block's run, in the row of all places.
struct Run {
    int64_t at, end, share;                // [at, end): this block's; share: places of every block's run
    int64_t base;                          // first place of sequence `seq`
    int seq;
    int keys, keys_after;                  // of `seq`, and (loaded ahead) of the sequence after it
};

__device__ __forceinline__ int keys_if(const AttnParams &p, int b) { return b < p.batch ? keys_of(p, b) : 0; }

// The run of block c.  All threads call it; `scratch` has blockDim.x / 32 + 3 int64.
__device__ __forceinline__ Run find_run(const AttnParams &p, int c, int64_t *scratch)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int64_t items = (int64_t)p.nkv * p.row_tiles;
    const int per = (p.batch + blockDim.x - 1) / blockDim.x;
    const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += places_of(p, keys_of(p, b));
    int64_t incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, incl, off);
        if (lane >= off) incl += y;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) incl += scratch[w];
        total += scratch[w];
    }
    Run r;
    total *= items;
    r.share = divide(total + p.grid - 1, p.grid);
    r.at = c * r.share;
    r.end = min(r.at + r.share, total);
    // the thread whose sequences hold place `at` walks them
    int64_t base = (incl - mine) * items;
    if (mine > 0 && base <= r.at && r.at < incl * items) {
        int b = b0, keys;
        for (;; ++b) {
            keys = keys_of(p, b);
            const int64_t n = places_of(p, keys) * items;
            if (r.at < base + n) break;
            base += n;
        }
        scratch[warps] = base;
        scratch[warps + 1] = b;
        scratch[warps + 2] = keys;
    }
    __syncthreads();
    r.base = scratch[warps];
    r.seq = (int)scratch[warps + 1];
    r.keys = (int)scratch[warps + 2];
    r.keys_after = r.at < r.end ? keys_if(p, r.seq + 1) : 0;
    return r;
}

// One item's part in a run.
struct Part {
    int seq, item, keys;                   // as in Join; keys of the sequence
    int64_t u0, u1;                        // units of the item
    bool begins, ends;                     // the item's first / last unit is among them
    int blocks;                            // where it begins and does not end: blocks it lies in
};

// The run's next part; advances it.  False where none is left.
__device__ __forceinline__ bool next_part(const AttnParams &p, Run &r, int c, Part &t)
{
    const int64_t items = (int64_t)p.nkv * p.row_tiles;
    while (r.at < r.end) {
        t.seq = r.seq;
        t.keys = r.keys;
        const int64_t n = places_of(p, t.keys), off = r.at - r.base;
        t.item = (int)divide(off, n);
        const int64_t from = off - t.item * n, to = min(n, from + (r.end - r.at));
        t.u0 = max(from - p.lead, (int64_t)0);
        t.u1 = to - p.lead;
        t.begins = t.u0 == 0;
        t.ends = to == n;
        t.blocks = t.begins && !t.ends ? (int)divide(r.base + (t.item + 1) * n - 1, r.share) - c + 1 : 0;
        r.at += to - from;
        if (t.ends && t.item == items - 1) {
            r.base += n * items;
            r.keys = r.keys_after;
            r.keys_after = keys_if(p, ++r.seq + 1);
        }
        if (t.u1 > t.u0) return true;      // (else the run ends within the item's lead)
    }
    return false;
}

// Query row `row` (token * group + head of the group) of a sequence sees this many keys.
__device__ __forceinline__ int keys_seen(const AttnParams &p, int keys, int row)
{
    return row < p.q_len * p.group ? keys - (p.q_len - 1 - row / p.group) : 0;
}

// o * sigmoid(g).  The exponential and the quotient are the fast ones (a few units in the last place of
// fp32): this is an elementwise tail, and what it feeds is rounded to 16 bits or scaled by a 16-bit gate.
__device__ __forceinline__ float gated(float o, float g) { return __fdividef(o, 1.0f + __expf(-g)); }

// Element c of query row `row`: o is the normalised sum.
__device__ __forceinline__ void write_out(const AttnParams &p, int seq, int head, int row, int c, float o)
{
    const int64_t r = (int64_t)seq * p.q_len + row / p.group;
    const int64_t h = (int64_t)head * p.group + row % p.group;
    if (p.gate != nullptr) {
        o = gated(o, load_elem(p.gate, r * p.gate_stride + h * p.gate_head_stride + c, p.dtype));
    }
    store_elem(p.out, r * p.out_stride + h * p.d + c, p.out_dtype, o);
}

// The natural logarithm of a row's softmax sum; m is in units of log2.
__device__ __forceinline__ float lse_of(float m, float l)
{
    return l == 0.f ? -__int_as_float(0x7f800000) : m * 0.69314718055994531f + logf(l);
}
__device__ __forceinline__ void write_lse(const AttnParams &p, int seq, int head, int row, float m, float l)
{
    const int64_t r = (int64_t)seq * p.q_len + row / p.group;
    if (p.lse != nullptr) p.lse[r * p.nq + (int64_t)head * p.group + row % p.group] = lse_of(m, l);
}

// Four sums of a row to outputs; norm: v_scale over the row's softmax sum, 0 for a row without keys.
__device__ __forceinline__ void finish4(const AttnParams &p, float4 &a, float norm, float4 gate)
{
    a = norm == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(a.x * norm, a.y * norm, a.z * norm, a.w * norm);
    if (p.gate != nullptr) a = make_float4(gated(a.x, gate.x), gated(a.y, gate.y), gated(a.z, gate.z), gated(a.w, gate.w));
}

// A row's sums stand for exp2(m) times them; m of a row without keys is -inf.
__device__ __forceinline__ float ex2(float x)              // 2^x, relative error below 2^-22
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float weight_of(float m, float top) { return m == -__int_as_float(0x7f800000) ? 0.f : ex2(m - top); }

// Adds up the items that lie in several blocks, after the kernel that left them.
cudaError_t launch_join(const AttnParams &p, cudaStream_t s);

// The tensor-core kernels, one translation unit per cache type.
template <int CACHE> cudaError_t launch_attn_tc(const AttnParams &p, cudaStream_t s);
// Bounded waits of theirs that ran out on the current device.
template <int CACHE> cudaError_t attn_wait_timeouts(unsigned *count);

}  // namespace gdna

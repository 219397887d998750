// gdnb_internal.cuh -- parameter blocks and launchers shared by the decoder-block
// translation units (include/gdnb.h).  Not part of the public ABI.
#pragma once

#include "gdna_internal.cuh"
#include "gdnb.h"

namespace gdnb {

using gdna::CacheLayout;
using gdna::Divisor;

struct NormParams {
    const void *x, *y, *gate;
    const float *post, *pre;
    void *x_out, *h;
    int64_t rows, x_stride, y_stride, gate_stride, x_out_stride, h_stride;
    int x_dtype, y_dtype, h_dtype, c;
    float scale, eps;
    int phase;                      // elements from a boundary of eight to the first row (set by the launcher)
    bool gate_pieces;               // the gate's rows begin where the others do
};

// How keys come into shared memory: 16-bit rows by tensor copies, E4M3 codes by tensor copies, or loads (16 bytes at a time, or
// element by element).
enum CopyMode { kTensorCopies = 0, kCodeCopies = 1, kLoads = 2, kPieces16 = 2, kElements = 3 };

// Attention of segments: runs of query rows with one list of keys each (the sequences of a prompt
// call; the groups of a shared prefix).
struct FlashParams {
    const void *q, *gate, *k, *v;
    const int32_t *table;           // NULL: keys lie in rows like the queries
    const int32_t *row_start;       // [segs + 1] (NULL: one segment), times row_mult
    const int32_t *kv_len;          // [segs], or NULL
    void *out;
    void *records;                  // of split tiles, and their partial results: the workspace (set by the launcher)
    float *parts;
    void *workspace;
    int64_t rows, table_stride, q_stride, gate_stride, gate_head_stride, out_stride;
    int64_t most_tiles, slots;      // that segments which do not overlap can make; partial results (set by the launcher)
    CacheLayout cache;
    int dtype, cache_dtype, out_dtype;
    int segs, row_mult, nq, nkv, group, d, max_pages;
    int causal;
    int all_parts;                  // every result is a partial one
    float scale2, v_scale;          // scores in units of log2
    // a shared call's requests' own keys: their attention, to be joined; or the last own_segs segments, row_mult tokens each
    const float *own, *own_lse;
    const int32_t *own_table, *own_kv_len;
    int64_t own_table_stride;
    int own_segs, own_max_pages;
    int64_t own_tiles;              // (set by the launcher)
    int q_vec, gate_vec, out_vec;   // rows and heads start on boundaries of 16 bytes, and are of eights
    int copy_mode, copy_keys;
    // set by the launcher
    int tile_tokens, tile_rows, grid;
    Divisor page_div, group_div;
};

cudaError_t launch_residual_norm(const NormParams &p, bool vec, cudaStream_t s);
cudaError_t launch_flash(FlashParams p, cudaStream_t s);
// Partial results: bytes that `segs` segments of `rows` rows need (prompt calls: a bound whatever the rows).
int64_t flash_parts_bytes(int64_t rows, int segs, int group, int nkv, int d, bool all_parts, int64_t own_tiles = 0);
// Tokens of a tile; tiles of `tokens` tokens of each of `segs` segments.
int flash_tile_tokens(int group, int d);
int64_t flash_tiles(int tokens, int segs, int group, int nkv, int d);
cudaError_t flash_wait_timeouts(unsigned *count);

}  // namespace gdnb

// gdna_attn.cu -- paged decode attention (gdna_attn_decode): the general kernel,
// the join of items that lie in several blocks, and the choice of kernel.
#include "gdna_attn.cuh"

namespace gdna {
namespace {

constexpr float kNegInf = -__builtin_huge_valf();

// ------------------------------------------------------------------ general kernel
//
// Any D <= 256, any strides and alignment.  One key a thread for the scores, one
// output column (or two) a thread for the sums; weights pass through shared
// memory.  Correct for everything and made for nothing: the calls that matter
// run on the tensor cores.
constexpr int kThreads = 128;
constexpr int kRows = 8;
constexpr int kMaxD = 256;

__global__ void __launch_bounds__(kThreads)
attn_general(const AttnParams p)
{
    __shared__ float q[kRows][kMaxD];
    __shared__ float weight[kRows][kThreads];
    __shared__ int64_t place[kThreads];    // element offset of a key's head; -1: a page of zeros
    __shared__ float red[kRows][kThreads / 32];
    __shared__ int64_t scratch[kThreads / 32 + 3];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x, D = p.d;
    Run run = find_run(p, c, scratch);
    Join join = {0, 0, 0, 0};
    Part part;
    while (next_part(p, run, c, part)) {
        const int head = part.item / p.row_tiles, row0 = (part.item % p.row_tiles) * kRows;
        __syncthreads();
        for (int i = tid; i < kRows * D; i += kThreads) {
            const int r = i / D, x = i - r * D, row = row0 + r;
            float v = 0.f;
            if (row < p.q_len * p.group)
                v = load_elem(p.q, ((int64_t)part.seq * p.q_len + row / p.group) * p.q_stride +
                                       ((int64_t)head * p.group + row % p.group) * D + x, p.dtype);
            q[r][x] = v;
        }
        int seen[kRows];
        float m[kRows], l[kRows], acc[kRows][2];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            seen[r] = keys_seen(p, part.keys, row0 + r);
            m[r] = kNegInf;
            l[r] = acc[r][0] = acc[r][1] = 0.f;
        }
        for (int64_t u = part.u0; u < part.u1; ++u) {
            const int64_t key = u * kThreads + tid;
            int64_t at = -1;
            if (key < part.keys) {
                const int64_t pg = key / p.cache.page_size;
                const int64_t page = p.table[part.seq * p.table_stride + pg];
                if (page >= 0 && page < p.cache.pages)
                    at = page * p.cache.page_stride + (key - pg * p.cache.page_size) * p.cache.token_stride +
                         head * p.cache.head_stride;
            }
            __syncthreads();               // the last unit's weights and places are used up; q is there
            place[tid] = at;
            float s[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) s[r] = 0.f;
            if (at >= 0)
                for (int x = 0; x < D; ++x) {
                    const float k = load_elem(p.k, at + x, p.cache_dtype);
#pragma unroll
                    for (int r = 0; r < kRows; ++r) s[r] = fmaf(q[r][x], k, s[r]);
                }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                s[r] = key < seen[r] ? s[r] * p.scale : kNegInf;
                float top = s[r];
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
                if (lane == 0) red[r][warp] = top;
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float top = fmaxf(m[r], fmaxf(fmaxf(red[r][0], red[r][1]), fmaxf(red[r][2], red[r][3])));
                const float from = top == kNegInf ? 0.f : top, down = weight_of(m[r], from);
                const float w = key < seen[r] ? exp2f(s[r] - from) : 0.f;
                l[r] = l[r] * down + w;
                acc[r][0] *= down;
                acc[r][1] *= down;
                m[r] = top;
                weight[r][tid] = w;
            }
            __syncthreads();
            const int here = (int)min((int64_t)kThreads, part.keys - u * kThreads);
            for (int j = 0; j < here; ++j) {
                if (place[j] < 0) continue;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int x = tid + e * kThreads;
                    if (x >= D) break;
                    const float v = load_elem(p.v, place[j] + x, p.cache_dtype);
#pragma unroll
                    for (int r = 0; r < kRows; ++r)     // a key a row does not see adds nothing, NaN or not
                        if (u * kThreads + j < seen[r]) acc[r][e] = fmaf(weight[r][j], v, acc[r][e]);
                }
            }
        }
        // a row's sum over the block (m is the same in all threads)
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float t = gdn::group_sum<32>(l[r]);
            __syncthreads();
            if (lane == 0) red[r][warp] = t;
            __syncthreads();
            l[r] = red[r][0] + red[r][1] + red[r][2] + red[r][3];
        }
        if (part.begins && part.ends) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (row0 + r >= p.q_len * p.group) break;
                const float norm = l[r] == 0.f ? 0.f : p.v_scale / l[r];
                for (int e = 0; e < 2; ++e)
                    if (tid + e * kThreads < D)
                        write_out(p, part.seq, head, row0 + r, tid + e * kThreads, l[r] == 0.f ? 0.f : acc[r][e] * norm);
                if (tid == 0) write_lse(p, part.seq, head, row0 + r, m[r], l[r]);
            }
        } else {
            float *to = part_of(p, 2 * c + (part.begins ? 1 : 0));
            const int width = part_width(D);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                for (int e = 0; e < 2; ++e)
                    if (tid + e * kThreads < D) to[r * width + tid + e * kThreads] = acc[r][e];
                if (tid == 0) { to[kRows * width + 2 * r] = m[r]; to[kRows * width + 2 * r + 1] = l[r]; }
            }
            if (part.begins) join = Join{part.seq, part.item, part.blocks, 0};
        }
    }
    if (tid == 0) joins_of(p)[c] = join;
}

// ------------------------------------------------------------------ join
//
// Block (c, r): row r of the item that begins in block c and continues.  All that it reads is a few
// hundred KB from the L2, so what counts is the chain of latencies: the Join first, then every part's
// maximum and sum, the first sums and the gate together.  The parts are dealt over the warps, a lane has
// up to two groups of four columns.  Small blocks: there are as many as blocks times rows, and one wave
// of them is to do.
constexpr int kJoinThreads = 128, kJoinWarps = kJoinThreads / 32;
constexpr int kFirst = 4;                  // parts a warp asks for at once

__global__ void __launch_bounds__(kJoinThreads)
attn_join(const AttnParams p)
{
    __shared__ float weight[kMaxGrid];
    __shared__ float red[kJoinWarps];
    __shared__ float4 sums[kJoinWarps][64];
    const int c = blockIdx.x, r = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int width = part_width(p.d), quads = width / 4;      // quads <= 64
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    auto part = [&](int i) { return part_of(p, 2 * (c + i) + (i == 0 ? 1 : 0)); };
    auto ml = [&](int i) { return __ldcs(reinterpret_cast<const float2 *>(part(i) + p.tile_rows * width + 2 * r)); };
    auto sum4 = [&](int i, int x) {
        return i < 0 || x >= quads ? zero : __ldcs(reinterpret_cast<const float4 *>(part(i) + r * width) + x);
    };
    gdn::early_start<true>(nullptr, 0);
    const Join join = joins_of(p)[c];
    const int n = join.parts;
    if (n == 0) return;
    const float2 mine = tid < n ? ml(tid) : make_float2(kNegInf, 0.f);
    float4 v[kFirst][2];
#pragma unroll
    for (int k = 0; k < kFirst; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) v[k][h] = sum4(warp + k * kJoinWarps < n ? warp + k * kJoinWarps : -1, lane + 32 * h);
    const int head = join.item / p.row_tiles, row = (join.item - head * p.row_tiles) * p.tile_rows + r;
    if (row >= p.q_len * p.group) return;
    const int token = row / p.group;
    const int64_t r_at = (int64_t)join.seq * p.q_len + token, h_at = (int64_t)head * p.group + (row - token * p.group);
    uint4 gate = make_uint4(0u, 0u, 0u, 0u);
    const bool four = p.d % 4 == 0;        // (else columns leave one by one)
    if (four && tid < quads && p.gate != nullptr)
        gate = ask4(p.gate, r_at * p.gate_stride + h_at * p.gate_head_stride + 4 * tid, p.dtype, p.gate_vec);

    // the parts' maximum, then their weights and the row's sum
    float top = mine.x;
    for (int i = tid + kJoinThreads; i < n; i += kJoinThreads) top = fmaxf(top, ml(i).x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
    if (lane == 0) red[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, red[w]);
    const float from = top == kNegInf ? 0.f : top;
    float l = 0.f;
    for (int i = tid; i < n; i += kJoinThreads) {
        const float2 u = i == tid ? mine : ml(i);
        weight[i] = weight_of(u.x, from);
        l = fmaf(weight[i], u.y, l);
    }
    l = gdn::group_sum<32>(l);
    __syncthreads();
    if (lane == 0) red[warp] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) l += red[w];

    float4 o[2] = {zero, zero};
    auto add = [&](int i, int h, float4 u) {
        const float w = weight[i];
        o[h].x = fmaf(w, u.x, o[h].x); o[h].y = fmaf(w, u.y, o[h].y);
        o[h].z = fmaf(w, u.z, o[h].z); o[h].w = fmaf(w, u.w, o[h].w);
    };
    for (int i0 = warp; i0 < n; i0 += kFirst * kJoinWarps) {
#pragma unroll
        for (int k = 0; k < kFirst; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (i0 + k * kJoinWarps < n) add(i0 + k * kJoinWarps, h, v[k][h]);
#pragma unroll
        for (int k = 0; k < kFirst; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = i0 + (kFirst + k) * kJoinWarps;
                v[k][h] = sum4(i < n ? i : -1, lane + 32 * h);
            }
    }
    sums[warp][lane] = o[0];
    sums[warp][lane + 32] = o[1];
    __syncthreads();
    const float norm = l == 0.f ? 0.f : p.v_scale / l;
    if (tid < quads) {
        float4 a = sums[0][tid];
#pragma unroll
        for (int w = 1; w < kJoinWarps; ++w) {
            const float4 u = sums[w][tid];
            a.x += u.x; a.y += u.y; a.z += u.z; a.w += u.w;
        }
        if (four) {
            finish4(p, a, norm, got4(gate, p.dtype, p.gate_vec));
            store4(p.out, r_at * p.out_stride + h_at * p.d + 4 * tid, p.out_dtype, p.out_vec, a);
        } else {
            const float u[4] = {a.x, a.y, a.z, a.w};
            for (int e = 0; e < 4 && 4 * tid + e < p.d; ++e)
                write_out(p, join.seq, head, row, 4 * tid + e, norm == 0.f ? 0.f : u[e] * norm);
        }
    }
    if (tid == 0) write_lse(p, join.seq, head, row, top, l);
}

// Query rows of a work item on the tensor cores.
int tc_rows(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

}  // namespace

cudaError_t attn_wait_timeouts(unsigned *count)
{
    unsigned n[3] = {0, 0, 0};
    cudaError_t e = attn_wait_timeouts<GDNA_F16>(&n[0]);
    if (e == cudaSuccess) e = attn_wait_timeouts<GDNA_BF16>(&n[1]);
    if (e == cudaSuccess) e = attn_wait_timeouts<GDNA_E4M3>(&n[2]);
    *count = n[0] + n[1] + n[2];
    return e;
}

int64_t attn_workspace_bytes(int64_t rows, int d)
{
    return kMaxGrid * (int64_t)sizeof(Join) + 2 * kMaxGrid * part_floats(tc_rows(rows), d) * (int64_t)sizeof(float);
}

cudaError_t launch_join(const AttnParams &p, cudaStream_t s)
{
    const int rows = p.q_len * p.group < p.tile_rows ? p.q_len * p.group : p.tile_rows;
    if (p.grid < 2) return cudaSuccess;
    return gdn::launch_early(attn_join, dim3(p.grid, rows), kJoinThreads, 0, s, true, p);
}

cudaError_t launch_attn_decode(const AttnParams &params, bool fast, cudaStream_t s)
{
    if (fast) {
        if (params.cache_dtype == GDNA_F16) return launch_attn_tc<GDNA_F16>(params, s);
        if (params.cache_dtype == GDNA_BF16) return launch_attn_tc<GDNA_BF16>(params, s);
        return launch_attn_tc<GDNA_E4M3>(params, s);
    }
    AttnParams p = params;
    p.unit = kThreads;
    p.lead = 0;
    p.tile_rows = kRows;
    p.row_tiles = (int)(((int64_t)p.q_len * p.group + kRows - 1) / kRows);
    const int sms = gdn::sm_count();
    p.grid = 4 * sms < kMaxGrid ? 4 * sms : kMaxGrid;
    attn_general<<<p.grid, kThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join(p, s);
}

}  // namespace gdna

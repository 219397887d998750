// gdna_internal.cuh -- parameter blocks, launcher declarations and device
// helpers shared by the attention-layer translation units (include/gdna.h).
// Not part of the public ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_internal.cuh"
#include "gdna.h"

namespace gdna {

using gdn::kFull;

// Where the cache's elements are: strides in elements.
struct CacheLayout {
    int64_t page_stride, token_stride, head_stride;
    int64_t pages;
    int page_size;
};

// Division of x < 2^31 by a fixed d >= 1 as a product: with 2^s >= d the quotient is
// floor(x m / 2^(31+s)), m = ceil(2^(31+s) / d) < 2^32 (the error x (m d - 2^(31+s)) / (d 2^(31+s))
// stays below 1 / d: Granlund and Montgomery, PLDI 1994).
struct Divisor {
    unsigned m, s;
    static Divisor of(unsigned d)
    {
        unsigned s = 0;
        while ((1ull << s) < d) ++s;
        return Divisor{(unsigned)(((1ull << (31 + s)) + d - 1) / d), s};
    }
    __device__ __forceinline__ unsigned quotient(unsigned x) const { return (unsigned)(((uint64_t)x * m) >> (31 + s)); }
};

struct PageParams {
    const int32_t *cached, *fresh;
    int32_t *table;
    int64_t table_stride;
    const int32_t *free_pages;
    int64_t n_free;
    const int32_t *free_head;
    int32_t *kv_len, *row_start;
    int64_t *slots;
    int32_t *positions, *free_head_out, *unserved;
    int64_t rows;
    int batch, page_size, max_pages;
    Divisor page_div;       // by the page size (set by the launcher)
};

struct RopeParams {
    const void *q, *k, *v;
    const float *qn, *kn, *cos_sin;
    const int32_t *positions;
    const int64_t *slots;
    void *q_out, *k_out, *k_cache, *v_cache;
    int64_t rows, n_pos;
    int64_t q_stride, q_head_stride, k_stride, v_stride, q_out_stride, k_out_stride;
    CacheLayout cache;
    int dtype, cache_dtype, nq, nkv, d, rot, interleaved;
    float eps, k_scale, v_scale;
    Divisor page_div;       // by the page size (set by the launcher)
};

struct AttnParams {
    const void *q, *gate, *k, *v;
    const int32_t *table, *kv_len;
    void *out;
    float *lse;
    void *workspace;
    int64_t table_stride, q_stride, gate_stride, gate_head_stride, out_stride;
    CacheLayout cache;
    int dtype, cache_dtype, out_dtype;
    int batch, q_len, nq, nkv, group, d, max_pages;
    float scale;            // scale * k_scale * log2(e): scores in units of log2
    float v_scale;
    int q_vec, gate_vec, out_vec;   // rows and heads start on boundaries of four elements
    // set by the launcher
    int unit;               // keys of one unit of work
    int lead;               // units that an item costs beside its keys
    int tile_rows;          // query rows (token, head of the group) of one work item
    int row_tiles;          // ceil(q_len * group / tile_rows)
    int grid;               // blocks that share the work
    Divisor page_div;       // by the page size
};

cudaError_t launch_page_assign(PageParams p, cudaStream_t s);
cudaError_t launch_qk_norm_rope(const RopeParams &p, bool fast, cudaStream_t s);
cudaError_t launch_attn_decode(const AttnParams &p, bool fast, cudaStream_t s);
// Bounded waits of the attention kernels that ran out on the current device.
cudaError_t attn_wait_timeouts(unsigned *count);
int64_t attn_workspace_bytes(int64_t rows, int d);

// ---------------------------------------------------------------- device helpers

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__nv_fp8_storage_t x)
{
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(x, __NV_E4M3)));
}

// One element of an array whose type is known at run time.
__device__ __forceinline__ float load_elem(const void *p, int64_t i, int dtype)
{
    if (dtype == GDNA_F32) return static_cast<const float *>(p)[i];
    if (dtype == GDNA_F16) return to_f32(static_cast<const __half *>(p)[i]);
    if (dtype == GDNA_BF16) return to_f32(static_cast<const __nv_bfloat16 *>(p)[i]);
    return to_f32(static_cast<const __nv_fp8_storage_t *>(p)[i]);
}

// The same, rounded to nearest even once (E4M3 saturates at +-448).
__device__ __forceinline__ void store_elem(void *p, int64_t i, int dtype, float x)
{
    if (dtype == GDNA_F32) static_cast<float *>(p)[i] = x;
    else if (dtype == GDNA_F16) static_cast<__half *>(p)[i] = __float2half_rn(x);
    else if (dtype == GDNA_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
    else static_cast<__nv_fp8_storage_t *>(p)[i] = __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

// Four elements that follow one another, as they lie in memory (`vec`: they start on a boundary of four; else as
// fp32), so that several can be on their way before the first is looked at.
__device__ __forceinline__ uint4 ask4(const void *p, int64_t i, int dtype, bool vec)
{
    if (!vec)
        return make_uint4(__float_as_uint(load_elem(p, i, dtype)), __float_as_uint(load_elem(p, i + 1, dtype)),
                          __float_as_uint(load_elem(p, i + 2, dtype)), __float_as_uint(load_elem(p, i + 3, dtype)));
    if (dtype == GDNA_F32) return *reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i);
    const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
    return make_uint4(u.x, u.y, 0u, 0u);
}
// What ask4 brought.
__device__ __forceinline__ float4 got4(uint4 u, int dtype, bool vec)
{
    if (!vec || dtype == GDNA_F32)
        return make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
    if (dtype == GDNA_F16) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}

__device__ __forceinline__ void store4(void *p, int64_t i, int dtype, bool vec, float4 x)
{
    if (!vec) {
        store_elem(p, i, dtype, x.x);
        store_elem(p, i + 1, dtype, x.y);
        store_elem(p, i + 2, dtype, x.z);
        store_elem(p, i + 3, dtype, x.w);
    } else if (dtype == GDNA_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = x;
    } else {
        uint2 u;
        if (dtype == GDNA_F16) {
            const __half2 a = __floats2half2_rn(x.x, x.y), b = __floats2half2_rn(x.z, x.w);
            u = make_uint2(*reinterpret_cast<const unsigned *>(&a), *reinterpret_cast<const unsigned *>(&b));
        } else {
            const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
            u = make_uint2(*reinterpret_cast<const unsigned *>(&a), *reinterpret_cast<const unsigned *>(&b));
        }
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i) = u;
    }
}

}  // namespace gdna

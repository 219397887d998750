// gdna_rope.cu -- per-head RMS norm of queries and keys, rotary positions and the
// cache's new rows in one pass (gdna_qk_norm_rope), and the host's table of
// cosines and sines (gdna_rope_table).
//
//     y = w x / sqrt(mean x^2 + eps);   (a, b) -> (a cos - b sin, a sin + b cos)
//
// on the first `rot` elements in pairs.  A stream: every input is read once and
// every output written once; the norm and the rotation stay in registers.
#include <cmath>

#include "gdna_internal.cuh"

namespace gdna {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxD = 256;

// General kernel: any 1 <= D <= 256, any alignment.  One warp per (row, head):
// heads 0..NQ-1 are the queries', then NKV keys', then NKV values'.
__global__ void __launch_bounds__(kThreads)
norm_rope_general(const RopeParams p)
{
    __shared__ float line[kWarps][kMaxD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int heads = p.nq + p.nkv * (p.v != nullptr ? 2 : 1), D = p.d;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
    if (unit >= p.rows * heads) return;                 // whole warps leave together
    const int64_t row = unit / heads;
    const int h = (int)(unit - row * heads);
    const int kind = h < p.nq ? 0 : h < p.nq + p.nkv ? 1 : 2;
    const int hh = kind == 0 ? h : kind == 1 ? h - p.nq : h - p.nq - p.nkv;
    const void *src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    const int64_t from = kind == 0 ? row * p.q_stride + hh * p.q_head_stride
                                   : row * (kind == 1 ? p.k_stride : p.v_stride) + (int64_t)hh * D;
    float *x = line[warp];
    float sum = 0.f;
    for (int i = lane; i < D; i += 32) {
        const float a = load_elem(src, from + i, p.dtype);
        x[i] = a;
        sum = fmaf(a, a, sum);
    }
    const float *w = kind == 0 ? p.qn : kind == 1 ? p.kn : nullptr;
    if (w != nullptr) {
        sum = gdn::group_sum<32>(sum);
        const float r = rsqrtf(sum / (float)D + p.eps);
        for (int i = lane; i < D; i += 32) x[i] = x[i] * r * w[i];
    }
    __syncwarp();

    const int half = p.rot / 2;
    const int64_t pos = p.rot > 0 ? p.positions[row] : 0;
    const bool known = pos >= 0 && pos < p.n_pos;
    const float *cs = p.cos_sin + (known ? pos : 0) * p.rot;
    const bool caching = kind > 0 && p.k_cache != nullptr;
    const int64_t slot = caching ? p.slots[row] : -1;
    const bool stored = slot >= 0 && slot < p.cache.pages * p.cache.page_size;
    int64_t at = 0;
    if (stored) {
        const int64_t page = slot / p.cache.page_size;
        at = page * p.cache.page_stride + (slot - page * p.cache.page_size) * p.cache.token_stride +
             hh * p.cache.head_stride;
    }
    for (int i = lane; i < D; i += 32) {
        float y = x[i];
        if (kind < 2 && i < p.rot) {
            const bool first = p.interleaved ? (i & 1) == 0 : i < half;
            const int pair = p.interleaved ? i >> 1 : first ? i : i - half;
            const float other = x[p.interleaved ? i ^ 1 : first ? i + half : i - half];
            const float c = known ? cs[pair] : __int_as_float(0x7fc00000), s = known ? cs[half + pair] : 0.f;
            y = first ? y * c - other * s : other * s + y * c;
        }
        if (kind == 0) store_elem(p.q_out, row * p.q_out_stride + (int64_t)hh * D + i, p.dtype, y);
        if (kind == 1 && p.k_out != nullptr)
            store_elem(p.k_out, row * p.k_out_stride + (int64_t)hh * D + i, p.dtype, y);
        if (stored)
            store_elem(kind == 1 ? p.k_cache : p.v_cache, at + i, p.cache_dtype, y / (kind == 1 ? p.k_scale : p.v_scale));
    }
}

// ------------------------------------------------------------------ vector kernel
//
// Head sizes 64, 128 and 256 on 16-byte boundaries, D/8 lanes a head, eight elements a lane as two runs of four.  In
// the rotated part of the half layout the runs are `half` apart, so that a lane holds both elements of its four
// pairs; elsewhere they follow one another.  No element crosses lanes but in the mean of squares, a butterfly over
// the head's lanes.  A block takes up to kInFlight heads a lane of one token row: their loads, the row's position and
// slot go out together, and its cosines and sines are loaded once for all of them.
//   A stream that the issue slots bound as much as the memory does (some hundred instructions for eight elements):
// 32768 rows of 24 + 4 fp32 heads of 256 take 314 us (2.02 GB: 6.4 TB/s, 0.95 of the measured copy rate).  With the
// pairs exchanged by shuffles they took 386; with blocks that stay and load the next row into the registers that a
// head leaves, 614 (half the warps fit).  With 64 registers eight blocks of 128 fit an SM: 316 us against 327 without
// that bound, 324 in blocks of 256.
constexpr int kInFlight = 4;
constexpr int kBlock = 128, kFit = 8;      // threads of a block, blocks on an SM (64 registers)

template <typename T> struct Four;         // four elements in registers as they lie in memory
template <> struct Four<float> {
    float4 u;
    __device__ __forceinline__ void load(const float *p) { u = __ldcs(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ float4 get() const { return u; }
};
template <> struct Four<__half> {
    uint2 u;
    __device__ __forceinline__ void load(const __half *p) { u = __ldcs(reinterpret_cast<const uint2 *>(p)); }
    __device__ __forceinline__ float4 get() const
    {
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u.x)), b = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
};
template <> struct Four<__nv_bfloat16> {
    uint2 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = __ldcs(reinterpret_cast<const uint2 *>(p)); }
    __device__ __forceinline__ float4 get() const
    {
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                           __uint_as_float(u.y & 0xffff0000u));
    }
};

// Four fp32 values to four elements of a type, rounded once.
__device__ __forceinline__ void put4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void put4(__half *p, float4 x)
{
    const __half2 a = __floats2half2_rn(x.x, x.y), b = __floats2half2_rn(x.z, x.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const unsigned *>(&a), *reinterpret_cast<const unsigned *>(&b));
}
__device__ __forceinline__ void put4(__nv_bfloat16 *p, float4 x)
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const unsigned *>(&a), *reinterpret_cast<const unsigned *>(&b));
}
__device__ __forceinline__ void put4(__nv_fp8_storage_t *p, float4 x)
{
    const unsigned a = __nv_cvt_float2_to_fp8x2(make_float2(x.x, x.y), __NV_SATFINITE, __NV_E4M3);
    const unsigned b = __nv_cvt_float2_to_fp8x2(make_float2(x.z, x.w), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<unsigned *>(p) = a | (b << 16);
}

__device__ __forceinline__ float squares(float4 x, float sum)
{
    return fmaf(x.x, x.x, fmaf(x.y, x.y, fmaf(x.z, x.z, fmaf(x.w, x.w, sum))));
}
__device__ __forceinline__ void turn(float &a, float &b, float c, float s)
{
    const float t = a * c - b * s;
    b = a * s + b * c;
    a = t;
}
__device__ __forceinline__ float4 scaled(float4 x, float by) { return make_float4(x.x / by, x.y / by, x.z / by, x.w / by); }

template <typename T, int D, bool INTERLEAVED, int FLIGHT>
__global__ void __launch_bounds__(kBlock, kFit)
norm_rope_vec(const RopeParams p, const int passes)
{
    constexpr int kLanes = D / 8, kAtOnce = kBlock / kLanes;                 // lanes of a head, heads of a block
    const int s = threadIdx.x % kLanes, first = threadIdx.x / kLanes;
    const int64_t row = blockIdx.x;
    const int heads = p.nq + p.nkv * (p.v != nullptr ? 2 : 1), half = p.rot / 2;
    const int from = blockIdx.y * passes * kAtOnce, to = min(heads, from + passes * kAtOnce);
    const bool turned = 8 * s < p.rot;
    // this lane's two runs of four elements
    const int e0 = !INTERLEAVED && turned ? 4 * s : 8 * s, e1 = !INTERLEAVED && turned ? half + 4 * s : 8 * s + 4;
    gdn::early_start<true>(nullptr, 0);

    const int64_t pos = turned ? p.positions[row] : 0, slot = p.k_cache != nullptr ? p.slots[row] : -1;
    Four<T> raw[FLIGHT][2];
    auto load = [&](int h0) {
#pragma unroll
        for (int k = 0; k < FLIGHT; ++k) {
            const int h = h0 + k * kAtOnce;
            raw[k][0] = raw[k][1] = Four<T>{};
            if (h < to) {
                const T *src = h < p.nq ? static_cast<const T *>(p.q) + row * p.q_stride + h * p.q_head_stride
                             : h < p.nq + p.nkv ? static_cast<const T *>(p.k) + row * p.k_stride + (int64_t)(h - p.nq) * D
                                                : static_cast<const T *>(p.v) + row * p.v_stride + (int64_t)(h - p.nq - p.nkv) * D;
                raw[k][0].load(src + e0);
                raw[k][1].load(src + e1);
            }
        }
    };
    load(from + first);

    // the four pairs' cosines and sines: pairs 4s .. 4s + 3 in either layout
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), n = make_float4(0.f, 0.f, 0.f, 0.f);
    if (turned) {
        const bool known = pos >= 0 && pos < p.n_pos;
        const float *at = p.cos_sin + (known ? pos : 0) * p.rot + 4 * s;
        c = __ldg(reinterpret_cast<const float4 *>(at));
        n = __ldg(reinterpret_cast<const float4 *>(at + half));
        if (!known) c.x = c.y = c.z = c.w = __int_as_float(0x7fc00000);
    }
    int64_t cache_at = -1;
    if (slot >= 0 && slot < p.cache.pages * p.cache.page_size) {
        const int64_t page = (slot >> 31) == 0 ? (int64_t)p.page_div.quotient((unsigned)slot) : slot / p.cache.page_size;
        cache_at = page * p.cache.page_stride + (slot - page * p.cache.page_size) * p.cache.token_stride;
    }

    for (int h0 = from + first; h0 - first < to; h0 += FLIGHT * kAtOnce) {  // (whole warps stay for the shuffles)
        if (h0 - first > from) load(h0);
#pragma unroll
        for (int k = 0; k < FLIGHT; ++k) {
            if (h0 - first + k * kAtOnce >= to) break;         // the block's
            const int h = h0 + k * kAtOnce;
            const bool query = h < p.nq, value = h >= p.nq + p.nkv;
            float4 x = raw[k][0].get(), y = raw[k][1].get();
            const float *w = value ? nullptr : query ? p.qn : p.kn;
            const float sum = gdn::group_sum<kLanes>(squares(x, squares(y, 0.f)));
            if (w != nullptr) {
                const float r = rsqrtf(sum * (1.0f / D) + p.eps);
                const float4 a = __ldg(reinterpret_cast<const float4 *>(w + e0)), b = __ldg(reinterpret_cast<const float4 *>(w + e1));
                x = make_float4(x.x * (r * a.x), x.y * (r * a.y), x.z * (r * a.z), x.w * (r * a.w));
                y = make_float4(y.x * (r * b.x), y.y * (r * b.y), y.z * (r * b.z), y.w * (r * b.w));
            }
            if (turned && !value) {
                if constexpr (INTERLEAVED) {
                    turn(x.x, x.y, c.x, n.x);
                    turn(x.z, x.w, c.y, n.y);
                    turn(y.x, y.y, c.z, n.z);
                    turn(y.z, y.w, c.w, n.w);
                } else {
                    turn(x.x, y.x, c.x, n.x);
                    turn(x.y, y.y, c.y, n.y);
                    turn(x.z, y.z, c.z, n.z);
                    turn(x.w, y.w, c.w, n.w);
                }
            }
            if (h >= to) continue;
            if (query) {
                T *out = static_cast<T *>(p.q_out) + row * p.q_out_stride + (int64_t)h * D;
                put4(out + e0, x);
                put4(out + e1, y);
                continue;
            }
            const int hh = value ? h - p.nq - p.nkv : h - p.nq;
            if (!value && p.k_out != nullptr) {
                T *out = static_cast<T *>(p.k_out) + row * p.k_out_stride + (int64_t)hh * D;
                put4(out + e0, x);
                put4(out + e1, y);
            }
            if (cache_at < 0) continue;
            const float scale = value ? p.v_scale : p.k_scale;
            if (scale != 1.f) { x = scaled(x, scale); y = scaled(y, scale); }
            const int64_t at = cache_at + hh * p.cache.head_stride;
            void *cache = value ? p.v_cache : p.k_cache;
            if (p.cache_dtype == GDNA_F16) {
                put4(static_cast<__half *>(cache) + at + e0, x);
                put4(static_cast<__half *>(cache) + at + e1, y);
            } else if (p.cache_dtype == GDNA_BF16) {
                put4(static_cast<__nv_bfloat16 *>(cache) + at + e0, x);
                put4(static_cast<__nv_bfloat16 *>(cache) + at + e1, y);
            } else {
                put4(static_cast<__nv_fp8_storage_t *>(cache) + at + e0, x);
                put4(static_cast<__nv_fp8_storage_t *>(cache) + at + e1, y);
            }
        }
    }
}

template <typename T, int D>
cudaError_t launch_vec(RopeParams p, cudaStream_t s)
{
    const int heads = p.nq + p.nkv * (p.v != nullptr ? 2 : 1), at_once = kBlock / (D / 8);
    const int all = (heads + at_once - 1) / at_once;           // passes over a whole row
    p.page_div = Divisor::of(p.cache.page_size > 0 ? (unsigned)p.cache.page_size : 1u);
    // Where one head a lane makes no more blocks than fit the GPU at once, that many blocks of a smaller kernel (one
    // row of 24 + 4 heads of 256: 2.2 us against 3.8; 64 rows of 16 + 2: 2.7 against 3.4); else kInFlight heads a lane,
    // whose loads are in flight together (256 rows of 48 + 8 heads of 128: 4.0 us against 4.2 with one).
    const bool few = p.rows * all <= kFit * gdn::sm_count() && all <= 65535;
    const int flight = few ? 1 : kInFlight, passes = (all + flight - 1) / flight <= 65535 ? flight : all;
    const dim3 grid((unsigned)p.rows, (unsigned)((all + passes - 1) / passes));
    auto launch = [&](auto kern) { return gdn::launch_early(kern, grid, kBlock, 0, s, few, p, passes); };
    if (few) return p.interleaved ? launch(norm_rope_vec<T, D, true, 1>) : launch(norm_rope_vec<T, D, false, 1>);
    return p.interleaved ? launch(norm_rope_vec<T, D, true, kInFlight>) : launch(norm_rope_vec<T, D, false, kInFlight>);
}

template <typename T>
cudaError_t launch_typed(const RopeParams &p, cudaStream_t s)
{
    return p.d == 64 ? launch_vec<T, 64>(p, s) : p.d == 128 ? launch_vec<T, 128>(p, s) : launch_vec<T, 256>(p, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams &p, bool fast, cudaStream_t s)
{
    if (fast)
        return p.dtype == GDNA_F32 ? launch_typed<float>(p, s) : p.dtype == GDNA_F16 ? launch_typed<__half>(p, s)
                                                                                     : launch_typed<__nv_bfloat16>(p, s);
    const int64_t units = p.rows * (p.nq + (int64_t)p.nkv * (p.v != nullptr ? 2 : 1));
    norm_rope_general<<<(unsigned)((units + kWarps - 1) / kWarps), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace gdna

extern "C" GDN_API int gdna_rope_table(float *table, int64_t n_pos, int rot, double base, gdna_rope_kind kind,
                                       double factor, double original_len, double beta_fast, double beta_slow,
                                       double amplitude)
{
    const double pi = 3.14159265358979323846;
    if (n_pos < 0 || rot < 2 || rot % 2 != 0) return GDN_ERR_ARG;
    if (!(base > 0) || !std::isfinite(base) || !(amplitude > 0) || !std::isfinite(amplitude)) return GDN_ERR_ARG;
    if (kind != GDNA_ROPE_PLAIN && kind != GDNA_ROPE_LINEAR && kind != GDNA_ROPE_NTK && kind != GDNA_ROPE_YARN)
        return GDN_ERR_UNSUPPORTED;
    if (kind != GDNA_ROPE_PLAIN && (!(factor >= 1) || !std::isfinite(factor))) return GDN_ERR_ARG;
    if (kind == GDNA_ROPE_NTK && rot < 4) return GDN_ERR_ARG;
    if (kind == GDNA_ROPE_YARN && (!(base > 1) || !(original_len > 0) || !std::isfinite(original_len) ||
                                   !(beta_slow > 0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast)))
        return GDN_ERR_ARG;
    if (n_pos == 0) return GDN_OK;
    if (table == nullptr) return GDN_ERR_ARG;
    if ((uintptr_t)table % 4 != 0) return GDN_ERR_ALIGN;
    const int half = rot / 2;
    if (kind == GDNA_ROPE_NTK) base *= std::pow(factor, (double)rot / (rot - 2));
    // YaRN: the (real) pair index at which a pair turns `turns` times within original_len, from
    // original_len * base^(-2i/rot) = 2 pi turns; the ramp goes between the two, rounded outwards.
    auto index_of = [&](double turns) {
        return rot * std::log(original_len / (turns * 2 * pi)) / (2 * std::log(base));
    };
    double low = 0, high = 0;
    if (kind == GDNA_ROPE_YARN) {
        low = std::fmax(std::floor(index_of(beta_fast)), 0.0);
        high = std::fmin(std::ceil(index_of(beta_slow)), (double)(rot - 1));
        if (!(high > low)) high = low + 0.001;
    }
    for (int i = 0; i < half; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (kind == GDNA_ROPE_LINEAR) f /= factor;
        if (kind == GDNA_ROPE_YARN) {
            const double ramp = std::fmin(std::fmax((i - low) / (high - low), 0.0), 1.0);   // 0: kept, 1: divided
            f = f * (1 - ramp) + f / factor * ramp;
        }
        for (int64_t n = 0; n < n_pos; ++n) {
            table[n * rot + i] = (float)(amplitude * std::cos(n * f));
            table[n * rot + half + i] = (float)(amplitude * std::sin(n * f));
        }
    }
    return GDN_OK;
}

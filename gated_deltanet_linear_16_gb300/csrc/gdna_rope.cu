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

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams &p, bool fast, cudaStream_t s)
{
    (void)fast;
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

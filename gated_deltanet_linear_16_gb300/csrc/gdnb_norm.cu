// gdnb_norm.cu -- norm after a block, gate, residual scale and norm before the
// next block in one pass (include/gdnb.h, gdnb_residual_norm).
//
//     u = post y / sqrt(mean y^2 + eps),  x' = x + scale gate u,  h = pre x' / sqrt(mean x'^2 + eps)
//
// Two sums over a row, the second of what the first decides, so a row stays in the registers
// of one block: eight or sixteen elements a thread, the threads as many as the row needs.
// Bound by HBM for many rows and by the chain load, sum, sum, store for few: with many rows sixteen elements, so that
// an SM has more rows in hand, with few eight, so that the chain is short.  A block takes row after row and asks for the
// next one's elements before it adds up this one's (16-bit rows), so that loads are in flight behind a row's two barriers.
// 32768 rows of 4096, bf16: 194 us, 5.5 TB/s (eight elements a thread: 250); fp32 throughout, 16384 rows: 171 us, 0.93 of the copy
// rate; one row: 6 us, the call.  Rows of an odd width that lie side by side are taken in eights from the
// boundary before them (16384 rows of 4095: 221 us, element by element 394; 20000 of 2881 in fp16 171, 393); rows that begin
// at unequal distances from a boundary go element by element, bound by its instructions.
#include "gdnb_internal.cuh"

namespace gdnb {
namespace {

// How a row's elements are taken: kWide: c and all rows are of eights on 16-byte boundaries.  kShifted: all rows begin equally far
// behind such a boundary (rows of an odd width that lie side by side), and groups of eight are counted from the boundary, the
// first and the last of a row element by element.  kSingly: any.
enum Mode { kSingly, kWide, kShifted };

// Eight elements of a row as they lie in memory (WIDE: fp32, else 16 bits), so that all are on their way before the first is
// looked at: elements first, first + step, ...; kWide, kShifted: first .. first + 7, 16 bytes at a time.
template <bool WIDE, int MODE> struct Row8 {
    static constexpr bool kVec = MODE != kSingly;
    uint4 a[kVec ? (WIDE ? 2 : 1) : 1];
    uint32_t one[kVec ? 1 : (WIDE ? 8 : 4)];

    // (`pieces`: 16 bytes at a time after all, a kShifted row of another stride not)
    __device__ __forceinline__ void ask(const void *p, int64_t row, int first, int step, int c, bool real, bool pieces = true)
    {
        if constexpr (kVec) {
            const bool in = real && first < c && (MODE == kWide || (pieces && first >= 0 && first + 8 <= c));
            a[0] = make_uint4(0u, 0u, 0u, 0u);
            if constexpr (WIDE) {
                const uint4 *at = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + row + first);
                a[1] = a[0];
                if (in) { a[0] = at[0]; a[1] = at[1]; }
            } else {
                if (in) a[0] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + row + first);
            }
            if constexpr (MODE == kShifted) {
                if (in || !real || first >= c) return;
                uint32_t u[WIDE ? 8 : 4];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool mine = first + j >= 0 && first + j < c;
                    if constexpr (WIDE) {
                        u[j] = mine ? (static_cast<const uint32_t *>(p) + row)[first + j] : 0u;
                    } else {
                        const uint32_t x = mine ? (static_cast<const uint16_t *>(p) + row)[first + j] : 0u;
                        u[j / 2] = j & 1 ? u[j / 2] | x << 16 : x;
                    }
                }
                a[0] = make_uint4(u[0], u[1], u[2], u[3]);
                if constexpr (WIDE) a[1] = make_uint4(u[4], u[5], u[6], u[7]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = real && first + j * step < c;
                if constexpr (WIDE) {
                    one[j] = in ? (static_cast<const uint32_t *>(p) + row + first)[j * step] : 0u;
                } else {
                    const uint32_t x = in ? (static_cast<const uint16_t *>(p) + row + first)[j * step] : 0u;
                    one[j / 2] = j & 1 ? one[j / 2] | x << 16 : x;
                }
            }
        }
    }
    __device__ __forceinline__ void get(float (&x)[8], int dtype) const
    {
        uint32_t u[WIDE ? 8 : 4];
        if constexpr (!kVec) {
#pragma unroll
            for (int j = 0; j < (WIDE ? 8 : 4); ++j) u[j] = one[j];
        } else {
#pragma unroll
            for (int j = 0; j < (WIDE ? 2 : 1); ++j) { u[4 * j] = a[j].x; u[4 * j + 1] = a[j].y; u[4 * j + 2] = a[j].z; u[4 * j + 3] = a[j].w; }
        }
        if constexpr (WIDE) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(u[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (dtype == GDNA_BF16) {
                    x[2 * j] = __uint_as_float(u[j] << 16);
                    x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[j]));
                    x[2 * j] = f.x;
                    x[2 * j + 1] = f.y;
                }
            }
        }
    }
};

template <int MODE>
__device__ __forceinline__ void put8(void *p, int64_t row, int first, int step, int c, int dtype, const float (&x)[8])
{
    if (MODE == kWide || (MODE == kShifted && first >= 0 && first + 8 <= c)) {
        if (first >= c) return;
        if (dtype == GDNA_F32) {
            float4 *at = reinterpret_cast<float4 *>(static_cast<float *>(p) + row + first);
            at[0] = make_float4(x[0], x[1], x[2], x[3]);
            at[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            unsigned u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (dtype == GDNA_BF16) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
                    u[j] = *reinterpret_cast<const unsigned *>(&b);
                } else {
                    const __half2 b = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
                    u[j] = *reinterpret_cast<const unsigned *>(&b);
                }
            }
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + row + first) = make_uint4(u[0], u[1], u[2], u[3]);
        }
    } else {
        if (MODE == kShifted && first >= c) return;
        auto mine = [&](int j) { return first + j * step < c && (MODE != kShifted || first + j >= 0); };
        // (the type decided once, not for each element)
        if (dtype == GDNA_F32) {
            float *at = static_cast<float *>(p) + row + first;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (mine(j)) at[j * step] = x[j];
        } else {
            uint16_t *at = static_cast<uint16_t *>(p) + row + first;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint16_t h = dtype == GDNA_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x[j])) : __half_as_ushort(__float2half_rn(x[j]));
                if (mine(j)) at[j * step] = h;
            }
        }
    }
}

template <int MODE>
__device__ __forceinline__ void weights8(const float *w, int first, int step, int c, float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 1.f;
    if (w == nullptr) return;
    if constexpr (MODE == kWide) {
        if (first >= c) return;
        const float4 a = *reinterpret_cast<const float4 *>(w + first), b = *reinterpret_cast<const float4 *>(w + first + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (first + j * step < c && first + j >= 0) x[j] = w[first + j * step];
    }
}
// Weights of kShifted rows, which begin at no boundary of eight, are kept in shared memory, element e at kBefore + e with one place
// left free after eight: lanes' elements, eight apart, then lie in 32 banks.
constexpr int kBefore = 8, kLeastShifted = 64, kMostShifted = 16370;   // (two groups a thread, 1024 threads)
__host__ __device__ constexpr int place_of(int i) { return i + (i >> 3); }
__host__ __device__ constexpr int places(int c) { return place_of(c + 2 * kBefore); }
__device__ __forceinline__ void keep(const float *w, int c, float *s)
{
    if (w == nullptr) return;
    for (int i = threadIdx.x; i < c + 2 * kBefore; i += blockDim.x)
        s[place_of(i)] = i >= kBefore && i < kBefore + c ? w[i - kBefore] : 1.f;
}
__device__ __forceinline__ void kept8(const float *w, const float *s, int first, int c, float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 1.f;
    if (w == nullptr || first >= c) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = s[place_of(kBefore + first + j)];
}

// The block's sum of `x`, in the warps' order; `red` alternates between two buffers, so that one barrier a sum is enough.
__device__ __forceinline__ float block_sum(float x, float *red)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    x = gdn::group_sum<32>(x);
    if (warps == 1) return x;
    if (lane == 0) red[warp] = x;
    __syncthreads();
    return gdn::group_sum<32>(lane < warps ? red[lane] : 0.f);
}

// XW, YW: x, y (and gate) are fp32.  K: groups of eight elements a thread.  EARLY: launched early, where all rows are in hand at
// once.
template <bool XW, bool YW, int MODE, int K, int THREADS, int BLOCKS, bool EARLY>
__global__ void __launch_bounds__(THREADS, BLOCKS) residual_norm(const NormParams p)
{
    gdn::early_start<EARLY>(nullptr, 0);
    __shared__ float red[2][32];
    const int t = threadIdx.x, n = blockDim.x, c = p.c;
    const int step = MODE != kSingly ? 1 : n * K;    // between a group's elements
    auto first = [&](int64_t row, int k) {
        if (MODE == kSingly) return t + k * n;
        return 8 * (t + k * n) - (MODE == kShifted ? (int)((p.phase + row * p.x_stride) & 7) : 0);
    };
    const float inv_c = 1.f / (float)c;
    constexpr bool kAhead = !XW && !YW && MODE != kSingly;   // the next row's elements in registers
    constexpr bool kKept = MODE == kShifted && !EARLY;         // the weights in shared memory
    constexpr bool kKeep = K == 1 && !kKept;                   // or in registers
    extern __shared__ float kept[];
    float post[8], pre[8];
    Row8<XW, MODE> x[K], x_next[kAhead ? K : 1];
    Row8<YW, MODE> y[K], y_next[kAhead ? K : 1], g[K];
    const bool has_y = p.y != nullptr, has_gate = p.gate != nullptr;
    auto ask = [&](int64_t row, int k, Row8<XW, MODE> &xr, Row8<YW, MODE> &yr) {
        const bool real = row < p.rows;
        xr.ask(p.x, row * p.x_stride, first(row, k), step, c, real);
        yr.ask(p.y, row * p.y_stride, first(row, k), step, c, real && has_y);
    };
    int64_t row = blockIdx.x;
    if constexpr (kAhead) {
#pragma unroll
        for (int k = 0; k < K; ++k) ask(row, k, x_next[k], y_next[k]);
    }
    if constexpr (kKeep) {
        weights8<MODE>(p.post, first(row, 0), step, c, post);
        weights8<MODE>(p.pre, first(row, 0), step, c, pre);
    }
    if constexpr (kKept) {
        keep(p.post, c, kept);
        keep(p.pre, c, kept + places(c));
        __syncthreads();
    }
    for (; row < p.rows; row += gridDim.x) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            g[k].ask(p.gate, row * p.gate_stride, first(row, k), step, c, has_gate, p.gate_pieces);
            if constexpr (kAhead) {
                x[k] = x_next[k]; y[k] = y_next[k];
                ask(row + gridDim.x, k, x_next[k], y_next[k]);
            } else {
                ask(row, k, x[k], y[k]);
            }
        }
        float factor = p.scale;
        if (has_y && p.post != nullptr) {              // (for all threads alike)
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float v[8];
                y[k].get(v, p.y_dtype);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = fmaf(v[j], v[j], sum);
            }
            factor = p.scale / sqrtf(block_sum(sum, red[0]) * inv_c + p.eps);
        }
        float sum = 0.f, to[K][8];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k].get(to[k], p.x_dtype);
            if (has_y) {
                float v[8], w[8];
                y[k].get(v, p.y_dtype);
                if constexpr (kKept) kept8(p.post, kept, first(row, k), c, post);
                else if constexpr (!kKeep) weights8<MODE>(p.post, first(row, k), step, c, post);
                g[k].get(w, p.y_dtype);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float u = v[j] * factor * post[j];
                    to[k][j] += has_gate ? u * w[j] : u;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(to[k][j], to[k][j], sum);
            if (p.x_out != nullptr) put8<MODE>(p.x_out, row * p.x_out_stride, first(row, k), step, c, p.x_dtype, to[k]);
        }
        if (p.h == nullptr) {
            // (the first sum's buffer is written again only after every thread has passed its barrier: two rows' barriers
            // would otherwise meet in one buffer)
            if (has_y && p.post != nullptr) __syncthreads();
            continue;
        }
        const float norm = 1.f / sqrtf(block_sum(sum, red[1]) * inv_c + p.eps);
        // without a first sum the same buffer is used row after row
        if (!(has_y && p.post != nullptr)) __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if constexpr (kKept) kept8(p.pre, kept + places(c), first(row, k), c, pre);
            else if constexpr (!kKeep) weights8<MODE>(p.pre, first(row, k), step, c, pre);
#pragma unroll
            for (int j = 0; j < 8; ++j) to[k][j] *= norm * pre[j];
            put8<MODE>(p.h, row * p.h_stride, first(row, k), step, c, p.h_dtype, to[k]);
        }
    }
}

template <bool XW, bool YW, int MODE, int K, int THREADS, int BLOCKS>
cudaError_t launch_as(const NormParams &p, unsigned blocks, int threads, cudaStream_t s)
{
    constexpr auto kern = residual_norm<XW, YW, MODE, K, THREADS, BLOCKS, false>;
    const int bytes = MODE == kShifted ? 2 * places(p.c) * (int)sizeof(float) : 0;
    if (MODE == kShifted) {
        const cudaError_t e = gdn::allow_dynamic_smem<kern>(2 * places(kMostShifted) * (int)sizeof(float));
        if (e != cudaSuccess) return e;
    }
    kern<<<blocks, threads, bytes, s>>>(p);
    return cudaGetLastError();
}
template <bool XW, bool YW, int MODE>
cudaError_t launch(const NormParams &p, cudaStream_t s)
{
    const int groups = (p.c + 7 + (MODE == kShifted ? 7 : 0)) / 8, sms = gdn::sm_count();
    // Sixteen elements a thread where the row needs them, or where there are rows for it: four or more an SM.
    const bool wide = groups > 1024 || (groups > 128 && p.rows >= 4 * (int64_t)sms);
    const int threads = ((wide ? (groups + 1) / 2 : groups) + 31) / 32 * 32;
    auto grid = [&](int resident) {                    // as many blocks as are resident at once, and no more than rows
        const int64_t most = (int64_t)sms * resident;
        return (unsigned)(p.rows < most ? p.rows : most);
    };
    const int some = threads >= 1024 ? 1 : threads <= 64 ? 16 : 1024 / threads;
    const unsigned blocks = grid(some);
    if (!wide && blocks == p.rows) return gdn::launch_early(residual_norm<XW, YW, MODE, 1, 1024, 1, true>, blocks, threads, 0, s, true, p);
    if (!wide) return launch_as<XW, YW, MODE, 1, 1024, 1>(p, blocks, threads, s);
    if (threads <= 256) return launch_as<XW, YW, MODE, 2, 256, 4>(p, blocks, threads, s);
    return launch_as<XW, YW, MODE, 2, 1024, 1>(p, blocks, threads, s);
}

template <int MODE> cudaError_t by_types(const NormParams &p, cudaStream_t s)
{
    const bool xw = p.x_dtype == GDNA_F32, yw = p.y != nullptr && p.y_dtype == GDNA_F32;
    if (xw) return yw ? launch<true, true, MODE>(p, s) : launch<true, false, MODE>(p, s);
    return yw ? launch<false, true, MODE>(p, s) : launch<false, false, MODE>(p, s);
}

// Whether all rows begin equally far behind a boundary of eight elements, and how far the first does.
bool equally_shifted(NormParams &p)
{
    auto size = [](int dtype) { return dtype == GDNA_F32 ? 4 : 2; };
    auto behind = [&](const void *a, int dtype) { return (int)(reinterpret_cast<uintptr_t>(a) / size(dtype) % 8); };
    auto like_x = [&](const void *a, int dtype, int64_t stride) {
        return a == nullptr || (behind(a, dtype) == p.phase && (p.rows == 1 || (stride - p.x_stride) % 8 == 0));
    };
    p.phase = behind(p.x, p.x_dtype);
    p.gate_pieces = like_x(p.gate, p.y_dtype, p.gate_stride);
    return p.c >= kLeastShifted && p.c <= kMostShifted && like_x(p.y, p.y_dtype, p.y_stride) &&
           like_x(p.x_out, p.x_dtype, p.x_out_stride) && like_x(p.h, p.h_dtype, p.h_stride);
}

}  // namespace

cudaError_t launch_residual_norm(const NormParams &args, bool vec, cudaStream_t s)
{
    NormParams p = args;
    if (vec) return by_types<kWide>(p, s);
    return equally_shifted(p) ? by_types<kShifted>(p, s) : by_types<kSingly>(p, s);
}

}  // namespace gdnb

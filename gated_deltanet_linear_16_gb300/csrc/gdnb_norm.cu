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
// rate; one row: 6 us, the call.  Rows that are not of eights on 16-byte boundaries go element by element, four times slower
// (16384 rows of 4095: 400 us): bound by its instructions.
#include "gdnb_internal.cuh"

namespace gdnb {
namespace {


// Eight elements of a row as they lie in memory (WIDE: fp32, else 16 bits), so that all are on their way before the first is
// looked at: elements first .. first + 7 (VEC: 16 bytes at a time), else first, first + step, ...
template <bool WIDE, bool VEC> struct Row8 {
    uint4 a[VEC ? (WIDE ? 2 : 1) : 1];
    uint32_t one[VEC ? 1 : (WIDE ? 8 : 4)];

    __device__ __forceinline__ void ask(const void *p, int64_t row, int first, int step, int c, bool real)
    {
        if constexpr (VEC) {
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            const bool in = real && first < c;
            if constexpr (WIDE) {
                const uint4 *at = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + row + first);
                a[0] = in ? at[0] : zero;
                a[1] = in ? at[1] : zero;
            } else {
                a[0] = in ? *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + row + first) : zero;
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
        if constexpr (!VEC) {
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

template <bool VEC>
__device__ __forceinline__ void put8(void *p, int64_t row, int first, int step, int c, int dtype, const float (&x)[8])
{
    if constexpr (VEC) {
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
        // (the type decided once, not for each element)
        if (dtype == GDNA_F32) {
            float *at = static_cast<float *>(p) + row + first;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (first + j * step < c) at[j * step] = x[j];
        } else {
            uint16_t *at = static_cast<uint16_t *>(p) + row + first;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint16_t h = dtype == GDNA_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x[j])) : __half_as_ushort(__float2half_rn(x[j]));
                if (first + j * step < c) at[j * step] = h;
            }
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void weights8(const float *w, int first, int step, int c, float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 1.f;
    if (w == nullptr) return;
    if constexpr (VEC) {
        if (first >= c) return;
        const float4 a = *reinterpret_cast<const float4 *>(w + first), b = *reinterpret_cast<const float4 *>(w + first + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (first + j * step < c) x[j] = w[first + j * step];
    }
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
template <bool XW, bool YW, bool VEC, int K, int THREADS, int BLOCKS, bool EARLY>
__global__ void __launch_bounds__(THREADS, BLOCKS) residual_norm(const NormParams p)
{
    gdn::early_start<EARLY>(nullptr, 0);
    __shared__ float red[2][32];
    const int t = threadIdx.x, n = blockDim.x, c = p.c;
    const int step = VEC ? 1 : n * K;                  // between a group's elements
    auto first = [&](int k) { return VEC ? 8 * (t + k * n) : t + k * n; };
    const float inv_c = 1.f / (float)c;
    constexpr bool kAhead = !XW && !YW && VEC;         // the next row's elements in registers
    constexpr bool kKeep = K == 1;                     // and the weights
    float post[8], pre[8];
    Row8<XW, VEC> x[K], x_next[kAhead ? K : 1];
    Row8<YW, VEC> y[K], y_next[kAhead ? K : 1], g[K];
    const bool has_y = p.y != nullptr, has_gate = p.gate != nullptr;
    auto ask = [&](int64_t row, int k, Row8<XW, VEC> &xr, Row8<YW, VEC> &yr) {
        const bool real = row < p.rows;
        xr.ask(p.x, row * p.x_stride, first(k), step, c, real);
        yr.ask(p.y, row * p.y_stride, first(k), step, c, real && has_y);
    };
    int64_t row = blockIdx.x;
    if constexpr (kAhead) {
#pragma unroll
        for (int k = 0; k < K; ++k) ask(row, k, x_next[k], y_next[k]);
    }
    if constexpr (kKeep) {
        weights8<VEC>(p.post, first(0), step, c, post);
        weights8<VEC>(p.pre, first(0), step, c, pre);
    }
    for (; row < p.rows; row += gridDim.x) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            g[k].ask(p.gate, row * p.gate_stride, first(k), step, c, has_gate);
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
                if constexpr (!kKeep) weights8<VEC>(p.post, first(k), step, c, post);
                g[k].get(w, p.y_dtype);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float u = v[j] * factor * post[j];
                    to[k][j] += has_gate ? u * w[j] : u;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(to[k][j], to[k][j], sum);
            if (p.x_out != nullptr) put8<VEC>(p.x_out, row * p.x_out_stride, first(k), step, c, p.x_dtype, to[k]);
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
            if constexpr (!kKeep) weights8<VEC>(p.pre, first(k), step, c, pre);
#pragma unroll
            for (int j = 0; j < 8; ++j) to[k][j] *= norm * pre[j];
            put8<VEC>(p.h, row * p.h_stride, first(k), step, c, p.h_dtype, to[k]);
        }
    }
}

template <bool XW, bool YW, bool VEC>
cudaError_t launch(const NormParams &p, cudaStream_t s)
{
    const int groups = (p.c + 7) / 8, sms = gdn::sm_count();
    // Sixteen elements a thread where the row needs them, or where there are rows for it: four or more an SM.
    const bool wide = groups > 1024 || (groups > 128 && p.rows >= 4 * (int64_t)sms);
    const int threads = ((wide ? (groups + 1) / 2 : groups) + 31) / 32 * 32;
    auto grid = [&](int resident) {                    // as many blocks as are resident at once, and no more than rows
        const int64_t most = (int64_t)sms * resident;
        return (unsigned)(p.rows < most ? p.rows : most);
    };
    const int some = threads >= 1024 ? 1 : threads <= 64 ? 16 : 1024 / threads;
    const unsigned blocks = grid(some);
    if (!wide) {
        if (blocks == p.rows) return gdn::launch_early(residual_norm<XW, YW, VEC, 1, 1024, 1, true>, blocks, threads, 0, s, true, p);
        residual_norm<XW, YW, VEC, 1, 1024, 1, false><<<blocks, threads, 0, s>>>(p);
    } else if (threads <= 256) {
        residual_norm<XW, YW, VEC, 2, 256, 4, false><<<blocks, threads, 0, s>>>(p);
    } else {
        residual_norm<XW, YW, VEC, 2, 1024, 1, false><<<blocks, threads, 0, s>>>(p);
    }
    return cudaGetLastError();
}

template <bool VEC> cudaError_t by_types(const NormParams &p, cudaStream_t s)
{
    const bool xw = p.x_dtype == GDNA_F32, yw = p.y != nullptr && p.y_dtype == GDNA_F32;
    if (xw) return yw ? launch<true, true, VEC>(p, s) : launch<true, false, VEC>(p, s);
    return yw ? launch<false, true, VEC>(p, s) : launch<false, false, VEC>(p, s);
}

}  // namespace

cudaError_t launch_residual_norm(const NormParams &p, bool vec, cudaStream_t s)
{
    return vec ? by_types<true>(p, s) : by_types<false>(p, s);
}

}  // namespace gdnb

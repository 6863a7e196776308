// moe_dispatch, its gradient, and the gradients of moe_finalize: the copies
// between token order and expert order.
//
// A workgroup owns a token.  The token's k places are scalars (the same for
// the whole workgroup), and each thread moves 16-byte words of the row: a
// token's row is read once and written to all its places, or its places'
// rows are read and summed.  No atomics: every row belongs to one token.
#include <algorithm>

#include "rowops.h"

namespace moe {
namespace {

constexpr int kMaxGrid = 1 << 20;

// A thread for each 16-byte word (or 8 values) of a row, up to 1024: the whole
// row moves at once, which the memory likes better than four steps of 4 KiB
// (DeepSeek-V3-shaped training batch, 256 -> 1024 threads at most: gradients of
// the weighted sum 413 -> 391 us, dispatch and its gradient 456 -> 446 us).
int threads_for(int n) { return std::min(1024, (n + 63) / 64 * 64); }

// 16 bytes at byte `off` of a row at a wave-uniform address.  Streamed rows are
// written once by one workgroup and fill the caches with nothing but
// themselves.  THROUGH: past this XCD's L2 as well (a buffer store with the
// device scope and non-temporal bits), so that no dirty lines are left for the
// next kernel to write back.  Dispatch and gradient of the DeepSeek-V3-shaped
// training batch: plain 442 us, non-temporal 439, THROUGH 427; its fp8 rows
// alone 107, 88, 80; the 33 MB of a decode batch 7.9, 7.1, 7.8 us.
template <bool THROUGH>
__device__ __forceinline__ void store_row16(u32x4_t v, char* row, unsigned row_bytes, unsigned off)
{
    if constexpr (THROUGH) {
        constexpr int kNt = 2, kSc1 = 16;
        const auto r = __builtin_amdgcn_make_buffer_rsrc(row, 0, (int)row_bytes, 0x00027000);
        __builtin_amdgcn_raw_buffer_store_b128(v, r, (int)off, 0, kNt | kSc1);
    } else {
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(row + off));
    }
}

// Rows of `bytes` bytes (a multiple of 16); with scales, nsc floats a row.
template <bool THROUGH>
__global__ __launch_bounds__(1024) void dispatch_kernel(const char* __restrict__ x,
                                                        const float* __restrict__ x_scale, int T, int k,
                                                        int n_shared, unsigned bytes, int nsc,
                                                        const int32_t* __restrict__ unpermute,
                                                        char* __restrict__ rows, float* __restrict__ rows_scale)
{
    const int P = T * k;
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        int at[MOE_MAX_TOPK];
#pragma unroll
        for (int j = 0; j < MOE_MAX_TOPK; ++j) at[j] = j < k ? unpermute[(size_t)t * k + j] : -1;
        for (unsigned c = threadIdx.x * 16; c < bytes; c += blockDim.x * 16) {
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(x + (size_t)t * bytes + c);
#pragma unroll
            for (int j = 0; j < MOE_MAX_TOPK; ++j)
                if ((unsigned)at[j] < (unsigned)P)
                    store_row16<THROUGH>(v, rows + (size_t)at[j] * bytes, bytes, c);
            for (int i = 0; i < n_shared; ++i)
                store_row16<THROUGH>(v, rows + ((size_t)P + (size_t)i * T + t) * bytes, bytes, c);
        }
        for (int c = threadIdx.x; c < nsc; c += blockDim.x) {
            const float v = x_scale[(size_t)t * nsc + c];
#pragma unroll
            for (int j = 0; j < MOE_MAX_TOPK; ++j)
                if ((unsigned)at[j] < (unsigned)P) rows_scale[(size_t)at[j] * nsc + c] = v;
            for (int i = 0; i < n_shared; ++i)
                rows_scale[((size_t)P + (size_t)i * T + t) * nsc + c] = v;
        }
    }
}

template <class Tin, class Tout, bool NT>
__global__ __launch_bounds__(1024) void dispatch_backward_kernel(const Tin* __restrict__ d_rows,
                                                                     const int32_t* __restrict__ unpermute,
                                                                     int T, int k, int H, int n_shared,
                                                                     Tout* __restrict__ dx)
{
    const int P = T * k, nch = H >> 3;
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        int at[MOE_MAX_TOPK];
#pragma unroll
        for (int j = 0; j < MOE_MAX_TOPK; ++j) at[j] = j < k ? unpermute[(size_t)t * k + j] : -1;
        for (int c = threadIdx.x; c < nch; c += blockDim.x) {
            Raw8<Tin> v[MOE_MAX_TOPK];
#pragma unroll
            for (int j = 0; j < MOE_MAX_TOPK; ++j) {
                v[j].zero();
                if ((unsigned)at[j] < (unsigned)P) v[j].template load<NT>(d_rows + (size_t)at[j] * H + 8 * c);
            }
            float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < MOE_MAX_TOPK; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] += v[j][e];
            for (int i = 0; i < n_shared; ++i) {
                Raw8<Tin> b;
                b.template load<NT>(d_rows + ((size_t)P + (size_t)i * T + t) * H + 8 * c);
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] += b[e];
            }
            store8_f32(dx + (size_t)t * H + 8 * c, a);
        }
    }
}

// No __restrict__ on fc2 and d_fc2: they may be the same rows.  A thread
// reads a word of a row before it writes the same word.
template <class Ty, class T, bool NT>
__global__ __launch_bounds__(1024) void finalize_backward_kernel(const Ty* __restrict__ dy, const T* fc2,
                                                                     const int32_t* __restrict__ unpermute,
                                                                     const float* __restrict__ scales, int Tn,
                                                                     int k, int H, int n_shared, T* d_fc2,
                                                                     float* __restrict__ d_scales)
{
    __shared__ float s_dot[16][MOE_MAX_TOPK];
    const int P = Tn * k, nch = H >> 3;
    for (int t = blockIdx.x; t < Tn; t += gridDim.x) {
        int at[MOE_MAX_TOPK];
        float sc[MOE_MAX_TOPK], dot[MOE_MAX_TOPK];
#pragma unroll
        for (int j = 0; j < MOE_MAX_TOPK; ++j) {
            at[j] = j < k ? unpermute[(size_t)t * k + j] : -1;
            sc[j] = j < k ? scales[(size_t)t * k + j] : 0.0f;
            dot[j] = 0.0f;
        }
        for (int c = threadIdx.x; c < nch; c += blockDim.x) {
            Raw8<Ty> g;
            g.template load<NT>(dy + (size_t)t * H + 8 * c);
            Raw8<T> v[MOE_MAX_TOPK];
#pragma unroll
            for (int j = 0; j < MOE_MAX_TOPK; ++j)
                if ((unsigned)at[j] < (unsigned)P) v[j].template load<NT>(fc2 + (size_t)at[j] * H + 8 * c);
#pragma unroll
            for (int j = 0; j < MOE_MAX_TOPK; ++j) {
                if ((unsigned)at[j] >= (unsigned)P) continue;
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dot[j] += g[e] * v[j][e];
                    o[e] = sc[j] * g[e];
                }
                Raw8<T> w;
                w.set(o);
                w.template store<NT>(d_fc2 + (size_t)at[j] * H + 8 * c);
            }
            if (n_shared > 0) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = g[e];
                Raw8<T> w;
                w.set(o);
                for (int i = 0; i < n_shared; ++i)
                    w.template store<NT>(d_fc2 + ((size_t)P + (size_t)i * Tn + t) * H + 8 * c);
            }
        }
#pragma unroll
        for (int j = 0; j < MOE_MAX_TOPK; ++j)
            if (j < k) {
                const float d = wave_sum_f32(dot[j]);
                if ((threadIdx.x & 63) == 0) s_dot[threadIdx.x >> 6][j] = d;
            }
        __syncthreads();
        if ((int)threadIdx.x < k) {
            float d = 0.0f;
            for (int w = 0; w < (int)(blockDim.x >> 6); ++w) d += s_dot[w][threadIdx.x];
            d_scales[(size_t)t * k + threadIdx.x] = d;
        }
        __syncthreads();
    }
}

}  // namespace

moe_status launch_dispatch(const void* x, const float* x_scale, int dt, int T, int H, int k, int n_shared,
                           const int32_t* unpermute, void* rows, float* rows_scale, hipStream_t s)
{
    const unsigned bytes = (unsigned)H * (dt == MOE_F32 ? 4 : dt == MOE_BF16 ? 2 : 1);
    const bool through = (long)T * (k + n_shared + 1) * bytes > kStream;
    auto* kernel = through ? dispatch_kernel<true> : dispatch_kernel<false>;
    {
        TimedLaunch tl(MOE_KID_DISPATCH, s);
        hipLaunchKernelGGL(kernel, dim3(std::min(T, kMaxGrid)), dim3(threads_for(bytes / 16)), 0, s,
                           static_cast<const char*>(x), x_scale, T, k, n_shared, bytes,
                           dt == MOE_FP8_E4M3 ? H / 128 : 0, unpermute, static_cast<char*>(rows), rows_scale);
    }
    return launch_status("dispatch_kernel");
}

namespace {

template <class Tin, class Tout>
void launch_sum(const void* d_rows, const int32_t* unpermute, int T, int k, int H, int n_shared, void* dx,
                hipStream_t s)
{
    const bool nt = (long)T * (k + n_shared + 1) * H * (long)sizeof(Tin) > kStream;
    auto* kernel = nt ? dispatch_backward_kernel<Tin, Tout, true> : dispatch_backward_kernel<Tin, Tout, false>;
    TimedLaunch tl(MOE_KID_DISPATCH_BWD, s);
    hipLaunchKernelGGL(kernel, dim3(std::min(T, kMaxGrid)), dim3(threads_for(H / 8)), 0, s,
                       static_cast<const Tin*>(d_rows), unpermute, T, k, H, n_shared, static_cast<Tout*>(dx));
}

template <class Ty, class T>
void launch_fin(const void* dy, const void* fc2, const int32_t* unpermute, const float* scales, int Tn, int k,
                int H, int n_shared, void* d_fc2, float* d_scales, hipStream_t s)
{
    const bool nt = (long)Tn * (2 * (k + n_shared) + 1) * H * (long)sizeof(T) > kStream;
    auto* kernel = nt ? finalize_backward_kernel<Ty, T, true> : finalize_backward_kernel<Ty, T, false>;
    TimedLaunch tl(MOE_KID_FINALIZE_BWD, s);
    hipLaunchKernelGGL(kernel, dim3(std::min(Tn, kMaxGrid)), dim3(threads_for(H / 8)), 0, s,
                       static_cast<const Ty*>(dy), static_cast<const T*>(fc2), unpermute, scales, Tn, k, H,
                       n_shared, static_cast<T*>(d_fc2), d_scales);
}

}  // namespace

moe_status launch_dispatch_backward(const void* d_rows, int dt, const int32_t* unpermute, int T, int k, int H,
                                    int n_shared, void* dx, int dxt, hipStream_t s)
{
    if (dt == MOE_BF16 && dxt == MOE_BF16)
        launch_sum<bf16_t, bf16_t>(d_rows, unpermute, T, k, H, n_shared, dx, s);
    else if (dt == MOE_BF16)
        launch_sum<bf16_t, float>(d_rows, unpermute, T, k, H, n_shared, dx, s);
    else if (dxt == MOE_BF16)
        launch_sum<float, bf16_t>(d_rows, unpermute, T, k, H, n_shared, dx, s);
    else
        launch_sum<float, float>(d_rows, unpermute, T, k, H, n_shared, dx, s);
    return launch_status("dispatch_backward_kernel");
}

moe_status launch_finalize_backward(const void* dy, int dyt, const void* fc2, int dt, const int32_t* unpermute,
                                    const float* scales, int T, int k, int H, int n_shared, void* d_fc2,
                                    float* d_scales, hipStream_t s)
{
    if (dyt == MOE_BF16 && dt == MOE_BF16)
        launch_fin<bf16_t, bf16_t>(dy, fc2, unpermute, scales, T, k, H, n_shared, d_fc2, d_scales, s);
    else if (dyt == MOE_BF16)
        launch_fin<bf16_t, float>(dy, fc2, unpermute, scales, T, k, H, n_shared, d_fc2, d_scales, s);
    else if (dt == MOE_BF16)
        launch_fin<float, bf16_t>(dy, fc2, unpermute, scales, T, k, H, n_shared, d_fc2, d_scales, s);
    else
        launch_fin<float, float>(dy, fc2, unpermute, scales, T, k, H, n_shared, d_fc2, d_scales, s);
    return launch_status("finalize_backward_kernel");
}

}  // namespace moe

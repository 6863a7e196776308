// moe_dispatch, its gradient, and the gradients of moe_finalize: the copies
// between token order and expert order.
//
// A workgroup owns a token.  The token's k places are scalars (the same for
// the whole workgroup), and each thread moves 16-byte words of the row: a
// token's row is read once and written to all its places, or its places'
// rows are read and summed.  No atomics: every row belongs to one token.
//
// Bound by memory.  Measured on MI355X, 8192 tokens x 7168 bf16, k = 8, one shared
// expert, skewed routing (1.17 GB a copy): dispatch and its gradient in turn 441
// us (5.3 TB/s; each alone 237 and 211 us, 5.0 and 5.6 TB/s), the gradients of
// finalize 384 us (2.1 GB, 5.5 TB/s; 357 us with rows in token order).  Decode
// batch of 512 tokens' codes 7.1 us.
// Every pair of types, 4096 x 7168, k = 4, rows' type first: the gradient of
// dispatch bf16/bf16 53 us, bf16/fp32 66, fp32/bf16 96, fp32/fp32 106 (5.3 to 5.5
// TB/s); the gradients of finalize 105, 120, 198, 212 us (4.9 to 5.0 TB/s).
#include <algorithm>

#include "rowops.h"

namespace moe {
namespace {

constexpr int kMaxGrid = 1 << 20;

// A thread for each 16-byte word of a row, up to 512 or (wide) 1024.  With many
// rows a token the whole row at once is what the memory likes best; with few, a
// workgroup of 1024 threads waits too long for too little.  512 / 1024 threads:
//   dispatch and gradient, 4096 x 7168 bf16  k = 1 47 / 64 us, k = 2 65 / 74 us,
//     k = 4 110 / 105 us; 8192 tokens, k = 8 and a shared expert 452 / 439 us
//   finalize_backward, 4096 x 7168 bf16  k = 1 34 / 52 us, k = 2 53 / 63 us, k = 4
//     96.5 / 97.0 us, k = 6 142 / 140 us, 8192 tokens, k = 8 and a shared expert 396 /
//     385 us; 512 tokens, k = 8 25.8 / 27.7 us; 64 x 7168 fp32, k = 8 12.9 / 10.8 us
int threads_for(int n, bool wide) { return std::min(wide ? 1024 : 512, (n + 63) / 64 * 64); }

// Rows of nch 16-byte words; with scales, nsc floats a row.  A row is written
// once, by one workgroup, and fills the caches with nothing but itself: the
// stores carry the non-temporal hint at every size (plain / hinted: 33 MB of a
// decode batch's codes 7.9 / 7.1 us, with a reader behind them equal; 530 MB of
// codes 107 / 88 us).
__global__ __launch_bounds__(1024) void dispatch_kernel(const u32x4_t* __restrict__ x,
                                                        const float* __restrict__ x_scale, int T, int k,
                                                        int n_shared, int nch, int nsc,
                                                        const int32_t* __restrict__ unpermute,
                                                        u32x4_t* __restrict__ rows,
                                                        float* __restrict__ rows_scale)
{
    const int P = T * k;
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        int at[MOE_MAX_TOPK];
#pragma unroll
        for (int j = 0; j < MOE_MAX_TOPK; ++j) at[j] = j < k ? unpermute[(size_t)t * k + j] : -1;
        for (int c = threadIdx.x; c < nch; c += blockDim.x) {
            const u32x4_t v = x[(size_t)t * nch + c];
#pragma unroll
            for (int j = 0; j < MOE_MAX_TOPK; ++j)
                if ((unsigned)at[j] < (unsigned)P)
                    __builtin_nontemporal_store(v, rows + (size_t)at[j] * nch + c);
            for (int i = 0; i < n_shared; ++i)
                __builtin_nontemporal_store(v, rows + ((size_t)P + (size_t)i * T + t) * nch + c);
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

// Values that a lane takes at a time where rows of two types meet.
template <class A, class B>
constexpr int kShared = 16 / (sizeof(A) > sizeof(B) ? sizeof(A) : sizeof(B));

template <class Tin, class Tout, bool NT>
__global__ __launch_bounds__(1024) void dispatch_backward_kernel(const Tin* __restrict__ d_rows,
                                                                     const int32_t* __restrict__ unpermute,
                                                                     int T, int k, int H, int n_shared,
                                                                     Tout* __restrict__ dx)
{
    constexpr int V = kShared<Tin, Tout>;
    const int P = T * k, nch = H / V;
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        int at[MOE_MAX_TOPK];
#pragma unroll
        for (int j = 0; j < MOE_MAX_TOPK; ++j) at[j] = j < k ? unpermute[(size_t)t * k + j] : -1;
        for (int c = threadIdx.x; c < nch; c += blockDim.x) {
            Raw<Tin, V> v[MOE_MAX_TOPK];
#pragma unroll
            for (int j = 0; j < MOE_MAX_TOPK; ++j) {
                v[j].zero();
                if ((unsigned)at[j] < (unsigned)P) v[j].template load<NT>(d_rows + (size_t)at[j] * H + V * c);
            }
            float a[V] = {};
#pragma unroll
            for (int j = 0; j < MOE_MAX_TOPK; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e) a[e] += v[j][e];
            for (int i = 0; i < n_shared; ++i) {
                Raw<Tin, V> b;
                b.template load<NT>(d_rows + ((size_t)P + (size_t)i * T + t) * H + V * c);
#pragma unroll
                for (int e = 0; e < V; ++e) a[e] += b[e];
            }
            Raw<Tout, V> w;
            w.set(a);
            w.store(dx + (size_t)t * H + V * c);
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
    constexpr int V = kShared<Ty, T>;
    const int P = Tn * k, nch = H / V;
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
            Raw<Ty, V> g;
            g.template load<NT>(dy + (size_t)t * H + V * c);
            Raw<T, V> v[MOE_MAX_TOPK];
#pragma unroll
            for (int j = 0; j < MOE_MAX_TOPK; ++j)
                if ((unsigned)at[j] < (unsigned)P) v[j].template load<NT>(fc2 + (size_t)at[j] * H + V * c);
#pragma unroll
            for (int j = 0; j < MOE_MAX_TOPK; ++j) {
                if ((unsigned)at[j] >= (unsigned)P) continue;
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    dot[j] += g[e] * v[j][e];
                    o[e] = sc[j] * g[e];
                }
                Raw<T, V> w;
                w.set(o);
                w.template store<NT>(d_fc2 + (size_t)at[j] * H + V * c);
            }
            if (n_shared > 0) {
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = g[e];
                Raw<T, V> w;
                w.set(o);
                for (int i = 0; i < n_shared; ++i)
                    w.template store<NT>(d_fc2 + ((size_t)P + (size_t)i * Tn + t) * H + V * c);
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
    const int nch = (int)((size_t)H * (dt == MOE_F32 ? 4 : dt == MOE_BF16 ? 2 : 1) / 16);
    {
        TimedLaunch tl(MOE_KID_DISPATCH, s);
        hipLaunchKernelGGL(dispatch_kernel, dim3(std::min(T, kMaxGrid)), dim3(threads_for(nch, k > 2)), 0, s,
                           static_cast<const u32x4_t*>(x), x_scale, T, k, n_shared, nch,
                           dt == MOE_FP8_E4M3 ? H / 128 : 0, unpermute, static_cast<u32x4_t*>(rows), rows_scale);
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
    hipLaunchKernelGGL(kernel, dim3(std::min(T, kMaxGrid)), dim3(threads_for(H / kShared<Tin, Tout>, k > 2)), 0, s,
                       static_cast<const Tin*>(d_rows), unpermute, T, k, H, n_shared, static_cast<Tout*>(dx));
}

template <class Ty, class T>
void launch_fin(const void* dy, const void* fc2, const int32_t* unpermute, const float* scales, int Tn, int k,
                int H, int n_shared, void* d_fc2, float* d_scales, hipStream_t s)
{
    const bool nt = (long)Tn * (2 * (k + n_shared) + 1) * H * (long)sizeof(T) > kStream;
    const bool wide = k > 4 && (nt || Tn < device_cu_count());
    auto* kernel = nt ? finalize_backward_kernel<Ty, T, true> : finalize_backward_kernel<Ty, T, false>;
    TimedLaunch tl(MOE_KID_FINALIZE_BWD, s);
    hipLaunchKernelGGL(kernel, dim3(std::min(Tn, kMaxGrid)), dim3(threads_for(H / kShared<Ty, T>, wide)), 0, s,
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

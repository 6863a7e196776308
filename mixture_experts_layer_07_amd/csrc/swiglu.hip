// moe_swiglu and its gradient from the 8-bit checkpoint.
//
//     h = g s u,  s = 1 / (1 + e^-g)
//     d_g = dh u s (1 + g (1 - s)),  d_u = dh g s
//
// Element by element, bound by memory.  A thread takes 16 bytes of gates and
// the ups of the same columns; 16 (bf16) or 32 (fp32) consecutive lanes hold one
// 128-value block of each.  A thread's chunk (row, col) moves by a fixed stride
// a step; the stride's whole rows and rest come from the host, so no division
// is made in the loop.
//
// Measured on MI355X, 73728 x 2048 bf16: forward with the checkpoint 202 us (1.22
// GB, 6.0 TB/s), backward with h again 253 us (1.52 GB, 6.0 TB/s), 461 us for the
// two in turn; 4096 rows to codes of h 8.9 us.  64, 128, 256 threads a workgroup 457, 460,
// 475 us; two or four chunks a thread in flight 470, 494 us; 32 bytes a lane in the
// backward 590 us (half lines a store).
#include <algorithm>

#include "rowops.h"

namespace moe {
namespace {

constexpr int kThreads = 128;

// e^-g: bf16 outputs keep 9 bits, so the product form of exp (relative error
// below 2^-22 |g|) serves; fp32 outputs take the library's function.
template <class T>
__device__ __forceinline__ float exp_neg(float g)
{
    if constexpr (sizeof(T) == 2) return __expf(-g);
    else return expf(-g);
}

template <class T>
__device__ __forceinline__ float sigmoid(float g)
{
    if constexpr (sizeof(T) == 2) return __builtin_amdgcn_rcpf(1.0f + exp_neg<T>(g));
    else return 1.0f / (1.0f + exp_neg<T>(g));
}

template <class T, bool NT>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(const T* __restrict__ gu, int rows, int nch, int drow,
                                                          int dcol, T* __restrict__ h, uint8_t* __restrict__ hq,
                                                          float* __restrict__ h_scale, uint8_t* __restrict__ guq,
                                                          float* __restrict__ gu_scale)
{
    constexpr int V = Raw<T>::kValues;
    constexpr int kLanes = 128 / V;  // of a block
    const unsigned first = blockIdx.x * kThreads + threadIdx.x;
    int row = (int)(first / (unsigned)nch), col = (int)(first % (unsigned)nch);
    const size_t I = (size_t)nch * V;
    while (row < rows) {
        const size_t g0 = (size_t)row * 2 * I + V * col, h0 = (size_t)row * I + V * col;
        Raw<T> rg, ru;
        rg.load(gu + g0);
        ru.load(gu + g0 + I);
        float g[V], u[V], o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            g[e] = rg[e];
            u[e] = ru[e];
            o[e] = g[e] * sigmoid<T>(g[e]) * u[e];
        }
        if (h) {
            Raw<T> w;
            w.set(o);
            w.template store<NT>(h + h0);
        }
        // 8-bit outputs: I is a multiple of 128, so a block's lanes share a row and a step
        if (hq) {
            const float s = block_absmax(o) / 448.0f;
            store_codes(o, s, hq + h0);
            if ((col & (kLanes - 1)) == 0) h_scale[h0 >> 7] = s;
        }
        if (guq) {
            const float sg = block_absmax(g) / 448.0f, su = block_absmax(u) / 448.0f;
            store_codes(g, sg, guq + g0);
            store_codes(u, su, guq + g0 + I);
            if ((col & (kLanes - 1)) == 0) {
                gu_scale[g0 >> 7] = sg;
                gu_scale[(g0 + I) >> 7] = su;
            }
        }
        row += drow;
        col += dcol;
        if (col >= nch) {
            col -= nch;
            ++row;
        }
    }
}

// No __restrict__ on dh and h: they may be the same rows.
template <class T, bool NT>
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(const T* dh, const uint8_t* __restrict__ guq,
                                                                   const float* __restrict__ gu_scale, int rows,
                                                                   int nch, int drow, int dcol,
                                                                   T* __restrict__ d_gu, T* h)
{
    constexpr int V = Raw<T>::kValues;
    const unsigned first = blockIdx.x * kThreads + threadIdx.x;
    int row = (int)(first / (unsigned)nch), col = (int)(first % (unsigned)nch);
    const size_t I = (size_t)nch * V;
    while (row < rows) {
        const size_t g0 = (size_t)row * 2 * I + V * col, h0 = (size_t)row * I + V * col;
        Raw<T> rd;
        rd.load(dh + h0);
        float g[V], u[V], dg[V], du[V], o[V];
        load_codes(guq + g0, gu_scale[g0 >> 7], g);
        load_codes(guq + g0 + I, gu_scale[(g0 + I) >> 7], u);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float s = sigmoid<T>(g[e]), gs = g[e] * s, d = rd[e];
            dg[e] = d * u[e] * (s + gs * (1.0f - s));
            du[e] = d * gs;
            o[e] = gs * u[e];
        }
        Raw<T> w;
        w.set(dg);
        w.template store<NT>(d_gu + g0);
        w.set(du);
        w.template store<NT>(d_gu + g0 + I);
        if (h) {
            w.set(o);
            w.template store<NT>(h + h0);
        }
        row += drow;
        col += dcol;
        if (col >= nch) {
            col -= nch;
            ++row;
        }
    }
}

int grid_of(int rows, int nch)
{
    const long chunks = (long)rows * nch;
    return (int)std::min((chunks + kThreads - 1) / kThreads, 1l << 20);
}

}  // namespace

namespace {

template <class T>
void launch_fwd(int rows, int I, const void* gu, void* h, uint8_t* hq, float* h_scale, uint8_t* guq,
                float* gu_scale, hipStream_t s)
{
    const int nch = I / Raw<T>::kValues, grid = grid_of(rows, nch), stride = grid * kThreads;
    const bool nt = (long)rows * I * ((h ? 3 : 2) * (long)sizeof(T) + (hq ? 1 : 0) + (guq ? 2 : 0)) > kStream;
    auto* kernel = nt ? swiglu_kernel<T, true> : swiglu_kernel<T, false>;
    TimedLaunch tl(MOE_KID_SWIGLU, s);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), 0, s, static_cast<const T*>(gu), rows, nch, stride / nch,
                       stride % nch, static_cast<T*>(h), hq, h_scale, guq, gu_scale);
}

template <class T>
void launch_bwd(int rows, int I, const void* dh, const uint8_t* guq, const float* gu_scale, void* d_gu,
                void* h, hipStream_t s)
{
    const int nch = I / Raw<T>::kValues, grid = grid_of(rows, nch), stride = grid * kThreads;
    const bool nt = (long)rows * I * ((h ? 4 : 3) * (long)sizeof(T) + 2) > kStream;
    auto* kernel = nt ? swiglu_backward_kernel<T, true> : swiglu_backward_kernel<T, false>;
    TimedLaunch tl(MOE_KID_SWIGLU_BWD, s);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), 0, s, static_cast<const T*>(dh), guq, gu_scale, rows, nch,
                       stride / nch, stride % nch, static_cast<T*>(d_gu), static_cast<T*>(h));
}

}  // namespace

moe_status launch_swiglu(const void* gu, int dt, int rows, int I, void* h, uint8_t* hq, float* h_scale,
                         uint8_t* guq, float* gu_scale, hipStream_t s)
{
    auto* f = dt == MOE_BF16 ? launch_fwd<bf16_t> : launch_fwd<float>;
    f(rows, I, gu, h, hq, h_scale, guq, gu_scale, s);
    return launch_status("swiglu_kernel");
}

moe_status launch_swiglu_backward(const void* dh, int dt, const uint8_t* guq, const float* gu_scale, int rows,
                                  int I, void* d_gu, void* h, hipStream_t s)
{
    auto* f = dt == MOE_BF16 ? launch_bwd<bf16_t> : launch_bwd<float>;
    f(rows, I, dh, guq, gu_scale, d_gu, h, s);
    return launch_status("swiglu_backward_kernel");
}

}  // namespace moe

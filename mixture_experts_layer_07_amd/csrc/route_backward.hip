// moe_route_backward: the gradient of the routing weights.
//
// With a kept expert's unnormalised weight w (an exponential or a sigmoid), S
// the sum that divides the weights and d the incoming gradients,
//     v_j - sum_i v_i w_i / S  =  (sum_i w_i (d_j - d_i) + (S - sum_i w_i) d_j) scaling / S
// where S - sum_i w_i is what the sum holds besides the kept weights: the
// other experts' exponentials (plain softmax), the 1e-20 (DeepSeek-V3) or
// nothing.  Written so, nothing cancels where one weight is near 1, and one
// renormalised weight alone has gradient exactly 0.
//
// Latency-bound: it writes T*E floats and reads little.  A wave owns eight
// tokens, eight lanes each: they compute the kept experts' gradients in fp64 (k
// exponentials a token) and put them into a tile of the output in LDS, which is
// then written as one contiguous run.  Plain softmax, where every logit has a
// gradient, first reads the tile's logits as one run and takes each row's
// statistics; the rows' walks start 8 columns apart so that the eight rows do
// not meet in the same LDS banks.
#include <algorithm>

#include "rowops.h"

namespace moe {
namespace {

constexpr int kTok = 8;       // tokens a wave
constexpr int kThreads = 64;  // a workgroup is one wave: its barriers cost nothing
constexpr int kMaxGrid = 1 << 20;

template <class V>
__device__ __forceinline__ V sum8(V v)
{
    v += __shfl_xor(v, 1, 64);
    v += __shfl_xor(v, 2, 64);
    v += __shfl_xor(v, 4, 64);
    return v;
}

template <class V>
__device__ __forceinline__ V max8(V v)
{
    v = fmax(v, __shfl_xor(v, 1, 64));
    v = fmax(v, __shfl_xor(v, 2, 64));
    return fmax(v, __shfl_xor(v, 4, 64));
}

// Calls f with the columns that lane j takes of its token's row: 8 q + j for q
// from tl on, around the end.
template <class F>
__device__ __forceinline__ void walk(int E, int tl, int j, F f)
{
    const int n = (E + 7) >> 3;
    int q = tl % n;
#pragma unroll 4
    for (int s = 0; s < n; ++s) {
        const int i = 8 * q + j;
        if (i < E) f(i);
        q = q + 1 == n ? 0 : q + 1;
    }
}

__global__ __launch_bounds__(kThreads) void route_backward_kernel(const float* __restrict__ logits,
                                                             const int32_t* __restrict__ ids,
                                                             const float* __restrict__ d_scales, int T, int E,
                                                             int method, int k, float scaling, bool whole,
                                                             bool aligned, float* __restrict__ d_logits)
{
    __shared__ __align__(16) float s_out[kTok * MOE_MAX_EXPERTS];
    const int lane = threadIdx.x & 63;
    const int tl = threadIdx.x >> 3, j = threadIdx.x & 7;
    const bool sigm = method == MOE_ROUTE_DEEPSEEKV3 || method == MOE_ROUTE_MINIMAX2 ||
                      method == MOE_ROUTE_SIGMOID_RENORM || method == MOE_ROUTE_LLAMA4;
    for (long t0 = (long)blockIdx.x * kTok; t0 < T; t0 += (long)gridDim.x * kTok) {
        const int nt = (int)min((long)kTok, T - t0);
        const long t = t0 + tl;
        int e = -1;
        double d = 0.0, l = 0.0;
        if (tl < nt && j < k) {
            e = ids[t * k + j];
            d = d_scales[t * k + j];
        }
        float* row = s_out + tl * E;
        // the tile: zeros, or its logits (t0 * E is a multiple of 4, so a run starts on a 16-byte boundary)
        const int n = nt * E;
        const float* in = logits + t0 * E;
        if (!whole || aligned) {
#pragma unroll 4
            for (int i = threadIdx.x; i < (n >> 2); i += kThreads)
                reinterpret_cast<float4*>(s_out)[i] =
                    whole ? reinterpret_cast<const float4*>(in)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i = (n & ~3) + threadIdx.x; i < n; i += kThreads) s_out[i] = whole ? in[i] : 0.0f;
        } else {
            for (int i = threadIdx.x; i < n; i += kThreads) s_out[i] = in[i];
        }
        if ((unsigned)e >= (unsigned)E) {  // a dropped pair
            e = -1;
            d = 0.0;
        }
        if (!whole && e >= 0) l = logits[t * E + e];
        double m = 0.0, rest = 0.0;  // maximum, and the sum of what is not kept
        if (whole) {
            // every expert once: the first of several pairs takes the others' gradients
            double sum = 0.0;
            bool first = true;
#pragma unroll
            for (int i = 0; i < MOE_MAX_TOPK; ++i) {
                const int ei = __shfl(e, (lane & ~7) | i, 64);
                const double di = __shfl(d, (lane & ~7) | i, 64);
                if (ei == e) {
                    sum += di;
                    first = first && i >= j;
                }
            }
            d = first ? sum : 0.0;
            e = first ? e : -1;
            __syncthreads();
            if (e >= 0) l = row[e];
            float mx = -INFINITY;
            if (tl < nt) walk(E, tl, j, [&](int i) { mx = fmaxf(mx, row[i]); });
            mx = max8(mx);
            m = mx;
            __syncthreads();
            if (e >= 0) row[e] = -INFINITY;  // the kept ones are added in fp64 below
            __syncthreads();
            float z = 0.0f;
            if (tl < nt)
                walk(E, tl, j, [&](int i) {
                    const float p = mx == -INFINITY ? 0.0f : expf(row[i] - mx);
                    row[i] = p;
                    z += p;
                });
            rest = sum8((double)z);
        } else if (!sigm) {
            m = max8(e >= 0 ? l : (double)-INFINITY);
        }
        double w = 0.0, slope = 1.0;  // the weight before division, and its own slope over itself
        if (e >= 0) {
            if (sigm) {
                const double x = exp(-fabs(l));
                w = l >= 0.0 ? 1.0 / (1.0 + x) : x / (1.0 + x);
                slope = l >= 0.0 ? x / (1.0 + x) : 1.0 / (1.0 + x);
            } else {
                w = m == -INFINITY ? 0.0 : exp(l - m);
            }
        }
        if (method == MOE_ROUTE_DEEPSEEKV3) rest = 1e-20;
        double v = 0.0, mean = 0.0;
        const double S = sum8(w) + rest;
        if (method == MOE_ROUTE_LLAMA4) {
            v = d * w * slope;
        } else {
            double a = rest * d;
#pragma unroll
            for (int i = 0; i < MOE_MAX_TOPK; ++i) {
                const double wi = __shfl(w, (lane & ~7) | i, 64), di = __shfl(d, (lane & ~7) | i, 64);
                a += wi * (d - di);
                mean += wi * di;
            }
            v = S > 0.0 ? w / S * slope * (a / S) : 0.0;
            mean = S > 0.0 ? mean / S / S : 0.0;
        }
        v *= scaling;
        // an expert listed twice gets the sum, written by both lanes
        double both = 0.0;
#pragma unroll
        for (int i = 0; i < MOE_MAX_TOPK; ++i) {
            const int ei = __shfl(e, (lane & ~7) | i, 64);
            const double vi = __shfl(v, (lane & ~7) | i, 64);
            if (ei == e) both += vi;
        }
        __syncthreads();
        if (whole && tl < nt) {
            const float f = (float)(-mean * scaling);
            walk(E, tl, j, [&](int i) { row[i] *= f; });
        }
        if (whole) __syncthreads();
        if (e >= 0) row[e] = (float)both;
        __syncthreads();
        float* out = d_logits + t0 * E;
        for (int i = threadIdx.x; i < (n >> 2); i += kThreads)
            reinterpret_cast<float4*>(out)[i] = reinterpret_cast<const float4*>(s_out)[i];
        for (int i = (n & ~3) + threadIdx.x; i < n; i += kThreads) out[i] = s_out[i];
        __syncthreads();
    }
}

}  // namespace

moe_status launch_route_backward(const float* logits, const int32_t* ids, const float* d_scales, int T, int E,
                                 int method, int k, float scaling, unsigned flags, float* d_logits,
                                 hipStream_t s)
{
    const bool whole = method == MOE_ROUTE_DEFAULT && !(flags & MOE_ROUTE_FLAG_RENORMALIZE);
    const int grid = (int)std::min(((long)T + kTok - 1) / kTok, (long)kMaxGrid);
    {
        TimedLaunch tl(MOE_KID_ROUTE_BWD, s);
        hipLaunchKernelGGL(route_backward_kernel, dim3(grid), dim3(kThreads), 0, s, logits, ids, d_scales, T, E, method,
                           k, scaling, whole, (reinterpret_cast<uintptr_t>(logits) & 15) == 0, d_logits);
    }
    return launch_status("route_backward_kernel");
}

}  // namespace moe

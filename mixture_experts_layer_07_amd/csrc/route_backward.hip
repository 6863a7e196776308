// moe_route_backward: the gradient of the routing weights.
//
// With a kept expert's unnormalised weight w (an exponential or a sigmoid), S
// the sum that divides the weights and d the incoming gradients, a renormalised
// weight's gradient and a plain softmax's are both
//     scaling * slope_j w_j / S * (d_j S - sum_i w_i d_i) / S
// where S holds the kept weights and, for plain softmax, the other experts'
// exponentials, for DeepSeek-V3 its 1e-20; slope is 1 for exponentials and
// 1 - sig for sigmoids.  The kept experts are computed in fp64, so that the
// difference keeps more digits than the output where one weight is near 1.
// The products of the difference are rounded alike (no fused multiply-add):
// one renormalised weight alone, which is constant, has gradient exactly 0.
//
// Latency-bound while small (8192 x 256, k = 8: 4.4 us in a captured graph; plain
// softmax 1021 x 65 5.6 us), then bound by the writes and by the lines that the
// kept logits are gathered from (65536 x 256: 24 us).  Plain softmax passes over
// its tile in LDS five times, with four waves a SIMD (108 registers) to hide it:
// 36 us, where its bytes take 26.  A wave
// owns eight tokens, eight lanes each: they compute the kept experts' gradients
// (an exponential and three divisions each; sums over a token's lanes by lane
// permutations) and put them into a tile of the output in LDS, which then goes
// out in whole rows.  Plain softmax, where every logit has a gradient, keeps
// the tile's logits there first and walks each row with its eight lanes.  The
// tile's rows are 8 floats longer than E so that the eight rows' walks meet
// different banks at E = 256.  A row's result does not depend on its place.
#include <algorithm>

#include "rowops.h"

namespace moe {
namespace {

constexpr int kTok = 8;       // tokens a wave
constexpr int kThreads = 64;  // a workgroup is one wave: its barriers cost nothing
constexpr int kMaxGrid = 1 << 20;

// The value of the lane that DPP control `ctrl` names.
template <int ctrl>
__device__ __forceinline__ double dpp_f64(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, ctrl, 0xf, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), ctrl, 0xf, 0xf, false);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Sums and maxima over aligned groups of 8 lanes, in every lane of them.
__device__ __forceinline__ double sum8(double v)
{
    v += dpp_f64<0xb1>(v);   // quad_perm [1,0,3,2]
    v += dpp_f64<0x4e>(v);   // quad_perm [2,3,0,1]
    v += dpp_f64<0x141>(v);  // row_half_mirror
    return v;
}

__device__ __forceinline__ float sum8(float v)
{
    v += dpp_f32<0xb1>(v);
    v += dpp_f32<0x4e>(v);
    v += dpp_f32<0x141>(v);
    return v;
}

__device__ __forceinline__ float max8(float v)
{
    v = fmaxf(v, dpp_f32<0xb1>(v));
    v = fmaxf(v, dpp_f32<0x4e>(v));
    return fmaxf(v, dpp_f32<0x141>(v));
}

// Calls f(tile index, output index) with the lane's elements of nt rows of E.
// W: floats at a time.
template <int W, class F>
__device__ __forceinline__ void rows_of(int nt, int E, int pitch, F f)
{
#pragma unroll
    for (int r = 0; r < kTok; ++r)
        if (r < nt)
            for (int c = (int)threadIdx.x * W; c < E; c += kThreads * W) f(r * pitch + c, r * E + c);
}

// WHOLE: plain softmax.  W: 4 where E and logits allow 16-byte accesses to the
// rows, else 1.
template <bool WHOLE, int W>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(const float* __restrict__ logits,
                                                                  const int32_t* __restrict__ ids,
                                                                  const float* __restrict__ d_scales, int T,
                                                                  int E, int method, int k, float scaling,
                                                                  float* __restrict__ d_logits)
{
#pragma clang fp contract(off)
    typedef float vec_t __attribute__((ext_vector_type(W)));
    __shared__ __align__(16) float s_out[kTok * (MOE_MAX_EXPERTS + 8)];
    const int lane = threadIdx.x;
    const int tl = lane >> 3, j = lane & 7, first_lane = lane & ~7;
    const int pitch = E + 8;
    float* row = s_out + tl * pitch;
    const bool sigm = method == MOE_ROUTE_DEEPSEEKV3 || method == MOE_ROUTE_MINIMAX2 ||
                      method == MOE_ROUTE_SIGMOID_RENORM || method == MOE_ROUTE_LLAMA4;
    for (long t0 = (long)blockIdx.x * kTok; t0 < T; t0 += (long)gridDim.x * kTok) {
        const int nt = (int)min((long)kTok, T - t0);
        const long t = t0 + tl;
        int e = -1;
        double d = 0.0;
        float l = -INFINITY;
        if (tl < nt && j < k) {
            e = ids[t * k + j];
            d = d_scales[t * k + j];
        }
        // the tile: the rows' logits, or zeros
        const float* in = logits + t0 * E;
        rows_of<W>(nt, E, pitch, [&](int s, int g) {
            *reinterpret_cast<vec_t*>(s_out + s) = WHOLE ? *reinterpret_cast<const vec_t*>(in + g) : vec_t(0.0f);
        });
        if ((unsigned)e >= (unsigned)E) {  // a dropped pair
            e = -1;
            d = 0.0;
        }
        if (!WHOLE && e >= 0) l = logits[t * E + e];
        // does a token list an expert twice?  (moe_route's ids do not.)  Every lane takes part in every
        // shuffle: a lane that is masked off has nothing to read
        bool again = false;
#pragma unroll
        for (int i = 0; i < MOE_MAX_TOPK; ++i) {
            const int other = __shfl(e, first_lane | i, 64);
            again |= i != j && e >= 0 && other == e;
        }
        const bool twice = __any(again);
        __syncthreads();
        double rest = 0.0;  // what S holds besides the kept weights
        float top = 0.0f;   // maximum logit
        if constexpr (WHOLE) {
            if (twice) {  // every expert once: the first of its pairs takes the others' gradients
                double sum = -0.0;  // a pair alone keeps its bits, the sign of a zero too
                bool first = true;
                for (int i = 0; i < MOE_MAX_TOPK; ++i) {
                    const int ei = __shfl(e, first_lane | i, 64);
                    const double di = __shfl(d, first_lane | i, 64);
                    if (ei == e) {
                        sum += di;
                        first = first && i >= j;
                    }
                }
                d = first ? sum : 0.0;
                e = first ? e : -1;
            }
            if (e >= 0) l = row[e];
            top = -INFINITY;
            if (tl < nt) {
#pragma unroll 8
                for (int i = j; i < E; i += 8) top = fmaxf(top, row[i]);
            }
            top = max8(top);
            __syncthreads();
            if (e >= 0) row[e] = -INFINITY;  // the kept ones are added in fp64 below
            __syncthreads();
            float z = 0.0f;
            if (tl < nt) {
#pragma unroll 8
                for (int i = j; i < E; i += 8) {
                    const float p = top == -INFINITY ? 0.0f : expf(row[i] - top);
                    row[i] = p;
                    z += p;
                }
            }
            rest = sum8(z);
        } else if (!sigm) {
            top = max8(l);
        }
        double w = 0.0, slope = 1.0;
        if (e >= 0) {
            if (sigm) {
                const double x = exp(-fabs((double)l)), y = 1.0 / (1.0 + x);
                w = l >= 0.0f ? y : x * y;
                slope = l >= 0.0f ? x * y : y;
            } else {
                w = top == -INFINITY ? 0.0 : exp((double)l - top);
            }
        }
        if (method == MOE_ROUTE_DEEPSEEKV3) rest = 1e-20;
        const double S = sum8(w) + rest, wd = sum8(w * d);
        double v;
        if (method == MOE_ROUTE_LLAMA4) v = w * slope * d;
        else v = S > 0.0 ? w / S * slope * ((S * d - wd) / S) : 0.0;
        v *= scaling;
        if constexpr (WHOLE) {
            const float f = S > 0.0 ? (float)(wd / S / S * -scaling) : 0.0f;
            if (tl < nt) {
#pragma unroll 8
                for (int i = j; i < E; i += 8) row[i] *= f;
            }
            __syncthreads();
        } else if (twice) {  // both lanes write the sum
            double both = -0.0;
            for (int i = 0; i < MOE_MAX_TOPK; ++i) {
                const int ei = __shfl(e, first_lane | i, 64);
                const double vi = __shfl(v, first_lane | i, 64);
                if (ei == e) both += vi;
            }
            v = both;
        }
        if (e >= 0) row[e] = (float)v;
        __syncthreads();
        float* out = d_logits + t0 * E;
        rows_of<W>(nt, E, pitch, [&](int s, int g) {
            *reinterpret_cast<vec_t*>(out + g) = *reinterpret_cast<const vec_t*>(s_out + s);
        });
        __syncthreads();
    }
}

}  // namespace

moe_status launch_route_backward(const float* logits, const int32_t* ids, const float* d_scales, int T, int E,
                                 int method, int k, float scaling, unsigned flags, float* d_logits,
                                 hipStream_t s)
{
    const bool whole = method == MOE_ROUTE_DEFAULT && !(flags & MOE_ROUTE_FLAG_RENORMALIZE);
    const bool wide = E % 4 == 0 && !(whole && (reinterpret_cast<uintptr_t>(logits) & 15));
    auto* kernel = whole ? (wide ? route_backward_kernel<true, 4> : route_backward_kernel<true, 1>)
                         : (wide ? route_backward_kernel<false, 4> : route_backward_kernel<false, 1>);
    const int grid = (int)std::min(((long)T + kTok - 1) / kTok, (long)kMaxGrid);
    {
        TimedLaunch tl(MOE_KID_ROUTE_BWD, s);
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), 0, s, logits, ids, d_scales, T, E, method, k, scaling,
                           d_logits);
    }
    return launch_status("route_backward_kernel");
}

}  // namespace moe

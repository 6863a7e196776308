// moe_route kernel: one 64-lane wavefront per token.
//
// Methods (TensorRT-LLM page "MoE 层前向执行", sections "路由方法枚举" and
// "DeepSeek-V3 的 noaux_tc"; vLLM page, section "FusedTopKRouter"):
//   Default            softmax over all E, keep top-k (optionally renormalised)
//   Renormalize        top-k, then softmax over the k kept logits
//   RenormalizeNaive   softmax, top-k, renormalise (same values as above)
//   DeepSeekV3         sigmoid scores; bias added for selection only; group
//                      score = sum of the group's two best biased keys; keep
//                      topk_group groups; top-k experts among them; weights
//                      = unbiased sigmoid / (sum + 1e-20) * scaling.
//   Llama4             top-k logits, each weighted by its own sigmoid
//   MiniMax2           sigmoid + bias for selection, top-k, unbiased sigmoids
//                      renormalised (DeepSeekV3 with one group, no 1e-20)
//   SigmoidRenorm      sigmoid, top-k, renormalise
//
// The selection itself is route_token in route.h.
#include "route.h"

namespace moe {
namespace {

constexpr int kWaves = 4;  // tokens per 256-thread block

__global__ __launch_bounds__(256) void route_kernel(RouteArgs a, int32_t* __restrict__ ids,
                                                    float* __restrict__ scales)
{
    __shared__ RouteLds s[kWaves];
    const int wave = threadIdx.x >> 6;
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * kWaves + wave;
    if (t >= a.T) return;  // a wave's LDS is its own: nothing waits for it
    float logit[4], scale;
    int id;
    load_logits(a, t, lane, logit);
    route_token<true>(a, logit, lane, s[wave], id, scale);
    if (lane < a.k) {
        ids[(size_t)t * a.k + lane] = id;
        scales[(size_t)t * a.k + lane] = scale;
    }
}

}  // namespace

moe_status launch_route(const float* logits, int T, int E, int method, int k, int n_group,
                        int topk_group, const float* bias, float scaling, unsigned flags,
                        int32_t* ids, float* scales, hipStream_t s)
{
    const int blocks = (T + kWaves - 1) / kWaves;
    const RouteArgs a{logits, bias, T, E, method, k, n_group, topk_group, scaling, flags};
    {
        TimedLaunch tl(MOE_KID_ROUTE, s);
        hipLaunchKernelGGL(route_kernel, dim3(blocks), dim3(256), 0, s, a, ids, scales);
    }
    return launch_status("route_kernel");
}

}  // namespace moe

// moe_quantize_mxfp4, moe_dequantize_mxfp4: rows of values to microscaled 4-bit
// codes and back.  The quantise-input step of the TensorRT-LLM page
// ("“自适应顺序”里的一个细节") in the 4-bit form that its fused backends read
// ("后端的三种形态与两个调度器家族"), with the scales of the OCP format.
//
// Memory-bound: 2 or 4 bytes a value on one side, 17/32 on the other.  Blocks of
// a row are consecutive and rows are dense, so block b of the whole array is
// values 32 b .. 32 b + 31 whatever the shape.  A thread takes 16 bytes of values
// (8 bf16 or 4 fp32), so 4 or 8 neighbouring lanes share a block and its largest
// magnitude goes round by lane permutations.  4096 x 7168 fp32 (133 MB each way):
// quantised in 25.1 us (5.3 TB/s), back in 18.3 (7.3, a part of the writes still in the
// memory-side cache); one bf16 row of 7168 in 1.9 and 1.8 us, where the calls take 4 each.
#include <algorithm>

#include "mxfp4.h"
#include "rowops.h"

namespace moe {
namespace {

template <int ctrl>
__device__ __forceinline__ uint32_t dpp_max_u32(uint32_t v)
{
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, ctrl, 0xf, 0xf, false);
    return o > v ? o : v;
}

template <class T, bool NT>
__global__ __launch_bounds__(256) void quantize_mxfp4_kernel(const T* __restrict__ x, long nchunks,
                                                             uint8_t* __restrict__ q, uint8_t* __restrict__ scale)
{
    constexpr int V = Raw<T>::kValues;  // values a thread
    constexpr int L = 32 / V;           // lanes a block
    // nchunks and the stride are multiples of L: a block's lanes leave together
    for (long c = (long)blockIdx.x * 256 + threadIdx.x; c < nchunks; c += (long)gridDim.x * 256) {
        Raw<T> r;
        r.template load<NT>(x + c * V);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(r[i]) & 0x7fffffffu);
        m = dpp_max_u32<0xb1>(m);                         // quad_perm [1,0,3,2]
        m = dpp_max_u32<0x4e>(m);                         // quad_perm [2,3,0,1]
        if constexpr (L == 8) m = dpp_max_u32<0x141>(m);  // row_half_mirror
        const uint32_t s = mxfp4_scale(m);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < V ? r[i % V] : 0.0f;
        const uint32_t w = mxfp4_codes(v, s);
        if constexpr (V == 8) *reinterpret_cast<uint32_t*>(q + c * 4) = w;
        else *reinterpret_cast<uint16_t*>(q + c * 2) = (uint16_t)w;
        if (threadIdx.x % L == 0) scale[c / L] = (uint8_t)s;
    }
}

template <class T, bool NT>
__global__ __launch_bounds__(256) void dequantize_mxfp4_kernel(const uint8_t* __restrict__ q,
                                                               const uint8_t* __restrict__ scale, long nchunks,
                                                               T* __restrict__ x)
{
    constexpr int V = Raw<T>::kValues;
    constexpr int L = 32 / V;
    for (long c = (long)blockIdx.x * 256 + threadIdx.x; c < nchunks; c += (long)gridDim.x * 256) {
        const uint32_t s = scale[c / L];
        Raw<T> r;
        if constexpr (V == 8) {
            r.w = mxfp4_to_bf16x8(*reinterpret_cast<const uint32_t*>(q + c * 4), s);
        } else {
            typedef float f32x2_t __attribute__((ext_vector_type(2)));
            const uint32_t w = *reinterpret_cast<const uint16_t*>(q + c * 2);
            const float f = __uint_as_float(s << 23);
            const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, f, 0);
            const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, f, 1);
            const float v[4] = {a.x, a.y, b.x, b.y};
            r.set(v);
        }
        r.template store<NT>(x + c * V);
    }
}

// One thread for each 16 bytes of values (a launch holds less than 2^32 threads: past
// 2^31 they loop); past kStream bytes of them the hinted form.
template <class T, class F>
moe_status for_chunks(long n, const char* what, F launch)
{
    const long nchunks = n / Raw<T>::kValues;
    const long grid = std::min((nchunks + 255) / 256, 1l << 23);
    launch(dim3((unsigned)grid), nchunks, n * (long)sizeof(T) > kStream);
    return launch_status(what);
}

template <class T>
moe_status quantize(const T* x, long n, uint8_t* q, uint8_t* scale, hipStream_t s)
{
    return for_chunks<T>(n, "quantize_mxfp4_kernel", [&](dim3 grid, long nchunks, bool nt) {
        TimedLaunch tl(MOE_KID_QUANT_MXFP4, s);
        auto kern = nt ? quantize_mxfp4_kernel<T, true> : quantize_mxfp4_kernel<T, false>;
        hipLaunchKernelGGL(kern, grid, dim3(256), 0, s, x, nchunks, q, scale);
    });
}

template <class T>
moe_status dequantize(const uint8_t* q, const uint8_t* scale, long n, T* x, hipStream_t s)
{
    return for_chunks<T>(n, "dequantize_mxfp4_kernel", [&](dim3 grid, long nchunks, bool nt) {
        TimedLaunch tl(MOE_KID_DEQUANT_MXFP4, s);
        auto kern = nt ? dequantize_mxfp4_kernel<T, true> : dequantize_mxfp4_kernel<T, false>;
        hipLaunchKernelGGL(kern, grid, dim3(256), 0, s, q, scale, nchunks, x);
    });
}

}  // namespace

moe_status launch_quantize_mxfp4(const void* x, int dt, int rows, int cols, uint8_t* q, uint8_t* scale,
                                 hipStream_t s)
{
    const long n = (long)rows * cols;
    if (dt == MOE_BF16) return quantize(static_cast<const bf16_t*>(x), n, q, scale, s);
    return quantize(static_cast<const float*>(x), n, q, scale, s);
}

moe_status launch_dequantize_mxfp4(const uint8_t* q, const uint8_t* scale, int rows, int cols, int dt, void* x,
                                   hipStream_t s)
{
    const long n = (long)rows * cols;
    if (dt == MOE_BF16) return dequantize(q, scale, n, static_cast<bf16_t*>(x), s);
    return dequantize(q, scale, n, static_cast<float*>(x), s);
}

}  // namespace moe

// Device helpers of the row operators (norm, dispatch, activation and the
// gradients): 8-value chunks of a row, sums over lanes, 1x128 e4m3 blocks.
#pragma once

#include "common.h"

namespace moe {
namespace {

// Calls that move more bytes than this stream past the caches: loads and
// stores carry the non-temporal hint (template argument NT).  Plain / hinted,
// inputs and outputs of three calls in turn: rmsnorm 66 MB 11.7 / 14.3 us, 132
// MB 28.6 / 26.1 us, 528 MB 94.6 / 84.4 us; finalize_backward 84 MB 16.6 / 20.1
// us, 125 MB 30.9 / 27.4 us, 1.0 GB 104.6 / 96.0 us; swiglu_backward 170 MB
// 60.0 / 55.7 us with its forward call.  With a producer before it and a
// quantiser that reads y after it, rmsnorm gains as well at 528 MB (165.6 ->
// 156.2 us for the three) and loses nothing below.
constexpr long kStream = 96l << 20;

// 8 consecutive values of a row as raw 16-byte words (bf16: one, fp32: two),
// widened to fp32 only where they are used.
template <class T>
struct Raw8 {
    static constexpr int W = sizeof(T) / 2;
    u32x4_t w[W];
    template <bool NT = false>
    __device__ __forceinline__ void load(const T* p)
    {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const u32x4_t* q = reinterpret_cast<const u32x4_t*>(reinterpret_cast<const char*>(p) + 16 * i);
            w[i] = NT ? __builtin_nontemporal_load(q) : *q;
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = u32x4_t{0, 0, 0, 0};
    }
    __device__ __forceinline__ float operator[](int i) const
    {
        if constexpr (W == 1) {
            const uint32_t u = w[0][i >> 1];
            return __uint_as_float((i & 1) ? (u & 0xffff0000u) : (u << 16));
        } else {
            return __uint_as_float(w[i >> 2][i & 3]);
        }
    }
    __device__ __forceinline__ void set(const float v[8])
    {
        if constexpr (W == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[0][i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i >> 2][i & 3] = __float_as_uint(v[i]);
        }
    }
    template <bool NT = false>
    __device__ __forceinline__ void store(T* p) const
    {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            u32x4_t* q = reinterpret_cast<u32x4_t*>(reinterpret_cast<char*>(p) + 16 * i);
            if constexpr (NT) __builtin_nontemporal_store(w[i], q);
            else *q = w[i];
        }
    }
};

template <int ctrl>
__device__ __forceinline__ float dpp_f32(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), ctrl, 0xf, 0xf, false));
}

// Sum over each aligned group of 16 lanes, in every lane of it: pairs, quads,
// half-rows and rows by lane permutations inside the vector unit.
__device__ __forceinline__ float sum16(float v)
{
    v += dpp_f32<0xb1>(v);   // quad_perm [1,0,3,2]
    v += dpp_f32<0x4e>(v);   // quad_perm [2,3,0,1]
    v += dpp_f32<0x141>(v);  // row_half_mirror
    v += dpp_f32<0x140>(v);  // row_mirror
    return v;
}

__device__ __forceinline__ float max16(float v)
{
    v = fmaxf(v, dpp_f32<0xb1>(v));
    v = fmaxf(v, dpp_f32<0x4e>(v));
    v = fmaxf(v, dpp_f32<0x141>(v));
    v = fmaxf(v, dpp_f32<0x140>(v));
    return v;
}

__device__ __forceinline__ float wave_sum_f32(float v)
{
    v = sum16(v);
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
    return v;
}

__device__ __forceinline__ float absmax8(const float v[8])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
}

// fl32(v / s) from r = fl32(1 / s): the product v r is within two units in the
// last place, one correction by the exact residual makes it the quotient or a
// neighbour, and a second one rounds it correctly (Markstein's theorem on
// quotients from correctly rounded reciprocals).  The sign is v's also where
// the result is zero.
__device__ __forceinline__ float quotient(float v, float s, float r)
{
    float q = v * r;
    q = __builtin_fmaf(__builtin_fmaf(-q, s, v), r, q);
    q = __builtin_fmaf(__builtin_fmaf(-q, s, v), r, q);
    return __builtin_copysignf(q, v);
}

// Eight values -> their e4m3 codes with block scale s = fl32(amax / 448), the
// codes that fp8x4_code gives (fl32(v / s) rounded to nearest even).  One
// reciprocal a block instead of a division a value, where no residual can
// underflow (s >= 2^-60: a value that does not round to zero has |v| >= 2^-70,
// so its residual is a multiple of 2^-118) and nothing overflows; the quotient
// is then at most 448 (1 + 2^-23), which needs no clamp.  The activation with
// its checkpoint: 222 -> 219 us alone, 222 -> 188 us with the narrow
// workgroups and hinted stores of swiglu.hip.
__device__ __forceinline__ uint2 fp8x8_code(const float v[8], float s)
{
    if (s >= 0x1p-60f && s <= 0x1p+100f) {
        const float r = 1.0f / s;
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = quotient(v[i], s, r);
        int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
        int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
        return make_uint2((uint32_t)lo, (uint32_t)hi);
    }
    const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
    return make_uint2(fp8x4_code(lo, s), fp8x4_code(hi, s));
}

// v = code * scale of eight e4m3 codes.
__device__ __forceinline__ void fp8x8_value(uint2 q, float s, float v[8])
{
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
        const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        v[4 * i] = a.x * s;
        v[4 * i + 1] = a.y * s;
        v[4 * i + 2] = b.x * s;
        v[4 * i + 3] = b.y * s;
    }
}

}  // namespace
}  // namespace moe

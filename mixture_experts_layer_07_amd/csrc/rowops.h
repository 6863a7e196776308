// Device helpers of the row operators (norm, dispatch, activation and the
// gradients): 16-byte chunks of a row, sums over lanes, 1x128 e4m3 blocks.
#pragma once

#include "common.h"

namespace moe {
namespace {

// Calls that move more bytes than this stream past the caches: loads and
// stores carry the non-temporal hint (template argument NT).  Plain / hinted,
// the inputs and outputs of three calls in turn:
//   rmsnorm            66 MB 11.9 / 14.4 us   132 MB 28.6 / 26.1   528 MB 93.9 / 84.2
//   its gradients      59 MB 17.6 / 19.1      235 MB 52.7 / 47.2   470 MB 94.3 / 84.1
//   finalize_backward  62 MB 12.2 / 13.7      125 MB 28.2 / 27.4   2.1 GB 410 / 385
//   swiglu + gradient  152 MB 32.4 / 26.3     304 MB 56.1 / 51.5   2.7 GB 466 / 460
// With a producer of x before it and a quantiser that reads y after it, rmsnorm
// gains as well at 528 MB (165.6 -> 156.2 us for the three).
constexpr long kStream = 96l << 20;

// V consecutive values of a row as raw words, widened to fp32 only where they
// are used.  A lane takes 16 bytes at a time, 8 bf16 or 4 fp32 values, so that
// a wave's access is one contiguous kilobyte (8 fp32 values a lane made each
// store half lines: swiglu_backward of 16384 x 2048 fp32 160 us against 106
// without the hint).  Where bf16 and fp32 rows meet, both take 4 values.
template <class T, int V = 16 / (int)sizeof(T)>
struct Raw {
    static constexpr int kValues = V, W = V * (int)sizeof(T) / 4;
    typedef uint32_t words_t __attribute__((ext_vector_type(W)));
    words_t w;
    template <bool NT = false>
    __device__ __forceinline__ void load(const T* p)
    {
        const words_t* q = reinterpret_cast<const words_t*>(p);
        if constexpr (NT) w = __builtin_nontemporal_load(q);
        else w = *q;
    }
    __device__ __forceinline__ void zero() { w = words_t(0u); }
    __device__ __forceinline__ float operator[](int i) const
    {
        if constexpr (sizeof(T) == 2) {
            const uint32_t u = w[i >> 1];
            return __uint_as_float((i & 1) ? (u & 0xffff0000u) : (u << 16));
        } else {
            return __uint_as_float(w[i]);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[V])
    {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(v[i]);
        }
    }
    template <bool NT = false>
    __device__ __forceinline__ void store(T* p) const
    {
        words_t* q = reinterpret_cast<words_t*>(p);
        if constexpr (NT) __builtin_nontemporal_store(w, q);
        else *q = w;
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

// Maximum, NaN if either is (fmaxf would drop it): one v_maximum3_f32.
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

__device__ __forceinline__ float max16(float v)
{
    v = max_nan(v, dpp_f32<0xb1>(v));
    v = max_nan(v, dpp_f32<0x4e>(v));
    v = max_nan(v, dpp_f32<0x141>(v));
    v = max_nan(v, dpp_f32<0x140>(v));
    return v;
}

__device__ __forceinline__ float wave_sum_f32(float v)
{
    v = sum16(v);
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
    return v;
}

// Maximum of |v| over a 1x128 block, V values a lane: 128 / V consecutive lanes.
// NaN if the block holds one: its scale is then NaN and no code of it stands for
// a finite value (a block of NaN alone would otherwise have scale 0 and pass for
// zeros).
template <int V>
__device__ __forceinline__ float block_absmax(const float (&v)[V])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) m = max_nan(m, fabsf(v[i]));
    m = max16(m);
    if constexpr (V == 4) m = max_nan(m, __shfl_xor(m, 16, 64));
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

// V values -> their e4m3 codes with block scale s = fl32(amax / 448), stored at
// q: the codes that fp8x4_code gives (fl32(v / s) rounded to nearest even).  One
// reciprocal a block instead of a division a value, where no residual can
// underflow (s >= 2^-60: a value that does not round to zero has |v| >= 2^-70,
// so its residual is a multiple of 2^-118) and nothing overflows; the quotient
// is then at most 448 (1 + 2^-23), which needs no clamp.  A scale that is
// infinite or NaN takes the other branch.  swiglu with a
// checkpoint of 73728 x 2048: 210 -> 191 us against a division a value.
template <int V>
__device__ __forceinline__ void store_codes(const float (&v)[V], float s, uint8_t* q)
{
    typedef uint32_t words_t __attribute__((ext_vector_type(V / 4)));
    words_t w;
    if (s >= 0x1p-60f && s <= 0x1p+100f) {
        const float r = 1.0f / s;
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            int c = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[4 * i], s, r), quotient(v[4 * i + 1], s, r), 0, false);
            c = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[4 * i + 2], s, r), quotient(v[4 * i + 3], s, r), c, true);
            w[i] = (uint32_t)c;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float f[4] = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
            w[i] = fp8x4_code(f, s);
        }
    }
    *reinterpret_cast<words_t*>(q) = w;
}

// v = code * scale of the V e4m3 codes at q.
template <int V>
__device__ __forceinline__ void load_codes(const uint8_t* q, float s, float (&v)[V])
{
    typedef uint32_t words_t __attribute__((ext_vector_type(V / 4)));
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    const words_t w = *reinterpret_cast<const words_t*>(q);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
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

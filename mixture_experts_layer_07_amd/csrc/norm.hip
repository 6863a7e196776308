// moe_rmsnorm and its gradients.
//
//     z = x (+ residual, rounded),  c = 1 / sqrt(mean(z^2) + eps),  y = z c w
//     g = dy w,  dz = c g - z c^3 mean(g z) (+ dtotal),  dw = sum_t dy z c
//
// A row stays in registers between its reduction and its outputs, so every
// array is read and written once.  A wave owns a row of up to 2048 values,
// a workgroup a longer one; a thread holds NV chunks of 8 consecutive values
// at chunk indices tid, tid + stride, ...
#include <algorithm>

#include "rowops.h"

namespace moe {
namespace {

constexpr int kMaxWaves = 8;
constexpr int kPartials = 512;  // most partial rows of dweight (sets the workspace's size)

// Sums of N values over the row's threads: one wave, or the workgroup through
// LDS.  `buf` alternates between two halves on consecutive calls, so one
// barrier a call is enough.
template <bool WAVE, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*s)[kMaxWaves][N], int& buf)
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum_f32(v[i]);
    if constexpr (!WAVE) {
        const int nw = blockDim.x >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) s[buf][threadIdx.x >> 6][i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float a = 0.0f;
            for (int w = 0; w < nw; ++w) a += s[buf][w][i];
            v[i] = a;
        }
        buf ^= 1;
    }
}

// No __restrict__: total and y may be x or residual.
template <class T, int NV, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 512) void rmsnorm_kernel(const T* x, const T* residual, const T* weight,
                                                       int rows, int H, float eps, T* total, T* y,
                                                       uint8_t* yq, float* y_scale)
{
    __shared__ float s_sum[2][kMaxWaves][1];
    int buf = 0;
    const int tid = WAVE ? (threadIdx.x & 63) : threadIdx.x;
    const int stride = WAVE ? 64 : blockDim.x;
    const int per = WAVE ? (blockDim.x >> 6) : 1;  // rows a workgroup takes at a time
    const int nch = H >> 3;
    const float inv = 1.0f / (float)H;
    for (long row = (long)blockIdx.x * per + (WAVE ? threadIdx.x >> 6 : 0); row < rows;
         row += (long)gridDim.x * per) {
        const size_t r0 = (size_t)row * H;
        Raw8<T> a[NV], b[NV], w[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * stride;
            a[i].zero();
            b[i].zero();
            w[i].zero();
            if (c < nch) {
                a[i].load(x + r0 + 8 * c);
                if (residual) b[i].load(residual + r0 + 8 * c);
                w[i].load(weight + 8 * c);
            }
        }
        float sum[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (residual) {
                float z[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = a[i][e] + b[i][e];
                a[i].set(z);  // the norm is taken of the stored sum
                const int c = tid + i * stride;
                if (c < nch) a[i].store(total + r0 + 8 * c);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[0] += a[i][e] * a[i][e];
        }
        row_sum<WAVE, 1>(sum, s_sum, buf);
        const float cn = rsqrtf(sum[0] * inv + eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * stride;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = a[i][e] * cn * w[i][e];
            if (y && c < nch) {
                Raw8<T> o;
                o.set(v);
                o.store(y + r0 + 8 * c);
            }
            if (yq) {  // H is a multiple of 128: the 16 lanes of a block are in or out together
                const float s = max16(absmax8(v)) / 448.0f;
                if (c < nch) {
                    *reinterpret_cast<uint2*>(yq + r0 + 8 * c) = fp8x8_code(v, s);
                    if ((c & 15) == 0) y_scale[(r0 >> 7) + (c >> 4)] = s;
                }
            }
        }
    }
}

// Workgroup b takes rows b, b + grid, ... and adds its rows' dy z c in
// registers; its sum is one row of `part`.
template <class T, int NV, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 512) void rmsnorm_backward_kernel(
    const T* dy, const T* z, const T* weight, const T* dtotal, int rows, int H, float eps, T* dz,
    float* __restrict__ part)
{
    __shared__ float s_sum[2][kMaxWaves][2];
    __shared__ float s_dw[WAVE ? 4 : 1][WAVE ? 512 * NV : 1];
    int buf = 0;
    const int wave = threadIdx.x >> 6;
    const int tid = WAVE ? (threadIdx.x & 63) : threadIdx.x;
    const int stride = WAVE ? 64 : blockDim.x;
    const int per = WAVE ? (blockDim.x >> 6) : 1;
    const int nch = H >> 3;
    const float inv = 1.0f / (float)H;
    Raw8<T> w[NV];
    float dw[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tid + i * stride;
        w[i].zero();
        if (c < nch) w[i].load(weight + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
    }
    for (long row = (long)blockIdx.x * per + (WAVE ? wave : 0); row < rows; row += (long)gridDim.x * per) {
        const size_t r0 = (size_t)row * H;
        Raw8<T> a[NV], g[NV], d[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * stride;
            a[i].zero();
            g[i].zero();
            d[i].zero();
            if (c < nch) {
                a[i].load(z + r0 + 8 * c);
                g[i].load(dy + r0 + 8 * c);
                if (dtotal) d[i].load(dtotal + r0 + 8 * c);
            }
        }
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sum[0] += a[i][e] * a[i][e];
                sum[1] += g[i][e] * w[i][e] * a[i][e];
            }
        row_sum<WAVE, 2>(sum, s_sum, buf);
        const float cn = rsqrtf(sum[0] * inv + eps);
        const float m = sum[1] * inv * cn * cn * cn;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * stride;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = cn * (g[i][e] * w[i][e]) - a[i][e] * m + d[i][e];
                dw[i][e] += g[i][e] * (a[i][e] * cn);
            }
            if (c < nch) {
                Raw8<T> o;
                o.set(v);
                o.store(dz + r0 + 8 * c);
            }
        }
    }
    float* out = part + (size_t)blockIdx.x * H;
    if constexpr (WAVE) {  // the four waves' sums, in order
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s_dw[wave][8 * (tid + 64 * i) + e] = dw[i][e];
        __syncthreads();
        for (int h = threadIdx.x; h < H; h += blockDim.x) {
            float v = 0.0f;
            for (int k = 0; k < per; ++k) v += s_dw[k][h];
            out[h] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * stride;
            if (c < nch) store8_f32(out + 8 * c, dw[i]);
        }
    }
}

// dweight[h] = sum over n rows of part: 32 columns a workgroup, 32 threads a
// column, each a run of rows; the runs' sums are added in order.
__global__ __launch_bounds__(1024) void rmsnorm_dweight_kernel(const float* __restrict__ part, int n, int H,
                                                               float* __restrict__ dweight)
{
    __shared__ float s[32][33];
    const int col = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int h = blockIdx.x * 32 + col;
    const int len = (n + 31) / 32;
    float v = 0.0f;
    if (h < H) {
        const int r1 = min(n, (run + 1) * len);
#pragma unroll 8
        for (int r = run * len; r < r1; ++r) v += part[(size_t)r * H + h];
    }
    s[run][col] = v;
    __syncthreads();
    if (threadIdx.x < 32 && h < H) {
        float a = 0.0f;
#pragma unroll
        for (int r = 0; r < 32; ++r) a += s[r][col];
        dweight[h] = a;
    }
}

struct Shape {
    bool wave;    // a wave a row, else a workgroup
    int threads;  // of a workgroup
    int nv;       // chunks a thread: 1, 2 or 4
    int per;      // rows a workgroup takes at a time
};

Shape shape_of(int H)
{
    const int nch = H / 8;
    Shape s;
    s.wave = nch <= 256;
    s.threads = s.wave ? 256 : nch <= 1024 ? 256 : 512;
    const int each = (nch + (s.wave ? 64 : s.threads) - 1) / (s.wave ? 64 : s.threads);
    s.nv = each <= 1 ? 1 : each <= 2 ? 2 : 4;
    s.per = s.wave ? 4 : 1;
    return s;
}

template <class T, int NV, bool WAVE>
void launch_fwd(const Shape& sh, int grid, const void* x, const void* residual, const void* weight, int T_,
                int H, float eps, void* total, void* y, uint8_t* yq, float* ys, hipStream_t s)
{
    hipLaunchKernelGGL((rmsnorm_kernel<T, NV, WAVE>), dim3(grid), dim3(sh.threads), 0, s,
                       static_cast<const T*>(x), static_cast<const T*>(residual),
                       static_cast<const T*>(weight), T_, H, eps, static_cast<T*>(total),
                       static_cast<T*>(y), yq, ys);
}

template <class T, int NV, bool WAVE>
void launch_bwd(const Shape& sh, int grid, const void* dy, const void* z, const void* weight,
                const void* dtotal, int T_, int H, float eps, void* dz, float* part, hipStream_t s)
{
    hipLaunchKernelGGL((rmsnorm_backward_kernel<T, NV, WAVE>), dim3(grid), dim3(sh.threads), 0, s,
                       static_cast<const T*>(dy), static_cast<const T*>(z), static_cast<const T*>(weight),
                       static_cast<const T*>(dtotal), T_, H, eps, static_cast<T*>(dz), part);
}

// Calls f with T, NV and WAVE as template arguments.
#define MOE_NORM_SHAPE(T, f, ...)                                                       \
    do {                                                                                \
        if (sh.wave) {                                                                  \
            if (sh.nv == 1) f<T, 1, true>(__VA_ARGS__);                                 \
            else if (sh.nv == 2) f<T, 2, true>(__VA_ARGS__);                            \
            else f<T, 4, true>(__VA_ARGS__);                                            \
        } else {                                                                        \
            if (sh.nv == 2) f<T, 2, false>(__VA_ARGS__);                                \
            else f<T, 4, false>(__VA_ARGS__);                                           \
        }                                                                               \
    } while (0)

int partials(int T, int H)
{
    const Shape sh = shape_of(H);
    return std::min((T + sh.per - 1) / sh.per, kPartials);
}

}  // namespace

size_t rmsnorm_backward_scratch_bytes(int T, int H) { return (size_t)partials(T, H) * H * sizeof(float); }

moe_status launch_rmsnorm(const void* x, const void* residual, const void* weight, int dt, int T, int H,
                          float eps, void* total, void* y, uint8_t* yq, float* y_scale, hipStream_t s)
{
    const Shape sh = shape_of(H);
    const int grid = std::min((T + sh.per - 1) / sh.per, 1 << 20);
    {
        TimedLaunch tl(MOE_KID_RMSNORM, s);
        if (dt == MOE_BF16)
            MOE_NORM_SHAPE(bf16_t, launch_fwd, sh, grid, x, residual, weight, T, H, eps, total, y, yq, y_scale, s);
        else
            MOE_NORM_SHAPE(float, launch_fwd, sh, grid, x, residual, weight, T, H, eps, total, y, yq, y_scale, s);
    }
    return launch_status("rmsnorm_kernel");
}

moe_status launch_rmsnorm_backward(const void* dy, const void* z, const void* weight, const void* dtotal,
                                   int dt, int T, int H, float eps, void* dz, float* dweight, void* ws,
                                   hipStream_t s)
{
    const int n = T ? partials(T, H) : 0;
    float* part = static_cast<float*>(ws);
    if (n > 0) {
        const Shape sh = shape_of(H);
        TimedLaunch tl(MOE_KID_RMSNORM_BWD, s);
        if (dt == MOE_BF16)
            MOE_NORM_SHAPE(bf16_t, launch_bwd, sh, n, dy, z, weight, dtotal, T, H, eps, dz, part, s);
        else
            MOE_NORM_SHAPE(float, launch_bwd, sh, n, dy, z, weight, dtotal, T, H, eps, dz, part, s);
    }
    {
        TimedLaunch tl(MOE_KID_RMSNORM_DWEIGHT, s);
        hipLaunchKernelGGL(rmsnorm_dweight_kernel, dim3((H + 31) / 32), dim3(1024), 0, s, part, n, H, dweight);
    }
    return launch_status("rmsnorm_backward_kernel");
}

}  // namespace moe

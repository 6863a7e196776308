// moe_rmsnorm and its gradients.
//
//     z = x (+ residual, rounded),  c = 1 / sqrt(mean(z^2) + eps),  n = z c,  y = n w
//     g = dy w,  dz = c (g - n mean(g n)) (+ dtotal),  dw = sum_t dy n
//
// Bound by memory: a row stays in registers between its reduction and its
// outputs, so every array is read and written once.  (The gradients of fp32 rows
// wider than 8192 hold more than fits: 30 registers of a lane go out to scratch
// memory and come back.)  A wave or, for longer rows, a workgroup owns a row; a
// thread holds NV 16-byte chunks of V consecutive values at chunk indices tid,
// tid + stride, ...
//
// Measured on MI355X (8192 x 7168 bf16; a copy moves 5.1 TB/s, 6.5 at best):
//   forward with residual, y and codes  84 us, 6.3 TB/s.  Two chunks a thread:
//     one 91 us, four 85 us.
//   backward with dtotal  84 us, 5.6 TB/s (the kernel 79 us, the sum of the
//     partial rows 5 us).  256 or 1024 partial rows instead of 512: 104 / 90 us;
//     two chunks a thread 85 us, one 104 us; the next row's loads in flight over
//     the reduction 85-105 us (registers), kept only where a row is a chunk a
//     lane.
//   backward of 2048 x 16384 fp32 with dtotal, which spills  103 us, 5.2 TB/s
//     (2048 x 8192 fp32 48 us, 5.6 TB/s).
//   one token 5.0 us a call, the kernel 3.4 in a captured graph; the gradients of
//   63 x 256 fp32 5.2 us, the kernel 4.9.
#include <algorithm>

#include "rowops.h"

namespace moe {
namespace {

constexpr int kMaxWaves = 16;
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

template <int V>
__device__ __forceinline__ void store_f32(float* p, const float (&v)[V])
{
#pragma unroll
    for (int i = 0; i < V; i += 4)
        *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}

// No __restrict__: total and y may be x or residual.
template <class T, int NV, bool WAVE, bool NT>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void rmsnorm_kernel(const T* x, const T* residual, const T* weight,
                                                       int rows, int H, float eps, T* total, T* y,
                                                       uint8_t* yq, float* y_scale)
{
    constexpr int V = Raw<T>::kValues;
    __shared__ float s_sum[2][kMaxWaves][1];
    int buf = 0;
    const int tid = WAVE ? (threadIdx.x & 63) : threadIdx.x;
    const int stride = WAVE ? 64 : blockDim.x;
    const int per = WAVE ? (blockDim.x >> 6) : 1;  // rows a workgroup takes at a time
    const int nch = H / V;
    const float inv = 1.0f / (float)H;
    for (long row = (long)blockIdx.x * per + (WAVE ? threadIdx.x >> 6 : 0); row < rows;
         row += (long)gridDim.x * per) {
        const size_t r0 = (size_t)row * H;
        Raw<T> a[NV], b[NV], w[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * stride;
            a[i].zero();
            b[i].zero();
            w[i].zero();
            if (c < nch) {
                a[i].template load<NT>(x + r0 + V * c);
                if (residual) b[i].template load<NT>(residual + r0 + V * c);
                w[i].load(weight + V * c);
            }
        }
        float sum[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (residual) {
                float z[V];
#pragma unroll
                for (int e = 0; e < V; ++e) z[e] = a[i][e] + b[i][e];
                a[i].set(z);  // the norm is taken of the stored sum
                const int c = tid + i * stride;
                if (c < nch) a[i].template store<NT>(total + r0 + V * c);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) sum[0] += a[i][e] * a[i][e];
        }
        row_sum<WAVE, 1>(sum, s_sum, buf);
        const float cn = rsqrtf(sum[0] * inv + eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * stride;
            float v[V];
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = a[i][e] * cn * w[i][e];
            if (y && c < nch) {
                Raw<T> o;
                o.set(v);
                o.template store<NT>(y + r0 + V * c);
            }
            if (yq) {  // H is a multiple of 128: the lanes of a block are in or out together
                constexpr int kLanes = 128 / V;
                const float s = block_absmax(v) / 448.0f;
                if (c < nch) {
                    store_codes(v, s, yq + r0 + V * c);
                    if ((c & (kLanes - 1)) == 0) y_scale[(r0 >> 7) + c / kLanes] = s;
                }
            }
        }
    }
}

// Workgroup b takes rows b, b + grid, ... and adds its rows' dy n in
// registers; its sum is one row of `part`.  The next row's loads are issued
// before the current row's reduction where the registers hold both rows.
template <class T, int NV, bool WAVE, bool NT>
__global__ __launch_bounds__(!WAVE ? 512 : NV == 4 ? 256 : 1024) void rmsnorm_backward_kernel(
    const T* dy, const T* z, const T* weight, const T* dtotal, int rows, int H, float eps, T* dz,
    float* __restrict__ part)
{
    constexpr int V = Raw<T>::kValues;
    constexpr bool kAhead = WAVE && NV == 1;
    __shared__ float s_sum[2][kMaxWaves][2];
    constexpr int kAdd = NV == 4 ? 4 : 8;  // waves whose sums are in LDS together
    __shared__ float s_dw[WAVE ? kAdd : 1][WAVE ? 64 * NV * V : 1];
    int buf = 0;
    const int wave = threadIdx.x >> 6;
    const int tid = WAVE ? (threadIdx.x & 63) : threadIdx.x;
    const int stride = WAVE ? 64 : blockDim.x;
    const int per = WAVE ? (blockDim.x >> 6) : 1;
    const int nch = H / V;
    const float inv = 1.0f / (float)H;
    struct Row {
        Raw<T> z[NV], g[NV], d[NV];
    };
    Raw<T> w[NV];
    float dw[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tid + i * stride;
        w[i].zero();
        if (c < nch) w[i].load(weight + V * c);
#pragma unroll
        for (int e = 0; e < V; ++e) dw[i][e] = 0.0f;
    }
    const long step = (long)gridDim.x * per;
    auto fetch = [&](Row& r, long row) {
        const size_t r0 = (size_t)row * H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * stride;
            r.z[i].zero();
            r.g[i].zero();
            r.d[i].zero();
            if (c < nch && row < rows) {
                r.z[i].template load<NT>(z + r0 + V * c);
                r.g[i].template load<NT>(dy + r0 + V * c);
                if (dtotal) r.d[i].template load<NT>(dtotal + r0 + V * c);
            }
        }
    };
    Row cur, next;
    long row = (long)blockIdx.x * per + (WAVE ? wave : 0);
    if constexpr (kAhead) fetch(cur, row);
    for (; row < rows; row += step) {
        if constexpr (kAhead) fetch(next, row + step);
        else fetch(cur, row);
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                sum[0] += cur.z[i][e] * cur.z[i][e];
                sum[1] += cur.g[i][e] * w[i][e] * cur.z[i][e];
            }
        row_sum<WAVE, 2>(sum, s_sum, buf);
        const float cn = rsqrtf(sum[0] * inv + eps);
        const float mean = sum[1] * inv * cn;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * stride;
            float v[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float n = cur.z[i][e] * cn;
                v[e] = cn * (cur.g[i][e] * w[i][e] - n * mean) + cur.d[i][e];
                dw[i][e] += cur.g[i][e] * n;
            }
            if (c < nch) {
                Raw<T> o;
                o.set(v);
                o.template store<NT>(dz + (size_t)row * H + V * c);
            }
        }
        if constexpr (kAhead) cur = next;
    }
    float* out = part + (size_t)blockIdx.x * H;
    if constexpr (WAVE) {  // the waves' sums, added in order, kAdd waves at a time
        constexpr int kCols = NV * V / 4;  // columns a thread of a 256-thread workgroup has at most
        float v[kCols] = {};
        for (int k0 = 0; k0 < per; k0 += kAdd) {
            if (wave >= k0 && wave < k0 + kAdd) {
#pragma unroll
                for (int i = 0; i < NV; ++i) store_f32(&s_dw[wave - k0][V * (tid + 64 * i)], dw[i]);
            }
            __syncthreads();
#pragma unroll
            for (int q = 0; q < kCols; ++q) {
                const int h = threadIdx.x + q * blockDim.x;
                if (h < H)
                    for (int k = 0; k < min(kAdd, per - k0); ++k) v[q] += s_dw[k][h];
            }
            __syncthreads();
        }
#pragma unroll
        for (int q = 0; q < kCols; ++q) {
            const int h = threadIdx.x + q * blockDim.x;
            if (h < H) out[h] = v[q];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * stride;
            if (c < nch) store_f32(out + V * c, dw[i]);
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
    int nv;       // chunks a thread
    int per;      // rows a workgroup takes at a time
    int grid;
};

// V: values of a chunk.  The same for every T, so a row's result does not
// depend on how many rows there are beside it.
Shape forward_shape(int T, int H, int V)
{
    const int nch = H / V;
    Shape s;
    s.wave = nch <= 128;
    s.nv = nch <= 64 ? 1 : nch <= 2048 ? 2 : 4;
    s.threads = s.wave ? 256 : (nch + 64 * s.nv - 1) / (64 * s.nv) * 64;
    s.per = s.wave ? 4 : 1;
    s.grid = std::min((T + s.per - 1) / s.per, 1 << 20);
    return s;
}

Shape backward_shape(int T, int H, int V)
{
    const int nch = H / V;
    Shape s;
    s.wave = nch <= 256;
    if (s.wave) {
        s.nv = nch <= 64 ? 1 : nch <= 128 ? 2 : 4;
        s.threads = T <= 64 && s.nv <= 2 ? 1024 : 256;
        s.per = s.threads / 64;
    } else {
        s.nv = nch <= 512 ? 2 : nch <= 2048 ? 4 : 8;
        s.threads = nch <= 1024 ? 256 : 512;
        s.per = 1;
    }
    // up to four rows one after the other cost less than the second launch that sums the partial rows
    s.grid = T <= 4 * s.per ? 1 : std::min((T + s.per - 1) / s.per, kPartials);
    return s;
}

template <class T, int NV, bool WAVE>
void launch_fwd(const Shape& sh, const void* x, const void* residual, const void* weight, int T_,
                int H, float eps, void* total, void* y, uint8_t* yq, float* ys, hipStream_t s)
{
    const bool nt = (long)T_ * H * (long)sizeof(T) * (residual ? 4 : 2) > kStream;
    auto* kernel = nt ? rmsnorm_kernel<T, NV, WAVE, true> : rmsnorm_kernel<T, NV, WAVE, false>;
    hipLaunchKernelGGL(kernel, dim3(sh.grid), dim3(sh.threads), 0, s,
                       static_cast<const T*>(x), static_cast<const T*>(residual),
                       static_cast<const T*>(weight), T_, H, eps, static_cast<T*>(total),
                       static_cast<T*>(y), yq, ys);
}

template <class T, int NV, bool WAVE>
void launch_bwd(const Shape& sh, const void* dy, const void* z, const void* weight,
                const void* dtotal, int T_, int H, float eps, void* dz, float* part, hipStream_t s)
{
    const bool nt = (long)T_ * H * (long)sizeof(T) * (dtotal ? 4 : 3) > kStream;
    auto* kernel = nt ? rmsnorm_backward_kernel<T, NV, WAVE, true> : rmsnorm_backward_kernel<T, NV, WAVE, false>;
    hipLaunchKernelGGL(kernel, dim3(sh.grid), dim3(sh.threads), 0, s,
                       static_cast<const T*>(dy), static_cast<const T*>(z), static_cast<const T*>(weight),
                       static_cast<const T*>(dtotal), T_, H, eps, static_cast<T*>(dz), part);
}

}  // namespace

size_t rmsnorm_backward_scratch_bytes(int T, int H)
{
    // whatever the type
    return (size_t)std::max(backward_shape(T, H, 4).grid, backward_shape(T, H, 8).grid) * H * sizeof(float);
}

moe_status launch_rmsnorm(const void* x, const void* residual, const void* weight, int dt, int T, int H,
                          float eps, void* total, void* y, uint8_t* yq, float* y_scale, hipStream_t s)
{
    const Shape sh = forward_shape(T, H, dt == MOE_F32 ? 4 : 8);
    {
        TimedLaunch tl(MOE_KID_RMSNORM, s);
        auto go = [&](auto type) {
            using V = decltype(type);
            constexpr int kWide = sizeof(V) == 4 ? 4 : 2;  // rows of more than 2048 chunks are fp32
            auto* f = !sh.wave ? (sh.nv == 2 ? launch_fwd<V, 2, false> : launch_fwd<V, kWide, false>)
                      : sh.nv == 1 ? launch_fwd<V, 1, true> : launch_fwd<V, 2, true>;
            f(sh, x, residual, weight, T, H, eps, total, y, yq, y_scale, s);
        };
        if (dt == MOE_BF16) go(bf16_t{});
        else go(float{});
    }
    return launch_status("rmsnorm_kernel");
}

moe_status launch_rmsnorm_backward(const void* dy, const void* z, const void* weight, const void* dtotal,
                                   int dt, int T, int H, float eps, void* dz, float* dweight, void* ws,
                                   hipStream_t s)
{
    const Shape sh = backward_shape(T, H, dt == MOE_F32 ? 4 : 8);
    // a single workgroup's sum is the answer
    float* part = T > 0 && sh.grid == 1 ? dweight : static_cast<float*>(ws);
    if (T > 0) {
        TimedLaunch tl(MOE_KID_RMSNORM_BWD, s);
        auto go = [&](auto type) {
            using V = decltype(type);
            constexpr int kWide = sizeof(V) == 4 ? 8 : 4;  // rows of more than 2048 chunks are fp32
            auto* f = !sh.wave ? (sh.nv == 2   ? launch_bwd<V, 2, false>
                                  : sh.nv == 4 ? launch_bwd<V, 4, false> : launch_bwd<V, kWide, false>)
                      : sh.nv == 1 ? launch_bwd<V, 1, true>
                      : sh.nv == 2 ? launch_bwd<V, 2, true> : launch_bwd<V, 4, true>;
            f(sh, dy, z, weight, dtotal, T, H, eps, dz, part, s);
        };
        if (dt == MOE_BF16) go(bf16_t{});
        else go(float{});
    }
    if (part != dweight) {
        TimedLaunch tl(MOE_KID_RMSNORM_DWEIGHT, s);
        hipLaunchKernelGGL(rmsnorm_dweight_kernel, dim3((H + 31) / 32), dim3(1024), 0, s, part, T ? sh.grid : 0, H,
                           dweight);
    }
    return launch_status("rmsnorm_backward_kernel");
}

}  // namespace moe

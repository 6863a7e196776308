// moe_layer_few: the whole layer for at most MOE_FEW_MAX_T tokens in two kernels.
//
//   FC1   h[r, c] = silu(x_t . W1_e[c]) * (x_t . W3_e[c])   for each (expert, token) pair r
//   FC2   y[t, n] = sum_j s_tj (h[r_tj] . W2_{e_tj}[n])  (+ shared experts)
//
// A few tokens are bound by the weights of the experts that they choose, each read
// once, and by latency.  So the routing is done inside FC1, by every workgroup for
// itself (a wave a token, the tables in LDS), and the weighted sum inside FC2,
// whose workgroups own output columns and walk through all experts: two launches
// instead of the five or more of the four-call layer, and no row of FC2 goes
// through memory.  The pairs' rows are numbered as moe_permute numbers them, by
// expert and token, then those of the shared experts.
//
// A workgroup of eight waves takes 16 columns (of h: 16 gate and 16 up rows of the
// weights) at a time; the waves share out the reduction length in pieces and add
// their sums through LDS.  Weights go from memory to registers, the next pieces'
// loads in flight while a piece is multiplied, 128 whole bytes of a row in eight lanes
// (a lane's own row, 64 bytes of 16 rows a load, is what the MFMA takes, but streams
// 4.5 TB/s where this does 6: the lanes of a wave exchange a piece through LDS of
// their own).  The 16 rows of a column tile are the first operand of the MFMA, up
// to 16 of the expert's tokens the second (rows past the last token repeat it: a
// column of the result depends on its own token alone).  An expert with more
// tokens is taken in chunks of 16.
// MFMA forms: fp32 16x16x4, else bf16 16x16x32; e4m3 codes are widened to bf16 (exact)
// and each 128-wide block's sum is scaled in fp32, MXFP4 codes with their scales (exact).
// A lane feeds the K positions that 16 bytes of its weight row hold, and loads the
// same positions of its token.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.h"
#include "dma.h"
#include "mxfp4.h"
#include "route.h"

namespace moe {
namespace {

struct fp4_t {};  // two e2m1 codes a byte

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
constexpr int kMaxPairs = MOE_FEW_MAX_T * MOE_MAX_TOPK;                     // routed rows
constexpr int kMaxChunks = kMaxPairs + 64 * ((MOE_FEW_MAX_T + 15) / 16);    // one expert's at most 16 rows each

struct FewArgs {
    const char* x;      // [T, H]
    const char* w13;    // [G, 2I, H]
    const char* w2;     // [G, H, I]
    const void* s13;    // block scales or null
    const void* s2;
    char* h;            // [R, I], activations' type
    char* y;            // [T, H]
    int32_t* ids;       // [T, k], written by FC1, read by FC2
    float* scales;
    int T, H, I, E, k, n_shared;
};

// ---------------------------------------------------------------- tables
// Which experts have tokens, and whose rows are whose.
struct Tables {
    uint32_t mask[MOE_MAX_EXPERTS];  // tokens of each expert
    int first[MOE_MAX_EXPERTS];      // first row of each expert
    int token[kMaxPairs];            // token of each routed row
    int chunk[kMaxChunks];           // expert << 16 | first row
    int nchunks;
};

// From the masks: chunks in the experts' order, first rows.  One wave, four
// neighbouring experts a lane; the shared experts' chunks follow.
__device__ __forceinline__ void make_chunks(const FewArgs& a, Tables& tb, int lane)
{
    int rows = 0, chunks = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = __popc(tb.mask[4 * lane + i]);
        rows += n;
        chunks += (n + 15) / 16;
    }
    int sum = rows << 16 | chunks;
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(sum, d, 64);
        if (lane >= d) sum += v;
    }
    int row = (sum >> 16) - rows, at = (sum & 0xffff) - chunks;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 4 * lane + i, n = __popc(tb.mask[e]);
        tb.first[e] = row;
        for (int r = 0; r < n; r += 16) tb.chunk[at++] = e << 16 | (row + r);
        row += n;
    }
    const int routed = __shfl(sum & 0xffff, 63, 64), per = (a.T + 15) / 16;
    for (int i = lane; i < a.n_shared * per; i += 64)
        tb.chunk[routed + i] = (a.E + i / per) << 16 | (a.T * a.k + (i / per) * a.T + (i % per) * 16);
    if (lane == 0) tb.nchunks = routed + a.n_shared * per;
}

// Row of token t at expert e.
__device__ __forceinline__ int row_of(const Tables& tb, int e, int t)
{
    return tb.first[e] + __popc(tb.mask[e] & ((1u << t) - 1u));
}

// The tables from thread i's pair (expert e0 of token i / k); every thread comes here.
__device__ __forceinline__ void make_tables(const FewArgs& a, Tables& tb, int i, int e0)
{
    const int t = i / a.k;  // kThreads >= kMaxPairs
    if (i < MOE_MAX_EXPERTS) tb.mask[i] = 0;
    __syncthreads();
    if (t < a.T) atomicOr(&tb.mask[e0], 1u << t);
    __syncthreads();
    if (i < 64) make_chunks(a, tb, i);
    __syncthreads();
    if (t < a.T) tb.token[row_of(tb, e0, t)] = t;
    __syncthreads();
}

// An expert's rows [row0, row0 + n) of a chunk (scalar), and the row of a lane.
struct Chunk {
    int e, row0, n;
};
__device__ __forceinline__ Chunk get_chunk(const FewArgs& a, const Tables& tb, int c)
{
    const int v = __builtin_amdgcn_readfirstlane(tb.chunk[c]);
    Chunk k{v >> 16, v & 0xffff, 0};
    const int end = k.e < a.E ? __builtin_amdgcn_readfirstlane(tb.first[k.e] + __popc(tb.mask[k.e]))
                              : a.T * a.k + (k.e - a.E + 1) * a.T;
    k.n = min(16, end - k.row0);
    return k;
}
__device__ __forceinline__ int token_of(const FewArgs& a, const Tables& tb, const Chunk& c, int row)
{
    return c.e < a.E ? tb.token[row] : row - a.T * a.k - (c.e - a.E) * a.T;
}

// ---------------------------------------------------------------- pieces
// Memory as the buffer instructions address it: a scalar base, a scalar offset and
// one of the lane's, so that no lane holds a pointer.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer make_buffer(const char* p)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(uniform_ptr(p)), 0, 0xffffffffu, 0x00020000);
}
template <bool NT>  // NT: streamed past the caches
__device__ __forceinline__ u32x4_t load16(Buffer b, uint32_t lane_offset, uint32_t offset)
{
    return __builtin_amdgcn_raw_buffer_load_b128(b, lane_offset, offset, NT ? 2 : 0);
}

// One piece: PE values of K of NR weight tiles (16 rows each) and of the tokens.
template <class WT> struct Form;
template <> struct Form<float> {
    using act = float;
    static constexpr int kPE = 64, kPerLoad = 16;  // K values of a piece, and of 64 bytes of a row
    static constexpr int kDepth = 2;               // pieces in registers: one multiplied, the others on their way
    static constexpr int bytes(int n) { return n * 4; }
};
template <> struct Form<bf16_t> {
    using act = bf16_t;
    static constexpr int kPE = 128, kPerLoad = 32;
    static constexpr int kDepth = 2;
    static constexpr int bytes(int n) { return n * 2; }
};
template <> struct Form<fp8_t> {
    using act = bf16_t;
    static constexpr int kPE = 128, kPerLoad = 64;
    static constexpr int kDepth = 3;
    static constexpr int bytes(int n) { return n; }
};
template <> struct Form<fp4_t> {
    using act = bf16_t;
    static constexpr int kPE = 256, kPerLoad = 128;
    static constexpr int kDepth = 2;
    static constexpr int bytes(int n) { return n / 2; }
};

template <class WT, int NR>
struct Piece {
    using F = Form<WT>;
    using act = typename F::act;
    static constexpr int RB = F::bytes(F::kPE);                     // bytes of a row
    static constexpr int WL = RB / 64;                              // weight fragments of a tile
    static constexpr int PL = F::kPerLoad / 4 * (int)sizeof(act) / 16;  // activation fragments for each of them
    static constexpr int kStage = NR * 16 * RB;                     // LDS bytes of the exchange
    u32x4_t w[NR][WL];  // load j: rows 8 (j % 2) + lane / 8, bytes 128 (j / 2) + 16 (lane % 8)
    u32x4_t v[WL][PL];
    float s[NR];            // fp8: the block's scale
    uint32_t s4[NR][2];     // MXFP4: the eight scale bytes of the lane's row

    // The piece at scalar byte offset `wat` of an expert's weights (tile i `stride`
    // bytes on, rows ld bytes apart) and `vat` of the activations, with the lane's
    // offsets in both.  HALF: the row ends after half of the piece (MXFP4); the
    // weights and activations of the first half stand in for the other one.
    template <bool HALF>
    __device__ __forceinline__ void load(Buffer wb, uint32_t wat, uint32_t stride, uint32_t ld, uint32_t woff, Buffer vb,
                                         uint32_t vat, uint32_t voff)
    {
        const uint32_t back = HALF && (threadIdx.x & 4) ? RB / 2 : 0;  // lanes of the second 64 bytes
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int j = 0; j < WL; ++j)
                w[i][j] = load16<true>(wb, woff - back + (j >> 1) * 128, wat + i * stride + (j & 1) * 8 * ld);
#pragma unroll
        for (int j = 0; j < WL; ++j)
#pragma unroll
            for (int i = 0; i < PL; ++i)
                v[j][i] = load16<false>(vb, voff + (HALF ? 0 : j) * F::kPerLoad * (int)sizeof(act) + i * 16, vat);
    }

    // Lane l's rows become fragments: tile row l % 16, chunk 4 (j % 2) + l / 16 of 128 bytes.
    __device__ __forceinline__ void exchange(char* stage, int lane, u32x4_t (&f)[NR][WL]) const
    {
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int j = 0; j < WL; ++j)
                *reinterpret_cast<u32x4_t*>(stage + (i * (WL / 2) + (j >> 1)) * 2048 +
                                            dma_off((j & 1) * 8 + (lane >> 3), lane & 7)) = w[i][j];
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int j = 0; j < WL; ++j)
                f[i][j] = *reinterpret_cast<const u32x4_t*>(stage + (i * (WL / 2) + (j >> 1)) * 2048 +
                                                            dma_off(lane & 15, (j & 1) * 4 + (lane >> 4)));
    }

    // HALF: of the second half nothing.
    template <bool HALF>
    __device__ __forceinline__ void add(f32x4_t (&acc)[NR], char* stage, int lane) const
    {
        u32x4_t f[NR][WL];
        exchange(stage, lane, f);
        constexpr int N = HALF ? WL / 2 : WL;
        if constexpr (std::is_same_v<WT, float>) {
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int i = 0; i < NR; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(f[i][j][c]), __uint_as_float(v[j][0][c]),
                                                                      acc[i], 0, 0, 0);
        } else if constexpr (std::is_same_v<WT, bf16_t>) {
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int i = 0; i < NR; ++i) acc[i] = mfma_frag(f[i][j], v[j][0], acc[i], bf16_t());
        } else if constexpr (std::is_same_v<WT, fp8_t>) {
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                f32x4_t part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    part = mfma_frag(fp8x8_to_bf16x8(f[i][j].x, f[i][j].y), v[j][0], part, bf16_t());
                    part = mfma_frag(fp8x8_to_bf16x8(f[i][j].z, f[i][j].w), v[j][1], part, bf16_t());
                }
                acc[i] += s[i] * part;
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const uint32_t sc = (s4[i][j] >> (8 * (lane >> 4))) & 0xffu;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        acc[i] = mfma_frag(mxfp4_to_bf16x8(f[i][j][q], sc), v[j][q], acc[i], bf16_t());
                }
        }
    }
};

// The scales of piece p of NR tiles whose first rows are row[]: fp8, one value a tile
// (scalar); MXFP4, eight bytes of the lane's row (HALF: four).
template <bool HALF, class WT, int NR>
__device__ __forceinline__ void load_scales(Piece<WT, NR>& r, const void* scale, int e, int N, int K, const int (&row)[NR],
                                            int p, int lane)
{
    if constexpr (std::is_same_v<WT, fp8_t>) {
        const __attribute__((address_space(4))) float* s = (const __attribute__((address_space(4))) float*)scale;
#pragma unroll
        for (int i = 0; i < NR; ++i) r.s[i] = s[((size_t)e * (N / 128) + row[i] / 128) * (K / 128) + p];
    } else if constexpr (std::is_same_v<WT, fp4_t>) {
        const Buffer b = make_buffer(static_cast<const char*>(scale) + (size_t)e * N * (K / 32));
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int j = 0; j < (HALF ? 1 : 2); ++j)
                r.s4[i][j] = __builtin_amdgcn_raw_buffer_load_b32(b, (uint32_t)(lane & 15) * (uint32_t)(K / 32),
                                                                  (uint32_t)row[i] * (uint32_t)(K / 32) + p * 8 + j * 4, 0);
    }
}

// f(true) for the last, half piece of a row, else f(false): MXFP4 pieces hold 256
// values, and rows a multiple of 128.
template <class WT, class Fn>
__device__ __forceinline__ void by_half(bool half, const Fn& f)
{
    if constexpr (std::is_same_v<WT, fp4_t>) {
        if (half) {
            f(std::true_type());
            return;
        }
    }
    f(std::false_type());
}

// Fills D - 1 buffers, then calls one(buffer, next buffer to fill) until it is false;
// unrolled, so that every buffer is a set of registers.
template <int D, class P, class Fetch, class One, class More>
__device__ __forceinline__ void run_pipeline(P (&buf)[D], Fetch& fetch, One& one, const More& more)
{
#pragma unroll
    for (int i = 0; i < D - 1; ++i)
        if (more()) fetch(buf[i]);
    while (true) {
#pragma unroll
        for (int i = 0; i < D; ++i)
            if (!one(buf[i], buf[(i + D - 1) % D])) return;
    }
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16_t* p, float v) { *p = f32_to_bf16(v); }

// ------------------------------------------------------------------- FC1
template <class WT>
__global__ __launch_bounds__(kThreads) void few_fc1_kernel(FewArgs a, RouteArgs ra)
{
    using F = Form<WT>;
    using act = typename F::act;
    __shared__ Tables tb;
    __shared__ union {
        RouteLds route[kWaves];
        struct {
            f32x4_t red[2][kWaves][2][64];  // [turn][wave][gate, up][lane]
            char stage[kWaves][Piece<WT, 2>::kStage];
        } s;
    } lds;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // ---- routing of every token, by every workgroup; the first one writes it out
    __shared__ int ids[kMaxPairs];
#pragma unroll 1
    for (int t = wave; t < a.T; t += kWaves) {
        int id[MOE_MAX_TOPK];
        float scale[MOE_MAX_TOPK];
        const bool first = blockIdx.x == 0;
        if (first) route_token<true>(ra, t, lane, lds.route[wave], id, scale);
        else route_token<false>(ra, t, lane, lds.route[wave], id, scale);
#pragma unroll
        for (int j = 0; j < MOE_MAX_TOPK; ++j)
            if (j < a.k && lane == j) {
                ids[t * a.k + j] = id[j];
                if (first) {
                    a.ids[t * a.k + j] = id[j];
                    a.scales[t * a.k + j] = scale[j];
                }
            }
    }
    __syncthreads();
    make_tables(a, tb, tid, tid < a.T * a.k ? ids[tid] : 0);

    // ---- (chunk, column tile) items.  Piece p of an item is wave p % 8's; every wave
    // takes the same number of steps (past the end it loads the last piece and adds
    // nothing).  The loads run kDepth - 1 steps ahead, across items.  Each step has its
    // registers by name (unrolled), and loads and multiplies in one branch: copied
    // registers or a join between the two would make the compiler wait for them.
    const int tiles = a.I / 16, np = (a.H + F::kPE - 1) / F::kPE, items = __builtin_amdgcn_readfirstlane(tb.nchunks) * tiles;
    const int steps = (np + kWaves - 1) / kWaves;
    const bool ragged = a.H % F::kPE != 0;  // the last piece is half a one
    const uint32_t ld = F::bytes(a.H), woff = (lane >> 3) * ld + (lane & 7) * 16;
    const Buffer xb = make_buffer(a.x);
    char* stage = lds.s.stage[wave];
    struct Loads {  // where the loads are
        int item, step, e, row[2];
        uint32_t voff;
    } ahead;
    auto enter = [&](int item) {
        ahead.item = item;
        ahead.step = 0;
        if (item >= items) return;
        const Chunk c = get_chunk(a, tb, item / tiles);
        const int col = item % tiles * 16, row = c.row0 + min(lane & 15, c.n - 1);
        ahead.e = c.e;
        ahead.row[0] = col;
        ahead.row[1] = a.I + col;
        ahead.voff = (uint32_t)(token_of(a, tb, c, row) * a.H + g * (F::kPerLoad / 4)) * (uint32_t)sizeof(act);
    };
    Piece<WT, 2> buf[F::kDepth];
    auto fetch = [&](Piece<WT, 2>& r) {
        const int p = min(wave + ahead.step * kWaves, np - 1);
        by_half<WT>(ragged && p == np - 1, [&](auto half) {
            r.template load<decltype(half)::value>(make_buffer(a.w13 + (size_t)ahead.e * 2 * a.I * ld),
                                                   ahead.row[0] * ld + F::bytes(p * F::kPE), a.I * ld, ld, woff, xb,
                                                   p * F::kPE * (uint32_t)sizeof(act), ahead.voff);
            load_scales<decltype(half)::value>(r, a.s13, ahead.e, 2 * a.I, a.H, ahead.row, p, lane);
        });
        if (++ahead.step == steps) enter(ahead.item + gridDim.x);
    };
    int item = blockIdx.x, step = 0, turn = 0;
    if (item >= items) return;
    f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    auto multiply = [&](const Piece<WT, 2>& r) {
        const int p = wave + step * kWaves;
        if (p < np)
            by_half<WT>(ragged && p == np - 1, [&](auto half) { r.template add<decltype(half)::value>(acc, stage, lane); });
    };
    auto one = [&](const Piece<WT, 2>& r, Piece<WT, 2>& next) {  // false after the last item
        if (ahead.item < items) {
            fetch(next);
            multiply(r);
        } else {
            multiply(r);
        }
        if (++step < steps) return true;
        lds.s.red[turn][wave][0][lane] = acc[0];
        lds.s.red[turn][wave][1][lane] = acc[1];
        acc[0] = acc[1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        lds_barrier();  // the other turn's buffer is free once every wave has come here
        if (wave < 4) {
            const float* sums = reinterpret_cast<const float*>(lds.s.red[turn]);
            float gt = 0.0f, up = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                gt += sums[w * 512 + tid];
                up += sums[w * 512 + 256 + tid];
            }
            const Chunk c = get_chunk(a, tb, item / tiles);
            const int n = (tid >> 2) & 15, col = item % tiles * 16 + (tid >> 6) * 4 + (tid & 3);
            if (n < c.n)
                put(reinterpret_cast<act*>(a.h) + (size_t)(c.row0 + n) * a.I + col,
                    gt * __builtin_amdgcn_rcpf(1.0f + expf(-gt)) * up);
        }
        turn ^= 1;
        step = 0;
        item += gridDim.x;
        return item < items;
    };
    enter(item);
    run_pipeline<F::kDepth>(buf, fetch, one, [&] { return ahead.item < items; });
}

// ------------------------------------------------------------------- FC2
template <class WT>
__global__ __launch_bounds__(kThreads) void few_fc2_kernel(FewArgs a)
{
    using F = Form<WT>;
    using act = typename F::act;
    __shared__ Tables tb;
    __shared__ float weight[kMaxPairs];                      // of each routed row
    __shared__ __attribute__((aligned(16))) char stage[kWaves][Piece<WT, 1>::kStage];
    __shared__ f32x4_t ys[kWaves][MOE_FEW_MAX_T][4];         // each wave's sums: 16 columns a token
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // ---- the tables again, from the ids
    const int pairs = a.T * a.k, e0 = tid < pairs ? a.ids[tid] : 0;
    make_tables(a, tb, tid, e0);
    if (tid < pairs) weight[row_of(tb, e0, tid / a.k)] = a.scales[tid];
    __syncthreads();

    // ---- column tiles.  A wave's pieces are every eighth of all (chunk, piece) pairs;
    // the loads run ahead as in FC1, within a tile.
    const int np = (a.I + F::kPE - 1) / F::kPE, all = __builtin_amdgcn_readfirstlane(tb.nchunks) * np, tiles = a.H / 16;
    const bool ragged = a.I % F::kPE != 0;
    const uint32_t ld = F::bytes(a.I), woff = (lane >> 3) * ld + (lane & 7) * 16;
    const Buffer hb = make_buffer(a.h);
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        for (int i = lane; i < a.T * 4; i += 64) ys[wave][i >> 2][i & 3] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        struct Loads {
            int q, chunk, p, e, row[1];
            uint32_t vat, voff;  // the chunk's first row; the lane's place
        } ahead;
        const int row0 = tile * 16;
        auto enter = [&](int q) {
            ahead.q = q;
            if (q >= all) return;
            const int chunk = q / np;
            ahead.p = q - chunk * np;
            if (chunk == ahead.chunk) return;
            ahead.chunk = chunk;
            const Chunk c = get_chunk(a, tb, chunk);
            ahead.e = c.e;
            ahead.row[0] = row0;
            ahead.vat = (uint32_t)(c.row0 * a.I) * (uint32_t)sizeof(act);
            ahead.voff = (uint32_t)(min(lane & 15, c.n - 1) * a.I + g * (F::kPerLoad / 4)) * (uint32_t)sizeof(act);
        };
        Piece<WT, 1> buf[F::kDepth];
        auto fetch = [&](Piece<WT, 1>& r) {
            by_half<WT>(ragged && ahead.p == np - 1, [&](auto half) {
                r.template load<decltype(half)::value>(make_buffer(a.w2 + (size_t)ahead.e * a.H * ld),
                                                       row0 * ld + F::bytes(ahead.p * F::kPE), 0, ld, woff, hb,
                                                       ahead.vat + ahead.p * F::kPE * (uint32_t)sizeof(act), ahead.voff);
                load_scales<decltype(half)::value>(r, a.s2, ahead.e, a.H, a.I, ahead.row, ahead.p, lane);
            });
            enter(ahead.q + kWaves);
        };
        int q = wave;
        f32x4_t acc[1] = {{0.f, 0.f, 0.f, 0.f}};
        auto one = [&](const Piece<WT, 1>& r, Piece<WT, 1>& next) {
            const int chunk = q / np;
            auto multiply = [&] {
                by_half<WT>(ragged && q - chunk * np == np - 1,
                            [&](auto half) { r.template add<decltype(half)::value>(acc, stage[wave], lane); });
            };
            if (ahead.q < all) {
                fetch(next);
                multiply();
            } else {
                multiply();
            }
            q += kWaves;
            if (q >= all || q / np != chunk) {  // the wave's last piece of this chunk: its rows to their tokens
                const Chunk c = get_chunk(a, tb, chunk);
                const int n = lane & 15, row = c.row0 + n;
                if (n < c.n) {
                    const float w = c.e < a.E ? weight[row] : 1.0f;
                    ys[wave][token_of(a, tb, c, row)][g] += w * acc[0];  // the wave's own; a token is in a chunk once
                }
                acc[0] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            }
            return q < all;
        };
        ahead.chunk = -1;
        enter(q);
        if (q < all) run_pipeline<F::kDepth>(buf, fetch, one, [&] { return ahead.q < all; });
        __syncthreads();
        for (int i = tid; i < a.T * 16; i += kThreads) {
            const int t = i >> 4, c = i & 15;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) v += reinterpret_cast<const float*>(&ys[w][t][0])[c];
            put(reinterpret_cast<act*>(a.y) + (size_t)t * a.H + row0 + c, v);
        }
        __syncthreads();
    }
}

template <class WT>
moe_status run_few(const FewArgs& a, const RouteArgs& ra, hipStream_t s)
{
    static const int occ1 = [] {
        int n = 0;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, few_fc1_kernel<WT>, kThreads, 0) != hipSuccess || n < 1) n = 1;
        return n;
    }();
    static const int occ2 = [] {
        int n = 0;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, few_fc2_kernel<WT>, kThreads, 0) != hipSuccess || n < 1) n = 1;
        return n;
    }();
    const long cus = device_cu_count(), per = (a.T + 15) / 16;
    const long chunks = std::min((long)a.T * a.k, (long)a.E * per) + a.n_shared * per;  // at most
    const long g1 = std::min(chunks * (a.I / 16), cus * occ1), g2 = std::min((long)a.H / 16, cus * occ2);
    {
        TimedLaunch tl(MOE_KID_FEW_FC1, s);
        hipLaunchKernelGGL(few_fc1_kernel<WT>, dim3((unsigned)g1), dim3(kThreads), 0, s, a, ra);
    }
    moe_status st = launch_status("few_fc1_kernel");
    if (st != MOE_OK) return st;
    {
        TimedLaunch tl(MOE_KID_FEW_FC2, s);
        hipLaunchKernelGGL(few_fc2_kernel<WT>, dim3((unsigned)g2), dim3(kThreads), 0, s, a);
    }
    return launch_status("few_fc2_kernel");
}

}  // namespace

size_t few_scratch_bytes(int T, int I, int k, int n_shared, int act)
{
    return (size_t)T * (k + n_shared) * I * (act == MOE_F32 ? 4 : 2);
}

moe_status launch_layer_few(const void* x, const float* logits, int T, int H, int I, int E, int method, int k,
                            int n_group, int topk_group, const float* bias, float scaling, unsigned flags,
                            int n_shared, const void* w13, const void* w2, int wdt, const void* w13_scale,
                            const void* w2_scale, int32_t* ids, float* scales, void* y, void* ws, hipStream_t s)
{
    FewArgs a{};
    a.x = static_cast<const char*>(x);
    a.w13 = static_cast<const char*>(w13);
    a.w2 = static_cast<const char*>(w2);
    a.s13 = w13_scale;
    a.s2 = w2_scale;
    a.h = static_cast<char*>(ws);
    a.y = static_cast<char*>(y);
    a.ids = ids;
    a.scales = scales;
    a.T = T; a.H = H; a.I = I; a.E = E; a.k = k; a.n_shared = n_shared;
    const RouteArgs ra{logits, bias, T, E, method, k, n_group, topk_group, scaling, flags};
    if (wdt == MOE_F32) return run_few<float>(a, ra, s);
    if (wdt == MOE_BF16) return run_few<bf16_t>(a, ra, s);
    if (wdt == MOE_FP8_E4M3) return run_few<fp8_t>(a, ra, s);
    return run_few<fp4_t>(a, ra, s);
}

}  // namespace moe

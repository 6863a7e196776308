// moe_layer_few: the whole layer for at most MOE_FEW_MAX_T tokens in two kernels, or
// three.
//
//   FC1   h[r, c] = silu(x_t . W1_e[c]) * (x_t . W3_e[c])   for each (expert, token) pair r
//   FC2   y[t, n] = sum_j s_tj (h[r_tj] . W2_{e_tj}[n])  (+ shared experts)
//
// A few tokens are bound by the weights of the experts that they choose, each read
// once (twice past 16 tokens of an expert), and by latency.  So the routing of up to
// eight tokens is done inside FC1, by every workgroup for itself (a wave a token, the
// tables in LDS), and the weighted sum inside FC2, whose workgroups own output columns
// and walk through all experts: two launches instead of the five or more of the
// four-call layer, and no row of FC2 goes through memory.  With more tokens moe_route's kernel goes first, where a wave would
// have had several to route (32 tokens of H 512, I 512, E 256 with groups: 119 us with
// four a wave, 105 so).  The pairs' rows are numbered as moe_permute numbers them, by
// expert and token, then those of the shared experts.
//
// A workgroup of eight waves takes 16 columns (of h: 16 gate and 16 up rows of the
// weights) at a time; the waves share out the reduction length in pieces and add
// their sums through LDS.  The next pieces' loads are in flight, to registers, while
// a piece is multiplied.  A load takes 128 whole bytes of a row in eight lanes: the
// lane's own row, 64 bytes of 16 rows a load, is what the MFMA takes, but streams
// 4.5 TB/s where this does 6 to 7, so the lanes of a wave exchange a piece through
// LDS of their own.  So are the activations: loads, not bytes, are what bounds the
// narrow weights (one token of the DeepSeek-V3-shaped layer in MXFP4: 83 us when each
// lane loaded its own activations and scales, 16 loads for 4 KB of weights, 56 with 5
// to 8), and where no expert has more than four tokens a piece of theirs is one or two.
// The 16 rows of a column tile are the first operand of the MFMA, up to 16 of the
// expert's tokens the second (rows past the last token repeat it: a column of the
// result depends on its own token alone).  An expert with 17 to 32 tokens is two chunks,
// each with its own pass over the expert's weights: 17 tokens that all choose one bf16
// expert of H 4096, I 14336 take 117 us where 16 take 68 (MXFP4 63 and 42), and past 16
// tokens a shared expert is read twice (32 tokens of H 4096, I 2048, E 64, k 6, 61 experts
// chosen: 458 us without one, 474 with).
// MFMA forms: fp32 16x16x4, else bf16 16x16x32; e4m3 codes are widened to bf16 (exact)
// and each 128-wide block's sum is scaled in fp32, MXFP4 codes with their scales (exact).
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
constexpr int kMaxPairs = MOE_FEW_MAX_T * MOE_MAX_TOPK;                   // routed rows
constexpr int kMaxChunks = kMaxPairs + 64 * ((MOE_FEW_MAX_T + 15) / 16);  // one expert's at most 16 rows each
constexpr int kFew = 4;                                                   // tokens of a chunk up to which activations are few

// What FC2 has to know of the routing; FC1 leaves it in the workspace.
struct Plan {
    int nchunks;
    int most;                 // rows of the largest chunk
    int chunk[kMaxChunks];    // expert << 18 | first row << 5 | rows
    int token[kMaxPairs];     // token of each routed row
    float weight[kMaxPairs];  // ... and its weight
};

struct FewArgs {
    const char* x;      // [T, H]
    const char* w13;    // [G, 2I, H]
    const char* w2;     // [G, H, I]
    const void* s13;    // block scales or null
    const void* s2;
    char* h;            // [R, I], activations' type
    Plan* plan;
    char* y;            // [T, H]
    int32_t* ids;       // [T, k]
    float* scales;
    int T, H, I, E, k, n_shared;
    int splits;         // workgroups that share a column tile of FC2
    float* part;        // ... [H/16, splits, T, 16] their sums, if more than one
    int* arrived;       // [H/16] how many of them are there
};

// ---------------------------------------------------------------- tables
struct Tables {
    uint32_t mask[MOE_MAX_EXPERTS];  // tokens of each expert
    int first[MOE_MAX_EXPERTS];      // first row of each expert
};

__device__ __forceinline__ int pack_chunk(int e, int row, int n) { return e << 18 | row << 5 | n; }

// From the masks: chunks in the experts' order, first rows.  One wave, four
// neighbouring experts a lane; the shared experts' chunks follow.
__device__ __forceinline__ void make_chunks(const FewArgs& a, Tables& tb, Plan& plan, int lane)
{
    int rows = 0, chunks = 0, most = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = __popc(tb.mask[4 * lane + i]);
        rows += n;
        chunks += (n + 15) / 16;
        most = max(most, n);
    }
    int sum = rows << 16 | chunks;
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(sum, d, 64);
        if (lane >= d) sum += v;
    }
    const bool many = __ballot(most > kFew) != 0;
    int row = (sum >> 16) - rows, at = (sum & 0xffff) - chunks;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 4 * lane + i, n = __popc(tb.mask[e]);
        tb.first[e] = row;
        for (int r = 0; r < n; r += 16) plan.chunk[at++] = pack_chunk(e, row + r, min(16, n - r));
        row += n;
    }
    const int routed = __shfl(sum & 0xffff, 63, 64), per = (a.T + 15) / 16;
    for (int i = lane; i < a.n_shared * per; i += 64)
        plan.chunk[routed + i] = pack_chunk(a.E + i / per, a.T * a.k + (i / per) * a.T + (i % per) * 16,
                                            min(16, a.T - (i % per) * 16));
    if (lane == 0) {
        plan.nchunks = routed + a.n_shared * per;
        plan.most = many || (a.n_shared > 0 && a.T > kFew) ? 16 : kFew;
    }
}

// Row of token t at expert e.
__device__ __forceinline__ int row_of(const Tables& tb, int e, int t)
{
    return tb.first[e] + __popc(tb.mask[e] & ((1u << t) - 1u));
}

// Rows [row0, row0 + n) of expert e (all scalar).
struct Chunk {
    int e, row0, n;
};
__device__ __forceinline__ Chunk get_chunk(const Plan& plan, int c)
{
    const int v = __builtin_amdgcn_readfirstlane(plan.chunk[c]);
    return {v >> 18, (v >> 5) & 0x1fff, v & 31};
}
__device__ __forceinline__ int token_of(const FewArgs& a, const Plan& plan, const Chunk& c, int row)
{
    return c.e < a.E ? plan.token[row] : row - a.T * a.k - (c.e - a.E) * a.T;
}

// Memory as the buffer instructions address it: a scalar base, a scalar offset and
// one of the lane's, so that no lane holds a pointer.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer make_buffer(const char* p, bool valid)  // not valid: loads are zeros, and no traffic
{
    const int bytes = __builtin_amdgcn_readfirstlane(valid ? -1 : 0);  // scalar, as the base
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(uniform_ptr(p)), 0, bytes, 0x00020000);
}
template <bool NT>  // NT: streamed past the caches
__device__ __forceinline__ u32x4_t load16(Buffer b, uint32_t lane_offset, uint32_t offset)
{
    return __builtin_amdgcn_raw_buffer_load_b128(b, lane_offset, offset, NT ? 2 : 0);
}

// ---------------------------------------------------------------- pieces
// The weights' forms: K values of a piece, and of 64 bytes of a row; pieces in
// registers (one multiplied, the others on their way) with few and with many tokens
// a chunk; whether a row may end after half a piece.
template <class WT> struct Form;
template <> struct Form<float> {
    using act = float;
    static constexpr int kPE = 64, kPer64 = 16, kDepthFew = 2, kDepthMany = 2;
    static constexpr bool kHalves = false;
    static constexpr int bytes(int n) { return n * 4; }
};
template <> struct Form<bf16_t> {
    using act = bf16_t;
    static constexpr int kPE = 128, kPer64 = 32, kDepthFew = 2, kDepthMany = 2;
    static constexpr bool kHalves = false;
    static constexpr int bytes(int n) { return n * 2; }
};
template <> struct Form<fp8_t> {
    using act = bf16_t;
    static constexpr int kPE = 128, kPer64 = 64, kDepthFew = 3, kDepthMany = 3;
    static constexpr bool kHalves = false;
    static constexpr int bytes(int n) { return n; }
};
template <> struct Form<fp4_t> {
    using act = bf16_t;
    static constexpr int kPE = 256, kPer64 = 128, kDepthFew = 3, kDepthMany = 2;
    static constexpr bool kHalves = true;
    static constexpr int bytes(int n) { return n / 2; }
};

// One piece: kPE values of K of NR weight tiles (16 rows each) and of the chunk's
// tokens, of which there are at most kFew or 16.
template <class WT, int NR, bool MANY>
struct Piece {
    using F = Form<WT>;
    using act = typename F::act;
    static constexpr bool kFp4 = std::is_same_v<WT, fp4_t>;
    static constexpr int RB = F::bytes(F::kPE);                     // bytes of a weight row
    static constexpr int WL = RB / 64;                              // weight loads, and fragments, of a tile
    static constexpr int VB = F::kPE * (int)sizeof(act);            // bytes of a token
    static constexpr int VT = 1024 / VB;                            // tokens of a load
    static constexpr int VL = (MANY ? 16 : kFew) / VT;              // loads of the tokens
    static constexpr int PL = VB / 64 / WL;                         // activation fragments for a weight fragment
    static constexpr int kWStage = 16 * RB;                         // LDS of the exchange: a tile at a time,
    static constexpr int kStage = kWStage + VL * 1024 + (kFp4 ? 256 : 0);  // the tokens, the scales
    u32x4_t w[NR][WL];  // load j: rows 8 (j % 2) + lane / 8, bytes 128 (j / 2) + 16 (lane % 8)
    u32x4_t v[VL];      // load i: token i VT + lane / (64 / VT), 16-byte chunk lane % (64 / VT)
    float s[NR];        // fp8: the block's scale
    uint32_t s4;        // MXFP4: four scale bytes of tile lane / 32, row lane / 2 % 16

    // The lane's token of load i and its bytes of it.
    static __device__ __forceinline__ int token(int lane, int i) { return i * VT + lane / (64 / VT); }
    static __device__ __forceinline__ int chunk16(int lane) { return lane % (64 / VT) * 16; }

    // The piece at scalar byte offset `wat` of an expert's weights (tile i `stride`
    // bytes on, rows ld bytes apart) and `vat` of the activations, with the lane's
    // offsets in both.  half: the row ends after half of the piece (MXFP4); the
    // first half stands in for the other one.
    __device__ __forceinline__ void load(Buffer wb, uint32_t wat, uint32_t stride, uint32_t ld, uint32_t woff, Buffer vb,
                                         uint32_t vat, const uint32_t (&voff)[VL], bool half)
    {
        wat = __builtin_amdgcn_readfirstlane(wat);
        vat = __builtin_amdgcn_readfirstlane(vat);
        uint32_t vback = 0;
        if constexpr (F::kHalves) {
            woff -= half && (threadIdx.x & 4) ? RB / 2 : 0;
            vback = half && (threadIdx.x & (32 / VT)) ? VB / 2 : 0;
        }
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int j = 0; j < WL; ++j)
                w[i][j] = load16<true>(wb, woff + (j >> 1) * 128, wat + i * stride + (j & 1) * 8 * ld);
#pragma unroll
        for (int i = 0; i < VL; ++i) v[i] = load16<false>(vb, voff[i] - vback, vat);
    }

    // The scales of piece p of tiles whose first rows are row[] of an expert's N.
    __device__ __forceinline__ void load_scales(const void* scale, int e, int N, int K, const int (&row)[NR], int p, int lane,
                                                bool half, bool valid)
    {
        if constexpr (std::is_same_v<WT, fp8_t>) {
            const __attribute__((address_space(4))) float* sp = (const __attribute__((address_space(4))) float*)scale;
#pragma unroll
            for (int i = 0; i < NR; ++i) s[i] = sp[((size_t)e * (N / 128) + row[i] / 128) * (K / 128) + p];
        } else if constexpr (kFp4) {
            const Buffer b = make_buffer(static_cast<const char*>(scale) + (size_t)e * N * (K / 32), valid);
            const uint32_t r = row[NR == 2 && lane >= 32 ? NR - 1 : 0] + (lane >> 1) % 16;
            s4 = __builtin_amdgcn_raw_buffer_load_b32(b, r * (uint32_t)(K / 32) + (half ? 0 : (lane & 1) * 4),
                                                      __builtin_amdgcn_readfirstlane(p * 8), 0);
        }
    }

    // acc += the piece's product with the chunk's n tokens, through the wave's own
    // `stage`.  Row l % 16 of a tile and token l % 16 (the last one's past it) are
    // lane l's, with 16-byte chunk 4 (j % 2) + l / 16 of each 128 bytes of the weights.
    __device__ __forceinline__ void add(f32x4_t (&acc)[NR], char* stage, int lane, int n, bool half) const
    {
        const int r = lane & 15, g = lane >> 4;
        char* vs = stage + kWStage;
#pragma unroll
        for (int i = 0; i < VL; ++i) {
            const int c = chunk16(lane);
            *reinterpret_cast<u32x4_t*>(vs + (c >> 7) * (VL * VT * 128) + dma_off(token(lane, i), (c >> 4) & 7)) = v[i];
        }
        if constexpr (kFp4) *reinterpret_cast<uint32_t*>(vs + VL * 1024 + lane * 4) = s4;
        u32x4_t a[WL][PL];
        const int t = min(r, n - 1);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            u32x4_t f[WL];
#pragma unroll
            for (int j = 0; j < WL; ++j)
                *reinterpret_cast<u32x4_t*>(stage + (j >> 1) * 2048 + dma_off((j & 1) * 8 + (lane >> 3), lane & 7)) = w[i][j];
            wave_lds_fence();
            if (i == 0) {
#pragma unroll
                for (int j = 0; j < WL; ++j)
#pragma unroll
                    for (int q = 0; q < PL; ++q) {
                        const int c = (j * 4 + g) * PL + q;  // of the token's 16-byte chunks
                        a[j][q] = *reinterpret_cast<const u32x4_t*>(vs + (c >> 3) * (VL * VT * 128) + dma_off(t, c & 7));
                    }
            }
#pragma unroll
            for (int j = 0; j < WL; ++j)
                f[j] = *reinterpret_cast<const u32x4_t*>(stage + (j >> 1) * 2048 + dma_off(r, (j & 1) * 4 + g));
            if constexpr (std::is_same_v<WT, float>) {
#pragma unroll
                for (int j = 0; j < WL; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(f[j][c]), __uint_as_float(a[j][0][c]),
                                                                      acc[i], 0, 0, 0);
            } else if constexpr (std::is_same_v<WT, bf16_t>) {
#pragma unroll
                for (int j = 0; j < WL; ++j) acc[i] = mfma_frag(f[j], a[j][0], acc[i], bf16_t());
            } else if constexpr (std::is_same_v<WT, fp8_t>) {
                f32x4_t part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < WL; ++j) {
                    part = mfma_frag(fp8x8_to_bf16x8(f[j].x, f[j].y), a[j][0], part, bf16_t());
                    part = mfma_frag(fp8x8_to_bf16x8(f[j].z, f[j].w), a[j][1], part, bf16_t());
                }
                acc[i] += s[i] * part;
            } else {
                typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
                const u32x2_t sc = *reinterpret_cast<const u32x2_t*>(vs + VL * 1024 + (i * 16 + r) * 8);
#pragma unroll
                for (int j = 0; j < WL; ++j) {
                    if (j > 0 && half) break;
                    const uint32_t byte = (sc[j] >> (8 * g)) & 0xffu;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        acc[i] = mfma_frag(mxfp4_to_bf16x8(f[j][q], byte), a[j][q], acc[i], bf16_t());
                }
            }
        }
    }
};

// Fills D - 1 buffers, then calls one(buffer, next buffer to fill) until it is false;
// unrolled, so that every buffer is a set of registers.
template <int D, class P, class Fetch, class One>
__device__ __forceinline__ void run_pipeline(P (&buf)[D], Fetch& fetch, One& one)
{
#pragma unroll
    for (int i = 0; i < D - 1; ++i) fetch(buf[i]);
    while (true) {
#pragma unroll
        for (int i = 0; i < D; ++i)
            if (!one(buf[i], buf[(i + D - 1) % D])) return;
    }
}

// h and y in the activations' type.  h is a product's operand next, and rounded here as
// the experts' FFN in separate calls rounds it: with bf16 the listed layers are 2.3e-3
// from the exact ones, where y's rounding alone leaves 1.7e-3.  (Two bf16 parts of h would
// cost FC2 a second product for each fragment and no byte of weights.)
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16_t* p, float v) { *p = f32_to_bf16(v); }

// ------------------------------------------------------------------- FC1
typedef f32x4_t Sums[2][kWaves][2][64];  // [turn][wave][gate, up][lane]

// The (chunk, column tile) items of this workgroup.  Piece p of an item is wave
// p % 8's; every wave takes the same number of steps (past the end it loads and adds
// nothing).  The loads run D - 1 steps ahead, across items, and go on past the last
// one with an empty buffer: each step has its registers by name (unrolled) and its
// loads under no condition, where copied registers or a join of two branches would
// make the compiler wait for them.
template <class WT, bool MANY>
__device__ __forceinline__ void fc1_items(const FewArgs& a, const Plan& plan, Sums& red, char* stage, int wave, int lane)
{
    using F = Form<WT>;
    using act = typename F::act;
    using P = Piece<WT, 2, MANY>;
    const int tiles = a.I / 16, np = (a.H + F::kPE - 1) / F::kPE;
    const int items = __builtin_amdgcn_readfirstlane(plan.nchunks) * tiles;
    const int steps = (np + kWaves - 1) / kWaves;
    const bool ragged = a.H % F::kPE != 0;  // the last piece is half a one
    const uint32_t ld = F::bytes(a.H), woff = (lane >> 3) * ld + (lane & 7) * 16;
    struct Loads {  // where the loads are
        int item, step, e, row[2];
        uint32_t voff[P::VL];
        bool valid;
    } ahead;
    auto enter = [&](int item) {
        ahead.item = item;
        ahead.step = 0;
        ahead.valid = item < items;
        if (!ahead.valid) return;
        const Chunk c = get_chunk(plan, item / tiles);
        ahead.e = c.e;
        ahead.row[0] = item % tiles * 16;
        ahead.row[1] = a.I + ahead.row[0];
#pragma unroll
        for (int i = 0; i < P::VL; ++i) {
            const int row = c.row0 + min(P::token(lane, i), c.n - 1);
            ahead.voff[i] = (uint32_t)(token_of(a, plan, c, row) * a.H) * (uint32_t)sizeof(act) + P::chunk16(lane);
        }
    };
    P buf[MANY ? F::kDepthMany : F::kDepthFew];
    auto fetch = [&](P& r) {
        const int p = min(wave + ahead.step * kWaves, np - 1);
        const bool valid = ahead.valid && wave + ahead.step * kWaves < np, half = F::kHalves && ragged && p == np - 1;
        r.load(make_buffer(a.w13 + (size_t)ahead.e * 2 * a.I * ld, valid), ahead.row[0] * ld + F::bytes(p * F::kPE),
               a.I * ld, ld, woff, make_buffer(a.x, valid), p * P::VB, ahead.voff, half);
        r.load_scales(a.s13, ahead.e, 2 * a.I, a.H, ahead.row, p, lane, half, valid);
        if (++ahead.step == steps) enter(ahead.item + gridDim.x);
    };
    int item = blockIdx.x, step = 0, turn = 0;
    if (item >= items) return;
    Chunk c = get_chunk(plan, item / tiles);
    f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    auto one = [&](const P& r, P& next) {  // false after the last item
        fetch(next);
        const int p = wave + step * kWaves;
        if (p < np) r.add(acc, stage, lane, c.n, F::kHalves && ragged && p == np - 1);
        if (++step < steps) return true;
        red[turn][wave][0][lane] = acc[0];
        red[turn][wave][1][lane] = acc[1];
        acc[0] = acc[1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        lds_barrier();  // the other turn's buffer is free once every wave has come here
        if (wave < 4) {
            const int i = wave * 64 + lane, n = (i >> 2) & 15, col = item % tiles * 16 + (i >> 6) * 4 + (i & 3);
            const float* sums = reinterpret_cast<const float*>(red[turn]);
            float gt = 0.0f, up = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                gt += sums[w * 512 + i];
                up += sums[w * 512 + 256 + i];
            }
            if (n < c.n)
                put(reinterpret_cast<act*>(a.h) + (size_t)(c.row0 + n) * a.I + col,
                    gt * __builtin_amdgcn_rcpf(1.0f + expf(-gt)) * up);
        }
        turn ^= 1;
        step = 0;
        item += gridDim.x;
        if (item >= items) return false;
        c = get_chunk(plan, item / tiles);
        return true;
    };
    enter(item);
    run_pipeline(buf, fetch, one);
}

// MAYBE: an expert may have more than kFew tokens (a call of at most kFew has a
// kernel of its own, whose smaller stage leaves LDS for a second workgroup on the CU;
// its registers allow one too but with MXFP4 weights in FC1, whose 153 are three waves
// a SIMD where a workgroup is two: there the CU has one).
template <class WT, bool MAYBE>
__global__ __launch_bounds__(kThreads) void few_fc1_kernel(FewArgs a, RouteArgs ra)
{
    constexpr int kStage = Piece<WT, 2, MAYBE>::kStage;
    __shared__ Tables tb;
    __shared__ Plan plan;
    __shared__ __attribute__((aligned(16))) union {
        RouteLds route[kWaves];
        struct {
            Sums red;
            char stage[kWaves][kStage];
        } s;
    } lds;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // ---- routing, by every workgroup; the last one, which has the fewest items,
    // writes it out
    const bool last = blockIdx.x == gridDim.x - 1;
    const int pairs = a.T * a.k;  // kThreads >= kMaxPairs
    __shared__ int ids[kMaxPairs];
    const bool routed = a.T > kWaves;  // moe_route's kernel has run: ids and weights are there
    float logit[4], scale = 0.0f;
    int id = 0;
    if (!routed && wave < a.T) load_logits(ra, wave, lane, logit);
    if (routed && tid < pairs) {
        id = a.ids[tid];
        if (last) scale = a.scales[tid];
    }
    if (tid < MOE_MAX_EXPERTS) tb.mask[tid] = 0;
    __syncthreads();
    auto enter = [&](int pair, int t) {
        ids[pair] = id;
        atomicOr(&tb.mask[id], 1u << t);
        if (last) plan.weight[pair] = scale;  // by pair until the rows are known
    };
    if (routed) {
        if (tid < pairs) enter(tid, tid / a.k);
    } else if (wave < a.T) {
        if (last) route_token<true>(ra, logit, lane, lds.route[wave], id, scale);
        else route_token<false>(ra, logit, lane, lds.route[wave], id, scale);
        if (lane < a.k) {
            enter(wave * a.k + lane, wave);
            if (last) {
                a.ids[wave * a.k + lane] = id;
                a.scales[wave * a.k + lane] = scale;
            }
        }
    }
    __syncthreads();
    if (wave == 0) make_chunks(a, tb, plan, lane);
    __syncthreads();
    if (tid < pairs) {
        const int row = row_of(tb, ids[tid], tid / a.k);
        plan.token[row] = tid / a.k;
        if (last) {
            a.plan->token[row] = tid / a.k;
            a.plan->weight[row] = plan.weight[tid];
        }
    }
    __syncthreads();
    if (last) {
        if (a.splits > 1)
            for (int i = tid; i < a.H / 16; i += kThreads) a.arrived[i] = 0;
        for (int i = tid; i < plan.nchunks; i += kThreads) a.plan->chunk[i] = plan.chunk[i];
        if (tid == 0) {
            a.plan->nchunks = plan.nchunks;
            a.plan->most = plan.most;
        }
    }
    if (!MAYBE || __builtin_amdgcn_readfirstlane(plan.most) <= kFew)
        fc1_items<WT, false>(a, plan, lds.s.red, lds.s.stage[wave], wave, lane);
    else
        fc1_items<WT, MAYBE>(a, plan, lds.s.red, lds.s.stage[wave], wave, lane);
}

// ------------------------------------------------------------------- FC2
typedef f32x4_t Columns[kWaves][MOE_FEW_MAX_T][4];  // each wave's sums: 16 columns a token

// The column tiles of this workgroup.  A wave's pieces are every eighth of all
// (chunk, piece) pairs; the loads run ahead as in FC1, within a tile.  Where there are
// fewer tiles than CUs, a.splits workgroups share one, and its pieces: each leaves its
// sums in the workspace, and the last to arrive adds them up, in the workgroups' order
// (32 bf16 tokens: H 2048, I 1024, E 64 159 -> 142 us for the layer, H 512, I 512, E 256
// 106 -> 60).
template <class WT, bool MANY>
__device__ __forceinline__ void fc2_tiles(const FewArgs& a, const Plan& plan, Columns& ys, char* stage, int wave, int lane)
{
    using F = Form<WT>;
    using act = typename F::act;
    using P = Piece<WT, 1, MANY>;
    const int np = (a.I + F::kPE - 1) / F::kPE, all = __builtin_amdgcn_readfirstlane(plan.nchunks) * np;
    const int items = a.H / 16 * a.splits, waves = kWaves * a.splits;
    const bool ragged = a.I % F::kPE != 0;
    const uint32_t ld = F::bytes(a.I), woff = (lane >> 3) * ld + (lane & 7) * 16;
    const int g = lane >> 4;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int tile = item / a.splits, split = item % a.splits, first = split * kWaves + wave;
        for (int i = lane; i < a.T * 4; i += 64) ys[wave][i >> 2][i & 3] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        struct Loads {
            int chunk, p, e, row[1];
            uint32_t vat, voff[P::VL];
            bool valid;
        } ahead;
        ahead.row[0] = tile * 16;
        auto enter = [&](int chunk) {
            ahead.valid = chunk * np + ahead.p < all;
            if (!ahead.valid) return;
            const Chunk c = get_chunk(plan, chunk);
            ahead.chunk = chunk;
            ahead.e = c.e;
            ahead.vat = (uint32_t)c.row0 * (uint32_t)a.I * (uint32_t)sizeof(act);  // h is under 4 GiB
#pragma unroll
            for (int i = 0; i < P::VL; ++i)
                ahead.voff[i] = (uint32_t)(min(P::token(lane, i), c.n - 1) * a.I) * (uint32_t)sizeof(act) + P::chunk16(lane);
        };
        P buf[MANY ? F::kDepthMany : F::kDepthFew];
        auto fetch = [&](P& r) {
            const bool half = F::kHalves && ragged && ahead.p == np - 1;
            r.load(make_buffer(a.w2 + (size_t)ahead.e * a.H * ld, ahead.valid), ahead.row[0] * ld + F::bytes(ahead.p * F::kPE),
                   0, ld, woff, make_buffer(a.h, ahead.valid), ahead.vat + ahead.p * P::VB, ahead.voff, half);
            r.load_scales(a.s2, ahead.e, a.H, a.I, ahead.row, ahead.p, lane, half, ahead.valid);
            if (!ahead.valid) return;
            int chunk = ahead.chunk;
            ahead.p += waves;
            while (ahead.p >= np) {
                ahead.p -= np;
                ++chunk;
            }
            if (chunk != ahead.chunk) enter(chunk);
        };
        int chunk = first / np, p = first - chunk * np, q = first;
        f32x4_t acc[1] = {{0.f, 0.f, 0.f, 0.f}};
        if (q < all) {
            Chunk c = get_chunk(plan, chunk);
            auto one = [&](const P& r, P& next) {
                fetch(next);
                r.add(acc, stage, lane, c.n, F::kHalves && ragged && p == np - 1);
                q += waves;
                p += waves;
                if (p < np && q < all) return true;
                // the wave's last piece of this chunk: its rows to their tokens
                const int n = lane & 15, row = c.row0 + n;
                if (n < c.n) {
                    const float w = c.e < a.E ? plan.weight[row] : 1.0f;
                    ys[wave][token_of(a, plan, c, row)][g] += w * acc[0];  // the wave's own; a token is in a chunk once
                }
                acc[0] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                if (q >= all) return false;
                while (p >= np) {
                    p -= np;
                    ++chunk;
                }
                c = get_chunk(plan, chunk);
                return true;
            };
            ahead.p = p;
            enter(chunk);
            run_pipeline(buf, fetch, one);
        }
        __syncthreads();
        static_assert(MOE_FEW_MAX_T * 16 <= kThreads);
        const int i = wave * 64 + lane, t = i >> 4, col = i & 15;
        float v = 0.0f;
        if (t < a.T) {
#pragma unroll
            for (int w = 0; w < kWaves; ++w) v += reinterpret_cast<const float*>(&ys[w][t][0])[col];
        }
        bool writes = t < a.T;
        if (a.splits > 1) {
            __shared__ int before;
            float* part = a.part + (size_t)tile * a.splits * a.T * 16 + i;
            // Stores and loads that go past the XCD's own L2, the stores complete before
            // the count goes up: a release fence would write that L2 back (35 us and more).
            if (writes) __hip_atomic_store(part + split * a.T * 16, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            if (i == 0) before = __hip_atomic_fetch_add(a.arrived + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            writes = writes && before == a.splits - 1;
            if (writes) {
                v = 0.0f;
                for (int s = 0; s < a.splits; ++s)
                    v += __hip_atomic_load(part + s * a.T * 16, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
        if (writes) put(reinterpret_cast<act*>(a.y) + (size_t)t * a.H + tile * 16 + col, v);
        __syncthreads();
    }
}

template <class WT, bool MAYBE>
__global__ __launch_bounds__(kThreads) void few_fc2_kernel(FewArgs a)
{
    constexpr int kStage = Piece<WT, 1, MAYBE>::kStage;
    __shared__ Plan plan;
    __shared__ __attribute__((aligned(16))) char stage[kWaves][kStage];
    __shared__ Columns ys;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (int i = tid; i < (int)(sizeof(Plan) / 4); i += kThreads)
        reinterpret_cast<int*>(&plan)[i] = reinterpret_cast<const int*>(a.plan)[i];
    __syncthreads();
    if (!MAYBE || __builtin_amdgcn_readfirstlane(plan.most) <= kFew)
        fc2_tiles<WT, false>(a, plan, ys, stage[wave], wave, lane);
    else
        fc2_tiles<WT, MAYBE>(a, plan, ys, stage[wave], wave, lane);
}

template <class WT, bool MAYBE>
moe_status run_few(const FewArgs& a, const RouteArgs& ra, hipStream_t s)
{
    static const int occ1 = [] {
        int n = 0;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, few_fc1_kernel<WT, MAYBE>, kThreads, 0) != hipSuccess || n < 1)
            n = 1;
        return n;
    }();
    static const int occ2 = [] {
        int n = 0;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, few_fc2_kernel<WT, MAYBE>, kThreads, 0) != hipSuccess || n < 1)
            n = 1;
        return n;
    }();
    const long cus = device_cu_count(), per = (a.T + 15) / 16;
    const long chunks = std::min((long)a.T * a.k, (long)a.E * per) + a.n_shared * per;  // at most
    const long g1 = std::min(chunks * (a.I / 16), cus * occ1), g2 = std::min((long)a.H / 16 * a.splits, cus * occ2);
    {
        TimedLaunch tl(MOE_KID_FEW_FC1, s);
        hipLaunchKernelGGL((few_fc1_kernel<WT, MAYBE>), dim3((unsigned)g1), dim3(kThreads), 0, s, a, ra);
    }
    moe_status st = launch_status("few_fc1_kernel");
    if (st != MOE_OK) return st;
    {
        TimedLaunch tl(MOE_KID_FEW_FC2, s);
        hipLaunchKernelGGL((few_fc2_kernel<WT, MAYBE>), dim3((unsigned)g2), dim3(kThreads), 0, s, a);
    }
    return launch_status("few_fc2_kernel");
}

template <class WT>
moe_status run_few(const FewArgs& a, const RouteArgs& ra, hipStream_t s)
{
    return a.T <= kFew ? run_few<WT, false>(a, ra, s) : run_few<WT, true>(a, ra, s);
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

size_t few_h_bytes(int T, int I, int k, int n_shared, int act)
{
    const size_t n = (size_t)T * (k + n_shared) * I * (act == MOE_F32 ? 4 : 2);
    return align256(n);
}

// Workgroups for a column tile of FC2: by H alone, so that a token's sums have the
// same order whatever else is in the call.  (kCus stands for the card's CUs also where
// no device is asked: the workspace's size.)
int few_splits(int H)
{
    constexpr int kCus = 256, kMost = 8;
    int n = 1;
    while (n < kMost && H / 16 * n * 2 <= kCus) n *= 2;
    return n;
}

}  // namespace

size_t few_scratch_bytes(int T, int H, int I, int k, int n_shared, int act)
{
    const int splits = few_splits(H);
    return few_h_bytes(T, I, k, n_shared, act) + align256(sizeof(Plan)) +
           (splits > 1 ? align256((size_t)H / 16 * 4) + (size_t)splits * T * H * 4 : 0);
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
    a.plan = reinterpret_cast<Plan*>(a.h + few_h_bytes(T, I, k, n_shared, wdt == MOE_F32 ? MOE_F32 : MOE_BF16));
    a.splits = few_splits(H);
    a.arrived = reinterpret_cast<int*>(reinterpret_cast<char*>(a.plan) + align256(sizeof(Plan)));
    a.part = reinterpret_cast<float*>(reinterpret_cast<char*>(a.arrived) + align256((size_t)H / 16 * 4));
    a.y = static_cast<char*>(y);
    a.ids = ids;
    a.scales = scales;
    a.T = T; a.H = H; a.I = I; a.E = E; a.k = k; a.n_shared = n_shared;
    const RouteArgs ra{logits, bias, T, E, method, k, n_group, topk_group, scaling, flags};
    if (T > kWaves) {
        const moe_status st = launch_route(logits, T, E, method, k, n_group, topk_group, bias, scaling, flags, ids, scales, s);
        if (st != MOE_OK) return st;
    }
    if (wdt == MOE_F32) return run_few<float>(a, ra, s);
    if (wdt == MOE_BF16) return run_few<bf16_t>(a, ra, s);
    if (wdt == MOE_FP8_E4M3) return run_few<fp8_t>(a, ra, s);
    return run_few<fp4_t>(a, ra, s);
}

}  // namespace moe

// dq4_moe.hip -- a mixture-of-experts layer for a few tokens (include/dq4_moe.h):
// the router, and the chosen experts' gated feed-forward blocks over nested 4-bit
// weights.
//
// Few tokens choose few experts, and each chosen expert's matrices are read once:
// the layer is bound by that and by the decode.  Four launches: the router, a
// plan (which experts, which tokens each, and x in operand fragments), the gate
// and up products of every chosen expert in one kernel, and the down products of
// all of them with the weighted sum over a token's experts in another.
//
// The weight is decoded in operand registers as in dq4_linear_fused.hip's few-row
// kernels, through one lookup table of byte pairs in LDS, and multiplied on
// v_mfma_f32_16x16x32_{f16,bf16}: 16 weight rows by a tile of 16 tokens.  An
// expert's tokens are gathered into tiles (with up to 16 tokens in all, the one
// tile of all tokens serves every expert), so that an expert costs its own
// tokens, not everybody's.
//
// Operand order of x and h: chunks of 512 k, [tile][chunk][16 steps][64 lanes][8],
// lane 16 g + c of step 4 j + s holding column c's k 512 chunk + 128 g + 32 j + 8
// s .. + 7: what a lane that decodes 16 packed bytes (32 k) four times needs.

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <utility>

#include "dq4.h"
#include "dq4_device.h"
#include "dq4_linear.h"
#include "dq4_linear_device.h"
#include "dq4_moe.h"

#pragma clang fp contract(off)

namespace dq4 {
namespace {

constexpr int kMaxTokens = DQ4_MOE_MAX_TOKENS, kMaxExperts = DQ4_MOE_MAX_EXPERTS,
              kMaxTopK = DQ4_MOE_MAX_TOP_K;
constexpr int64_t kMaxWidth = int64_t{1} << 17, kMaxWeight = int64_t{1} << 40, kMaxRows = int64_t{1} << 21;
constexpr int kSpan = 512;                     // k of a chunk
constexpr int kTileChunk = 16 * 64 * 8;        // elements of a tile's chunk

// ---------------------------------------------------------------------------
// the router
// ---------------------------------------------------------------------------
struct RouteArgs {
    const uint16_t *x;
    int64_t m, n_in, ld_x;
    const uint16_t *router;
    const float *bias;
    int32_t n_experts, top_k, renormalize;
    int32_t vec;
    int32_t *ids;
    float *weights;
};

// A token per workgroup.  A wave takes every 16th expert, four at a time; the
// products are exact in FP32 and their sums run in 64 bits, since the choice
// between two experts hangs on the last place.  An expert's rank is the number of
// experts before it.  Bound by the reading of the router's matrix from cache by
// one CU (64 experts x 2048: 256 KiB).
constexpr int kRouteWaves = 16, kRouteExperts = 4;

template <int OUT>
__global__ __launch_bounds__(64 * kRouteWaves) void moe_route_kernel(RouteArgs a)
{
    __shared__ double logit[kMaxExperts];
    __shared__ double best[kMaxTopK];
    __shared__ float share[kMaxExperts];
    __shared__ int any_nan;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int E = a.n_experts;
    const int k = static_cast<int>(a.n_in);
    for (int64_t t = blockIdx.x; t < a.m; t += gridDim.x) {
        const uint16_t *x = a.x + t * a.ld_x;
        for (int e0 = wave * kRouteExperts; e0 < E; e0 += kRouteWaves * kRouteExperts) {
            double sum[kRouteExperts] = {};
            for (int c = lane * 8; c < k; c += 512) {
                const int valid = k - c < 8 ? k - c : 8;
                float xv[8];
                load_values<OUT, 8>(x + c, a.vec, valid, xv);
#pragma unroll
                for (int q = 0; q < kRouteExperts; ++q) {
                    const int e = e0 + q < E ? e0 + q : E - 1;
                    float r[8];
                    load_values<OUT, 8>(a.router + static_cast<int64_t>(e) * k + c, a.vec, valid, r);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        sum[q] = sum[q] + static_cast<double>(xv[j] * r[j]);
                }
            }
#pragma unroll
            for (int q = 0; q < kRouteExperts; ++q) {
#pragma unroll
                for (int d = 32; d > 0; d /= 2)
                    sum[q] = sum[q] + __shfl_xor(sum[q], d);
                if (lane == 0 && e0 + q < E)
                    logit[e0 + q] = a.bias ? sum[q] + static_cast<double>(a.bias[e0 + q]) : sum[q];
            }
        }
        if (tid == 0)
            any_nan = 0;
        __syncthreads();
        const double minus_infinity = -__builtin_inf();
        if (tid < E) {
            const double mine = logit[tid];
            const bool nan = mine != mine;
            if (nan)
                any_nan = 1;
            int rank = 0;
            for (int e = 0; e < E; ++e) {
                const double other = logit[e];
                const bool before = nan ? other == other ? other != minus_infinity : e < tid
                                        : other > mine || (other == mine && e < tid);
                rank += before ? 1 : 0;
            }
            if (mine != minus_infinity && rank < a.top_k) {
                a.ids[t * a.top_k + rank] = tid;
                best[rank] = mine;
            }
        }
        // places that no expert is left for: as many experts as are not masked
        int chosen = 0;
        for (int e = 0; e < E && chosen < a.top_k; ++e)
            chosen += logit[e] != minus_infinity ? 1 : 0;
        __syncthreads();
        const double top = chosen > 0 ? best[0] : 0.0;
        if (tid < E)
            share[tid] = exp_f32(static_cast<float>(logit[tid] - top));
        __syncthreads();
        if (tid < a.top_k) {
            float total = 0.0f;
            if (a.renormalize) {
                for (int j = 0; j < chosen; ++j)
                    total = total + exp_f32(static_cast<float>(best[j] - top));
            } else {
                for (int e = 0; e < E; ++e)
                    total = total + share[e];
            }
            float w = 0.0f;
            if (tid < chosen)
                w = any_nan ? __builtin_nanf("")
                            : exp_f32(static_cast<float>(best[tid] - top)) * __builtin_amdgcn_rcpf(total);
            else
                a.ids[t * a.top_k + tid] = -1;
            a.weights[t * a.top_k + tid] = w;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// the plan
// ---------------------------------------------------------------------------
// A pass goes over one expert's matrices with up to `tf` tiles of its tokens.
struct Pass {
    int32_t expert, x_tile, h_tile, tiles;
};

struct MoeArgs {
    Weight w[3];             // gate, up, down
    int32_t log2_block, log2_down;
    int32_t n_experts, top_k;
    int64_t n_ff, n_in, m;
    int32_t act, tf;
    const uint16_t *x;
    int64_t ld_x;
    const int32_t *ids;
    const float *weights;
    int32_t vec_x, vec_y;
    int32_t max_tiles;
    int32_t *n_units;
    Pass *units;
    int32_t *token_of;       // [h tile][16]: the column's token, or -1
    float *share_of;         // [h tile][16]: its weight for the tile's expert
    uint16_t *x_frags, *h_frags;
    const uint16_t *residual;
    int64_t ld_residual;
    uint16_t *y;
    int64_t ld_y;
};

__device__ __forceinline__ int chunks_of(int64_t k)
{
    return static_cast<int>((k + kSpan - 1) / kSpan);
}

// Every workgroup works the plan out for itself (up to 1024 choices, a mask of
// tokens for each expert); workgroup 0 writes it, and all write x tiles in operand
// order, with zeros where there is no token or no k, and zeros for the k of h that
// the products leave out.
__global__ __launch_bounds__(512) void moe_plan_zero_fill(MoeArgs a)
{
    __shared__ uint32_t mask[kMaxExperts][2];
    __shared__ int tile0[kMaxExperts];
    __shared__ int sums[8];
    __shared__ int token[16];
    const int tid = threadIdx.x;
    const int m = static_cast<int>(a.m), pairs = m * a.top_k;
    mask[tid][0] = mask[tid][1] = 0;
    __syncthreads();
    for (int p = tid; p < pairs; p += 512) {
        const int e = a.ids[p], t = p / a.top_k;
        if (e >= 0 && e < a.n_experts)
            atomicOr(&mask[e][t >> 5], 1u << (t & 31));
    }
    __syncthreads();
    const bool one_tile = m <= 16;  // the tile of all tokens
    const int count = __builtin_popcount(mask[tid][0]) + __builtin_popcount(mask[tid][1]);
    const int tiles = count == 0 ? 0 : one_tile ? 1 : (count + 15) / 16;
    const int passes = (tiles + a.tf - 1) / a.tf;
    int n_tiles, n_units;
    const int my_tile = list_position<512>(tiles, &n_tiles, sums);
    tile0[tid] = my_tile;
    const int my_unit = list_position<512>(passes, &n_units, sums);
    // where a choice's token lies among its expert's
    const auto tile_column = [&](int e, int t) {
        const uint32_t below = (1u << (t & 31)) - 1;
        const int slot = one_tile ? t
                         : t < 32 ? __builtin_popcount(mask[e][0] & below)
                                  : __builtin_popcount(mask[e][0]) + __builtin_popcount(mask[e][1] & below);
        return tile0[e] * 16 + slot;
    };
    if (blockIdx.x == 0) {
        if (tid == 0)
            *a.n_units = n_units;
        for (int q = 0; q < passes; ++q) {
            const int left = tiles - q * a.tf;
            a.units[my_unit + q] = Pass{tid, one_tile ? 0 : my_tile + q * a.tf, my_tile + q * a.tf,
                                        left < a.tf ? left : a.tf};
        }
        for (int i = tid; i < n_tiles * 16; i += 512)
            a.token_of[i] = -1;
        __syncthreads();  // (and tile0 is complete)
        for (int p = tid; p < pairs; p += 512) {
            const int e = a.ids[p], t = p / a.top_k, j = p - t * a.top_k;
            if (e < 0 || e >= a.n_experts)
                continue;
            // an expert's first place in the row stands for all of its places
            bool first = true;
            for (int i = 0; i < j; ++i)
                first = first && a.ids[t * a.top_k + i] != e;
            if (!first)
                continue;
            float w = a.weights[p];
            for (int i = j + 1; i < a.top_k; ++i)
                if (a.ids[t * a.top_k + i] == e)
                    w = w + a.weights[t * a.top_k + i];
            const int at = tile_column(e, t);
            a.token_of[at] = t;
            a.share_of[at] = w;
        }
    }
    const int x_tiles = one_tile ? (n_tiles > 0 ? 1 : 0) : n_tiles;
    const int chunks = chunks_of(a.n_in), h_chunks = chunks_of(a.n_ff);
    const int h_from = static_cast<int>((a.n_ff + 15) / 16 * 16);
    // pieces of a tile's x: one chunk each
    for (int item = blockIdx.x; item < n_tiles * chunks; item += gridDim.x) {
        const int tile = item / chunks, ch = item - tile * chunks;
        __syncthreads();  // the last item's tokens are read
        if (tid < 16)
            token[tid] = one_tile && tid < m ? tid : -1;
        __syncthreads();
        if (!one_tile)
            for (int p = tid; p < pairs; p += 512) {
                const int e = a.ids[p], t = p / a.top_k;
                if (e < 0 || e >= a.n_experts)
                    continue;
                const int at = tile_column(e, t);
                if (at >> 4 == tile)
                    token[at & 15] = t;
            }
        __syncthreads();
        if (tile < x_tiles) {
            uint16_t *to = a.x_frags + (static_cast<int64_t>(tile) * chunks + ch) * kTileChunk;
            for (int u = tid; u < 1024; u += 512) {
                const int lane = u & 63, step = u >> 6;
                const int t = token[lane & 15];
                const int k0 = ch * kSpan + 128 * (lane >> 4) + 8 * step;
                u32x4 q = {0, 0, 0, 0};
                if (t >= 0 && k0 < a.n_in) {
                    const uint16_t *from = a.x + t * a.ld_x + k0;
                    if (a.vec_x) {
                        q = *reinterpret_cast<const u32x4 *>(from);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (k0 + j < a.n_in)
                                q[j / 2] |= static_cast<uint32_t>(from[j]) << (16 * (j & 1));
                    }
                }
                *reinterpret_cast<u32x4 *>(to + u * 8) = q;
            }
        }
        if (ch == 0 && h_chunks > 0) {
            uint16_t *to = a.h_frags + (static_cast<int64_t>(tile) * h_chunks + h_chunks - 1) * kTileChunk;
            for (int u = tid; u < 1024; u += 512) {
                const int k0 = (h_chunks - 1) * kSpan + 128 * ((u & 63) >> 4) + 8 * (u >> 6);
                if (k0 >= h_from)
                    *reinterpret_cast<u32x4 *>(to + u * 8) = u32x4{0, 0, 0, 0};
            }
        }
    }
}

// ---------------------------------------------------------------------------
// 16 rows of a 4-bit weight, one chunk of 512 k, as 16 operands
// ---------------------------------------------------------------------------
// Rows of a weight matrix of one expert: `rows` of them from global row `row0` on.
struct RowBlock {
    int64_t row0;
    int rows;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_from(const void *p, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0,
                                             static_cast<int32_t>(bytes < 0x7FFFFFF0 ? bytes : 0x7FFFFFF0),
                                             kRawBufferWord3);
}

// Row lengths that are multiples of 32, packed codes at 4-byte boundaries.  A load
// takes 256 bytes of 4 rows, a quad of lanes on 64 of them; 4 such loads are
// transposed between the lanes of each quad; the scales, S blocks per 128 k, are
// looked up four lanes to a row and handed over.  S = 2: blocks of 64 k or more and
// row lengths that are multiples of 64; else S = 4.
template <int OUT, int S>
struct EvenRows {
    static constexpr bool kAhead = true;  // the registers hold the next chunk's loads
    u32x4 packed[4];
    uint32_t code[S];
    float absmax[S];
    uint32_t from[4];
    float s[4];

    __device__ __forceinline__ void load(const Weight &w, int lb, int64_t n_elems, const RowBlock &b,
                                         uint32_t n, int c, int lane)
    {
        const int64_t e0 = b.row0 * n, b0 = e0 >> lb;
        const uint32_t phase = static_cast<uint32_t>(e0) & ((1u << lb) - 1);
        const uint32_t group_phase = static_cast<uint32_t>(b0) & 255;
        const int64_t blocks = (n_elems + (int64_t{1} << lb) - 1) >> lb;
        const auto rp = buffer_from(w.packed + (e0 >> 1), ((n_elems + 1) >> 1) - (e0 >> 1));
        const auto rc = buffer_from(w.scale_codes + b0, blocks - b0);
        const auto rm = buffer_from(w.nested_absmax + (b0 >> kNestedLog2),
                                    (((blocks + 255) >> kNestedLog2) - (b0 >> kNestedLog2)) * 4);
        const uint32_t k = c * kSpan + 32 * (((lane >> 4) << 2) | (lane & 3));
        const int row = 4 * ((lane >> 2) & 3);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            packed[q] = __builtin_amdgcn_raw_buffer_load_b128(
                rp, k < n && row + q < b.rows ? ((row + q) * n + k) >> 1 : 0x80000000u, 0, 0);
#pragma unroll
        for (int h = 0; h < S; ++h) {
            const uint32_t e = (lane >> 2) * n + c * kSpan + 128 * (lane & 3) + h * (128 / S);
            const uint32_t blk = (phase + e) >> lb;
            code[h] = __builtin_amdgcn_raw_buffer_load_b8(rc, blk, 0, 0);
            absmax[h] = __builtin_bit_cast(
                float, __builtin_amdgcn_raw_buffer_load_b32(rm, ((group_phase + blk) >> kNestedLog2) * 4, 0, 0));
        }
    }

    // `zeros`: the table's row of zeros, which a piece beyond the row or the last
    // row (its load gave zeros) reads, times 0.
    __device__ __forceinline__ void prepare(const float *scb, float offset, const RowBlock &b, uint32_t n, int c,
                                            uint32_t lane_byte, int lane)
    {
        const int g = lane >> 4, r = lane & 15;
        float given[S];
#pragma unroll
        for (int h = 0; h < S; ++h) {
            const float q = block_scale(scb[code[h]], absmax[h], offset);
            // lane 16 g + r multiplies quarter g of row r
            given[h] = __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute((4 * r + g) * 4,
                                                                              __builtin_bit_cast(int, q)));
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            uint32_t v[4] = {packed[0][d], packed[1][d], packed[2][d], packed[3][d]};
            transpose_quads(v, lane & 1, lane & 2);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                packed[j][d] = v[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool beyond = c * kSpan + 128 * g + 32 * j >= n || r >= b.rows;
            from[j] = beyond ? lane_byte | kPairTableBytes : lane_byte;
            s[j] = beyond ? 0.0f : given[j * S / 4];
        }
    }

    __device__ __forceinline__ Pairs look(const uint8_t *table, int step) const
    {
        return lookup_dword(packed[step / 4][step % 4], table, from[step / 4]);
    }

    __device__ __forceinline__ u32x4 operand(const Pairs &p, int step) const
    {
        return scaled_dword<OUT>(p, s[step / 4]);
    }
};

// Any row length and alignment: a lane takes its own row's 32 k, five dwords that
// are shifted to its first nibble.  Blocks are at least 32 elements long, so a
// piece meets at most two; each element picks its scale.  Dwords are read up to the
// one with the last byte.
template <int OUT>
struct AnyRows {
    static constexpr bool kAhead = false;
    u32x4 lo[4];
    uint32_t hi[4];
    uint32_t code[4][2];
    float absmax[4][2];
    uint32_t shift;
    int meet[4], valid[4];
    float s[4][2];
    uint32_t from;

    __device__ __forceinline__ void load(const Weight &w, int lb, int64_t n_elems, const RowBlock &b, uint32_t n,
                                         int c, int lane)
    {
        const int64_t e0 = b.row0 * n, b0 = e0 >> lb;
        const uint32_t phase = static_cast<uint32_t>(e0) & ((1u << lb) - 1);
        const uint32_t group_phase = static_cast<uint32_t>(b0) & 255;
        const int64_t blocks = (n_elems + (int64_t{1} << lb) - 1) >> lb;
        const uintptr_t at = reinterpret_cast<uintptr_t>(w.packed) + (e0 >> 1);
        const uint32_t skew = static_cast<uint32_t>(at & 3);
        const auto rp = buffer_from(reinterpret_cast<const void *>(at - skew),
                                    (((n_elems + 1) >> 1) - (e0 >> 1) + skew + 3) & ~int64_t{3});
        const auto rc = buffer_from(w.scale_codes + b0, blocks - b0);
        const auto rm = buffer_from(w.nested_absmax + (b0 >> kNestedLog2),
                                    (((blocks + 255) >> kNestedLog2) - (b0 >> kNestedLog2)) * 4);
        const int r = lane & 15;
        const uint32_t nibble0 = 2 * skew + (static_cast<uint32_t>(e0) & 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t k = c * kSpan + 128 * (lane >> 4) + 32 * j;
            const int left = r < b.rows ? static_cast<int>(n) - static_cast<int>(k) : 0;
            valid[j] = left < 0 ? 0 : left > 32 ? 32 : left;
            const uint32_t e = r * n + k;
            const uint32_t nibble = nibble0 + e;
            shift = 4 * (nibble & 7);  // the same for all j
            const uint32_t word = valid[j] > 0 ? (nibble >> 3) * 4 : 0x80000000u;
            lo[j] = __builtin_amdgcn_raw_buffer_load_b128(rp, word, 0, 0);
            hi[j] = __builtin_amdgcn_raw_buffer_load_b32(rp, word + 16, 0, 0);
            const uint32_t blk = (phase + e) >> lb;
            meet[j] = static_cast<int>(((blk + 1) << lb) - phase - e);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                code[j][h] = __builtin_amdgcn_raw_buffer_load_b8(rc, valid[j] > 0 ? blk + h : 0x80000000u, 0, 0);
                absmax[j][h] = __builtin_bit_cast(
                    float, __builtin_amdgcn_raw_buffer_load_b32(
                               rm, valid[j] > 0 ? ((group_phase + blk + h) >> kNestedLog2) * 4 : 0x80000000u, 0, 0));
            }
        }
    }

    __device__ __forceinline__ void prepare(const float *scb, float offset, const RowBlock &, uint32_t, int,
                                            uint32_t lane_byte, int)
    {
        from = lane_byte;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                s[j][h] = block_scale(scb[code[j][h]], absmax[j][h], offset);
    }

    __device__ __forceinline__ Pairs look(const uint8_t *table, int step) const
    {
        const int j = step / 4, d = step % 4;
        return lookup_dword(__builtin_amdgcn_alignbit(d < 3 ? lo[j][d + 1] : hi[j], lo[j][d], shift), table, from);
    }

    __device__ __forceinline__ u32x4 operand(const Pairs &p, int step) const
    {
        const int j = step / 4, d = step % 4;
        u32x4 q;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = 8 * d + 2 * i + h;
                const float z = p.v[i][h] * (at < meet[j] ? s[j][0] : s[j][1]);
                v[h] = at < valid[j] ? z : 0.0f;
            }
            q[i] = Half<OUT>::pack2(v[0], v[1]);
        }
        return q;
    }
};

// ---------------------------------------------------------------------------
// gate and up
// ---------------------------------------------------------------------------
// An item is a unit's row block: 16 rows of the expert's gate and the same of its
// up matrix.  The 8 waves take its chunks in turn, their sums meet in LDS in a
// fixed order, and h goes out in the down product's operand order.  The next
// chunk's weight, also that of the next item, is in flight while one is
// multiplied.
template <int OUT, class Rows, int TF>
__global__ __launch_bounds__(512) void moe_gate_up_kernel(MoeArgs a)
{
    __shared__ __attribute__((aligned(1024))) uint8_t table[kPairTableBytes + 256];
    __shared__ float scb[2][256], cb4[2][16];
    __shared__ __attribute__((aligned(16))) f32x4 partial[8][2 * TF][64];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t n = static_cast<uint32_t>(a.n_in);
    const int n_ff = static_cast<int>(a.n_ff);
    const int chunks = chunks_of(a.n_in), h_chunks = chunks_of(a.n_ff);
    const int row_blocks = (n_ff + 15) >> 4;
    const int64_t n_elems = static_cast<int64_t>(a.n_experts) * a.n_ff * a.n_in;
    const Weight pair[2] = {a.w[0], a.w[1]};

    const Codebooks codebooks = fetch_codebooks<2>(pair);
    const int items = *a.n_units * row_blocks;
    int next_item = blockIdx.x, next_c = wave;
    Pass unit{}, next_unit{};
    RowBlock rows{}, next_rows{};
    const auto enter = [&](int item) {
        const int u = item / row_blocks;
        next_unit = a.units[u];
        const int row = (item - u * row_blocks) * 16;
        next_rows = RowBlock{static_cast<int64_t>(next_unit.expert) * n_ff + row, n_ff - row < 16 ? n_ff - row : 16};
    };
    Rows cur[2], next[2];
    const bool some = wave < chunks;
    if (next_item < items) {
        enter(next_item);
        if (some && Rows::kAhead)
#pragma unroll
            for (int f = 0; f < 2; ++f)
                next[f].load(a.w[f], a.log2_block, n_elems, next_rows, n, next_c, lane);
    }
    fill_tables<2, 1>(codebooks, table, scb, cb4);
    const uint32_t lane_byte = (lane & 15) * 16;

    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        unit = next_unit;
        rows = next_rows;
        f32x4 acc[2][TF];
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                acc[f][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int c = wave; c < chunks; c += 8) {
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                if constexpr (Rows::kAhead)
                    cur[f] = next[f];
                else
                    cur[f].load(a.w[f], a.log2_block, n_elems, rows, n, c, lane);
            }
            next_c += 8;
            if (next_c >= chunks) {
                next_c = wave;
                next_item += gridDim.x;
                if (next_item < items)
                    enter(next_item);
            }
            // past the last item: the last one's again, unused
            if constexpr (Rows::kAhead)
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    next[f].load(a.w[f], a.log2_block, n_elems, next_rows, n, next_c, lane);
#pragma unroll
            for (int f = 0; f < 2; ++f)
                cur[f].prepare(scb[f], a.w[f].offset, rows, n, c, lane_byte, lane);
            const uint16_t *x[TF];
#pragma unroll
            for (int t = 0; t < TF; ++t)  // past the unit's last tile: that again, unused
                x[t] = a.x_frags +
                       (static_cast<int64_t>(unit.x_tile + (t < unit.tiles ? t : unit.tiles - 1)) * chunks + c) *
                           kTileChunk + lane * 8;
            constexpr int kAhead = 4;
            u32x4 xf[kAhead][TF];
#pragma unroll
            for (int st = 0; st < kAhead; ++st)
#pragma unroll
                for (int t = 0; t < TF; ++t)
                    xf[st][t] = *reinterpret_cast<const u32x4 *>(x[t] + st * 512);
            Pairs now[2], then[2];
#pragma unroll
            for (int f = 0; f < 2; ++f)
                now[f] = cur[f].look(table + f * 8, 0);
#pragma unroll
            for (int st = 0; st < 16; ++st) {
                if (st < 15)
#pragma unroll
                    for (int f = 0; f < 2; ++f)
                        then[f] = cur[f].look(table + f * 8, st + 1);
                keep_order();
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const u32x4 wf = cur[f].operand(now[f], st);
#pragma unroll
                    for (int t = 0; t < TF; ++t)
                        acc[f][t] = Half<OUT>::mfma(wf, xf[st % kAhead][t], acc[f][t]);
                    now[f] = then[f];
                }
                if (st + kAhead < 16)
#pragma unroll
                    for (int t = 0; t < TF; ++t)
                        xf[st % kAhead][t] = *reinterpret_cast<const u32x4 *>(x[t] + (st + kAhead) * 512);
            }
        }
        if (!some) {  // this wave has no chunk: it follows the items all the same
            next_item += gridDim.x;
            if (next_item < items)
                enter(next_item);
        }
        lds_barrier();  // the last item's sums are read
        if (some)
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int t = 0; t < TF; ++t)
                    partial[wave][f * TF + t][lane] = acc[f][t];
        lds_barrier();
        const int live = chunks < 8 ? chunks : 8;
        if (wave < unit.tiles) {  // a wave finishes one tile
            const int t = wave;
            f32x4 gate = {0.0f, 0.0f, 0.0f, 0.0f}, up = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int q = 0; q < live; ++q) {
                gate = gate + partial[q][t][lane];
                up = up + partial[q][TF + t][lane];
            }
            // the lane's four neighbouring k of h, column lane % 16
            const int k = (item - item / row_blocks * row_blocks) * 16 + 4 * (lane >> 4);
            float h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[i] = k + i < n_ff ? act_f32(a.act, gate[i]) * up[i] : 0.0f;
            const int ch = k / kSpan, in = k % kSpan;
            uint16_t *to = a.h_frags + (static_cast<int64_t>(unit.h_tile + t) * h_chunks + ch) * kTileChunk +
                           (((in & 127) >> 3) * 64 + (in >> 7) * 16 + (lane & 15)) * 8 + (in & 7);
            *reinterpret_cast<u32x2 *>(to) = u32x2{Half<OUT>::pack2(h[0], h[1]), Half<OUT>::pack2(h[2], h[3])};
        }
    }
}

// ---------------------------------------------------------------------------
// down, and the sum over a token's experts
// ---------------------------------------------------------------------------
// A workgroup takes 16 output columns and walks all units: its waves take the
// (unit, chunk) pairs in turn, multiply a unit's sums by its tokens' weights and
// add them to their own sums for every token, in a fixed order; the waves' sums
// meet at the end.  So a token's experts are added up without a pass of their own.
template <int OUT, class Rows, int TF>
__global__ __launch_bounds__(512) void moe_down_kernel(MoeArgs a)
{
    __shared__ __attribute__((aligned(1024))) uint8_t table[kPairTableBytes + 256];
    __shared__ float scb[1][256], cb4[1][16];
    __shared__ __attribute__((aligned(16))) float sums[8][kMaxTokens][16];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t n = static_cast<uint32_t>(a.n_ff);
    const int n_out = static_cast<int>(a.n_in);
    const int chunks = chunks_of(a.n_ff);
    const int64_t n_elems = static_cast<int64_t>(a.n_experts) * a.n_ff * a.n_in;
    const Weight one[2] = {a.w[2], a.w[2]};

    const Codebooks codebooks = fetch_codebooks<1>(one);
    const int items = *a.n_units * chunks;
    const int row_blocks = (n_out + 15) >> 4;
    Pass next_unit{};
    RowBlock next_rows{};
    int next_c = 0;
    const auto enter = [&](int row_block, int item) {
        const int u = item / chunks;
        next_unit = a.units[u];
        next_c = item - u * chunks;
        const int row = row_block * 16;
        next_rows = RowBlock{static_cast<int64_t>(next_unit.expert) * n_out + row,
                             n_out - row < 16 ? n_out - row : 16};
    };
    Rows cur, next;
    const bool some = wave < items;
    if (some) {
        enter(blockIdx.x, wave);
        if constexpr (Rows::kAhead)
            next.load(a.w[2], a.log2_down, n_elems, next_rows, n, next_c, lane);
    }
    fill_tables<1, 1>(codebooks, table, scb, cb4);
    const uint32_t lane_byte = (lane & 31) * 8;

    for (int row_block = blockIdx.x; row_block < row_blocks; row_block += gridDim.x) {
        for (int i = lane; i < kMaxTokens * 4; i += 64)
            reinterpret_cast<f32x4 *>(&sums[wave][0][0])[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        f32x4 acc[TF];
#pragma unroll
        for (int t = 0; t < TF; ++t)
            acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int item = wave; item < items; item += 8) {
            if constexpr (Rows::kAhead)
                cur = next;
            else
                cur.load(a.w[2], a.log2_down, n_elems, next_rows, n, next_c, lane);
            const Pass unit = next_unit;
            const RowBlock rows = next_rows;
            const int c = next_c;
            const bool last = item + 8 >= items;
            if (!last)
                enter(row_block, item + 8);
            else if (row_block + static_cast<int>(gridDim.x) < row_blocks)
                enter(row_block + gridDim.x, wave);
            // past the last item: the same again, unused
            if constexpr (Rows::kAhead)
                next.load(a.w[2], a.log2_down, n_elems, next_rows, n, next_c, lane);
            cur.prepare(scb[0], a.w[2].offset, rows, n, c, lane_byte, lane);
            const uint16_t *h[TF];
#pragma unroll
            for (int t = 0; t < TF; ++t)
                h[t] = a.h_frags +
                       (static_cast<int64_t>(unit.h_tile + (t < unit.tiles ? t : unit.tiles - 1)) * chunks + c) *
                           kTileChunk + lane * 8;
            constexpr int kAhead = 4;
            u32x4 hf[kAhead][TF];
#pragma unroll
            for (int st = 0; st < kAhead; ++st)
#pragma unroll
                for (int t = 0; t < TF; ++t)
                    hf[st][t] = *reinterpret_cast<const u32x4 *>(h[t] + st * 512);
            Pairs now = cur.look(table, 0), then{};
#pragma unroll
            for (int st = 0; st < 16; ++st) {
                if (st < 15)
                    then = cur.look(table, st + 1);
                keep_order();
                const u32x4 wf = cur.operand(now, st);
#pragma unroll
                for (int t = 0; t < TF; ++t)
                    acc[t] = Half<OUT>::mfma(wf, hf[st % kAhead][t], acc[t]);
                now = then;
                if (st + kAhead < 16)
#pragma unroll
                    for (int t = 0; t < TF; ++t)
                        hf[st % kAhead][t] = *reinterpret_cast<const u32x4 *>(h[t] + (st + kAhead) * 512);
            }
            // the wave's next pair is of another unit: this one's sums to its tokens
            if (last || next_unit.h_tile != unit.h_tile) {
#pragma unroll
                for (int t = 0; t < TF; ++t) {
                    if (t < unit.tiles) {
                        const int at = (unit.h_tile + t) * 16 + (lane & 15);
                        const int token = a.token_of[at];
                        if (token >= 0) {
                            const float w = a.share_of[at];
                            f32x4 *to = reinterpret_cast<f32x4 *>(&sums[wave][token][4 * (lane >> 4)]);
                            f32x4 v = *to;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                v[i] = v[i] + w * acc[t][i];
                            *to = v;
                        }
                    }
                    acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                }
            }
        }
        lds_barrier();
        if (tid < a.m * 4) {
            const int token = tid >> 2, i0 = 4 * (tid & 3);
            f32x4 z = *reinterpret_cast<const f32x4 *>(&sums[0][token][i0]);
#pragma unroll
            for (int q = 1; q < 8; ++q)
                z = z + *reinterpret_cast<const f32x4 *>(&sums[q][token][i0]);
            const int n0 = row_block * 16 + i0;
            const int valid = n_out - n0 < 4 ? n_out - n0 : 4;
            if (valid > 0) {
                const bool vec = a.vec_y && valid == 4;
                float out[4] = {z[0], z[1], z[2], z[3]};
                if (a.residual) {
                    float r[4];
                    load_values<OUT, 4>(a.residual + token * a.ld_residual + n0, vec, valid, r);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        out[i] = out[i] + r[i];
                }
                store_values<OUT, 4>(a.y + token * a.ld_y + n0, vec, valid, out);
            }
        }
        lds_barrier();  // the sums are read
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Tiles of a pass over an expert: as many as its share of the tokens is likely to
// fill, if they spread evenly, up to two (registers); an expert with more takes
// more passes.  (Up to 16 tokens there is one tile.)
int tiles_per_pass(int64_t m, int64_t top_k, int64_t n_experts)
{
    return m <= 16 || m * top_k <= 8 * n_experts ? 1 : 2;
}

// What the workspace holds, in this order.
struct Layout {
    int64_t max_tiles;  // at most this many tiles, and units
    int64_t units, tokens, shares, x, h, all;
};

Layout layout_of(int64_t n_experts, int64_t n_ff, int64_t n_in, int64_t m, int64_t top_k)
{
    Layout l{};
    const int64_t pairs = m * top_k;
    // an expert's last tile may hold one token alone
    l.max_tiles = (pairs < n_experts ? pairs : n_experts) + pairs / 16;
    l.units = 256;
    l.tokens = l.units + align256(l.max_tiles * static_cast<int64_t>(sizeof(Pass)));
    l.shares = l.tokens + align256(l.max_tiles * 64);
    l.x = l.shares + align256(l.max_tiles * 64);
    l.h = l.x + (m <= 16 ? 1 : l.max_tiles) * ceil_div(n_in, kSpan) * kTileChunk * 2;
    l.all = l.h + l.max_tiles * ceil_div(n_ff, kSpan) * kTileChunk * 2;
    return l;
}

bool sizes_fit(int64_t n_experts, int64_t n_ff, int64_t n_in, int64_t m, int64_t top_k)
{
    return n_experts <= kMaxExperts && top_k <= kMaxTopK && m <= kMaxTokens && n_ff <= kMaxWidth &&
           n_in <= kMaxWidth && n_experts * n_ff * n_in <= kMaxWeight;
}

bool four_aligned(const void *p)
{
    return reinterpret_cast<uintptr_t>(p) % 4 == 0;
}

template <int OUT, class Rows>
const void *gate_up_kernel(int tf)
{
    return tf == 1 ? reinterpret_cast<const void *>(&moe_gate_up_kernel<OUT, Rows, 1>)
                   : reinterpret_cast<const void *>(&moe_gate_up_kernel<OUT, Rows, 2>);
}

template <int OUT, class Rows>
const void *down_kernel(int tf)
{
    return tf == 1 ? reinterpret_cast<const void *>(&moe_down_kernel<OUT, Rows, 1>)
                   : reinterpret_cast<const void *>(&moe_down_kernel<OUT, Rows, 2>);
}

template <int OUT>
dq4_status_t run_moe(MoeArgs a, int cus, hipStream_t s)
{
    void *params[] = {&a};
    const int64_t pieces = a.max_tiles * ceil_div(a.n_in, kSpan);
    dq4_status_t st = launch(reinterpret_cast<const void *>(&moe_plan_zero_fill), pieces < cus ? pieces : cus, 1, 512,
                             params, s);
    if (st != DQ4_OK)
        return st;
    if (a.n_ff > 0) {
        const bool even = a.n_in % 32 == 0 && four_aligned(a.w[0].packed) && four_aligned(a.w[1].packed);
        const void *kernel = !even ? gate_up_kernel<OUT, AnyRows<OUT>>(a.tf)
                             : a.log2_block >= 6 && a.n_in % 64 == 0 ? gate_up_kernel<OUT, EvenRows<OUT, 2>>(a.tf)
                                                                     : gate_up_kernel<OUT, EvenRows<OUT, 4>>(a.tf);
        const int64_t most = a.max_tiles * ceil_div(a.n_ff, 16);
        st = launch(kernel, most < cus ? most : cus, 1, 512, params, s);
        if (st != DQ4_OK)
            return st;
    }
    const bool even = a.n_ff % 32 == 0 && four_aligned(a.w[2].packed);
    const void *kernel = !even ? down_kernel<OUT, AnyRows<OUT>>(a.tf)
                         : a.log2_down >= 6 && a.n_ff % 64 == 0 ? down_kernel<OUT, EvenRows<OUT, 2>>(a.tf)
                                                                : down_kernel<OUT, EvenRows<OUT, 4>>(a.tf);
    const int64_t row_blocks = ceil_div(a.n_in, 16);
    return launch(kernel, row_blocks < cus ? row_blocks : cus, 1, 512, params, s);
}

}  // namespace
}  // namespace dq4

using namespace dq4;

extern "C" {

dq4_status_t dq4_moe_route(const void *x, int64_t m, int64_t n_in, int64_t ld_x, int32_t dtype,
                           const void *router, const float *bias, int32_t n_experts, int32_t top_k,
                           int32_t renormalize, int32_t *ids, float *weights, void *stream)
{
    if (m < 0 || n_in < 0 || n_experts < 0 || (dtype != DQ4_F16 && dtype != DQ4_BF16) || top_k < 1 ||
        top_k > n_experts)
        return DQ4_EINVAL;
    if (n_experts > kMaxExperts || top_k > kMaxTopK || m > kMaxRows || n_in > kMaxWidth)
        return DQ4_EUNSUPPORTED;
    if (m == 0)
        return DQ4_OK;
    if (!ids || !weights || (n_in > 0 && (!x || !router)) || bad_ld(ld_x, m, n_in))
        return DQ4_EINVAL;
    RouteArgs a{};
    a.x = static_cast<const uint16_t *>(x);
    a.m = m;
    a.n_in = n_in;
    a.ld_x = ld_x;
    a.router = static_cast<const uint16_t *>(router);
    a.bias = bias;
    a.n_experts = n_experts;
    a.top_k = top_k;
    a.renormalize = renormalize != 0;
    a.vec = rows_aligned(x, ld_x, m, n_in) && reinterpret_cast<uintptr_t>(router) % 16 == 0;
    a.ids = ids;
    a.weights = weights;
    void *params[] = {&a};
    const int64_t most = current_compute_units() * int64_t{8};
    return launch(dtype == DQ4_F16 ? reinterpret_cast<const void *>(&moe_route_kernel<DQ4_F16>)
                                   : reinterpret_cast<const void *>(&moe_route_kernel<DQ4_BF16>),
                  m < most ? m : most, 1, 64 * kRouteWaves, params, static_cast<hipStream_t>(stream));
}

int64_t dq4_moe_fused_workspace_bytes(int32_t n_experts, int64_t n_ff, int64_t n_in, int64_t m, int32_t top_k)
{
    if (n_experts <= 0 || n_ff < 0 || n_in <= 0 || m <= 0 || top_k <= 0 ||
        !sizes_fit(n_experts, n_ff, n_in, m, top_k))
        return 0;
    return layout_of(n_experts, n_ff, n_in, m, top_k).all;
}

dq4_status_t dq4_moe_fused(const dq4_weight_t *gate, const dq4_weight_t *up, const dq4_weight_t *down,
                           int32_t n_experts, int64_t n_ff, int64_t n_in, int32_t dtype, int32_t activation,
                           const void *x, int64_t m, int64_t ld_x, const int32_t *ids, const float *weights,
                           int32_t top_k, const void *residual, int64_t ld_residual, void *y, int64_t ld_y,
                           void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!gate || !up || !down || (dtype != DQ4_F16 && dtype != DQ4_BF16))
        return DQ4_EINVAL;
    int log2_block = 0, log2_up = 0, log2_down = 0;
    for (const auto &[w, log2] : {std::pair<const dq4_weight_t *, int *>{gate, &log2_block}, {up, &log2_up},
                                  {down, &log2_down}}) {
        const dq4_status_t st = validate_layout(w->blocksize, w->nested_blocksize, dtype, log2);
        if (st != DQ4_OK)
            return st;
    }
    if (log2_up != log2_block)
        return DQ4_EUNSUPPORTED;
    if (n_experts < 1 || n_ff < 0 || n_in < 0 || m < 0 || top_k < 1 || activation < DQ4_ACT_RELU ||
        activation > DQ4_ACT_GELU_TANH)
        return DQ4_EINVAL;
    if (!sizes_fit(n_experts, n_ff, n_in, m, top_k))
        return DQ4_EUNSUPPORTED;
    if (m == 0 || n_in == 0)
        return DQ4_OK;
    if (!x || !y || !ids || !weights || bad_ld(ld_x, m, n_in) || bad_ld(ld_y, m, n_in) ||
        (residual && bad_ld(ld_residual, m, n_in)) ||
        (n_ff > 0 && (weight_missing(gate) || weight_missing(up) || weight_missing(down))) ||
        !down->scale_codebook || !down->codebook4)
        return DQ4_EINVAL;
    const Layout l = layout_of(n_experts, n_ff, n_in, m, top_k);
    if (workspace_bytes < l.all || bad_workspace(workspace, workspace_bytes))
        return DQ4_EINVAL;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    MoeArgs a{};
    a.w[0] = device_weight(*gate);
    a.w[1] = device_weight(*up);
    a.w[2] = device_weight(*down);
    a.log2_block = log2_block;
    a.log2_down = log2_down;
    a.n_experts = n_experts;
    a.top_k = top_k;
    a.n_ff = n_ff;
    a.n_in = n_in;
    a.m = m;
    a.act = activation;
    a.tf = tiles_per_pass(m, top_k, n_experts);
    a.x = static_cast<const uint16_t *>(x);
    a.ld_x = ld_x;
    a.ids = ids;
    a.weights = weights;
    a.vec_x = rows_aligned(x, ld_x, m, n_in);
    a.vec_y = rows_aligned(y, ld_y, m, 8) && (!residual || rows_aligned(residual, ld_residual, m, 8));
    a.max_tiles = static_cast<int32_t>(l.max_tiles);
    a.n_units = reinterpret_cast<int32_t *>(ws);
    a.units = reinterpret_cast<Pass *>(ws + l.units);
    a.token_of = reinterpret_cast<int32_t *>(ws + l.tokens);
    a.share_of = reinterpret_cast<float *>(ws + l.shares);
    a.x_frags = reinterpret_cast<uint16_t *>(ws + l.x);
    a.h_frags = reinterpret_cast<uint16_t *>(ws + l.h);
    a.residual = static_cast<const uint16_t *>(residual);
    a.ld_residual = ld_residual;
    a.y = static_cast<uint16_t *>(y);
    a.ld_y = ld_y;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int cus = current_compute_units();
    return dtype == DQ4_F16 ? run_moe<DQ4_F16>(a, cus, s) : run_moe<DQ4_BF16>(a, cus, s);
}

}  // extern "C"

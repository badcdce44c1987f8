// dq4_moe.hip -- a mixture-of-experts layer for a few tokens (include/dq4_moe.h):
// the router, and the chosen experts' gated feed-forward blocks over nested 4-bit
// weights.
//
// Few tokens choose few experts, and each chosen expert's matrices are read once for
// 16 of its tokens (32 where tiles_per_pass says two): the layer is bound by that and by
// the decode.  Two launches route (the logits, the
// choice), three multiply: a plan (which experts, which tokens each, and x in operand
// fragments; a single token's kernels plan for themselves), the gate and up products
// of every chosen expert, and the down products of all of them with the weighted sum
// over a token's experts.
//
// Measured on one MI355X (gate and up | down, us): one token, 8 of 64 experts of 1024
// x 2048, 26 MB of weight, 11.9 | 8.4, a wave has one chunk, and launch, plan, tables
// and the memory's latency are most of it; 16 tokens, all of 8 experts of 14336 x 4096,
// 727 MB, 145 | 76 (3.3 | 3.2 TB/s; vector instructions and lookups fill half of the
// time, the wait for the next chunk the rest); 64 tokens, 4 of 16 experts of 1000 x
// 2376, 60 MB, 25.6 | 19.4.
//
// The weight is decoded in operand registers as in dq4_linear_fused.hip's few-row
// kernels, through one lookup table of byte pairs in LDS, and multiplied on
// v_mfma_f32_16x16x32_{f16,bf16}: 16 weight rows by a tile of 16 tokens.  An
// expert's tokens are gathered into tiles, so that an expert costs its own tokens,
// not everybody's.
//
// Operand order of x and h: chunks of 512 k, [tile][chunk][16 steps][64 lanes][8],
// lane 16 g + c of step 4 j + s holding column c's k 512 chunk + 128 g + 32 j + 8
// s .. + 7: what a lane that decodes 16 packed bytes (32 k) four times needs.

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <initializer_list>
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
    double *logits;  // m x n_experts
    int32_t *ids;
    float *weights;
};

// Logits.  kExperts = 1: a workgroup for one token and expert, its waves share k.
// kExperts = 4: a wave for one token and four experts, so that x is read less often
// (with router and choice, from Python, BF16, us, one expert | four: 128 tokens, 64
// experts x 2048 17.0 | 13.4, 512 tokens 45 | 30, 2048 tokens 168 | 106; 16 tokens and 8
// experts x 4096 13.9 | 14.7).
// The sums run in 64 bits, since the choice between two experts hangs on the last
// place.  The products are exact: of FP16 values in FP32, of BF16 values, whose
// products leave FP32's range at both ends, in FP64 (2048 tokens, 64 experts x 2048:
// FP16 103, BF16 106).  (One workgroup per token for everything took 16.6 us for 64
// experts x 2048: the conversions to 64 bits on one CU.)
template <int OUT, int kExperts>
__global__ __launch_bounds__(256) void moe_logits_kernel(RouteArgs a)
{
    __shared__ double part[4];
    constexpr int kWaves = kExperts == 1 ? 4 : 1;  // that share an item
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int k = static_cast<int>(a.n_in), E = a.n_experts;
    const int groups = (E + kExperts - 1) / kExperts;
    const int64_t items = a.m * groups;
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * (4 / kWaves) + wave / kWaves; item < items;
         item += static_cast<int64_t>(gridDim.x) * (4 / kWaves)) {
        const int64_t t = static_cast<uint32_t>(item) / static_cast<uint32_t>(groups);
        const int e0 = static_cast<int>(item - t * groups) * kExperts;
        const uint16_t *x = a.x + t * a.ld_x;
        double sum[kExperts] = {};
#pragma unroll 4
        for (int c = (wave % kWaves * 64 + lane) * 8; c < k; c += kWaves * 512) {
            const int valid = k - c < 8 ? k - c : 8;
            float xv[8];
            load_values<OUT, 8>(x + c, a.vec, valid, xv);
#pragma unroll
            for (int q = 0; q < kExperts; ++q) {
                const int e = e0 + q < E ? e0 + q : E - 1;
                float r[8];
                load_values<OUT, 8>(a.router + static_cast<int64_t>(e) * k + c, a.vec, valid, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if constexpr (OUT == DQ4_F16)
                        sum[q] = sum[q] + static_cast<double>(xv[j] * r[j]);
                    else
                        sum[q] = sum[q] + static_cast<double>(xv[j]) * static_cast<double>(r[j]);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < kExperts; ++q) {
#pragma unroll
            for (int d = 32; d > 0; d /= 2)
                sum[q] = sum[q] + __shfl_xor(sum[q], d);
            if constexpr (kWaves == 4) {
                if (lane == 0)
                    part[wave] = sum[q];
                __syncthreads();
                sum[q] = part[0] + part[1] + part[2] + part[3];
                __syncthreads();
            }
            if (lane == 0 && wave % kWaves == 0 && e0 + q < E) {
                const float bias = a.bias ? a.bias[e0 + q] : 0.0f;
                // (a masked expert's sum may be an infinity or NaN: it is not looked at)
                a.logits[t * E + e0 + q] = bias == -__builtin_inff() ? static_cast<double>(bias)
                                                                     : sum[q] + static_cast<double>(bias);
            }
        }
    }
}

// A logit as a whole number in the same order: -infinity, NaN, the values upwards.
constexpr uint64_t kMasked = 0x000FFFFFFFFFFFFFull;

__device__ __forceinline__ uint64_t key_of(double logit)
{
    const uint64_t bits = __builtin_bit_cast(uint64_t, logit + 0.0);  // -0 is 0
    const uint64_t key = bits >> 63 ? ~bits : bits | 0x8000000000000000ull;
    return logit != logit ? kMasked + 1 : key;
}

// A token per workgroup, a thread per expert: an expert's rank is the number of
// experts before it.
__global__ __launch_bounds__(kMaxExperts) void moe_select_kernel(RouteArgs a)
{
    __shared__ __attribute__((aligned(16))) uint64_t keys[kMaxExperts];
    __shared__ double best[kMaxTopK];
    __shared__ float share[kMaxExperts];
    __shared__ int masked, any_nan;
    const int tid = threadIdx.x;
    const int E = a.n_experts, padded = (E + 63) & ~63;  // the workgroup's threads
    const double minus_infinity = -__builtin_inf();
    for (int64_t t = blockIdx.x; t < a.m; t += gridDim.x) {
        const double mine = tid < E ? a.logits[t * E + tid] : minus_infinity;
        const uint64_t key = tid < E ? key_of(mine) : 0;
        keys[tid] = key;
        if (tid == 0)
            masked = any_nan = 0;
        __syncthreads();
        const bool nan = mine != mine;
        int rank = 0;
#pragma unroll 16
        for (int e = 0; e < padded; ++e)
            rank += keys[e] >= (e < tid ? key : key + 1) ? 1 : 0;
        if (nan)
            any_nan = 1;
        if (key == kMasked)
            atomicAdd(&masked, 1);
        if (key > kMasked && rank < a.top_k) {
            a.ids[t * a.top_k + rank] = tid;
            best[rank] = mine;
        }
        __syncthreads();
        // as many places as there are experts left
        const int chosen = E - masked < a.top_k ? E - masked : a.top_k;
        const double top = chosen > 0 ? best[0] : 0.0;
        share[tid] = exp_f32(static_cast<float>(mine - top));
        __syncthreads();
        if (tid < a.top_k) {
            float total = 0.0f;
            if (a.renormalize) {
                for (int j = 0; j < chosen; ++j)
                    total = total + exp_f32(static_cast<float>(best[j] - top));
            } else {
#pragma unroll 8
                for (int e = 0; e < padded; ++e)
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
    int32_t expert, tile, tiles;  // the first of its tiles
    int32_t columns;              // of them all: 16 in each but the last
};

struct MoeArgs {
    Weight w[2];             // gate, up
    Weight down;
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
    int32_t *n_passes;
    Pass *passes;
    int32_t *token_of;       // [tile][16]: the column's token
    float *share_of;         // [tile][16]: its weight for the tile's expert
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
// order, with zeros where there is no k, and zeros for the k of h that the products
// leave out.  Columns without a token are not written and never read.
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
    const int count = __builtin_popcount(mask[tid][0]) + __builtin_popcount(mask[tid][1]);
    const int tiles = (count + 15) / 16;
    const int passes = (tiles + a.tf - 1) / a.tf;
    int n_tiles, n_passes;
    const int my_tile = list_position<512>(tiles, &n_tiles, sums);
    tile0[tid] = my_tile;
    const int my_pass = list_position<512>(passes, &n_passes, sums);
    // where a choice's token lies among its expert's
    const auto tile_column = [&](int e, int t) {
        const uint32_t below = (1u << (t & 31)) - 1;
        return tile0[e] * 16 + (t < 32 ? __builtin_popcount(mask[e][0] & below)
                                       : __builtin_popcount(mask[e][0]) + __builtin_popcount(mask[e][1] & below));
    };
    if (blockIdx.x == 0) {
        if (tid == 0)
            *a.n_passes = n_passes;
        for (int q = 0; q < passes; ++q) {
            const int left = tiles - q * a.tf, columns = count - q * a.tf * 16;
            a.passes[my_pass + q] = Pass{tid, my_tile + q * a.tf, left < a.tf ? left : a.tf,
                                         columns < a.tf * 16 ? columns : a.tf * 16};
        }
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
    const int chunks = chunks_of(a.n_in), h_chunks = chunks_of(a.n_ff);
    const int h_from = static_cast<int>((a.n_ff + 15) / 16 * 16);
    // pieces of a tile's x: one chunk each, the columns that have a token
    for (int item = blockIdx.x; item < n_tiles * chunks; item += gridDim.x) {
        const int tile = item / chunks, ch = item - tile * chunks;
        __syncthreads();  // the last item's tokens are read
        if (tid < 16)
            token[tid] = -1;
        __syncthreads();
        for (int p = tid; p < pairs; p += 512) {
            const int e = a.ids[p], t = p / a.top_k;
            if (e < 0 || e >= a.n_experts)
                continue;
            const int at = tile_column(e, t);
            if (at >> 4 == tile)
                token[at & 15] = t;
        }
        __syncthreads();
        uint16_t *to = a.x_frags + (static_cast<int64_t>(tile) * chunks + ch) * kTileChunk;
        for (int u = tid; u < 1024; u += 512) {
            const int lane = u & 63, step = u >> 6;
            const int t = token[lane & 15];
            if (t < 0)
                continue;
            const int k0 = ch * kSpan + 128 * (lane >> 4) + 8 * step;
            u32x4 q = {0, 0, 0, 0};
            if (k0 < a.n_in) {
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
        if (ch == 0 && h_chunks > 0) {
            uint16_t *to_h = a.h_frags + (static_cast<int64_t>(tile) * h_chunks + h_chunks - 1) * kTileChunk;
            for (int u = tid; u < 1024; u += 512) {
                const int k0 = (h_chunks - 1) * kSpan + 128 * ((u & 63) >> 4) + 8 * (u >> 6);
                if (k0 >= h_from)
                    *reinterpret_cast<u32x4 *>(to_h + u * 8) = u32x4{0, 0, 0, 0};
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

// One weight matrix and where a chunk of its rows begins.
struct Source {
    Weight w;
    int log2_block;
    int64_t n_elems;
    uint32_t n;  // row length
};

// (field by field: an array or a choice of structs would pass through memory)
__device__ __forceinline__ Weight either(const Weight &a, const Weight &b, int second)
{
    return Weight{second ? b.packed : a.packed,
                  second ? b.scale_codes : a.scale_codes,
                  second ? b.nested_absmax : a.nested_absmax,
                  second ? b.scale_codebook : a.scale_codebook,
                  second ? b.codebook4 : a.codebook4,
                  second ? b.offset : a.offset};
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_from(const void *p, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0,
                                             static_cast<int32_t>(bytes < 0x7FFFFFF0 ? bytes : 0x7FFFFFF0),
                                             kRawBufferWord3);
}

// The buffers of a row block, and the place of its first element in them.
struct Buffers {
    __amdgpu_buffer_rsrc_t packed, codes, absmax;
    uint32_t nibble0;      // of the first element in `packed`, which starts at a dword
    uint32_t phase;        // elements of the first block before it
    uint32_t group_phase;  // blocks of the first group before that block
};

__device__ __forceinline__ Buffers buffers_of(const Source &s, const RowBlock &b)
{
    const int64_t e0 = b.row0 * s.n, b0 = e0 >> s.log2_block;
    const int64_t blocks = (s.n_elems + (int64_t{1} << s.log2_block) - 1) >> s.log2_block;
    const uintptr_t at = reinterpret_cast<uintptr_t>(s.w.packed) + (e0 >> 1);
    const uint32_t skew = static_cast<uint32_t>(at & 3);
    Buffers q;
    // whole dwords, up to the one with the last byte
    q.packed = buffer_from(reinterpret_cast<const void *>(at - skew),
                           (((s.n_elems + 1) >> 1) - (e0 >> 1) + skew + 3) & ~int64_t{3});
    q.codes = buffer_from(s.w.scale_codes + b0, blocks - b0);
    q.absmax = buffer_from(s.w.nested_absmax + (b0 >> kNestedLog2),
                           (((blocks + 255) >> kNestedLog2) - (b0 >> kNestedLog2)) * 4);
    q.nibble0 = 2 * skew + (static_cast<uint32_t>(e0) & 1);
    q.phase = static_cast<uint32_t>(e0) & ((1u << s.log2_block) - 1);
    q.group_phase = static_cast<uint32_t>(b0) & 255;
    return q;
}

__device__ __forceinline__ void load_scale(const Buffers &q, uint32_t block, bool in, uint32_t *code, float *absmax)
{
    *code = __builtin_amdgcn_raw_buffer_load_b8(q.codes, in ? block : 0x80000000u, 0, 0);
    *absmax = __builtin_bit_cast(
        float, __builtin_amdgcn_raw_buffer_load_b32(
                   q.absmax, in ? ((q.group_phase + block) >> kNestedLog2) * 4 : 0x80000000u, 0, 0));
}

// Row lengths that are multiples of 32, packed codes at 4-byte boundaries.  A load
// takes 256 bytes of 4 rows, a quad of lanes on 64 of them; 4 such loads are
// transposed between the lanes of each quad; the scales, S blocks per 128 k, are
// looked up four lanes to a row and handed over.  S = 2: blocks of 64 k or more and
// row lengths that are multiples of 64; else S = 4.
template <int OUT, int S>
struct EvenRows {
    static constexpr bool kEven = true;
    u32x4 packed[4];
    uint32_t code[S];
    float absmax[S];
    float s[S];

    __device__ __forceinline__ void load_scales(const Source &w, const RowBlock &b, int c, int lane)
    {
        const Buffers q = buffers_of(w, b);
#pragma unroll
        for (int h = 0; h < S; ++h) {
            const uint32_t e = (lane >> 2) * w.n + c * kSpan + 128 * (lane & 3) + h * (128 / S);
            load_scale(q, (q.phase + e) >> w.log2_block, true, &code[h], &absmax[h]);
        }
    }

    __device__ __forceinline__ void load_packed(int i, const Source &w, const RowBlock &b, int c, int lane)
    {
        const Buffers q = buffers_of(w, b);
        const uint32_t k = c * kSpan + 32 * (((lane >> 4) << 2) | (lane & 3));
        const int row = 4 * ((lane >> 2) & 3) + i;
        packed[i] = __builtin_amdgcn_raw_buffer_load_b128(
            q.packed, k < w.n && row < b.rows ? ((row * w.n + k) >> 1) + (q.nibble0 >> 1) : 0x80000000u, 0, 0);
    }

    __device__ __forceinline__ void load(const Source &w, const RowBlock &b, int c, int lane)
    {
        load_scales(w, b, c, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            load_packed(i, w, b, c, lane);
    }

    __device__ __forceinline__ void prepare(const float *scb, float offset, int lane)
    {
        const int g = lane >> 4, r = lane & 15;
#pragma unroll
        for (int h = 0; h < S; ++h) {
            const float q = block_scale(scb[code[h]], absmax[h], offset);
            // lane 16 g + r multiplies quarter g of row r
            s[h] = __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute((4 * r + g) * 4,
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
    }

    // A piece beyond the row or the last row: its load gave zeros; it reads the
    // table's row of zeros, times 0.
    static __device__ __forceinline__ bool beyond(const Source &w, const RowBlock &b, int c, int j, int lane)
    {
        return c * kSpan + 128 * (lane >> 4) + 32 * j >= static_cast<int>(w.n) || (lane & 15) >= b.rows;
    }

    __device__ __forceinline__ Pairs look(const uint8_t *table, uint32_t lane_byte, int step) const
    {
        return lookup_dword(packed[step / 4][step % 4], table, lane_byte);
    }

    __device__ __forceinline__ u32x4 operand(const Pairs &p, bool beyond, int step) const
    {
        return scaled_dword<OUT>(p, beyond ? 0.0f : s[step / 4 * S / 4]);
    }
};

// Any row length and alignment: a lane takes its own row's 32 k at a time.  Blocks
// are at least 32 elements long, so a piece meets at most two.
// kEights: row lengths that are multiples of 8, packed codes at 4-byte boundaries;
// a step's 8 k are one dword, of one block, and all in the row or none.  Else five
// dwords are shifted to their first nibble and each element picks its scale
// (16 experts of 1000 x 2376, 64 tokens, gate and up: 26 us, against 40 without kEights).
template <int OUT, bool kEights>
struct AnyRows {
    static constexpr bool kEven = false;
    u32x4 lo;
    uint32_t hi;
    uint32_t code[2];
    float absmax[2];
    uint32_t shift;
    int meet, valid;
    float s[2];

    __device__ __forceinline__ void load(const Source &w, const RowBlock &b, int c, int j, int lane)
    {
        const Buffers q = buffers_of(w, b);
        const int r = lane & 15;
        const uint32_t k = c * kSpan + 128 * (lane >> 4) + 32 * j;
        const int left = r < b.rows ? static_cast<int>(w.n) - static_cast<int>(k) : 0;
        valid = left < 0 ? 0 : left > 32 ? 32 : left;
        const uint32_t e = r * w.n + k, nibble = q.nibble0 + e;
        shift = kEights ? 0 : 4 * (nibble & 7);
        const uint32_t word = valid > 0 ? (nibble >> 3) * 4 : 0x80000000u;
        lo = __builtin_amdgcn_raw_buffer_load_b128(q.packed, word, 0, 0);
        hi = kEights ? 0 : __builtin_amdgcn_raw_buffer_load_b32(q.packed, word + 16, 0, 0);
        const uint32_t block = (q.phase + e) >> w.log2_block;
        meet = static_cast<int>(((block + 1) << w.log2_block) - q.phase - e);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            load_scale(q, block + h, valid > 0, &code[h], &absmax[h]);
    }

    __device__ __forceinline__ void prepare(const float *scb, float offset)
    {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            s[h] = block_scale(scb[code[h]], absmax[h], offset);
    }

    __device__ __forceinline__ Pairs look(const uint8_t *table, uint32_t lane_byte, int d) const
    {
        return lookup_dword(kEights ? lo[d] : __builtin_amdgcn_alignbit(d < 3 ? lo[d + 1] : hi, lo[d], shift), table,
                            lane_byte);
    }

    __device__ __forceinline__ u32x4 operand(const Pairs &p, int d) const
    {
        u32x4 q;
        if constexpr (kEights) {
            q = scaled_dword<OUT>(p, 8 * d < meet ? s[0] : s[1]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q[i] = 8 * d < valid ? q[i] : 0;
            return q;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = 8 * d + 2 * i + h;
                const float z = p.v[i][h] * (at < meet ? s[0] : s[1]);
                v[h] = at < valid ? z : 0.0f;
            }
            q[i] = Half<OUT>::pack2(v[0], v[1]);
        }
        return q;
    }
};

// The other operand: fragments of TF tiles, in operand order; or (kOne) the one
// token's row, in the lanes of column 0.  Columns without a token lie past the buffer:
// their lanes get zeros and move nothing (with 16 columns always, an expert that 4 of
// 16 tokens chose moved 16 KiB of h for 4 KiB of weight).
template <int TF, bool kOne>
struct Columns {
    const uint16_t *at;
    uint32_t bytes;
    uint32_t offset[TF];

    __device__ __forceinline__ u32x4 load(int t, int step) const
    {
        return __builtin_amdgcn_raw_buffer_load_b128(buffer_from(at, bytes), offset[t] + (kOne ? 16 : 1024) * step, 0,
                                                     0);
    }
};

// Chunk c of a pass over tiles of `chunks` chunks.
template <int TF>
__device__ __forceinline__ Columns<TF, false> tile_columns(const uint16_t *frags, const Pass &p, int chunks, int c,
                                                           int lane)
{
    Columns<TF, false> x;
    x.at = frags + (static_cast<int64_t>(p.tile) * chunks + c) * kTileChunk;
    x.bytes = 0x7FFFFFF0;
#pragma unroll
    for (int t = 0; t < TF; ++t)
        x.offset[t] = 16 * t + (lane & 15) < p.columns
                          ? static_cast<uint32_t>(t) * chunks * (kTileChunk * 2) + lane * 16
                          : 0x80000000u;
    return x;
}

// Chunk c of one row of k values; zeros behind it.
__device__ __forceinline__ Columns<1, true> row_columns(const uint16_t *row, int64_t k, int c, int lane)
{
    Columns<1, true> x;
    x.at = row;
    x.bytes = static_cast<uint32_t>(k * 2);
    x.offset[0] = (lane & 15) == 0 ? (c * kSpan + 128 * (lane >> 4)) * 2 : 0x80000000u;
    return x;
}

// Steps that the other operand is loaded ahead; what the registers hold.
template <int W>
constexpr int kAheadOf = W == 2 ? 2 : 4;

// What a wave holds: of a row block an even one's chunk, or two pieces in turn; and
// the other operand's next steps.
template <class Rows, int W, int TF>
struct Held {
    Rows r[W][Rows::kEven ? 1 : 2];
    static constexpr int kAhead = kAheadOf<W>;
    u32x4 x[kAhead][TF];

    template <bool kOne>
    __device__ __forceinline__ void load_first(const Source (&src)[W], const RowBlock &rows, int c,
                                               const Columns<TF, kOne> &columns, int lane)
    {
#pragma unroll
        for (int f = 0; f < W; ++f) {
            if constexpr (Rows::kEven)
                r[f][0].load(src[f], rows, c, lane);
            else
                r[f][0].load(src[f], rows, c, 0, lane);
        }
#pragma unroll
        for (int st = 0; st < kAhead; ++st)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                x[st][t] = columns.load(t, st);
    }
};

// Where the wave's next chunk lies (the same again after the last one: unused).
template <int TF, bool kOne>
struct Place {
    RowBlock rows;
    int c;
    Columns<TF, kOne> x;
};

// acc[f][t] += 16 rows of each of W weights x a chunk of 512 k x TF tiles.  Lookups
// run one weight's step ahead (weight f's table lies f * 8 bytes behind the first's).
// Loads return in the order of their issue: the next chunk's weight, which comes from
// memory, goes out behind this chunk's last load from cache.
template <int OUT, class Rows, int W, int TF, bool kOne>
__device__ __forceinline__ void multiply_chunk(Held<Rows, W, TF> &held, const Source (&src)[W],
                                               const Place<TF, kOne> &at, const Place<TF, kOne> &next,
                                               const float *scb, const uint8_t *table, uint32_t lane_byte,
                                               uint32_t zero_byte, f32x4 (&acc)[W][TF], int lane)
{
    constexpr int kAhead = kAheadOf<W>;
    Rows ahead[W];
    if constexpr (Rows::kEven)
#pragma unroll
        for (int f = 0; f < W; ++f)
            held.r[f][0].prepare(scb + 256 * f, src[f].w.offset, lane);
    Pairs now{}, then{};
#pragma unroll
    for (int st = 0; st < 16; ++st) {
        const int j = st / 4, d = st % 4;
        if constexpr (!Rows::kEven)
            if (d == 0)
#pragma unroll
                for (int f = 0; f < W; ++f) {
                    held.r[f][j & 1].prepare(scb + 256 * f, src[f].w.offset);
                    if (j < 3)
                        held.r[f][(j + 1) & 1].load(src[f], at.rows, at.c, j + 1, lane);
                    else
                        held.r[f][0].load(src[f], next.rows, next.c, 0, lane);
                }
#pragma unroll
        for (int f = 0; f < W; ++f) {
            const int nf = f + 1 < W ? f + 1 : 0, ns = f + 1 < W ? st : st + 1;
            u32x4 wf;
            if constexpr (Rows::kEven) {
                const bool beyond = Rows::beyond(src[f], at.rows, at.c, j, lane);
                if (st == 0 && f == 0)
                    now = held.r[0][0].look(table, beyond ? zero_byte : lane_byte, 0);
                if (ns < 16)
                    then = held.r[nf][0].look(
                        table + nf * 8, Rows::beyond(src[nf], at.rows, at.c, ns / 4, lane) ? zero_byte : lane_byte, ns);
                keep_order();
                wf = held.r[f][0].operand(now, beyond, st);
            } else {
                if (d == 0 && f == 0)
                    now = held.r[0][j & 1].look(table, lane_byte, 0);
                if (ns / 4 == j)
                    then = held.r[nf][j & 1].look(table + nf * 8, lane_byte, ns % 4);
                keep_order();
                wf = held.r[f][j & 1].operand(now, d);
            }
#pragma unroll
            for (int t = 0; t < TF; ++t)
                acc[f][t] = Half<OUT>::mfma(wf, held.x[st % kAhead][t], acc[f][t]);
            now = then;
        }
        if constexpr (Rows::kEven)
            if (st == 16 - kAhead)
#pragma unroll
                for (int f = 0; f < W; ++f)
                    ahead[f].load(src[f], next.rows, next.c, lane);
#pragma unroll
        for (int t = 0; t < TF; ++t)
            held.x[st % kAhead][t] =
                st + kAhead < 16 ? at.x.load(t, st + kAhead) : next.x.load(t, st + kAhead - 16);
    }
    if constexpr (Rows::kEven)
#pragma unroll
        for (int f = 0; f < W; ++f)
            held.r[f][0] = ahead[f];
}

// A single token's plan: its valid experts, each once, in the order of its row.
struct OnePlan {
    int n;
    int expert[kMaxTopK];
    float share[kMaxTopK];
};

__device__ __forceinline__ void plan_one(const MoeArgs &a, OnePlan &p)
{
    const int lane = threadIdx.x;
    if (lane >= 64)
        return;
    const bool in = lane < a.top_k;
    const int e = in ? a.ids[lane] : -1;
    const float w = in ? a.weights[lane] : 0.0f;
    bool first = e >= 0 && e < a.n_experts;
    float share = w;
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
        const int other = __shfl(e, j);
        const float more = __shfl(w, j);
        first = first && !(j < lane && other == e);
        share = j > lane && other == e ? share + more : share;
    }
    const uint64_t mask = __ballot(first);
    if (first) {
        const int at = __builtin_popcountll(mask & ((uint64_t{1} << lane) - 1));
        p.expert[at] = e;
        p.share[at] = share;
    }
    if (lane == 0)
        p.n = __builtin_popcountll(mask);
}

// The tables in two parts.  A workgroup's first loads of weight go out between them:
// behind those, what waits for the codebooks would wait for the weight too (one token,
// 8 of 64 experts of 1024 x 2048: 7.5 of the gate and up kernel's 14 us).
template <int kWeights, int kTables>
__device__ __forceinline__ void store_codebooks(const Codebooks &c, uint8_t *table, float (&scb)[kWeights][256],
                                                float (&cb4)[kWeights][16])
{
    const int tid = threadIdx.x, threads = blockDim.x;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int i = tid + q * threads;
        if (i < kWeights * 256)
            scb[i >> 8][i & 255] = c.scb[q];
    }
    if (tid < kWeights * 16)
        cb4[tid >> 4][tid & 15] = c.cb4;
    if (tid < 64)
        *reinterpret_cast<uint32_t *>(&table[kTables * kPairTableBytes + tid * 4]) = 0;
}

// A thread writes two neighbours of a pair's 32 places, one of each weight where two
// share a table; its first value is always the same.
template <int THREADS, int kWeights, int kTables>
__device__ __forceinline__ void fill_pairs(uint8_t *table, const float (&cb4)[kWeights][16])
{
    static_assert(THREADS % 256 == 0 && 4096 % THREADS == 0, "a thread keeps its first value");
    const int tid = threadIdx.x;
    constexpr bool kShared = kWeights == 2 && kTables == 1;
    float first[kWeights];
#pragma unroll
    for (int w = 0; w < kWeights; ++w)
        first[w] = cb4[w][(tid >> 4) & 15];
#pragma unroll
    for (int q = 0; q < kTables * 4096 / THREADS; ++q) {
        const int which = q * THREADS / 4096, second = (tid >> 8) + q * THREADS % 4096 / 256;
        *reinterpret_cast<f32x4 *>(&table[(tid + q * THREADS) * 16]) =
            f32x4{first[which], cb4[which][second], first[kShared ? 1 : which], cb4[kShared ? 1 : which][second]};
    }
    lds_barrier();
}

// ---------------------------------------------------------------------------
// gate and up
// ---------------------------------------------------------------------------
// An item is a pass's row block: 16 rows of the expert's gate and the same of its up
// matrix.  `wk` waves for each of both take its chunks in turn, and a workgroup takes
// as many items at a time as it has such groups of waves; a group's sums meet in LDS
// in a fixed order, and h goes out in the down product's operand order.  The next
// chunk's weight, also that of the next item, is in flight while one is multiplied.
// h is rounded to T, the width of the matrix instruction's operands in the down product
// (kept in two parts, it would take twice the instructions and the reads of h).  This
// rounding and y's own are as large, so y's error is up to sqrt 2 times that with FP32 h:
// against 64 bits (norm) 1.8e-3 for 1.65e-3 in BF16 (one token, 8 of 64 experts of 1024 x
// 2048), 2.9e-4 for 2.1e-4 in FP16 (16 tokens, 8 of 14336 x 4096).  An FP16 h beyond
// 65504 is an infinity.
// (A wave for each matrix: 16 waves hold one matrix's chunk and the next, and with
// four waves a SIMD lookups, vector instructions and loads overlap; a wave for both
// left room for 8 waves.)
template <int OUT, class Rows, int W, int TF, bool kOne, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void moe_gate_up_kernel(MoeArgs a, int32_t wk_waves)
{
    constexpr int kTables = 3 - W;  // W == 2: one table of both weights
    __shared__ __attribute__((aligned(1024))) uint8_t table[kTables * kPairTableBytes + 256];
    __shared__ float scb[2][256], cb4[2][16];
    __shared__ __attribute__((aligned(16))) f32x4 partial[WAVES][W * TF][64];
    __shared__ OnePlan one;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr int kShare = 3 - W;  // waves that share a chunk
    const int WK = wk_waves, WR = WAVES / (kShare * WK);
    const int which = W == 2 ? 0 : wave & 1, wk = wave / kShare % WK, wr = wave / (kShare * WK);
    const int n_ff = static_cast<int>(a.n_ff);
    const int chunks = chunks_of(a.n_in), h_chunks = chunks_of(a.n_ff);
    const int row_blocks = (n_ff + 15) >> 4;
    const int64_t n_elems = static_cast<int64_t>(a.n_experts) * a.n_ff * a.n_in;
    Source src[W];
#pragma unroll
    for (int f = 0; f < W; ++f)
        src[f] = Source{either(a.w[0], a.w[1], which + f), a.log2_block, n_elems, static_cast<uint32_t>(a.n_in)};

    const Codebooks codebooks = fetch_codebooks<2>(a.w);
    int n_passes;
    if constexpr (kOne)
        plan_one(a, one);
    else
        n_passes = *a.n_passes;
    store_codebooks<2, kTables>(codebooks, table, scb, cb4);
    __syncthreads();
    if constexpr (kOne)
        n_passes = one.n;
    const int items = n_passes * row_blocks;
    const int step = gridDim.x * WR;
    int next_item = blockIdx.x * WR + wr;
    Pass pass{}, next_pass{};
    Place<TF, kOne> at{}, next{};
    const auto columns = [&](const Pass &p, int c) {
        if constexpr (kOne)
            return row_columns(a.x, a.n_in, c, lane);
        else
            return tile_columns<TF>(a.x_frags, p, chunks, c, lane);
    };
    const auto enter = [&](int item) {
        const int u = item / row_blocks;
        if constexpr (kOne)
            next_pass = Pass{one.expert[u], u, 1, 1};
        else
            next_pass = a.passes[u];
        const int row = (item - u * row_blocks) * 16;
        next.rows = RowBlock{static_cast<int64_t>(next_pass.expert) * n_ff + row, n_ff - row < 16 ? n_ff - row : 16};
        next.c = wk;
        next.x = columns(next_pass, wk);
    };
    Held<Rows, W, TF> held;
    // (without a branch around the loads: what waits for some where branches meet waits
    // for them all; no rows, no columns: nothing is moved)
    next.x = columns(Pass{0, 0, 0, 0}, 0);
    if (next_item < items)
        enter(next_item);
    held.load_first(src, next.rows, next.c, next.x, lane);
    fill_pairs<64 * WAVES, 2, kTables>(table, cb4);
    const uint32_t copy = W == 2 ? (lane & 15) * 16 : (lane & 31) * 8;
    const uint32_t lane_byte = copy + which * kPairTableBytes, zero_byte = copy % 248 + kTables * kPairTableBytes;

    for (int item0 = blockIdx.x * WR; item0 < items; item0 += step) {
        const int item = item0 + wr;
        pass = next_pass;
        f32x4 acc[W][TF];
#pragma unroll
        for (int f = 0; f < W; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                acc[f][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (item < items)
            for (int c = wk; c < chunks; c += WK) {  // wk < chunks
                at = next;
                if (c + WK < chunks) {
                    next.c = c + WK;
                    next.x = columns(pass, c + WK);
                } else {
                    next_item += step;
                    if (next_item < items)
                        enter(next_item);
                }
                multiply_chunk<OUT, Rows, W, TF, kOne>(held, src, at, next, scb[which], table, lane_byte, zero_byte,
                                                       acc, lane);
            }
        lds_barrier();  // the last items' sums are read
        if (item < items)
#pragma unroll
            for (int f = 0; f < W; ++f)
#pragma unroll
                for (int t = 0; t < TF; ++t)
                    partial[wave][f * TF + t][lane] = acc[f][t];
        lds_barrier();
        if (item < items) {  // a wave of the group finishes a tile
            for (int t = wave - wr * (kShare * WK); t < pass.tiles; t += kShare * WK) {
                f32x4 gate = {0.0f, 0.0f, 0.0f, 0.0f}, up = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int q = wr * (kShare * WK); q < (wr + 1) * (kShare * WK); q += kShare) {
                    gate = gate + partial[q][t][lane];
                    up = up + (W == 2 ? partial[q][(W - 1) * TF + t][lane] : partial[q + kShare - 1][t][lane]);
                }
                // the lane's four neighbouring k of h, column lane % 16
                const int k = (item - item / row_blocks * row_blocks) * 16 + 4 * (lane >> 4);
                float h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    h[i] = k + i < n_ff ? act_f32(a.act, gate[i]) * up[i] : 0.0f;
                const u32x2 out = {Half<OUT>::pack2(h[0], h[1]), Half<OUT>::pack2(h[2], h[3])};
                if constexpr (kOne) {  // a row of its own
                    if ((lane & 15) == 0)
                        *reinterpret_cast<u32x2 *>(a.h_frags + static_cast<int64_t>(pass.tile) * h_chunks * kSpan + k) = out;
                } else if (16 * t + (lane & 15) < pass.columns) {
                    const int ch = k / kSpan, in = k % kSpan;
                    uint16_t *to = a.h_frags + (static_cast<int64_t>(pass.tile + t) * h_chunks + ch) * kTileChunk +
                                   (((in & 127) >> 3) * 64 + (in >> 7) * 16 + (lane & 15)) * 8 + (in & 7);
                    *reinterpret_cast<u32x2 *>(to) = out;
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// down, and the sum over a token's experts
// ---------------------------------------------------------------------------
// A workgroup takes 16 output columns and walks all passes: its waves take the
// (pass, chunk) pairs in turn, multiply a pass's sums by its tokens' weights and add
// them to their own sums for every token, in a fixed order; the waves' sums meet at
// the end.  So a token's experts are added up without a pass of their own.
template <int OUT, class Rows, int TF, bool kOne, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void moe_down_kernel(MoeArgs a)
{
    constexpr int kTokens = kOne ? 1 : kMaxTokens;
    __shared__ __attribute__((aligned(1024))) uint8_t table[kPairTableBytes + 256];
    __shared__ float scb[1][256], cb4[1][16];
    __shared__ __attribute__((aligned(16))) float sums[WAVES][kTokens][16];
    __shared__ OnePlan one;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n_out = static_cast<int>(a.n_in);
    const int chunks = chunks_of(a.n_ff);
    const int64_t n_elems = static_cast<int64_t>(a.n_experts) * a.n_ff * a.n_in;
    const Weight both[2] = {a.down, a.down};
    const Source src[1] = {{a.down, a.log2_down, n_elems, static_cast<uint32_t>(a.n_ff)}};

    const Codebooks codebooks = fetch_codebooks<1>(both);
    int n_passes;
    if constexpr (kOne)
        plan_one(a, one);
    else
        n_passes = *a.n_passes;
    store_codebooks<1, 1>(codebooks, table, scb, cb4);
    __syncthreads();
    if constexpr (kOne)
        n_passes = one.n;
    const int items = n_passes * chunks;
    const int row_blocks = (n_out + 15) >> 4;
    Pass next_pass{};
    Place<TF, kOne> at{}, next{};
    const auto columns = [&](const Pass &p, int c) {
        if constexpr (kOne)  // (up to the last k that the products wrote)
            return row_columns(a.h_frags + static_cast<int64_t>(p.tile) * chunks * kSpan, (a.n_ff + 15) / 16 * 16, c, lane);
        else
            return tile_columns<TF>(a.h_frags, p, chunks, c, lane);
    };
    const auto enter = [&](int row_block, int item) {
        const int u = item / chunks;
        if constexpr (kOne)
            next_pass = Pass{one.expert[u], u, 1, 1};
        else
            next_pass = a.passes[u];
        next.c = item - u * chunks;
        const int row = row_block * 16;
        next.rows = RowBlock{static_cast<int64_t>(next_pass.expert) * n_out + row,
                             n_out - row < 16 ? n_out - row : 16};
        next.x = columns(next_pass, next.c);
    };
    Held<Rows, 1, TF> held;
    next.x = columns(Pass{0, 0, 0, 0}, 0);
    if (wave < items)
        enter(blockIdx.x, wave);
    held.load_first(src, next.rows, next.c, next.x, lane);
    fill_pairs<64 * WAVES, 1, 1>(table, cb4);
    const uint32_t lane_byte = (lane & 31) * 8, zero_byte = lane_byte + kPairTableBytes;

    for (int row_block = blockIdx.x; row_block < row_blocks; row_block += gridDim.x) {
        for (int i = lane; i < (kOne ? 1 : static_cast<int>(a.m)) * 4; i += 64)
            reinterpret_cast<f32x4 *>(&sums[wave][0][0])[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        f32x4 acc[1][TF];
#pragma unroll
        for (int t = 0; t < TF; ++t)
            acc[0][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int item = wave; item < items; item += WAVES) {
            const Pass pass = next_pass;
            at = next;
            const bool last = item + WAVES >= items;
            if (!last)
                enter(row_block, item + WAVES);
            else if (row_block + static_cast<int>(gridDim.x) < row_blocks)
                enter(row_block + gridDim.x, wave);
            multiply_chunk<OUT, Rows, 1, TF, kOne>(held, src, at, next, scb[0], table, lane_byte, zero_byte, acc, lane);
            // the wave's next pair is of another pass: this one's sums to its tokens
            if (last || next_pass.tile != pass.tile) {
#pragma unroll
                for (int t = 0; t < TF; ++t) {
                    if (16 * t + (lane & 15) < pass.columns) {
                        const int place = (pass.tile + t) * 16 + (lane & 15);
                        const int token = kOne ? 0 : a.token_of[place];
                        const float w = kOne ? one.share[pass.tile] : a.share_of[place];
                        f32x4 *to = reinterpret_cast<f32x4 *>(&sums[wave][token][4 * (lane >> 4)]);
                        f32x4 v = *to;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i] = v[i] + w * acc[0][t][i];
                        *to = v;
                    }
                    acc[0][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                }
            }
        }
        lds_barrier();
        if (tid < a.m * 4) {
            const int token = tid >> 2, i0 = 4 * (tid & 3);
            f32x4 z = *reinterpret_cast<const f32x4 *>(&sums[0][token][i0]);
#pragma unroll
            for (int q = 1; q < WAVES; ++q)
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
// more passes.  (The whole call, us, with one | two: 64 tokens, 8 of 64 experts of 1024
// x 2048, 8 tokens each, 94 | 121; 40 and 64 tokens, 4 of 16 experts of 1000 x 2376, 10
// and 16 tokens each, 50.7 | 48.6 and 69 | 50.)
int tiles_per_pass(int64_t m, int64_t top_k, int64_t n_experts)
{
    return m <= 16 || m * top_k <= 8 * n_experts ? 1 : 2;
}

// What the workspace holds, in this order.
struct Layout {
    int64_t max_tiles;  // at most this many tiles, and passes
    int64_t passes, tokens, shares, x, h, all;
};

Layout layout_of(int64_t n_experts, int64_t n_ff, int64_t n_in, int64_t m, int64_t top_k)
{
    Layout l{};
    const int64_t pairs = m * top_k;
    // an expert's last tile may hold one token alone
    l.max_tiles = (pairs < n_experts ? pairs : n_experts) + pairs / 16;
    l.passes = 256;
    l.tokens = l.passes + align256(l.max_tiles * static_cast<int64_t>(sizeof(Pass)));
    l.shares = l.tokens + align256(l.max_tiles * 64);
    l.x = l.shares + align256(l.max_tiles * 64);
    l.h = l.x + l.max_tiles * ceil_div(n_in, kSpan) * kTileChunk * 2;
    l.all = l.h + l.max_tiles * ceil_div(n_ff, kSpan) * kTileChunk * 2;
    return l;
}

bool sizes_fit(int64_t n_experts, int64_t n_ff, int64_t n_in, int64_t m, int64_t top_k)
{
    return n_experts <= kMaxExperts && top_k <= kMaxTopK && m <= kMaxTokens && n_ff <= kMaxWidth &&
           n_in <= kMaxWidth && n_experts * n_ff * n_in <= kMaxWeight;
}

// A single token's kernels read x and h as they lie, and plan for themselves.
bool one_token(const MoeArgs &a)
{
    return a.m == 1 && a.vec_x;
}

// One token, up to a tile a pass, more.
template <int OUT, class Rows>
struct Kernels {
    // (Two tiles' sums and operands do not leave EvenRows the registers for 16 waves: 9
    // and 11 spill in gate and up, 2 and 5 in down.  AnyRows would fit and has the same
    // number.)
    static constexpr int kWaves = 16, kWavesOfTwo = 8;

    static dq4_status_t gate_up(const MoeArgs &a, int cus, hipStream_t s)
    {
        const void *kernel = one_token(a)
                                 ? reinterpret_cast<const void *>(&moe_gate_up_kernel<OUT, Rows, 1, 1, true, kWaves>)
                             : a.tf == 1
                                 ? reinterpret_cast<const void *>(&moe_gate_up_kernel<OUT, Rows, 2, 1, false, kWaves>)
                                 : reinterpret_cast<const void *>(&moe_gate_up_kernel<OUT, Rows, 2, 2, false, kWavesOfTwo>);
        const int waves = a.tf == 1 ? kWaves : kWavesOfTwo;
        const int share = one_token(a) ? 2 : 1;  // waves of a chunk
        // Waves along k for each matrix, no more than chunks: what leaves a wave the
        // fewest chunks if the tokens spread over the experts, the fewer waves of two
        // (the whole call, us, with 1, 2, 4, 8: 16 tokens, 8 of 64 experts of 1024 x
        // 2048 80, 83, 85; 64 tokens, 2 of 8 experts of 2048 x 4096 61, 48, 49, 51; 64
        // tokens, 4 of 16 experts of 1000 x 2376 61, 50, 55).
        const int64_t chunks = ceil_div(a.n_in, kSpan), pairs = a.m * a.top_k;
        const int64_t items = (pairs < a.n_experts ? pairs : a.n_experts) * ceil_div(a.n_ff, 16);
        int32_t wk = 0;
        int64_t least = 0;
        for (int w = waves / share; w > 0; w /= 2) {
            const int64_t each = ceil_div(items, static_cast<int64_t>(cus) * (waves / share / w)) * ceil_div(chunks, w);
            if (w <= chunks && (wk == 0 || each <= least)) {
                wk = w;
                least = each;
            }
        }
        MoeArgs args = a;
        void *params[] = {&args, &wk};
        const int64_t most = ceil_div(a.max_tiles * ceil_div(a.n_ff, 16), waves / (share * wk));
        return launch(kernel, most < cus ? most : cus, 1, 64 * waves, params, s);
    }

    static dq4_status_t down(const MoeArgs &a, int cus, hipStream_t s)
    {
        const void *kernel = one_token(a) ? reinterpret_cast<const void *>(&moe_down_kernel<OUT, Rows, 1, true, kWaves>)
                             : a.tf == 1
                                 ? reinterpret_cast<const void *>(&moe_down_kernel<OUT, Rows, 1, false, kWaves>)
                                 : reinterpret_cast<const void *>(&moe_down_kernel<OUT, Rows, 2, false, kWavesOfTwo>);
        MoeArgs args = a;
        void *params[] = {&args};
        const int64_t row_blocks = ceil_div(a.n_in, 16);
        return launch(kernel, row_blocks < cus ? row_blocks : cus, 1, 64 * (a.tf == 1 ? kWaves : kWavesOfTwo), params, s);
    }
};

template <int OUT>
dq4_status_t run_moe(MoeArgs a, int cus, hipStream_t s)
{
    dq4_status_t st;
    if (!one_token(a)) {  // (a single token's kernels plan for themselves)
        void *params[] = {&a};
        const int64_t pieces = a.max_tiles * ceil_div(a.n_in, kSpan);
        st = launch(reinterpret_cast<const void *>(&moe_plan_zero_fill), pieces < cus ? pieces : cus, 1, 512, params, s);
        if (st != DQ4_OK)
            return st;
    }
    // which rows a row length and the packed codes' addresses allow
    const auto rows_of = [](int64_t n, int log2_block, std::initializer_list<const void *> packed) {
        bool aligned = true;
        for (const void *p : packed)
            aligned = aligned && reinterpret_cast<uintptr_t>(p) % 4 == 0;
        return !aligned || n % 8 ? 0 : n % 32 ? 1 : n % 64 || log2_block < 6 ? 2 : 3;
    };
    if (a.n_ff > 0) {
        const int kind = rows_of(a.n_in, a.log2_block, {a.w[0].packed, a.w[1].packed});
        st = kind == 0   ? Kernels<OUT, AnyRows<OUT, false>>::gate_up(a, cus, s)
             : kind == 1 ? Kernels<OUT, AnyRows<OUT, true>>::gate_up(a, cus, s)
             : kind == 2 ? Kernels<OUT, EvenRows<OUT, 4>>::gate_up(a, cus, s)
                         : Kernels<OUT, EvenRows<OUT, 2>>::gate_up(a, cus, s);
        if (st != DQ4_OK)
            return st;
    }
    const int kind = rows_of(a.n_ff, a.log2_down, {a.down.packed});
    return kind == 0   ? Kernels<OUT, AnyRows<OUT, false>>::down(a, cus, s)
           : kind == 1 ? Kernels<OUT, AnyRows<OUT, true>>::down(a, cus, s)
           : kind == 2 ? Kernels<OUT, EvenRows<OUT, 4>>::down(a, cus, s)
                       : Kernels<OUT, EvenRows<OUT, 2>>::down(a, cus, s);
}

}  // namespace
}  // namespace dq4

using namespace dq4;

extern "C" {

int64_t dq4_moe_route_workspace_bytes(int64_t m, int32_t n_experts)
{
    if (m <= 0 || n_experts <= 0 || m > kMaxRows || n_experts > kMaxExperts)
        return 0;
    return align256(m * n_experts * 8);
}

dq4_status_t dq4_moe_route(const void *x, int64_t m, int64_t n_in, int64_t ld_x, int32_t dtype,
                           const void *router, const float *bias, int32_t n_experts, int32_t top_k,
                           int32_t renormalize, int32_t *ids, float *weights, void *workspace,
                           int64_t workspace_bytes, void *stream)
{
    if (m < 0 || n_in < 0 || n_experts < 0 || (dtype != DQ4_F16 && dtype != DQ4_BF16) || top_k < 1 ||
        top_k > n_experts)
        return DQ4_EINVAL;
    if (n_experts > kMaxExperts || top_k > kMaxTopK || m > kMaxRows || n_in > kMaxWidth)
        return DQ4_EUNSUPPORTED;
    if (m == 0)
        return DQ4_OK;
    if (!ids || !weights || (n_in > 0 && (!x || !router)) || bad_ld(ld_x, m, n_in) ||
        workspace_bytes < dq4_moe_route_workspace_bytes(m, n_experts) || bad_workspace(workspace, workspace_bytes))
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
    a.logits = static_cast<double *>(workspace);
    a.ids = ids;
    a.weights = weights;
    void *params[] = {&a};
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t cus = current_compute_units();
    const bool four = m * n_experts > cus * 16;
    const int64_t groups = four ? ceil_div(m * ceil_div(n_experts, 4), 4) : m * n_experts;
    const void *kernel = dtype == DQ4_F16 ? (four ? reinterpret_cast<const void *>(&moe_logits_kernel<DQ4_F16, 4>)
                                                  : reinterpret_cast<const void *>(&moe_logits_kernel<DQ4_F16, 1>))
                                          : (four ? reinterpret_cast<const void *>(&moe_logits_kernel<DQ4_BF16, 4>)
                                                  : reinterpret_cast<const void *>(&moe_logits_kernel<DQ4_BF16, 1>));
    const dq4_status_t st = launch(kernel, groups < cus * 8 ? groups : cus * 8, 1, 256, params, s);
    if (st != DQ4_OK)
        return st;
    return launch(reinterpret_cast<const void *>(&moe_select_kernel), m < cus * 8 ? m : cus * 8, 1,
                  static_cast<int>(ceil_div(n_experts, 64)) * 64, params, s);
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
    a.down = device_weight(*down);
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
    a.n_passes = reinterpret_cast<int32_t *>(ws);
    a.passes = reinterpret_cast<Pass *>(ws + l.passes);
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

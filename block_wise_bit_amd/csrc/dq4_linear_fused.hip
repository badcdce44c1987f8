// dq4_linear_fused.hip -- products over nested 4-bit weights with a fused
// epilogue: the linear layer (bias, activation, residual), the gated half of a
// feed-forward block, and the backward passes (include/dq4_linear.h).
//
// Route for any size: the weight is decoded once into 16-bit operand fragments
// of the matrix instruction in the workspace (weight_fragments_kernel,
// weight_row_fragments_kernel), then one matrix kernel (fragment_product_kernel,
// fragment_product_wide_kernel) multiplies and finishes each output in its
// epilogue.  The decode moves 2.5 bytes per weight element, the product 2 m
// operations per element: the decode is small against the product once m is
// above a thousand.
//
// Fewer rows: the call is bound by reading the 4-bit weight and by decoding it,
// so the weight is decoded straight into operand registers and no copy is
// written: token_rows_kernel (forward, m <= 2), batch_rows_kernel (forward, m <=
// 64), tile_rows_kernel (forward, m <= 1024), ragged_rows_kernel (forward, m <=
// 64, rows of whole dwords only), weight_columns_kernel (backward, m <= 128).
//
// Fragment layout.  The output columns n (weight rows forward, weight columns
// backward) are taken in groups of 128, the summed index k in chunks of 64.
// One (group, chunk) is 16 KiB: [2 k-steps of 32][8 fragments f][64 lanes][8
// k], so that a fragment is 1 KiB in lane order: it moves from HBM to LDS and
// from LDS to registers in straight lines, without bank conflicts, whatever
// the weight's own layout.  Row r of fragment f is output column 8 r + f of
// the group: a lane, which holds D rows 4 g + i of every fragment, then holds
// 8 neighbouring columns per i and writes 16 bytes at once.  The gated
// forward puts 64 gate columns (fragments 0-3, column 4 r + f) beside the same
// 64 up columns (fragments 4-7) in one group, so that act(g) * u is formed in
// registers.  The gated backward lays the chunks of Wg and Wu one after the
// other: one sum over both.  Columns and k beyond the matrix are zeros.

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "dq4.h"
#include "dq4_device.h"
#include "dq4_int8.h"
#include "dq4_linear.h"
#include "dq4_linear_device.h"

#pragma clang fp contract(off)

namespace dq4 {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 128;                  // output columns per fragment group
constexpr int kChunk = 64;                   // k per chunk
constexpr int kFrags = 8;                    // fragments per group and k-step
constexpr int kFragBytes = 1024;
constexpr int kUnitBytes = 2 * kFrags * kFragBytes;  // one (group, chunk): 16 KiB
constexpr int kXcds = 8;
// m, n_out, n_in, and an m x n_out or m x n_in matrix: what keeps every grid and
// 32-bit offset below in range.
constexpr int64_t kMaxDim = int64_t{1} << 21, kMaxMatrix = int64_t{1} << 39;

// How the fragments of a call are laid out from its weight or weights.
enum Layout {
    kSingle = 0,   // one weight
    kSideBySide = 1,  // gated forward: 64 gate and 64 up columns per group
    kStacked = 2   // gated backward: the k-chunks of Wg, then those of Wu
};

struct FragmentArgs {
    Weight w[2];
    uint16_t *out;
    int64_t n_out, n_in;  // the weight's shape (both weights)
    int32_t log2_block;
    int32_t group0;       // first fragment group of this launch
    int32_t groups;
    int32_t chunks;       // per weight
    int32_t layout;
};

// One weight's lookup tables in LDS.
struct Tables {
    float scb[256];
    float cb4[16];
};

__device__ __forceinline__ void load_tables(const Weight &w, Tables &t)
{
    const int i = threadIdx.x;
    if (i < 256)
        t.scb[i] = w.scale_codebook[i];
    if (i < 16)
        t.cb4[i] = w.codebook4[i];
}

__device__ __forceinline__ float scale_of(const Weight &w, const Tables &t, int64_t block)
{
    return block_scale(t.scb[w.scale_codes[block]], w.nested_absmax[block >> kNestedLog2],
                       w.offset);
}

// The FP32 products of elements e .. e + valid - 1 (valid in 1 .. 8) of the flat
// weight, before their rounding to T, zeros after them; any alignment.  The
// codes are 32 bits out of two neighbouring dwords (the dword with the last
// byte is read whole, nothing beyond it), and since blocks are longer than 8
// elements at most two of them meet.
__device__ __forceinline__ void octet_of(const Weight &w, const Tables &t, int log2_block,
                                         int64_t last_byte, int64_t e, int valid, float (&v)[8])
{
    const uintptr_t address = reinterpret_cast<uintptr_t>(w.packed);
    const uint32_t skew = static_cast<uint32_t>(address & 3);
    const uint32_t *words = reinterpret_cast<const uint32_t *>(address - skew);
    const int64_t bit = static_cast<int64_t>(skew) * 8 + 4 * e;
    const int64_t at = bit >> 5, last = (last_byte + skew) >> 2;
    const uint32_t lo = words[at], hi = words[at < last ? at + 1 : at];
    const uint32_t word = __builtin_amdgcn_alignbit(hi, lo, static_cast<uint32_t>(bit) & 31);
    const int64_t b = e >> log2_block;
    const int64_t b_last = (e + valid - 1) >> log2_block;
    const float s_lo = scale_of(w, t, b), s_hi = scale_of(w, t, b_last);
    const int64_t meet = ((b + 1) << log2_block) - e;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float p = t.cb4[(word >> (4 * j)) & 15u] * (j < meet ? s_lo : s_hi);
        v[j] = j < valid ? p : 0.0f;
    }
}

// ---------------------------------------------------------------------------
// what a call does beside the decode, before its product
// ---------------------------------------------------------------------------
// One row block of x rows (any alignment and stride) into rows of ld_out
// elements, zeros from column k on: the form the product reads in 16-byte
// pieces.
struct CopyArgs {
    const uint16_t *x;
    int64_t ld_x, m, k;
    uint16_t *out;
    int64_t ld_out;
};

constexpr int kRowBlock = 32;  // rows of a block beside the decode

__device__ __forceinline__ void copy_rows_zero_padded(const CopyArgs &a, int64_t bx, int64_t by)
{
    const int64_t c = bx * kThreads + threadIdx.x;
    if (c >= a.ld_out)
        return;
    const int64_t r0 = by * kRowBlock, r1 = r0 + kRowBlock < a.m ? r0 + kRowBlock : a.m;
#pragma unroll 8
    for (int64_t r = r0; r < r1; ++r)
        a.out[r * a.ld_out + c] = c < a.k ? a.x[r * a.ld_x + c] : static_cast<uint16_t>(0);
}

struct SlopeArgs {
    const uint16_t *dy;
    int64_t ld_dy;
    const uint16_t *pre[2];     // z, or g and u
    int64_t ld_pre;
    uint16_t *dz[2];
    int64_t ld_dz;
    uint16_t *pad[2];           // padded copies for the product, or null
    int64_t ld_pad;             // their columns
    int64_t pad_rows;           // their rows
    int32_t frag_rows;          // 0: copies in rows; else in operand fragments, 16 frag_rows
                                // rows a slice: [slice][32 columns][16 rows][lane][8]
    float *partial;             // column sums, one row per row block, or null
    int64_t m, n;
    int32_t act;
};

// dz = T(dy act'(pre)), or dgate and dup, of one block of rows.  A thread takes
// N neighbouring columns (8, a 16-byte load, where every matrix has 16-byte
// aligned rows; else 1) and every eighth row; the column sums of the unrounded
// products (the bias gradient) are FP32 additions in a fixed order: a thread's
// rows, then the eight threads of a column.
// The product that follows takes dz in T, as it is written here and as an
// adapter's gradient takes it: the matrix instruction's operands are 16 bits
// wide, and dz as a sum of two of them would double its work (gated 11008 x
// 4096 with 2048 rows: 330 us of 425 once more).  The rounding of dz and that
// of dx are of one size, so dx's error is sqrt 2 times that of a product of the
// unrounded dz (relative to dx, root mean square: BF16 2.3e-3 against 1.7e-3,
// FP16 2.9e-4 against 2.1e-4).
template <int OUT, bool kGated, int N>
__device__ __forceinline__ void activation_slopes(const SlopeArgs &a, int64_t bx, int64_t by,
                                                  float (&sums)[8][32 * N])
{
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = (bx * 32 + tx) * N;
    const int64_t width = a.pad[0] ? a.ld_pad : a.n;
    const int64_t r0 = by * kRowBlock;
    const int64_t rows = a.pad[0] ? a.pad_rows : a.m;
    const int64_t r1 = r0 + kRowBlock < rows ? r0 + kRowBlock : rows;
    float sum[N] = {};
    if (c < width) {
        for (int64_t r = r0 + ty; r < r1; r += 8) {
            float z0[N] = {}, z1[N] = {};
            if (c < a.n && r < a.m) {
                float dy[N], pre[N], up[N];
                load_values<OUT, N>(a.dy + r * a.ld_dy + c, N > 1, N, dy);
                if (a.act != DQ4_ACT_NONE)
                    load_values<OUT, N>(a.pre[0] + r * a.ld_pre + c, N > 1, N, pre);
                if constexpr (kGated)
                    load_values<OUT, N>(a.pre[1] + r * a.ld_pre + c, N > 1, N, up);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    float value, slope;
                    if constexpr (kGated) {
                        act_and_slope_f32(a.act, pre[j], &value, &slope);
                        z0[j] = dy[j] * up[j] * slope;
                        z1[j] = dy[j] * value;
                    } else {
                        z0[j] = dy[j];
                        if (a.act != DQ4_ACT_NONE) {
                            act_and_slope_f32(a.act, pre[j], &value, &slope);
                            z0[j] = dy[j] * slope;
                        }
                        sum[j] = sum[j] + z0[j];
                    }
                }
                if (a.dz[0])
                    store_values<OUT, N>(a.dz[0] + r * a.ld_dz + c, N > 1, N, z0);
                if constexpr (kGated)
                    store_values<OUT, N>(a.dz[1] + r * a.ld_dz + c, N > 1, N, z1);
            }
            if (a.pad[0]) {
                int64_t at = r * a.ld_pad + c;
                if (a.frag_rows) {
                    const uint32_t tf = a.frag_rows, block = static_cast<uint32_t>(r) >> 4;
                    const int64_t slice = block / tf, t = block - slice * tf;
                    at = ((slice * (a.ld_pad >> 5) + (c >> 5)) * tf + t) * 512 +
                         (((c >> 3) & 3) * 16 + (r & 15)) * 8 + (c & 7);
                }
                store_values<OUT, N>(a.pad[0] + at, N > 1, N, z0);
                if constexpr (kGated)
                    store_values<OUT, N>(a.pad[1] + at, N > 1, N, z1);
            }
        }
    }
    if constexpr (!kGated) {
        if (a.partial) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                sums[ty][tx * N + j] = sum[j];
            __syncthreads();
            for (int i = threadIdx.x; i < 32 * N; i += kThreads) {
                float total = sums[0][i];
#pragma unroll
                for (int q = 1; q < 8; ++q)
                    total = total + sums[q][i];
                const int64_t col = bx * (32 * N) + i;
                if (col < a.n)
                    a.partial[by * a.n + col] = total;
            }
        }
    }
}

// The work that goes with a decode launch.
enum Beside {
    kNothing = 0,
    kCopy = 1,
    kSlopes8 = 2,       // linear backward, 8 columns a thread
    kSlopes1 = 3,
    kGatedSlopes8 = 4,  // gated backward
    kGatedSlopes1 = 5
};

struct BesideArgs {
    int32_t blocks;     // workgroups of this work, after those of the decode: one a piece
    int32_t first;      // their first piece
    int32_t columns;    // pieces along the columns
    CopyArgs copy;
    SlopeArgs slope;
};

template <int OUT, int kBeside>
__device__ __forceinline__ void work_beside(const BesideArgs &b, int block)
{
    const int item = b.first + block;
    const int by = item / b.columns, bx = item - by * b.columns;
    if constexpr (kBeside == kCopy) {
        copy_rows_zero_padded(b.copy, bx, by);
    } else if constexpr (kBeside >= kSlopes8) {
        constexpr bool kGated = kBeside >= kGatedSlopes8;
        constexpr int N = kBeside == kSlopes8 || kBeside == kGatedSlopes8 ? 8 : 1;
        __shared__ float sums[8][32 * N];
        activation_slopes<OUT, kGated, N>(b.slope, bx, by, sums);
    }
}

// Decode into fragments.  kForward: k runs along the weight's rows (n_in), a
// 16-byte unit is 8 neighbouring elements of one row, one packed dword.
// Backward: k runs down the weight's columns; a thread takes the dwords of 8
// rows (8 columns each) and writes 8 units, each pairing the same column of
// the 8 rows.  kAligned: rows start on packed dwords (n_in % 8 == 0, 4-byte
// aligned codes); otherwise eight elements are cut out of two dwords.
// Bound by memory: 0.5 B read and 2 B written per element.  Workgroups behind
// the decode's do the call's other work before the product (kBeside), which
// does not depend on the weight: one launch, and neither waits for the other.
template <int OUT, bool kForward, bool kAligned, int kBeside>
__global__ __launch_bounds__(kThreads) void weight_fragments_kernel(FragmentArgs a, BesideArgs b)
{
    if constexpr (kBeside != kNothing) {
        const int first = static_cast<int>(gridDim.x) - b.blocks;
        if (static_cast<int>(blockIdx.x) >= first) {
            work_beside<OUT, kBeside>(b, static_cast<int>(blockIdx.x) - first);
            return;
        }
    }
    __shared__ Tables tables[2];
    const int n_weights = a.layout == kSingle ? 1 : 2;
    load_tables(a.w[0], tables[0]);
    if (n_weights == 2)
        load_tables(a.w[1], tables[1]);
    __syncthreads();

    const int tid = threadIdx.x;
    const int lb = a.log2_block;
    const int64_t last_byte = (a.n_out * a.n_in - 1) >> 1;
    const int all_chunks = a.layout == kStacked ? 2 * a.chunks : a.chunks;
    if constexpr (kForward) {
        // a workgroup decodes 4 chunks (256 k, 128 packed bytes a row) of a group
        const int spans = (all_chunks + 3) / 4;
        const int group = blockIdx.x / spans;
        const int span = blockIdx.x - group * spans;
        uint16_t *base = a.out + static_cast<int64_t>(group) * all_chunks * (kUnitBytes / 2);
        for (int it = 0; it < 16; ++it) {
            const int u = it * kThreads + tid;  // unit within the 4 chunks
            const int lane = u & 63, f = (u >> 6) & 7, ks = (u >> 9) & 1;
            const int chunk = span * 4 + (u >> 10);
            if (chunk >= all_chunks)
                break;
            const int r = lane & 15;
            int which = 0;
            int64_t o;
            if (a.layout == kSideBySide) {
                which = f >> 2;
                o = static_cast<int64_t>(a.group0 + group) * 64 + 4 * r + (f & 3);
            } else {
                o = static_cast<int64_t>(a.group0 + group) * kGroup + 8 * r + f;
            }
            const int64_t k = static_cast<int64_t>(chunk) * kChunk + ks * 32 + (lane >> 4) * 8;
            u32x4 q = {0, 0, 0, 0};
            if (o < a.n_out && k < a.n_in) {
                const Weight &w = a.w[which];
                const Tables &t = tables[which];
                const int64_t e0 = o * a.n_in + k;
                float v[8];
                if constexpr (kAligned) {
                    const uint32_t word = *reinterpret_cast<const uint32_t *>(w.packed + (e0 >> 1));
                    const float s = scale_of(w, t, e0 >> lb);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] = t.cb4[(word >> (4 * j)) & 15u] * s;
                } else {
                    octet_of(w, t, lb, last_byte, e0, static_cast<int>(a.n_in - k < 8 ? a.n_in - k : 8), v);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    q[j] = Half<OUT>::pack2(v[2 * j], v[2 * j + 1]);
            }
            *reinterpret_cast<u32x4 *>(base + static_cast<int64_t>(chunk) * (kUnitBytes / 2) +
                                       (u & 1023) * 8) = q;
        }
    } else {
        // a workgroup decodes one chunk (64 weight rows) of two groups
        const int pair = blockIdx.x / all_chunks;
        const int chunk = blockIdx.x - pair * all_chunks;
        const int lane = tid & 63, ks = (tid >> 6) & 1, group = pair * 2 + (tid >> 7);
        if (group >= a.groups)
            return;
        const int which = chunk >= a.chunks ? 1 : 0;
        const Weight &w = a.w[which];
        const Tables &t = tables[which];
        const int64_t o0 = static_cast<int64_t>(chunk - which * a.chunks) * kChunk + ks * 32 +
                           (lane >> 4) * 8;
        const int64_t j0 = static_cast<int64_t>(a.group0 + group) * kGroup + 8 * (lane & 15);
        u32x4 q[8];
#pragma unroll
        for (int f = 0; f < 8; ++f)
            q[f] = u32x4{0, 0, 0, 0};
        if (j0 < a.n_in) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {  // two weight rows at a time
                float v[2][8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t o = o0 + 2 * p + h;
                    const int64_t e0 = o * a.n_in + j0;
                    if (o >= a.n_out) {
#pragma unroll
                        for (int f = 0; f < 8; ++f)
                            v[h][f] = 0.0f;
                    } else if constexpr (kAligned) {
                        const uint32_t word =
                            *reinterpret_cast<const uint32_t *>(w.packed + (e0 >> 1));
                        const float s = scale_of(w, t, e0 >> lb);
#pragma unroll
                        for (int f = 0; f < 8; ++f)
                            v[h][f] = t.cb4[(word >> (4 * f)) & 15u] * s;
                    } else {
                        octet_of(w, t, lb, last_byte, e0,
                                 static_cast<int>(a.n_in - j0 < 8 ? a.n_in - j0 : 8), v[h]);
                    }
                }
#pragma unroll
                for (int f = 0; f < 8; ++f)
                    q[f][p] = Half<OUT>::pack2(v[0][f], v[1][f]);
            }
        }
        uint16_t *base = a.out + (static_cast<int64_t>(group) * all_chunks + chunk) * (kUnitBytes / 2) +
                         ks * (kFrags * kFragBytes / 2) + lane * 8;
#pragma unroll
        for (int f = 0; f < 8; ++f)
            *reinterpret_cast<u32x4 *>(base + f * (kFragBytes / 2)) = q[f];
    }
}

// 8 codes of a row at byte address `at`; kAligned: one load.  Else dwords, none past
// the one that holds the weight's last byte.
template <bool kAligned>
__device__ __forceinline__ u32x2 load_codes8(uintptr_t at, uintptr_t last)
{
    if constexpr (kAligned) {
        return *reinterpret_cast<const u32x2 *>(at);
    } else {
        uint32_t d[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const uintptr_t w = (at & ~uintptr_t{3}) + 4 * i;
            d[i] = *reinterpret_cast<const uint32_t *>(w < last ? w : last);
        }
        return u32x2{__builtin_amdgcn_alignbyte(d[1], d[0], static_cast<uint32_t>(at) & 3),
                     __builtin_amdgcn_alignbyte(d[2], d[1], static_cast<uint32_t>(at) & 3)};
    }
}

// 8 rows of 8 columns to the 8 columns' pieces of 8 rows, as dq4_int8_prep rounds.
template <int OUT>
__device__ __forceinline__ void decode_codes(const u32x2 (&code)[8], const float (&scale)[8], u32x4 (&q)[8])
{
    constexpr float kR127 = 0x1.020408p-7f;  // the FP32 value nearest 1/127
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int f = 0; f < 8; ++f) {
            float v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int8_t c = static_cast<int8_t>(code[2 * p + h][f / 4] >> (8 * (f & 3)));
                const float scaled = static_cast<float>(c) * scale[2 * p + h];
                // columns past the last one: products that nobody takes
                v[h] = scaled * kR127;
            }
            q[f][p] = Half<OUT>::pack2(v[0], v[1]);
        }
}

// The columns of an LLM.int8 weight (include/dq4_int8.h) as fragments of 16-bit
// values, laid out as in the backward decode above.  kAligned: 8 codes of a row are
// an aligned 8-byte load; otherwise they are cut out of three dwords (the dword
// with the weight's last byte is read whole, nothing beyond it).  Bound by memory:
// 1 byte read and 2 written per element (11008 x 4096: 33 us, 4.1 TB/s).  Workgroups
// behind these do the call's work beside the decode, as above.
struct Int8FragmentArgs {
    const int8_t *codes;
    const float *scales;
    uint16_t *out;
    int64_t n_out, n_in;
    int32_t groups, chunks;
};

template <int OUT, bool kAligned, int kBeside>
__global__ __launch_bounds__(kThreads) void int8_column_fragments_kernel(Int8FragmentArgs a, BesideArgs b)
{
    if constexpr (kBeside != kNothing) {
        const int first = static_cast<int>(gridDim.x) - b.blocks;
        if (static_cast<int>(blockIdx.x) >= first) {
            work_beside<OUT, kBeside>(b, static_cast<int>(blockIdx.x) - first);
            return;
        }
    }
    const int tid = threadIdx.x;
    const int pair = blockIdx.x / a.chunks, chunk = blockIdx.x - pair * a.chunks;
    const int lane = tid & 63, ks = (tid >> 6) & 1, group = pair * 2 + (tid >> 7);
    if (group >= a.groups)
        return;
    const int64_t o0 = static_cast<int64_t>(chunk) * kChunk + ks * 32 + (lane >> 4) * 8;
    const int64_t j0 = static_cast<int64_t>(group) * kGroup + 8 * (lane & 15);
    const uintptr_t base = reinterpret_cast<uintptr_t>(a.codes);
    const uintptr_t last = (base + a.n_out * a.n_in - 1) & ~uintptr_t{3};
    u32x4 q[8];
#pragma unroll
    for (int f = 0; f < 8; ++f)
        q[f] = u32x4{0, 0, 0, 0};
    if (j0 < a.n_in) {
        u32x2 code[8];
        float scale[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            const int64_t o = o0 + h;
            code[h] = u32x2{0, 0};
            scale[h] = 0.0f;
            if (o < a.n_out) {
                scale[h] = a.scales[o];
                code[h] = load_codes8<kAligned>(base + o * a.n_in + j0, last);
            }
        }
        decode_codes<OUT>(code, scale, q);
    }
    uint16_t *to = a.out + (static_cast<int64_t>(group) * a.chunks + chunk) * (kUnitBytes / 2) +
                   ks * (kFrags * kFragBytes / 2) + lane * 8;
#pragma unroll
    for (int f = 0; f < 8; ++f)
        *reinterpret_cast<u32x4 *>(to + f * (kFragBytes / 2)) = q[f];
}

// ---------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------
struct ProductArgs {
    const uint16_t *wfrag;      // group-major fragments of this launch's groups
    const uint16_t *x[2];       // the second is read by chunks [chunks, 2 chunks)
    int64_t ld_x;
    int64_t k;                  // readable columns of an x matrix, a multiple of 8
    int64_t m, n;               // rows; output columns in all (gated: h's columns)
    int64_t n0;                 // first output column of this launch
    int32_t groups;             // of this launch
    int32_t chunks;             // per x matrix
    int32_t n_x;
    int32_t act;
    int32_t vec;                // outputs and residual take whole vectors
    int32_t tiles_t;
    int32_t splits;             // of the chunks; above 1 the sums go to `partial`
    f32x4 *partial;             // [split][tile][wave][f][16 rows][lane]
    const uint16_t *bias;
    const uint16_t *residual;
    int64_t ld_residual;
    uint16_t *y;
    int64_t ld_y;
    uint16_t *pre[2];
    int64_t ld_pre;
    const float *bias_partial;  // column sums of row blocks, added up by workgroups
    float *dbias;               // of their own (blockIdx.y == splits), or null
    int64_t bias_n;
    int32_t bias_blocks;
};

// dbias[c] = the row blocks' sums, added in order.
__device__ __forceinline__ void add_bias_blocks(const float *partial, int64_t n, int32_t blocks,
                                                float *dbias)
{
    for (int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; c < n;
         c += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        float sum = 0.0f;
#pragma unroll 8
        for (int32_t b = 0; b < blocks; ++b)
            sum = sum + partial[b * n + c];
        dbias[c] = sum;
    }
}

// Outputs of one row: columns n0 .. n0 + 7 of a linear call.
template <int OUT>
__device__ __forceinline__ void finish_linear(const ProductArgs &a, int64_t row, int64_t n0,
                                              float (&z)[8])
{
    const int64_t left = a.n - n0;
    if (row >= a.m || left <= 0)
        return;
    const int valid = left < 8 ? static_cast<int>(left) : 8;
    const bool vec = a.vec && valid == 8;
    if (a.bias) {
        float b[8];
        load_values<OUT, 8>(a.bias + n0, vec, valid, b);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            z[j] = z[j] + b[j];
    }
    if (a.pre[0])
        store_values<OUT, 8>(a.pre[0] + row * a.ld_pre + n0, vec, valid, z);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        z[j] = act_f32(a.act, z[j]);
    if (a.residual) {
        float r[8];
        load_values<OUT, 8>(a.residual + row * a.ld_residual + n0, vec, valid, r);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            z[j] = z[j] + r[j];
    }
    store_values<OUT, 8>(a.y + row * a.ld_y + n0, vec, valid, z);
}

// Columns n0 .. n0 + 3 of a gated call.
template <int OUT>
__device__ __forceinline__ void finish_gated(const ProductArgs &a, int64_t row, int64_t n0,
                                             float (&g)[4], float (&u)[4])
{
    const int64_t left = a.n - n0;
    if (row >= a.m || left <= 0)
        return;
    const int valid = left < 4 ? static_cast<int>(left) : 4;
    const bool vec = a.vec && valid == 4;
    if (a.pre[0]) {
        store_values<OUT, 4>(a.pre[0] + row * a.ld_pre + n0, vec, valid, g);
        store_values<OUT, 4>(a.pre[1] + row * a.ld_pre + n0, vec, valid, u);
    }
    float h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        h[j] = act_f32(a.act, g[j]) * u[j];
    store_values<OUT, 4>(a.y + row * a.ld_y + n0, vec, valid, h);
}

constexpr int kFinishLd = kGroup + 4;  // floats per row of a wave's epilogue slab

// Rows 4 it .. 4 it + 3 of a slab of 16 rows: a lane finishes 8 columns of one.
template <int OUT, bool kGated>
__device__ __forceinline__ void finish_slab_rows(const ProductArgs &a, const float *slab,
                                                 int64_t row0, int group, int it, int lane)
{
    const int g = lane >> 4, c = lane & 15;
    const float *from = slab + (it * 4 + g) * kFinishLd + 8 * c;
    const f32x4 lo = *reinterpret_cast<const f32x4 *>(from);
    const f32x4 hi = *reinterpret_cast<const f32x4 *>(from + 4);
    const int64_t row = row0 + it * 4 + g;
    if constexpr (kGated) {
        float gv[4] = {lo[0], lo[1], lo[2], lo[3]}, uv[4] = {hi[0], hi[1], hi[2], hi[3]};
        finish_gated<OUT>(a, row, a.n0 + static_cast<int64_t>(group) * 64 + 4 * c, gv, uv);
    } else {
        float z[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        finish_linear<OUT>(a, row, a.n0 + static_cast<int64_t>(group) * kGroup + 8 * c, z);
    }
}

// The epilogue of one wave's 128 columns x 16 TF rows.  16 rows at a time pass
// through a slab of LDS that only this wave uses: a lane holds 8 neighbouring
// columns of one row per D register, so the slab takes and gives whole
// vectors, and the code after it is there once instead of once per register.
template <int OUT, bool kGated, int TF>
__device__ __forceinline__ void finish_wave(const ProductArgs &a, const f32x4 (&acc)[kFrags][TF],
                                            float *slab, int64_t row0, int group, int lane)
{
    const int g = lane >> 4, c = lane & 15;
#pragma unroll
    for (int t = 0; t < TF; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float *to = slab + c * kFinishLd + 8 * (4 * g + i);
            *reinterpret_cast<f32x4 *>(to) =
                f32x4{acc[0][t][i], acc[1][t][i], acc[2][t][i], acc[3][t][i]};
            *reinterpret_cast<f32x4 *>(to + 4) =
                f32x4{acc[4][t][i], acc[5][t][i], acc[6][t][i], acc[7][t][i]};
        }
        // the wave's LDS operations complete in order; the compiler must not
        // move the reads of other lanes' values above the writes
        __asm__ volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int it = 0; it < 4; ++it)
            finish_slab_rows<OUT, kGated>(a, slab, row0 + t * 16, group, it, lane);
        __asm__ volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
    }
}

// Tile of 128 WN output columns x 16 TF WT rows; wave (wn, wt) takes group wn
// of the tile and 16 TF rows.  Both operands go from HBM to LDS without
// passing registers, double-buffered by chunks of 64 k.  Bound by the waits at
// each chunk's barrier, which two or three workgroups per CU cover in part:
// 0.77 PFLOP/s with 128 x 128, 0.45 with 128 x 64 (large products; the sizes
// that take them have too few tiles of 256 x 256 to fill the GPU).
template <int OUT, bool kGated, int WN, int WT, int TF>
__global__ __launch_bounds__(64 * WN * WT) void fragment_product_kernel(ProductArgs a)
{
    constexpr int kRows = 16 * TF * WT;
    constexpr int kWBytes = WN * kUnitBytes;
    constexpr int kXBytes = kRows * kChunk * 2;
    constexpr int kStage = kWBytes + kXBytes;
    constexpr int kWaves = WN * WT;
    constexpr int kWLoads = WN * 16 / kWaves;          // 1 KiB loads per wave and chunk
    constexpr int kXLoads = 2 * TF * WT / kWaves;
    if (static_cast<int>(blockIdx.y) == a.splits) {
        add_bias_blocks(a.bias_partial, a.bias_n, a.bias_blocks, a.dbias);
        return;
    }
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage];
    static_assert(kWaves * 16 * kFinishLd * 4 <= 2 * kStage, "the epilogue slabs fit the stages");

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % WN, wt = wave / WN;

    // consecutive workgroups go to the XCDs in turn: give each XCD a
    // contiguous run of tiles, so that its L2 serves their shared operands
    const int tiles = gridDim.x;
    const int per = tiles / kXcds, extra = tiles % kXcds;
    const int xcd = blockIdx.x % kXcds, idx = blockIdx.x / kXcds;
    const int tile = xcd * per + (xcd < extra ? xcd : extra) + idx;
    const int tile_n = tile / a.tiles_t, tile_t = tile - tile_n * a.tiles_t;
    const int group0 = tile_n * WN;
    const int64_t row0 = static_cast<int64_t>(tile_t) * kRows;

    const int all_chunks = a.chunks * a.n_x;
    // loads: W fragments are straight 1 KiB runs; group wl of the tile
    u32x4 rs_w[WN];
#pragma unroll
    for (int q = 0; q < WN; ++q) {
        const int group = group0 + q < a.groups ? group0 + q : a.groups - 1;
        rs_w[q] = make_rsrc(reinterpret_cast<const uint8_t *>(a.wfrag) +
                                static_cast<int64_t>(group) * all_chunks * kUnitBytes,
                            static_cast<uint32_t>(all_chunks) * kUnitBytes);
    }
    // x: 16 rows x 32 k per load; rows past the end lie past the buffer
    const int64_t rows_left = a.m - row0;
    const int64_t rows_here = rows_left < kRows ? rows_left : kRows;
    const uint32_t x_bytes = static_cast<uint32_t>(((rows_here - 1) * a.ld_x + a.k) * 2);
    u32x4 rs_x[2];
    rs_x[0] = make_rsrc(a.x[0] + row0 * a.ld_x, x_bytes);
    rs_x[1] = make_rsrc(a.x[a.n_x - 1] + row0 * a.ld_x, x_bytes);
    uint32_t x_off[kXLoads], x_lds[kXLoads];
    int32_t x_k[kXLoads];
#pragma unroll
    for (int q = 0; q < kXLoads; ++q) {
        const int fr = wave * kXLoads + q;  // fragment: k-step fr & 1 of row block fr >> 1
        const int row = (fr >> 1) * 16 + (lane & 15);
        x_k[q] = (fr & 1) * 32 + (lane >> 4) * 8;
        // a single row's stride is not looked at: rows past the end get an
        // offset past any buffer
        x_off[q] = row < rows_here
                       ? static_cast<uint32_t>(row * static_cast<int32_t>(a.ld_x) + x_k[q]) * 2u
                       : 0x80000000u;
        x_lds[q] = kWBytes + fr * kFragBytes;
    }
    const uint32_t lds0 = lds_offset(lds);
    const uint32_t w_voff = lane * 16;

    auto issue = [&](int c, int buf) {
        const uint32_t to = lds0 + buf * kStage;
#pragma unroll
        for (int q = 0; q < kWLoads; ++q) {
            const int fr = wave * kWLoads + q;  // of WN * 16
            buffer_to_lds(rs_w[fr / 16], w_voff,
                          static_cast<uint32_t>(c) * kUnitBytes + (fr % 16) * kFragBytes,
                          to + fr * kFragBytes);
        }
        const int second = c >= a.chunks ? 1 : 0;
        const int ck = c - second * a.chunks;
        const u32x4 rs = second ? rs_x[1] : rs_x[0];
        const int32_t k_left = static_cast<int32_t>(a.k - static_cast<int64_t>(ck) * kChunk);
#pragma unroll
        for (int q = 0; q < kXLoads; ++q) {
            const uint32_t off = x_off[q] + static_cast<uint32_t>(ck) * (kChunk * 2);
            buffer_to_lds(rs, x_k[q] < k_left ? off : 0x80000000u, 0, to + x_lds[q]);
        }
    };

    f32x4 acc[kFrags][TF];
#pragma unroll
    for (int f = 0; f < kFrags; ++f)
#pragma unroll
        for (int t = 0; t < TF; ++t)
            acc[f][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // this split's chunks
    const int split = blockIdx.y;
    const int c_first = static_cast<int>(static_cast<uint32_t>(all_chunks) * split / a.splits);
    const int c_last = static_cast<int>(static_cast<uint32_t>(all_chunks) * (split + 1) / a.splits);
    if (c_first < c_last) {
        issue(c_first, c_first & 1);
        wait_all_and_barrier();
    }
    for (int c = c_first; c < c_last; ++c) {
        const int buf = c & 1;
        if (c + 1 < c_last)
            issue(c + 1, buf ^ 1);
        const uint8_t *w_lds = lds + buf * kStage + wn * kUnitBytes + lane * 16;
        const uint8_t *x_l = lds + buf * kStage + kWBytes + wt * (TF * 2 * kFragBytes) + lane * 16;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            u32x4 wf[kFrags], xf[TF];
#pragma unroll
            for (int t = 0; t < TF; ++t)
                xf[t] = *reinterpret_cast<const u32x4 *>(x_l + (2 * t + ks) * kFragBytes);
#pragma unroll
            for (int f = 0; f < kFrags; ++f)
                wf[f] = *reinterpret_cast<const u32x4 *>(w_lds + (ks * kFrags + f) * kFragBytes);
#pragma unroll
            for (int f = 0; f < kFrags; ++f)
#pragma unroll
                for (int t = 0; t < TF; ++t)
                    acc[f][t] = Half<OUT>::mfma(wf[f], xf[t], acc[f][t]);
        }
        wait_all_and_barrier();
    }

    if (group0 + wn >= a.groups)
        return;
    if (a.splits > 1) {
        f32x4 *to = a.partial + ((static_cast<int64_t>(split) * tiles + tile) * kWaves + wave) *
                                    (kFrags * TF * 64) + lane;
#pragma unroll
        for (int f = 0; f < kFrags; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                to[(f * TF + t) * 64] = acc[f][t];
        return;
    }
    finish_wave<OUT, kGated, TF>(a, acc, reinterpret_cast<float *>(lds) + wave * (16 * kFinishLd),
                                 row0 + wt * (TF * 16), group0 + wn, lane);
}

// The 256 x 256 tile, for large products: 8 waves in two halves, one of each
// half on every SIMD.  A wave alternates between a load phase (its operand
// fragments of one k-step of 32 from LDS, and the loads from HBM to LDS of the
// k-step three ahead) and a product phase (32 matrix instructions); every phase
// ends on a barrier and the halves are one phase apart, so that while one
// wave of a SIMD multiplies the other one loads.  Four buffers of one k-step
// each: the step three ahead goes where step h - 1 lay, which both halves have
// read by then, and it has four phases (about 2000 cycles) or more to arrive.
// Bound by the matrix pipe at the clock it runs at under this load, and by the
// last round of tiles: 22016 x 4096 columns by 4096 rows in 638 us, 1.16 PFLOP/s;
// 57344 x 8192 by 512 rows, 448 tiles on 256 CUs, 453 us, 1.06.
template <int OUT, bool kGated>
__global__ __launch_bounds__(512) void fragment_product_wide_kernel(ProductArgs a)
{
    constexpr int WN = 2, WT = 4, TF = 4;
    constexpr int kRows = 16 * TF * WT;
    constexpr int kStepW = kFrags * kFragBytes;      // one group's fragments of one k-step
    constexpr int kStage = WN * kStepW + kRows * 64;  // 32 KiB
    if (static_cast<int>(blockIdx.y) == a.splits) {
        add_bias_blocks(a.bias_partial, a.bias_n, a.bias_blocks, a.dbias);
        return;
    }
    __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * kStage];
    static_assert(8 * 16 * kFinishLd * 4 <= 4 * kStage, "the epilogue slabs fit the stages");

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % WN, wt = wave / WN;

    // each XCD takes a contiguous run of tiles, as in fragment_product_kernel
    const int tiles = gridDim.x;
    const int per = tiles / kXcds, extra = tiles % kXcds;
    const int xcd = blockIdx.x % kXcds, idx = blockIdx.x / kXcds;
    const int tile = xcd * per + (xcd < extra ? xcd : extra) + idx;
    const int tile_n = tile / a.tiles_t, tile_t = tile - tile_n * a.tiles_t;
    const int group0 = tile_n * WN;
    const int64_t row0 = static_cast<int64_t>(tile_t) * kRows;
    const int all_steps = a.chunks * a.n_x * 2;

    // this wave's loads of a step: W fragments 2 wave, 2 wave + 1 (of 16), x
    // fragments 2 wave, 2 wave + 1 (of 16)
    const int w_group = group0 + wave / 4 < a.groups ? group0 + wave / 4 : a.groups - 1;
    const u32x4 rs_w = make_rsrc(reinterpret_cast<const uint8_t *>(a.wfrag) +
                                     static_cast<int64_t>(w_group) * all_steps * kStepW,
                                 static_cast<uint32_t>(all_steps) * kStepW);
    const int64_t rows_left = a.m - row0;
    const int64_t rows_here = rows_left < kRows ? rows_left : kRows;
    const uint32_t x_bytes = static_cast<uint32_t>(((rows_here - 1) * a.ld_x + a.k) * 2);
    const u32x4 rs_x0 = make_rsrc(a.x[0] + row0 * a.ld_x, x_bytes);
    const u32x4 rs_x1 = make_rsrc(a.x[a.n_x - 1] + row0 * a.ld_x, x_bytes);
    uint32_t x_off[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int row = (2 * wave + q) * 16 + (lane & 15);
        x_off[q] = row < rows_here
                       ? static_cast<uint32_t>(row * static_cast<int32_t>(a.ld_x) + (lane >> 4) * 8) * 2u
                       : 0x80000000u;
    }
    const int32_t x_k = (lane >> 4) * 8;
    const uint32_t lds0 = lds_offset(lds);
    const uint32_t w_off = (wave % 4) * (2 * kFragBytes) + lane * 16;

    // this split's steps
    const int split = blockIdx.y;
    const int h_first = 2 * static_cast<int>(static_cast<uint32_t>(all_steps / 2) * split / a.splits);
    const int h_last = 2 * static_cast<int>(static_cast<uint32_t>(all_steps / 2) * (split + 1) / a.splits);

    // always 4 loads: past the last step they fetch nothing and write zeros
    // where nothing is read, so that the waits below count the same loads
    auto issue = [&](int h) {
        const uint32_t to = lds0 + (h & 3) * kStage;
        const bool real = h < h_last;
        const uint32_t w_at = real ? w_off : 0x80000000u;
        const uint32_t soff = real ? static_cast<uint32_t>(h) * kStepW : 0u;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            buffer_to_lds(rs_w, w_at + q * kFragBytes, soff,
                          to + (wave / 4) * kStepW + ((wave % 4) * 2 + q) * kFragBytes);
        const int second = h >= 2 * a.chunks ? 1 : 0;
        const int hk = h - second * 2 * a.chunks;
        const u32x4 rs = second ? rs_x1 : rs_x0;
        const int32_t k_left = static_cast<int32_t>(a.k) - hk * 32;
        const bool in = real && x_k < k_left;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            buffer_to_lds(rs, in ? x_off[q] + static_cast<uint32_t>(hk) * 64u : 0x80000000u, 0,
                          to + WN * kStepW + (2 * wave + q) * kFragBytes);
    };

    f32x4 acc[kFrags][TF];
#pragma unroll
    for (int f = 0; f < kFrags; ++f)
#pragma unroll
        for (int t = 0; t < TF; ++t)
            acc[f][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    issue(h_first);
    issue(h_first + 1);
    issue(h_first + 2);
    __asm__ volatile("s_waitcnt vmcnt(8)" ::: "memory");
    if (h_first == h_last)
        __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    if (wave >= 4)
        __builtin_amdgcn_s_barrier();  // the second half is one phase behind
    for (int h = h_first; h < h_last; ++h) {
        const uint8_t *stage = lds + (h & 3) * kStage;
        const uint8_t *w_lds = stage + wn * kStepW + lane * 16;
        const uint8_t *x_lds = stage + WN * kStepW + wt * (TF * kFragBytes) + lane * 16;
        u32x4 wf[kFrags], xf[TF];
#pragma unroll
        for (int t = 0; t < TF; ++t)
            xf[t] = *reinterpret_cast<const u32x4 *>(x_lds + t * kFragBytes);
#pragma unroll
        for (int f = 0; f < kFrags; ++f)
            wf[f] = *reinterpret_cast<const u32x4 *>(w_lds + f * kFragBytes);
        issue(h + 3);
        // this wave's share of step h + 1 has arrived (steps h + 2 and h + 3
        // are still under way), and its reads of step h are done
        __asm__ volatile("s_waitcnt vmcnt(8) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int f = 0; f < kFrags; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                acc[f][t] = Half<OUT>::mfma(wf[f], xf[t], acc[f][t]);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        // after the last barrier the buffers are the epilogue's: no load may
        // still be on its way into them
        if (h + 1 == h_last)
            __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    }
    if (wave < 4)
        __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");

    if (group0 + wn >= a.groups)
        return;
    if (a.splits > 1) {
        f32x4 *to = a.partial + ((static_cast<int64_t>(split) * tiles + tile) * 8 + wave) *
                                    (kFrags * TF * 64) + lane;
#pragma unroll
        for (int f = 0; f < kFrags; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                to[(f * TF + t) * 64] = acc[f][t];
        return;
    }
    finish_wave<OUT, kGated, TF>(a, acc, reinterpret_cast<float *>(lds) + wave * (16 * kFinishLd),
                                 row0 + wt * (TF * 16), group0 + wn, lane);
}

// The splits' sums of one wave's 128 columns x 16 rows, added in order, and
// the epilogue.  Four waves share the 8 fragments, so that a wave has the
// loads of 8 splits in flight: the kernel is short and its time is latency
// (about 4 us for up to a few MB of sums).
template <int OUT, bool kGated, int WN, int WT, int TF>
__global__ __launch_bounds__(256) void product_reduce_kernel(ProductArgs a, int32_t tiles)
{
    __shared__ __attribute__((aligned(16))) float slab[16 * kFinishLd];
    const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int t = blockIdx.y;
    const int tile = blockIdx.x / (WN * WT), wave = blockIdx.x % (WN * WT);
    const int wn = wave % WN, wt = wave / WN;
    const int tile_n = tile / a.tiles_t, tile_t = tile - tile_n * a.tiles_t;
    const int group = tile_n * WN + wn;
    const int64_t row0 = (static_cast<int64_t>(tile_t) * WT + wt) * (16 * TF) + 16 * t;
    if (group >= a.groups || row0 >= a.m)
        return;
    const f32x4 *from = a.partial + (static_cast<int64_t>(tile) * (WN * WT) + wave) * (kFrags * TF * 64) +
                        (2 * q * TF + t) * 64 + lane;
    const int64_t split_step = static_cast<int64_t>(tiles) * (WN * WT) * (kFrags * TF * 64);
    f32x4 acc[2];
#pragma unroll
    for (int f = 0; f < 2; ++f)
        acc[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < a.splits; s += 8) {
        f32x4 part[8][2];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int f = 0; f < 2; ++f)  // past the last split: the first again, left out below
                part[i][f] = from[(s + i < a.splits ? s + i : s) * split_step + f * TF * 64];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (s + i < a.splits)
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    acc[f] = acc[f] + part[i][f];
    }
    const int g = lane >> 4, c = lane & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x2 *>(slab + c * kFinishLd + 8 * (4 * g + i) + 2 * q) =
            f32x2{acc[0][i], acc[1][i]};
    __syncthreads();
    finish_slab_rows<OUT, kGated>(a, slab, row0, group, q, lane);
}

// ---------------------------------------------------------------------------
// few rows of an LLM.int8 layer's gradient: no fragments in memory
// ---------------------------------------------------------------------------
// A workgroup takes 128 columns and a share of the weight's rows for 16 TF tokens, its
// waves every eighth step of 32 rows: a wave loads 8 codes of 8 rows a lane, decodes
// them to operands in registers and multiplies; the next step is in flight meanwhile.
// The waves' sums meet in LDS, the workgroups' in product_reduce_kernel, both in a fixed
// order.  The last `bias_rows` rows of workgroups add up the bias gradient.  Bound by reading the
// weight: 28672 x 8192, 16 tokens, 3.7 TB/s, from 33 tokens on by reading it for each 32
// (sums of 64 do not fit the registers beside two steps).
struct Int8ColumnArgs {
    const int8_t *codes;
    const float *scales;
    const uint16_t *dy;
    int64_t ld_dy;
    int64_t n_out, n_in, m;
    int32_t steps, slices, splits, bias_rows;
    f32x4 *partial;
    float *dbias;  // or null
};

template <int OUT, int TF, bool kAligned, bool kVec>
__global__ __launch_bounds__(512) void int8_columns_kernel(Int8ColumnArgs a)
{
    __shared__ __attribute__((aligned(16))) f32x4 part[8][kFrags * TF][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (static_cast<int>(blockIdx.y) >= a.splits * a.slices) {
        const int64_t block = (static_cast<int64_t>(blockIdx.y) - a.splits * a.slices) * gridDim.x + blockIdx.x;
        const int64_t stride = static_cast<int64_t>(a.bias_rows) * gridDim.x * 512;
        for (int64_t c = block * 512 + tid; c < a.n_out; c += stride) {
            float sum = 0.0f;
#pragma unroll 8
            for (int64_t r = 0; r < a.m; ++r)
                sum = sum + Half<OUT>::widen(a.dy[r * a.ld_dy + c]);
            a.dbias[c] = sum;
        }
        return;
    }
    const int split = static_cast<uint32_t>(blockIdx.y) / static_cast<uint32_t>(a.slices);
    const int slice = blockIdx.y - split * a.slices, group = blockIdx.x;
    const int first = static_cast<int>(static_cast<uint32_t>(a.steps) * split / static_cast<uint32_t>(a.splits));
    const int last = static_cast<int>(static_cast<uint32_t>(a.steps) * (split + 1) / static_cast<uint32_t>(a.splits));
    const uintptr_t base = reinterpret_cast<uintptr_t>(a.codes);
    const uintptr_t last_dword = (base + a.n_out * a.n_in - 1) & ~uintptr_t{3};
    int64_t j0 = static_cast<int64_t>(group) * kGroup + 8 * (lane & 15);
    j0 = j0 < a.n_in ? j0 : 0;  // sums that nobody takes
    struct Step {
        u32x2 code[8];
        float scale[8];
        u32x4 x[TF];
    };
    // (without branches: rows past the end load the last one's, times 0)
    const auto load = [&](Step &s, int step) {
        const int64_t o0 = static_cast<int64_t>(step < last ? step : last - 1) * 32 + 8 * (lane >> 4);
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            const int64_t o = o0 + h < a.n_out ? o0 + h : a.n_out - 1;
            s.code[h] = load_codes8<kAligned>(base + o * a.n_in + j0, last_dword);
            const float scale = a.scales[o];
            s.scale[h] = o0 + h < a.n_out ? scale : 0.0f;
        }
#pragma unroll
        for (int t = 0; t < TF; ++t) {
            const int64_t token = (static_cast<int64_t>(slice) * TF + t) * 16 + (lane & 15);
            const bool in = token < a.m;
            const uint16_t *row = a.dy + (in ? token : 0) * a.ld_dy;
            if constexpr (kVec) {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(row + (o0 < a.n_out ? o0 : 0));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s.x[t][i] = in && o0 < a.n_out ? v[i] : 0;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t k = o0 + 2 * i;
                    const uint32_t lo = row[k < a.n_out ? k : 0], hi = row[k + 1 < a.n_out ? k + 1 : 0];
                    s.x[t][i] = !in ? 0u : (k < a.n_out ? lo : 0u) | (k + 1 < a.n_out ? hi << 16 : 0u);
                }
            }
        }
    };
    f32x4 acc[kFrags][TF];
#pragma unroll
    for (int f = 0; f < kFrags; ++f)
#pragma unroll
        for (int t = 0; t < TF; ++t)
            acc[f][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    Step now, next;
    if (first + wave < last)
        load(now, first + wave);
    for (int step = first + wave; step < last; step += 8) {
        load(next, step + 8);
        u32x4 q[8];
        decode_codes<OUT>(now.code, now.scale, q);
#pragma unroll
        for (int f = 0; f < kFrags; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                acc[f][t] = Half<OUT>::mfma(q[f], now.x[t], acc[f][t]);
        now = next;
    }
#pragma unroll
    for (int f = 0; f < kFrags; ++f)
#pragma unroll
        for (int t = 0; t < TF; ++t)
            part[wave][f * TF + t][lane] = acc[f][t];
    __syncthreads();
    f32x4 *to = a.partial + (static_cast<int64_t>(split) * gridDim.x * a.slices +
                             static_cast<int64_t>(group) * a.slices + slice) * (kFrags * TF * 64);
    for (int i = tid; i < kFrags * TF * 64; i += 512) {
        f32x4 z = part[0][i >> 6][i & 63];
#pragma unroll
        for (int w = 1; w < 8; ++w)
            z = z + part[w][i >> 6][i & 63];
        to[i] = z;
    }
}

// ---------------------------------------------------------------------------
// few rows: the weight decoded straight into operand registers
// ---------------------------------------------------------------------------
struct RowsArgs {
    Weight w[2];
    int64_t n_out, n_in;        // the weight's shape (both weights)
    int64_t n_elems;            // n_out * n_in
    int32_t log2_block;
    int32_t row_blocks;
    int32_t whole, rest;        // tiles: those over all of k, those in out.splits parts
    ProductArgs out;            // x and the epilogue's matrices
};

// Output row r of the linear call's columns n0 .. n0 + 3.
template <int OUT>
__device__ __forceinline__ void finish_linear4(const ProductArgs &a, int64_t row, int64_t n0,
                                               f32x4 acc)
{
    const int64_t left = a.n - n0;
    if (row >= a.m || left <= 0)
        return;
    const int valid = left < 4 ? static_cast<int>(left) : 4;
    const bool vec = a.vec && valid == 4;
    float z[4] = {acc[0], acc[1], acc[2], acc[3]};
    if (a.bias) {
        float b[4];
        load_values<OUT, 4>(a.bias + n0, vec, valid, b);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            z[j] = z[j] + b[j];
    }
    if (a.pre[0])
        store_values<OUT, 4>(a.pre[0] + row * a.ld_pre + n0, vec, valid, z);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        z[j] = act_f32(a.act, z[j]);
    if (a.residual) {
        float r[4];
        load_values<OUT, 4>(a.residual + row * a.ld_residual + n0, vec, valid, r);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            z[j] = z[j] + r[j];
    }
    store_values<OUT, 4>(a.y + row * a.ld_y + n0, vec, valid, z);
}

// Weight rows of whole dwords whose length is no multiple of 32: m <= 16 TF
// rows of x against the 4-bit weight, which is read once and never written
// out.  A lane loads 16 packed bytes (32 k) of one weight row, decodes each
// dword into the matrix instruction's operand registers, and multiplies it
// with the x fragments of the same k; its 32 k may straddle two blocks, and
// each dword picks one.  A workgroup takes R fragments of 16 weight rows
// (gated: R / 2 of each weight, the same columns) at a time; its waves split
// the chunks of 128 k, and the partial sums meet in LDS.  Workgroups walk the
// row blocks; the next chunk's loads, also those of the next row block, are
// issued before the current chunk is decoded.  Bound by the latency of a few
// chunks and of the sums' meeting at small sizes (1000 x 2376 with 37 rows: 15
// us), by the decode's vector instructions at large ones (4096 x 11000 with 64
// rows: 58 us a call).
template <int OUT, bool kGated, int R, int TF, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void ragged_rows_kernel(RowsArgs a)
{
    constexpr int kW = kGated ? 2 : 1;
    constexpr int kPer = R / kW;                 // fragments per weight and row wave
    constexpr int WK = WAVES;                    // waves along k
    constexpr int kBlockRows = 16 * kPer;        // weight rows per row block
    constexpr int kSpan = 128;                   // k per chunk
    constexpr int kBounds = 2;                   // blocks a lane's 32 k may touch
    __shared__ __attribute__((aligned(1024))) uint8_t table[kPairTableBytes + 256];
    __shared__ float scb[kW][256], cb4[kW][16];
    __shared__ __attribute__((aligned(16))) f32x4 partial[WAVES][R][64];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave;
    const int r = lane & 15, g = lane >> 4;
    const int lb = a.log2_block;
    const uint32_t n_in = static_cast<uint32_t>(a.n_in);
    const int chunks = static_cast<int>((n_in + kSpan - 1) / kSpan);

    struct Loads {
        u32x4 packed[R];
        uint32_t code[R][kBounds];
        float absmax[R][kBounds];
    };
    u32x4 x[4][TF];  // the current chunk's; each step's is reloaded once used
    // buffers of the row block whose chunks are being loaded
    u32x4 rs_packed[kW], rs_code[kW], rs_absmax[kW];
    uint32_t block_phase = 0, group_phase = 0;  // of the row block's first element
    auto enter = [&](int64_t rb) {
        const int64_t e0 = rb * kBlockRows * a.n_in;
        const int64_t b0 = e0 >> lb;
        block_phase = static_cast<uint32_t>(e0 - (b0 << lb));
        group_phase = static_cast<uint32_t>(b0 & 255);
        const int64_t blocks = (a.n_elems + (int64_t{1} << lb) - 1) >> lb;
        const int64_t most = 0x7FFFFFF0;
        const int64_t pb = ((a.n_elems + 1) >> 1) - (e0 >> 1), cb = blocks - b0,
                      gb = (((blocks + 255) >> 8) - (b0 >> 8)) * 4;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            rs_packed[w] = make_rsrc(a.w[w].packed + (e0 >> 1), static_cast<uint32_t>(pb < most ? pb : most));
            rs_code[w] = make_rsrc(a.w[w].scale_codes + b0, static_cast<uint32_t>(cb < most ? cb : most));
            rs_absmax[w] = make_rsrc(a.w[w].nested_absmax + (b0 >> 8), static_cast<uint32_t>(gb < most ? gb : most));
        }
    };
    auto rsrc = [](u32x4 q) {
        return __builtin_amdgcn_make_buffer_rsrc(
            reinterpret_cast<void *>((static_cast<uint64_t>(q[1]) << 32) | q[0]), 0,
            static_cast<int32_t>(q[2]), kRawBufferWord3);
    };
    const u32x4 rs_x = make_rsrc(a.out.x[0],
                                 static_cast<uint32_t>(((a.out.m - 1) * a.out.ld_x + a.out.k) * 2));
    uint32_t x_row[TF];
#pragma unroll
    for (int t = 0; t < TF; ++t)
        x_row[t] = t * 16 + r < a.out.m
                       ? static_cast<uint32_t>((t * 16 + r) * a.out.ld_x * 2)
                       : 0x80000000u;
    auto load = [&](Loads &l, int c) {
        const uint32_t k = c * kSpan + 32 * g;
#pragma unroll
        for (int f = 0; f < R; ++f) {
            const int w = kGated ? f / kPer : 0;
            const uint32_t row = (kGated ? f % kPer : f) * 16 + r;
            const uint32_t e = row * n_in + k;
            l.packed[f] = __builtin_amdgcn_raw_buffer_load_b128(
                rsrc(rs_packed[w]), e >> 1, 0, 0);
#pragma unroll
            for (int h = 0; h < kBounds; ++h) {
                const uint32_t b = (block_phase + e + (h ? 31 : 0)) >> lb;
                l.code[f][h] = __builtin_amdgcn_raw_buffer_load_b8(rsrc(rs_code[w]), b, 0, 0);
                l.absmax[f][h] = __builtin_bit_cast(
                    float, __builtin_amdgcn_raw_buffer_load_b32(rsrc(rs_absmax[w]),
                                                                ((group_phase + b) >> 8) * 4, 0, 0));
            }
        }
    };
    auto load_x = [&](int c, int st) {
        const uint32_t k = c * kSpan + 32 * g + 8 * st;
#pragma unroll
        for (int t = 0; t < TF; ++t)
            x[st][t] = __builtin_amdgcn_raw_buffer_load_b128(
                rsrc(rs_x), k < static_cast<uint32_t>(a.out.k) ? x_row[t] + k * 2 : 0x80000000u, 0, 0);
    };

    const Codebooks codebooks = fetch_codebooks<kW>(a.w);
    Loads cur;
    int64_t load_rb = blockIdx.x;
    int load_c = wk;
    const bool any = wk < chunks;  // this wave has chunks at all
    if (any) {
        enter(load_rb);
        load(cur, load_c);
#pragma unroll
        for (int st = 0; st < 4; ++st)
            load_x(load_c, st);
    }

    // the lookup tables, while the first loads are in flight
    fill_tables<kW, 1>(codebooks, table, scb, cb4);

    const uint32_t lane_byte = kGated ? (lane & 15) * 16 : (lane & 31) * 8;
    for (int64_t rb = blockIdx.x; rb < a.row_blocks; rb += gridDim.x) {
        f32x4 acc[R][TF];
#pragma unroll
        for (int f = 0; f < R; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                acc[f][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const uint32_t phase = static_cast<uint32_t>((rb * kBlockRows * a.n_in) & ((1 << lb) - 1));
        for (int c = wk; c < chunks; c += WK) {
            // the following chunk, of this row block or the next one
            load_c += WK;
            if (load_c >= chunks) {
                load_c = wk;
                load_rb += gridDim.x;
                if (load_rb < a.row_blocks)
                    enter(load_rb);
            }
            Loads next = cur;
            if (load_rb < a.row_blocks)
                load(next, load_c);
            float s[R][kBounds];
#pragma unroll
            for (int f = 0; f < R; ++f)
#pragma unroll
                for (int h = 0; h < kBounds; ++h)
                    s[f][h] = block_scale(scb[kGated ? f / kPer : 0][cur.code[f][h]], cur.absmax[f][h],
                                          a.w[kGated ? f / kPer : 0].offset);
            const uint32_t k = c * kSpan + 32 * g;
#pragma unroll
            for (int st = 0; st < 4; ++st) {
#pragma unroll
                for (int f = 0; f < R; ++f) {
                    float sc = s[f][0];
                    const uint32_t row = (kGated ? f % kPer : f) * 16 + r;
                    const uint32_t e = phase + row * n_in + k;
                    if (((e + 8 * st) >> lb) != (e >> lb))
                        sc = s[f][kBounds - 1];
                    u32x4 wf = decode_dword<OUT>(cur.packed[f][st], sc,
                                                 table + (kGated ? f / kPer : 0) * 8, lane_byte);
                    if (k + 8 * st >= n_in)  // beyond the row there is no value at all
                        wf = u32x4{0, 0, 0, 0};
#pragma unroll
                    for (int t = 0; t < TF; ++t)
                        acc[f][t] = Half<OUT>::mfma(wf, x[st][t], acc[f][t]);
                }
                load_x(load_c, st);  // after the last row block: a chunk again, unused
            }
            cur = next;
        }
        // the k-waves' partial sums, 16 rows of x at a time
#pragma unroll
        for (int t = 0; t < TF; ++t) {
            lds_barrier();
#pragma unroll
            for (int f = 0; f < R; ++f)
                partial[wave][f][lane] = acc[f][t];
            lds_barrier();
            for (int i = tid; i < kPer * 64; i += 64 * WAVES) {
                const int ln = i & 63, f = i >> 6;
                f32x4 sum = partial[0][f][ln];
                for (int q = 1; q < WK; ++q)
                    sum = sum + partial[q][f][ln];
                const int64_t n0 = rb * kBlockRows + f * 16 + (ln >> 4) * 4;
                const int64_t row = t * 16 + (ln & 15);
                if constexpr (kGated) {
                    f32x4 up = partial[0][f + kPer][ln];
                    for (int q = 1; q < WK; ++q)
                        up = up + partial[q][f + kPer][ln];
                    float gv[4] = {sum[0], sum[1], sum[2], sum[3]}, uv[4] = {up[0], up[1], up[2], up[3]};
                    finish_gated<OUT>(a.out, row, n0, gv, uv);
                } else {
                    finish_linear4<OUT>(a.out, row, n0, sum);
                }
            }
        }
    }
}

// Forward decode of weights whose rows are whole 16-byte pieces (n_in % 32 ==
// 0): a wave takes the 16 rows of one fragment f and 256 k.  A load takes 64
// neighbouring bytes of each row (lane 4 r + p: 32 k of row r), the decoded 16
// byte units change places in LDS, and every store is a whole fragment.  Each
// scale is looked up once per 32 k.  Workgroups walk the (group, 256 k) items
// with the next item's loads in flight.  Bound by memory: 0.5 B read, 2 B
// written per element; 2 x 28672 x 8192 in 226 us, 5.2 TB/s.
constexpr int kDecodeWaves = 16;
constexpr int kUnitLd = 1024 + 32;  // bytes between a wave's fragments in LDS: 8 neighbouring
                                    // lanes' writes then meet 8 different bank groups

template <int OUT, bool kTwo>
__global__ __launch_bounds__(64 * kDecodeWaves) void weight_row_fragments_kernel(FragmentArgs a,
                                                                                int32_t spans,
                                                                                int32_t items)
{
    constexpr int kW = kTwo ? 2 : 1;
    __shared__ __attribute__((aligned(1024))) uint8_t table[kPairTableBytes + 256];
    __shared__ float scb[kW][256], cb4[kW][16];
    __shared__ __attribute__((aligned(16))) uint8_t units[kDecodeWaves][4 * kUnitLd];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int f = wave & 7, which = kTwo ? f >> 2 : 0;
    const Weight w = a.w[which];
    const int r = lane >> 2, p = lane & 3;
    const int lb = a.log2_block;
    const int64_t n_in = a.n_in;
    const int row_of = kTwo ? 4 * r + (f & 3) : 8 * r + f;

    struct Loads {
        u32x4 packed[2];
        uint32_t code[2];
        float absmax[2];
    };
    // a workgroup's two halves of 8 waves take neighbouring items
    auto load = [&](Loads &l, int item) {
        const int group = item / spans, span = item - group * spans;
        const int64_t o = static_cast<int64_t>(a.group0 + group) * (kTwo ? 64 : kGroup) + row_of;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t k = static_cast<int64_t>(span) * 256 + h * 128 + 32 * p;
            l.packed[h] = u32x4{0, 0, 0, 0};
            l.code[h] = 0;
            l.absmax[h] = 0.0f;
            if (o < a.n_out && k < n_in) {
                const int64_t e = o * n_in + k;
                const int64_t b = e >> lb;
                typedef uint32_t Dwords __attribute__((ext_vector_type(4), aligned(4)));
                l.packed[h] = *reinterpret_cast<const Dwords *>(w.packed + (e >> 1));
                l.code[h] = w.scale_codes[b];
                l.absmax[h] = w.nested_absmax[b >> kNestedLog2];
            }
        }
    };
    const Codebooks codebooks = fetch_codebooks<kW>(a.w);
    int item = blockIdx.x * 2 + (wave >> 3);
    const int step = gridDim.x * 2;
    Loads cur;
    if (item < items)
        load(cur, item);
    fill_tables<kW, 1>(codebooks, table, scb, cb4);

    const uint32_t lane_byte = kTwo ? (lane & 15) * 16 + which * 8 : (lane & 31) * 8;
    const int chunks = a.chunks;
    for (; item < items; item += step) {
        Loads next = cur;
        if (item + step < items)
            load(next, item + step);
        const int group = item / spans, span = item - group * spans;
        const int64_t o = static_cast<int64_t>(a.group0 + group) * (kTwo ? 64 : kGroup) + row_of;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t k = static_cast<int64_t>(span) * 256 + h * 128 + 32 * p;
            const bool beyond = o >= a.n_out || k >= n_in;  // zeros, whatever the codebooks hold
            const uint32_t from = beyond ? (lane_byte & 255) | kPairTableBytes : lane_byte;
            float s = block_scale(scb[which][cur.code[h]], cur.absmax[h], w.offset);
            s = beyond ? 0.0f : s;
            uint8_t *to = units[wave] + p * kUnitLd + r * 16;
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<u32x4 *>(to + g * 256) =
                    decode_dword<OUT>(cur.packed[h][g], s, table, from);
            // only this wave uses these units: its LDS operations are in order,
            // the compiler must not move the reads above the writes
            __asm__ volatile("" ::: "memory");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int chunk = span * 4 + h * 2 + (q >> 1);
                const u32x4 v = *reinterpret_cast<const u32x4 *>(units[wave] + q * kUnitLd + lane * 16);
                if (chunk < chunks)
                    *reinterpret_cast<u32x4 *>(a.out + (static_cast<int64_t>(group) * chunks + chunk) * (kUnitBytes / 2) +
                                               ((q & 1) * kFrags + f) * (kFragBytes / 2) + lane * 8) = v;
            }
            __asm__ volatile("" ::: "memory");
            __builtin_amdgcn_wave_barrier();
        }
        cur = next;
    }
}

// ---------------------------------------------------------------------------
// one or two rows of x: weight rows read in straight lines
// ---------------------------------------------------------------------------
// The products are dot products of whole weight rows, and the 4-bit weight is
// all the memory traffic, so every load of it is 1 KiB of one row: lane l takes
// the 16 bytes (32 k) l of a chunk of 2048 k.  The matrix instruction still
// does the sum: with operand lane l holding the same 8 k of the weight row (A)
// and of x (B), D[i][i] is the sum over the pieces i, 16 + i, 32 + i, 48 + i,
// and the diagonal's 16 values add up to the chunk's dot product.  15 of 16
// results are unused; the instruction is still cheaper than widening the
// rounded weight for the vector unit (4 vector instructions per packed byte
// against 10), and x stays in registers: a wave keeps one chunk of k and walks
// rows.  The waves' partial sums meet in LDS, in a fixed order.  Bound by the
// reading of the weight where it is long (gated 28672 x 8192, one token: 242 MB
// in 60 us, 4.07 TB/s), by the lookup tables' filling and the launch where it is
// short (4096 x 4096: 7.6 us).
struct TokenArgs {
    Weight w[2];
    int64_t n_in;
    int32_t log2_block;
    int32_t chunks;             // of 2048 k
    int32_t wk;                 // waves along k
    int32_t rows_per, rows_extra;  // weight rows of a workgroup; the first ones take one more
    int32_t batch;              // weight rows per pass through LDS
    ProductArgs out;
};

constexpr int kTokenSpan = 2048;   // k per wave and chunk
constexpr int kTokenDepth = 3;     // pairs of row chunks in flight per wave
constexpr int kTokenMaxChunks = 16;

template <int OUT>
__device__ __forceinline__ void finish_one(const ProductArgs &a, int64_t row, int64_t n, float z)
{
    if (a.bias)
        z = z + Half<OUT>::widen(a.bias[n]);
    if (a.pre[0])
        a.pre[0][row * a.ld_pre + n] = static_cast<uint16_t>(Half<OUT>::pack2(z, 0.0f));
    z = act_f32(a.act, z);
    if (a.residual)
        z = z + Half<OUT>::widen(a.residual[row * a.ld_residual + n]);
    a.y[row * a.ld_y + n] = static_cast<uint16_t>(Half<OUT>::pack2(z, 0.0f));
}

// Floats of partial sums: what the tables leave of the LDS.
template <bool kGated>
constexpr int kTokenPartials = kGated ? 6144 : 12288;

template <int OUT, bool kGated, int M, int WAVES, int DEPTH>
__global__ __launch_bounds__(64 * WAVES) void token_rows_kernel(TokenArgs a)
{
    constexpr int kW = kGated ? 2 : 1;
    constexpr int kRows = kGated ? 1 : 2;  // weight rows of a pair of row chunks
    __shared__ __attribute__((aligned(1024))) uint8_t table[kW * kPairTableBytes + 256];
    __shared__ float scb[kW][256], cb4[kW][16];
    __shared__ __attribute__((aligned(16))) float partial[2][kTokenPartials<kGated> / 2];
    __shared__ float unused[64];

    const int tid = threadIdx.x;
    const int threads = blockDim.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int WK = a.wk, WR = (threads >> 6) / WK;
    const int wk = wave % WK, wr = wave / WK;
    const int lb = a.log2_block;
    const uint32_t n_in = static_cast<uint32_t>(a.n_in);
    const int chunks = a.chunks;
    const int passes = (chunks + WK - 1) / WK;

    // this workgroup's weight rows
    const int block = blockIdx.x;
    const int row_first = block * a.rows_per + (block < a.rows_extra ? block : a.rows_extra);
    const int row_last = row_first + a.rows_per + (block < a.rows_extra ? 1 : 0);

    struct Row {
        u32x4 packed;
        uint32_t code;
        float absmax;
    };
    Row ring[DEPTH][2];  // gated: a row of each weight; else two rows
    u32x4 x[M][4];
    uint32_t k_lane = 0, packed_off = 0;
    auto load_one = [&](Row &to, int w, int row) {
        row = row < row_last ? row : row_last - 1;  // loaded again, unused
        const int64_t e0 = row * a.n_in;
        const int64_t b0 = e0 >> lb;
        const uint32_t phase = static_cast<uint32_t>(e0) & ((1u << lb) - 1);
        const uint32_t b = (phase + k_lane) >> lb;
        const uint32_t gr = ((static_cast<uint32_t>(b0) & 255) + b) >> 8;
        const auto rsrc = [](const void *p) {
            return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, 0x7FFFFFFF,
                                                     kRawBufferWord3);
        };
        // lanes beyond the row: an offset past every buffer, zeros
        const uint32_t past = packed_off & 0x80000000u;
        to.packed = __builtin_amdgcn_raw_buffer_load_b128(rsrc(a.w[w].packed + (e0 >> 1)), packed_off,
                                                          0, 0);
        to.code = __builtin_amdgcn_raw_buffer_load_b8(rsrc(a.w[w].scale_codes + b0), b | past, 0, 0);
        to.absmax = __builtin_bit_cast(
            float, __builtin_amdgcn_raw_buffer_load_b32(rsrc(a.w[w].nested_absmax + (b0 >> 8)),
                                                        (gr * 4) | past, 0, 0));
    };
    // pair i of this wave's rows from `row0` on
    auto load = [&](Row (&to)[2], int row0, int i) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            load_one(to[j], kGated ? j : 0, row0 + (i * kRows + (kGated ? 0 : j)) * WR + wr);
    };
    const auto rs_x = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t *>(a.out.x[0]), 0,
        static_cast<int32_t>(((a.out.m - 1) * a.out.ld_x + a.out.k) * 2), kRawBufferWord3);
    auto enter_chunk = [&](int chunk) {
        k_lane = chunk * kTokenSpan + 32 * lane;
        packed_off = k_lane < n_in ? k_lane / 2 : 0x80000000u;
#pragma unroll
        for (int t = 0; t < M; ++t)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                // rows and k beyond x lie past the buffer: zeros
                const uint32_t at = static_cast<uint32_t>(t * a.out.ld_x + k_lane + 8 * s) * 2;
                x[t][s] = __builtin_amdgcn_raw_buffer_load_b128(
                    rs_x, k_lane < n_in && t < a.out.m ? at : 0x80000000u, 0, 0);
            }
    };

    const Codebooks codebooks = fetch_codebooks<kW>(a.w);
    // the first rows' loads go out before the tables are built
    enter_chunk(wk);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        load(ring[d], row_first, d);
    fill_tables<kW, kW>(codebooks, table, scb, cb4);

    const uint32_t lane_byte = (lane & 31) * 8;
    const int G = lane >> 4, c = lane & 15;
    const bool writer = G == (c >> 2) && (c & 3) == 0;
    int parity = 0;
    for (int b0 = row_first; b0 < row_last; b0 += a.batch, parity ^= 1) {
        const int rows = row_last - b0 < a.batch ? row_last - b0 : a.batch;
        float *part = partial[parity];
        for (int pass = 0; pass < passes; ++pass) {
            const int chunk = wk + pass * WK;
            if (chunk >= chunks)
                break;
            if (passes > 1 && (pass > 0 || b0 != row_first)) {  // else the ring is filled
                enter_chunk(chunk);
#pragma unroll
                for (int d = 0; d < DEPTH; ++d)
                    load(ring[d], b0, d);
            }
            // a lane beyond the row (its loads gave zeros) reads the row of
            // zeros behind the tables, times 0
            const bool beyond = k_lane >= n_in;
            uint32_t from[kW];
#pragma unroll
            for (int w = 0; w < kW; ++w)
                from[w] = lane_byte + (beyond ? kW * kPairTableBytes : w * kPairTableBytes);
            for (int i0 = 0; i0 * kRows * WR + wr < rows; i0 += DEPTH) {
#pragma unroll
                for (int d = 0; d < DEPTH; ++d) {
                    const int i = i0 + d;
                    // a turn loads as often past the last row: were the number
                    // of loads in flight not known, every turn would begin by
                    // waiting for all of them
                    if (i * kRows * WR + wr < rows) {
                        float s[2];
                        f32x4 acc[2][M];
                        Pairs now[2], next[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int w = kGated ? j : 0;
                            now[j] = lookup_dword(ring[d][j].packed[0], table, from[w]);
                            s[j] = block_scale(scb[w][ring[d][j].code], ring[d][j].absmax, a.w[w].offset);
                            s[j] = beyond ? 0.0f : s[j];
                        }
#pragma unroll
                        for (int st = 0; st < 4; ++st) {
                            if (st < 3) {
#pragma unroll
                                for (int j = 0; j < 2; ++j)
                                    next[j] = lookup_dword(ring[d][j].packed[st + 1], table, from[kGated ? j : 0]);
                            }
                            keep_order();
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const u32x4 wf = scaled_dword<OUT>(now[j], s[j]);
#pragma unroll
                                for (int t = 0; t < M; ++t)
                                    acc[j][t] = Half<OUT>::mfma(wf, x[t][st],
                                                                st == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f}
                                                                        : acc[j][t]);
                                now[j] = next[j];
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int r = (i * kRows + (kGated ? 0 : j)) * WR + wr;
#pragma unroll
                            for (int t = 0; t < M; ++t) {
                                // the diagonal value of this lane's column, its quad's sum
                                const f32x4 q = acc[j][t];
                                const float lo = (c & 1) ? q[1] : q[0], hi = (c & 1) ? q[3] : q[2];
                                float v = (c & 2) ? hi : lo;
                                v = v + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, true));
                                v = v + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, true));
                                // no branch: other lanes and rows past the end
                                // write where nothing is read
                                float *to = part + (((r * M + t) * kW + (kGated ? j : 0)) * chunks + chunk) * 4 + G;
                                *(writer && r < rows ? to : &unused[lane]) = v;
                            }
                        }
                    }
                    // batches are whole rings long: with one pass the ring
                    // runs on into the next batch
                    load(ring[d], b0, i + DEPTH);
                }
            }
        }
        lds_barrier();
        for (int i = tid; i < rows * M; i += threads) {
            const int r = i / M, t = i % M;
            if (t >= a.out.m)
                continue;
            float z[kW];
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const float *from = part + ((r * M + t) * kW + w) * chunks * 4;
                float sum = 0.0f;
                for (int q = 0; q < chunks; ++q) {
                    const f32x4 v = *reinterpret_cast<const f32x4 *>(from + 4 * q);
                    sum = sum + ((v[0] + v[1]) + (v[2] + v[3]));
                }
                z[w] = sum;
            }
            const int64_t n = b0 + r;
            if constexpr (kGated) {
                if (a.out.pre[0]) {
                    a.out.pre[0][t * a.out.ld_pre + n] = static_cast<uint16_t>(Half<OUT>::pack2(z[0], 0.0f));
                    a.out.pre[1][t * a.out.ld_pre + n] = static_cast<uint16_t>(Half<OUT>::pack2(z[1], 0.0f));
                }
                a.out.y[t * a.out.ld_y + n] =
                    static_cast<uint16_t>(Half<OUT>::pack2(act_f32(a.out.act, z[0]) * z[1], 0.0f));
            } else {
                finish_one<OUT>(a.out, t, n, z[0]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// 3 to 64 rows of x: weight rows read 64 bytes at a time, transposed in registers
// ---------------------------------------------------------------------------
// x in operand fragments: fragment (chunk of 512 k, step, 16 rows of x) is 1
// KiB in lane order; lane (r, g) of step 4 j + s holds row r's k 512 c + 128 g
// + 32 j + 8 s .. + 7.  Rows and k beyond x are zeros.  More than 128 rows are
// cut into slices of 128 (blockIdx.y), one after the other.
__global__ __launch_bounds__(kThreads) void x_fragments_zero_fill(const uint16_t *x, int64_t ld_x,
                                                                  int64_t m, int64_t k, int32_t tf,
                                                                  int32_t frags, bool aligned,
                                                                  uint16_t *out)
{
    const int lane = threadIdx.x & 63;
    const int fr = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    if (fr >= frags)
        return;
    const int step = fr / tf, t = fr - step * tf;
    const int64_t row = static_cast<int64_t>(blockIdx.y) * (16 * tf) + t * 16 + (lane & 15);
    const int64_t k0 = static_cast<int64_t>(step >> 4) * 512 + 128 * (lane >> 4) + 8 * (step & 15);
    u32x4 q = {0, 0, 0, 0};
    if (row < m && k0 < k) {
        const uint16_t *from = x + row * ld_x + k0;
        if (aligned) {
            q = *reinterpret_cast<const u32x4 *>(from);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k0 + j < k)
                    q[j / 2] |= static_cast<uint32_t>(from[j]) << (16 * (j & 1));
        }
    }
    const int64_t at = static_cast<int64_t>(blockIdx.y) * frags + fr;
    *reinterpret_cast<u32x4 *>(out + (at * 64 + lane) * 8) = q;
}

// 16 TF rows of x against the 4-bit weight, which is read once and never
// written out.  A wave takes two fragments of 16 weight rows (gated: one of
// each weight, the same columns) and chunks of 512 k.  The matrix instruction
// wants neighbouring lanes in different weight rows, memory wants them side by
// side (a load whose neighbouring lanes lie in 16 rows took 64 accesses of the
// vector cache, this one 16): so a load takes 256 bytes of 4 rows, a quad of
// lanes on 64 of them, and 4 such loads are transposed between the lanes of
// each quad; the scales are looked up four lanes to a row too, and handed over.
// Waves along k (wk of them) meet in LDS, in a fixed order.  The
// next chunk's loads, also those of the next row block, are in flight while a
// chunk is multiplied; each x fragment is reloaded kAhead steps ahead.
// S: blocks looked up per lane and 128 k (2: blocks of 64 k or more and n_in
// % 64 == 0; else 4).
// Bound by the lookups, the decode's vector instructions and the x loads, which
// two waves per SIMD overlap in part: about 9 us until the tables are filled and
// the last sums have met, then per 33.5 M weight elements 4.8 us with 16 rows
// of x and 7 to 9 with 64 (gated 28672 x 8192: 80 and 135 us).
template <int OUT, bool kGated, int TF, int S>
__global__ __launch_bounds__(512) void batch_rows_kernel(RowsArgs a, const uint16_t *x_frags, int wk_waves)
{
    constexpr int R = 2, kW = kGated ? 2 : 1;
    constexpr int kPer = R / kW;
    constexpr int kSpan = 512;
    __shared__ __attribute__((aligned(1024))) uint8_t table[kPairTableBytes + 256];
    __shared__ float scb[kW][256], cb4[kW][16];
    __shared__ __attribute__((aligned(16))) f32x4 partial[8][R * TF][64];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int WK = wk_waves, WR = 8 / WK;
    const int wk = wave % WK, wr = wave / WK;
    const int g = lane >> 4;
    const int block_rows = 16 * kPer * WR;
    const int lb = a.log2_block;
    const uint32_t n_in = static_cast<uint32_t>(a.n_in);
    const int chunks = static_cast<int>((n_in + kSpan - 1) / kSpan);
    const bool odd = lane & 1, high = lane & 2;

    struct Loads {
        u32x4 packed[R][4];
        uint32_t code[R][S];
        float absmax[R][S];
    };
    const auto rsrc_of = [](const void *p, int64_t bytes) {
        return __builtin_amdgcn_make_buffer_rsrc(
            const_cast<void *>(p), 0, static_cast<int32_t>(bytes < 0x7FFFFFF0 ? bytes : 0x7FFFFFF0),
            kRawBufferWord3);
    };
    const uint32_t k_load = 32 * (((lane >> 4) << 2) | (lane & 3));  // of the loaded piece
    const uint32_t row_load = 4 * ((lane >> 2) & 3);
    const int64_t blocks = (a.n_elems + (int64_t{1} << lb) - 1) >> lb;
    auto load = [&](Loads &l, int64_t rb, int c) {
        const int64_t row0 = rb * block_rows + wr * (16 * kPer);
        const int64_t e0 = row0 * a.n_in;
        const int64_t b0 = e0 >> lb;
        const uint32_t phase = static_cast<uint32_t>(e0) & ((1u << lb) - 1);
        const uint32_t group_phase = static_cast<uint32_t>(b0) & 255;
        const int64_t packed_left = ((a.n_elems + 1) >> 1) - (e0 >> 1);
        if (packed_left <= 0) {  // row waves past the last row
#pragma unroll
            for (int f = 0; f < R; ++f) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    l.packed[f][q] = u32x4{0, 0, 0, 0};
#pragma unroll
                for (int h = 0; h < S; ++h) {
                    l.code[f][h] = 0;
                    l.absmax[f][h] = 0.0f;
                }
            }
            return;
        }
        const uint32_t k = c * kSpan + k_load;
        const uint32_t past = k < n_in ? 0u : 0x80000000u;
#pragma unroll
        for (int f = 0; f < R; ++f) {
            const int w = kGated ? f : 0;
            const uint32_t frag_row = kGated ? 0 : f * 16;
            const auto rp = rsrc_of(a.w[w].packed + (e0 >> 1), packed_left);
            const auto rc = rsrc_of(a.w[w].scale_codes + b0, blocks - b0);
            const auto rm = rsrc_of(a.w[w].nested_absmax + (b0 >> 8), (((blocks + 255) >> 8) - (b0 >> 8)) * 4);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                l.packed[f][q] = __builtin_amdgcn_raw_buffer_load_b128(
                    rp, (((frag_row + row_load + q) * n_in + k) >> 1) | past, 0, 0);
#pragma unroll
            for (int h = 0; h < S; ++h) {
                // of row lane / 4, the lane's quarter of the chunk
                const uint32_t e = (frag_row + (lane >> 2)) * n_in + c * kSpan + 128 * (lane & 3) + h * (128 / S);
                const uint32_t b = (phase + e) >> lb;
                l.code[f][h] = __builtin_amdgcn_raw_buffer_load_b8(rc, b, 0, 0);
                l.absmax[f][h] = __builtin_bit_cast(
                    float, __builtin_amdgcn_raw_buffer_load_b32(rm, ((group_phase + b) >> 8) * 4, 0, 0));
            }
        }
    };
    constexpr int kAhead = TF == 4 && S == 4 ? 2 : 4;  // steps; what the registers hold
    u32x4 x[kAhead][TF];
    auto load_x = [&](int c, int step) {  // step in 0 .. 15 of chunk c
#pragma unroll
        for (int t = 0; t < TF; ++t)
            x[step % kAhead][t] = *reinterpret_cast<const u32x4 *>(
                x_frags + ((static_cast<int64_t>(c) * 16 + step) * TF + t) * 512 + lane * 8);
    };

    const Codebooks codebooks = fetch_codebooks<kW>(a.w);
    Loads cur;
    int64_t load_rb = blockIdx.x;
    int load_c = wk;  // wk < chunks: the host takes no more waves along k than chunks
    load(cur, load_rb, load_c);
#pragma unroll
    for (int st = 0; st < kAhead; ++st)
        load_x(load_c, st);

    // the lookup tables, while the first loads are in flight
    fill_tables<kW, 1>(codebooks, table, scb, cb4);

    const uint32_t lane_byte = kGated ? (lane & 15) * 16 : (lane & 31) * 8;
    for (int64_t rb = blockIdx.x; rb < a.row_blocks; rb += gridDim.x) {
        f32x4 acc[R][TF];
#pragma unroll
        for (int f = 0; f < R; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                acc[f][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int c = wk; c < chunks; c += WK) {
            // the following chunk, of this row block or the next one
            load_c += WK;
            if (load_c >= chunks) {
                load_c = wk;
                load_rb += gridDim.x;
            }
            Loads next;
            if (load_rb < a.row_blocks)
                load(next, load_rb, load_c);
            else
                next = cur;
            float s[R][S];
#pragma unroll
            for (int f = 0; f < R; ++f) {
#pragma unroll
                for (int h = 0; h < S; ++h) {
                    const float q = block_scale(scb[kGated ? f : 0][cur.code[f][h]], cur.absmax[f][h],
                                                a.w[kGated ? f : 0].offset);
                    // lane 16 g + r multiplies quarter g of row r
                    s[f][h] = __builtin_bit_cast(
                        float, __builtin_amdgcn_ds_bpermute((4 * (lane & 15) + g) * 4, __builtin_bit_cast(int, q)));
                }
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    uint32_t v[4] = {cur.packed[f][0][d], cur.packed[f][1][d], cur.packed[f][2][d],
                                     cur.packed[f][3][d]};
                    transpose_quads(v, odd, high);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        cur.packed[f][j][d] = v[j];
                }
            }
            const uint32_t k = c * kSpan + 128 * g;
            uint32_t from[4];
            float sj[4][R];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // a piece beyond the row (its load gave zeros) reads the row
                // of zeros behind the table, times 0
                const bool beyond = k + 32 * j >= n_in;
                from[j] = beyond ? lane_byte | kPairTableBytes : lane_byte;
#pragma unroll
                for (int f = 0; f < R; ++f)
                    sj[j][f] = beyond ? 0.0f : s[f][j * S / 4];
            }
            Pairs now[R], then[R];
#pragma unroll
            for (int f = 0; f < R; ++f)
                now[f] = lookup_dword(cur.packed[f][0][0], table + (kGated ? f : 0) * 8, from[0]);
#pragma unroll
            for (int st = 0; st < 16; ++st) {
                // with 64 rows of x the products cover the lookups, and there
                // are no registers to spare
                const int ahead = TF < 4 ? st + 1 : st;
                if (ahead < 16) {
#pragma unroll
                    for (int f = 0; f < R; ++f)
                        then[f] = lookup_dword(cur.packed[f][ahead / 4][ahead % 4],
                                               table + (kGated ? f : 0) * 8, from[ahead / 4]);
                }
                if constexpr (TF < 4)
                    keep_order();
#pragma unroll
                for (int f = 0; f < R; ++f) {
                    const u32x4 wf = scaled_dword<OUT>(TF < 4 ? now[f] : then[f], sj[st / 4][f]);
#pragma unroll
                    for (int t = 0; t < TF; ++t)
                        acc[f][t] = Half<OUT>::mfma(wf, x[st % kAhead][t], acc[f][t]);
                    now[f] = then[f];
                }
                if (st + kAhead < 16)
                    load_x(c, st + kAhead);
                else
                    load_x(load_c, st + kAhead - 16);  // after the last row block: unused
            }
            cur = next;
        }
        lds_barrier();  // the last row block's sums are read
#pragma unroll
        for (int f = 0; f < R; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                partial[wave][f * TF + t][lane] = acc[f][t];
        lds_barrier();
        for (int i = tid; i < WR * kPer * TF * 64; i += 512) {
            const int ln = i & 63, ft = (i >> 6) % (kPer * TF), row_wave = (i >> 6) / (kPer * TF);
            const int f = ft / TF, t = ft - f * TF;
            f32x4 sum = partial[row_wave * WK][f * TF + t][ln];
            for (int q = 1; q < WK; ++q)
                sum = sum + partial[row_wave * WK + q][f * TF + t][ln];
            const int64_t n0 = rb * block_rows + row_wave * (16 * kPer) + f * 16 + (ln >> 4) * 4;
            const int64_t row = t * 16 + (ln & 15);
            if constexpr (kGated) {
                f32x4 up = partial[row_wave * WK][TF + t][ln];
                for (int q = 1; q < WK; ++q)
                    up = up + partial[row_wave * WK + q][TF + t][ln];
                float gv[4] = {sum[0], sum[1], sum[2], sum[3]}, uv[4] = {up[0], up[1], up[2], up[3]};
                finish_gated<OUT>(a.out, row, n0, gv, uv);
            } else {
                finish_linear4<OUT>(a.out, row, n0, sum);
            }
        }
    }
}

// 65 to 1024 rows of x: a tile of 128 rows of x and 256 weight rows (gated: 128
// of each weight), over all of k or one of `splits` parts of it.  The weight
// comes as in batch_rows_kernel, but a wave walks all the tile's k for 32
// weight rows of its own, so that the 8 waves share x's fragments: four steps
// of them at a time go straight to LDS, double buffered.  Lookups run one or
// two steps ahead, the next chunk's scales and transposition are done within
// this chunk's last steps, and a wave that multiplies goes first.  Per step of
// 32 k a wave looks up 2 packed dwords per lane, reads 8 x fragments and issues
// 16 matrix instructions; what bounds it is the LDS (about 880 cycles per step
// of the workgroup, 370 of them lookups, against 512 of the matrix pipe), of
// which about 0.7 is reached: 0.5 us per step, a tile of 8192 k in 130 us; gated
// 28672 x 8192 with 512 rows 524 us, 0.92 PFLOP/s, where decode and product
// take 676.
template <int OUT, bool kGated, int S>
__global__ __launch_bounds__(512) void tile_rows_kernel(RowsArgs a, const uint16_t *x_frags)
{
    constexpr int R = 2, TF = 8, kW = kGated ? 2 : 1;
    constexpr int kPer = R / kW;
    constexpr int kSpan = 512;
    constexpr int kStage = 4 * TF * kFragBytes;  // x's fragments of 4 steps: 32 KiB
    constexpr int kLook = S == 2 ? 2 : 1;        // steps that the lookups run ahead: what the registers hold
    __shared__ __attribute__((aligned(1024))) uint8_t table[kPairTableBytes + 256];
    __shared__ float scb[kW][256], cb4[kW][16];
    __shared__ __attribute__((aligned(1024))) uint8_t stage[2 * kStage];

    // this workgroup's tile, and its part of k
    int tile = blockIdx.x, split = 0, splits = 1;
    if (tile >= a.whole) {
        splits = a.out.splits;
        const int at = (tile - a.whole) / splits;
        split = tile - a.whole - at * splits;
        tile = a.whole + at;
    }
    // 128 rows of x; the weight is read again for each such slice
    const int slice = tile / a.row_blocks;
    const int64_t rb = tile - slice * a.row_blocks;
    const int64_t x_row0 = static_cast<int64_t>(slice) * (16 * TF);
    x_frags += static_cast<int64_t>(slice) * ((a.n_in + 511) / 512) * (16 * TF * 512);
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave;
    const int g = lane >> 4;
    constexpr int block_rows = 16 * kPer * 8;
    const int lb = a.log2_block;
    const uint32_t n_in = static_cast<uint32_t>(a.n_in);
    const int chunks = static_cast<int>((n_in + kSpan - 1) / kSpan);
    const int begin = split * chunks / splits, end = (split + 1) * chunks / splits;
    const bool odd = lane & 1, high = lane & 2;

    struct Loads {
        u32x4 packed[R][4];
        uint32_t code[R][S];
        float absmax[R][S];
    };
    const auto rsrc_of = [](const void *p, int64_t bytes) {
        return __builtin_amdgcn_make_buffer_rsrc(
            const_cast<void *>(p), 0,
            static_cast<int32_t>(bytes < 0 ? 0 : bytes < 0x7FFFFFF0 ? bytes : 0x7FFFFFF0),
            kRawBufferWord3);
    };
    const uint32_t k_load = 32 * (((lane >> 4) << 2) | (lane & 3));  // of the loaded piece
    const uint32_t row_load = 4 * ((lane >> 2) & 3);
    const int64_t blocks = (a.n_elems + (int64_t{1} << lb) - 1) >> lb;
    auto load = [&](Loads &l, int c) {
        const int64_t row0 = rb * block_rows + wr * (16 * kPer);
        const int64_t e0 = row0 * a.n_in;
        const int64_t b0 = e0 >> lb;
        const uint32_t phase = static_cast<uint32_t>(e0) & ((1u << lb) - 1);
        const uint32_t group_phase = static_cast<uint32_t>(b0) & 255;
        const int64_t packed_left = ((a.n_elems + 1) >> 1) - (e0 >> 1);
        const uint32_t k = c * kSpan + k_load;
        const uint32_t past = k < n_in ? 0u : 0x80000000u;
#pragma unroll
        for (int f = 0; f < R; ++f) {
            const int w = kGated ? f : 0;
            const uint32_t frag_row = kGated ? 0 : f * 16;
            const auto rp = rsrc_of(a.w[w].packed + (e0 >> 1), packed_left);
            const auto rc = rsrc_of(a.w[w].scale_codes + b0, blocks - b0);
            const auto rm = rsrc_of(a.w[w].nested_absmax + (b0 >> 8), (((blocks + 255) >> 8) - (b0 >> 8)) * 4);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                l.packed[f][q] = __builtin_amdgcn_raw_buffer_load_b128(
                    rp, (((frag_row + row_load + q) * n_in + k) >> 1) | past, 0, 0);
#pragma unroll
            for (int h = 0; h < S; ++h) {
                // of row lane / 4, the lane's quarter of the chunk
                const uint32_t e = (frag_row + (lane >> 2)) * n_in + c * kSpan + 128 * (lane & 3) + h * (128 / S);
                const uint32_t b = (phase + e) >> lb;
                l.code[f][h] = __builtin_amdgcn_raw_buffer_load_b8(rc, b, 0, 0);
                l.absmax[f][h] = __builtin_bit_cast(
                    float, __builtin_amdgcn_raw_buffer_load_b32(rm, ((group_phase + b) >> 8) * 4, 0, 0));
            }
        }
    };
    // four steps' x fragments, 32 KiB in a row, straight to LDS: 4 KiB a wave
    const u32x4 rs_x = make_rsrc(x_frags, static_cast<uint32_t>(chunks) * (4 * kStage));
    const uint32_t lds0 = lds_offset(stage);
    auto issue_x = [&](int q) {  // stage q = 4 chunk + j
        const uint32_t at = static_cast<uint32_t>(q) * kStage + wave * (4 * kFragBytes);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            buffer_to_lds(rs_x, lane * 16, at + i * kFragBytes,
                          lds0 + (q & 1) * kStage + wave * (4 * kFragBytes) + i * kFragBytes);
    };

    // one register, hidden from the compiler, so that each read is it plus an
    // immediate offset; without it every read's address took a register of its own
    uint32_t x_at = lds0 + lane * 16;
    __asm__("" : "+v"(x_at));
    const auto *x_lane = reinterpret_cast<const __attribute__((address_space(3))) u32x4 *>(x_at);

    const Codebooks codebooks = fetch_codebooks<kW>(a.w);
    Loads cur;
    issue_x(4 * begin);
    load(cur, begin);

    // the lookup tables, while the first loads are in flight
    fill_tables<kW, 1>(codebooks, table, scb, cb4);

    const uint32_t lane_byte = kGated ? (lane & 15) * 16 : (lane & 31) * 8;
    wait_all_and_barrier();
    f32x4 acc[R][TF];
#pragma unroll
    for (int f = 0; f < R; ++f)
#pragma unroll
        for (int t = 0; t < TF; ++t)
            acc[f][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // a fragment's scales, and its packed dwords into operand order
    auto prepare = [&](Loads &l, float (&s)[R][S], int f) {
#pragma unroll
        for (int h = 0; h < S; ++h) {
            const float q = block_scale(scb[kGated ? f : 0][l.code[f][h]], l.absmax[f][h],
                                        a.w[kGated ? f : 0].offset);
            // lane 16 g + r multiplies quarter g of row r
            s[f][h] = __builtin_bit_cast(
                float, __builtin_amdgcn_ds_bpermute((4 * (lane & 15) + g) * 4, __builtin_bit_cast(int, q)));
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            uint32_t v[4] = {l.packed[f][0][d], l.packed[f][1][d], l.packed[f][2][d], l.packed[f][3][d]};
            transpose_quads(v, odd, high);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                l.packed[f][j][d] = v[j];
        }
    };
    // step st's lookups; a piece beyond the row (its load gave zeros) reads the
    // row of zeros behind the table, and is multiplied with 0
    const uint32_t k_lane = 128 * g;
    auto lookup = [&](Pairs (&to)[R], const Loads &l, int c, int st) {
        const uint32_t from =
            c * kSpan + k_lane + 32 * (st / 4) >= n_in ? lane_byte | kPairTableBytes : lane_byte;
#pragma unroll
        for (int f = 0; f < R; ++f)
            to[f] = lookup_dword(l.packed[f][st / 4][st % 4], table + (kGated ? f : 0) * 8, from);
    };
    float s[R][S];
#pragma unroll
    for (int f = 0; f < R; ++f)
        prepare(cur, s, f);
    Pairs now[kLook][R];
#pragma unroll
    for (int i = 0; i < kLook; ++i)
        lookup(now[i], cur, begin, i);
    for (int c = begin; c < end; ++c) {
        Loads next;
        const int c_next = c + 1 < end ? c + 1 : c;  // at the end: the chunk again, unused
        float s_next[R][S];
        const uint32_t k = c * kSpan + k_lane;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int q = 4 * c + j;
            u32x4 x[2][TF / 2];  // the first half of a step's, the second
            auto read_x = [&](int d, int half) {
#pragma unroll
                for (int t = 0; t < TF / 2; ++t)
                    x[half][t] =
                        x_lane[((j & 1) * kStage + (d * TF + half * (TF / 2) + t) * kFragBytes) / 16];
            };
            read_x(0, 0);
            issue_x(q + 1 < 4 * end ? q + 1 : q - 1);  // at the end: a stage nobody reads
            if (j == 1)
                load(next, c_next);
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int st = 4 * j + d;
                u32x4 wf[R];
                read_x(d, 1);
#pragma unroll
                for (int f = 0; f < R; ++f)
                    wf[f] = scaled_dword<OUT>(now[st % kLook][f], k + 32 * j >= n_in ? 0.0f : s[f][j * S / 4]);
                keep_order();
                if (st + kLook < 16)
                    lookup(now[st % kLook], cur, c, st + kLook);
                else
                    lookup(now[st % kLook], next, c_next, st + kLook - 16);
                keep_order();
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int f = 0; f < R; ++f)
#pragma unroll
                    for (int t = 0; t < TF / 2; ++t)
                        acc[f][t] = Half<OUT>::mfma(wf[f], x[0][t], acc[f][t]);
                keep_order();
                if (d < 3)
                    read_x(d + 1, 0);
                if (j == 3 && d < R)  // the next chunk has arrived
                    prepare(next, s_next, d);
#pragma unroll
                for (int f = 0; f < R; ++f)
#pragma unroll
                    for (int t = 0; t < TF / 2; ++t)
                        acc[f][TF / 2 + t] = Half<OUT>::mfma(wf[f], x[1][t], acc[f][TF / 2 + t]);
                __builtin_amdgcn_s_setprio(0);
                keep_order();
            }
            // the next stage has arrived: behind its loads only the next
            // chunk's weight loads (more than 8) may be under way
            if (j == 1)
                __asm__ volatile("s_waitcnt vmcnt(8) lgkmcnt(0)" ::: "memory");
            else
                __asm__ volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            __asm__ volatile("" ::: "memory");
        }
        cur = next;
#pragma unroll
        for (int f = 0; f < R; ++f)
#pragma unroll
            for (int h = 0; h < S; ++h)
                s[f][h] = s_next[f][h];
    }
    if (splits > 1) {
        f32x4 *to = a.out.partial +
                    ((static_cast<int64_t>(split) * a.rest + tile - a.whole) * 8 + wave) * (TF * R * 64) + lane;
#pragma unroll
        for (int t = 0; t < TF; ++t)
#pragma unroll
            for (int f = 0; f < R; ++f)
                to[(t * R + f) * 64] = acc[f][t];
        return;
    }
    // the epilogue, 4 x 16 rows of x at a time through this wave's part of
    // the stages, so that its code is there once
    f32x4 *mine = reinterpret_cast<f32x4 *>(stage + wave * (8 * kFragBytes));
    const int64_t n0 = rb * block_rows + wr * (16 * kPer) + g * 4;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int f = 0; f < R; ++f)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                mine[(t * R + f) * 64 + lane] = acc[f][half * 4 + t];
#pragma unroll 1
        for (int t = 0; t < 4; ++t) {
            const int64_t row = x_row0 + (half * 4 + t) * 16 + (lane & 15);
            const f32x4 u = mine[(t * R) * 64 + lane], v = mine[(t * R + 1) * 64 + lane];
            if constexpr (kGated) {
                float gv[4] = {u[0], u[1], u[2], u[3]}, uv[4] = {v[0], v[1], v[2], v[3]};
                finish_gated<OUT>(a.out, row, n0, gv, uv);
            } else {
                finish_linear4<OUT>(a.out, row, n0, u);
                finish_linear4<OUT>(a.out, row, n0 + 16, v);
            }
        }
    }
}

// The splits' sums of 16 rows of x and one wave's 32 weight rows, added in
// order, and the epilogue: a wave each, with the loads of 8 splits in flight.
template <int OUT, bool kGated>
__global__ __launch_bounds__(256) void tile_rows_reduce_kernel(RowsArgs a)
{
    constexpr int R = 2, TF = 8;
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x % 2 * 4 + (threadIdx.x >> 6);
    const int wave = blockIdx.x / 2 % 8, at = blockIdx.x / 16;
    const int tile = a.whole + at;
    const int slice = tile / a.row_blocks, rb = tile - slice * a.row_blocks;
    const int64_t row0 = (static_cast<int64_t>(slice) * TF + t) * 16;
    if (row0 >= a.out.m)
        return;
    const int64_t step = static_cast<int64_t>(a.rest) * (8 * TF * R * 64);
    const f32x4 *from = a.out.partial + ((static_cast<int64_t>(at) * 8 + wave) * TF + t) * (R * 64) + lane;
    f32x4 sum[R];
#pragma unroll
    for (int f = 0; f < R; ++f)
        sum[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < a.out.splits; s += 8) {
        f32x4 v[8][R];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int f = 0; f < R; ++f)  // past the last split: the first again, left out below
                v[i][f] = from[(s + i < a.out.splits ? s + i : s) * step + f * 64];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (s + i < a.out.splits)
#pragma unroll
                for (int f = 0; f < R; ++f)
                    sum[f] = sum[f] + v[i][f];
    }
    const int64_t row = row0 + (lane & 15);
    const int64_t n0 = (static_cast<int64_t>(rb) * 8 + wave) * (16 * (kGated ? 1 : R)) + (lane >> 4) * 4;
    if constexpr (kGated) {
        float g[4] = {sum[0][0], sum[0][1], sum[0][2], sum[0][3]};
        float u[4] = {sum[1][0], sum[1][1], sum[1][2], sum[1][3]};
        finish_gated<OUT>(a.out, row, n0, g, u);
    } else {
        finish_linear4<OUT>(a.out, row, n0, sum[0]);
        finish_linear4<OUT>(a.out, row, n0 + 16, sum[1]);
    }
}

// ---------------------------------------------------------------------------
// few rows of dz: dx = dz W with the weight decoded straight into operands
// ---------------------------------------------------------------------------
struct ColumnArgs {
    Weight w[2];
    int64_t n_out, n_in;
    int32_t log2_block;
    int32_t steps;              // of 32 weight rows, per weight
    int32_t splits;             // of all steps
    int32_t slices;             // of 16 TF rows of dz
    const uint16_t *dz_frags[2];  // [slice][step][16 rows][lane][8], zeros beyond dz
    ProductArgs out;            // partial, groups, bias sums
};

// 16 TF rows of dz (dgate and dup: kTwo, one sum over both) against 128 weight
// columns: the sum runs down the weight's rows, so a lane takes the packed
// dwords of 8 rows, 8 neighbouring columns each, looks up their values and
// pairs the same column of two rows in one conversion: that transposes them
// into operand fragments (column 8 r + f in row r of fragment f) for nothing.
// A load takes 64 neighbouring bytes of 4 rows.  The 8 waves take steps of 32
// rows in turn, their sums meet in LDS, and those of the workgroups that share
// a column group in the workspace (product_reduce_kernel), in a fixed order.
// Bound by the lookups in LDS and the decode's vector instructions: W is read
// once for 16 TF rows of dz and never written out.  Whole calls: linear 11008 x
// 4096 with up to 16 rows 27 us, with 64 33; gated 28672 x 8192 with 64 rows 183,
// where decode and product take 547.
template <int OUT, bool kTwo, int TF>
__global__ __launch_bounds__(512) void weight_columns_kernel(ColumnArgs a)
{
    constexpr int kW = kTwo ? 2 : 1;
    __shared__ __attribute__((aligned(1024))) uint8_t table[kPairTableBytes + 256];
    __shared__ float scb[kW][256], cb4[kW][16];
    __shared__ __attribute__((aligned(16))) f32x4 partial[8][kFrags][64];
    if (static_cast<int>(blockIdx.y) == a.splits * a.slices) {
        add_bias_blocks(a.out.bias_partial, a.out.bias_n, a.out.bias_blocks, a.out.dbias);
        return;
    }
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int group = blockIdx.x;
    const int slice = static_cast<int>(blockIdx.y) / a.splits;
    const int split = static_cast<int>(blockIdx.y) - slice * a.splits;
    const int lb = a.log2_block;
    const uint32_t n_in = static_cast<uint32_t>(a.n_in);
    const uint32_t j0 = group * kGroup + 8 * r;
    // columns beyond the weight: nothing is loaded, and their sums are not kept
    const uint32_t past = j0 < n_in ? 0u : 0x80000000u;
    const int64_t n_elems = a.n_out * a.n_in;
    const int64_t blocks = (n_elems + (int64_t{1} << lb) - 1) >> lb;
    const int all_steps = a.steps * kW;
    const int first = static_cast<int>(static_cast<uint32_t>(all_steps) * split / a.splits);
    const int last = static_cast<int>(static_cast<uint32_t>(all_steps) * (split + 1) / a.splits);

    struct Loads {
        uint32_t packed[8], code[8];
        float absmax[8];
        u32x4 x[TF];
    };
    const auto rsrc_of = [](const void *p, int64_t bytes) {
        return __builtin_amdgcn_make_buffer_rsrc(
            const_cast<void *>(p), 0, static_cast<int32_t>(bytes < 0x7FFFFFF0 ? bytes : 0x7FFFFFF0),
            kRawBufferWord3);
    };
    auto load = [&](Loads &l, int step) {
        step = step < last ? step : last - 1;  // loaded again, unused
        const int which = kTwo && step >= a.steps ? 1 : 0;
        const int s = step - which * a.steps;
        const Weight &w = a.w[which];
        const int64_t e0 = static_cast<int64_t>(s) * 32 * a.n_in;
        const int64_t b0 = e0 >> lb;
        const uint32_t phase = static_cast<uint32_t>(e0) & ((1u << lb) - 1);
        const uint32_t group_phase = static_cast<uint32_t>(b0) & 255;
        const auto rp = rsrc_of(w.packed + (e0 >> 1), ((n_elems + 1) >> 1) - (e0 >> 1));
        const auto rc = rsrc_of(w.scale_codes + b0, blocks - b0);
        const auto rm = rsrc_of(w.nested_absmax + (b0 >> 8), (((blocks + 255) >> 8) - (b0 >> 8)) * 4);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint32_t e = (8 * g + q) * n_in + j0;
            const uint32_t b = (phase + e) >> lb;
            l.packed[q] = __builtin_amdgcn_raw_buffer_load_b32(rp, (e >> 1) | past, 0, 0);
            l.code[q] = __builtin_amdgcn_raw_buffer_load_b8(rc, b | past, 0, 0);
            l.absmax[q] = __builtin_bit_cast(
                float, __builtin_amdgcn_raw_buffer_load_b32(rm, (((group_phase + b) >> 8) * 4) | past, 0, 0));
        }
#pragma unroll
        for (int t = 0; t < TF; ++t)
            l.x[t] = *reinterpret_cast<const u32x4 *>(
                a.dz_frags[which] + ((static_cast<int64_t>(slice) * a.steps + s) * TF + t) * 512 + lane * 8);
    };

    const Codebooks codebooks = fetch_codebooks<kW>(a.w);
    Loads cur;
    load(cur, first + wave);
    fill_tables<kW, 1>(codebooks, table, scb, cb4);

    f32x4 acc[kFrags][TF];
#pragma unroll
    for (int f = 0; f < kFrags; ++f)
#pragma unroll
        for (int t = 0; t < TF; ++t)
            acc[f][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int step = first + wave; step < last; step += 8) {
        Loads next;
        load(next, step + 8);
        const int which = kTwo && step >= a.steps ? 1 : 0;
        const uint32_t from = kTwo ? (lane & 15) * 16 + which * 8 : (lane & 31) * 8;
        const float offset = a.w[which].offset;
        float s[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            s[q] = block_scale(scb[which][cur.code[q]], cur.absmax[q], offset);
        u32x4 wf[kFrags];
        Pairs row[2];
        row[0] = lookup_dword(cur.packed[0], table, from);
        row[1] = lookup_dword(cur.packed[1], table, from);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            Pairs then[2];
            if (p < 3) {
                then[0] = lookup_dword(cur.packed[2 * p + 2], table, from);
                then[1] = lookup_dword(cur.packed[2 * p + 3], table, from);
            }
            keep_order();
#pragma unroll
            for (int f = 0; f < kFrags; ++f)
                wf[f][p] = Half<OUT>::pack2(row[0].v[f / 2][f % 2] * s[2 * p],
                                            row[1].v[f / 2][f % 2] * s[2 * p + 1]);
            if (p < 3) {
                row[0] = then[0];
                row[1] = then[1];
            }
        }
        // rows beyond the weight hold no value at all
        const int left = static_cast<int>(a.n_out) - ((step - which * a.steps) * 32 + 8 * g);
        if (__builtin_amdgcn_readfirstlane(static_cast<int>(a.n_out) - (step - which * a.steps) * 32) < 32) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t mask = left >= 2 * p + 2 ? 0xFFFFFFFFu : left == 2 * p + 1 ? 0xFFFFu : 0u;
#pragma unroll
                for (int f = 0; f < kFrags; ++f)
                    wf[f][p] &= mask;
            }
        }
#pragma unroll
        for (int f = 0; f < kFrags; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                acc[f][t] = Half<OUT>::mfma(wf[f], cur.x[t], acc[f][t]);
        cur = next;
    }
    // the waves' sums, 16 rows of dz at a time; wave f adds up fragment f
    const int tile = group * a.slices + slice;
    f32x4 *to = a.out.partial + (static_cast<int64_t>(split) * (gridDim.x * a.slices) + tile) * (kFrags * TF * 64);
#pragma unroll
    for (int t = 0; t < TF; ++t) {
        if (t > 0)
            lds_barrier();
#pragma unroll
        for (int f = 0; f < kFrags; ++f)
            partial[wave][f][lane] = acc[f][t];
        lds_barrier();
        f32x4 sum = partial[0][wave][lane];
#pragma unroll
        for (int q = 1; q < 8; ++q)
            sum = sum + partial[q][wave][lane];
        to[(wave * TF + t) * 64 + lane] = sum;
    }
}

// ---------------------------------------------------------------------------
// the bias gradient on its own
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kThreads) void bias_grad_reduce_kernel(const float *partial,
                                                                    int64_t n, int32_t blocks,
                                                                    float *dbias)
{
    add_bias_blocks(partial, n, blocks, dbias);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// The product reads this matrix where it lies, or a padded copy of it.
bool needs_copy(const void *x, int64_t ld, int64_t m, int64_t k)
{
    return !rows_aligned(x, ld, m, k) || (m > 1 && ld > (int64_t{1} << 22));
}

// The row stride of a matrix that the product reads where it lies, at most 2^22
// (needs_copy): a tile's 256 rows then end below byte 2^31, the offset that the
// kernels give to what must not be read.  One row's stride, and that of rows
// without columns, may be anything and is not used.
int64_t product_ld(int64_t ld, int64_t m, int64_t k)
{
    return m > 1 && k > 0 ? ld : k;
}

int64_t padded_ld(int64_t k)
{
    return ceil_div(k, kChunk) * kChunk;
}

// How a product is cut: the tile (128 WN columns x 16 TF WT rows) and the
// splits of the summed index.  It follows from the call's sizes and the GPU
// alone, so that a smaller workspace changes nothing in the sums.
struct Plan {
    int tile;      // 0: 256 x 256, 1: 128 x 128, 2: 128 x 64
    int splits;
    double cost;   // microseconds, roughly
};

constexpr int kTileCols[3] = {256, 128, 128}, kTileRows[3] = {256, 128, 64};
constexpr int kTileResident[3] = {1, 2, 3};        // workgroups per CU (LDS)
// Microseconds of one chunk of 64 k with every CU full, as measured: 1.2, 0.77
// and 0.45 PFLOP/s over 256 CUs.
constexpr double kTileChunk[3] = {1.78, 1.40, 1.80};

Plan plan_of(int64_t m, int64_t groups, int64_t all_chunks, int cus)
{
    Plan best{2, 1, 1e300};
    for (int tile = 0; tile < 3; ++tile) {
        const int64_t tiles = ceil_div(groups * kGroup, kTileCols[tile]) * ceil_div(m, kTileRows[tile]);
        for (int splits = 1; splits <= 16; ++splits) {
            if (splits > 1 && splits * 2 > all_chunks)
                break;
            const int64_t rounds = ceil_div(tiles * splits, static_cast<int64_t>(cus) * kTileResident[tile]);
            double cost = static_cast<double>(rounds) *
                          (static_cast<double>(ceil_div(all_chunks, splits)) * kTileChunk[tile] + 2.0);
            if (splits > 1)  // the partial sums, written and read at about 4 TB/s, and a launch
                cost += 3.0 + static_cast<double>(splits) * static_cast<double>(m) *
                                  static_cast<double>(groups * kGroup) * 8.0 / 4e6;
            if (cost < best.cost)
                best = Plan{tile, splits, cost};
        }
    }
    return best;
}

// The sizes of one call's product.
struct Shape {
    int64_t m, n, k;   // rows, output columns, summed index per x matrix
    int32_t layout;
    int n_x() const { return layout == kStacked ? 2 : 1; }
    int64_t per_group() const { return layout == kSideBySide ? 64 : kGroup; }
    int64_t groups() const { return ceil_div(n, per_group()); }
    int64_t chunks() const { return ceil_div(k, kChunk); }
    int64_t group_bytes() const { return chunks() * n_x() * kUnitBytes; }
    Plan plan(int cus) const { return plan_of(m, groups(), chunks() * n_x(), cus); }
    // partial sums of `g` groups
    int64_t split_bytes(const Plan &p, int64_t g) const
    {
        return p.splits == 1 ? 0
                             : p.splits * ceil_div(g * kGroup, kTileCols[p.tile]) * kTileCols[p.tile] *
                                   ceil_div(m, kTileRows[p.tile]) * kTileRows[p.tile] * 4;
    }
    int64_t window_bytes(const Plan &p, int64_t g) const
    {
        return g * group_bytes() + split_bytes(p, g);
    }
};

// Workspace: [padded x copies][column sums][fragments of a window of groups]
int64_t copy_bytes(const Shape &s, bool copy)
{
    return copy ? align256(s.m * padded_ld(s.k) * 2) * s.n_x() : 0;
}

int64_t partial_bytes(int64_t m, int64_t n)
{
    return align256(ceil_div(m, kRowBlock) * n * 4);
}

int64_t workspace_need(const Shape &s, int64_t fixed, bool least)
{
    const int64_t groups = least ? (s.groups() < 2 ? s.groups() : 2) : s.groups();
    return fixed + s.window_bytes(s.plan(current_compute_units()), groups);
}

// How the tile route is cut: whole rounds of 128 x 256 tiles, one per CU, and
// the tiles of the last round, each over one of `splits` parts of k where they
// alone leave CUs idle (gated 28672 x 8192 with 512 rows: 3.5 rounds take the
// time of 3.5, not of 4).
struct TilePlan {
    int64_t row_blocks, whole, rest;
    int splits;
    double cost;  // microseconds, roughly
    int64_t partial_bytes() const { return splits == 1 ? 0 : splits * rest * (128 * 256 * 4); }
};

TilePlan tile_plan(int64_t m, int64_t n_out, int64_t n_in, bool gated, int cus)
{
    const int64_t row_blocks = ceil_div(n_out, gated ? 128 : 256);
    const int64_t tiles = row_blocks * ceil_div(m, 128), chunks = ceil_div(n_in, 512);
    const int64_t whole = tiles / cus * cus, rest = tiles - whole;
    // microseconds, as measured: 8 a chunk of 512 k, 9 until the tables are
    // filled and the first loads have come; the partial sums, written and read
    // at about 4 TB/s, and a launch
    const double rounds = static_cast<double>(whole / cus) * (static_cast<double>(chunks) * 8.0 + 9.0);
    TilePlan p{row_blocks, tiles, 0, 1, 1e300};
    for (int splits = 1; splits <= 16 && splits <= chunks; ++splits) {
        double cost = rounds + static_cast<double>(ceil_div(rest * splits, cus)) *
                                   (static_cast<double>(ceil_div(chunks, splits)) * 8.0 + 9.0);
        if (splits > 1)
            cost += 3.0 + static_cast<double>(rest * splits) * (128 * 256 * 8.0 / 4e6);
        if (cost < p.cost)
            p = splits == 1 ? TilePlan{row_blocks, tiles, 0, 1, cost}
                            : TilePlan{row_blocks, whole, rest, splits, cost};
    }
    return p;
}

// Which kernel a forward call takes.
enum Route {
    kTokenRoute,    // one or two rows of x, weight rows of up to 32768
    kBatchRoute,    // up to 64 rows: x's fragments from memory, waves along k
    kTileRoute,     // up to 1024: tiles of 128 rows of x, x's fragments through LDS
    kRaggedRoute,   // up to 64, weight rows of whole dwords that are not 32 k apart
    kProductRoute   // decode to fragments, then the product
};

// Where the routes meet, in whole calls (BF16 unless said otherwise, us):
//   token | batch: gated 28672 x 8192 at m = 2 75 | 80, at m = 4 97 | 80; gated
//     11008 x 4096 at m = 2 19 | 23, at m = 4 24 | 23
//   batch | tile, which costs the same for 1 to 128 rows: gated 28672 x 8192 at
//     m = 64 135 | 150, two readings at m = 128 232 | 150; gated 11008 x 4096 at
//     m = 64 34 | 48, at m = 128 63 | 48
//   tile | product: the lesser of the two plans' costs: gated 28672 x 8192 at
//     m = 512 524 | 676, at m = 1024 999 | 1083; gated 11008 x 4096 at m = 320
//     90 | 152, at m = 768 165 | 235; linear 11008 x 4096 at m = 700 95 | 110.
//     Beyond 1024 rows the decode is a small part, and the plans' costs are
//     too rough to choose.  They would take the tiles each time (tile | product
//     as planned, then as measured): gated 11008 x 4096 at m = 1280 275 | 280,
//     267 | 246; linear 4096 x 11008 at m = 2048 185 | 218, 216 | 206; gated
//     11008 x 4096 at m = 1536 316 | 396, 310 | 340.  The limit is 8 and 5 % the
//     better for the first two, 10 % the worse for the third.
//   ragged | product: FP16 4096 x 11000 at m = 64 58 | 73; more rows would
//     read the weight twice
constexpr int64_t kTokenMost = 2, kBatchMost = 64, kTileMost = 1024, kRaggedMost = 64;

Route route_of(const dq4_weight_t *w0, const dq4_weight_t *w1, const Shape &s, int cus)
{
    if (s.m > kTileMost || s.k == 0 || s.k % 8 != 0 ||
        reinterpret_cast<uintptr_t>(w0->packed) % 4 != 0 ||
        (w1 && reinterpret_cast<uintptr_t>(w1->packed) % 4 != 0))
        return kProductRoute;
    if (s.k % 32 != 0)
        return s.m <= kRaggedMost ? kRaggedRoute : kProductRoute;
    if (s.m <= kTokenMost && s.k <= kTokenMaxChunks * kTokenSpan)
        return kTokenRoute;
    if (s.m <= kBatchMost)
        return kBatchRoute;
    // the product's decode: 5.2 TB/s, and a launch
    const double decode = 5.0 + static_cast<double>(s.n * s.k) * (w1 ? 2.0 : 1.0) * 4.8e-7;
    return tile_plan(s.m, s.n, s.k, w1 != nullptr, cus).cost < s.plan(cus).cost + decode ? kTileRoute
                                                                                        : kProductRoute;
}

// A backward call with few rows of dz whose weight rows are whole dwords
// decodes in registers (weight_columns_kernel), once for 32 rows.  Against the
// product over a decoded copy, in whole calls (BF16, us): linear 4096 x 4096 at
// m = 128 29 | 39, gated 11008 x 4096 at m = 128 74 | 118.  With the fifth
// reading of the weight, from m = 129 on, one gains what the other loses: at m =
// 192 gated 28672 x 8192 570 | about 600, linear 11008 x 4096 69 | 60.
constexpr int64_t kColumnsMost = 128;

struct ColumnPlan {
    bool use;
    int tf, slices, splits;
    int64_t steps, groups;  // steps per weight
    int64_t frag_bytes() const { return slices * steps * tf * kFragBytes; }  // per matrix
    int64_t partial_bytes() const { return splits * groups * slices * kFrags * tf * kFragBytes; }
};

ColumnPlan column_plan(const dq4_weight_t *w0, const dq4_weight_t *w1, int64_t n_out, int64_t n_in,
                       int64_t m, int cus)
{
    ColumnPlan p{};
    p.use = m <= kColumnsMost && n_out > 0 && n_in > 0 && n_in % 8 == 0 &&
            reinterpret_cast<uintptr_t>(w0->packed) % 4 == 0 &&
            (!w1 || reinterpret_cast<uintptr_t>(w1->packed) % 4 == 0);
    if (!p.use)
        return p;
    p.tf = m <= 16 ? 1 : 2;
    p.slices = static_cast<int>(ceil_div(m, 16 * p.tf));
    p.steps = ceil_div(n_out, 32);
    p.groups = ceil_div(n_in, kGroup);
    // one workgroup per CU, each wave with a step at least
    const int64_t all = p.steps * (w1 ? 2 : 1);
    int64_t splits = cus / (p.groups * p.slices);
    if (splits > ceil_div(all, 8))
        splits = ceil_div(all, 8);
    p.splits = static_cast<int>(splits < 1 ? 1 : splits);
    return p;
}

int x_row_frags(int64_t m)
{
    return m <= 16 ? 1 : m <= 32 ? 2 : m <= 64 ? 4 : 8;
}

// Bytes of x in operand fragments.
int64_t x_fragment_bytes(int64_t m, int64_t k)
{
    const int64_t tf = x_row_frags(m);
    return ceil_div(m, 16 * tf) * ceil_div(k, 512) * 16 * tf * kFragBytes;
}

// Whether a forward call needs x in 16-byte aligned rows and x is not (the
// batch and tile routes lay x out in fragments, from any rows).
bool forward_copies(const Shape &s, const dq4_weight_t *w0, const dq4_weight_t *w1, const void *x,
                    int64_t ld_x)
{
    const Route route = route_of(w0, w1, s, current_compute_units());
    return route != kBatchRoute && route != kTileRoute && needs_copy(x, ld_x, s.m, s.k);
}

// Workspace of a forward call.
int64_t forward_need(const Shape &s, const dq4_weight_t *w0, const dq4_weight_t *w1, bool copy,
                     bool least)
{
    const int64_t fixed = copy_bytes(s, copy);
    switch (route_of(w0, w1, s, current_compute_units())) {
    case kProductRoute:
        return workspace_need(s, fixed, least);
    case kBatchRoute:
        return x_fragment_bytes(s.m, s.k);
    case kTileRoute:
        return x_fragment_bytes(s.m, s.k) +
               tile_plan(s.m, s.n, s.k, w1 != nullptr, current_compute_units()).partial_bytes();
    default:
        return fixed;
    }
}

template <int OUT, bool kGated, int WN, int WT, int TF>
dq4_status_t launch_product_tile(ProductArgs a, hipStream_t s)
{
    a.tiles_t = static_cast<int32_t>(ceil_div(a.m, 16 * TF * WT));
    const int64_t tiles = ceil_div(a.groups, WN) * a.tiles_t;
    void *params[] = {&a};
    const void *kernel;
    if constexpr (WN == 2)
        kernel = reinterpret_cast<const void *>(&fragment_product_wide_kernel<OUT, kGated>);
    else
        kernel = reinterpret_cast<const void *>(&fragment_product_kernel<OUT, kGated, WN, WT, TF>);
    dq4_status_t st = launch(kernel, tiles, a.splits + (a.dbias ? 1 : 0), 64 * WN * WT, params, s);
    if (st != DQ4_OK || a.splits == 1)
        return st;
    int32_t n_tiles = static_cast<int32_t>(tiles);
    void *rp[] = {&a, &n_tiles};
    return launch(reinterpret_cast<const void *>(&product_reduce_kernel<OUT, kGated, WN, WT, TF>),
                  tiles * WN * WT, TF, 256, rp, s);
}

template <int OUT, bool kGated>
dq4_status_t launch_product(const ProductArgs &a, const Plan &plan, hipStream_t s)
{
    if (plan.tile == 0)
        return launch_product_tile<OUT, kGated, 2, 4, 4>(a, s);
    if (plan.tile == 1)
        return launch_product_tile<OUT, kGated, 1, 4, 2>(a, s);
    return launch_product_tile<OUT, kGated, 1, 4, 1>(a, s);
}

template <int OUT, bool kGated, int R, int TF, int WAVES>
dq4_status_t launch_ragged_tile(RowsArgs a, int cus, hipStream_t s)
{
    a.row_blocks = static_cast<int32_t>(ceil_div(a.n_out, 16 * (kGated ? R / 2 : R)));
    void *params[] = {&a};
    return launch(reinterpret_cast<const void *>(&ragged_rows_kernel<OUT, kGated, R, TF, WAVES>),
                  a.row_blocks < cus ? a.row_blocks : cus, 1, 64 * WAVES, params, s);
}

template <int OUT, bool kGated>
dq4_status_t launch_ragged(const RowsArgs &a, int cus, hipStream_t s)
{
    if (a.out.m > 32)
        return launch_ragged_tile<OUT, kGated, 2, 4, 8>(a, cus, s);
    if (a.out.m > 16)
        return launch_ragged_tile<OUT, kGated, kGated ? 4 : 2, 2, 8>(a, cus, s);
    if constexpr (!kGated)
        if (ceil_div(a.n_out, 16) <= cus)
            return launch_ragged_tile<OUT, false, 1, 1, 16>(a, cus, s);
    return launch_ragged_tile<OUT, kGated, 2, 1, kGated ? 8 : 16>(a, cus, s);
}

template <int OUT, bool kGated, int M>
dq4_status_t launch_token_rows(const RowsArgs &r, int cus, hipStream_t s)
{
    // a wave's registers hold x's chunk and the rows in flight
    constexpr int kWaves = M == 1 ? 16 : 8;
    TokenArgs a{};
    a.w[0] = r.w[0];
    a.w[1] = r.w[1];
    a.n_in = r.n_in;
    a.log2_block = r.log2_block;
    a.chunks = static_cast<int32_t>(ceil_div(r.n_in, kTokenSpan));
    a.wk = static_cast<int32_t>(ceil_div(a.chunks, ceil_div(a.chunks, kWaves)));
    const int wr = kWaves / a.wk;
    const int64_t grid = r.n_out < cus ? r.n_out : cus;
    a.rows_per = static_cast<int32_t>(r.n_out / grid);
    a.rows_extra = static_cast<int32_t>(r.n_out % grid);
    const int pair = (kGated ? 1 : 2) * wr;  // rows of one pair of every wave
    const int fit = kTokenPartials<kGated> / 2 / (M * (kGated ? 2 : 1) * a.chunks * 4);
    a.out = r.out;
    void *params[] = {&a};
    // with a single pair for each wave there is nothing to load ahead: 4096 x
    // 4096 at m = 1 takes 10.6 us with a ring of three, 7.6 us with one
    if (a.rows_per + (a.rows_extra ? 1 : 0) <= pair && pair <= fit) {
        a.batch = pair;
        return launch(reinterpret_cast<const void *>(&token_rows_kernel<OUT, kGated, M, kWaves, 1>), grid,
                      1, 64 * a.wk * wr, params, s);
    }
    a.batch = fit / (kTokenDepth * pair) * (kTokenDepth * pair);
    return launch(reinterpret_cast<const void *>(&token_rows_kernel<OUT, kGated, M, kWaves, kTokenDepth>),
                  grid, 1, 64 * a.wk * wr, params, s);
}

template <int OUT, bool kGated, int TF>
dq4_status_t launch_batch_rows(RowsArgs a, const uint16_t *x_frags, int cus, hipStream_t s)
{
    // waves along k: as many rounds of row blocks as fit the GPU, each as long
    // as its chunks per wave plus about one for the sums' meeting
    const int64_t tasks = ceil_div(a.n_out, kGated ? 16 : 32), chunks = ceil_div(a.n_in, 512);
    int best = 1;
    int64_t least = INT64_MAX;
    for (int wk = 1; wk <= 8 && wk <= chunks; wk *= 2) {
        const int64_t row_blocks = ceil_div(tasks, 8 / wk);
        const int64_t cost = ceil_div(row_blocks, cus) * (ceil_div(chunks, wk) + 1);
        if (cost < least) {
            least = cost;
            best = wk;
        }
    }
    a.row_blocks = static_cast<int32_t>(ceil_div(tasks, 8 / best));
    void *params[] = {&a, &x_frags, &best};
    const void *kernel = a.log2_block >= 6 && a.n_in % 64 == 0
                             ? reinterpret_cast<const void *>(&batch_rows_kernel<OUT, kGated, TF, 2>)
                             : reinterpret_cast<const void *>(&batch_rows_kernel<OUT, kGated, TF, 4>);
    return launch(kernel, a.row_blocks < cus ? a.row_blocks : cus, 1, 512, params, s);
}

template <int OUT, bool kGated>
dq4_status_t launch_batch(const RowsArgs &a, uint8_t *workspace, int cus, hipStream_t s)
{
    const uint16_t *x = a.out.x[0];
    int64_t ld = a.out.ld_x, m = a.out.m, k = a.n_in;
    int32_t tf = x_row_frags(m);
    int32_t frags = static_cast<int32_t>(ceil_div(k, 512) * 16 * tf);
    bool aligned = rows_aligned(x, ld, m, k);
    uint16_t *out = reinterpret_cast<uint16_t *>(workspace);
    void *params[] = {&x, &ld, &m, &k, &tf, &frags, &aligned, &out};
    const dq4_status_t st = launch(reinterpret_cast<const void *>(&x_fragments_zero_fill),
                                   ceil_div(frags, kThreads / 64), ceil_div(m, 16 * tf), kThreads, params, s);
    if (st != DQ4_OK)
        return st;
    if (tf == 1)
        return launch_batch_rows<OUT, kGated, 1>(a, out, cus, s);
    if (tf == 2)
        return launch_batch_rows<OUT, kGated, 2>(a, out, cus, s);
    if (tf == 4)
        return launch_batch_rows<OUT, kGated, 4>(a, out, cus, s);
    const TilePlan p = tile_plan(m, a.n_out, k, kGated, cus);
    RowsArgs b = a;
    b.row_blocks = static_cast<int32_t>(p.row_blocks);
    b.whole = static_cast<int32_t>(p.whole);
    b.rest = static_cast<int32_t>(p.rest);
    b.out.splits = p.splits;
    b.out.partial = reinterpret_cast<f32x4 *>(workspace + x_fragment_bytes(m, k));
    void *tile_params[] = {&b, &out};
    const dq4_status_t tiles = launch(a.log2_block >= 6 && a.n_in % 64 == 0
                                          ? reinterpret_cast<const void *>(&tile_rows_kernel<OUT, kGated, 2>)
                                          : reinterpret_cast<const void *>(&tile_rows_kernel<OUT, kGated, 4>),
                                      p.whole + p.rest * p.splits, 1, 512, tile_params, s);
    if (tiles != DQ4_OK || p.splits == 1)
        return tiles;
    void *reduce_params[] = {&b};
    return launch(reinterpret_cast<const void *>(&tile_rows_reduce_kernel<OUT, kGated>), p.rest * 16,
                  1, 256, reduce_params, s);
}

// Few rows of x, by one of the kernels that read the 4-bit weight itself.
template <int OUT, bool kGated>
dq4_status_t launch_few_rows(const RowsArgs &a, Route route, uint8_t *workspace, int cus,
                             hipStream_t s)
{
    if (route == kRaggedRoute)
        return launch_ragged<OUT, kGated>(a, cus, s);
    if (route == kBatchRoute || route == kTileRoute)
        return launch_batch<OUT, kGated>(a, workspace, cus, s);
    if (a.out.m == 1)
        return launch_token_rows<OUT, kGated, 1>(a, cus, s);
    return launch_token_rows<OUT, kGated, 2>(a, cus, s);
}

// The work beside a decode: which, and in how many workgroups.
struct BesideWork {
    Beside kind;
    BesideArgs args;
};

// More pieces than these (matrices of 2^33 elements in odd rows), 2^31 threads,
// take launches of their own.
constexpr int32_t kMostBeside = 1 << 23;

BesideWork copy_work(const void *x, int64_t ld, int64_t m, int64_t k, void *out)
{
    BesideWork w{kCopy, {}};
    w.args.copy = CopyArgs{static_cast<const uint16_t *>(x), ld, m, k, static_cast<uint16_t *>(out),
                           padded_ld(k)};
    w.args.columns = static_cast<int32_t>(ceil_div(padded_ld(k), kThreads));
    w.args.blocks = static_cast<int32_t>(ceil_div(m, kRowBlock)) * w.args.columns;
    return w;
}

BesideWork slope_work(const SlopeArgs &a, bool gated)
{
    bool vec = rows_aligned(a.dy, a.ld_dy, a.m, a.n);
    for (const void *p : {static_cast<const void *>(a.pre[0]), static_cast<const void *>(a.pre[1])})
        vec = vec && (!p || rows_aligned(p, a.ld_pre, a.m, a.n));
    for (const void *p : {static_cast<const void *>(a.dz[0]), static_cast<const void *>(a.dz[1])})
        vec = vec && (!p || rows_aligned(p, a.ld_dz, a.m, a.n));
    BesideWork w{gated ? (vec ? kGatedSlopes8 : kGatedSlopes1) : (vec ? kSlopes8 : kSlopes1), {}};
    w.args.slope = a;
    w.args.columns = static_cast<int32_t>(ceil_div(a.pad[0] ? a.ld_pad : a.n, vec ? 256 : 32));
    w.args.blocks = static_cast<int32_t>(ceil_div(a.pad[0] ? a.pad_rows : a.m, kRowBlock)) * w.args.columns;
    return w;
}

template <int OUT, bool kForward, bool kAligned>
const void *fragments_kernel(Beside kind)
{
    if constexpr (kForward) {
        if (kind == kCopy)
            return reinterpret_cast<const void *>(&weight_fragments_kernel<OUT, true, kAligned, kCopy>);
        return reinterpret_cast<const void *>(&weight_fragments_kernel<OUT, true, kAligned, kNothing>);
    } else {
        switch (kind) {
        case kSlopes8:
            return reinterpret_cast<const void *>(&weight_fragments_kernel<OUT, false, kAligned, kSlopes8>);
        case kSlopes1:
            return reinterpret_cast<const void *>(&weight_fragments_kernel<OUT, false, kAligned, kSlopes1>);
        case kGatedSlopes8:
            return reinterpret_cast<const void *>(&weight_fragments_kernel<OUT, false, kAligned, kGatedSlopes8>);
        case kGatedSlopes1:
            return reinterpret_cast<const void *>(&weight_fragments_kernel<OUT, false, kAligned, kGatedSlopes1>);
        default:
            return reinterpret_cast<const void *>(&weight_fragments_kernel<OUT, false, kAligned, kNothing>);
        }
    }
}

// A decode of a.groups (none: 0) and the work beside it.
template <int OUT, bool kForward>
dq4_status_t launch_fragments(FragmentArgs a, bool aligned, BesideWork beside, int cus, hipStream_t s)
{
    const int64_t all_chunks = a.layout == kStacked ? 2 * a.chunks : a.chunks;
    if (kForward && aligned && a.n_in % 32 == 0 && beside.kind == kNothing) {
        int32_t spans = static_cast<int32_t>(ceil_div(all_chunks, 4));
        int64_t items64 = static_cast<int64_t>(a.groups) * spans;
        if (items64 > INT32_MAX / 2)
            return DQ4_EUNSUPPORTED;
        int32_t items = static_cast<int32_t>(items64);
        void *params[] = {&a, &spans, &items};
        const void *kernel =
            a.layout == kSideBySide
                ? reinterpret_cast<const void *>(&weight_row_fragments_kernel<OUT, true>)
                : reinterpret_cast<const void *>(&weight_row_fragments_kernel<OUT, false>);
        const int64_t pairs = ceil_div(items, 2);
        return launch(kernel, pairs < cus ? pairs : cus, 1, 64 * kDecodeWaves, params, s);
    }
    const int64_t grid = kForward ? a.groups * ceil_div(all_chunks, 4) : ceil_div(a.groups, 2) * all_chunks;
    const void *kernel = aligned ? fragments_kernel<OUT, kForward, true>(beside.kind)
                                 : fragments_kernel<OUT, kForward, false>(beside.kind);
    while (beside.args.blocks > kMostBeside) {
        BesideArgs part = beside.args;
        part.blocks = kMostBeside;
        void *params[] = {&a, &part};  // no decode: the grid has this work's workgroups alone
        const dq4_status_t st = launch(kernel, kMostBeside, 1, kThreads, params, s);
        if (st != DQ4_OK)
            return st;
        beside.args.first += kMostBeside;
        beside.args.blocks -= kMostBeside;
    }
    void *params[] = {&a, &beside.args};
    return launch(kernel, grid + beside.args.blocks, 1, kThreads, params, s);
}

// Decode and multiply, window by window of output columns.
template <int OUT, bool kForward>
dq4_status_t run_product(const Shape &sh, const dq4_weight_t *w0, const dq4_weight_t *w1,
                         int64_t n_out, int64_t n_in, int log2_block, ProductArgs p,
                         BesideWork beside, uint8_t *fragments, int64_t fragment_bytes,
                         hipStream_t s)
{
    int device = 0;
    const hipError_t e = hipGetDevice(&device);
    if (e != hipSuccess)
        return hip_failed(e);
    const int cus = compute_units(device);
    p.m = sh.m;
    p.n = sh.n;
    if constexpr (kForward) {
        const Route route = route_of(w0, w1, sh, cus);
        if (route != kProductRoute) {
            if (beside.kind != kNothing) {
                const dq4_status_t st = launch_fragments<OUT, true>(FragmentArgs{}, true, beside, cus, s);
                if (st != DQ4_OK)
                    return st;
            }
            RowsArgs r{};
            r.w[0] = device_weight(*w0);
            r.w[1] = device_weight(w1 ? *w1 : *w0);
            r.n_out = n_out;
            r.n_in = n_in;
            r.n_elems = n_out * n_in;
            r.log2_block = log2_block;
            r.out = p;
            return w1 ? launch_few_rows<OUT, true>(r, route, fragments, cus, s)
                      : launch_few_rows<OUT, false>(r, route, fragments, cus, s);
        }
    }
    const int64_t groups = sh.groups();
    const Plan plan = sh.plan(cus);
    // the widest window that fits, in pairs of groups (a tile's columns)
    int64_t window = groups;
    while (window > 2 && sh.window_bytes(plan, window) > fragment_bytes)
        window = window / 2 + (window / 2) % 2;
    FragmentArgs f{};
    f.w[0] = device_weight(*w0);
    f.w[1] = device_weight(w1 ? *w1 : *w0);
    const int64_t split_bytes = sh.split_bytes(plan, window);
    f.out = reinterpret_cast<uint16_t *>(fragments + split_bytes);
    f.n_out = n_out;
    f.n_in = n_in;
    f.log2_block = log2_block;
    f.chunks = static_cast<int32_t>(sh.chunks());
    f.layout = sh.layout;
    const bool aligned = n_in % 8 == 0 && reinterpret_cast<uintptr_t>(w0->packed) % 4 == 0 &&
                         (!w1 || reinterpret_cast<uintptr_t>(w1->packed) % 4 == 0);
    p.wfrag = f.out;
    p.splits = plan.splits;
    p.partial = reinterpret_cast<f32x4 *>(fragments);
    p.chunks = f.chunks;
    p.n_x = sh.n_x();
    for (int64_t g0 = 0; g0 < groups; g0 += window) {
        f.group0 = static_cast<int32_t>(g0);
        f.groups = static_cast<int32_t>(groups - g0 < window ? groups - g0 : window);
        if (f.chunks > 0) {
            const dq4_status_t st = launch_fragments<OUT, kForward>(f, aligned, beside, cus, s);
            if (st != DQ4_OK)
                return st;
            beside = BesideWork{kNothing, {}};  // it went with the first window
        }
        p.groups = f.groups;
        p.n0 = g0 * sh.per_group();
        dq4_status_t st;
        if constexpr (kForward)
            st = sh.layout == kSideBySide ? launch_product<OUT, true>(p, plan, s)
                                          : launch_product<OUT, false>(p, plan, s);
        else
            st = launch_product<OUT, false>(p, plan, s);
        if (st != DQ4_OK)
            return st;
        p.dbias = nullptr;
    }
    return DQ4_OK;
}

template <int OUT>
const void *int8_fragments_kernel(bool aligned, Beside kind)
{
    if (kind == kSlopes8)
        return aligned ? reinterpret_cast<const void *>(&int8_column_fragments_kernel<OUT, true, kSlopes8>)
                       : reinterpret_cast<const void *>(&int8_column_fragments_kernel<OUT, false, kSlopes8>);
    if (kind == kSlopes1)
        return aligned ? reinterpret_cast<const void *>(&int8_column_fragments_kernel<OUT, true, kSlopes1>)
                       : reinterpret_cast<const void *>(&int8_column_fragments_kernel<OUT, false, kSlopes1>);
    return aligned ? reinterpret_cast<const void *>(&int8_column_fragments_kernel<OUT, true, kNothing>)
                   : reinterpret_cast<const void *>(&int8_column_fragments_kernel<OUT, false, kNothing>);
}

// Tokens up to which the columns are multiplied as they are decoded (whole calls, us, decode
// and product | this: 16 tokens, 11008 x 4096 56 | 17, 28672 x 8192 288 | 63; 64 tokens 60 |
// 27, 289 | 100; 128 tokens 63 | 46, 300 | 187, 1001 x 1377 17.4 | 17.0).
constexpr int64_t kInt8ColumnsMost = 128;

struct Int8ColumnPlan {
    int tf;
    int64_t slices, groups, steps, splits;
    int64_t bytes() const { return splits * groups * slices * kFrags * tf * kFragBytes; }
};

Int8ColumnPlan int8_column_plan(int64_t n_out, int64_t n_in, int64_t m, int cus)
{
    Int8ColumnPlan p{};
    p.tf = m <= 16 ? 1 : 2;
    p.slices = ceil_div(m, 16 * p.tf);
    p.groups = ceil_div(n_in, kGroup);
    p.steps = ceil_div(n_out, 32);
    // one workgroup per CU, each wave with a step at least
    p.splits = cus / (p.groups * p.slices);
    if (p.splits > ceil_div(p.steps, 8))
        p.splits = ceil_div(p.steps, 8);
    if (p.splits < 1)
        p.splits = 1;
    return p;
}

template <int OUT, int TF>
dq4_status_t run_int8_few(const Int8ColumnPlan &plan, Int8ColumnArgs a, ProductArgs p, hipStream_t s)
{
    const bool aligned = a.n_in % 8 == 0 && reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
    const bool vec = rows_aligned(a.dy, a.ld_dy, a.m, a.n_out);
    const void *kernel = aligned ? (vec ? reinterpret_cast<const void *>(&int8_columns_kernel<OUT, TF, true, true>)
                                        : reinterpret_cast<const void *>(&int8_columns_kernel<OUT, TF, true, false>))
                                 : (vec ? reinterpret_cast<const void *>(&int8_columns_kernel<OUT, TF, false, true>)
                                        : reinterpret_cast<const void *>(&int8_columns_kernel<OUT, TF, false, false>));
    a.steps = static_cast<int32_t>(plan.steps);
    a.slices = static_cast<int32_t>(plan.slices);
    a.splits = static_cast<int32_t>(plan.splits);
    const int64_t bias_rows = !a.dbias ? 0 : ceil_div(a.n_out, 512 * plan.groups);
    a.bias_rows = static_cast<int32_t>(bias_rows < 256 ? bias_rows : 256);
    void *params[] = {&a};
    const dq4_status_t st = launch(kernel, plan.groups, plan.splits * plan.slices + a.bias_rows, 512, params, s);
    if (st != DQ4_OK)
        return st;
    p.partial = a.partial;
    p.splits = a.splits;
    p.tiles_t = a.slices;
    p.groups = static_cast<int32_t>(plan.groups);
    int32_t tiles = static_cast<int32_t>(plan.groups * plan.slices);
    void *rp[] = {&p, &tiles};
    return launch(reinterpret_cast<const void *>(&product_reduce_kernel<OUT, false, 1, 1, TF>), tiles, TF, 256, rp, s);
}

// dx = dy W for an LLM.int8 weight: its columns to 16-bit fragments, then the
// product.
template <int OUT>
dq4_status_t run_int8_columns(const Shape &sh, const int8_t *codes, const float *scales, ProductArgs p,
                              BesideWork beside, uint8_t *ws, hipStream_t s)
{
    int device = 0;
    const hipError_t e = hipGetDevice(&device);
    if (e != hipSuccess)
        return hip_failed(e);
    const int cus = compute_units(device);
    const Plan plan = sh.plan(cus);
    if (beside.args.blocks > kMostBeside) {
        const dq4_status_t st = launch_fragments<OUT, false>(FragmentArgs{}, true, beside, cus, s);
        if (st != DQ4_OK)
            return st;
        beside = BesideWork{kNothing, {}};
    }
    p.m = sh.m;
    p.n = sh.n;
    p.splits = plan.splits;
    p.partial = reinterpret_cast<f32x4 *>(ws);
    p.n_x = 1;
    p.groups = static_cast<int32_t>(sh.groups());
    p.chunks = static_cast<int32_t>(sh.chunks());
    Int8FragmentArgs f{};
    f.codes = codes;
    f.scales = scales;
    f.out = reinterpret_cast<uint16_t *>(ws + sh.split_bytes(plan, sh.groups()));
    f.n_out = sh.k;
    f.n_in = sh.n;
    f.groups = p.groups;
    f.chunks = p.chunks;
    p.wfrag = f.out;
    if (f.chunks > 0) {
        const bool aligned = sh.n % 8 == 0 && reinterpret_cast<uintptr_t>(codes) % 8 == 0;
        void *params[] = {&f, &beside.args};
        const dq4_status_t st = launch(int8_fragments_kernel<OUT>(aligned, beside.kind),
                                       ceil_div(sh.groups(), 2) * f.chunks + beside.args.blocks, 1, kThreads, params, s);
        if (st != DQ4_OK)
            return st;
    }
    return launch_product<OUT, false>(p, plan, s);
}

template <int OUT, bool kTwo, int TF>
dq4_status_t launch_columns_tile(ColumnArgs a, hipStream_t s)
{
    const int64_t tiles = static_cast<int64_t>(a.out.groups) * a.slices;
    void *params[] = {&a};
    const dq4_status_t st =
        launch(reinterpret_cast<const void *>(&weight_columns_kernel<OUT, kTwo, TF>), a.out.groups,
               static_cast<int64_t>(a.splits) * a.slices + (a.out.dbias ? 1 : 0), 512, params, s);
    if (st != DQ4_OK)
        return st;
    ProductArgs p = a.out;
    p.splits = a.splits;
    p.tiles_t = a.slices;
    int32_t n_tiles = static_cast<int32_t>(tiles);
    void *rp[] = {&p, &n_tiles};
    return launch(reinterpret_cast<const void *>(&product_reduce_kernel<OUT, false, 1, 1, TF>), tiles, TF,
                  256, rp, s);
}

// dz's fragments and slopes, the product, the epilogue.
template <int OUT>
dq4_status_t run_columns(const ColumnPlan &plan, const dq4_weight_t *w0, const dq4_weight_t *w1,
                         int64_t n_out, int64_t n_in, int64_t m, int log2_block, ProductArgs p,
                         const BesideWork &beside, hipStream_t s)
{
    const dq4_status_t st = launch_fragments<OUT, false>(FragmentArgs{}, true, beside, 0, s);
    if (st != DQ4_OK)
        return st;
    p.m = m;
    p.n = n_in;
    p.groups = static_cast<int32_t>(plan.groups);
    ColumnArgs a{};
    a.w[0] = device_weight(*w0);
    a.w[1] = device_weight(w1 ? *w1 : *w0);
    a.n_out = n_out;
    a.n_in = n_in;
    a.log2_block = log2_block;
    a.steps = static_cast<int32_t>(plan.steps);
    a.splits = plan.splits;
    a.slices = plan.slices;
    a.dz_frags[0] = beside.args.slope.pad[0];
    a.dz_frags[1] = beside.args.slope.pad[1];
    a.out = p;
    if (plan.tf == 1)
        return w1 ? launch_columns_tile<OUT, true, 1>(a, s) : launch_columns_tile<OUT, false, 1>(a, s);
    return w1 ? launch_columns_tile<OUT, true, 2>(a, s) : launch_columns_tile<OUT, false, 2>(a, s);
}

// Sizes, type, activation and layout of a call; *empty when there is nothing
// to write.
dq4_status_t check_call(const dq4_weight_t *w0, const dq4_weight_t *w1, int64_t n_out,
                        int64_t n_in, int64_t m, int32_t dtype, int32_t act, bool gated,
                        int *log2_block)
{
    if (!w0 || (gated && !w1))
        return DQ4_EINVAL;
    if (dtype != DQ4_F16 && dtype != DQ4_BF16)
        return DQ4_EINVAL;
    const dq4_status_t st = validate_layout(w0->blocksize, w0->nested_blocksize, dtype, log2_block);
    if (st != DQ4_OK)
        return st;
    if (gated && (w1->blocksize != w0->blocksize || w1->nested_blocksize != w0->nested_blocksize))
        return DQ4_EUNSUPPORTED;
    if (n_out < 0 || n_in < 0 || m < 0)
        return DQ4_EINVAL;
    if (act < (gated ? DQ4_ACT_RELU : DQ4_ACT_NONE) || act > DQ4_ACT_GELU_TANH)
        return DQ4_EINVAL;
    if (n_out > kMaxDim || n_in > kMaxDim || m > kMaxDim || m * n_out > kMaxMatrix ||
        m * n_in > kMaxMatrix)
        return DQ4_EUNSUPPORTED;
    return DQ4_OK;
}

int64_t int8_backward_need(int64_t n_out, int64_t n_in, int64_t m, const void *dy, int64_t ld_dy)
{
    if (m <= kInt8ColumnsMost && n_in > 0)
        return int8_column_plan(n_out, n_in, m, current_compute_units()).bytes();
    const Shape s{m, n_in, n_out, kSingle};
    const bool copy = n_in > 0 && needs_copy(dy, ld_dy, m, n_out);
    return workspace_need(s, copy_bytes(s, copy) + partial_bytes(m, n_out), false);
}

bool sizes_ok(int64_t n_out, int64_t n_in, int64_t m)
{
    return n_out > 0 && n_in >= 0 && m > 0 && n_out <= kMaxDim && n_in <= kMaxDim && m <= kMaxDim &&
           m * n_out <= kMaxMatrix && m * n_in <= kMaxMatrix;
}

int64_t linear_backward_need(const dq4_weight_t *w, int64_t n_out, int64_t n_in, int64_t m,
                             const void *lhs, int64_t ld_lhs, bool least)
{
    const ColumnPlan cp = column_plan(w, nullptr, n_out, n_in, m, current_compute_units());
    if (cp.use)
        return partial_bytes(m, n_out) + cp.frag_bytes() + cp.partial_bytes();
    const Shape s{m, n_in, n_out, kSingle};
    const bool copy = n_in > 0 && needs_copy(lhs, ld_lhs, m, n_out);
    return workspace_need(s, copy_bytes(s, copy) + partial_bytes(m, n_out), least);
}

int64_t gated_backward_need(const dq4_weight_t *gate, const dq4_weight_t *up, int64_t n_ff,
                            int64_t n_in, int64_t m, const void *dgate, const void *dup,
                            int64_t ld_dpre, bool least)
{
    const ColumnPlan cp = column_plan(gate, up, n_ff, n_in, m, current_compute_units());
    if (cp.use)
        return 2 * cp.frag_bytes() + cp.partial_bytes();
    const Shape s{m, n_in, n_ff, kStacked};
    const bool copy = n_in > 0 && (needs_copy(dgate, ld_dpre, m, n_ff) || needs_copy(dup, ld_dpre, m, n_ff));
    return workspace_need(s, copy_bytes(s, copy), least);
}

}  // namespace
}  // namespace dq4

using namespace dq4;

extern "C" {

int64_t dq4_linear_fused_workspace_bytes(const dq4_weight_t *w, int64_t n_out, int64_t n_in,
                                         int64_t m, const void *x, int64_t ld_x, int32_t least)
{
    if (!w || !sizes_ok(n_out, n_in, m))
        return 0;
    const Shape s{m, n_out, n_in, kSingle};
    return forward_need(s, w, nullptr, forward_copies(s, w, nullptr, x, ld_x), least != 0);
}

int64_t dq4_gated_fused_workspace_bytes(const dq4_weight_t *gate, const dq4_weight_t *up,
                                        int64_t n_ff, int64_t n_in, int64_t m, const void *x,
                                        int64_t ld_x, int32_t least)
{
    if (!gate || !up || !sizes_ok(n_ff, n_in, m))
        return 0;
    const Shape s{m, n_ff, n_in, kSideBySide};
    return forward_need(s, gate, up, forward_copies(s, gate, up, x, ld_x), least != 0);
}

int64_t dq4_linear_fused_backward_workspace_bytes(const dq4_weight_t *w, int64_t n_out,
                                                  int64_t n_in, int64_t m, const void *dz,
                                                  int64_t ld_dz, int32_t least)
{
    if (!w || !sizes_ok(n_out, n_in, m))
        return 0;
    return linear_backward_need(w, n_out, n_in, m, dz, ld_dz, least != 0);
}

int64_t dq4_gated_fused_backward_workspace_bytes(const dq4_weight_t *gate,
                                                 const dq4_weight_t *up, int64_t n_ff,
                                                 int64_t n_in, int64_t m, const void *dgate,
                                                 const void *dup, int64_t ld_dpre,
                                                 int32_t least)
{
    if (!gate || !up || !sizes_ok(n_ff, n_in, m))
        return 0;
    return gated_backward_need(gate, up, n_ff, n_in, m, dgate, dup, ld_dpre, least != 0);
}

dq4_status_t dq4_linear_fused(const dq4_weight_t *w, int64_t n_out, int64_t n_in, int32_t dtype,
                              int32_t activation, const void *x, int64_t m, int64_t ld_x,
                              const void *bias, const void *residual, int64_t ld_residual,
                              void *y, int64_t ld_y, void *pre, int64_t ld_pre, void *workspace,
                              int64_t workspace_bytes, void *stream)
{
    int log2_block = 0;
    const dq4_status_t st = check_call(w, nullptr, n_out, n_in, m, dtype, activation, false, &log2_block);
    if (st != DQ4_OK)
        return st;
    if (m == 0 || n_out == 0)
        return DQ4_OK;
    if (!y || (n_in > 0 && (!x || weight_missing(w))))
        return DQ4_EINVAL;
    if (bad_ld(ld_x, m, n_in) || bad_ld(ld_y, m, n_out) || (residual && bad_ld(ld_residual, m, n_out)) ||
        (pre && bad_ld(ld_pre, m, n_out)))
        return DQ4_EINVAL;
    const Shape sh{m, n_out, n_in, kSingle};
    const bool copy = forward_copies(sh, w, nullptr, x, ld_x);
    const int64_t fixed = copy_bytes(sh, copy);
    if (workspace_bytes < forward_need(sh, w, nullptr, copy, true) ||
        bad_workspace(workspace, workspace_bytes))
        return DQ4_EINVAL;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    hipStream_t s = static_cast<hipStream_t>(stream);
    ProductArgs p{};
    p.x[0] = p.x[1] = static_cast<const uint16_t *>(x);
    p.ld_x = product_ld(ld_x, m, n_in);
    p.k = n_in;
    BesideWork beside{kNothing, {}};
    if (copy && n_in > 0) {
        beside = copy_work(x, ld_x, m, n_in, ws);
        p.x[0] = p.x[1] = reinterpret_cast<uint16_t *>(ws);
        p.ld_x = p.k = padded_ld(n_in);
    }
    p.act = activation;
    p.bias = static_cast<const uint16_t *>(bias);
    p.residual = static_cast<const uint16_t *>(residual);
    p.ld_residual = ld_residual;
    p.y = static_cast<uint16_t *>(y);
    p.ld_y = ld_y;
    p.pre[0] = static_cast<uint16_t *>(pre);
    p.ld_pre = ld_pre;
    p.vec = rows_aligned(y, ld_y, m, 8) && (!bias || reinterpret_cast<uintptr_t>(bias) % 16 == 0) &&
            (!residual || rows_aligned(residual, ld_residual, m, 8)) &&
            (!pre || rows_aligned(pre, ld_pre, m, 8));
    if (dtype == DQ4_F16)
        return run_product<DQ4_F16, true>(sh, w, nullptr, n_out, n_in, log2_block, p, beside, ws + fixed,
                                          workspace_bytes - fixed, s);
    return run_product<DQ4_BF16, true>(sh, w, nullptr, n_out, n_in, log2_block, p, beside, ws + fixed,
                                       workspace_bytes - fixed, s);
}

dq4_status_t dq4_gated_fused(const dq4_weight_t *gate, const dq4_weight_t *up, int64_t n_ff,
                             int64_t n_in, int32_t dtype, int32_t activation, const void *x,
                             int64_t m, int64_t ld_x, void *h, int64_t ld_h, void *gate_pre,
                             void *up_pre, int64_t ld_pre, void *workspace,
                             int64_t workspace_bytes, void *stream)
{
    int log2_block = 0;
    const dq4_status_t st = check_call(gate, up, n_ff, n_in, m, dtype, activation, true, &log2_block);
    if (st != DQ4_OK)
        return st;
    if (m == 0 || n_ff == 0)
        return DQ4_OK;
    if (!h || (n_in > 0 && (!x || weight_missing(gate) || weight_missing(up))))
        return DQ4_EINVAL;
    if ((gate_pre == nullptr) != (up_pre == nullptr))
        return DQ4_EINVAL;
    if (bad_ld(ld_x, m, n_in) || bad_ld(ld_h, m, n_ff) || (gate_pre && bad_ld(ld_pre, m, n_ff)))
        return DQ4_EINVAL;
    const Shape sh{m, n_ff, n_in, kSideBySide};
    const bool copy = forward_copies(sh, gate, up, x, ld_x);
    const int64_t fixed = copy_bytes(sh, copy);
    if (workspace_bytes < forward_need(sh, gate, up, copy, true) ||
        bad_workspace(workspace, workspace_bytes))
        return DQ4_EINVAL;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    hipStream_t s = static_cast<hipStream_t>(stream);
    ProductArgs p{};
    p.x[0] = p.x[1] = static_cast<const uint16_t *>(x);
    p.ld_x = product_ld(ld_x, m, n_in);
    p.k = n_in;
    BesideWork beside{kNothing, {}};
    if (copy && n_in > 0) {
        beside = copy_work(x, ld_x, m, n_in, ws);
        p.x[0] = p.x[1] = reinterpret_cast<uint16_t *>(ws);
        p.ld_x = p.k = padded_ld(n_in);
    }
    p.act = activation;
    p.y = static_cast<uint16_t *>(h);
    p.ld_y = ld_h;
    p.pre[0] = static_cast<uint16_t *>(gate_pre);
    p.pre[1] = static_cast<uint16_t *>(up_pre);
    p.ld_pre = ld_pre;
    p.vec = rows_aligned(h, ld_h, m, 8) && (!gate_pre || (rows_aligned(gate_pre, ld_pre, m, 8) &&
                                                          rows_aligned(up_pre, ld_pre, m, 8)));
    if (dtype == DQ4_F16)
        return run_product<DQ4_F16, true>(sh, gate, up, n_ff, n_in, log2_block, p, beside, ws + fixed,
                                          workspace_bytes - fixed, s);
    return run_product<DQ4_BF16, true>(sh, gate, up, n_ff, n_in, log2_block, p, beside, ws + fixed,
                                       workspace_bytes - fixed, s);
}

dq4_status_t dq4_linear_fused_backward(const dq4_weight_t *w, int64_t n_out, int64_t n_in,
                                       int32_t dtype, int32_t activation, const void *dy,
                                       int64_t m, int64_t ld_dy, const void *pre, int64_t ld_pre,
                                       void *dx, int64_t ld_dx, void *dz, int64_t ld_dz,
                                       float *dbias, void *workspace, int64_t workspace_bytes,
                                       void *stream)
{
    int log2_block = 0;
    const dq4_status_t st = check_call(w, nullptr, n_out, n_in, m, dtype, activation, false, &log2_block);
    if (st != DQ4_OK)
        return st;
    const bool act = activation != DQ4_ACT_NONE;
    if (!act && dz)
        return DQ4_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (m == 0) {  // empty sums
        if (!dbias || n_out == 0)
            return DQ4_OK;
        const float *none = nullptr;
        int64_t n = n_out;
        int32_t blocks = 0;
        void *params[] = {&none, &n, &blocks, &dbias};
        return launch(reinterpret_cast<const void *>(&bias_grad_reduce_kernel), ceil_div(n, kThreads),
                      1, kThreads, params, s);
    }
    if (n_out > 0 && (!dy || (act && (!pre || !dz)) || bad_ld(ld_dy, m, n_out) ||
                      (act && (bad_ld(ld_pre, m, n_out) || bad_ld(ld_dz, m, n_out)))))
        return DQ4_EINVAL;
    if (n_in > 0 && (!dx || bad_ld(ld_dx, m, n_in) || (n_out > 0 && weight_missing(w))))
        return DQ4_EINVAL;
    const Shape sh{m, n_in, n_out, kSingle};
    const void *lhs = act ? dz : dy;
    const int64_t ld_lhs = act ? ld_dz : ld_dy;
    const ColumnPlan cp = column_plan(w, nullptr, n_out, n_in, m, current_compute_units());
    const bool copy = cp.use || (n_in > 0 && needs_copy(lhs, ld_lhs, m, n_out));
    const int64_t copied = cp.use ? cp.frag_bytes() : copy_bytes(sh, copy);
    const int64_t fixed = copied + partial_bytes(m, n_out);
    if (n_out > 0 &&
        (workspace_bytes < linear_backward_need(w, n_out, n_in, m, lhs, ld_lhs, true) ||
         bad_workspace(workspace, workspace_bytes)))
        return DQ4_EINVAL;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    ProductArgs p{};
    p.x[0] = p.x[1] = static_cast<const uint16_t *>(lhs);
    p.ld_x = product_ld(ld_lhs, m, n_out);
    p.k = n_out;
    BesideWork beside{kNothing, {}};
    const int64_t blocks = ceil_div(m, kRowBlock);
    if (n_out > 0 && (act || dbias || copy)) {
        SlopeArgs a{};
        a.dy = static_cast<const uint16_t *>(dy);
        a.ld_dy = ld_dy;
        a.pre[0] = static_cast<const uint16_t *>(pre);
        a.ld_pre = ld_pre;
        a.dz[0] = static_cast<uint16_t *>(dz);
        a.ld_dz = ld_dz;
        if (copy) {
            a.pad[0] = reinterpret_cast<uint16_t *>(ws);
            a.ld_pad = cp.use ? cp.steps * 32 : padded_ld(n_out);
            a.pad_rows = cp.use ? cp.slices * 16 * cp.tf : m;
            a.frag_rows = cp.use ? cp.tf : 0;
            p.x[0] = p.x[1] = a.pad[0];
            p.ld_x = p.k = a.ld_pad;
        }
        a.partial = !dbias ? nullptr : blocks == 1 ? dbias : reinterpret_cast<float *>(ws + copied);
        a.m = m;
        a.n = n_out;
        a.act = activation;
        beside = slope_work(a, false);
        if (dbias && blocks > 1) {
            p.bias_partial = a.partial;
            p.bias_n = n_out;
            p.bias_blocks = static_cast<int32_t>(blocks);
            p.dbias = dbias;
        }
    }
    if (n_in == 0) {  // no product: the slopes and the bias gradient alone
        if (beside.kind == kNothing)
            return DQ4_OK;
        const dq4_status_t ls =
            dtype == DQ4_F16 ? launch_fragments<DQ4_F16, false>(FragmentArgs{}, true, beside, 0, s)
                             : launch_fragments<DQ4_BF16, false>(FragmentArgs{}, true, beside, 0, s);
        if (ls != DQ4_OK || !p.dbias)
            return ls;
        void *rp[] = {&p.bias_partial, &p.bias_n, &p.bias_blocks, &p.dbias};
        return launch(reinterpret_cast<const void *>(&bias_grad_reduce_kernel),
                      ceil_div(n_out, kThreads), 1, kThreads, rp, s);
    }
    p.act = DQ4_ACT_NONE;
    p.y = static_cast<uint16_t *>(dx);
    p.ld_y = ld_dx;
    p.vec = rows_aligned(dx, ld_dx, m, 8);
    if (cp.use) {
        p.partial = reinterpret_cast<f32x4 *>(ws + fixed);
        return dtype == DQ4_F16
                   ? run_columns<DQ4_F16>(cp, w, nullptr, n_out, n_in, m, log2_block, p, beside, s)
                   : run_columns<DQ4_BF16>(cp, w, nullptr, n_out, n_in, m, log2_block, p, beside, s);
    }
    if (dtype == DQ4_F16)
        return run_product<DQ4_F16, false>(sh, w, nullptr, n_out, n_in, log2_block, p, beside, ws + fixed,
                                           workspace_bytes - fixed, s);
    return run_product<DQ4_BF16, false>(sh, w, nullptr, n_out, n_in, log2_block, p, beside, ws + fixed,
                                        workspace_bytes - fixed, s);
}

dq4_status_t dq4_gated_fused_backward(const dq4_weight_t *gate, const dq4_weight_t *up,
                                      int64_t n_ff, int64_t n_in, int32_t dtype,
                                      int32_t activation, const void *dh, int64_t m,
                                      int64_t ld_dh, const void *gate_pre, const void *up_pre,
                                      int64_t ld_pre, void *dx, int64_t ld_dx, void *dgate,
                                      void *dup, int64_t ld_dpre, void *workspace,
                                      int64_t workspace_bytes, void *stream)
{
    int log2_block = 0;
    const dq4_status_t st = check_call(gate, up, n_ff, n_in, m, dtype, activation, true, &log2_block);
    if (st != DQ4_OK)
        return st;
    if (m == 0)
        return DQ4_OK;
    if (n_ff > 0 && (!dh || !gate_pre || !up_pre || !dgate || !dup || bad_ld(ld_dh, m, n_ff) ||
                     bad_ld(ld_pre, m, n_ff) || bad_ld(ld_dpre, m, n_ff)))
        return DQ4_EINVAL;
    if (n_in > 0 && (!dx || bad_ld(ld_dx, m, n_in) ||
                     (n_ff > 0 && (weight_missing(gate) || weight_missing(up)))))
        return DQ4_EINVAL;
    const Shape sh{m, n_in, n_ff, kStacked};
    const ColumnPlan cp = column_plan(gate, up, n_ff, n_in, m, current_compute_units());
    const bool copy = cp.use || (n_in > 0 && (needs_copy(dgate, ld_dpre, m, n_ff) ||
                                              needs_copy(dup, ld_dpre, m, n_ff)));
    const int64_t fixed = cp.use ? 2 * cp.frag_bytes() : copy_bytes(sh, copy);
    if (n_ff > 0 && (workspace_bytes < gated_backward_need(gate, up, n_ff, n_in, m, dgate, dup, ld_dpre, true) ||
                     bad_workspace(workspace, workspace_bytes)))
        return DQ4_EINVAL;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    hipStream_t s = static_cast<hipStream_t>(stream);
    ProductArgs p{};
    p.x[0] = static_cast<const uint16_t *>(dgate);
    p.x[1] = static_cast<const uint16_t *>(dup);
    p.ld_x = product_ld(ld_dpre, m, n_ff);
    p.k = n_ff;
    BesideWork beside{kNothing, {}};
    if (n_ff > 0) {
        SlopeArgs a{};
        a.dy = static_cast<const uint16_t *>(dh);
        a.ld_dy = ld_dh;
        a.pre[0] = static_cast<const uint16_t *>(gate_pre);
        a.pre[1] = static_cast<const uint16_t *>(up_pre);
        a.ld_pre = ld_pre;
        a.dz[0] = static_cast<uint16_t *>(dgate);
        a.dz[1] = static_cast<uint16_t *>(dup);
        a.ld_dz = ld_dpre;
        if (copy) {
            a.ld_pad = cp.use ? cp.steps * 32 : padded_ld(n_ff);
            a.pad_rows = cp.use ? cp.slices * 16 * cp.tf : m;
            a.frag_rows = cp.use ? cp.tf : 0;
            a.pad[0] = reinterpret_cast<uint16_t *>(ws);
            a.pad[1] = reinterpret_cast<uint16_t *>(ws + fixed / 2);
            p.x[0] = a.pad[0];
            p.x[1] = a.pad[1];
            p.ld_x = p.k = a.ld_pad;
        }
        a.m = m;
        a.n = n_ff;
        a.act = activation;
        beside = slope_work(a, true);
    }
    if (n_in == 0) {  // no product: the slopes alone
        if (beside.kind == kNothing)
            return DQ4_OK;
        return dtype == DQ4_F16
                   ? launch_fragments<DQ4_F16, false>(FragmentArgs{}, true, beside, 0, s)
                   : launch_fragments<DQ4_BF16, false>(FragmentArgs{}, true, beside, 0, s);
    }
    p.act = DQ4_ACT_NONE;
    p.y = static_cast<uint16_t *>(dx);
    p.ld_y = ld_dx;
    p.vec = rows_aligned(dx, ld_dx, m, 8);
    if (cp.use) {
        p.partial = reinterpret_cast<f32x4 *>(ws + fixed);
        return dtype == DQ4_F16
                   ? run_columns<DQ4_F16>(cp, gate, up, n_ff, n_in, m, log2_block, p, beside, s)
                   : run_columns<DQ4_BF16>(cp, gate, up, n_ff, n_in, m, log2_block, p, beside, s);
    }
    if (dtype == DQ4_F16)
        return run_product<DQ4_F16, false>(sh, gate, up, n_ff, n_in, log2_block, p, beside, ws + fixed,
                                           workspace_bytes - fixed, s);
    return run_product<DQ4_BF16, false>(sh, gate, up, n_ff, n_in, log2_block, p, beside, ws + fixed,
                                        workspace_bytes - fixed, s);
}

int64_t dq4_int8_linear_backward_workspace_bytes(int64_t n_out, int64_t n_in, int64_t m, const void *dy,
                                                 int64_t ld_dy)
{
    if (!sizes_ok(n_out, n_in, m))
        return 0;
    return int8_backward_need(n_out, n_in, m, dy, ld_dy);
}

dq4_status_t dq4_int8_linear_backward(const int8_t *CB, const float *SCB, int64_t n_out, int64_t n_in,
                                      int32_t dtype, const void *dy, int64_t m, int64_t ld_dy, void *dx,
                                      int64_t ld_dx, float *dbias, void *workspace, int64_t workspace_bytes,
                                      void *stream)
{
    if (n_out < 0 || n_in < 0 || m < 0 || (dtype != DQ4_F16 && dtype != DQ4_BF16))
        return DQ4_EINVAL;
    if (n_out > kMaxDim || n_in > kMaxDim || m > kMaxDim || m * n_out > kMaxMatrix / 2 ||
        m * n_in > kMaxMatrix / 2)
        return DQ4_EUNSUPPORTED;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (m == 0) {  // empty sums
        if (!dbias || n_out == 0)
            return DQ4_OK;
        const float *none = nullptr;
        int64_t n = n_out;
        int32_t blocks = 0;
        void *params[] = {&none, &n, &blocks, &dbias};
        return launch(reinterpret_cast<const void *>(&bias_grad_reduce_kernel), ceil_div(n, kThreads), 1,
                      kThreads, params, s);
    }
    if (n_out > 0 && (!dy || bad_ld(ld_dy, m, n_out)))
        return DQ4_EINVAL;
    if (n_in > 0 && (!dx || bad_ld(ld_dx, m, n_in) || (n_out > 0 && (!CB || !SCB))))
        return DQ4_EINVAL;
    if (n_out > 0 && (workspace_bytes < int8_backward_need(n_out, n_in, m, dy, ld_dy) ||
                      bad_workspace(workspace, workspace_bytes)))
        return DQ4_EINVAL;
    const Shape sh{m, n_in, n_out, kSingle};
    const bool copy = n_in > 0 && needs_copy(dy, ld_dy, m, n_out);
    const int64_t copied = copy_bytes(sh, copy), fixed = copied + partial_bytes(m, n_out);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    ProductArgs p{};
    if (m <= kInt8ColumnsMost && n_in > 0 && n_out > 0) {
        const Int8ColumnPlan plan = int8_column_plan(n_out, n_in, m, current_compute_units());
        p.m = m;
        p.n = n_in;
        p.act = DQ4_ACT_NONE;
        p.y = static_cast<uint16_t *>(dx);
        p.ld_y = ld_dx;
        p.vec = rows_aligned(dx, ld_dx, m, 8);
        Int8ColumnArgs a{CB, SCB, static_cast<const uint16_t *>(dy), ld_dy, n_out, n_in, m, 0, 0, 0, 0,
                         reinterpret_cast<f32x4 *>(ws), dbias};
        if (plan.tf == 1)
            return dtype == DQ4_F16 ? run_int8_few<DQ4_F16, 1>(plan, a, p, s) : run_int8_few<DQ4_BF16, 1>(plan, a, p, s);
        return dtype == DQ4_F16 ? run_int8_few<DQ4_F16, 2>(plan, a, p, s) : run_int8_few<DQ4_BF16, 2>(plan, a, p, s);
    }
    p.x[0] = p.x[1] = static_cast<const uint16_t *>(dy);
    p.ld_x = product_ld(ld_dy, m, n_out);
    p.k = n_out;
    BesideWork beside{kNothing, {}};
    const int64_t blocks = ceil_div(m, kRowBlock);
    if (n_out > 0 && (dbias || copy)) {
        SlopeArgs a{};
        a.dy = static_cast<const uint16_t *>(dy);
        a.ld_dy = ld_dy;
        if (copy) {
            a.pad[0] = reinterpret_cast<uint16_t *>(ws);
            a.ld_pad = padded_ld(n_out);
            a.pad_rows = m;
            p.x[0] = p.x[1] = a.pad[0];
            p.ld_x = p.k = a.ld_pad;
        }
        a.partial = !dbias ? nullptr : blocks == 1 ? dbias : reinterpret_cast<float *>(ws + copied);
        a.m = m;
        a.n = n_out;
        a.act = DQ4_ACT_NONE;
        beside = slope_work(a, false);
        if (dbias && blocks > 1) {
            p.bias_partial = a.partial;
            p.bias_n = n_out;
            p.bias_blocks = static_cast<int32_t>(blocks);
            p.dbias = dbias;
        }
    }
    if (n_in == 0) {  // no product: the bias gradient alone
        if (beside.kind == kNothing)
            return DQ4_OK;
        const dq4_status_t st =
            dtype == DQ4_F16 ? launch_fragments<DQ4_F16, false>(FragmentArgs{}, true, beside, 0, s)
                             : launch_fragments<DQ4_BF16, false>(FragmentArgs{}, true, beside, 0, s);
        if (st != DQ4_OK || !p.dbias)
            return st;
        void *rp[] = {&p.bias_partial, &p.bias_n, &p.bias_blocks, &p.dbias};
        return launch(reinterpret_cast<const void *>(&bias_grad_reduce_kernel), ceil_div(n_out, kThreads), 1,
                      kThreads, rp, s);
    }
    p.act = DQ4_ACT_NONE;
    p.y = static_cast<uint16_t *>(dx);
    p.ld_y = ld_dx;
    p.vec = rows_aligned(dx, ld_dx, m, 8);
    return dtype == DQ4_F16 ? run_int8_columns<DQ4_F16>(sh, CB, SCB, p, beside, ws + fixed, s)
                            : run_int8_columns<DQ4_BF16>(sh, CB, SCB, p, beside, ws + fixed, s);
}

}  // extern "C"

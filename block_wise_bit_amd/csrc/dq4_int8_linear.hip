// dq4_int8_linear.hip -- the LLM.int8 linear layer (include/dq4_int8.h): tokens
// quantized to 8-bit codes, and the product of the codes with a scale for each
// token and channel, the outlier columns in 16 bits.  (Its gradient is in
// dq4_linear_fused.hip: up to 128 tokens the weight's columns are multiplied as they
// are decoded, beyond it is a product over a 16-bit copy of the weight.)
//
// The sum of a product is one of 8-bit integers in 32 bits, exact in any order,
// on v_mfma_i32_16x16x64_i8: D (16 x 16) += A (16 x 64) B (64 x 16).  Lane l
// holds A[l % 16][16 (l / 16) .. + 15] and the same of B's columns, one 16-byte
// register quad each, and D[4 (l / 16) + i][l % 16] for i = 0 .. 3.  A is the
// weight (16 output columns), B the codes (16 tokens).
//
// LDS layout of such a fragment: 1 KiB, 16 rows of 64 bytes, the 16-byte piece p
// of row r in slot 4 r + (p ^ turn(r / 4)), turn = 0, 2, 3, 1.  A load takes 64
// neighbouring bytes of a row with a quad of lanes straight to LDS, lane l to slot
// l.  Of a wave's 16-byte LDS reads 16 lanes are served together, and they have to
// lie in 16 different slots of a 256-byte line.  With this turn they do, whether
// those are 16 lanes in a row or quads of two pieces (with turn(q) = q a product
// lost 17 % of its cycles to bank conflicts).
//
// Few tokens (up to 32 or 64): int8_rows_kernel, the weight read once.  More:
// int8_product_kernel, tiles of both operands in LDS.

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "dq4.h"
#include "dq4_device.h"
#include "dq4_int8.h"
#include "dq4_linear_device.h"

#pragma clang fp contract(off)

namespace dq4 {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int kFragBytes = 1024;
constexpr int kStep = 64;                     // k per matrix instruction
constexpr int kXcds = 8;
constexpr int64_t kMaxDim = int64_t{1} << 21, kMaxMatrix = int64_t{1} << 38;
// 128 * 128 * kMaxSum stays below 2^31.
constexpr int64_t kMaxSum = (int64_t{1} << 17) - 1;
constexpr float kR127 = 0x1.020408p-7f;       // the FP32 value nearest 1/127
constexpr float kR16129 = 1.0f / 16129.0f;    // 1 / 127^2
constexpr uint32_t kPast = 0x80000000u;       // an offset past every buffer

// ---------------------------------------------------------------------------
// quantization
// ---------------------------------------------------------------------------
struct QuantArgs {
    const uint16_t *x;
    int64_t m, k, ld_x;
    uint32_t limit;       // the least 15-bit pattern of a magnitude at the threshold
    uint32_t non_finite;  // T's infinity
    int8_t *codes;
    int64_t ld_codes;
    float *scales;
    int32_t *outliers;    // null: no threshold
    uint8_t *flags;       // one byte a column, 0 before the rows are read
    int32_t vec_in, vec_out;
};

// The code of x in a row of scale s: round(127 x / s), half to even.  x and s are
// multiplied by `up`, a power of two that keeps what follows inside FP32's normal
// range.  The quotient is at most 127 and its FP32 value within 3e-5, so only the
// whole numbers next to it come into question, and the remainder 127 x - q s,
// exact in FP32 (127 x has 18 bits, q s 19, and both are multiples of x's last
// place where q is not 0), decides.
__device__ __forceinline__ int code_of(float x, float up, float s, float inv)
{
    const float xs = x * up;
    float q = __builtin_rintf(xs * inv);
    const float r = 127.0f * xs - q * s;
    const float twice = 2.0f * __builtin_fabsf(r);
    const int odd = static_cast<int>(q) & 1;
    const bool move = twice > s || (twice == s && odd);
    q = q + (move ? __builtin_copysignf(1.0f, r) : 0.0f);
    return static_cast<int>(q);
}

// A row of x per workgroup and turn: its scale, then its codes.  A thread holds up
// to kHeld pieces of 8 elements between the two, the rest is read again.  Bound by
// memory's latency, which a workgroup waits for twice a row with nothing else in flight:
// 2 bytes read and 1 written per element, 4096 x 4096 18 us (2.8 TB/s); a wave per row
// took 21.  (kHeld is one for all widths, 8192 elements: 5 waves a SIMD; with two pieces,
// enough for 4096, the registers would allow 8.)
// kOne: the only row, by one workgroup, which also makes the list of outliers.
constexpr int kHeld = 4;

template <int OUT, bool kOne>
__global__ __launch_bounds__(kOne ? 1024 : 256) void int8_quant_rows_kernel(QuantArgs a)
{
    constexpr int THREADS = kOne ? 1024 : 256;
    constexpr int kWords = kOne ? (kMaxSum + 31) / 32 : 1;
    __shared__ uint32_t peaks[2][THREADS / 64];
    __shared__ uint32_t flagged[kWords];
    __shared__ int sums[THREADS / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int k = static_cast<int>(a.k);
    if constexpr (kOne) {
        for (int i = tid; i < kWords; i += THREADS)
            flagged[i] = 0;
        __syncthreads();
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x, turn ^= 1) {
        const uint16_t *x = a.x + row * a.ld_x;
        auto load = [&](int c) {
            u32x4 q = {0, 0, 0, 0};
            if (a.vec_in) {
                q = *reinterpret_cast<const u32x4 *>(x + c);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < k)
                        q[j / 2] |= static_cast<uint32_t>(x[c + j]) << (16 * (j & 1));
            }
            return q;
        };
        uint32_t peak = 0;
        auto look = [&](const u32x4 &q, int c) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = (q[j / 2] >> (16 * (j & 1))) & 0x7FFFu;
                if (b >= a.limit) {  // not below the threshold (a NaN is not)
                    if constexpr (kOne)
                        atomicOr(&flagged[(c + j) >> 5], 1u << ((c + j) & 31));
                    else
                        a.flags[c + j] = 1;
                } else {
                    peak = b > peak ? b : peak;
                }
            }
        };
        u32x4 held[kHeld];
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            const int c = (h * THREADS + tid) * 8;
            held[h] = u32x4{0, 0, 0, 0};
            if (c < k)
                held[h] = load(c);
        }
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            const int c = (h * THREADS + tid) * 8;
            if (c < k)
                look(held[h], c);
        }
        for (int c = (kHeld * THREADS + tid) * 8; c < k; c += THREADS * 8)
            look(load(c), c);
#pragma unroll
        for (int d = 32; d > 0; d /= 2) {
            const uint32_t other = __shfl_xor(peak, d);
            peak = other > peak ? other : peak;
        }
        if (lane == 0)
            peaks[turn][wave] = peak;
        __syncthreads();  // the next row's peaks go to the other half
#pragma unroll
        for (int w = 0; w < THREADS / 64; ++w)
            peak = peaks[turn][w] > peak ? peaks[turn][w] : peak;
        float scale = Half<OUT>::widen(peak);
        if (peak >= a.non_finite)
            scale = __builtin_nanf("");
        if (tid == 0)
            a.scales[row] = scale;
        const bool none = peak == 0 || peak >= a.non_finite;
        const float up = scale < 0x1p-100f ? 0x1p64f : scale > 0x1p100f ? 0x1p-64f : 1.0f;
        const float s = scale * up;
        const float inv = 127.0f * __builtin_amdgcn_rcpf(s);
        int8_t *codes = a.codes + row * a.ld_codes;
        auto write = [&](const u32x4 &q, int c) {
            uint32_t out[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = (q[j / 2] >> (16 * (j & 1))) & 0xFFFFu;
                const bool zero = none || (b & 0x7FFFu) >= a.limit;
                const int code = zero ? 0 : code_of(Half<OUT>::widen(b), up, s, inv);
                out[j / 4] |= (static_cast<uint32_t>(code) & 0xFFu) << (8 * (j & 3));
            }
            if (a.vec_out) {
                *reinterpret_cast<u32x2 *>(codes + c) = u32x2{out[0], out[1]};
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < k)
                        codes[c + j] = static_cast<int8_t>(out[j / 4] >> (8 * (j & 3)));
            }
        };
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            const int c = (h * THREADS + tid) * 8;
            if (c < k)
                write(held[h], c);
        }
        for (int c = (kHeld * THREADS + tid) * 8; c < k; c += THREADS * 8)
            write(load(c), c);
    }
    if constexpr (kOne) {
        if (!a.outliers)
            return;
        // (the flags are complete: every thread passed the row's barrier)
        int count = 0;
        uint32_t word[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            word[q] = 4 * tid + q < kWords ? flagged[4 * tid + q] : 0;
            count += __builtin_popcount(word[q]);
        }
        int total;
        int at = list_position<THREADS>(count, &total, sums);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            for (uint32_t w = word[q]; w; w &= w - 1)
                a.outliers[1 + at++] = (4 * tid + q) * 32 + __builtin_ctz(w);
        for (int i = total + tid; i < k; i += THREADS)
            a.outliers[1 + i] = -1;
        if (tid == 0)
            a.outliers[0] = total;
    }
}

__global__ __launch_bounds__(256) void int8_flags_zero_fill(uint32_t *flags, int32_t words)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < words)
        flags[i] = 0;
}

// The flagged columns: workgroup 0 lists them, the others set their codes to zero
// in the rows blockIdx.x - 1, ... .
constexpr int kListed = 4096;  // columns looked at in one go

__global__ __launch_bounds__(1024) void int8_outliers_zero_fill(QuantArgs a)
{
    __shared__ int sums[16];
    __shared__ int list[kListed];
    const int tid = threadIdx.x;
    const int k = static_cast<int>(a.k);
    int before = 0;
    for (int c0 = 0; c0 < k; c0 += kListed) {
        // the flags behind column k - 1 are zero
        const int c = c0 + 4 * tid;
        const uint32_t word = c < k ? *reinterpret_cast<const uint32_t *>(a.flags + c) : 0;
        int total;
        int at = list_position<1024>(__builtin_popcount(word), &total, sums);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if ((word >> (8 * j)) & 1)
                list[at++] = c + j;
        __syncthreads();
        if (blockIdx.x == 0) {
            for (int i = tid; i < total; i += 1024)
                a.outliers[1 + before + i] = list[i];
        } else if (total > 0) {
            // 32 threads a row
            const int64_t step = gridDim.x - 1;
            for (int64_t row = blockIdx.x - 1 + (tid >> 5) * step; row < a.m; row += 32 * step)
                for (int i = tid & 31; i < total; i += 32)
                    a.codes[row * a.ld_codes + list[i]] = 0;
        }
        before += total;
        __syncthreads();
    }
    if (blockIdx.x == 0) {
        for (int i = before + tid; i < k; i += 1024)
            a.outliers[1 + i] = -1;
        if (tid == 0)
            a.outliers[0] = before;
    }
}

// ---------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------
struct Int8Args {
    const int8_t *codes;
    int64_t ld_codes;
    const float *scales;
    const int8_t *w;
    int64_t ld_w;
    const float *w_scales;
    int64_t m, n;
    int32_t k;                  // bytes of a row to read, zeros behind column n_in included
    int32_t n_in;
    const uint16_t *x;          // of the outlier columns
    int64_t ld_x;
    const int32_t *outliers;    // null: none
    const uint16_t *w_outliers, *x_outliers;  // fragments of the first kOutlierChunks * 32 of them
    const uint16_t *bias, *residual;
    int64_t ld_residual;
    uint16_t *y;
    int64_t ld_y;
    int32_t vec;                // bias, residual and y take whole vectors
    int32_t rows_per, rows_extra;  // weight rows of a workgroup; the first ones take one more
    int32_t tiles_n, tiles_t;
    int32_t splits;             // of the steps of k; above 1 the sums go to `partial`
    i32x4 *partial;             // [split][tile][wave][fragment][16 tokens][lane]
};

__device__ __forceinline__ i32x4 mfma_i8(u32x4 a, u32x4 b, i32x4 c)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                                 __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

__device__ __forceinline__ int turn(int q)
{
    return (0x78 >> (2 * q)) & 3;
}

// Byte of piece `g` of row `r` in a fragment in LDS.
__device__ __forceinline__ uint32_t piece_at(int r, int g)
{
    return static_cast<uint32_t>(4 * r + (g ^ turn(r >> 2))) * 16;
}

// The piece that lane l loads, of row l / 4.
__device__ __forceinline__ int piece_of(int lane)
{
    return (lane & 3) ^ turn(lane >> 4);
}

// --- outlier columns ---------------------------------------------------------
// They enter through the 16-bit matrix instruction, on the FP32 value of the
// integer sum: 32 of them a chunk.  With more than 16 tokens their operands are
// gathered once per call into fragments (int8_outlier_fragments_kernel) for the
// first 128 columns; with up to 16 the row kernel gathers two chunks itself while
// it multiplies, and saves the launch.  Columns beyond are gathered where they are
// used, which is slow but needs no memory: at a threshold of 6, models have a few
// dozen.
constexpr int kOutlierChunks = 4;

__device__ __forceinline__ int outlier_count(const Int8Args &a)
{
    if (!a.outliers)
        return 0;
    const int c = a.outliers[0];
    return c < 0 ? 0 : c > a.n_in ? a.n_in : c;
}

template <int OUT>
constexpr uint32_t kNan = OUT == DQ4_F16 ? 0x7E00u : 0x7FC0u;

// A lane's 8 columns of a chunk: kNone past the last one, kBad for an index that is
// no column.  (All loads without branches, so that they are under way together.)
constexpr int kNone = -1, kBad = -2;

struct Columns {
    int c[8];
};

__device__ __forceinline__ Columns load_columns(const Int8Args &a, int l0, int count)
{
    Columns q;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = a.outliers[1 + (l0 + j < a.n_in ? l0 + j : a.n_in - 1)];
        q.c[j] = l0 + j >= count ? kNone : c < 0 || c >= a.n_in ? kBad : c;
    }
    return q;
}

// The codes W[n][c] is made of, and it; zeros past the last row.
struct Codes {
    int8_t b[8];
    float s;
};

__device__ __forceinline__ Codes load_codes(const Int8Args &a, int64_t n, const Columns &q)
{
    Codes w;
    const int64_t row = n < a.n ? n : 0;
    w.s = a.w_scales[row];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        w.b[j] = a.w[row * a.ld_w + (q.c[j] < 0 ? 0 : q.c[j])];
    return w;
}

template <int OUT>
__device__ __forceinline__ u32x4 weight_fragment(const Int8Args &a, int64_t n, const Columns &q, const Codes &w)
{
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float scaled = static_cast<float>(w.b[j]) * w.s;
        v[j] = Half<OUT>::pack2(scaled * kR127, 0.0f) & 0xFFFFu;
        v[j] = q.c[j] == kNone || n >= a.n ? 0u : q.c[j] == kBad ? kNan<OUT> : v[j];
    }
    return u32x4{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
}

template <int OUT>
__device__ __forceinline__ u32x4 x_fragment(const Int8Args &a, int64_t t, const Columns &q)
{
    const int64_t row = t < a.m ? t : 0;
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = a.x[row * a.ld_x + (q.c[j] < 0 ? 0 : q.c[j])];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = q.c[j] == kNone || t >= a.m ? 0u : q.c[j] == kBad ? kNan<OUT> : v[j];
    return u32x4{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
}

// Row (output column) of lane row r of weight fragment f: kWide as the product's
// tiles take them, 8 r + f of 128; else 16 in a row.
template <bool kWide>
__device__ __forceinline__ int64_t fragment_row(int64_t f, int r)
{
    return kWide ? (f >> 3) * 128 + 8 * r + (f & 7) : f * 16 + r;
}

// A wave gathers one chunk of one fragment of 16 rows: of the weight, or of x.
template <int OUT, bool kWide>
__global__ __launch_bounds__(256) void int8_outlier_fragments_kernel(Int8Args a, int64_t w_frags,
                                                                     int64_t x_frags, uint16_t *out)
{
    const int lane = threadIdx.x & 63;
    const int count = outlier_count(a);
    const int chunks = (count + 31) / 32 < kOutlierChunks ? (count + 31) / 32 : kOutlierChunks;
    const int64_t items = (w_frags + x_frags) * kOutlierChunks;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); i < items;
         i += static_cast<int64_t>(gridDim.x) * 4) {
        const int64_t f = i / kOutlierChunks;
        const int c = static_cast<int>(i % kOutlierChunks);
        if (c >= chunks)
            continue;
        const Columns q = load_columns(a, 32 * c + 8 * (lane >> 4), count);
        u32x4 v;
        if (f < w_frags) {
            const int64_t n = fragment_row<kWide>(f, lane & 15);
            v = weight_fragment<OUT>(a, n, q, load_codes(a, n, q));
        } else {
            v = x_fragment<OUT>(a, (f - w_frags) * 16 + (lane & 15), q);
        }
        *reinterpret_cast<u32x4 *>(out + (i * 64 + lane) * 8) = v;
    }
}

// One column after the other: the tiles' epilogue has no registers for more.
template <int OUT>
__device__ __forceinline__ uint32_t weight_value(const Int8Args &a, int64_t n, int c)
{
    if (n >= a.n)
        return 0;
    const float scaled = static_cast<float>(a.w[n * a.ld_w + c]) * a.w_scales[n];
    return Half<OUT>::pack2(scaled * kR127, 0.0f) & 0xFFFFu;
}

template <int OUT>
__device__ __forceinline__ uint32_t x_value(const Int8Args &a, int64_t t, int c)
{
    return t < a.m ? a.x[t * a.ld_x + c] : 0u;
}

template <int OUT, class Value>
__device__ __forceinline__ u32x4 gather_slowly(const Int8Args &a, int l0, int count, Value value)
{
    uint64_t q[2] = {0, 0};
#pragma unroll 1
    for (int j = 0; j < 8 && l0 + j < count; ++j) {
        const int c = a.outliers[1 + l0 + j];
        const uint64_t v = c < 0 || c >= a.n_in ? kNan<OUT> : value(c);
        q[0] |= j < 4 ? v << (16 * j) : 0;
        q[1] |= j < 4 ? 0 : v << (16 * (j - 4));
    }
    return u32x4{static_cast<uint32_t>(q[0]), static_cast<uint32_t>(q[0] >> 32), static_cast<uint32_t>(q[1]),
                 static_cast<uint32_t>(q[1] >> 32)};
}

// Chunk c of fragment f that int8_outlier_fragments_kernel wrote.
__device__ __forceinline__ u32x4 held_fragment(const uint16_t *frags, int64_t f, int c, int lane)
{
    return *reinterpret_cast<const u32x4 *>(frags + ((f * kOutlierChunks + c) * 64 + lane) * 8);
}

// --- the epilogue --------------------------------------------------------------
// A token's scale s as two factors, 2^a / 127^2 and s / 2^a, a its exponent held to
// [-100, 100].  The sum's value is sum (2^a / 127^2) S (s / 2^a), in this order.  sum /
// 127^2 is 0 or lies between 2^-14 and 2^17, so the first product is normal.  The next
// is the value over s / 2^a, which lies in [1, 2) unless s is beyond 2^+-100: there
// s / 2^a >= 1 (or <= 1) moves the product away from overflow (underflow), and S alone
// cannot reach the other end.  So no step leaves FP32's range where the value does not
// (with s itself as the last factor, large S gave infinities and small S lost bits that
// s brings back), at no cost per output: fractions and exponents of both scales took
// 2 % longer for 4096 tokens, 11008 x 4096.
struct TokenScale {
    float first, last;
};

__device__ __forceinline__ TokenScale token_scale(float s)
{
    const int e = static_cast<int>((__builtin_bit_cast(uint32_t, s) >> 23) & 255) - 127;
    const int a = e < -100 ? -100 : e > 100 ? 100 : e;
    return TokenScale{__builtin_ldexpf(kR16129, a), __builtin_ldexpf(s, -a)};
}

__device__ __forceinline__ float scaled_sum(int sum, float w_scale, const TokenScale &s)
{
    return static_cast<float>(sum) * s.first * w_scale * s.last;
}

// Bias, residual and the rounding of N neighbouring outputs, up to column last - 1.
template <int OUT, int N>
__device__ __forceinline__ void finish(const Int8Args &a, int64_t row, int64_t n0, int64_t last, float (&z)[N])
{
    const int64_t left = last - n0;
    if (row >= a.m || left <= 0)
        return;
    const int valid = left < N ? static_cast<int>(left) : N;
    const bool vec = a.vec && valid == N && n0 % N == 0;
    float v[N];
    if (a.bias) {
        load_values<OUT, N>(a.bias + n0, vec, valid, v);
#pragma unroll
        for (int j = 0; j < N; ++j)
            z[j] = z[j] + v[j];
    }
    if (a.residual) {
        load_values<OUT, N>(a.residual + row * a.ld_residual + n0, vec, valid, v);
#pragma unroll
        for (int j = 0; j < N; ++j)
            z[j] = z[j] + v[j];
    }
    store_values<OUT, N>(a.y + row * a.ld_y + n0, vec, valid, z);
}

// --- few tokens ----------------------------------------------------------------
// 16 TF tokens against a workgroup's share of the weight's rows, which is the same
// for all up to one row, 16 R at a time.  The 8 waves split k, steps
// of 64 in turn, and each keeps the codes of its steps in registers over all its row
// blocks (up to XF steps; a memory pipeline that also carried the codes again for
// every row block took 60 us instead of 42 for 28672 x 8192 with 16 tokens).  A wave
// has a ring of kUnits fragments in LDS that only it fills and reads, first with
// codes, then with weight rows, so nothing but the meeting of the sums, integer
// additions in LDS, needs a barrier, and the next row block's loads are under way
// across it.
// XF = 0: k is too long for that, and each step brings its codes along.
constexpr int kUnits = 16;  // fragments of a wave's ring

// The weight rows of this workgroup.
struct RowRange {
    int64_t first, last;
};

__device__ __forceinline__ RowRange row_range(const Int8Args &a)
{
    const int b = blockIdx.x;
    const int64_t first = static_cast<int64_t>(b) * a.rows_per + (b < a.rows_extra ? b : a.rows_extra);
    return RowRange{first, first + a.rows_per + (b < a.rows_extra ? 1 : 0)};
}

// A wave each finishes 16 rows x 16 tokens of the row block from `row0` to `last`,
// and clears their sums for the row block after the next.
template <int OUT, int TF, int R, class Gathered>
__device__ __forceinline__ void finish_rows(const Int8Args &a, int32_t *sum, int64_t row0, int64_t last, int wave,
                                            int lane, int count, const Gathered &gathered)
{
    const int r = lane & 15, g = lane >> 4;
    if (wave >= R * TF)
        return;
    const int f = wave / TF, t = wave - f * TF;
    i32x4 *at = reinterpret_cast<i32x4 *>(&sum[wave * 256 + r * 16 + 4 * g]);
    const i32x4 q = *at;
    *at = i32x4{0, 0, 0, 0};
    const int64_t n0 = row0 + f * 16 + 4 * g, row = t * 16 + r;
    const int64_t n = row0 + f * 16 + r;  // the lane's row of the weight's operand
    const TokenScale scale = token_scale(row < a.m ? a.scales[row] : 0.0f);
    f32x4 z;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        z[i] = scaled_sum(q[i], n0 + i < last ? a.w_scales[n0 + i] : 0.0f, scale);
    constexpr int kFirst = Gathered::kChunks;
    if constexpr (kFirst > 0)
#pragma unroll
        for (int c = 0; c < kFirst; ++c)
            if (32 * c < count)
                z = Half<OUT>::mfma(weight_fragment<OUT>(a, n, gathered.columns[c], gathered.codes[c]), gathered.x[c], z);
    for (int c = kFirst; 32 * c < count; ++c) {
        if (kFirst == 0 && c < kOutlierChunks) {
            // (rows of any fragment: the workgroup's first row is no multiple of 16)
            const int64_t held = n < a.n ? n : a.n - 1;
            z = Half<OUT>::mfma(held_fragment(a.w_outliers, held >> 4, c, 16 * g + static_cast<int>(held & 15)),
                                held_fragment(a.x_outliers, t, c, lane), z);
            continue;
        }
        const Columns q2 = load_columns(a, 32 * c + 8 * g, count);
        z = Half<OUT>::mfma(weight_fragment<OUT>(a, n, q2, load_codes(a, n, q2)), x_fragment<OUT>(a, row, q2), z);
    }
    float out[4] = {z[0], z[1], z[2], z[3]};
    finish<OUT, 4>(a, row, n0, last, out);
}

// Up to 16 tokens: the columns of the first two chunks of outliers and x's operands,
// by the waves that finish; the weight's codes at the start of a row block.
template <int OUT, int TF, int R>
struct Gathered {
    static constexpr int kChunks = TF == 1 ? 2 : 0;
    Columns columns[2];
    u32x4 x[2];
    Codes codes[2];

    __device__ __forceinline__ void begin(const Int8Args &a, int wave, int lane, int count)
    {
        if constexpr (kChunks > 0) {
            if (wave < R)
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    if (32 * c < count) {
                        columns[c] = load_columns(a, 32 * c + 8 * (lane >> 4), count);
                        x[c] = x_fragment<OUT>(a, lane & 15, columns[c]);
                    }
        }
    }
    __device__ __forceinline__ void row_block(const Int8Args &a, int64_t row0, int wave, int lane, int count)
    {
        if constexpr (kChunks > 0) {
            if (wave < R)
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    if (32 * c < count)
                        codes[c] = load_codes(a, row0 + wave * 16 + (lane & 15), columns[c]);
        }
    }
};

// Bytes of rows row0 .. last - 1.
__device__ __forceinline__ uint32_t weight_bytes(const Int8Args &a, int64_t row0, int64_t last)
{
    const int64_t left = (last - row0 - 1) * a.ld_w + a.k;
    return static_cast<uint32_t>(left < 0x7FFFFFF0 ? left : 0x7FFFFFF0);
}

template <int R, int TF>
__device__ __forceinline__ void add_sums(int32_t *sum, const i32x4 (&acc)[R][TF], int lane)
{
#pragma unroll
    for (int f = 0; f < R; ++f)
#pragma unroll
        for (int t = 0; t < TF; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                atomicAdd(&sum[(f * TF + t) * 256 + (lane & 15) * 16 + 4 * (lane >> 4) + i], acc[f][t][i]);
}

template <int OUT, int TF, int R, int XF>
__global__ __launch_bounds__(512) void int8_rows_kernel(Int8Args a)
{
    constexpr int kStepUnits = XF > 0 ? R : R + TF;                    // of the ring
    constexpr int kSteps = kUnits / kStepUnits;                        // steps that fit it
    constexpr int kSlots = kSteps * kStepUnits;
    __shared__ __attribute__((aligned(1024))) uint8_t ring[8 * kSlots * kFragBytes];
    __shared__ __attribute__((aligned(16))) int32_t sums[2][R * TF * 256];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int steps = (a.k + kStep - 1) / kStep;
    const int mine = wave < steps ? (steps - wave + 7) / 8 : 0;
    const int count = outlier_count(a);

    for (int i = tid; i < 2 * R * TF * 256; i += 512)
        (&sums[0][0])[i] = 0;
    __syncthreads();
    Gathered<OUT, TF, R> gathered;
    gathered.begin(a, wave, lane, count);

    // the loads run ahead of the products: the codes' (XF > 0), then by steps, then by
    // row blocks; rows past the last one lie past the buffers
    const int piece = piece_of(lane);
    const uint32_t ring0 = lds_offset(ring) + wave * (kSlots * kFragBytes);
    const u32x4 rs_x = make_rsrc(a.codes, static_cast<uint32_t>((a.m - 1) * a.ld_codes + a.k));
    const RowRange rows = row_range(a);
    u32x4 rs_w = make_rsrc(a.w + rows.first * a.ld_w, weight_bytes(a, rows.first, rows.last));
    const uint32_t w_off = static_cast<uint32_t>((lane >> 2) * a.ld_w) + 16 * piece;
    const auto load_x = [&](int t, int i, int slot) {
        const int row = 16 * t + (lane >> 2);
        const uint32_t k0 = static_cast<uint32_t>(wave + 8 * i) * kStep;
        const bool in = row < a.m && i < mine && k0 + 16 * piece < static_cast<uint32_t>(a.k);
        buffer_to_lds(rs_x, in ? static_cast<uint32_t>(row * a.ld_codes) + k0 + 16 * piece : kPast, 0,
                      ring0 + slot * kFragBytes);
    };
    int64_t l_row = rows.first;
    int l_i = 0;
    // past the last step the loads fetch zeros that nobody reads
    const auto load_w = [&](int f, int slot) {
        const uint32_t k0 = static_cast<uint32_t>(wave + 8 * l_i) * kStep;
        const bool in = l_row < rows.last && k0 + 16 * piece < static_cast<uint32_t>(a.k);
        u32x4 rs;
#pragma unroll
        for (int d = 0; d < 4; ++d)
            rs[d] = __builtin_amdgcn_readfirstlane(rs_w[d]);
        buffer_to_lds(rs, in ? w_off + f * 16 * static_cast<uint32_t>(a.ld_w) + k0 : kPast, 0,
                      ring0 + slot * kFragBytes);
    };
    const auto next_step = [&]() {
        if (++l_i == mine) {
            l_i = 0;
            l_row += 16 * R;
            if (l_row < rows.last)
                rs_w = make_rsrc(a.w + l_row * a.ld_w, weight_bytes(a, l_row, rows.last));
        }
    };
    const auto load_step = [&](int slot) {
#pragma unroll
        for (int f = 0; f < R; ++f)
            load_w(f, slot + f);
        if constexpr (XF == 0)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                load_x(t, l_row < rows.last ? l_i : mine, slot + R + t);
        next_step();
    };
    const auto at = [&](int slot) {
        return ring + (wave * kSlots + slot) * kFragBytes + piece_at(lane & 15, lane >> 4);
    };

    u32x4 x[XF > 0 ? XF : 1][TF];
    int slot = 0;
    if (mine > 0) {
        if constexpr (XF > 0) {
            // one row of fragments through the ring: the codes' (an even number of
            // steps, so that the weight's steps lie whole behind them), then the weight's
            static_assert(kSlots == kUnits && kSlots % R == 0, "a step of the weight is not cut");
            const int code_steps = (mine + 1) & ~1, codes = code_steps * TF;
            const auto load_unit = [&](int u) {
                if (u < codes) {
                    load_x(u % TF, u / TF, u % kSlots);
                } else {
                    const int f = (u - codes) % R;
                    load_w(f, u % kSlots);
                    if (f == R - 1)
                        next_step();
                }
            };
#pragma unroll
            for (int u = 0; u < kSlots; ++u)
                load_unit(u);
#pragma unroll
            for (int i = 0; i < XF; ++i)
                if (i < code_steps)
#pragma unroll
                    for (int t = 0; t < TF; ++t) {
                        const int u = i * TF + t;
                        __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(kSlots - 1) : "memory");
                        x[i][t] = *reinterpret_cast<const u32x4 *>(at(u % kSlots));
                        __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                        __builtin_amdgcn_sched_barrier(0);
                        load_unit(u + kSlots);
                    }
            slot = codes % kSlots;
        } else {
#pragma unroll
            for (int d = 0; d < kSteps; ++d)
                load_step(d * kStepUnits);
        }
    }
    int parity = 0;
    for (int64_t row0 = rows.first; row0 < rows.last; row0 += 16 * R, parity ^= 1) {
        i32x4 acc[R][TF];
#pragma unroll
        for (int f = 0; f < R; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                acc[f][t] = i32x4{0, 0, 0, 0};
        gathered.row_block(a, row0, wave, lane, count);
        const auto step = [&](const u32x4 (&held)[TF]) {
            __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"((kSteps - 1) * kStepUnits) : "memory");
            u32x4 wf[R], xf[TF];
#pragma unroll
            for (int f = 0; f < R; ++f)
                wf[f] = *reinterpret_cast<const u32x4 *>(at(slot + f));
#pragma unroll
            for (int t = 0; t < TF; ++t)
                if constexpr (XF > 0)
                    xf[t] = held[t];
                else
                    xf[t] = *reinterpret_cast<const u32x4 *>(at(slot + R + t));
            // the step's places are read: they may be filled again
            __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            load_step(slot);
            slot = slot + kStepUnits == kSlots ? 0 : slot + kStepUnits;
#pragma unroll
            for (int f = 0; f < R; ++f)
#pragma unroll
                for (int t = 0; t < TF; ++t)
                    acc[f][t] = mfma_i8(wf[f], xf[t], acc[f][t]);
        };
        if constexpr (XF > 0) {
#pragma unroll
            for (int i = 0; i < XF; ++i)
                if (i < mine)
                    step(x[i]);
        } else {
            for (int i = 0; i < mine; ++i)
                step(x[0]);
        }
        if (mine > 0)
            add_sums<R, TF>(sums[parity], acc, lane);
        lds_barrier();
        finish_rows<OUT, TF, R>(a, sums[parity], row0, rows.last, wave, lane, count, gathered);
    }
}

// The same for rows that are no multiple of 16 bytes, or not aligned so: dwords into
// registers, shifted to bytes, and no ring.
template <int OUT, int TF, int R>
__global__ __launch_bounds__(512) void int8_any_rows_kernel(Int8Args a)
{
    constexpr int kFrags = R + TF;
    __shared__ __attribute__((aligned(16))) int32_t sums[2][R * TF * 256];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int steps = (a.k + kStep - 1) / kStep;
    const int mine = wave < steps ? (steps - wave + 7) / 8 : 0;
    const int count = outlier_count(a);
    const uint32_t x_bytes = static_cast<uint32_t>((a.m - 1) * a.ld_codes + a.k);
    for (int i = tid; i < 2 * R * TF * 256; i += 512)
        (&sums[0][0])[i] = 0;
    __syncthreads();
    Gathered<OUT, TF, R> gathered;
    gathered.begin(a, wave, lane, count);

    const RowRange rows = row_range(a);

    // 16 bytes at any address: 5 dwords, those past the buffer are zeros
    const auto load_bytes = [&](__amdgpu_buffer_rsrc_t rsrc, uint32_t at, int left) {
        const u32x4 lo = __builtin_amdgcn_raw_buffer_load_b128(rsrc, at & ~3u, 0, 0);
        const uint32_t hi = __builtin_amdgcn_raw_buffer_load_b32(rsrc, (at & ~3u) + 16, 0, 0);
        u32x4 q;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const uint32_t v = __builtin_amdgcn_alignbyte(d < 3 ? lo[d + 1] : hi, lo[d], at & 3);
            const int valid = left - 4 * d;  // bytes of the row
            q[d] = valid >= 4 ? v : valid <= 0 ? 0u : v & ((1u << (8 * valid)) - 1);
        }
        return q;
    };
    int parity = 0;
    for (int64_t row0 = rows.first; row0 < rows.last; row0 += 16 * R, parity ^= 1) {
        i32x4 acc[R][TF];
#pragma unroll
        for (int f = 0; f < R; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                acc[f][t] = i32x4{0, 0, 0, 0};
        gathered.row_block(a, row0, wave, lane, count);
        const uintptr_t w_at = reinterpret_cast<uintptr_t>(a.w + row0 * a.ld_w);
        const uintptr_t x_at = reinterpret_cast<uintptr_t>(a.codes);
        const uint32_t w_skew = w_at & 3, x_skew = x_at & 3;
        // whole dwords, up to the one with the last byte
        const auto rw = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(w_at - w_skew), 0,
                                                          (weight_bytes(a, row0, rows.last) + w_skew + 3) & ~3u, kRawBufferWord3);
        const auto rx = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(x_at - x_skew), 0,
                                                          (x_bytes + x_skew + 3) & ~3u, kRawBufferWord3);
        const int64_t rows_left = rows.last - row0;
        const auto load = [&](u32x4 (&q)[kFrags], int i) {
            const int k0 = (wave + 8 * i) * kStep + 16 * g;
            const int left = i < mine ? a.k - k0 : 0;  // bytes of the row from here on
#pragma unroll
            for (int f = 0; f < R; ++f) {
                const int row = 16 * f + r;
                q[f] = load_bytes(rw, left > 0 && row < rows_left
                                          ? static_cast<uint32_t>(row * a.ld_w) + k0 + w_skew : kPast, left);
            }
#pragma unroll
            for (int t = 0; t < TF; ++t) {
                const int row = 16 * t + r;
                q[R + t] = load_bytes(rx, left > 0 && row < a.m
                                              ? static_cast<uint32_t>(row * a.ld_codes) + k0 + x_skew : kPast, left);
            }
        };
        u32x4 now[kFrags], next[kFrags];
        load(now, 0);
        for (int i = 0; i < mine; ++i) {
            load(next, i + 1);
#pragma unroll
            for (int f = 0; f < R; ++f)
#pragma unroll
                for (int t = 0; t < TF; ++t)
                    acc[f][t] = mfma_i8(now[f], now[R + t], acc[f][t]);
#pragma unroll
            for (int f = 0; f < kFrags; ++f)
                now[f] = next[f];
        }
        if (mine > 0)
            add_sums<R, TF>(sums[parity], acc, lane);
        lds_barrier();
        finish_rows<OUT, TF, R>(a, sums[parity], row0, rows.last, wave, lane, count, gathered);
    }
}

// --- more tokens ------------------------------------------------------------------
constexpr int kGroup = 128, kGroupFrags = 8;
constexpr int kFinishLd = kGroup + 4;  // floats per row of a wave's epilogue slab

// 16 tokens x 128 columns of sums to outputs, through a slab of LDS that only this
// wave uses: a lane holds 8 neighbouring columns of one token per D register, so
// the slab takes and gives whole vectors.
template <int OUT>
__device__ __forceinline__ void finish_slab_rows(const Int8Args &a, const float *slab, int64_t row0,
                                                 int64_t group, int it, int lane)
{
    const int g = lane >> 4, c = lane & 15;
    const float *from = slab + (it * 4 + g) * kFinishLd + 8 * c;
    const f32x4 lo = *reinterpret_cast<const f32x4 *>(from);
    const f32x4 hi = *reinterpret_cast<const f32x4 *>(from + 4);
    float z[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    finish<OUT, 8>(a, row0 + it * 4 + g, group * kGroup + 8 * c, a.n, z);
}

// FP32 values of fragments F0 .. F0 + N - 1 of a group and 16 tokens, outliers
// included.
template <int OUT, int N>
__device__ __forceinline__ void tile_values(const Int8Args &a, const i32x4 *sum, int stride, int f0,
                                            int64_t group, int64_t row0, int count, int lane,
                                            f32x4 (&z)[N])
{
    const int g = lane >> 4;
    const int64_t row = row0 + (lane & 15);
    const TokenScale scale = token_scale(row < a.m ? a.scales[row] : 0.0f);
#pragma unroll
    for (int f = 0; f < N; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t n = group * kGroup + 8 * (4 * g + i) + f0 + f;
            z[f][i] = scaled_sum(sum[f * stride][i], n < a.n ? a.w_scales[n] : 0.0f, scale);
        }
    for (int c = 0; c < kOutlierChunks && 32 * c < count; ++c) {
        const u32x4 xf = held_fragment(a.x_outliers, row0 >> 4, c, lane);
#pragma unroll
        for (int f = 0; f < N; ++f)
            z[f] = Half<OUT>::mfma(held_fragment(a.w_outliers, group * kGroupFrags + f0 + f, c, lane), xf, z[f]);
    }
#pragma unroll 1
    for (int c = kOutlierChunks; 32 * c < count; ++c) {
        const int l0 = 32 * c + 8 * g;
        const u32x4 xf = gather_slowly<OUT>(a, l0, count, [&](int column) { return x_value<OUT>(a, row, column); });
#pragma unroll
        for (int f = 0; f < N; ++f) {
            const int64_t n = fragment_row<true>(group * kGroupFrags + f0 + f, lane & 15);
            const u32x4 wf = gather_slowly<OUT>(a, l0, count, [&](int column) { return weight_value<OUT>(a, n, column); });
            z[f] = Half<OUT>::mfma(wf, xf, z[f]);
        }
    }
}

// The epilogue of one wave's 128 columns x 16 TF tokens.
template <int OUT, int TF>
__device__ __forceinline__ void finish_wave(const Int8Args &a, const i32x4 (&acc)[kGroupFrags][TF], float *slab,
                                            int64_t group, int64_t row0, int lane)
{
    const int count = outlier_count(a);
    const int g = lane >> 4, c = lane & 15;
    if (group * kGroup >= a.n)
        return;
#pragma unroll
    for (int t = 0; t < TF; ++t) {
        if (row0 + t * 16 >= a.m)
            return;
        f32x4 z[kGroupFrags];
        tile_values<OUT, kGroupFrags>(a, &acc[0][t], TF, 0, group, row0 + t * 16, count, lane, z);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float *to = slab + c * kFinishLd + 8 * (4 * g + i);
            *reinterpret_cast<f32x4 *>(to) = f32x4{z[0][i], z[1][i], z[2][i], z[3][i]};
            *reinterpret_cast<f32x4 *>(to + 4) = f32x4{z[4][i], z[5][i], z[6][i], z[7][i]};
        }
        // the wave's LDS operations complete in order; the compiler must not move
        // the reads of other lanes' values above the writes
        __asm__ volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int it = 0; it < 4; ++it)
            finish_slab_rows<OUT>(a, slab, row0 + t * 16, group, it, lane);
        __asm__ volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
    }
}

// Tile of 128 WN output columns x 16 TF WT tokens; wave (wn, wt) takes group wn of
// the tile and 16 TF tokens.  Both operands go from memory straight to LDS, 128 k
// at a time: a load takes whole 128-byte lines of 8 rows, lane l the 16 bytes l % 8
// of row l / 8 (with 64 bytes of 16 rows each line was fetched twice, and an 8192^3
// product took 18 % longer).  A chunk is 8 rows of every fragment of the tile; two
// chunks make 128 k, two steps of matrix instructions, and a ring of five lets each
// chunk be under way for two steps.  In it the piece p of row r lies in place p ^ (r
// / 2) of its 128 bytes, for reads without bank conflicts as above.
//
// The 256 x 256 tile (WN = 2), 8 waves, has two halves of waves, one of each half
// on every SIMD, one phase apart: while one multiplies, the other reads its operands
// of the next step from LDS and issues its loads.  The other tiles have several
// workgroups per CU instead, and one barrier for 128 k.
constexpr int kRing = 5;

// Tiles go in bands of kBand columns, row by row: the 32 that an XCD works on at a
// time are then about as many rows as columns, and its L2 fetches the least (8192^3:
// see below).
constexpr int kBand = 4;

__device__ __forceinline__ void place_of(const Int8Args &a, int tile, int *tile_n, int *tile_t)
{
    const int band = tile / (kBand * a.tiles_t);
    const int left = a.tiles_n - band * kBand, width = left < kBand ? left : kBand;
    const int in = tile - band * (kBand * a.tiles_t);
    *tile_t = in / width;
    *tile_n = band * kBand + in - *tile_t * width;
}

template <int OUT, int WN, int WT, int TF>
__global__ __launch_bounds__(64 * WN * WT) void int8_product_kernel(Int8Args a)
{
    constexpr int kWaves = WN * WT;
    constexpr int kRows = 16 * TF * WT;
    constexpr int kTileFrags = WN * kGroupFrags + TF * WT;
    constexpr int kChunk = kTileFrags * kFragBytes;
    constexpr int kLoads = kTileFrags / kWaves;
    static_assert(kLoads * kWaves == kTileFrags, "the waves share the loads evenly");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kRing * kChunk];
    static_assert(kWaves * 16 * kFinishLd * 4 <= kRing * kChunk, "the epilogue slabs fit the ring");

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % WN, wt = wave / WN;

    // consecutive workgroups go to the XCDs in turn: give each XCD a contiguous
    // run of tiles, so that its L2 serves their shared operands
    const int tiles = gridDim.x;
    const int per = tiles / kXcds, extra = tiles % kXcds;
    const int xcd = blockIdx.x % kXcds, idx = blockIdx.x / kXcds;
    const int tile = xcd * per + (xcd < extra ? xcd : extra) + idx;
    int tile_n, tile_t;
    place_of(a, tile, &tile_n, &tile_t);
    const int64_t col0 = static_cast<int64_t>(tile_n) * (WN * kGroup);
    const int64_t row0 = static_cast<int64_t>(tile_t) * kRows;

    // this wave's loads of a chunk: fragments wave * kLoads .. of the weight's, then
    // the codes'; rows past the end get an offset past any buffer
    const int64_t cols_left = a.n - col0, rows_left = a.m - row0;
    const int cols_here = static_cast<int>(cols_left < WN * kGroup ? cols_left : WN * kGroup);
    const int rows_here = static_cast<int>(rows_left < kRows ? rows_left : kRows);
    const u32x4 rs_w = make_rsrc(a.w + col0 * a.ld_w, static_cast<uint32_t>((cols_here - 1) * a.ld_w + a.k));
    const u32x4 rs_x = make_rsrc(a.codes + row0 * a.ld_codes,
                                 static_cast<uint32_t>((rows_here - 1) * a.ld_codes + a.k));
    uint32_t off[2][kLoads];
    int from_k[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = (lane >> 3) + 8 * h;
        from_k[h] = 16 * ((lane & 7) ^ (r >> 1));
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int fr = wave * kLoads + q;
            if (fr < WN * kGroupFrags) {
                const int row = (fr >> 3) * kGroup + 8 * r + (fr & 7);
                off[h][q] = row < cols_here ? static_cast<uint32_t>(row * a.ld_w) + from_k[h] : kPast;
            } else {
                const int row = (fr - WN * kGroupFrags) * 16 + r;
                off[h][q] = row < rows_here ? static_cast<uint32_t>(row * a.ld_codes) + from_k[h] : kPast;
            }
        }
    }
    const uint32_t to0 = lds_offset(lds) + wave * (kLoads * kFragBytes);

    const int pairs = (a.k + 2 * kStep - 1) / (2 * kStep);
    const int split = blockIdx.y;
    const int p_first = static_cast<int>(static_cast<uint32_t>(pairs * split) / static_cast<uint32_t>(a.splits));
    const int p_last = static_cast<int>(static_cast<uint32_t>(pairs * (split + 1)) / static_cast<uint32_t>(a.splits));

    // always kLoads: past the last chunk they fetch zeros that nobody reads
    int slot = 0;  // of the next chunk
    auto issue = [&](int p, int h) {
        const int k0 = p * (2 * kStep);
        const bool in = p < p_last && k0 + from_k[h] < a.k;
        const uint32_t to = to0 + slot * kChunk;
#pragma unroll
        for (int q = 0; q < kLoads; ++q)
            buffer_to_lds(wave * kLoads + q < WN * kGroupFrags ? rs_w : rs_x, in ? off[h][q] + k0 : kPast, 0,
                          to + q * kFragBytes);
        slot = slot + 1 == kRing ? 0 : slot + 1;
    };

    i32x4 acc[kGroupFrags][TF];
#pragma unroll
    for (int f = 0; f < kGroupFrags; ++f)
#pragma unroll
        for (int t = 0; t < TF; ++t)
            acc[f][t] = i32x4{0, 0, 0, 0};

    // lane 16 g + r reads piece 4 s + g of row r for step s
    const int r = lane & 15, g = lane >> 4;
    const uint32_t in_row = (r & 7) * 128;
    const uint32_t at[2] = {in_row + 16 * (g ^ (r >> 1)), in_row + 16 * ((4 + g) ^ (r >> 1))};
    int first = 0;  // slot of the pair's first chunk
    u32x4 wf[kGroupFrags], xf[TF];
    auto read = [&](int s) {
        const int second = first + 1 == kRing ? 0 : first + 1;
        const uint8_t *from = lds + (r < 8 ? first : second) * kChunk + at[s];
#pragma unroll
        for (int t = 0; t < TF; ++t)
            xf[t] = *reinterpret_cast<const u32x4 *>(from + (WN * kGroupFrags + wt * TF + t) * kFragBytes);
#pragma unroll
        for (int f = 0; f < kGroupFrags; ++f)
            wf[f] = *reinterpret_cast<const u32x4 *>(from + (wn * kGroupFrags + f) * kFragBytes);
    };
    auto multiply = [&]() {
#pragma unroll
        for (int f = 0; f < kGroupFrags; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                acc[f][t] = mfma_i8(wf[f], xf[t], acc[f][t]);
    };

    issue(p_first, 0);
    issue(p_first, 1);
    issue(p_first + 1, 0);
    if constexpr (WN == 2) {
        __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads) : "memory");
        __builtin_amdgcn_s_barrier();
        if (wave >= kWaves / 2)
            __builtin_amdgcn_s_barrier();  // the second half is one phase behind
        for (int p = p_first; p < p_last; ++p) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                read(s);
                // into the places of pair p - 1, which both halves have read
                if (s == 0)
                    issue(p + 1, 1);
                else
                    issue(p + 2, 0);
                // this wave's reads are done, and before the next pair its share of
                // that has arrived (the chunk after it is under way)
                if (s == 0)
                    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                else
                    __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kLoads) : "memory");
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_setprio(1);
                multiply();
                __builtin_amdgcn_s_setprio(0);
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
            }
            first = first + 2 >= kRing ? first + 2 - kRing : first + 2;
        }
        if (wave < kWaves / 2)
            __builtin_amdgcn_s_barrier();
    } else {
        for (int p = p_first; p < p_last; ++p) {
            // the pair has arrived (the chunk after it is under way), and this wave's
            // reads of the last pair are done: its places are filled next
            __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kLoads) : "memory");
            __builtin_amdgcn_s_barrier();
            __asm__ volatile("" ::: "memory");
            read(0);
            issue(p + 1, 1);
            multiply();
            read(1);
            issue(p + 2, 0);
            multiply();
            first = first + 2 >= kRing ? first + 2 - kRing : first + 2;
        }
    }
    // the epilogue takes the ring: no load may still be on its way into it
    __asm__ volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");

    if (a.splits > 1) {
        i32x4 *to = a.partial +
                    ((static_cast<int64_t>(split) * tiles + tile) * kWaves + wave) * (kGroupFrags * TF * 64) + lane;
#pragma unroll
        for (int f = 0; f < kGroupFrags; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                to[(f * TF + t) * 64] = acc[f][t];
        return;
    }
    finish_wave<OUT, TF>(a, acc, reinterpret_cast<float *>(lds) + wave * (16 * kFinishLd),
                         static_cast<int64_t>(tile_n) * WN + wn, row0 + wt * (16 * TF), lane);
}

// The splits' sums of one wave's 128 columns x 16 tokens, and the epilogue.  Four
// waves share the 8 fragments.
template <int OUT, int WN, int WT, int TF>
__global__ __launch_bounds__(256) void int8_product_reduce_kernel(Int8Args a, int32_t tiles)
{
    __shared__ __attribute__((aligned(16))) float slab[16 * kFinishLd];
    const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int t = blockIdx.y;
    const int tile = blockIdx.x / (WN * WT), wave = blockIdx.x % (WN * WT);
    const int wn = wave % WN, wt = wave / WN;
    int tile_n, tile_t;
    place_of(a, tile, &tile_n, &tile_t);
    const int64_t group = static_cast<int64_t>(tile_n) * WN + wn;
    const int64_t row0 = (static_cast<int64_t>(tile_t) * WT + wt) * (16 * TF) + 16 * t;
    if (group * kGroup >= a.n || row0 >= a.m)
        return;
    const i32x4 *from = a.partial + (static_cast<int64_t>(tile) * (WN * WT) + wave) * (kGroupFrags * TF * 64) +
                        (2 * q * TF + t) * 64 + lane;
    const int64_t split_step = static_cast<int64_t>(tiles) * (WN * WT) * (kGroupFrags * TF * 64);
    i32x4 sum[2] = {};
    for (int s = 0; s < a.splits; s += 8) {
        i32x4 part[8][2];
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
                    sum[f] = sum[f] + part[i][f];
    }
    f32x4 z[2];
    tile_values<OUT, 2>(a, sum, 1, 2 * q, group, row0, outlier_count(a), lane, z);
    const int g = lane >> 4, c = lane & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x2 *>(slab + c * kFinishLd + 8 * (4 * g + i) + 2 * q) = f32x2{z[0][i], z[1][i]};
    __syncthreads();
    finish_slab_rows<OUT>(a, slab, row0, group, q, lane);
}

// Rows of bytes, any alignment and stride, into rows of ld_out bytes (a multiple of
// 16) with zeros behind column k.
struct CopyArgs {
    const int8_t *in;
    int64_t ld_in, rows;
    int8_t *out;
};

__global__ __launch_bounds__(256) void int8_rows_zero_fill(CopyArgs a, CopyArgs b, int32_t k, int32_t ld_out)
{
    const int words = ld_out / 4;
    for (int64_t item = blockIdx.x; item < a.rows + b.rows; item += gridDim.x) {
        const bool first = item < a.rows;
        const int64_t row = first ? item : item - a.rows;
        const int8_t *from = first ? a.in + row * a.ld_in : b.in + row * b.ld_in;
        uint32_t *to = reinterpret_cast<uint32_t *>((first ? a.out : b.out) + row * ld_out);
        for (int c = threadIdx.x; c < words; c += 256) {
            uint32_t q = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * c + j < k)
                    q |= static_cast<uint32_t>(static_cast<uint8_t>(from[4 * c + j])) << (8 * j);
            to[c] = q;
        }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// The least 15-bit pattern of T whose value is not below the threshold; T's
// infinity where every finite value is.
uint32_t threshold_pattern(float threshold, int32_t dtype)
{
    const auto value = [&](uint32_t bits) {
        if (dtype == DQ4_BF16) {
            const uint32_t wide = bits << 16;
            float f;
            __builtin_memcpy(&f, &wide, 4);
            return static_cast<double>(f);
        }
        const int e = static_cast<int>(bits >> 10);
        const double f = static_cast<double>(bits & 1023);
        return e == 0 ? f * 0x1p-24 : __builtin_ldexp(1024.0 + f, e - 25);
    };
    uint32_t low = 1, high = dtype == DQ4_F16 ? 0x7C00u : 0x7F80u;
    while (low < high) {
        const uint32_t mid = (low + high) / 2;
        if (value(mid) >= static_cast<double>(threshold))
            high = mid;
        else
            low = mid + 1;
    }
    return low;
}

bool sizes_fit(int64_t m, int64_t n_out, int64_t n_in)
{
    return m <= kMaxDim && n_out <= kMaxDim && n_in <= kMaxSum && m * n_out <= kMaxMatrix;
}

// Row strides up to this keep a tile's 256 rows below the offset 2^31.
constexpr int64_t kMaxStride = int64_t{1} << 22;

// Whether rows of bytes can be loaded 16 at a time.
bool byte_rows_aligned(const void *p, int64_t ld, int64_t rows, int64_t k)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && k % 16 == 0 &&
           (rows <= 1 || (ld % 16 == 0 && ld <= kMaxStride));
}

// Tokens of the row kernels, and of their form that gathers outliers itself.
constexpr int64_t kRowsMost = 64, kGatheredMost = 16;

// Whether a call takes a row kernel.  With more than 32 tokens and more than 4096 k
// a wave's codes do not fit its registers, and the tiles are faster (64 tokens, us,
// rows | tiles: 28672 x 8192 83 | 69, 4096 x 14336 23.1 | 19.8; 4096 x 4096 11.3 |
// 14.6; 32 tokens, 28672 x 8192: 53 | 67), unless they had to copy the weight first.
bool takes_rows(int64_t m, int64_t k, bool aligned)
{
    return m <= kRowsMost && (m <= 32 || k <= 4096 || !aligned);
}

// Tiles of 16 tokens that a row kernel works on.  It reads the outlier operands of all
// of them, also of those behind the last token, so the workspace holds as many.
int row_kernel_tiles(int64_t m)
{
    return m <= 16 ? 1 : m <= 32 ? 2 : 4;
}

constexpr int kTileCols[3] = {256, 128, 128}, kTileRows[3] = {256, 128, 64};
constexpr int kTileResident[3] = {1, 2, 2};  // workgroups per CU (LDS)
// Microseconds of one step of 64 k with every CU full, as measured at 8192^3 (438,
// 565 and 755 us).
constexpr double kTileStep[3] = {0.86, 0.55, 0.37};

struct Plan {
    int tile, splits;
    double cost;
};

Plan plan_of(int64_t m, int64_t n, int64_t k, int cus)
{
    Plan best{2, 1, 1e300};
    const int64_t steps = ceil_div(k, kStep);
    for (int tile = 0; tile < 3; ++tile) {
        const int64_t tiles = ceil_div(n, kTileCols[tile]) * ceil_div(m, kTileRows[tile]);
        for (int splits = 1; splits <= 16; ++splits) {
            if (splits > 1 && splits * 4 > steps)
                break;
            const int64_t rounds = ceil_div(tiles * splits, static_cast<int64_t>(cus) * kTileResident[tile]);
            double cost = static_cast<double>(rounds) *
                          (static_cast<double>(ceil_div(steps, splits)) * kTileStep[tile] + 3.0);
            if (splits > 1)  // the partial sums, written and read at about 8 TB/s (cache), and a launch
                cost += 3.0 + static_cast<double>(splits) * static_cast<double>(m) * static_cast<double>(n) * 8.0 / 8e6;
            if (cost < best.cost)
                best = Plan{tile, splits, cost};
        }
    }
    return best;
}

int64_t partial_bytes(const Plan &p, int64_t m, int64_t n)
{
    return p.splits == 1 ? 0
                         : p.splits * ceil_div(n, kTileCols[p.tile]) * kTileCols[p.tile] *
                               ceil_div(m, kTileRows[p.tile]) * kTileRows[p.tile] * 4;
}

// What a product's workspace holds, in this order.
struct Layout {
    bool rows;                       // int8_rows_kernel
    bool copy_codes, copy_weight;    // in rows of ld_copy bytes
    int64_t ld_copy;
    int64_t codes_bytes, weight_bytes;
    int64_t w_frags, x_frags;        // outlier fragments
    Plan plan;
    int64_t partial;
    int64_t frag_bytes() const { return (w_frags + x_frags) * kOutlierChunks * kFragBytes; }
    int64_t bytes() const { return codes_bytes + weight_bytes + frag_bytes() + partial; }
};

Layout layout_of(const void *codes, int64_t m, int64_t ld_codes, const void *w, int64_t n, int64_t k,
                 bool outliers, int cus)
{
    Layout l{};
    l.rows = takes_rows(m, k, byte_rows_aligned(codes, ld_codes, m, k) && byte_rows_aligned(w, k, n, k));
    l.copy_codes = l.rows ? m > 1 && ld_codes > kMaxStride : !byte_rows_aligned(codes, ld_codes, m, k);
    l.copy_weight = !l.rows && !byte_rows_aligned(w, k, n, k);
    l.ld_copy = ceil_div(k, kStep) * kStep;
    l.codes_bytes = l.copy_codes ? align256(m * l.ld_copy) : 0;
    l.weight_bytes = l.copy_weight ? align256(n * l.ld_copy) : 0;
    if (!l.rows) {
        l.plan = plan_of(m, n, k, cus);
        l.partial = partial_bytes(l.plan, m, n);
    }
    if (outliers && k > 0 && m > kGatheredMost) {
        l.w_frags = l.rows ? ceil_div(n, 16) : ceil_div(n, kGroup) * kGroupFrags;
        l.x_frags = l.rows ? row_kernel_tiles(m) : ceil_div(m, 16);
    }
    return l;
}

template <int OUT, int TF, int R>
dq4_status_t launch_rows_tile(Int8Args a, bool aligned, int cus, hipStream_t s)
{
    const int64_t grid = ceil_div(a.n, 16) < cus ? ceil_div(a.n, 16) : cus;
    a.rows_per = static_cast<int32_t>(a.n / grid);
    a.rows_extra = static_cast<int32_t>(a.n % grid);
    const void *kernel = aligned ? reinterpret_cast<const void *>(&int8_rows_kernel<OUT, TF, R, 0>)
                                 : reinterpret_cast<const void *>(&int8_any_rows_kernel<OUT, TF, R>);
    // codes are kept where there is more than one row block to keep them for (16
    // tokens, 4096 x 14336, one row block: 16.4 us kept, 13.3 not); with R = 1 there is one
    if constexpr (R == 2) {
        const int64_t steps = ceil_div(ceil_div(a.k, kStep), 8);  // of a wave
        if (aligned && a.n > grid * (16 * R)) {
            if (steps <= 8)
                kernel = reinterpret_cast<const void *>(&int8_rows_kernel<OUT, TF, R, 8>);
            else if (steps <= 16 && TF <= 2)
                kernel = reinterpret_cast<const void *>(&int8_rows_kernel<OUT, TF, R, TF <= 2 ? 16 : 8>);
            else if (steps <= 32 && TF == 1)
                kernel = reinterpret_cast<const void *>(&int8_rows_kernel<OUT, TF, R, TF == 1 ? 32 : 8>);
        }
    }
    void *params[] = {&a};
    return launch(kernel, grid, 1, 512, params, s);
}

template <int OUT>
dq4_status_t launch_rows(const Int8Args &a, int cus, hipStream_t s)
{
    const bool aligned = byte_rows_aligned(a.codes, a.ld_codes, a.m, a.k) && byte_rows_aligned(a.w, a.ld_w, a.n, a.k);
    const bool two = a.n > static_cast<int64_t>(16) * cus;  // more than 16 rows a workgroup
    const int tiles = row_kernel_tiles(a.m);
    if (tiles == 1)
        return two ? launch_rows_tile<OUT, 1, 2>(a, aligned, cus, s) : launch_rows_tile<OUT, 1, 1>(a, aligned, cus, s);
    if (tiles == 2)
        return two ? launch_rows_tile<OUT, 2, 2>(a, aligned, cus, s) : launch_rows_tile<OUT, 2, 1>(a, aligned, cus, s);
    return two ? launch_rows_tile<OUT, 4, 2>(a, aligned, cus, s) : launch_rows_tile<OUT, 4, 1>(a, aligned, cus, s);
}

template <int OUT, int WN, int WT, int TF>
dq4_status_t launch_tile(Int8Args a, hipStream_t s)
{
    a.tiles_t = static_cast<int32_t>(ceil_div(a.m, 16 * TF * WT));
    a.tiles_n = static_cast<int32_t>(ceil_div(a.n, WN * kGroup));
    const int64_t tiles = static_cast<int64_t>(a.tiles_n) * a.tiles_t;
    void *params[] = {&a};
    const dq4_status_t st = launch(reinterpret_cast<const void *>(&int8_product_kernel<OUT, WN, WT, TF>), tiles,
                                   a.splits, 64 * WN * WT, params, s);
    if (st != DQ4_OK || a.splits == 1)
        return st;
    int32_t n_tiles = static_cast<int32_t>(tiles);
    void *rp[] = {&a, &n_tiles};
    return launch(reinterpret_cast<const void *>(&int8_product_reduce_kernel<OUT, WN, WT, TF>), tiles * WN * WT, TF,
                  256, rp, s);
}

template <int OUT>
dq4_status_t run_linear(Int8Args a, const Layout &l, uint8_t *ws, int cus, hipStream_t s)
{
    dq4_status_t st = DQ4_OK;
    if ((l.copy_codes || l.copy_weight) && a.k > 0) {
        CopyArgs codes{}, weight{};
        if (l.copy_codes) {
            codes = CopyArgs{a.codes, a.ld_codes, a.m, reinterpret_cast<int8_t *>(ws)};
            a.codes = codes.out;
            a.ld_codes = l.ld_copy;
        }
        if (l.copy_weight) {
            weight = CopyArgs{a.w, a.ld_w, a.n, reinterpret_cast<int8_t *>(ws + l.codes_bytes)};
            a.w = weight.out;
            a.ld_w = l.ld_copy;
        }
        int32_t k = a.k, ld = static_cast<int32_t>(l.ld_copy);
        void *params[] = {&codes, &weight, &k, &ld};
        const int64_t rows = codes.rows + weight.rows;
        st = launch(reinterpret_cast<const void *>(&int8_rows_zero_fill), rows < cus * 8 ? rows : cus * 8, 1, 256,
                    params, s);
        if (st != DQ4_OK)
            return st;
    }
    uint16_t *frags = reinterpret_cast<uint16_t *>(ws + l.codes_bytes + l.weight_bytes);
    if (l.w_frags > 0) {
        int64_t w_frags = l.w_frags, x_frags = l.x_frags;
        void *params[] = {&a, &w_frags, &x_frags, &frags};
        const int64_t groups = w_frags + x_frags;  // (four chunks each)
        const void *kernel = l.rows ? reinterpret_cast<const void *>(&int8_outlier_fragments_kernel<OUT, false>)
                                    : reinterpret_cast<const void *>(&int8_outlier_fragments_kernel<OUT, true>);
        st = launch(kernel, groups < cus * 8 ? groups : cus * 8, 1, 256, params, s);
        if (st != DQ4_OK)
            return st;
        a.w_outliers = frags;
        a.x_outliers = frags + w_frags * kOutlierChunks * (kFragBytes / 2);
    }
    if (l.rows)
        return launch_rows<OUT>(a, cus, s);
    // copies end in zeros: the tiles read whole pieces of 16
    a.k = static_cast<int32_t>(l.copy_codes || l.copy_weight ? ceil_div(a.k, 16) * 16 : a.k);
    a.splits = l.plan.splits;
    a.partial = reinterpret_cast<i32x4 *>(ws + l.codes_bytes + l.weight_bytes + l.frag_bytes());
    if (l.plan.tile == 0)
        return launch_tile<OUT, 2, 4, 4>(a, s);
    if (l.plan.tile == 1)
        return launch_tile<OUT, 1, 4, 2>(a, s);
    return launch_tile<OUT, 1, 4, 1>(a, s);
}

}  // namespace
}  // namespace dq4

using namespace dq4;

extern "C" {

int64_t dq4_int8_quant_workspace_bytes(int64_t m, int64_t n_in, float threshold)
{
    if (!(threshold > 0.0f) || m <= 1 || n_in <= 0 || n_in > kMaxSum)
        return 0;
    return align256(n_in);
}

dq4_status_t dq4_int8_quant(const void *x, int64_t m, int64_t n_in, int64_t ld_x, int32_t dtype,
                            float threshold, int8_t *codes, int64_t ld_codes, float *scales,
                            int32_t *outliers, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (m < 0 || n_in < 0 || (dtype != DQ4_F16 && dtype != DQ4_BF16) || !(threshold >= 0.0f))
        return DQ4_EINVAL;
    if (!sizes_fit(m, 0, n_in) || m * n_in > kMaxMatrix)
        return DQ4_EUNSUPPORTED;
    const bool mixed = threshold > 0.0f;
    if (mixed != (outliers != nullptr))
        return DQ4_EINVAL;
    if (m > 0 && (!scales || (n_in > 0 && (!x || !codes || bad_ld(ld_x, m, n_in) || bad_ld(ld_codes, m, n_in)))))
        return DQ4_EINVAL;
    if (workspace_bytes < dq4_int8_quant_workspace_bytes(m, n_in, threshold) ||
        bad_workspace(workspace, workspace_bytes))
        return DQ4_EINVAL;
    if (m == 0 && !mixed)
        return DQ4_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int cus = current_compute_units();
    QuantArgs a{};
    a.x = static_cast<const uint16_t *>(x);
    a.m = m;
    a.k = n_in;
    a.ld_x = ld_x;
    a.non_finite = dtype == DQ4_F16 ? 0x7C00u : 0x7F80u;
    a.limit = mixed ? threshold_pattern(threshold, dtype) : 0x8000u;
    a.codes = codes;
    a.ld_codes = ld_codes;
    a.scales = scales;
    a.outliers = outliers;
    a.flags = static_cast<uint8_t *>(workspace);
    a.vec_in = rows_aligned(x, ld_x, m, n_in);
    a.vec_out = reinterpret_cast<uintptr_t>(codes) % 8 == 0 && n_in % 8 == 0 && (m <= 1 || ld_codes % 8 == 0);
    void *params[] = {&a};
    if (m <= 1) {
        const void *kernel = dtype == DQ4_F16
                                 ? reinterpret_cast<const void *>(&int8_quant_rows_kernel<DQ4_F16, true>)
                                 : reinterpret_cast<const void *>(&int8_quant_rows_kernel<DQ4_BF16, true>);
        return launch(kernel, 1, 1, 1024, params, s);
    }
    if (mixed && n_in > 0) {
        uint32_t *words = static_cast<uint32_t *>(workspace);
        int32_t n = static_cast<int32_t>(align256(n_in) / 4);
        void *fill[] = {&words, &n};
        const dq4_status_t st =
            launch(reinterpret_cast<const void *>(&int8_flags_zero_fill), ceil_div(n, 256), 1, 256, fill, s);
        if (st != DQ4_OK)
            return st;
    }
    const int64_t grid = m < cus * 8 ? m : cus * 8;
    const void *kernel = dtype == DQ4_F16
                             ? reinterpret_cast<const void *>(&int8_quant_rows_kernel<DQ4_F16, false>)
                             : reinterpret_cast<const void *>(&int8_quant_rows_kernel<DQ4_BF16, false>);
    const dq4_status_t st = launch(kernel, grid, 1, 256, params, s);
    if (st != DQ4_OK || !mixed)
        return st;
    const int64_t zero = ceil_div(m, 16) < cus ? ceil_div(m, 16) : cus;
    return launch(reinterpret_cast<const void *>(&int8_outliers_zero_fill), 1 + zero, 1, 1024, params, s);
}

int64_t dq4_int8_linear_workspace_bytes(const int8_t *codes, int64_t m, int64_t ld_codes, const int8_t *CB,
                                        int64_t n_out, int64_t n_in, int32_t outliers)
{
    if (m <= 0 || n_out <= 0 || n_in < 0 || !sizes_fit(m, n_out, n_in))
        return 0;
    return layout_of(codes, m, ld_codes, CB, n_out, n_in, outliers != 0, current_compute_units()).bytes();
}

dq4_status_t dq4_int8_linear(const int8_t *codes, int64_t m, int64_t ld_codes, const float *scales,
                             const int8_t *CB, const float *SCB, int64_t n_out, int64_t n_in, int32_t dtype,
                             const void *x, int64_t ld_x, const int32_t *outliers, const void *bias,
                             const void *residual, int64_t ld_residual, void *y, int64_t ld_y,
                             void *workspace, int64_t workspace_bytes, void *stream)
{
    if (m < 0 || n_out < 0 || n_in < 0 || (dtype != DQ4_F16 && dtype != DQ4_BF16))
        return DQ4_EINVAL;
    if (!sizes_fit(m, n_out, n_in))
        return DQ4_EUNSUPPORTED;
    if (m == 0 || n_out == 0)
        return DQ4_OK;
    if (!scales || !SCB || !y || (n_in > 0 && (!codes || !CB)) || ((x != nullptr) != (outliers != nullptr) && n_in > 0))
        return DQ4_EINVAL;
    if (bad_ld(ld_codes, m, n_in) || bad_ld(ld_y, m, n_out) || (residual && bad_ld(ld_residual, m, n_out)) ||
        (outliers && bad_ld(ld_x, m, n_in)))
        return DQ4_EINVAL;
    const int cus = current_compute_units();
    const Layout l = layout_of(codes, m, ld_codes, CB, n_out, n_in, outliers != nullptr, cus);
    if (workspace_bytes < l.bytes() || bad_workspace(workspace, workspace_bytes))
        return DQ4_EINVAL;
    Int8Args a{};
    a.codes = codes;
    a.ld_codes = m > 1 ? ld_codes : n_in;
    a.scales = scales;
    a.w = CB;
    a.ld_w = n_in;
    a.w_scales = SCB;
    a.m = m;
    a.n = n_out;
    a.k = a.n_in = static_cast<int32_t>(n_in);
    a.x = static_cast<const uint16_t *>(x);
    a.ld_x = ld_x;
    a.outliers = n_in > 0 ? outliers : nullptr;
    a.bias = static_cast<const uint16_t *>(bias);
    a.residual = static_cast<const uint16_t *>(residual);
    a.ld_residual = ld_residual;
    a.y = static_cast<uint16_t *>(y);
    a.ld_y = ld_y;
    a.vec = rows_aligned(y, ld_y, m, 8) && (!bias || reinterpret_cast<uintptr_t>(bias) % 16 == 0) &&
            (!residual || rows_aligned(residual, ld_residual, m, 8));
    a.splits = 1;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    hipStream_t s = static_cast<hipStream_t>(stream);
    return dtype == DQ4_F16 ? run_linear<DQ4_F16>(a, l, ws, cus, s) : run_linear<DQ4_BF16>(a, l, ws, cus, s);
}

}  // extern "C"

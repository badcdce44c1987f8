// dq4_linear_device.h -- pieces shared by the sources of the products (internal;
// not part of the C ABI): the 16-bit types, the activations, the operand layout
// of the matrix instruction, loads to LDS, the 4-bit weight's decode in
// registers, and the checks and launches of the host side.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "dq4_device.h"
#include "dq4.h"
#include "dq4_linear.h"

#pragma clang fp contract(off)

namespace dq4 {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// The 16-bit type T of a call (OUT = DQ4_F16 or DQ4_BF16): conversions from
// FP32 are one round-to-nearest-even step of a rounded FP32 value, and the
// products run on v_mfma_f32_16x16x32_{f16,bf16}: D (16 x 16, FP32) += A (16
// x 32) B (32 x 16).  Lane l holds A[l % 16][8 (l / 16) .. + 7] and
// B[8 (l / 16) .. + 7][l % 16], and D[4 (l / 16) + i][l % 16] for i = 0 .. 3.
template <int OUT>
struct Half;

template <>
struct Half<DQ4_F16> {
    typedef f16x8 Frag;
    static __device__ __forceinline__ float widen(uint32_t bits16)
    {
        return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits16)));
    }
    static __device__ __forceinline__ uint32_t pack2(float lo, float hi)
    {
        // one v_cvt_pk_f16_f32, round to nearest even
        return __builtin_bit_cast(
            uint32_t, __builtin_convertvector((f32x2{rounded_fp32(lo), rounded_fp32(hi)}), f16x2));
    }
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(Frag, a),
                                                      __builtin_bit_cast(Frag, b), c, 0, 0, 0);
    }
};

template <>
struct Half<DQ4_BF16> {
    typedef bf16x8 Frag;
    static __device__ __forceinline__ float widen(uint32_t bits16)
    {
        return __builtin_bit_cast(float, bits16 << 16);
    }
    static __device__ __forceinline__ uint32_t pack2(float lo, float hi)
    {
        // one v_cvt_pk_bf16_f32, round to nearest even
        return __builtin_bit_cast(
            uint32_t, __builtin_convertvector((f32x2{rounded_fp32(lo), rounded_fp32(hi)}), bf16x2));
    }
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(Frag, a),
                                                       __builtin_bit_cast(Frag, b), c, 0, 0, 0);
    }
};

// ---------------------------------------------------------------------------
// activations, in FP32
// ---------------------------------------------------------------------------
// exp(x) as 2^(x log2 e): the rounding of x log2 e leaves a relative error of
// about |x| 2^-24, at most 6e-6 where the result is a normal FP32 number, far
// below the half step of FP16 or BF16 that the results are rounded to (the
// bias gradient, in FP32, keeps it).
__device__ __forceinline__ float exp_f32(float x)
{
    return __builtin_amdgcn_exp2f(x * 1.44269504088896341f);
}

// 1 / (1 + exp(-x)); the reciprocal instruction is within 1 ulp.
__device__ __forceinline__ float sigmoid_f32(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + exp_f32(-x));
}

// erfc(|x|): the Chebyshev fit t exp(-x^2 + P(t)), t = 1 / (1 + |x| / 2), of
// Press, Teukolsky, Vetterling and Flannery, "Numerical Recipes" (erfcc).  The
// fit's own relative error is below 1.2e-7; here the exponent, about x^2 in
// size, is rounded three times, which adds up to 1.5 x^2 2^-23 (1.5e-5 at x =
// 9), and results below 2^-126, from |x| = 9.2 on, are flushed to 0.
__device__ __forceinline__ float erfc_abs_f32(float x)
{
    const float z = __builtin_fabsf(x);
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.5f * z);
    float p = 0.17087277f;
    p = -0.82215223f + t * p;
    p = 1.48851587f + t * p;
    p = -1.13520398f + t * p;
    p = 0.27886807f + t * p;
    p = -0.18628806f + t * p;
    p = 0.09678418f + t * p;
    p = 0.37409196f + t * p;
    p = 1.00002368f + t * p;
    p = -1.26551223f + t * p;
    return t * exp_f32(-z * z + p);
}

// The normal distribution's integral, erfc(-z / sqrt 2) / 2.
__device__ __forceinline__ float normal_cdf_f32(float z)
{
    const float half_tail = 0.5f * erfc_abs_f32(z * 0.70710678118654752f);
    return z > 0.0f ? 1.0f - half_tail : half_tail;
}

constexpr float kGeluTwoC = 1.59576912160573071f;     // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// The tanh form's 2 v, v = sqrt(2/pi) (z + 0.044715 z^3), with z held to [-64,
// 64]: the sigmoid is 0 or 1 long before that, and z^3 cannot overflow.  A NaN
// gives -64: what is computed from it has to take the NaN from z itself.
__device__ __forceinline__ float gelu_clamp(float z)
{
    return __builtin_amdgcn_fmed3f(z, -64.0f, 64.0f);
}

// z held to [-bound, bound]; a NaN stays.
__device__ __forceinline__ float held(float z, float bound)
{
    return z != z ? z : __builtin_amdgcn_fmed3f(z, -bound, bound);
}

// act(z); z/2 (1 + tanh v) is z sigmoid(2 v).
__device__ __forceinline__ float act_f32(int act, float z)
{
    switch (act) {
    case DQ4_ACT_RELU:
        return z < 0.0f ? 0.0f : z;
    case DQ4_ACT_SILU:
        return z * sigmoid_f32(z);
    case DQ4_ACT_GELU:
        return z * normal_cdf_f32(z);
    case DQ4_ACT_GELU_TANH: {
        const float c = gelu_clamp(z);
        return z * sigmoid_f32(kGeluTwoC * (c + kGeluCubic * (c * c * c)));
    }
    default:
        return z;
    }
}

// act(z) and its derivative, for a saved z: a NaN gives NaN, and the
// infinities, which a 16-bit z reaches by overflow, give the limits (the
// formulas alone give 0 times infinity there).  `c` is z with the infinities
// held to the largest finite number, whose products with a vanished sigmoid or
// density are 0; z itself is multiplied only where it is not negative infinity.
__device__ __forceinline__ void act_and_slope_f32(int act, float z, float *value, float *slope)
{
    constexpr float kMax = 3.402823466e+38f;
    switch (act) {
    case DQ4_ACT_RELU:
        *value = z < 0.0f ? 0.0f : z;
        *slope = z > 0.0f ? 1.0f : z != z ? z : 0.0f;
        return;
    case DQ4_ACT_SILU: {
        const float s = sigmoid_f32(z), c = held(z, kMax);
        *value = (z > 0.0f ? z : c) * s;
        *slope = s * (1.0f + c * (1.0f - s));
        return;
    }
    case DQ4_ACT_GELU: {
        const float p = normal_cdf_f32(z), c = held(z, kMax);
        *value = (z > 0.0f ? z : c) * p;
        *slope = p + c * (kInvSqrt2Pi * exp_f32(-0.5f * (z * z)));
        return;
    }
    case DQ4_ACT_GELU_TANH: {
        const float c = held(z, 64.0f);
        const float s = sigmoid_f32(kGeluTwoC * (c + kGeluCubic * (c * c * c)));
        *value = (z > 0.0f ? z : c) * s;
        *slope = s + c * s * (1.0f - s) * (kGeluTwoC * (1.0f + 3.0f * kGeluCubic * (c * c)));
        return;
    }
    default:
        *value = z;
        *slope = 1.0f;
        return;
    }
}

// ---------------------------------------------------------------------------
// matrices and weights
// ---------------------------------------------------------------------------
struct Weight {
    const uint8_t *packed;
    const uint8_t *scale_codes;
    const float *nested_absmax;
    const float *scale_codebook;
    const float *codebook4;
    float offset;
};

template <int OUT, int N>
__device__ __forceinline__ void load_values(const uint16_t *p, bool vec, int valid, float (&v)[N])
{
    if (vec) {
        if constexpr (N == 8) {
            const u32x4 q = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = Half<OUT>::widen((q[j / 2] >> (16 * (j & 1))) & 0xFFFFu);
        } else if constexpr (N == 4) {
            const u32x2 q = *reinterpret_cast<const u32x2 *>(p);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = Half<OUT>::widen((q[j / 2] >> (16 * (j & 1))) & 0xFFFFu);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            v[j] = j < valid ? Half<OUT>::widen(p[j]) : 0.0f;
    }
}

template <int OUT, int N>
__device__ __forceinline__ void store_values(uint16_t *p, bool vec, int valid, const float (&v)[N])
{
    if (vec && N > 1) {
        uint32_t q[N / 2 + 1];
#pragma unroll
        for (int j = 0; j < N / 2; ++j)
            q[j] = Half<OUT>::pack2(v[2 * j], v[2 * j + 1]);
        if constexpr (N == 8)
            *reinterpret_cast<u32x4 *>(p) = u32x4{q[0], q[1], q[2], q[3]};
        else if constexpr (N == 4)
            *reinterpret_cast<u32x2 *>(p) = u32x2{q[0], q[1]};
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < valid)
                p[j] = static_cast<uint16_t>(Half<OUT>::pack2(v[j], 0.0f));
    }
}

__device__ __forceinline__ uint32_t lds_offset(const void *p)
{
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) const void *)p));
}

// 16 bytes per lane from a buffer straight to LDS at `lds` + 16 lane; a lane
// whose offset is out of the buffer's range gets zeros.  In asm (there is no
// destination register): the compiler would make every LDS read wait for
// these loads, also where they fill the other half of the double buffer; the
// kernel's own wait and barrier order them.  (m0 needs one wait state before
// the load reads it; the compiler never keeps a value in it across statements.)
__device__ __forceinline__ void buffer_to_lds(u32x4 rsrc, uint32_t voffset, uint32_t soffset,
                                              uint32_t lds)
{
    __asm__ volatile("s_mov_b32 m0, %0\n\t"
                     "s_nop 0\n\t"
                     "buffer_load_dwordx4 %1, %2, %3 offen lds"
                     :
                     : "s"(lds), "v"(voffset), "s"(rsrc), "s"(soffset)
                     : "memory");
}

__device__ __forceinline__ u32x4 make_rsrc(const void *base, uint32_t bytes)
{
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    u32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b));
    r[1] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32) & 0xFFFFu);
    r[2] = __builtin_amdgcn_readfirstlane(bytes);
    r[3] = kRawBufferWord3;
    return r;
}

__device__ __forceinline__ void wait_all_and_barrier()
{
    __asm__ volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
// the 4-bit weight decoded in registers
// ---------------------------------------------------------------------------
// The two values of a packed byte, low nibble first, in copies that the lanes
// share out: entry b at byte 256 b, in it 32 copies of 8 bytes (one weight) or
// 16 copies of both weights' pairs (gated).  The address of a lookup is one
// byte permute, and lanes that are served together read different banks
// whatever their codes: of a wave's 8-byte lookups 16 lanes are served at a
// time (16 copies measured 2.7 ns per lookup and CU, 32 copies 2.4, 8 copies
// 4.4, a single table 26).
constexpr int kPairTableBytes = 256 * 32 * 8;

// A barrier for LDS alone: it does not wait for the loads that the wave has
// under way from memory, as __syncthreads() does.
__device__ __forceinline__ void lds_barrier()
{
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
}

// The codebooks' way into LDS, in two parts: `fetch_codebooks` goes before a
// kernel's first weight loads (loads return in order: behind them the tables
// would wait for the weight), `fill_tables` after them.  It fills kTables
// tables (kTables == 1 and two weights: one table of both, 16 copies each),
// the row of zeros behind them and the scale codebooks; every thread of the
// workgroup (256 or more) calls it, and it ends on a barrier.  The 16 values
// pass through LDS: taken from memory entry by entry they cost 5 us at the
// start of every call.
struct Codebooks {
    float scb[2];
    float cb4;
};

template <int kWeights>
__device__ __forceinline__ Codebooks fetch_codebooks(const Weight (&w)[2])
{
    const int tid = threadIdx.x, threads = blockDim.x;
    // without branches: a load that some threads skip makes the compiler lose
    // count of the loads under way, and wait for all of them
    Codebooks c;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int i = (tid + q * threads) % (kWeights * 256);
        c.scb[q] = w[kWeights == 2 ? i >> 8 : 0].scale_codebook[i & 255];
    }
    c.cb4 = w[kWeights == 2 ? (tid >> 4) & 1 : 0].codebook4[tid & 15];
    return c;
}

template <int kWeights, int kTables>
__device__ __forceinline__ void fill_tables(const Codebooks &c, uint8_t *table,
                                            float (&scb)[kWeights][256], float (&cb4)[kWeights][16])
{
    const int tid = threadIdx.x, threads = blockDim.x;
    // every thread stores (the rest over the table that is filled below), so
    // that no load is moved behind a branch
    float *rest = reinterpret_cast<float *>(table) + tid;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int i = tid + q * threads;
        *(i < kWeights * 256 ? &scb[i >> 8][i & 255] : rest) = c.scb[q];
    }
    *(tid < kWeights * 16 ? &cb4[tid >> 4][tid & 15] : rest) = c.cb4;
    if (tid < 64)
        *reinterpret_cast<uint32_t *>(&table[kTables * kPairTableBytes + tid * 4]) = 0;
    lds_barrier();
#pragma unroll 8
    for (int i = tid; i < kTables * 256 * 32; i += threads) {
        const int b = (i >> 5) & 255, which = kTables == 2 ? i >> 13 : kWeights == 2 ? i & 1 : 0;
        *reinterpret_cast<f32x2 *>(&table[i * 8]) = f32x2{cb4[which][b & 15], cb4[which][b >> 4]};
    }
    lds_barrier();
}

struct Pairs {
    f32x2 v[4];  // the eight codebook values of a packed dword
};

__device__ __forceinline__ Pairs lookup_dword(uint32_t word, const uint8_t *table,
                                              uint32_t lane_byte)
{
    Pairs p;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // lane_byte with the word's byte j as its byte 1
        const uint32_t at = __builtin_amdgcn_perm(word, lane_byte, 0x03020000u | ((4u + j) << 8));
        p.v[j] = *reinterpret_cast<const f32x2 *>(table + at);
    }
    return p;
}

template <int OUT>
__device__ __forceinline__ u32x4 scaled_dword(const Pairs &p, float s)
{
    u32x4 q;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        q[j] = Half<OUT>::pack2(p.v[j][0] * s, p.v[j][1] * s);
    return q;
}

template <int OUT>
__device__ __forceinline__ u32x4 decode_dword(uint32_t word, float s, const uint8_t *table,
                                              uint32_t lane_byte)
{
    return scaled_dword<OUT>(lookup_dword(word, table, lane_byte), s);
}

// The lookups before this line are issued before what follows it: left to
// itself the compiler waits for each lookup where it is used.
__device__ __forceinline__ void keep_order()
{
    __builtin_amdgcn_sched_barrier(0);
}

// Lane l of each quad exchanges register j for lane j's register l.
__device__ __forceinline__ void transpose_quads(uint32_t (&v)[4], bool odd, bool high)
{
    const auto xor1 = [](uint32_t a) {
        return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(a), 0xB1, 0xF, 0xF, true));
    };
    const auto xor2 = [](uint32_t a) {
        return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(a), 0x4E, 0xF, 0xF, true));
    };
    // every lane makes every exchange; only then does it choose
    const uint32_t x0 = xor1(v[0]), x1 = xor1(v[1]), x2 = xor1(v[2]), x3 = xor1(v[3]);
    const uint32_t a0 = odd ? x1 : v[0], a1 = odd ? v[1] : x0;
    const uint32_t a2 = odd ? x3 : v[2], a3 = odd ? v[3] : x2;
    const uint32_t y0 = xor2(a0), y1 = xor2(a1), y2 = xor2(a2), y3 = xor2(a3);
    v[0] = high ? y2 : a0;
    v[1] = high ? y3 : a1;
    v[2] = high ? a2 : y0;
    v[3] = high ? a3 : y1;
}

// ---------------------------------------------------------------------------
// lists
// ---------------------------------------------------------------------------
// Inclusive prefix sum over a wave.
__device__ __forceinline__ int wave_prefix(int v, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int other = __shfl_up(v, d);
        v += lane >= d ? other : 0;
    }
    return v;
}

// The positions of `count` entries of each of the workgroup's threads in a list:
// the number before this thread's, and all of them in *total.
template <int THREADS>
__device__ __forceinline__ int list_position(int count, int *total, int (&sums)[THREADS / 64])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int upto = wave_prefix(count, lane);
    __syncthreads();  // sums may still be read
    if (lane == 63)
        sums[wave] = upto;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
        before += w < wave ? sums[w] : 0;
        all += sums[w];
    }
    *total = all;
    return before + upto - count;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
inline int64_t ceil_div(int64_t a, int64_t b)
{
    return (a + b - 1) / b;
}

inline int64_t align256(int64_t b)
{
    return (b + 255) & ~int64_t{255};
}

inline dq4_status_t launch(const void *kernel, int64_t gx, int64_t gy, int threads, void **params,
                    hipStream_t s)
{
    // a launch of 2^32 threads or more along x runs a part of them, without an error
    if (gx * threads > 0xFFFFFFFF || gy > 65535)
        return DQ4_EUNSUPPORTED;
    const hipError_t e = hipLaunchKernel(kernel, dim3(static_cast<uint32_t>(gx), static_cast<uint32_t>(gy)),
                                         dim3(threads), params, 0, s);
    return e == hipSuccess ? DQ4_OK : hip_failed(e);
}

inline bool rows_aligned(const void *p, int64_t ld, int64_t rows, int64_t width)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld % 8 == 0) && width % 8 == 0;
}

inline int current_compute_units()
{
    int device = 0;
    if (hipGetDevice(&device) != hipSuccess) {
        (void)hipGetLastError();
        return 256;
    }
    return compute_units(device);
}

inline Weight device_weight(const dq4_weight_t &w)
{
    return Weight{w.packed, w.scale_codes, w.nested_absmax, w.scale_codebook, w.codebook4, w.offset};
}

inline bool bad_workspace(const void *workspace, int64_t bytes)
{
    return bytes > 0 && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0);
}

inline bool weight_missing(const dq4_weight_t *w)
{
    return !w->packed || !w->scale_codes || !w->nested_absmax || !w->scale_codebook || !w->codebook4;
}

// A row stride that rows of this width cannot have.
inline bool bad_ld(int64_t ld, int64_t m, int64_t width)
{
    return m > 1 && (ld < width || ld > INT64_MAX / 2 / m);
}

}  // namespace dq4

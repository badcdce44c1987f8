// Sanitizer driver for the host side of include/dq4_int8.h (without the gradient) and
// include/dq4_moe.h (a test, built by tests/test_int8_moe_sanitizers.py with
// AddressSanitizer and UBSan on the host code only): calls that are rejected or have
// nothing to do, and the workspace sizes, which choose the kernels, over sizes up to
// and beyond the limits.  No call reaches the GPU, so it runs on a machine without one.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "dq4_int8.h"
#include "dq4_moe.h"

static int failures = 0;
static void expect(int64_t got, int64_t want, const char *what)
{
    if (got != want) {
        printf("%s: got %lld want %lld\n", what, static_cast<long long>(got), static_cast<long long>(want));
        ++failures;
    }
}

static const int64_t kSizes[] = {INT64_MIN, -1, 0, 1, 8, 16, 17, 31, 64, 65, 1000, 4096, 4097, 131071, 131072, 131073,
                                 (1 << 21) - 1, 1 << 21, (1 << 21) + 1, int64_t{1} << 40, INT64_MAX};
static const int32_t kCounts[] = {INT32_MIN, -1, 0, 1, 2, 16, 17, 64, 512, 513, INT32_MAX};

int main()
{
    void *pv = reinterpret_cast<void *>(0x1000);
    uint8_t *p8 = reinterpret_cast<uint8_t *>(0x1000);
    int8_t *codes = reinterpret_cast<int8_t *>(0x1000);
    int32_t *ids = reinterpret_cast<int32_t *>(0x1000);
    float *pf = reinterpret_cast<float *>(0x1000);
    const dq4_weight_t w = {p8, p8, pf, pf, pf, 0.03f, 64, 256};
    const dq4_weight_t none = {nullptr, nullptr, nullptr, nullptr, nullptr, 0.f, 64, 256};
    const int64_t big = INT64_MAX, most = int64_t{1} << 38;

    for (int64_t m : kSizes)
        for (int64_t k : kSizes) {
            const bool fits = m >= 0 && k >= 0 && m <= (1 << 21) && k <= 131071 && (m == 0 || k <= most / m);
            for (float threshold : {0.0f, 6.0f, HUGE_VALF}) {
                expect(dq4_int8_quant_workspace_bytes(m, k, threshold) >= 0, 1, "quant workspace");
                if (!fits)
                    expect(dq4_int8_quant(pv, m, k, big, DQ4_F16, threshold, codes, big, pf,
                                          threshold > 0 ? ids : nullptr, pv, big, nullptr) != DQ4_OK, 1, "quant sizes");
            }
            for (int64_t n : kSizes) {
                const bool ok = fits && n >= 0 && n <= (1 << 21) && (m == 0 || n <= most / m);
                for (int32_t outliers = 0; outliers < 2; ++outliers)
                    for (int64_t ld : {k, int64_t{0}, INT64_MAX}) {
                        const int64_t s = dq4_int8_linear_workspace_bytes(codes, m, ld, codes + 1, n, k, outliers);
                        expect(ok && m > 0 && n > 0 ? s >= 0 : s == 0, 1, "linear workspace");
                    }
                const dq4_status_t st =
                    ok && m > 0 && n > 0
                        ? dq4_int8_linear(codes, m, big, pf, codes, pf, n, k, DQ4_BF16, nullptr, 0, nullptr, nullptr, nullptr,
                                          0, nullptr, big, pv, big, nullptr)
                        : dq4_int8_linear(codes, m, big, pf, codes, pf, n, k, DQ4_BF16, nullptr, 0, nullptr, nullptr, nullptr,
                                          0, pv, big, pv, big, nullptr);
                expect(st == DQ4_OK, ok && (m == 0 || n == 0), "linear sizes");
            }
        }
    for (int64_t ld : {INT64_MIN, int64_t{-1}, int64_t{0}, int64_t{63}, INT64_MAX / 2, INT64_MAX}) {
        expect(dq4_int8_quant(pv, 3, 64, ld, DQ4_F16, 0.0f, codes, 64, pf, nullptr, pv, big, nullptr), DQ4_EINVAL, "ld_x");
        expect(dq4_int8_quant(pv, 3, 64, 64, DQ4_F16, 0.0f, codes, ld, pf, nullptr, pv, big, nullptr), DQ4_EINVAL, "ld_codes");
        expect(dq4_int8_linear(codes, 3, ld, pf, codes, pf, 64, 64, DQ4_F16, nullptr, 0, nullptr, nullptr, nullptr, 0, pv, 64,
                               pv, big, nullptr), DQ4_EINVAL, "linear ld_codes");
        expect(dq4_int8_linear(codes, 3, 64, pf, codes, pf, 64, 64, DQ4_F16, nullptr, 0, nullptr, nullptr, pv, ld, pv, 64,
                               pv, big, nullptr), DQ4_EINVAL, "linear ld_residual");
        expect(dq4_moe_route(pv, 3, 64, ld, DQ4_F16, pv, nullptr, 8, 2, 1, ids, pf, pv, big, nullptr), DQ4_EINVAL, "route ld");
        expect(dq4_moe_fused(&w, &w, &w, 4, 64, 64, DQ4_F16, DQ4_ACT_SILU, pv, 3, 64, ids, pf, 2, nullptr, 0, pv, ld, pv, big,
                             nullptr), DQ4_EINVAL, "experts ld_y");
    }

    for (int64_t m : kSizes)
        for (int32_t E : kCounts) {
            expect(dq4_moe_route_workspace_bytes(m, E) >= 0, 1, "route workspace");
            for (int32_t top_k : kCounts)
                for (int64_t n : kSizes) {
                    const bool asked = m >= 0 && n >= 0 && E >= 0 && top_k >= 1;
                    const bool route = asked && top_k <= E && E <= 512 && top_k <= 16 && m <= (1 << 21) && n <= (1 << 17);
                    expect(dq4_moe_route(pv, m, n, big, DQ4_BF16, pv, nullptr, E, top_k, 0, nullptr, pf, pv, big, nullptr) ==
                               DQ4_OK, route && m == 0, "route sizes");
                    for (int64_t n_ff : {INT64_MIN, int64_t{0}, int64_t{1000}, int64_t{1} << 17, INT64_MAX}) {
                        const bool fits = asked && E >= 1 && n_ff >= 0 && E <= 512 && top_k <= 16 && m <= 64 &&
                                          n_ff <= (1 << 17) && n <= (1 << 17) &&
                                          E * n_ff * n <= (int64_t{1} << 40);
                        const int64_t s = dq4_moe_fused_workspace_bytes(E, n_ff, n, m, top_k);
                        expect(fits && m > 0 && n > 0 ? s > 0 : s == 0, 1, "experts workspace");
                        expect(dq4_moe_fused(&w, &w, &w, E, n_ff, n, DQ4_BF16, DQ4_ACT_GELU, pv, m, big, nullptr, pf, top_k,
                                             nullptr, 0, pv, big, pv, big, nullptr) == DQ4_OK,
                               fits && (m == 0 || n == 0), "experts sizes");
                    }
                }
        }
    for (const dq4_weight_t *wt : {static_cast<const dq4_weight_t *>(nullptr), &none}) {
        expect(dq4_moe_fused(wt, &w, &w, 4, 64, 64, DQ4_F16, 1, pv, 3, 64, ids, pf, 2, nullptr, 0, pv, 64, pv, big, nullptr),
               DQ4_EINVAL, "no gate");
        expect(dq4_moe_fused(&w, &w, wt, 4, 64, 64, DQ4_F16, 1, pv, 3, 64, ids, pf, 2, nullptr, 0, pv, 64, pv, big, nullptr),
               DQ4_EINVAL, "no down");
    }
    expect(dq4_int8_quant(pv, 3, 64, 64, DQ4_F16, NAN, codes, 64, pf, ids, pv, big, nullptr), DQ4_EINVAL, "threshold");
    expect(dq4_int8_quant(pv, 3, 64, 64, INT32_MAX, 6.0f, codes, 64, pf, ids, pv, big, nullptr), DQ4_EINVAL, "type");
    expect(dq4_moe_fused(&w, &w, &w, 4, 64, 64, DQ4_F16, INT32_MIN, pv, 3, 64, ids, pf, 2, nullptr, 0, pv, 64, pv, big,
                         nullptr), DQ4_EINVAL, "activation");
    expect(dq4_moe_fused(&w, &w, &w, 4, 64, 64, DQ4_F16, 1, pv, 3, 64, ids, pf, 2, nullptr, 0, pv, 64, pv, INT64_MIN,
                         nullptr), DQ4_EINVAL, "negative workspace");
    printf("int8 and experts abi sanitizer driver: %d failures\n", failures);
    return failures != 0;
}

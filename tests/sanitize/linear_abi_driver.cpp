// Sanitizer driver for the host side of include/dq4_linear.h (a test, built by
// tests/test_linear_sanitizers.py with AddressSanitizer and UBSan on the host
// code only): calls that are rejected or have nothing to do, and the workspace
// sizes, which choose the kernels, over sizes up to and beyond the limits.  No
// call reaches the GPU, so it runs on a machine without one.
#include <stdint.h>
#include <stdio.h>

#include "dq4_linear.h"

static int failures = 0;
static void expect(int64_t got, int64_t want, const char *what)
{
    if (got != want) {
        printf("%s: got %lld want %lld\n", what, static_cast<long long>(got), static_cast<long long>(want));
        ++failures;
    }
}

static const int64_t kSizes[] = {INT64_MIN, -1, 0, 1, 7, 8, 31, 32, 64, 65, 1000, 1024, 1025, 2048, 32768, 32800,
                                 (1 << 20) + 8, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, int64_t{1} << 40, INT64_MAX};

int main()
{
    void *pv = reinterpret_cast<void *>(0x1000);
    const uint8_t *p8 = reinterpret_cast<uint8_t *>(0x1000);
    const float *pf = reinterpret_cast<float *>(0x1000);
    float *out = reinterpret_cast<float *>(0x1000);
    const dq4_weight_t w = {p8, p8, pf, pf, pf, 0.03f, 64, 256};
    const dq4_weight_t odd = {p8 + 1, p8, pf, pf, pf, 0.03f, 64, 256};
    const dq4_weight_t none = {nullptr, nullptr, nullptr, nullptr, nullptr, 0.f, 64, 256};
    const int64_t big = INT64_MAX;

    for (const dq4_weight_t *wt : {&w, &odd})
        for (int64_t m : kSizes)
            for (int64_t n : kSizes)
                for (int64_t k : kSizes)
                    for (int32_t least = 0; least < 2; ++least) {
                        const bool ok = n > 0 && k >= 0 && m > 0 && n <= (1 << 21) && k <= (1 << 21) && m <= (1 << 21) &&
                                        m * n <= (int64_t{1} << 39) && m * k <= (int64_t{1} << 39);
                        for (const void *x : {static_cast<const void *>(pv), static_cast<const void *>(p8 + 2)})
                            for (int64_t ld : {k, int64_t{0}, INT64_MAX}) {
                                const int64_t sizes[4] = {
                                    dq4_linear_fused_workspace_bytes(wt, n, k, m, x, ld, least),
                                    dq4_gated_fused_workspace_bytes(wt, &w, n, k, m, x, ld, least),
                                    dq4_linear_fused_backward_workspace_bytes(wt, n, k, m, x, ld, least),
                                    dq4_gated_fused_backward_workspace_bytes(&w, wt, n, k, m, x, x, ld, least)};
                                for (int64_t s : sizes)
                                    expect(ok ? s >= 0 : s == 0, 1, "workspace size");
                            }
                        if (ok)
                            continue;
                        // sizes that the calls reject, or have nothing to write for
                        const dq4_status_t st = dq4_linear_fused(wt, n, k, DQ4_BF16, DQ4_ACT_SILU, pv, m, big, pv, pv, big, pv,
                                                                 big, pv, big, pv, big, nullptr);
                        const bool empty = m >= 0 && n >= 0 && k >= 0 && m <= (1 << 21) && n <= (1 << 21) && k <= (1 << 21) &&
                                           (m == 0 || n == 0);
                        expect(st == DQ4_OK, empty && m * k <= (int64_t{1} << 39), "linear of rejected sizes");
                        const dq4_status_t sg = dq4_gated_fused(wt, &w, n, k, DQ4_F16, DQ4_ACT_GELU, pv, m, big, pv, big, pv,
                                                                pv, big, pv, big, nullptr);
                        expect(sg, st, "gated of rejected sizes");
                    }

    // leading dimensions whose products overflow, missing operands and workspaces
    for (int64_t ld : {INT64_MIN, int64_t{-1}, int64_t{0}, int64_t{63}, INT64_MAX / 2, INT64_MAX}) {
        expect(dq4_linear_fused(&w, 64, 64, DQ4_F16, DQ4_ACT_NONE, pv, 3, ld, nullptr, nullptr, 0, pv, 64, nullptr, 0, pv, big,
                                nullptr), DQ4_EINVAL, "ld_x");
        expect(dq4_linear_fused(&w, 64, 64, DQ4_F16, DQ4_ACT_NONE, pv, 3, 64, nullptr, pv, ld, pv, 64, nullptr, 0, pv, big,
                                nullptr), DQ4_EINVAL, "ld_residual");
        expect(dq4_linear_fused_backward(&w, 64, 64, DQ4_F16, DQ4_ACT_GELU, pv, 3, ld, pv, 64, pv, 64, pv, 64, out, pv, big,
                                         nullptr), DQ4_EINVAL, "ld_dy");
        expect(dq4_gated_fused_backward(&w, &w, 64, 64, DQ4_F16, DQ4_ACT_GELU, pv, 3, 64, pv, pv, 64, pv, 64, pv, pv, ld, pv,
                                        big, nullptr), DQ4_EINVAL, "ld_dpre");
    }
    expect(dq4_linear_fused(nullptr, 64, 64, DQ4_F16, 0, pv, 3, 64, nullptr, nullptr, 0, pv, 64, nullptr, 0, pv, big, nullptr),
           DQ4_EINVAL, "no weight");
    expect(dq4_linear_fused(&none, 64, 64, DQ4_F16, 0, pv, 3, 64, nullptr, nullptr, 0, pv, 64, nullptr, 0, pv, big, nullptr),
           DQ4_EINVAL, "an empty weight");
    expect(dq4_linear_fused(&w, 64, 64, DQ4_F16, 0, pv, 3, 64, nullptr, nullptr, 0, pv, 64, nullptr, 0, pv, INT64_MIN, nullptr),
           DQ4_EINVAL, "negative workspace");
    expect(dq4_linear_fused(&w, 64, 64, DQ4_F16, 0, pv, 3, 64, nullptr, nullptr, 0, pv, 64, nullptr, 0,
                            reinterpret_cast<void *>(0x1010), big, nullptr), DQ4_EINVAL, "workspace off 256 bytes");
    expect(dq4_gated_fused(&w, nullptr, 64, 64, DQ4_F16, DQ4_ACT_SILU, pv, 3, 64, pv, 64, nullptr, nullptr, 0, pv, big, nullptr),
           DQ4_EINVAL, "no up weight");
    expect(dq4_gated_fused(&w, &w, 64, 64, DQ4_F16, DQ4_ACT_NONE, pv, 3, 64, pv, 64, nullptr, nullptr, 0, pv, big, nullptr),
           DQ4_EINVAL, "gated without activation");
    expect(dq4_linear_fused_backward(&w, 64, 64, DQ4_F16, INT32_MIN, pv, 3, 64, pv, 64, pv, 64, pv, 64, out, pv, big, nullptr),
           DQ4_EINVAL, "activation");
    expect(dq4_linear_fused_backward(&w, 64, 64, INT32_MAX, 1, pv, 3, 64, pv, 64, pv, 64, pv, 64, out, pv, big, nullptr),
           DQ4_EINVAL, "type");
    expect(dq4_linear_fused_backward(&w, 64, 64, DQ4_F16, 1, pv, 0, 64, pv, 64, pv, 64, pv, 64, nullptr, pv, big, nullptr),
           DQ4_OK, "no rows");
    expect(dq4_gated_fused_backward(&w, &w, 64, 64, DQ4_F16, 1, pv, 0, 64, pv, pv, 64, pv, 64, pv, pv, 64, pv, big, nullptr),
           DQ4_OK, "gated, no rows");
    printf("linear abi sanitizer driver: %d failures\n", failures);
    return failures != 0;
}

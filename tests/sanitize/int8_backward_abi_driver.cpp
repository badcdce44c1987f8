// Sanitizer driver for the host side of the gradient in include/dq4_int8.h (a test,
// built by tests/test_int8_backward_sanitizers.py with AddressSanitizer and UBSan on the
// host code only): calls that are rejected or have nothing to do, and the workspace
// sizes, which follow from the plans of both of its ways, over sizes up to and beyond
// the limits.  No call reaches the GPU, so it runs on a machine without one.
#include <stdint.h>
#include <stdio.h>

#include "dq4_int8.h"

static int failures = 0;
static void expect(int64_t got, int64_t want, const char *what, int64_t n_out, int64_t n_in, int64_t m)
{
    if (got != want) {
        printf("%s (%lld x %lld, %lld tokens): got %lld want %lld\n", what, static_cast<long long>(n_out),
               static_cast<long long>(n_in), static_cast<long long>(m), static_cast<long long>(got),
               static_cast<long long>(want));
        ++failures;
    }
}

static const int64_t kSizes[] = {INT64_MIN, -1, 0, 1, 7, 8, 16, 17, 32, 33, 64, 127, 128, 129, 130, 256, 1000, 2376, 4096,
                                 4097, 131073, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, int64_t{1} << 40, INT64_MAX};

int main()
{
    void *pv = reinterpret_cast<void *>(0x1000);
    const int8_t *codes = reinterpret_cast<const int8_t *>(0x1000);
    float *pf = reinterpret_cast<float *>(0x1000);
    const int64_t big = INT64_MAX, top = int64_t{1} << 21, most = int64_t{1} << 38;

    for (int64_t n_out : kSizes)
        for (int64_t n_in : kSizes)
            for (int64_t m : kSizes) {
                const bool asked = n_out >= 0 && n_in >= 0 && m >= 0;
                const bool fits = asked && n_out <= top && n_in <= top && m <= top && m * n_out <= most && m * n_in <= most;
                int64_t least = 0;
                for (const void *dy : {pv, reinterpret_cast<void *>(0x1002)})
                    for (int64_t ld : {n_out, int64_t{0}, (int64_t{1} << 22) + 8, INT64_MAX}) {
                        const int64_t s = dq4_int8_linear_backward_workspace_bytes(n_out, n_in, m, dy, ld);
                        if (!fits || n_out == 0 || m == 0)
                            expect(s >= 0, 1, "workspace", n_out, n_in, m);
                        else if (m <= 128 && n_in > 0) {
                            // split sums of whole tiles: 16 or 32 tokens by 128 columns, FP32
                            const int64_t tile = m <= 16 ? 16 : 32;
                            const int64_t once = (m + tile - 1) / tile * tile * ((n_in + 127) / 128 * 128) * 4;
                            expect(s > 0 && s % once == 0, 1, "few tokens' workspace", n_out, n_in, m);
                        } else if (n_in > 0) {
                            // the 16-bit copy of the weight, in groups of 128 columns by 64 rows
                            const int64_t copy = (n_in + 127) / 128 * 128 * ((n_out + 63) / 64 * 64) * 2;
                            expect(s >= copy, 1, "workspace with the copy", n_out, n_in, m);
                        }
                        least = s;
                    }
                if (!asked || !fits) {
                    expect(dq4_int8_linear_backward(codes, pf, n_out, n_in, DQ4_BF16, pv, m, big, pv, big, pf, pv, big, nullptr),
                           asked ? DQ4_EUNSUPPORTED : DQ4_EINVAL, "sizes", n_out, n_in, m);
                    continue;
                }
                if (m == 0)
                    expect(dq4_int8_linear_backward(nullptr, nullptr, n_out, n_in, DQ4_F16, nullptr, 0, 0, nullptr, 0, nullptr,
                                                    nullptr, 0, nullptr), DQ4_OK, "no tokens", n_out, n_in, m);
                if (m == 0 || n_out == 0)
                    continue;
                // every missing operand, row stride and workspace is refused before a launch
                expect(dq4_int8_linear_backward(codes, pf, n_out, n_in, DQ4_F16, nullptr, m, n_out, pv, n_in, nullptr, pv, big,
                                                nullptr), DQ4_EINVAL, "no dy", n_out, n_in, m);
                if (m > 1)
                    for (int64_t ld : {INT64_MIN, int64_t{-1}, n_out - 1, INT64_MAX})
                        expect(dq4_int8_linear_backward(codes, pf, n_out, n_in, DQ4_F16, pv, m, ld, pv, n_in, nullptr, pv, big,
                                                        nullptr), DQ4_EINVAL, "ld_dy", n_out, n_in, m);
                if (n_in > 0) {
                    expect(dq4_int8_linear_backward(nullptr, pf, n_out, n_in, DQ4_F16, pv, m, n_out, pv, n_in, nullptr, pv, big,
                                                    nullptr), DQ4_EINVAL, "no CB", n_out, n_in, m);
                    expect(dq4_int8_linear_backward(codes, nullptr, n_out, n_in, DQ4_F16, pv, m, n_out, pv, n_in, nullptr, pv,
                                                    big, nullptr), DQ4_EINVAL, "no SCB", n_out, n_in, m);
                    expect(dq4_int8_linear_backward(codes, pf, n_out, n_in, DQ4_F16, pv, m, n_out, nullptr, n_in, nullptr, pv,
                                                    big, nullptr), DQ4_EINVAL, "no dx", n_out, n_in, m);
                    if (m > 1)
                        for (int64_t ld : {INT64_MIN, int64_t{-1}, n_in - 1, INT64_MAX})
                            expect(dq4_int8_linear_backward(codes, pf, n_out, n_in, DQ4_F16, pv, m, n_out, pv, ld, nullptr, pv,
                                                            big, nullptr), DQ4_EINVAL, "ld_dx", n_out, n_in, m);
                    least = dq4_int8_linear_backward_workspace_bytes(n_out, n_in, m, pv, n_out);
                    for (int64_t bytes : {INT64_MIN, int64_t{-1}, least - 1})
                        expect(dq4_int8_linear_backward(codes, pf, n_out, n_in, DQ4_F16, pv, m, n_out, pv, n_in, pf, pv, bytes,
                                                        nullptr), DQ4_EINVAL, "workspace too small", n_out, n_in, m);
                    expect(dq4_int8_linear_backward(codes, pf, n_out, n_in, DQ4_F16, pv, m, n_out, pv, n_in, pf,
                                                    reinterpret_cast<void *>(0x1010), big, nullptr), DQ4_EINVAL,
                           "workspace not aligned", n_out, n_in, m);
                }
                expect(dq4_int8_linear_backward(codes, pf, n_out, n_in, INT32_MAX, pv, m, n_out, pv, n_in, pf, pv, big, nullptr),
                       DQ4_EINVAL, "type", n_out, n_in, m);
            }
    printf("int8 gradient abi sanitizer driver: %d failures\n", failures);
    return failures != 0;
}

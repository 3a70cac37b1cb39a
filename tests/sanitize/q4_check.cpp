// Host-sanitizer driver for the 4-bit layer calls (include/bakron_q4.h), built
// with AddressSanitizer and UndefinedBehaviorSanitizer on the host code only by
// tests/test_q4_sanitize.py and run on the CPU: sizes over many shapes and every
// host-side refusal.  Pointers are fake and never dereferenced.
#include <stdint.h>
#include <stdio.h>

#include "../../include/bakron_q4.h"

static int fails = 0;
#define EXPECT(cond)                                          \
    do {                                                      \
        if (!(cond)) {                                        \
            printf("FAIL line %d: %s\n", __LINE__, #cond);    \
            ++fails;                                          \
        }                                                     \
    } while (0)

int main()
{
    void* f = reinterpret_cast<void*>(4096);
    const float* ff = static_cast<const float*>(f);
    const uint8_t* fc = static_cast<const uint8_t*>(f);
    int32_t* fi = static_cast<int32_t*>(f);
    float* fo = static_cast<float*>(f);
    const size_t big = (size_t)1 << 60;
    const int64_t dims[] = {0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000, 4096, 14336, 65536, 65537, -1};
    const int64_t groups[] = {0, 64, 128, 192, 65536, 1 << 20, (int64_t)1 << 40};
    const int64_t tokens[] = {0, 1, 64, 65, 200, 1000, 8192, 100000, BAKRON_Q4_MAX_TOKENS, BAKRON_Q4_MAX_TOKENS + 1, -5};
    for (int64_t m : dims)
        for (int64_t n : dims) {
            const bool ok = m > 0 && n > 0 && m <= BAKRON_MAX_DIM && n <= BAKRON_MAX_DIM;
            for (int64_t g : groups) {
                const size_t one = bakron_q4_packed_bytes(1, m, n, g);
                EXPECT((one > 0) == ok);
                EXPECT(one % 256 == 0 && bakron_q4_packed_bytes(256, m, n, g) == 256 * one);
                if (ok) EXPECT(one >= (size_t)m * n / 2);
                for (int64_t t : tokens) {
                    const size_t a = bakron_q4_linear_workspace_bytes(t, m, n, g);
                    const size_t b = bakron_q4_linear_grad_workspace_bytes(t, m, n, g);
                    if (!ok || t <= 0 || t > BAKRON_Q4_MAX_TOKENS) EXPECT(a == 0 && b == 0);
                    EXPECT(a % 256 == 0 && b % 256 == 0);
                    if (ok && t > 0 && t <= BAKRON_Q4_MAX_TOKENS && b)
                        EXPECT(bakron_q4_linear_grad(f, m, t, BAKRON_Q4_BF16, f, m, n, g, f, n, f, b - 1, nullptr) ==
                               BAKRON_ERR_WORKSPACE);
                }
            }
            for (int64_t t : {1, 16, 64, 65})
                for (int64_t e : {1, 8, 256, 257}) {
                    const size_t w = bakron_q4_moe_workspace_bytes(t, m, n, e, 1, 0);
                    EXPECT((w > 0) == (t <= 64 && e <= 256 && m > 0 && n >= 0 && m <= BAKRON_MAX_DIM && n <= BAKRON_MAX_DIM));
                }
        }
    EXPECT(bakron_q4_packed_bytes(1, 64, 64, 63) == 0 && bakron_q4_packed_bytes(-1, 64, 64, 0) == 0);
    EXPECT(bakron_q4_pack(nullptr, ff, ff, 1, 64, 64, 0, f, nullptr) == BAKRON_ERR_NULL_POINTER);
    EXPECT(bakron_q4_pack(fc, ff, ff, 257, 64, 64, 0, f, nullptr) == BAKRON_ERR_BAD_SIZE);
    EXPECT(bakron_q4_pack(fc, ff, ff, 1, 64, 64, 1, f, nullptr) == BAKRON_ERR_BAD_ARG);
    EXPECT(bakron_q4_pack(fc, ff, ff, 0, 64, 64, 0, nullptr, nullptr) == BAKRON_SUCCESS);
    EXPECT(bakron_q4_linear(f, 63, 4, 0, f, 64, 64, 0, f, 64, f, big, nullptr) == BAKRON_ERR_BAD_ARG);
    EXPECT(bakron_q4_linear(f, 64, 4, 7, f, 64, 64, 0, f, 64, f, big, nullptr) == BAKRON_ERR_BAD_ARG);
    EXPECT(bakron_q4_linear(f, INT64_MAX, 4, 0, f, 64, 64, 0, f, 64, f, big, nullptr) == BAKRON_ERR_BAD_ARG);
    EXPECT(bakron_q4_linear(f, 64, INT64_MAX, 0, f, 64, 64, 0, f, 64, f, big, nullptr) == BAKRON_ERR_BAD_SIZE);
    EXPECT(bakron_q4_linear(f, 64, 4, 0, f, INT64_MIN, 64, 0, f, 64, f, big, nullptr) == BAKRON_ERR_BAD_SIZE);
    EXPECT(bakron_q4_linear(f, 64, 4, 0, nullptr, 64, 64, 0, f, 64, f, big, nullptr) == BAKRON_ERR_NULL_POINTER);
    EXPECT(bakron_q4_linear_grad(f, 64, 0, 0, nullptr, 64, 64, 0, nullptr, 64, nullptr, 0, nullptr) == BAKRON_SUCCESS);
    EXPECT(bakron_q4_moe(f, 64, 65, 0, f, f, f, f, 64, 64, 8, 2, 0, f, 64, fi, fo, f, big, nullptr) == BAKRON_ERR_BAD_SIZE);
    EXPECT(bakron_q4_moe(f, 64, 4, 0, f, f, f, f, 64, 64, 8, 9, 0, f, 64, fi, fo, f, big, nullptr) == BAKRON_ERR_BAD_ARG);
    EXPECT(bakron_q4_moe(f, 64, 4, 0, f, f, f, nullptr, 64, 64, 8, 2, 0, f, 64, fi, fo, f, big, nullptr) ==
           BAKRON_ERR_NULL_POINTER);
    EXPECT(bakron_q4_moe(f, 64, 4, 0, f, f, f, f, 64, 64, 8, 2, 0, f, 64, fi, fo, f, 1, nullptr) == BAKRON_ERR_WORKSPACE);
    EXPECT(bakron_q4_moe(f, 64, 0, 0, f, f, f, f, 64, 64, 8, 2, 0, f, 64, fi, fo, f, 1, nullptr) == BAKRON_SUCCESS);
    if (fails) return 1;
    printf("Q4 SANITIZE OK\n");
    return 0;
}

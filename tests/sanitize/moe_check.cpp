// Host-sanitizer driver for the calls of the expert layer for many tokens
// (include/bakron_moe.h), built with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code only by tests/test_moe_sanitize.py
// and run on the CPU: sizes over many shapes and host-side refusals.  Pointers are
// fake and never dereferenced.
#include <stdint.h>
#include <stdio.h>

#include "../../include/bakron_moe.h"

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
    float* fo = static_cast<float*>(f);
    int32_t* fi = static_cast<int32_t*>(f);
    const size_t big = (size_t)1 << 60;
    const int64_t most = BAKRON_MOE_MAX_ROWS;
    const int64_t dims[] = {0, 1, 15, 17, 64, 127, 129, 1000, 14336, 65536, 65537, -1, INT64_MAX, INT64_MIN};
    const int64_t groups[] = {0, 64, 128, 192, (int64_t)1 << 40, 65, -64};
    const int64_t rows[] = {0, 1, 33, 500, 4096, 49152, most, most + 1, -5, INT64_MAX, INT64_MIN};
    const int64_t experts[] = {1, 5, 64, 256, 0, 257, -1, INT64_MAX};
    for (int64_t m : dims)
        for (int64_t n : dims)
            for (int64_t g : groups)
                for (int64_t r : rows)
                    for (int64_t e : experts) {
                        const bool ok = m > 0 && n > 0 && m <= BAKRON_MAX_DIM && n <= BAKRON_MAX_DIM && g >= 0 && g % 64 == 0 && r > 0 &&
                                        r <= most && e >= 1 && e <= BAKRON_MOE_MAX_EXPERTS;
                        const size_t a = bakron_q4_experts_workspace_bytes(r, e, m, n, g);
                        const size_t b = bakron_q4_experts_grad_workspace_bytes(r, e, m, n, g);
                        EXPECT(a % 256 == 0 && b % 256 == 0);
                        if (!ok) EXPECT(a == 0 && b == 0);
                        if (ok && a) {
                            EXPECT(a >= (size_t)r * n * 2);   // the copy of x
                            EXPECT(bakron_q4_experts(f, n, r, 0, f, e, m, n, g, fi, f, m, f, a - 1, nullptr) == BAKRON_ERR_WORKSPACE);
                        }
                        if (ok && b)
                            EXPECT(bakron_q4_experts_grad(f, m, r, 1, f, e, m, n, g, fi, f, n, f, b - 1, nullptr) == BAKRON_ERR_WORKSPACE);
                    }
    for (int64_t t : rows)
        for (int64_t e : experts)
            for (int32_t k : {1, 6, 16, 17, 0, -1, INT32_MAX, INT32_MIN}) {
                const bool ok = t > 0 && t <= most && e >= 1 && e <= BAKRON_MOE_MAX_EXPERTS && k >= 1 && k <= 16 && k <= e && t * k <= most;
                const size_t a = bakron_moe_route_workspace_bytes(t, e, k);
                EXPECT(ok ? (a > 0) == (t > 64) : a == 0);
                if (ok && a) EXPECT(bakron_moe_route(f, e, t, 2, e, k, fi, fo, fi, fi, fi, f, a - 1, nullptr) == BAKRON_ERR_WORKSPACE);
                if (!ok && t != 0) EXPECT(bakron_moe_route(f, e > 0 ? e : 1, t, 2, e, k, fi, fo, fi, fi, fi, f, big, nullptr) < 0);
                if (!ok && t != 0) EXPECT(bakron_moe_route_grad(ff, ff, fi, t, e, k, f, e > 0 ? e : 1, 2, nullptr) < 0);
            }
    for (int64_t r : rows)
        for (int64_t c : dims) {
            const bool ok = r > 0 && r <= most && c > 0 && c <= BAKRON_MAX_DIM;
            const size_t a = bakron_ck8_bytes(r, c);
            EXPECT(ok ? a >= (size_t)r * c && a % 256 == 0 : a == 0);
            const bool none = (r == 0 && c >= 0 && c <= BAKRON_MAX_DIM) || (c == 0 && r >= 0 && r <= most);
            if (none) EXPECT(bakron_gated_act(f, c, f, c, r, 0, c, 0, nullptr, f, c, f, f, nullptr) == BAKRON_SUCCESS);
            else if (!ok) EXPECT(bakron_gated_act(f, c, f, c, r, 0, c, 0, nullptr, f, c, f, f, nullptr) == BAKRON_ERR_BAD_SIZE);
            if (!ok && !none) EXPECT(bakron_ck8_pack(f, c, r, 0, c, f, nullptr) == BAKRON_ERR_BAD_SIZE);
            if (!ok && !none) EXPECT(bakron_ck8_unpack(f, r, c, 2, f, c, nullptr) == BAKRON_ERR_BAD_SIZE);
            if (!ok && !none) EXPECT(bakron_gated_act_grad(f, c, f, f, r, 0, c, 0, nullptr, f, c, f, c, nullptr) == BAKRON_ERR_BAD_SIZE);
        }
    EXPECT(bakron_moe_gather(f, INT64_MAX, 4, 0, 64, 2, fi, f, 64, 8, nullptr) == BAKRON_ERR_BAD_ARG);
    EXPECT(bakron_moe_gather(f, 64, INT64_MAX, 0, 64, 2, fi, f, 64, 8, nullptr) == BAKRON_ERR_BAD_SIZE);
    EXPECT(bakron_moe_combine(f, 64, INT64_MIN, 0, 64, 2, fi, ff, 4, f, 64, nullptr) == BAKRON_ERR_BAD_SIZE);
    EXPECT(bakron_moe_combine(f, 64, 8, 0, 64, INT32_MAX, fi, ff, 4, f, 64, nullptr) == BAKRON_ERR_BAD_ARG);
    EXPECT(bakron_moe_combine_grad(f, 64, f, 64, 8, 0, 64, 2, fi, ff, 4, f, INT64_MIN, fo, nullptr) == BAKRON_ERR_BAD_ARG);
    EXPECT(bakron_moe_combine_grad(f, 64, f, 64, 8, 0, 64, 2, nullptr, ff, 4, f, 64, fo, nullptr) == BAKRON_ERR_NULL_POINTER);
    if (fails) return 1;
    printf("MOE SANITIZE OK\n");
    return 0;
}

// Host-only driver of the feed-forward operators' C entry points for the address
// and undefined-behaviour sanitizers: the choice of tiles and splits over a grid
// of sizes, types and layouts (through the workspace functions), and the
// argument checks of the four calls.  No GPU is touched: every call here is
// refused or has nothing to compute.  Prints "OK <calls>".
#include <cstdint>
#include <cstdio>

#include "../include/pgemm.h"

static int calls = 0;
#define EXPECT(cond)                                            \
    do {                                                        \
        ++calls;                                                \
        if (!(cond)) {                                          \
            std::printf("FAIL line %d: %s\n", __LINE__, #cond); \
            return 1;                                           \
        }                                                       \
    } while (0)

int main() {
    const int64_t dims[] = {0, 1, 15, 16, 17, 255, 256, 257, 1000, 4096, 100001, 0x7fffff00, 0x7fffff01, -1};
    for (int dtype = -1; dtype <= 4; ++dtype)
        for (int64_t M : dims)
            for (int64_t N : dims)
                for (int64_t K : dims) {
                    const int64_t a = pgemm_linear_workspace(M, N, K, dtype), b = pgemm_gated_workspace(M, N, K, dtype);
                    const int64_t c = pgemm_linear_backward_workspace(M, N, K, PGEMM_ACT_GELU, dtype);
                    const int64_t d = pgemm_gated_backward_workspace(M, N, K, dtype);
                    const bool bad = dtype < 0 || dtype > PGEMM_BF16 || M < 0 || N < 0 || K < 0;
                    EXPECT(bad ? a < 0 && b < 0 && c < 0 && d < 0 : (a >= 0) == (b >= 0) && (c >= 0) == (d >= 0));
                    EXPECT(a < 0 || (a % 256 == 0 && b % 256 == 0));
                    EXPECT(a == pgemm_linear_workspace(M, N, K, dtype));
                }
    void* p = (void*)(uintptr_t)(1 << 20);  // never dereferenced
    for (int order = -1; order <= 2; ++order)
        for (int act = -1; act <= 5; ++act)
            for (int out = -1; out <= 3; ++out)
                for (int64_t ld : {(int64_t)0, (int64_t)7, (int64_t)1 << 40}) {
                    EXPECT(pgemm_linear(8, 8, 8, p, ld, p, ld, order, p, p, ld, act, p, ld, p, ld, out, 2, nullptr, 0,
                                        nullptr) < 0);
                    EXPECT(pgemm_gated(8, 8, 8, p, ld, p, p, ld, order, p, p, act, p, ld, p, ld, p, ld, out, 2, nullptr,
                                       0, nullptr) < 0);
                    EXPECT(pgemm_linear_backward(8, 8, 8, p, ld, p, ld, p, ld, order, p, ld, act, p, ld, p, ld, order, p,
                                                 out, 2, nullptr, 0, nullptr) < 0);
                    EXPECT(pgemm_gated_backward(8, 8, 8, p, ld, p, ld, p, p, ld, order, p, ld, p, ld, act, p, ld, p, p,
                                                ld, order, p, p, out, 2, nullptr, 0, nullptr) < 0);
                }
    EXPECT(pgemm_linear(0, 8, 8, nullptr, 8, nullptr, 8, 0, nullptr, nullptr, 8, 0, nullptr, 8, nullptr, 8, 2, 2, nullptr,
                        0, nullptr) == PGEMM_OK);
    std::printf("OK %d\n", calls);
    return 0;
}

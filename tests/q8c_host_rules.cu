// q8c_host_rules.cu -- what the host decides about the 8-bit products, without a GPU.
//
// Built and run by tests/test_q8c_host_rules.py, linked against libqmm.so.  Prints one line per violation
// and "ok <checks>" at the end; exits 1 on any violation.
#include <cstdio>

#include "qmm_q8c.cuh"

using namespace qmm;

namespace {
int g_bad = 0, g_checks = 0;

#define CHECK(cond, ...)                                  \
    do {                                                  \
        ++g_checks;                                       \
        if (!(cond)) {                                    \
            ++g_bad;                                      \
            std::printf("FAIL %s: ", #cond);              \
            std::printf(__VA_ARGS__);                     \
            std::printf("\n");                            \
        }                                                 \
    } while (0)

// Results are stored 8 bytes at a time only where each of these stores is on an 8-byte boundary: column n of row
// m, n a multiple of 4, is element m N + n from y.
void wide_results() {
    for (int N = 1; N <= 4100; N = N < 12 ? N + 1 : N * 3 / 2)
        for (int yt : {(int)X_F32, (int)X_F16, (int)X_BF16})
            for (int ks = 1; ks <= 2; ++ks)
                for (long long at = 0; at < 16; at += x_size(yt)) {
                    QcCall c = {};
                    c.w.N = N;
                    c.yt = yt;
                    c.y = reinterpret_cast<void*>(0x10000 + at);
                    if (!qc_wide_results(c, ks)) continue;
                    CHECK(yt != X_F32 && ks == 1, "N %d type %d ks %d", N, yt, ks);
                    for (int m = 0; m < 4; ++m)
                        for (int n = 0; n < N; n += 4) {
                            CHECK((at + ((long long)m * N + n) * 2) % 8 == 0, "N %d, y %lld bytes from a boundary, row %d, column %d", N, at, m, n);
                            CHECK(n + 4 <= N, "N %d: four results from column %d", N, n);
                        }
                }
    QcCall c = {};  // and they are where they can be
    c.w.N = 64;
    c.yt = X_BF16;
    c.y = reinterpret_cast<void*>(0x10000);
    CHECK(qc_wide_results(c, 1), "aligned results of 64 columns");
}
}  // namespace

int main() {
    wide_results();
    if (g_bad) return 1;
    std::printf("ok %d\n", g_checks);
}

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

// Every plan of the GEMM is one that a kernel is compiled for, fits the block's shared memory, and a plan that none is
// compiled for is refused, before any CUDA call.
constexpr int kSms = 152, kSmem = 232448;  // GB300
bool compiled(const QcGemmPlan& p) { return (p.cg == 1 && p.kt == 2) || (p.cg == 2 && (p.kt == 1 || p.kt == 2)); }
void gemm_plans() {
    const int Ms[] = {1, 5, 16, 17, 33, 64, 65, 128, 129, 192, 200, 256, 257, 300, 512, 1000, 1024, 4000, 70000}, Ns[] = {1, 16, 100, 129, 576, 1536, 4096, 9000, 14336, 28672, 131072, 1 << 23},
              Ks[] = {1, 64, 128, 129, 576, 1000, 4096, 8192, 14336, 28672, 131071};
    for (int M : Ms)
        for (int N : Ns)
            for (int K : Ks)
                for (int sms : {kSms, 2, 77}) {
                    QcCall c = {};
                    if (!qc_describe(N, K, nullptr, c.w)) continue;
                    c.a.M = M;
                    const QcGemmPlan p = plan_q8c_gemm(c, sms, kSmem);
                    if (!p.ok) continue;
                    CHECK(compiled(p), "%d x %d x %d: cg %d kt %d", M, N, K, p.cg, p.kt);
                    CHECK(p.smem <= (size_t)kSmem && p.bx <= 256 && p.bx % (16 * p.cg) == 0, "%d x %d x %d: bx %d, %zu bytes", M, N, K, p.bx, p.smem);
                    CHECK((long long)p.mtiles * p.bx >= M && (long long)(p.mtiles - 1) * p.bx < M, "%d x %d x %d: %d tiles of %d", M, N, K, p.mtiles, p.bx);
                    CHECK(p.ks == 1 || M <= 65535, "%d x %d x %d: the slices' sums are a grid of M", M, N, K);
                }
    QcCall c = {};
    qc_describe(4096, 4096, nullptr, c.w);
    c.a.M = 256;
    QcGemmPlan p = plan_q8c_gemm(c, kSms, kSmem);
    const int forms[][2] = {{1, 1}, {0, 2}, {2, 0}, {2, 3}, {3, 2}};
    for (const auto& f : forms) {
        p.cg = f[0];
        p.kt = f[1];
        unsigned err = 0;
        CHECK(launch_q8c_gemm(p, c, nullptr, &err, 0, kSmem, nullptr) == cudaErrorInvalidConfiguration, "cg %d kt %d", p.cg, p.kt);
    }
}
}  // namespace

int main() {
    wide_results();
    gemm_plans();
    if (g_bad) return 1;
    std::printf("ok %d\n", g_checks);
}

// qmm_q4g_internal.h -- launchers of the 4-bit group-scale products and the
// mixture-of-experts operators, shared between their translation units.
#pragma once

#include "qmm_internal.h"
#include "qmm_q4g.cuh"

namespace qmm {

// What a product computes.
enum : int {
    P_DENSE = 0,    // y [M, N] = x W^T
    P_GATE_UP = 1,  // h [T k, F] = silu(x Wg_e^T) (x Wu_e^T), paired weights
    P_DOWN = 2      // y [T, N] = sum_j weight[t][j] h[t][j] Wd_e^T
};

// A routing: T tokens, top_k slots each (slot = t top_k + j).
struct QgRoute {
    const int* ids;       // [T][top_k]; a slot whose id is outside [0, E) is skipped
    const float* weights; // [T][top_k] (P_DOWN)
    const int* offsets;   // [E + 1]
    const int* order;     // slots sorted by expert
    int T, top_k;
};

struct QgCall {
    int op;
    QgWeights w;
    const void* x;
    void* y;
    int xt;           // type of x and y
    long long ldx;    // elements from a row of x to the next
    int M;            // rows of x (P_DENSE), slots T top_k otherwise
    QgRoute r;
};

cudaError_t launch_q4g_pack(const uint8_t* codes, const void* scales, int bf16, const uint8_t* zeros, int gsrc, const QgWeights& w,
                            void* out, cudaStream_t s);
cudaError_t launch_q4g_pack_q4_0(const uint8_t* wq, const QgWeights& w, void* out, cudaStream_t s);
cudaError_t launch_q4g_dequantize(const QgWeights& w, float* out, cudaStream_t s);

// The row kernel: warp MMAs, few activation rows per weight matrix.
struct QgRowsPlan {
    bool ok = false;
    int by_slot = 0;       // a block's rows are one slot's (P_GATE_UP) or one token's (P_DOWN): no sorted order needed
    int cols = 0;          // activation rows per item, at most
    int nb = 0;            // 8-column MMA blocks
    int np = 0;            // 16-bit pieces per activation value
    int warps = 0, wk = 0; // warps per block, warps that split K
    int blocks = 0;
    long long items = 0;
    int off_zero = 0, off_red = 0, off_ring = 0;
    size_t smem = 0;
    size_t workspace = 0;  // P_DOWN by expert: f32 partial rows [T top_k][N]
};
QgRowsPlan plan_q4g_rows(const QgCall& c, int sms, int smem_max);
cudaError_t launch_q4g_rows(const QgRowsPlan& pl, const QgCall& c, void* ws, int smem_max, cudaStream_t s);

// The tcgen05 GEMM.
struct QgGemmPlan {
    bool ok = false;
    int np = 0, pa = 0;    // pieces (hi, or hi and lo) of the activations: 2 for f32; of the weights
    int cg = 0, bx = 0, nacc = 0, accw = 0, mtiles = 0, ntiles = 0, nraw = 0, nx = 0, nstage = 0, grid = 0, ks = 0;
    int prep = 0;          // activations go through the preparation launch (f32, bf16)
    size_t smem = 0, ws_x = 0, ws_xs = 0, ws_part = 0, workspace = 0;
};
QgGemmPlan plan_q4g_gemm(const QgCall& c, int sms, int smem_max);
// stall: 0, or (test hook) one more than the tiles of raw weights that one block copies
cudaError_t launch_q4g_gemm(const QgGemmPlan& pl, const QgCall& c, void* ws, unsigned* err, int stall, int smem_max, cudaStream_t s);

// y [T, N] = sum_j weight[t][j] part[t top_k + j], in the order of j
cudaError_t launch_q4g_combine(const float* part, const QgRoute& r, int E, int N, void* y, int xt, cudaStream_t s);

// y [n] = the sum of ks slices of part [ks][n], in order
cudaError_t launch_q4g_sum(const float* part, int ks, long long n, void* y, int xt, cudaStream_t s);

struct RouteCall {
    const void* logits;
    int xt;
    long long ldl;
    int T, E, top_k;
    int sigmoid, renorm, groups, top_groups, top2;
    const float* bias;
    float scale;
    int* ids;
    float* weights;
    int* offsets;  // NULL: no sorted order wanted
    int* order;
};
size_t route_workspace(int T, int E, int top_k);
cudaError_t launch_route(const RouteCall& c, void* ws, cudaStream_t s);

}  // namespace qmm

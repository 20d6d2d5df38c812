// qmm_q4g_api.cu -- the C ABI (include/qmm.h) of the 4-bit group-scale
// products and the mixture-of-experts operators: argument checks, the choice
// between the row kernel and the GEMM, launches.
#include "qmm_q4g_internal.h"

#include "../../include/qmm.h"

using namespace qmm;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool float_type(qmm_float t) { return t == QMM_FLOAT_F32 || t == QMM_FLOAT_F16 || t == QMM_FLOAT_BF16; }

// a weight descriptor's checks; QMM_OK also for N = 0 (w.N == 0 then)
qmm_status describe(const qmm_q4g* d, QgWeights& w) {
    if (!d) return QMM_ERR_NULL;
    w = QgWeights();
    if (d->N == 0 && d->K > 0 && d->experts > 0) return QMM_OK;
    if (!qg_describe(d->experts, d->N, d->K, d->group, d->paired, d->data, w)) return QMM_ERR_SHAPE;
    return QMM_OK;
}
qmm_status check_data(const qmm_q4g* d) {
    if (!d->data) return QMM_ERR_NULL;
    return aligned(d->data, 16) ? QMM_OK : QMM_ERR_ALIGN;
}
qmm_status check_rows(const void* x, int xt, int64_t ldx, int64_t K) {
    if (ldx < K) return QMM_ERR_SHAPE;
    if (!aligned(x, 16) || (ldx * x_size(xt)) % 16 != 0) return QMM_ERR_ALIGN;
    return QMM_OK;
}

// The kernel a product goes to.  The row kernel streams the weights once per
// item of a few activation rows and turns every code into an MMA operand once
// per 8 columns (an f32 row is three).  The GEMM's conversion serves up to 256
// rows (f32: 64), but a call has some 8 us of fixed cost.  Measured (row kernel
// / GEMM, us): 4096 x 4096 bf16, 8 rows 7.2 / 10.4, 12 rows 8.5 / 10.2; 14336 x
// 4096 bf16, 12 rows 15.3 / 18.2, 16 rows 19.3 / 18.3; 4096 x 14336 bf16, 8 rows
// (two items) 22.3 / 19.5; 14336 x 4096 f32, 8 rows (two items) 23.1 / 28.1, 10
// rows 46 / 28; 1000 x 2048 bf16, 64 rows 6.2 / 8.7.  gate_up and down of 64
// experts, 2048 -> 2 x 1024 -> 2048, bf16: 8 slots an expert 59 + 41 / 59 + 37,
// 16 slots 117 + 60 / 59 + 38; f32: 4 slots 103 + 49 / 100 + 58, 8 slots 124 + 60
// / 101 + 59; of 128 experts with 768, f32: 4 slots 142 + 69 / 152 + 86.
struct Choice {
    bool gemm = false;
    QgRowsPlan rows;
    QgGemmPlan mm;
    size_t workspace = 0;
    bool ok = false;
};
Choice choose(const QgCall& c, int sms, int smem) {
    Choice ch;
    const int np = c.xt == X_F32 ? 3 : 1;
    const long long columns = (long long)c.M * np, size = (long long)c.w.N * c.w.K;
    const bool small = columns * size <= 160000000;
    const bool few = c.op == P_DENSE ? columns <= (np == 3 ? 24 : 12) || small : columns <= (np == 3 ? 12ll : 8ll) * c.w.E;
    if (few) ch.rows = plan_q4g_rows(c, sms, smem);
    // activations that do not fit one pass (f32: two) over a large matrix
    if (ch.rows.ok && c.op == P_DENSE && ch.rows.items > (np == 3 ? 2 : 1) && !small && (ch.mm = plan_q4g_gemm(c, sms, smem)).ok)
        ch.rows.ok = false;
    if (!ch.rows.ok) ch.mm = plan_q4g_gemm(c, sms, smem);
    if (!ch.rows.ok && !ch.mm.ok) ch.rows = plan_q4g_rows(c, sms, smem);
    ch.gemm = !ch.rows.ok && ch.mm.ok;
    ch.ok = ch.rows.ok || ch.mm.ok;
    ch.workspace = ch.gemm ? ch.mm.workspace : ch.rows.workspace;
    return ch;
}

size_t workspace_of(QgCall c) {
    int sms = 0, smem = 0;
    if (device_constants(nullptr, &sms, &smem) != cudaSuccess) return 0;
    const Choice ch = choose(c, sms, smem);
    return ch.ok ? ch.workspace : 0;
}

qmm_status product(const QgCall& c, void* ws, size_t ws_bytes, qmm_stream_t stream) {
    if (injected_launch_failure()) return QMM_ERR_CUDA;  // test hook: no CUDA call made
    unsigned* err = nullptr;
    int sms = 0, smem = 0;
    if (device_constants(&err, &sms, &smem) != cudaSuccess) return QMM_ERR_CUDA;
    const Choice ch = choose(c, sms, smem);
    if (!ch.ok) return QMM_ERR_SHAPE;
    if (ch.workspace) {
        if (!ws || ws_bytes < ch.workspace) return QMM_ERR_WORKSPACE;
        if (!aligned(ws, 16)) return QMM_ERR_ALIGN;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = ch.gemm ? launch_q4g_gemm(ch.mm, c, ws, err, injected_stall(), smem, s) : launch_q4g_rows(ch.rows, c, ws, smem, s);
    return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}

// the shape of an experts' product; slots = T top_k
qmm_status moe_shape(const QgWeights& w, int64_t T, int64_t top_k) {
    if (T < 0 || top_k < 1 || top_k > QMM_MOE_MAX_TOP_K || w.E > QMM_MOE_MAX_EXPERTS || T * top_k > INT32_MAX) return QMM_ERR_SHAPE;
    return QMM_OK;
}

qmm_status moe_product(int op, const qmm_q4g* wd, qmm_float xt, const void* x, int64_t ldx, const qmm_routing* r, void* y, void* ws,
                       size_t ws_bytes, qmm_stream_t stream) {
    if (!float_type(xt)) return QMM_ERR_TYPE;
    QgCall c = {};
    qmm_status st = describe(wd, c.w);
    if (st != QMM_OK) return st;
    if (!r) return QMM_ERR_NULL;
    st = moe_shape(c.w, r->T, r->top_k);
    if (st != QMM_OK) return st;
    if (c.w.N && (op == P_GATE_UP) != (c.w.paired != 0)) return QMM_ERR_SHAPE;
    if (r->T == 0 || c.w.N == 0) return QMM_OK;
    if (!x || !y || !r->ids || !r->offsets || !r->order || (op == P_DOWN && !r->weights)) return QMM_ERR_NULL;
    if ((st = check_data(wd)) != QMM_OK) return st;
    if ((st = check_rows(x, (int)xt, ldx, c.w.K)) != QMM_OK) return st;
    if (!aligned(y, x_size((int)xt)) || !aligned(r->ids, 4) || !aligned(r->weights, 4) || !aligned(r->offsets, 4) || !aligned(r->order, 4))
        return QMM_ERR_ALIGN;
    c.op = op;
    c.x = x;
    c.y = y;
    c.xt = (int)xt;
    c.ldx = ldx;
    c.M = (int)(r->T * r->top_k);
    c.r = QgRoute{r->ids, r->weights, r->offsets, r->order, (int)r->T, (int)r->top_k};
    return product(c, ws, ws_bytes, stream);
}

size_t moe_workspace(int op, const qmm_q4g* wd, qmm_float xt, int64_t T, int64_t top_k) {
    QgCall c = {};
    if (!float_type(xt) || describe(wd, c.w) != QMM_OK || c.w.N == 0 || moe_shape(c.w, T, top_k) != QMM_OK || T == 0) return 0;
    c.op = op;
    c.xt = (int)xt;
    c.ldx = c.w.K;
    c.M = (int)(T * top_k);
    c.r.T = (int)T;
    c.r.top_k = (int)top_k;
    return workspace_of(c);
}

}  // namespace

extern "C" {

size_t qmm_q4g_bytes(int64_t experts, int64_t N, int64_t K, int group, int paired) {
    QgWeights w;
    if (!qg_describe(experts, N, K, group, paired, nullptr, w)) return 0;
    return (size_t)(w.iscale_off + (long long)w.E * w.RB * 16 * 4);
}

qmm_status qmm_q4g_pack(const uint8_t* codes, const void* scales, qmm_float scale_type, const uint8_t* zeros, int64_t experts, int64_t N,
                        int64_t K, int group, int paired, void* out, qmm_stream_t stream) {
    if (scale_type != QMM_FLOAT_F16 && scale_type != QMM_FLOAT_BF16) return QMM_ERR_TYPE;
    const qmm_q4g d = {out, experts, N, K, group, paired};
    QgWeights w;
    qmm_status st = describe(&d, w);
    if (st != QMM_OK) return st;
    if (w.N == 0) return QMM_OK;
    if (!codes || !scales || !out) return QMM_ERR_NULL;
    if (!aligned(out, 16) || !aligned(scales, 2)) return QMM_ERR_ALIGN;
    return launch_q4g_pack(codes, scales, scale_type == QMM_FLOAT_BF16, zeros, group, w, out, reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? QMM_OK
               : QMM_ERR_CUDA;
}

qmm_status qmm_q4g_pack_q4_0(const void* wq, int64_t experts, int64_t N, int64_t K, int paired, void* out, qmm_stream_t stream) {
    const qmm_q4g d = {out, experts, N, K, 32, paired};
    QgWeights w;
    qmm_status st = describe(&d, w);
    if (st != QMM_OK) return st;
    if (w.N == 0) return QMM_OK;
    if (!wq || !out) return QMM_ERR_NULL;
    if (!aligned(wq, 16) || !aligned(out, 16)) return QMM_ERR_ALIGN;
    return launch_q4g_pack_q4_0(static_cast<const uint8_t*>(wq), w, out, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? QMM_OK
                                                                                                                               : QMM_ERR_CUDA;
}

qmm_status qmm_q4g_dequantize(const qmm_q4g* wd, float* out, qmm_stream_t stream) {
    QgWeights w;
    qmm_status st = describe(wd, w);
    if (st != QMM_OK) return st;
    if (w.N == 0) return QMM_OK;
    if (!out) return QMM_ERR_NULL;
    if ((st = check_data(wd)) != QMM_OK) return st;
    if (!aligned(out, 16)) return QMM_ERR_ALIGN;
    return launch_q4g_dequantize(w, out, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}

size_t qmm_q4g_matmul_workspace(const qmm_q4g* wd, qmm_float xtype, int64_t M) {
    QgCall c = {};
    if (!float_type(xtype) || describe(wd, c.w) != QMM_OK || c.w.N == 0 || c.w.paired || c.w.E != 1 || M <= 0 || M > INT32_MAX) return 0;
    c.op = P_DENSE;
    c.xt = (int)xtype;
    c.ldx = c.w.K;
    c.M = (int)M;
    return workspace_of(c);
}

qmm_status qmm_q4g_matmul(const qmm_q4g* wd, qmm_float xtype, const void* x, int64_t ldx, int64_t M, void* y, void* workspace,
                          size_t workspace_bytes, qmm_stream_t stream) {
    if (!float_type(xtype)) return QMM_ERR_TYPE;
    QgCall c = {};
    qmm_status st = describe(wd, c.w);
    if (st != QMM_OK) return st;
    if (M < 0 || M > INT32_MAX || (c.w.N && (c.w.paired || c.w.E != 1))) return QMM_ERR_SHAPE;
    if (M == 0 || c.w.N == 0) return QMM_OK;
    if (!x || !y) return QMM_ERR_NULL;
    if ((st = check_data(wd)) != QMM_OK) return st;
    if ((st = check_rows(x, (int)xtype, ldx, c.w.K)) != QMM_OK) return st;
    if (!aligned(y, x_size((int)xtype))) return QMM_ERR_ALIGN;
    c.op = P_DENSE;
    c.x = x;
    c.y = y;
    c.xt = (int)xtype;
    c.ldx = ldx;
    c.M = (int)M;
    return product(c, workspace, workspace_bytes, stream);
}

static bool route_shape(int64_t T, int64_t E, int64_t top_k) {
    return T >= 0 && E >= 1 && E <= QMM_MOE_MAX_EXPERTS && top_k >= 1 && top_k <= QMM_MOE_MAX_TOP_K && top_k <= E && T * top_k <= INT32_MAX;
}

size_t qmm_moe_route_workspace(int64_t T, int64_t E, int64_t top_k) {
    return route_shape(T, E, top_k) && T > 0 ? route_workspace((int)T, (int)E, (int)top_k) : 0;
}

qmm_status qmm_moe_route(const qmm_route_config* cfg, qmm_float type, const void* logits, int64_t ldl, int64_t T, int64_t E,
                         const float* bias, int32_t* ids, float* weights, int32_t* offsets, int32_t* order, void* workspace,
                         size_t workspace_bytes, qmm_stream_t stream) {
    if (!cfg) return QMM_ERR_NULL;
    if (!float_type(type)) return QMM_ERR_TYPE;
    if ((cfg->score != QMM_SCORE_SOFTMAX && cfg->score != QMM_SCORE_SIGMOID) ||
        (cfg->group_score != QMM_GROUP_MAX && cfg->group_score != QMM_GROUP_TOP2))
        return QMM_ERR_TYPE;
    if (!route_shape(T, E, cfg->top_k) || ldl < E) return QMM_ERR_SHAPE;
    if (cfg->groups < 1 || cfg->groups > 32 || E % cfg->groups != 0 || cfg->top_groups < 1 || cfg->top_groups > cfg->groups ||
        cfg->top_k > cfg->top_groups * (E / cfg->groups))
        return QMM_ERR_SHAPE;
    if (T > 0 && (offsets == nullptr) != (order == nullptr)) return QMM_ERR_NULL;
    if (T > 0 && (!logits || !ids || !weights)) return QMM_ERR_NULL;
    if (!aligned(logits, x_size((int)type)) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(offsets, 4) || !aligned(order, 4) ||
        !aligned(bias, 4))
        return QMM_ERR_ALIGN;
    if (order && T > 0) {
        const size_t need = route_workspace((int)T, (int)E, cfg->top_k);
        if (need && (!workspace || workspace_bytes < need)) return QMM_ERR_WORKSPACE;
        if (need && !aligned(workspace, 16)) return QMM_ERR_ALIGN;
    }
    if (injected_launch_failure()) return QMM_ERR_CUDA;
    RouteCall c;
    c.logits = logits;
    c.xt = (int)type;
    c.ldl = ldl;
    c.T = (int)T;
    c.E = (int)E;
    c.top_k = cfg->top_k;
    c.sigmoid = cfg->score == QMM_SCORE_SIGMOID;
    c.renorm = cfg->renorm != 0;
    c.groups = cfg->groups;
    c.top_groups = cfg->top_groups;
    c.top2 = cfg->group_score == QMM_GROUP_TOP2;
    c.bias = bias;
    c.scale = cfg->scale;
    c.ids = ids;
    c.weights = weights;
    c.offsets = offsets;
    c.order = order;
    return launch_route(c, workspace, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}

size_t qmm_moe_gate_up_workspace(const qmm_q4g* w, qmm_float xtype, int64_t T, int64_t top_k) {
    return moe_workspace(P_GATE_UP, w, xtype, T, top_k);
}
qmm_status qmm_moe_gate_up(const qmm_q4g* w, qmm_float xtype, const void* x, int64_t ldx, const qmm_routing* r, void* h, void* workspace,
                           size_t workspace_bytes, qmm_stream_t stream) {
    return moe_product(P_GATE_UP, w, xtype, x, ldx, r, h, workspace, workspace_bytes, stream);
}
size_t qmm_moe_down_workspace(const qmm_q4g* w, qmm_float xtype, int64_t T, int64_t top_k) {
    return moe_workspace(P_DOWN, w, xtype, T, top_k);
}
qmm_status qmm_moe_down(const qmm_q4g* w, qmm_float xtype, const void* h, int64_t ldh, const qmm_routing* r, void* y, void* workspace,
                        size_t workspace_bytes, qmm_stream_t stream) {
    return moe_product(P_DOWN, w, xtype, h, ldh, r, y, workspace, workspace_bytes, stream);
}

}  // extern "C"

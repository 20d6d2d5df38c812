// qmm_q8c_api.cu -- the C ABI (include/qmm.h) of the 8-bit channel-scaled
// products and of the norms around a block: argument checks, the choice
// between the row kernel and the GEMM, launches.
#include "qmm_q8c.cuh"

#include "../../include/qmm.h"

using namespace qmm;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool float_type(qmm_float t) { return t == QMM_FLOAT_F32 || t == QMM_FLOAT_F16 || t == QMM_FLOAT_BF16; }
cudaStream_t stream_of(qmm_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
qmm_status status(cudaError_t e) { return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA; }

// QMM_OK also for N = 0 (w.N == 0 then)
qmm_status describe(const qmm_q8c* d, QcWeights& w) {
    if (!d) return QMM_ERR_NULL;
    w = QcWeights();
    if (d->N == 0 && d->K > 0) return QMM_OK;
    return qc_describe(d->N, d->K, d->data, w) ? QMM_OK : QMM_ERR_SHAPE;
}

// The kernel that a product goes to: up to four rows to the row kernel, where they fit its shared memory.
// Measured (row kernel / GEMM, us, bf16): 576 x 576, 1, 4 and 8 rows 4.5 / 5.5, 5.1 / 5.5, 5.7 / 5.5; 4096 x 4096
// 7.6 / 10.1, 11.4 / 10.5, 11.9 / 11.0; 14336 x 4096 13.8 / 15.8, 15.8 / 15.9, 18.1 / 15.9; 28672 x 8192 41 / 48, 44 / 49,
// 48 / 50.  (The GEMM's time hardly depends on the rows until there are more than 64.)
struct Choice {
    bool gemm = false, ok = false;
    QcRowsPlan rows;
    QcGemmPlan mm;
    size_t workspace = 0;
};
Choice choose(const QcCall& c, int sms, int smem) {
    Choice ch;
    ch.rows = plan_q8c_rows(c, sms, smem);
    if (!ch.rows.ok) ch.mm = plan_q8c_gemm(c, sms, smem);
    ch.gemm = !ch.rows.ok;
    ch.ok = ch.rows.ok || ch.mm.ok;
    ch.workspace = ch.gemm ? ch.mm.workspace : ch.rows.workspace;
    return ch;
}

}  // namespace

extern "C" {

size_t qmm_q8c_bytes(int64_t N, int64_t K) {
    QcWeights w;
    return qc_describe(N, K, nullptr, w) ? qc_bytes(w) : 0;
}

qmm_status qmm_q8c_pack(const int8_t* codes, int64_t ldc, const float* scales, int64_t N, int64_t K, void* out, qmm_stream_t stream) {
    const qmm_q8c d = {out, N, K};
    QcWeights w;
    const qmm_status st = describe(&d, w);
    if (st != QMM_OK) return st;
    if (ldc < K) return QMM_ERR_SHAPE;
    if (w.N == 0) return QMM_OK;
    if (!codes || !scales || !out) return QMM_ERR_NULL;
    if (!aligned(out, 16) || !aligned(scales, 4)) return QMM_ERR_ALIGN;
    return status(launch_q8c_pack(codes, ldc, scales, w, out, stream_of(stream)));
}

qmm_status qmm_q8c_dequantize(const qmm_q8c* wd, float* out, qmm_stream_t stream) {
    QcWeights w;
    const qmm_status st = describe(wd, w);
    if (st != QMM_OK) return st;
    if (w.N == 0) return QMM_OK;
    if (!out || !wd->data) return QMM_ERR_NULL;
    if (!aligned(wd->data, 16) || !aligned(out, 4)) return QMM_ERR_ALIGN;
    return status(launch_q8c_dequantize(w, out, stream_of(stream)));
}

qmm_status qmm_q8c_quantize(qmm_float xtype, const void* x, int64_t ldx, int64_t M, int64_t K, int8_t* codes, int64_t ldc, float* scales,
                            qmm_stream_t stream) {
    if (!float_type(xtype)) return QMM_ERR_TYPE;
    if (M < 0 || M > INT32_MAX || K < 1 || K > kQcMaxK || ldx < K || ldc < K) return QMM_ERR_SHAPE;
    if (M == 0) return QMM_OK;
    if (!x || !codes || !scales) return QMM_ERR_NULL;
    if (!aligned(x, x_size((int)xtype)) || !aligned(scales, 4)) return QMM_ERR_ALIGN;
    if (injected_launch_failure()) return QMM_ERR_CUDA;
    return status(launch_q8c_quantize(QcRows{x, nullptr, ldx, (int)xtype, (int)M}, (int)K, codes, ldc, scales, stream_of(stream)));
}

size_t qmm_q8c_matmul_workspace(const qmm_q8c* wd, int quantized, int64_t M) {
    QcCall c = {};
    int sms = 0, smem = 0;
    if (describe(wd, c.w) != QMM_OK || c.w.N == 0 || M <= 0 || M > INT32_MAX || device_constants(nullptr, &sms, &smem) != cudaSuccess) return 0;
    static const float some = 0.0f;
    c.a = QcRows{reinterpret_cast<const void*>(4), quantized ? &some : nullptr, c.w.K, X_F32, (int)M};  // rows on no boundary: the most
    const Choice ch = choose(c, sms, smem);
    return ch.ok ? ch.workspace : 0;
}

qmm_status qmm_q8c_matmul(const qmm_q8c* wd, qmm_float xtype, const void* x, int64_t ldx, const float* x_scales, int64_t M, const float* bias,
                          qmm_float ytype, void* y, void* workspace, size_t workspace_bytes, qmm_stream_t stream) {
    if ((!x_scales && !float_type(xtype)) || !float_type(ytype)) return QMM_ERR_TYPE;
    QcCall c = {};
    const qmm_status st = describe(wd, c.w);
    if (st != QMM_OK) return st;
    if (M < 0 || M > INT32_MAX || ldx < wd->K) return QMM_ERR_SHAPE;
    if (M == 0 || c.w.N == 0) return QMM_OK;
    if (!x || !y || !wd->data) return QMM_ERR_NULL;
    if (!aligned(wd->data, 16) || (!x_scales && !aligned(x, x_size((int)xtype))) || !aligned(x_scales, 4) || !aligned(bias, 4) ||
        !aligned(y, x_size((int)ytype)))
        return QMM_ERR_ALIGN;
    c.a = QcRows{x, x_scales, ldx, (int)xtype, (int)M};
    c.bias = bias;
    c.y = y;
    c.yt = (int)ytype;
    if (injected_launch_failure()) return QMM_ERR_CUDA;  // test hook: no CUDA call made
    unsigned* err = nullptr;
    int sms = 0, smem = 0;
    if (device_constants(&err, &sms, &smem) != cudaSuccess) return QMM_ERR_CUDA;
    const Choice ch = choose(c, sms, smem);
    if (!ch.ok) return QMM_ERR_SHAPE;
    if (ch.workspace) {
        if (!workspace || workspace_bytes < ch.workspace) return QMM_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return QMM_ERR_ALIGN;
    }
    return status(ch.gemm ? launch_q8c_gemm(ch.mm, c, workspace, err, injected_stall(), smem, stream_of(stream))
                          : launch_q8c_rows(ch.rows, c, workspace, smem, stream_of(stream)));
}

qmm_status qmm_block_norm(const qmm_norm* n, int64_t T, int64_t K, qmm_stream_t stream) {
    if (!n) return QMM_ERR_NULL;
    if (!float_type(n->type) || !float_type(n->weight_type)) return QMM_ERR_TYPE;
    if (T < 0 || T > INT32_MAX || K < 1 || K > QMM_NORM_MAX_K) return QMM_ERR_SHAPE;
    if (n->ldy < K || (n->residual && n->ldr < K) || (n->gate && n->ldg != 0 && n->ldg < K) || (n->residual_out && n->ldro < K) || n->ldh < K)
        return QMM_ERR_SHAPE;
    if (T == 0) return QMM_OK;
    if (!n->y || !n->weight || (n->h == nullptr) == (n->codes == nullptr) || (n->codes && !n->scales)) return QMM_ERR_NULL;
    if (n->h && n->h == n->residual_out) return QMM_ERR_SHAPE;  // two results, one place
    // in place, row t's result lies on row t's input and on no other one's
    auto astray = [&](const void* out, int64_t ld) {
        return T > 1 && out && ((out == n->y && ld != n->ldy) || (out == n->residual && ld != n->ldr));
    };
    if (astray(n->residual_out, n->ldro) || astray(n->h, n->ldh)) return QMM_ERR_SHAPE;
    const uintptr_t a = (uintptr_t)x_size((int)n->type), wa = (uintptr_t)x_size((int)n->weight_type);
    if (!aligned(n->y, a) || !aligned(n->residual, a) || !aligned(n->gate, a) || !aligned(n->post_weight, wa) || !aligned(n->weight, wa) ||
        !aligned(n->residual_out, a) || !aligned(n->h, a) || !aligned(n->scales, 4))
        return QMM_ERR_ALIGN;
    // codes are a byte each: a row's do not lie where its values do
    if (n->codes && (n->codes == n->residual_out || n->codes == n->y || n->codes == n->residual)) return QMM_ERR_SHAPE;
    if (injected_launch_failure()) return QMM_ERR_CUDA;
    NormCall c;
    c.y = n->y;
    c.r = n->residual;
    c.gate = n->gate;
    c.post = n->post_weight;
    c.pre = n->weight;
    c.r_out = n->residual_out;
    c.h = n->h;
    c.codes = n->codes;
    c.scales = n->scales;
    c.ldy = n->ldy;
    c.ldr = n->ldr;
    c.ldg = n->ldg;
    c.ldro = n->ldro;
    c.ldh = n->ldh;
    c.T = (int)T;
    c.K = (int)K;
    c.xt = (int)n->type;
    c.wt = (int)n->weight_type;
    c.scale = n->scale;
    c.eps = n->eps;
    c.offset = n->weight_offset;
    return status(launch_block_norm(c, stream_of(stream)));
}

}  // extern "C"

// qmm_q4g_rows_2.cu -- row-kernel launches with 2 block(s) of 8 activation columns
#include "qmm_q4g_rows_go.cuh"

namespace qmm {
cudaError_t launch_q4g_rows_2(const QgRowsPlan& pl, const QgRowsParams& p, int smem_max, cudaStream_t s) {
    return q4g_rows_go<2>(pl, p, smem_max, s);
}
}  // namespace qmm

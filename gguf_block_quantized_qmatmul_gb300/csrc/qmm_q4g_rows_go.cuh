// qmm_q4g_rows_go.cuh -- instantiation and launch of the row kernel for one column-block count
#pragma once

#include "qmm_q4g_rows.cuh"

namespace qmm {

template <int NB, bool BF, int NG, bool TOK = false>
cudaError_t q4g_rows_one(const QgRowsPlan& pl, const QgRowsParams& p, int smem_max, cudaStream_t s) {
    static unsigned long long done = 0;
    auto* k = q4g_rows_kernel<NB, BF, NG, TOK>;
    const cudaError_t e = ensure_smem(k, smem_max - kQgRowStatic, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(k, (unsigned)pl.blocks, (unsigned)(pl.warps * 32), pl.smem, s, p);
}

template <int NB>
cudaError_t q4g_rows_go(const QgRowsPlan& pl, const QgRowsParams& p, int smem_max, cudaStream_t s) {
    const int ng = p.c.w.ng;
    if constexpr (NB == 1) {
        if (p.c.op == P_DOWN && pl.by_slot) {
            if (p.c.xt == X_F16)
                return ng == 1 ? q4g_rows_one<1, false, 1, true>(pl, p, smem_max, s)
                       : ng == 2 ? q4g_rows_one<1, false, 2, true>(pl, p, smem_max, s)
                                 : q4g_rows_one<1, false, 4, true>(pl, p, smem_max, s);
            return ng == 1 ? q4g_rows_one<1, true, 1, true>(pl, p, smem_max, s)
                   : ng == 2 ? q4g_rows_one<1, true, 2, true>(pl, p, smem_max, s)
                             : q4g_rows_one<1, true, 4, true>(pl, p, smem_max, s);
        }
    }
    if (p.c.xt == X_F16)
        return ng == 1 ? q4g_rows_one<NB, false, 1>(pl, p, smem_max, s)
               : ng == 2 ? q4g_rows_one<NB, false, 2>(pl, p, smem_max, s)
                         : q4g_rows_one<NB, false, 4>(pl, p, smem_max, s);
    return ng == 1 ? q4g_rows_one<NB, true, 1>(pl, p, smem_max, s)
           : ng == 2 ? q4g_rows_one<NB, true, 2>(pl, p, smem_max, s)
                     : q4g_rows_one<NB, true, 4>(pl, p, smem_max, s);
}

}  // namespace qmm

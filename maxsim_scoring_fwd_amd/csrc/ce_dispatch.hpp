// Launches of maxsim_linear_cross_entropy's kernels, for one storage type.
#pragma once

#include "ce_kernels.hpp"
#include "host_common.hpp"

namespace maxsim {

// Places of the rings: three of 24 KB, or four of 16, leave room for two workgroups a CU; twelve of 10 KB
// fill one's LDS.
constexpr int CE_STAGES = 3, CE_HALF_STAGES = 4, CE_FEW_STAGES = 12;

template <typename Kernel> int ce_launch(Kernel kernel, int64_t tiles, int lds, int cus, const CeArgs &a, hipStream_t st) {
  // the tiles are dealt out on the device, where their number is known: no more workgroups than
  // there can be tiles, nor than the chip holds at once
  const int64_t most = (int64_t)cus * blocks_per_cu((const void *)kernel, GEMM_THREADS, lds);
  const unsigned grid = (unsigned)(tiles < most ? tiles : most);
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(GEMM_THREADS), lds, st, a);
  return hipGetLastError() == hipSuccess ? MAXSIM_OK : MAXSIM_ERR_LAUNCH;
}

// Whether logits go in tiles of 128 rows: where there are no more rows, or fewer tiles of 256 than
// three quarters of the workgroups (forward, tiles of 256 and of 128: 2000 rows, 2000 x 768 in bf16, 128
// tiles, 30.1 and 24.7 us; 300 rows, 20000 x 768, 314 tiles, 31.6 and 26.5; 512 rows, 30522 x 768, 478
// tiles, 38.2 and 43.0; 346 rows, 1547 x 640 in fp32 93 and 61).
inline bool ce_half(const CeArgs &a) {
  return a.n <= CE_HALF_BN || 4 * blocks_of(a.vocab, CE_BM) * blocks_of(a.n, CE_BN) <= 3 * CE_LANES;
}

template <int DT> int ce_gathered(const CeArgs &a, bool count, hipStream_t st) {
  if (count)
    hipLaunchKernelGGL(ce_count_kernel<DT>, dim3((unsigned)blocks_of(a.n, CE_COUNT)), dim3(GEMM_THREADS), 0, st, a);
  if (count && hipGetLastError() != hipSuccess) return MAXSIM_ERR_LAUNCH;
  hipLaunchKernelGGL(ce_gather_kernel<DT>, dim3((unsigned)blocks_of(a.n, CE_GATHER)), dim3(GEMM_THREADS), 0, st, a);
  return hipGetLastError() == hipSuccess ? MAXSIM_OK : MAXSIM_ERR_LAUNCH;
}

template <int DT> int ce_forward(const CeArgs &a, int cus, hipStream_t st) {
  const int across = (int)blocks_of(a.vocab, CE_BM);
  if (ce_few(a)) {
    using G = TileGemm<DT, CE_BM, CE_FEW, 4, SIDE_ROWS, SIDE_ROWS, CE_FEW_STAGES>;
    constexpr int lds = G::lds + CE_FEW * sizeof(CeRow);
    hipLaunchKernelGGL((ce_few_kernel<DT, CE_FEW_STAGES>), dim3(across), dim3(GEMM_THREADS), lds, st, a);
    if (hipGetLastError() != hipSuccess) return MAXSIM_ERR_LAUNCH;
  } else {
    using Z = CeLogits<DT, CE_BM, CE_BN, 2, CE_STAGES>;
    using H = CeLogits<DT, CE_BM, CE_HALF_BN, 2, CE_HALF_STAGES>;
    int rc = ce_gathered<DT>(a, a.n > CE_DIRECT, st);
    if (rc == MAXSIM_OK)
      rc = ce_half(a)
               ? ce_launch(ce_forward_kernel<DT, CE_BM, CE_HALF_BN, 2, CE_HALF_STAGES>,
                           across * blocks_of(a.n, CE_HALF_BN), H::lds, cus, a, st)
               : ce_launch(ce_forward_kernel<DT, CE_BM, CE_BN, 2, CE_STAGES>, across * blocks_of(a.n, CE_BN), Z::lds,
                           cus, a, st);
    if (rc != MAXSIM_OK) return rc;
  }
  hipLaunchKernelGGL(ce_join_kernel<DT>, dim3((unsigned)blocks_of(a.n, 8)), dim3(GEMM_THREADS), 0, st, a, across);
  return hipGetLastError() == hipSuccess ? MAXSIM_OK : MAXSIM_ERR_LAUNCH;
}

template <int DT> int ce_backward(CeArgs &a, int64_t pieces, int cus, hipStream_t st) {
  int rc = ce_gathered<DT>(a, DT == DT_FP16 || a.n > CE_DIRECT, st);
  if (rc != MAXSIM_OK) return rc;
  const int64_t any = (int64_t)1 << 30;
  using Z = CeLogits<DT, CE_BM, CE_BN, 2, CE_STAGES>;
  using H = CeLogits<DT, CE_BM, CE_HALF_BN, 2, CE_HALF_STAGES>;
  using G = TileGemm<DT, CE_PM, CE_PN, 2, SIDE_COLS_P, SIDE_COLS_P, CE_STAGES>;
  // with fewer rows there are fewer pieces and more tiles of dw in one
  if (CeUnits(a, a.n, CePieces(a.n, a.vocab, a.p_elements), Elem<DT>::bytes).w_splits == 1) a.w_slots = 0;
  for (a.piece = 0; a.piece < pieces; a.piece++) {
    rc = ce_half(a)
             ? ce_launch(ce_p_kernel<DT, CE_BM, CE_HALF_BN, 2, CE_HALF_STAGES>, any, H::lds, cus, a, st)
             : ce_launch(ce_p_kernel<DT, CE_BM, CE_BN, 2, CE_STAGES>, any, Z::lds, cus, a, st);
    if (rc == MAXSIM_OK) rc = ce_launch(ce_products_kernel<DT, CE_STAGES>, any, G::lds, cus, a, st);
    if (rc != MAXSIM_OK) return rc;
  }
  return a.dh || a.w_slots ? ce_launch(ce_parts_kernel<DT>, any, 0, cus, a, st) : MAXSIM_OK;
}

}  // namespace maxsim

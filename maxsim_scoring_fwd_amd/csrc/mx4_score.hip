// maxsim_score_mx4: checks and the choice of the kernel (mx4_score_kernel.hpp).
#include "host_common.hpp"
#include "mx4_score_kernel.hpp"

using namespace maxsim;

namespace {

constexpr int MX4_LDS_QUERY = 64 * 1024;  // most bytes of a query's codes held in LDS

template <int KS, int QB, bool QLDS, int SUB = 1> int mx4_launch(Mx4Args &a, const DeviceInfo &di, hipStream_t st) {
  // about 8 KiB of codes in flight a wave; at wide rows two tiles
  constexpr int P = KS >= 4 ? 2 : 8 / KS;
  const size_t lds = QLDS ? (size_t)QB * KS * WAVE * 17 : 0;
  auto kernel = mx4_score_kernel<KS, QB, P, QLDS, SUB>;
  int bpc = blocks_per_cu((const void *)kernel, DENSE_THREADS, lds);
  // Packed documents go to waves in whole ones: with fewer waves the longest share is nearer the mean,
  // and 12 waves a CU have bytes enough under way (20000 documents of 20 to 300 tokens, 32 query tokens,
  // as many workgroups as fit and 3 of them a CU: d = 32 21.3 and 21.9 us, 64 28.6 and 28.4, 96 42.5 and
  // 39.8, 128 50.0 and 49.4; 10000 with d = 256 53.5 and 52.4, 5000 with 512 60.8 and 60.9, 3000 with 1024
  // 83.5 both; 64 query tokens, d = 128, 48.9 and 48.6; fixed documents of equal length 136.3 and 136.5).
  // A query in LDS makes the matrix cores and LDS the bound, and those want every wave (5000 documents of
  // 20 to 340, d = 128: 128 query tokens 26.5 and 28.6 us, 300 61.5 and 64.0).
  if (!QLDS && a.doc.offsets && bpc > 3) bpc = 3;
  int64_t grid = (int64_t)di.cus * bpc;
  const int64_t most = (a.doc.n_docs + DENSE_WAVES - 1) / DENSE_WAVES;
  if (grid > most) grid = most;
  a.doc.contiguous = a.doc.n_docs >= 4 * grid * DENSE_WAVES;
  log_launch("mx4", (const void *)kernel, grid, DENSE_THREADS, lds, bpc);
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(DENSE_THREADS), lds, st, a);
  return hipGetLastError() == hipSuccess ? MAXSIM_OK : MAXSIM_ERR_LAUNCH;
}

// Up to 64 query tokens stay in registers; more come from LDS, all blocks for every tile, so that
// the documents are still read once.
template <int SUB> int mx4_narrow(int qb, Mx4Args &a, const DeviceInfo &di, hipStream_t st) {
  if (qb <= 1) return mx4_launch<1, 1, false, SUB>(a, di, st);
  if (qb <= 2) return mx4_launch<1, 2, false, SUB>(a, di, st);
  return mx4_launch<1, 4, false, SUB>(a, di, st);
}
template <int KS> int mx4_pick(Mx4Args &a, const DeviceInfo &di, hipStream_t st) {
  const int qb = (a.q_len + 15) / 16;
  if (KS == 1 && qb <= 4 && a.blocks <= 2) return a.blocks == 1 ? mx4_narrow<4>(qb, a, di, st) : mx4_narrow<2>(qb, a, di, st);
  if (qb <= 1) return mx4_launch<KS, 1, false>(a, di, st);
  if (qb <= 2) return mx4_launch<KS, 2, false>(a, di, st);
  if (qb <= 4) return mx4_launch<KS, 4, false>(a, di, st);
  if (qb <= 8) return mx4_launch<KS, 8, true>(a, di, st);
  if constexpr (KS <= 4)
    if (qb <= 16) return mx4_launch<KS, 16, true>(a, di, st);
  if constexpr (KS <= 2)
    if (qb <= 32) return mx4_launch<KS, 32, true>(a, di, st);
  if constexpr (KS <= 1)
    if (qb <= 64) return mx4_launch<KS, 64, true>(a, di, st);
  return MAXSIM_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" int maxsim_score_mx4(const uint8_t *Q, const uint8_t *q_scale, int q_len, const uint8_t *D,
                                const uint8_t *d_scale, const int64_t *doc_offsets, int64_t n_docs, int nd,
                                const int32_t *doc_lens, int d, float *out, void *stream) {
  if (n_docs < 0 || q_len < 1 || q_len > MAXSIM_MAX_Q_LEN || d < MAXSIM_MIN_D || d > MAXSIM_MAX_D || d % 32 ||
      (!doc_offsets && nd < 1))
    return MAXSIM_ERR_SHAPE;
  if (doc_offsets && doc_lens) return MAXSIM_ERR_UNSUPPORTED;
  const int steps = (d + 127) / 128, ks = steps <= 1 ? 1 : steps <= 2 ? 2 : steps <= 4 ? 4 : 8;
  if (q_len > 64 && (int64_t)((q_len + 15) / 16) * 16 * ks * 64 > MX4_LDS_QUERY) return MAXSIM_ERR_UNSUPPORTED;
  if (n_docs == 0) return MAXSIM_OK;  // arrays of no documents have no address
  if (!Q || !q_scale || !D || !d_scale || !out) return MAXSIM_ERR_NULL;
  if (!aligned(Q, 16) || !aligned(D, 16) || !aligned(out, 4) || (doc_offsets && !aligned(doc_offsets, 8)) ||
      (doc_lens && !aligned(doc_lens, 4)))
    return MAXSIM_ERR_ALIGN;
  DeviceInfo di;
  const int rc = current_device(di);
  if (rc != MAXSIM_OK) return rc;
  Mx4Args a{};
  a.doc.D = (const char *)D;
  a.doc.offsets = doc_offsets;
  a.doc.n_docs = n_docs;
  a.doc.nd = doc_offsets ? 0 : nd;
  a.doc.doc_lens = doc_lens;
  a.doc.out = out;
  a.d_scale = d_scale;
  a.q_scale = q_scale;
  a.Q = (const char *)Q;
  a.q_len = q_len;
  a.blocks = d / 32;
  hipStream_t st = (hipStream_t)stream;
  switch (ks) {
  case 1: return mx4_pick<1>(a, di, st);
  case 2: return mx4_pick<2>(a, di, st);
  case 4: return mx4_pick<4>(a, di, st);
  default: return mx4_pick<8>(a, di, st);
  }
}

// maxsim_linear_cross_entropy and its backward: checks, workspaces and the choice of the kernels
// (ce_kernels.hpp).
#include "ce_kernels.hpp"
#include "host_common.hpp"

using namespace maxsim;

namespace {

// Room for P, one piece of the vocabulary, and at least one tile of it for all rows. Fewer and longer
// pieces are worth more than a P that stays in the chip's 256 MiB cache: each piece adds to dh's
// sums and ends with workgroups that wait for the last (8192 x 30522 x 768 in bf16, both products
// of all pieces: room of 128 MiB 818 us, 256 MiB 718, 512 MiB 677, where P is one piece). Rows are wide
// there and P's own way to memory and back hides behind the products; at narrow widths it does not, and
// no other room was tried there.
constexpr int64_t CE_P_BYTES = (int64_t)512 << 20;
// Room for dh's tiles in parts: two for every workgroup that the chip holds at once, so that CeUnits
// can make parts short enough where there are few tiles; and for dw's of a piece, where there are less
// than one for each.
constexpr int64_t CE_SLOTS = 2 * CE_LANES;

// A step's panels are reached by 32-bit offsets.
constexpr int64_t CE_MOST_ROWS = (int64_t)1 << 22, CE_MOST_VOCAB = (int64_t)1 << 26;

struct Carver {
  char *base;
  size_t at = 0;
  template <typename T> T *take(int64_t n) {
    T *p = base ? (T *)(base + at) : nullptr;
    at += ((size_t)n * sizeof(T) + 255) & ~(size_t)255;
    return p;
  }
};

bool ce_sizes(int64_t n, int64_t vocab, int d, int dtype) {
  return n >= 0 && n <= CE_MOST_ROWS && vocab >= 1 && vocab <= CE_MOST_VOCAB && d >= 1 && d <= 16384 &&
         d * elem_bytes(dtype) % 16 == 0 &&
         blocks_of(n, CE_BN) * blocks_of(vocab, CE_BM) < ((int64_t)1 << 31);  // tiles are counted in 32 bits
}

// The workspace, carved up; with base NULL only its size is worked out.
size_t ce_carve(CeArgs &a, int eb, bool backward, char *base) {
  Carver c{base};
  a.counted = c.take<int32_t>(1);
  a.counts = c.take<int32_t>(blocks_of(a.n, CE_COUNT));
  a.most = c.take<float>(blocks_of(a.n, CE_COUNT));
  a.info = c.take<int4>(a.n);
  a.hc = c.take<char>(a.n * (blocks_of((int64_t)a.d * eb, PANEL) * PANEL));
  if (!backward) {
    const int64_t tiles = blocks_of(a.vocab, CE_BM);
    a.part = c.take<float2>(tiles * a.n);
    a.picked = c.take<float>(a.n);
    return c.at;
  }
  const int64_t rows = blocks_of(a.n, CE_BN) * CE_BN, tiles = blocks_of(a.vocab, CE_BM);
  int64_t p = CE_P_BYTES / eb;
  if (p > rows * tiles * CE_BM) p = rows * tiles * CE_BM;
  if (p < rows * CE_BM) p = rows * CE_BM;
  a.p_elements = p;
  a.p = c.take<char>(p * eb);
  a.queue = c.take<int32_t>(8);
  const int64_t cols = CePieces(a.n, a.vocab, p).cols;
  const int64_t h = blocks_of(a.d, CE_PM) * blocks_of(a.n, CE_PN), w = blocks_of(a.d, CE_PM) * blocks_of(cols, CE_PN);
  // no more than tiles and parts can be: fewer rows have fewer tiles of as many parts
  const int64_t h_most = h * (cols * eb / 64 / CE_H_LEAST + 1), room = h_most < CE_SLOTS ? h_most : CE_SLOTS;
  a.slots = h > room ? h : room;
  a.dhp = c.take<float>(a.slots * CE_PM * CE_PN);
  a.w_slots = w < CE_LANES && blocks_of(a.n * eb, 64) >= 2 * CE_W_LEAST ? CE_SLOTS : 0;
  a.dwp = c.take<float>(a.w_slots * CE_PM * CE_PN);
  return c.at;
}

size_t ce_workspace(int64_t n, int64_t vocab, int d, int dtype, bool backward) {
  const int eb = elem_bytes(dtype);
  if (eb == 0 || !ce_sizes(n, vocab, d, dtype) || n == 0) return 0;
  CeArgs a{};
  a.n = n;
  a.vocab = vocab;
  a.d = d;
  return ce_carve(a, eb, backward, nullptr);
}

int ce_checked(const void *h, const void *w, const int64_t *labels, int64_t n, int64_t vocab, int d, int dtype,
               float scale) {
  if (elem_bytes(dtype) == 0) return MAXSIM_ERR_DTYPE;
  if (!ce_sizes(n, vocab, d, dtype) || !(scale > 0 && scale <= __FLT_MAX__)) return MAXSIM_ERR_SHAPE;
  if (n > 0 && (!h || !labels)) return MAXSIM_ERR_NULL;
  if (n > 0 && !w) return MAXSIM_ERR_NULL;
  if (!aligned(h, 16) || !aligned(w, 16) || !aligned(labels, 8)) return MAXSIM_ERR_ALIGN;
  return MAXSIM_OK;
}

// dw where there is no row: a multiple of 16 bytes
__global__ void __launch_bounds__(256) ce_zero_kernel(u32x4_t *p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = u32x4_t{0, 0, 0, 0};
}

}  // namespace

extern "C" {

size_t maxsim_linear_cross_entropy_workspace_size(int64_t n_rows, int64_t vocab, int d, int dtype) {
  return ce_workspace(n_rows, vocab, d, dtype, false);
}

size_t maxsim_linear_cross_entropy_backward_workspace_size(int64_t n_rows, int64_t vocab, int d, int dtype) {
  return ce_workspace(n_rows, vocab, d, dtype, true);
}

int maxsim_linear_cross_entropy(const void *h, const void *w, const int64_t *labels, int64_t n_rows,
                                int64_t vocab, int d, int dtype, float scale, float *loss, float *lse,
                                void *workspace, size_t workspace_bytes, void *stream) {
  int rc = ce_checked(h, w, labels, n_rows, vocab, d, dtype, scale);
  if (rc != MAXSIM_OK) return rc;
  if (n_rows == 0) return MAXSIM_OK;
  if (!loss || !lse || !workspace) return MAXSIM_ERR_NULL;
  if (!aligned(loss, 4) || !aligned(lse, 4) || !aligned(workspace, 16)) return MAXSIM_ERR_ALIGN;
  if (workspace_bytes < ce_workspace(n_rows, vocab, d, dtype, false)) return MAXSIM_ERR_SHAPE;
  DeviceInfo di;
  rc = current_device(di);
  if (rc != MAXSIM_OK) return rc;
  CeArgs a{};
  a.h = (const char *)h;
  a.w = (const char *)w;
  a.labels = labels;
  a.n = n_rows;
  a.vocab = vocab;
  a.d = d;
  a.row_bytes = d * elem_bytes(dtype);
  a.scale = scale;
  a.loss = loss;
  a.lse = lse;
  ce_carve(a, elem_bytes(dtype), false, (char *)workspace);
  hipStream_t st = (hipStream_t)stream;
  return dtype == MAXSIM_BF16   ? ce_forward_bf16(a, di.cus, st)
         : dtype == MAXSIM_FP16 ? ce_forward_fp16(a, di.cus, st)
                                : ce_forward_fp32(a, di.cus, st);
}

int maxsim_linear_cross_entropy_backward(const float *grad_loss, const void *h, const void *w,
                                         const int64_t *labels, const float *lse, int64_t n_rows, int64_t vocab,
                                         int d, int dtype, float scale, void *dh, void *dw, void *workspace,
                                         size_t workspace_bytes, void *stream) {
  int rc = ce_checked(h, w, labels, n_rows, vocab, d, dtype, scale);
  if (rc != MAXSIM_OK) return rc;
  if ((!dh && !dw) || (n_rows == 0 && !dw)) return MAXSIM_OK;
  if (n_rows > 0 && (!grad_loss || !lse || !workspace)) return MAXSIM_ERR_NULL;
  if (!aligned(grad_loss, 4) || !aligned(lse, 4) || !aligned(dh, 16) || !aligned(dw, 16) || !aligned(workspace, 16))
    return MAXSIM_ERR_ALIGN;
  if (workspace_bytes < ce_workspace(n_rows, vocab, d, dtype, true)) return MAXSIM_ERR_SHAPE;
  DeviceInfo di;
  rc = current_device(di);
  if (rc != MAXSIM_OK) return rc;
  if (n_rows == 0) {
    hipLaunchKernelGGL(ce_zero_kernel, dim3(4 * di.cus), dim3(256), 0, (hipStream_t)stream, (u32x4_t *)dw,
                       vocab * (d * elem_bytes(dtype) / 16));
    return hipGetLastError() == hipSuccess ? MAXSIM_OK : MAXSIM_ERR_LAUNCH;
  }
  CeArgs a{};
  a.h = (const char *)h;
  a.w = (const char *)w;
  a.labels = labels;
  a.grad = grad_loss;
  a.n = n_rows;
  a.vocab = vocab;
  a.d = d;
  a.row_bytes = d * elem_bytes(dtype);
  a.scale = scale;
  a.lse = const_cast<float *>(lse);
  a.dh = (char *)dh;
  a.dw = (char *)dw;
  ce_carve(a, elem_bytes(dtype), true, (char *)workspace);
  const int64_t pieces = CePieces(n_rows, vocab, a.p_elements).n;
  hipStream_t st = (hipStream_t)stream;
  return dtype == MAXSIM_BF16   ? ce_backward_bf16(a, pieces, di.cus, st)
         : dtype == MAXSIM_FP16 ? ce_backward_fp16(a, pieces, di.cus, st)
                                : ce_backward_fp32(a, pieces, di.cus, st);
}

}  // extern "C"

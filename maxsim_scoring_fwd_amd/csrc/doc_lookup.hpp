// Finding the document of a packed token, or of a tile of packed tokens, from doc_offsets.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace maxsim {

// Index of packed token t within its document (one thread's search, log2(n_docs) steps). A
// token before the first offset or past the last counts from the nearest offset below it, or
// from zero.
__device__ __forceinline__ int64_t place_in_document(const int64_t *offsets, int64_t n_docs,
                                                     int64_t t) {
  int64_t lo = 0, hi = n_docs + 1;  // the first offset past t lies in [lo, hi]
  while (lo < hi) {
    const int64_t mid = lo + (hi - lo) / 2;
    if (offsets[mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo == 0 ? t : t - offsets[lo - 1];
}

// Tiles over packed documents without a plan made beforehand and without reading the offsets
// on the host. The token range is cut at every offset, which gives n_docs + 2 spans: the tokens
// before the first offset (no document), the documents, and the tokens after the last offset
// (no document). Span s that begins at token `begin` owns the tile slots from
// begin / rows + s on: for any length that is at least ceil(length / rows) slots before the
// next span's first one, so n_tokens / rows + n_docs + 2 slots hold every tile, and a slot past
// its span's length is empty.
struct TileSpan {
  int64_t begin;  // first token of the span
  int64_t len;    // tokens of the span
  int64_t first;  // first row of this tile within the span
  int64_t doc;    // document, or -1
};

// One wave's search, 64 probes a step: two steps for up to 4096 documents. Offsets are clamped
// to the token range, so that no tile reaches past it whatever they hold.
__device__ __forceinline__ TileSpan find_tile(const int64_t *offsets, int64_t n_docs,
                                              int64_t n_tokens, int64_t slot, int rows) {
  const int lane = threadIdx.x & 63;
  auto begin_of = [&](int64_t s) -> int64_t {
    if (s == 0) return 0;
    if (s > n_docs + 1) return n_tokens;
    const int64_t o = offsets[s - 1];
    return o < 0 ? 0 : (o > n_tokens ? n_tokens : o);
  };
  int64_t lo = 0, hi = n_docs + 2;
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 63) / 64;
    const int64_t p = lo + lane * step;
    const bool in = p < hi && (p == lo || begin_of(p) / rows + p <= slot);
    const uint64_t mask = __ballot(in);
    const int last = 63 - __builtin_clzll(mask | 1);
    lo += last * step;
    hi = lo + step < hi ? lo + step : hi;
  }
  TileSpan t;
  t.begin = begin_of(lo);
  const int64_t end = begin_of(lo + 1);
  t.len = end > t.begin ? end - t.begin : 0;
  t.first = (slot - (t.begin / rows + lo)) * rows;
  t.doc = lo == 0 || lo == n_docs + 1 ? -1 : lo - 1;
  return t;
}

}  // namespace maxsim

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

// v of one lane, in all.
__device__ __forceinline__ int64_t lane_value(int64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)((uint64_t)v >> 32), lane);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// n / d for n < 2^31 by a multiplication: with 2^s the first power of two that is at least d and
// m = ceil(2^(31 + s) / d), m * d exceeds 2^(31 + s) by less than 2^s, which n < 2^31 does not
// carry into the quotient.
struct FastDiv {
  uint32_t d, m, shift;
  void set(uint32_t by) {
    d = by;
    uint32_t s = 0;
    while (((uint64_t)1 << s) < by) s++;
    m = by > 1 ? (uint32_t)((((uint64_t)1 << (31 + s)) + by - 1) / by) : 0;
    shift = s ? s - 1 : 0;
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    return d == 1 ? n : __umulhi(n, m) >> shift;
  }
};

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

// One wave's search, 63 probes a step: one step for up to 61 documents. Lane 63 looks one probe
// further, so that the last step also knows where the span ends. With more documents the first
// step looks at the 63 spans around the one that documents of equal length would put there, which
// is right for most tiles, and the next ones search what that has left. Offsets are clamped to the
// token range, so that no tile reaches past it whatever they hold.
__device__ __forceinline__ TileSpan find_tile(const int64_t *offsets, int64_t n_docs,
                                              int64_t n_tokens, int64_t slot, int rows) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, hi = n_docs + 2, begin = 0;
  const float spans = (float)(n_docs + 2), slots = (float)(n_tokens / rows + n_docs + 2);
  int64_t from = hi <= 63 ? 0 : (int64_t)((float)slot * (spans / slots)) - 31;
  from = from < 0 ? 0 : (from > hi - 63 ? (hi > 63 ? hi - 63 : 0) : from);
  int64_t step = 1;
  int last = 0;
  for (;;) {
    int64_t p = from + lane * step;
    p = p < hi ? p : hi;
    int64_t o = 0;
    if (p > 0) o = p > n_docs + 1 ? n_tokens : offsets[p - 1];
    begin = o < 0 ? 0 : (o > n_tokens ? n_tokens : o);
    const bool in = lane < 63 && p < hi && (p == lo || begin / rows + p <= slot);
    const uint64_t found = __ballot(in);
    if (found == 0) {  // before the window
      hi = from;
    } else {
      last = 63 - __builtin_clzll(found);
      const int64_t past = from + (last + 1) * step;
      lo = from + last * step;
      // the last probe of the window may have spans of its own behind it
      if (last < 62 || step > 1) hi = past < hi ? past : hi;
      if (hi - lo <= 1 || (step == 1 && last < 62)) break;
    }
    from = lo;
    step = (uint64_t)(hi - lo + 62) / 63;
  }
  TileSpan t;
  t.begin = lane_value(begin, last);
  const int64_t end = lane_value(begin, last + 1);
  t.len = end > t.begin ? end - t.begin : 0;
  t.first = (slot - (t.begin / rows + lo)) * rows;
  t.doc = lo == 0 || lo == n_docs + 1 ? -1 : lo - 1;
  return t;
}

}  // namespace maxsim

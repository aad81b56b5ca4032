// paged.cuh -- addressing of a paged key/value cache and the division of a decode batch's work.
//
// A cache is a pool of pages of `page_size` positions. Row b of the page table names the page of
// each block of page_size positions of sequence b, so position j of head h lies at
//   page_table[b][j / page_size] * page_stride + (j % page_size) * tok_stride + h * head_stride
// (elements; 64-bit, a pool may hold more than 2^31 elements).
#pragma once

#include "common.cuh"
#include "launch.h"

namespace sdpa {

// pos / page_size for 0 <= pos < 2^31 without a division: with l = ceil(log2 d) and
// m = floor(2^32 (2^l - d) / d) + 1, n / d = (mulhi(m, n) + n) >> l (Granlund and Montgomery,
// "Division by invariant integers using multiplication", 1994). The host computes m and l.
__device__ __forceinline__ int page_of(const PagedArgs& p, int pos) {
  return (int)((__umulhi(p.div_mul, (uint32_t)pos) + (uint32_t)pos) >> p.div_shift);
}

// What a query at position len - 1 sees of a sequence, in tiles of `tile` keys: positions
// 0 .. sinks - 1 and lo .. len - 1. Tiles that hold no visible key are left out: a unit's tile t
// covers positions start(t) .. start(t) + tile - 1, the sinks' tiles first, then those of the
// window. An empty sequence has one tile without a visible key, which writes its outputs.
struct KeySpan {
  int len, lo, sinks;  // visible: j < len and (j >= lo or j < sinks)
  int ns, gap, nt;     // tiles before the gap, tiles left out, tiles in all

  __device__ __forceinline__ void set(int length, int window, int sink_tokens, int tile) {
    len = length;
    lo = len > window ? len - window : 0;
    sinks = sink_tokens;
    const int all = (len + tile - 1) / tile;
    const int first = lo / tile;
    ns = (min(sinks, lo) + tile - 1) / tile;
    gap = first > ns ? first - ns : 0;
    nt = all - gap > 0 ? all - gap : 1;
  }
  __device__ __forceinline__ int start(int t, int tile) const { return (t < ns ? t : t + gap) * tile; }
  __device__ __forceinline__ bool sees(int j) const { return j < len && (j >= lo || j < sinks); }
};

// The length of row b, or 0 (with ATTN_ERR_DATA recorded) where it does not fit the page table.
__device__ __forceinline__ int row_length(const PagedArgs& p, int b, int* status) {
  const int len = __ldg(p.seq_lens + b);
  if (len < 0 || len > p.max_pages * p.page_size) {
    report(status, ATTN_ERR_DATA);
    return 0;
  }
  return len;
}

}  // namespace sdpa

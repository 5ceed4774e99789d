// Arguments of the attention kernels over the 8-bit paged cache (internal).
#pragma once

#include "kvcache.cuh"

namespace sv {

struct AttendArgs {
  KvCache c;
  const char* q;
  long qb, qt, qh;  // strides in elements
  int B, W, Hq, G;  // G = Hq / H query heads per KV head
  const int32_t* seq;
  const int32_t* win;
  const int32_t* masks;
  int words;        // mask words per row
  float scale_log2; // scale * log2(e)
  char* out;
  float* lse;
};

// A request's lengths; false when they are out of range.
__device__ __forceinline__ bool attend_lens(const AttendArgs& a, int b, long* seq, int* w) {
  *seq = a.seq[b];
  *w = a.win ? a.win[b] : a.W;
  return *seq >= 0 && *w >= 0 && *w <= a.W && *seq + *w <= (long)a.c.max_blocks * a.c.tpb;
}

}  // namespace sv

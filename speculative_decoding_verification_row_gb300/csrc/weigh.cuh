// Arguments of the kernels that weigh cached positions (internal).
#pragma once

#include "attend.cuh"

namespace sv {

struct WeighArgs : AttendArgs {  // what the work division reads, q, and the cache
  const float* row_lse;
  const float* old;
  float scale, decay;
  float* sum;
  int T;
};

// Four e4m3 codes as two pairs of T.
__device__ __forceinline__ void e4m3x4_to(uint32_t w, uint32_t& lo, uint32_t& hi, __half*) {
  e4m3x4_to_half(w, lo, hi);
}
__device__ __forceinline__ void e4m3x4_to(uint32_t w, uint32_t& lo, uint32_t& hi, __nv_bfloat16*) {
  uint32_t a, b;
  e4m3x4_to_half(w, a, b);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  lo = pack_out(x.x, x.y, (__nv_bfloat16*)nullptr);
  hi = pack_out(y.x, y.y, (__nv_bfloat16*)nullptr);
}

// weigh.cu: few rows per KV head.
cudaError_t launch_weigh_rows(const WeighArgs& a, int dtype, cudaStream_t st);
// weigh_tiles.cu: many rows per KV head.
size_t weigh_tiles_scratch();
cudaError_t launch_weigh_tiles(WeighArgs& a, int dtype, void* scratch, cudaStream_t st);

}  // namespace sv

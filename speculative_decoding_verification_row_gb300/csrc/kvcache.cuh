// The 8-bit paged KV cache on the device (internal): addressing, the scale
// rule and the e4m3 conversions shared by the store, the relocation and the
// attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kernels.cuh"

namespace sv {

struct KvCache {
  uint8_t* pool;
  float* scales;
  const int32_t* tables;
  int num_blocks, max_blocks, tpb, H, D;
  // Byte offset of row `off` of (block, kind, head): 64 bits, a pool passes 4 GB.
  __device__ __forceinline__ size_t row(int blk, int kind, int h, int off) const {
    return ((((size_t)blk * 2 + kind) * H + h) * tpb + off) * D;
  }
  __device__ __forceinline__ size_t scale_at(int blk, int kind, int h) const {
    return ((size_t)blk * 2 + kind) * H + h;
  }
  // Block of logical position t of request b, or -1 when it is unmapped.
  __device__ __forceinline__ int block(int b, long t) const {
    if (t < 0 || t >= (long)max_blocks * tpb) return -1;
    const int blk = tables[(size_t)b * max_blocks + t / tpb];
    return blk < 0 || blk >= num_blocks ? -1 : blk;
  }
};

// Host check of a cache descriptor; fills `c`.
inline int kv_setup(const spec_kv_cache* s, KvCache* c) {
  if (!s || s->size != sizeof(spec_kv_cache) || !s->pool || !s->scales || !s->block_tables)
    return SPEC_EINVAL;
  if (s->num_blocks < 1 || s->max_blocks < 1 || s->tokens_per_block < 16 ||
      s->tokens_per_block > 1024 || s->tokens_per_block % 16 != 0 || s->kv_heads < 1 ||
      s->kv_heads > 1024 || (s->head_dim != 64 && s->head_dim != 128) ||
      reinterpret_cast<uintptr_t>(s->pool) % 32 != 0)
    return SPEC_EINVAL;
  *c = KvCache{static_cast<uint8_t*>(s->pool), s->scales, s->block_tables, s->num_blocks,
               s->max_blocks, s->tokens_per_block, s->kv_heads, s->head_dim};
  return SPEC_OK;
}

// Host check of a strided [B, W, heads, D] array: 16-byte vectors along D.
inline bool kv_strides_ok(const void* p, const int64_t* st) {
  return p && st && reinterpret_cast<uintptr_t>(p) % 16 == 0 && st[0] % 8 == 0 &&
         st[1] % 8 == 0 && st[2] % 8 == 0;
}

// The least power of two s >= 2^-126 with amax <= 448 s (448 = 1.75 * 2^8 is
// the largest e4m3 value); 0 for amax = 0.  amax is finite.
__device__ __forceinline__ float scale_for(float amax) {
  if (!(amax > 0.f)) return 0.f;
  int e;
  const float m = frexpf(amax, &e);  // amax = m 2^e, m in [1/2, 1)
  e = m <= 0.875f ? e - 9 : e - 8;
  return ldexpf(1.f, e < -126 ? -126 : e);
}

// a / b, and 0 where b is 0.
__device__ __forceinline__ float scale_ratio(float a, float b) { return b > 0.f ? a / b : 0.f; }

// Two floats to e4m3, nearest, ties to even; not finite: NaN.
__device__ __forceinline__ unsigned short to_e4m3x2(float a, float b) {
  a = fabsf(a) < INFINITY ? a : NAN;
  b = fabsf(b) < INFINITY ? b : NAN;
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Four e4m3 codes times r, rounded again.
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t w, float r) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3));
    const float2 f = __half22float2(h);
    out |= (uint32_t)to_e4m3x2(f.x * r, f.y * r) << (16 * i);
  }
  return out;
}

__device__ __forceinline__ uint4 rescale_e4m3x16(uint4 v, float r) {
  return make_uint4(rescale_e4m3x4(v.x, r), rescale_e4m3x4(v.y, r), rescale_e4m3x4(v.z, r),
                    rescale_e4m3x4(v.w, r));
}

}  // namespace sv

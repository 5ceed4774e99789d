// Attention of a window's rows over the paged 8-bit cache (spec_attend_kv).
//
// out = sum_t p_t v_t, p = softmax(scale q . k_t), one pass over the keys
// with the running maximum m and sum l of 2^(s - m), s in log2 units.
#include "attend.cuh"

namespace sv {

namespace {

constexpr int kSimpleWarps = 4;

// One CTA = one window token and query head; each warp takes every fourth
// key, D / 32 elements per lane.
template <class T, int D>
__global__ void __launch_bounds__(kSimpleWarps * 32) attend_simple_kernel(const AttendArgs a) {
  constexpr int E = D / 32;
  const KvCache& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hq = blockIdx.x % a.Hq, i = blockIdx.x / a.Hq % a.W, b = blockIdx.x / a.Hq / a.W;
  const int h = hq / a.G;
  long seq;
  int w;
  const bool good = attend_lens(a, b, &seq, &w);
  if (good && i >= w) return;
  const size_t orow = ((size_t)b * a.W + i) * a.Hq + hq;
  T* out = reinterpret_cast<T*>(a.out) + orow * D;
  if (!good) {
    for (int e = threadIdx.x; e < D; e += blockDim.x) out[e] = (T)NAN;
    if (a.lse && threadIdx.x == 0) a.lse[orow] = NAN;
    return;
  }
  const T* q = reinterpret_cast<const T*>(a.q) + b * a.qb + i * a.qt + hq * a.qh;
  float qv[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) qv[e] = (float)q[lane * E + e], o[e] = 0.f;
  float m = -INFINITY, l = 0.f;
  bool bad = false;
  for (long t = (long)threadIdx.x * c.tpb; t < seq + w; t += (long)blockDim.x * c.tpb)
    bad = bad || c.block(b, t) < 0;
  const int32_t* mask = a.masks ? a.masks + ((size_t)b * a.W + i) * a.words : nullptr;
  for (long t = warp; t < seq + w; t += kSimpleWarps) {
    const long j = t - seq;
    if (j >= 0 && (mask ? !(mask[j >> 5] >> (j & 31) & 1) : j > i)) continue;
    const int blk = c.block(b, t);
    if (blk < 0) break;
    const uint8_t* kr = c.pool + c.row(blk, 0, h, (int)(t % c.tpb)) + lane * E;
    const uint8_t* vr = c.pool + c.row(blk, 1, h, (int)(t % c.tpb)) + lane * E;
    auto val = [](uint8_t x) { return __half2float(__half(__nv_cvt_fp8_to_halfraw(x, __NV_E4M3))); };
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += qv[e] * val(kr[e]);
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    s *= a.scale_log2 * c.scales[c.scale_at(blk, 0, h)];
    const float mn = fmaxf(m, s), al = exp2f(m - mn), p = exp2f(s - mn);
    const float pv = p * c.scales[c.scale_at(blk, 1, h)];
    l = l * al + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * al + pv * val(vr[e]);
    m = mn;
  }
  __shared__ float sM[kSimpleWarps], sL[kSimpleWarps], sO[kSimpleWarps][D];
  __shared__ int sBad;
  if (threadIdx.x == 0) sBad = 0;
  __syncthreads();
  if (bad) sBad = 1;
  if (lane == 0) sM[warp] = m, sL[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) sO[warp][lane * E + e] = o[e];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int k = 0; k < kSimpleWarps; ++k) M = fmaxf(M, sM[k]);
  auto none = [&](int k) { return sM[k] == -INFINITY && sL[k] == 0.f; };
  for (int k = 0; k < kSimpleWarps; ++k) L += none(k) ? 0.f : sL[k] * exp2f(sM[k] - M);
  for (int e = threadIdx.x; e < D; e += blockDim.x) {
    float x = 0.f;
    for (int k = 0; k < kSimpleWarps; ++k)
      x += none(k) ? 0.f : sO[k][e] * exp2f(sM[k] - M);
    out[e] = (T)(sBad ? NAN : L > 0.f ? x / L : x);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[orow] = sBad ? NAN : L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_attend_scratch_size(int B, int W, int q_heads, int kv_heads, int head_dim) {
  if (B < 1 || B > SPEC_MAX_BATCH || W < 1 || W > SPEC_MAX_WINDOW || kv_heads < 1 ||
      kv_heads > 1024 || q_heads < 1 || q_heads > 16384 || q_heads % kv_heads != 0 ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return 256;
}

int spec_attend_kv(const spec_kv_cache* cache, const spec_attend_params* p, void* scratch,
                   size_t scratch_bytes, spec_stream_t stream) {
  AttendArgs a{};
  const int rc = kv_setup(cache, &a.c);
  if (rc != SPEC_OK) return rc;
  if (!p || p->size != sizeof(spec_attend_params) || !kv_strides_ok(p->q, p->q_strides) ||
      (p->dtype != SPEC_BF16 && p->dtype != SPEC_F16) || !p->seq_lens || !p->out ||
      reinterpret_cast<uintptr_t>(p->out) % 16 != 0 || !isfinite(p->scale) ||
      (p->masks && p->W > SPEC_MAX_TREE_NODES))
    return SPEC_EINVAL;
  const size_t need = spec_attend_scratch_size(p->B, p->W, p->q_heads, a.c.H, a.c.D);
  if (need == 0) return SPEC_EINVAL;
  if (!scratch || reinterpret_cast<uintptr_t>(scratch) % 256 != 0 || scratch_bytes < need)
    return SPEC_EWORKSPACE;
  a.q = static_cast<const char*>(p->q);
  a.qb = p->q_strides[0];
  a.qt = p->q_strides[1];
  a.qh = p->q_strides[2];
  a.B = p->B;
  a.W = p->W;
  a.Hq = p->q_heads;
  a.G = p->q_heads / a.c.H;
  a.seq = p->seq_lens;
  a.win = p->window_lens;
  a.masks = p->masks;
  a.words = (p->W + 31) / 32;
  a.scale_log2 = (float)((double)p->scale * 1.4426950408889634073599246810019);
  a.out = static_cast<char*>(p->out);
  a.lse = p->out_lse;
  const long grid = (long)a.B * a.W * a.Hq;
  if (grid > INT_MAX) return SPEC_EINVAL;
  auto go = [&](auto kernel) {
    kernel<<<(unsigned)grid, kSimpleWarps * 32, 0, (cudaStream_t)stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
  };
  if (p->dtype == SPEC_BF16)
    return a.c.D == 64 ? go(attend_simple_kernel<__nv_bfloat16, 64>)
                       : go(attend_simple_kernel<__nv_bfloat16, 128>);
  return a.c.D == 64 ? go(attend_simple_kernel<__half, 64>) : go(attend_simple_kernel<__half, 128>);
}

}  // extern "C"

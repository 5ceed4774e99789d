// Rotary positions on the device (internal): the angle of a position and the
// rotation of a token's rows, shared by the rotation and the rotating store.
#pragma once

#include "kvcache.cuh"

namespace sv {

// Rows of one kind: [B, W, heads, D], strides in elements, in and out.
struct RotateRows {
  const char* in;
  char* out;
  long ib, it, ih, ob, ot, oh;
  int heads;
};

struct RotateArgs {
  RotateRows x[2];  // q, k
  int B, W, D;
  const int32_t* starts;
  const int32_t* win;
  const int32_t* masks;
  const double* inv_freq;
  int pairs, interleaved;
  float gain;
};

// |f| / (2 pi) modulo 1, in units of 2^-64 turns, with f's sign: what one position adds to the angle.
// Integers only: 53 bits of f times the first 64 bits of 1 / (2 pi).  The multiple
// by a position is exact modulo a turn, and off by |position f| 2^-64 turns for
// the constant's end and |position| 2^-64 for the shift's: less than 2^-30 + 2^-33
// turns while |position f| stays below 2^34 radians, and more beyond.  f is finite.
__device__ __forceinline__ uint64_t turns_of(double f) {
  constexpr uint64_t kInvTau = 0x28be60db9391054aull;  // floor(2^64 / (2 pi))
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int e = (int)(bits >> 52 & 2047) - 1023;
  if (e < -64) return 0;  // no position turns it by 2^-33
  const uint64_t m = (bits << 11) | 1ull << 63;  // |f| = m 2^(e - 63)
  const uint64_t lo = m * kInvTau, hi = __umul64hi(m, kInvTau);
  const int down = 63 - e;  // turns = (hi:lo) >> down
  uint64_t t = 0;
  if (down <= 0)
    t = down > -64 ? lo << -down : 0;
  else if (down < 64)
    t = hi << (64 - down) | lo >> down;
  else if (down < 128)
    t = hi >> (down - 64);
  return bits >> 63 ? 0 - t : t;
}

// Sine and cosine of position * f, times the gain.  The angle becomes a float
// within an eighth of a turn of a multiple of a quarter: off by at most 2^-26 of
// a half turn, where a whole turn's would be off by 2^-25.  Sine and cosine of a
// float, by sincospif in fp32, are up to 2^-22 off where 64-bit ones rounded once
// would be 2^-25: what follows is rounded to 8 or 11 bits, and prompts of 4001
// tokens in fp16 are 1.2e-4 off with either.
__device__ __forceinline__ float2 angle_at(uint64_t turns, long position, float gain) {
  const uint64_t at = (uint64_t)position * turns;  // modulo a turn
  const uint64_t quarter = (at + (1ull << 61)) >> 62;
  const int32_t rest = (int32_t)((int64_t)(at - (quarter << 62)) >> 30);  // 2^-34 turns
  float s, c;
  sincospif((float)rest * 0x1p-33f, &s, &c);
  const float x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s;
  return quarter & 2 ? make_float2(-x * gain, -y * gain) : make_float2(x * gain, y * gain);
}

// Depth of a window token: its place in a chain, else its mask's bits without its own.
__device__ __forceinline__ int depth_of(const int32_t* masks, int W, int b, int i) {
  if (!masks) return i;
  const int words = (W + 31) >> 5;
  const int32_t* row = masks + ((size_t)b * W + i) * words;
  int n = 0;
  for (int x = 0; x < words; ++x) {
    const int left = W - x * 32;
    n += __popc((uint32_t)row[x] & (left < 32 ? (1u << left) - 1 : ~0u));
  }
  return n > 0 ? n - 1 : 0;
}

template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(bf16_lo(w), bf16_hi(w));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <class T>
__device__ __forceinline__ uint32_t pack2(float x, float y);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float x, float y) {
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The elements of a turned pair.  One rounding order wherever a pair is turned:
// the rotation and the rotating store give the same bits.
__device__ __forceinline__ float turn_a(float a, float b, float2 t) {
  return __fmaf_rn(a, t.x, -__fmul_rn(b, t.y));
}
__device__ __forceinline__ float turn_b(float a, float b, float2 t) {
  return __fmaf_rn(b, t.x, __fmul_rn(a, t.y));
}

// Pairs that lie in one 16-byte vector (interleaved), four of them.
template <class T>
__device__ __forceinline__ void turn_inside(uint4& x, const float2* cs) {
  uint32_t* w = &x.x;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 v = unpack2<T>(w[k]), t = cs[k];
    w[k] = pack2<T>(turn_a(v.x, v.y, t), turn_b(v.x, v.y, t));
  }
}

// Pairs across two vectors (half layout), eight of them: their first elements
// (which 1), their second (2), or both (3).
template <class T, int WHICH>
__device__ __forceinline__ void turn_across(uint4& x, uint4& y, const float2* cs) {
  uint32_t *a = &x.x, *b = &y.x;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 u = unpack2<T>(a[k]), v = unpack2<T>(b[k]), t0 = cs[2 * k], t1 = cs[2 * k + 1];
    if (WHICH & 1) a[k] = pack2<T>(turn_a(u.x, v.x, t0), turn_a(u.y, v.y, t1));
    if (WHICH & 2) b[k] = pack2<T>(turn_b(u.x, v.x, t0), turn_b(u.y, v.y, t1));
  }
}

constexpr int kTurnThreads = 128;
constexpr int kMaxPairs = 256;

// One token of a window, by a CTA of kTurnThreads: its heads share the angles
// (cs, shared memory), which its threads compute while their first rows are on
// the way.
template <class T, bool INTER>
__device__ __forceinline__ void rotate_token(const RotateArgs& a, int b, int i, float2* cs) {
  const int tid = threadIdx.x;
  const int w = a.win ? a.win[b] : a.W;
  if (i >= w || w > a.W) return;
  const int per = a.D / 16;        // tasks of a row: 16 elements each
  const int turned = a.pairs / 8;  // those that turn; the others copy
  const int total = per * (a.x[0].heads + a.x[1].heads);
  uint4 u, v;
  char *to_u, *to_v;
  // the two vectors of a task, and where they go
  auto load = [&](int task) {
    int head = task / per;
    const int x = task - head * per;
    const bool second = head >= a.x[0].heads;
    const RotateRows& r = a.x[second];
    if (second) head -= a.x[0].heads;
    const bool half = !INTER && x < turned;
    const int eu = half ? 8 * x : 16 * x, ev = half ? a.pairs + 8 * x : 16 * x + 8;
    const char* in = r.in + 2 * (b * r.ib + i * r.it + head * r.ih);
    char* out = r.out + 2 * (b * r.ob + i * r.ot + head * r.oh);
    u = *reinterpret_cast<const uint4*>(in + 2 * eu);
    v = *reinterpret_cast<const uint4*>(in + 2 * ev);
    to_u = out + 2 * eu;
    to_v = out + 2 * ev;
    return x;
  };
  int x = tid < total ? load(tid) : 0;
  const long position = (long)a.starts[b] + depth_of(a.masks, a.W, b, i);
  for (int p = tid; p < a.pairs; p += kTurnThreads) cs[p] = angle_at(turns_of(a.inv_freq[p]), position, a.gain);
  __syncthreads();
  for (int task = tid; task < total; task += kTurnThreads) {
    if (task != tid) x = load(task);
    if (x < turned) {
      if (INTER) {
        turn_inside<T>(u, cs + 8 * x);
        turn_inside<T>(v, cs + 8 * x + 4);
      } else {
        turn_across<T, 3>(u, v, cs + 8 * x);
      }
    }
    *reinterpret_cast<uint4*>(to_u) = u;
    *reinterpret_cast<uint4*>(to_v) = v;
  }
}

// Host check of a rotation's arguments; fills `a`.
int rotate_setup(const spec_rotate_params* p, RotateArgs* a);
// Its arrays, eight of them.
void rotate_arrays(const spec_rotate_params* p, Arrays* x);
// Enqueues the rotation of all rows (rotary.cu).
cudaError_t launch_rotate(const RotateArgs& a, int dtype, cudaStream_t st);

}  // namespace sv

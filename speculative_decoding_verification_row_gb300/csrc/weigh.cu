// The attention that each cached position drew from a window's rows
// (spec_weigh_kv).
//
// Tensor cores through mma.sync m16n8k16, the keys as the left operand: a
// warp holds 16 keys in registers, converted from e4m3 to fp16 (exact) once,
// and lets the rows pass; each lane adds up the weights of its two keys, so that
// the sum over rows needs four shuffles per tile and no atomics.  bf16 rows are
// scaled by a power of two to a largest magnitude in [2^14, 2^15) and rounded to
// fp16: exact down to 2^-28 of the row's largest.  (Keys as bf16 instead took 128
// of a tile's some 250 instructions: 78 us for 64 windows of 1 to 4 tokens over
// 512 to 8192 positions, 32/8 heads of 128.)  A weight is exp of a score less
// the row's lse, at most 1 but for rounding; the tensor cores cut a score's partial
// sums off, and exp2 is ex2.approx: 8 rows of 4 heads of 128 in fp16 over 700
// positions are 2.4e-7 off (of the weights' norm), fp32 products and exp 2.0e-7.
//
// Bound by the bytes under way: 16 warps an SM with a tile each.  In a graph that
// case takes 75 us, 4.0 TB/s (0.60 of the measured copy rate); 100 requests of
// one token over 8192 positions 180 us, 5.0 TB/s.
#include "weigh.cuh"

namespace sv {

constexpr int kAllRows = 1 << 30;

// A unit of all rows of a request and KV head: every position it has, also where
// the window is empty; none for lengths out of range.
template <int KEYS>
struct Division<kAllRows, KEYS> {
  static __device__ __forceinline__ void lens(const AttendArgs& a, int b, int* seq, int* w) {
    Division<1, KEYS>::lens(a, b, seq, w);
  }
  static __device__ __forceinline__ int tiles(const AttendArgs&, int seq, int w, int) {
    return w < 0 ? 0 : (int)(((unsigned)seq + (unsigned)w + KEYS - 1) / KEYS);
  }
  static __device__ __forceinline__ bool next(const AttendArgs& a, Unit& u) {
    if (++u.h < a.c.H) return true;
    u.h = 0;
    do {
      if (++u.b == a.B) return false;
      lens(a, u.b, &u.seq, &u.w);
      u.tiles = tiles(a, u.seq, u.w, 0);
    } while (u.tiles == 0);
    return true;
  }
};

namespace {

constexpr int kWWarps = 4, kWThreads = kWWarps * 32;
constexpr int kWKeys = 16 * kWWarps;  // keys of a tile
constexpr int kWRows = 32;            // most rows of a KV head
constexpr int kWCost = 2;             // cells of a unit besides its tiles
constexpr int kWLeast = 4;            // cells below which a share is not worth a CTA
constexpr int kWCtas = 4 * kSms;

__device__ __forceinline__ void mma_k16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <class T, int D>
__global__ void __launch_bounds__(kWThreads, 4) weigh_kernel(const WeighArgs a) {
  constexpr int U = D / 64;           // 16-byte chunks of a key per thread
  constexpr int kPitch = 2 * D + 16;  // bytes of a staged row: its 16-byte reads hit all banks once
  constexpr float kLog2e = 1.4426950408889634f;
  __shared__ __align__(16) unsigned char sQ[kWRows * kPitch];
  __shared__ __align__(8) float sNeg[kWRows];  // -lse; -inf: no weight
  __shared__ __align__(8) float sUnit[kWRows];  // a row's power of two, inverted
  constexpr bool kScaled = !__is_same(T, __half);
  __shared__ Walk<kAllRows, kWKeys, kWCost> v;
  __shared__ int sMore;
  const KvCache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, cc = lane & 3;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!divide<kAllRows, kWKeys, kWCost, kWThreads>(a, kWLeast, v)) return;
  __syncthreads();  // every thread has stored the walk's beginning
  for (;;) {
    if (tid == 0) sMore = v.next(a);
    __syncthreads();
    if (!sMore) break;
    const Unit u = v.u;
    const int tile0 = v.tile0, tile1 = v.tile1, rows = u.w * a.G;
    const long end = (long)u.seq + u.w;  // positions the request has
    const int32_t* table = c.tables + (size_t)u.b * c.max_blocks;

    // ---- keys of a tile: the block looked up two tiles ahead, its rows one (two:
    // 79.5 us for the case above instead of 74)
    struct Keys {
      uint4 row[2 * U];
      float scale;
      int blk;
    } keys;
    int blk = -1;
    auto lookup = [&](int tile) {
      const unsigned x = (unsigned)tile * kWWarps + warp;  // group of 16 keys
      blk = tile < tile1 && (long)x * 16 < end ? table[col16(a, x)] : -1;
    };
    auto fetch = [&](int tile) {
      keys.blk = blk < c.num_blocks ? blk : -1;
      keys.scale = 0.f;
      if (keys.blk >= 0) {
        const unsigned x = (unsigned)tile * kWWarps + warp;
        const uint8_t* kp = c.pool + c.row(keys.blk, 0, u.h, (int)(x - col16(a, x) * (c.tpb / 16)) * 16);
        keys.scale = c.scales[c.scale_at(keys.blk, 0, u.h)];
#pragma unroll
        for (int y = 0; y < U; ++y) {
          keys.row[2 * y] = reinterpret_cast<const uint4*>(kp + g * D)[cc + 4 * y];
          keys.row[2 * y + 1] = reinterpret_cast<const uint4*>(kp + (g + 8) * D)[cc + 4 * y];
        }
      }
      lookup(tile + 1);
    };
    lookup(tile0);

    // ---- the rows, once for all tiles
    constexpr int V = 2 * D / 16;  // 16-byte vectors of a row
    for (int x = tid; x < kWRows * V; x += kWThreads) {
      const int r = x / V, at = x % V;
      uint4 q = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const int i = (unsigned)r / (unsigned)a.G, head = u.h * a.G + r - i * a.G;
        q = reinterpret_cast<const uint4*>(a.q + 2 * (u.b * a.qb + i * a.qt + head * a.qh))[at];
      }
      if constexpr (kScaled) {  // V lanes hold a row
        uint32_t* w = &q.x;
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = as_float2(w[e], (T*)nullptr);
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
#pragma unroll
        for (int d = 1; d < V; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        int e2;
        frexpf(top, &e2);  // top < 2^e2
        const int up = top > 0.f && top < INFINITY ? min(15 - e2, 126) : 0;
        const float f = ldexpf(1.f, up);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 y = as_float2(w[e], (T*)nullptr);
          w[e] = half2_of(y.x * f, y.y * f);
        }
        if (at == 0) sUnit[r] = ldexpf(1.f, -up);
      }
      *reinterpret_cast<uint4*>(sQ + r * kPitch + at * 16) = q;
    }
    float neg = -INFINITY;
    if (tid < rows) {
      const int i = (unsigned)tid / (unsigned)a.G;
      neg = -a.row_lse[((size_t)u.b * a.W + i) * a.Hq + u.h * a.G + tid - i * a.G];
      if (neg == INFINITY) neg = -INFINITY;
    }
    if (tid < kWRows) sNeg[tid] = neg;
    fetch(tile0);
    const bool some = __syncthreads_or(tid < rows && neg == -INFINITY);

    for (int tile = tile0; tile < tile1; ++tile) {
      const long t0 = (long)tile * kWKeys + warp * 16;
      // ---- the keys of this warp, as fragments
      uint32_t k[U * 4][4];
      const bool real = keys.blk >= 0;
      const float cs = a.scale * keys.scale;
#pragma unroll
      for (int y = 0; y < U; ++y) {
        const uint4 p = real ? keys.row[2 * y] : make_uint4(0, 0, 0, 0), q = real ? keys.row[2 * y + 1] : make_uint4(0, 0, 0, 0);
        const uint32_t pw[4] = {p.x, p.y, p.z, p.w}, qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          e4m3x4_to_half(pw[x], k[y * 4 + x][0], k[y * 4 + x][2]);
          e4m3x4_to_half(qw[x], k[y * 4 + x][1], k[y * 4 + x][3]);
        }
      }
      fetch(tile + 1);
      const long t = t0 + g + 8 * cc;  // the position that a lane of cc < 2 writes
      const bool mine = cc < 2 && t < end && t < a.T;
      const size_t at = ((size_t)u.b * c.H + u.h) * a.T + t;
      const float old = a.old && mine && t < u.seq ? a.old[at] : 0.f;
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};  // by key, of even and odd rows
      const bool plain = t0 + 15 <= u.seq && !some;  // every row sees every key
      for (int n = 0; n * 8 < rows; ++n) {
        // two chains: fewer roundings add up in each (the case above is off by 0.9e-6
        // instead of 1.2e-6, in the same time)
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int y = 0; y < U; ++y) {
          const uint4* qp = reinterpret_cast<const uint4*>(sQ + (n * 8 + g) * kPitch + (cc + 4 * y) * 32);
          const uint4 p = qp[0], q = qp[1];
          const uint32_t b[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) mma_k16(x & 1 ? s2 : s, k[y * 4 + x], b[2 * x], b[2 * x + 1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += s2[e];
        // element e: key g + 8 (e / 2), row 2 cc + e % 2
        const float2 l = *reinterpret_cast<const float2*>(sNeg + n * 8 + 2 * cc);
        float2 scale = make_float2(cs, cs);
        if constexpr (kScaled) scale = mul2(scale, *reinterpret_cast<const float2*>(sUnit + n * 8 + 2 * cc));
        if (plain && n * 8 + 8 <= rows) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float2 e = mul2(fma2(make_float2(s[2 * x], s[2 * x + 1]), scale, l),
                                  make_float2(kLog2e, kLog2e));
            sum[x] = add2(sum[x], make_float2(ex2(e.x), ex2(e.y)));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float ln = e & 1 ? l.y : l.x, p = ex2(fmaf(s[e], e & 1 ? scale.y : scale.x, ln) * kLog2e);
            // place j of the window is seen from its own token on
            const long since = max(0l, t0 + g + 8 * (e >> 1) - u.seq) * a.G;
            if (n * 8 + 2 * cc + (e & 1) >= since && ln != -INFINITY) (e & 1 ? sum[e >> 1].y : sum[e >> 1].x) += p;
          }
        }
      }
      float total[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        total[x] = sum[x].x + sum[x].y;
        total[x] += __shfl_xor_sync(~0u, total[x], 1);
        total[x] += __shfl_xor_sync(~0u, total[x], 2);
      }
      if (mine) {
        const float x = !real ? NAN : cc ? total[1] : total[0];
        a.sum[at] = a.old && t < u.seq ? fmaf(a.decay, old, x) : x;
      }
    }
    __syncthreads();  // the rows, and the walk, have been read
  }
}

}  // namespace

cudaError_t launch_weigh_rows(const WeighArgs& a, int dtype, cudaStream_t st) {
  if (a.c.D == 64)
    return dtype == SPEC_BF16 ? launch_first(weigh_kernel<__nv_bfloat16, 64>, kWCtas, kWThreads, st, a)
                              : launch_first(weigh_kernel<__half, 64>, kWCtas, kWThreads, st, a);
  return dtype == SPEC_BF16 ? launch_first(weigh_kernel<__nv_bfloat16, 128>, kWCtas, kWThreads, st, a)
                            : launch_first(weigh_kernel<__half, 128>, kWCtas, kWThreads, st, a);
}

namespace {

// Whether this file's kernel serves this many rows per KV head, as many as it
// stages; else weigh_tiles.cu.  8192 positions, 8 KV heads of 64 and of 128, 32 rows:
// 1 request 10 us here and 11 there, 12 and 12; 16 requests 43 and 70, 49 and 90; 64
// requests 126 and 251, 165 and 336; with fewer rows, and over 1000 positions, it is
// ahead by more.  With 64 rows 16 requests (heads of 128) took 77 here, if twice the
// rows are staged (which slows the case above to 80), and 79 there.
bool few_rows(int W, int G) { return (long)W * G <= kWRows; }

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_weigh_scratch_size(int B, int W, int q_heads, int kv_heads, int head_dim) {
  if (B < 1 || B > SPEC_MAX_BATCH || W < 1 || W > SPEC_MAX_WINDOW || kv_heads < 1 || kv_heads > 1024 ||
      q_heads < 1 || q_heads > 16384 || q_heads % kv_heads != 0 || (head_dim != 64 && head_dim != 128))
    return 0;
  return few_rows(W, q_heads / kv_heads) ? 256 : weigh_tiles_scratch();
}

int spec_weigh_kv(const spec_kv_cache* cache, const spec_weigh_params* p, void* scratch, size_t scratch_bytes,
                  spec_stream_t stream) {
  constexpr double kLog2e = 1.4426950408889634073599246810019;
  WeighArgs a{};
  const int rc = kv_setup(cache, &a.c);
  if (rc != SPEC_OK) return rc;
  if (!p || p->size != sizeof(spec_weigh_params) || !kv_strides_ok(p->q, p->q_strides) ||
      (p->dtype != SPEC_BF16 && p->dtype != SPEC_F16) || !p->seq_lens || !p->lse || !p->out || p->T < 1 ||
      !isfinite((float)(p->scale * kLog2e)) || !isfinite(p->decay) ||
      (long)a.c.max_blocks * a.c.tpb > kMaxPositions || (long)p->B * p->W * p->q_heads > kMaxRows)
    return SPEC_EINVAL;
  const size_t need = spec_weigh_scratch_size(p->B, p->W, p->q_heads, a.c.H, a.c.D);
  if (need == 0) return SPEC_EINVAL;
  if (!scratch || reinterpret_cast<uintptr_t>(scratch) % 256 != 0 || scratch_bytes < need) return SPEC_EWORKSPACE;
  const long B = p->B, weights = B * a.c.H * p->T * sizeof(float);
  Arrays x;
  const int old = x.read(dense(p->weights, weights));
  x.read(strided(p->q, p->q_strides, p->B, p->W, p->q_heads, a.c.D, 2));
  x.read(dense(p->lse, B * p->W * p->q_heads * sizeof(float)));
  x.read(dense(p->seq_lens, B * sizeof(int32_t)));
  x.read(dense(p->window_lens, B * sizeof(int32_t)));
  cache_arrays(a.c, p->B, false, &x);
  x.write(dense(p->out, weights), old);
  x.write(dense(scratch, need));
  if (!x.apart()) return SPEC_EINVAL;
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
  a.mtiles = 1;
  a.tpb16_div = (unsigned)((1ull << 32) / (a.c.tpb / 16) + ((1ull << 32) % (a.c.tpb / 16) != 0));
  a.row_lse = p->lse;
  a.scale = p->scale;
  a.old = p->weights;
  a.decay = p->decay;
  a.sum = p->out;
  a.T = p->T;
  const cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = few_rows(a.W, a.G) ? launch_weigh_rows(a, p->dtype, st)
                                           : launch_weigh_tiles(a, p->dtype, scratch, st);
  return e == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}

}  // extern "C"

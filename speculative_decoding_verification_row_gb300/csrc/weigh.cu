// The attention that each cached position drew from a window's rows
// (spec_weigh_kv).
//
// Tensor cores through mma.sync m16n8k16, the keys as the left operand: a
// warp holds 16 keys in registers, converted from e4m3 once, and lets the
// rows pass; each lane adds up the weights of its two keys, so that the sum
// over rows needs four shuffles per tile and no atomics.  e4m3 -> bf16 and
// fp16 is exact, so the products are those of the stored values; a weight is
// exp of a score less the row's lse, at most 1 but for rounding.
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
constexpr int kWRows = 64;            // rows staged at a time
constexpr int kWCost = 2;             // cells of a unit besides its tiles
constexpr int kWLeast = 4;            // cells below which a share is not worth a CTA
constexpr int kWCtas = 4 * kSms;

__device__ __forceinline__ void mma_k16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half*) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_k16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                        __nv_bfloat16*) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <class T, int D>
__global__ void __launch_bounds__(kWThreads, 4) weigh_kernel(const WeighArgs a) {
  constexpr int U = D / 64;              // 16-byte chunks of a key per thread
  constexpr int kPitch = 2 * D + 16;     // bytes of a staged row: its 16-byte reads hit all banks once
  __shared__ __align__(16) unsigned char sQ[kWRows * kPitch];
  __shared__ float sLse[kWRows];
  __shared__ Walk<kAllRows, kWKeys, kWCost> v;
  __shared__ int sMore;
  const KvCache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, cc = lane & 3;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!divide<kAllRows, kWKeys, kWCost, kWThreads>(a, kWLeast, v)) return;
  __syncthreads();  // every thread has stored the walk's beginning
  const int tpb16 = c.tpb / 16;
  for (;;) {
    if (tid == 0) sMore = v.next(a);
    __syncthreads();
    if (!sMore) break;
    const Unit u = v.u;
    const int tile0 = v.tile0, tile1 = v.tile1;
    __syncthreads();  // the walk has been read
    const int rows = u.w * a.G, chunks = (rows + kWRows - 1) / kWRows;
    const long end = (long)u.seq + u.w;  // positions the request has
    const int32_t* table = c.tables + (size_t)u.b * c.max_blocks;
    auto stage = [&](int chunk) {
      constexpr int V = 2 * D / 16;  // 16-byte vectors of a row
      __syncthreads();
      for (int x = tid; x < kWRows * V; x += kWThreads) {
        const int r = x / V, at = x % V, row = chunk * kWRows + r;
        uint4 q = make_uint4(0, 0, 0, 0);
        if (row < rows) {
          const int i = row / a.G, head = u.h * a.G + row % a.G;
          q = reinterpret_cast<const uint4*>(a.q + 2 * (u.b * a.qb + i * a.qt + head * a.qh))[at];
        }
        *reinterpret_cast<uint4*>(sQ + r * kPitch + at * 16) = q;
      }
      for (int r = tid; r < kWRows; r += kWThreads) {
        const int row = chunk * kWRows + r;
        float l = INFINITY;  // no weight
        if (row < rows) {
          l = a.row_lse[((size_t)u.b * a.W + row / a.G) * a.Hq + u.h * a.G + row % a.G];
          if (l == -INFINITY) l = INFINITY;
        }
        sLse[r] = l;
      }
      __syncthreads();
    };
    if (chunks == 1) stage(0);
    for (int tile = tile0; tile < tile1; ++tile) {
      const long t0 = (long)tile * kWKeys + warp * 16;
      const int col16 = tile * kWWarps + warp;
      int blk = t0 < end ? table[col16 / tpb16] : -1;
      if (blk >= c.num_blocks) blk = -1;
      // ---- the keys of this warp, as fragments
      uint32_t k[U * 4][4];
      float cs = 0.f;
      if (blk >= 0) {
        const uint8_t* kp = c.pool + c.row(blk, 0, u.h, col16 % tpb16 * 16);
        cs = a.scale * c.scales[c.scale_at(blk, 0, u.h)];
#pragma unroll
        for (int y = 0; y < U; ++y) {
          const uint4 p = reinterpret_cast<const uint4*>(kp + (size_t)g * D)[cc + 4 * y];
          const uint4 q = reinterpret_cast<const uint4*>(kp + (size_t)(g + 8) * D)[cc + 4 * y];
          const uint32_t pw[4] = {p.x, p.y, p.z, p.w}, qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            e4m3x4_to(pw[x], k[y * 4 + x][0], k[y * 4 + x][2], (T*)nullptr);
            e4m3x4_to(qw[x], k[y * 4 + x][1], k[y * 4 + x][3], (T*)nullptr);
          }
        }
      } else {
#pragma unroll
        for (int x = 0; x < U * 4; ++x) k[x][0] = k[x][1] = k[x][2] = k[x][3] = 0;
      }
      // the first row that sees the lane's keys: place j of the window is seen from its own token on
      long from[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) from[x] = max(0l, t0 + g + 8 * x - u.seq) * a.G;
      const long first = max(0l, t0 - u.seq) * a.G;  // of the warp's keys
      float sum[2] = {0.f, 0.f};
      for (int chunk = (int)(max(0l, (long)tile * kWKeys - u.seq) * a.G / kWRows); chunk < chunks; ++chunk) {
        if (chunks > 1) stage(chunk);
        float part[2] = {0.f, 0.f};  // a chunk's sum on its own: fewer roundings on the way
        for (int n = 0; n < kWRows / 8; ++n) {
          const int row = chunk * kWRows + n * 8;
          if (row >= rows) break;
          if (row + 8 <= first) continue;
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int y = 0; y < U; ++y) {
            const uint4* qp = reinterpret_cast<const uint4*>(sQ + (n * 8 + g) * kPitch + (cc + 4 * y) * 32);
            const uint4 p = qp[0], q = qp[1];
            const uint32_t b[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) mma_k16(s, k[y * 4 + x], b[2 * x], b[2 * x + 1], (T*)nullptr);
          }
          // element e: key g + 8 (e / 2), row 2 cc + e % 2
          const float2 l = *reinterpret_cast<const float2*>(sLse + n * 8 + 2 * cc);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float le = e & 1 ? l.y : l.x;
            const float p = ex2(fmaf(s[e], cs, -le) * 1.4426950408889634f);
            if (row + 2 * cc + (e & 1) >= from[e >> 1] && le != INFINITY) part[e >> 1] += p;
          }
        }
        sum[0] += part[0], sum[1] += part[1];
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        sum[x] += __shfl_xor_sync(~0u, sum[x], 1);
        sum[x] += __shfl_xor_sync(~0u, sum[x], 2);
      }
      const long t = t0 + g + 8 * cc;
      if (cc < 2 && t < end && t < a.T) {
        const size_t at = ((size_t)u.b * c.H + u.h) * a.T + t;
        float x = blk < 0 ? NAN : cc ? sum[1] : sum[0];
        if (a.old && t < u.seq) x = fmaf(a.decay, a.old[at], x);
        a.sum[at] = x;
      }
    }
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

// Whether this file's kernel serves this many rows per KV head; else weigh_tiles.cu.
bool few_rows(int W, int G) { return (long)W * G <= 32; }

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

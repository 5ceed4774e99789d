// The quantising store of a window's K and V rows into the paged 8-bit cache
// (spec_store_kv), and the relocation of accepted rows there
// (spec_relocate_quantised_kv).
//
// Why powers of two: e4m3 is a floating-point format, so the scale decides
// the range only, not the relative precision; with a power of two x / s and
// the re-rounding of codes to a larger scale are exact but for the codes that
// fall below the normal range (2^-6 s), and the consumers' products with the
// scales are exact as well.
//
// At a step's sizes both are bound by latency: table -> rows -> maximum ->
// codes.  In a graph (operands in L2) the store of 64 requests of 8 tokens, 8
// heads of 128 takes 4.6 us (4.2 with 1 to 8 tokens each), that of 4 prompts of
// 4001 tokens, 4 heads of 64, 7.2 us (of one beside three windows of 5 to 15
// tokens, 5.7); 64 prompts of 4096 tokens with 8 heads of 128, 276 us, 5.8 TB/s
// (0.86 of the measured copy rate).  The relocation of 16 requests' paths of 4 takes 3.9 us, of 256
// requests' paths of 17 7.2 us.
#include "kvcache.cuh"

namespace sv {

namespace {

struct StoreArgs {
  KvCache c;
  const char* x[2];
  long sb[2], st[2], sh[2];  // strides in elements
  const int32_t* seq;
  const int32_t* win;
  int B, W, pages;
  int split;  // CTAs per block of a request's window
};

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

// Largest finite magnitude of eight packed elements.
template <class T>
__device__ __forceinline__ float amax8(uint4 v, float m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<T>(w[i]);
    const float a = fabsf(f.x), b = fabsf(f.y);
    m = fmaxf(m, a < INFINITY ? a : 0.f);  // false for NaN too
    m = fmaxf(m, b < INFINITY ? b : 0.f);
  }
  return m;
}

template <class T>
__device__ __forceinline__ uint2 quant8(uint4 v, float r) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<T>(w[i]);
    q[i] = to_e4m3x2(f.x * r, f.y * r);
  }
  return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

constexpr int kStoreThreads = 128;

// A unit is one block of one request's window, one kind, one head: the
// largest magnitude of the new rows, the scale, the codes.  WARPS warps serve
// it (1, or the CTA's 4) and a CTA takes (kind, head) pairs of one block: one
// round of them in a small call, all in a large one, so that the window's
// blocks are checked once.  The rows stay in registers between the passes, VECS 16-byte vectors
// a lane; what a larger block holds beyond that is read again (from L2).  With
// the CTA per unit 9 CTAs share an SM (56 registers; 80 and 6 without the
// bound: 333 us instead of 300 with blocks of 64 tokens).
template <class T, int WARPS, int VECS>
__global__ void __launch_bounds__(kStoreThreads, WARPS > 1 ? 9 : 0) store_kernel(const StoreArgs a) {
  constexpr int kUnits = kStoreThreads / 32 / WARPS, kLanes = 32 * WARPS;
  const KvCache& c = a.c;
  const int groups = (2 * c.H + kUnits - 1) / kUnits;
  int u = blockIdx.x;
  const int group0 = u % a.split;
  u /= a.split;
  const int page = u % a.pages, b = u / a.pages;
  const long seq = a.seq[b];
  const int w = a.win ? a.win[b] : a.W;
  if (seq < 0 || w < 1 || w > a.W) return;
  const long col = seq / c.tpb + page;      // block table column
  const int last = (int)((seq + w - 1) / c.tpb);
  if (col > last || last >= c.max_blocks) return;
  __shared__ float sMax[kStoreThreads / 32];
  const int32_t* table = c.tables + (size_t)b * c.max_blocks;
  const int blk = table[col];
  const bool mapped = blk >= 0 && blk < c.num_blocks;
  const int lane = threadIdx.x % kLanes;
  const int first = page == 0 ? (int)(seq % c.tpb) : 0;  // first row written
  const int i0 = (int)(col * c.tpb + first - seq);        // its window token
  const int rows = min(c.tpb - first, w - i0);
  const int vpr = c.D / 8, shift = c.D == 128 ? 4 : 3;    // vectors per row: 16 or 8
#pragma unroll 1
  for (int group = group0; group < groups; group += a.split) {
    const int unit = group * kUnits + (int)threadIdx.x / kLanes;  // kind * H + h
    const bool real = unit < 2 * c.H;
    const int kind = real && unit >= c.H, h = real ? unit - kind * c.H : 0;
    const int nvec = real ? rows * vpr : 0;
    const char* src = a.x[kind] + 2 * (b * a.sb[kind] + i0 * a.st[kind] + h * a.sh[kind]);
    auto vec = [&](int v) {
      return *reinterpret_cast<const uint4*>(src + 2 * ((v >> shift) * a.st[kind] + (v & (vpr - 1)) * 8));
    };
    uint4 keep[VECS];
    float amax = 0.f;
#pragma unroll
    for (int q = 0; q < VECS; ++q) {
      const int v = lane + q * kLanes;
      if (v < nvec) keep[q] = vec(v);
    }
    // the old scale comes while the rows do
    float* ps = c.scales + c.scale_at(mapped ? blk : 0, kind, h);
    const float old = first > 0 ? *ps : 0.f;
    // every CTA of the request checks all of its window's blocks, so they agree
    int bad = 0;
    if (group == group0)
      for (int i = (int)(seq / c.tpb) + threadIdx.x; i <= last; i += kStoreThreads)
        bad |= table[i] < 0 || table[i] >= c.num_blocks;
#pragma unroll
    for (int q = 0; q < VECS; ++q)
      if (lane + q * kLanes < nvec) amax = amax8<T>(keep[q], amax);
    for (int v = lane + VECS * kLanes; v < nvec; v += kLanes) amax = amax8<T>(vec(v), amax);
#pragma unroll
    for (int d = 16; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, d));
    if (WARPS > 1 && (threadIdx.x & 31) == 0) sMax[threadIdx.x >> 5] = amax;
    if (__syncthreads_or(bad)) return;  // also: every warp has read the old scale
    if (!real) continue;
    if (WARPS > 1) {
#pragma unroll
      for (int i = 0; i < kStoreThreads / 32; ++i) amax = fmaxf(amax, sMax[i]);
    }
    float scale = scale_for(amax);
    uint8_t* dst = c.pool + c.row(blk, kind, h, 0);
    if (first > 0) {
      if (old >= scale) {
        scale = old;
      } else {  // the live rows move to the larger scale
        const float r = scale_ratio(old, scale);
        for (int v = lane; v < first * c.D / 16; v += kLanes) {
          uint4* p = reinterpret_cast<uint4*>(dst) + v;
          *p = rescale_e4m3x16(*p, r);
        }
      }
    }
    if (lane == 0) *ps = scale;
    const float inv = scale_ratio(1.f, scale);
    uint2* out = reinterpret_cast<uint2*>(dst + (size_t)first * c.D);
#pragma unroll
    for (int q = 0; q < VECS; ++q) {
      const int v = lane + q * kLanes;
      if (v < nvec) out[v] = quant8<T>(keep[q], inv);
    }
    for (int v = lane + VECS * kLanes; v < nvec; v += kLanes) out[v] = quant8<T>(vec(v), inv);
    if (WARPS > 1) break;  // such CTAs take one unit each
  }
}

struct MoveArgs {
  KvCache c;
  const int32_t* base;
  const int32_t* nodes;
  const int32_t* num_accepted;
  int B, L;
};

constexpr int kMoveWarps = 4;

// One warp = one request, kind and head; lane j holds what row j (and row
// j + 32) needs.  Nodes increase strictly from the root, so node_j >= j: a
// row is never written before a later row of the path has been read, as long
// as every batch loads before it stores and the batches go in increasing j.
__global__ void __launch_bounds__(kMoveWarps * 32) move_kernel(const MoveArgs a) {
  const KvCache& c = a.c;
  const int lane = threadIdx.x & 31;
  const long u = (long)blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
  if (u >= (long)a.B * 2 * c.H) return;
  const int h = (int)(u % c.H), kind = (int)(u / c.H & 1), b = (int)(u / c.H / 2);
  const int n = a.num_accepted[b];
  if (n <= 0 || n >= a.L) return;
  const int32_t* nodes = a.nodes + (size_t)b * a.L;
  const long base = a.base[b];
  // rows j = lane + 1 and lane + 33 of the path: source and target blocks
  int src[2], dst[2];
  float had[2];
  bool ok = nodes[0] == 0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int j = lane + 1 + 32 * q;
    src[q] = dst[q] = -1;
    had[q] = 0.f;
    if (j <= n) {
      const int nd = nodes[j];
      src[q] = c.block(b, base + nd);
      dst[q] = c.block(b, base + j);
      ok = ok && nd > nodes[j - 1] && src[q] >= 0 && dst[q] >= 0;
      if (ok) had[q] = c.scales[c.scale_at(src[q], kind, h)];
    }
  }
  if (!__all_sync(~0u, ok)) return;
  __syncwarp();  // every source scale has been read
  // the blocks written to: their largest scale among the rows they receive
  const long p0 = (base + 1) / c.tpb, p1 = (base + n) / c.tpb;
  const int off0 = (int)((base + 1) % c.tpb);
  float now[2] = {0.f, 0.f};  // the new scale of the rows' target blocks
  for (long p = p0; p <= p1; ++p) {
    float m = 0.f;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int j = lane + 1 + 32 * q;
      if (j <= n && (base + j) / c.tpb == p) m = fmaxf(m, had[q]);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
    const int blk = c.block(b, p * c.tpb);
    float* ps = c.scales + c.scale_at(blk, kind, h);
    if (p == p0 && off0 > 0) {
      const float old = *ps;
      if (old >= m) {
        m = old;
      } else {
        const float r = scale_ratio(old, m);
        uint4* row = reinterpret_cast<uint4*>(c.pool + c.row(blk, kind, h, 0));
        for (int v = lane; v < off0 * c.D / 16; v += 32) row[v] = rescale_e4m3x16(row[v], r);
      }
    }
    __syncwarp();
    if (lane == 0) *ps = m;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int j = lane + 1 + 32 * q;
      if (j <= n && (base + j) / c.tpb == p) now[q] = m;
    }
  }
  // the rows, 16 bytes per lane, several rows at a time
  const int vpr = c.D / 16, per = 32 / vpr;
  for (int j0 = 1; j0 <= n; j0 += per) {
    const int j = j0 + lane / vpr;
    const int from = (j - 1) & 31;
    const bool hi = j > 32;
    const int s0 = __shfl_sync(~0u, src[0], from), s1 = __shfl_sync(~0u, src[1], from);
    const int d0 = __shfl_sync(~0u, dst[0], from), d1 = __shfl_sync(~0u, dst[1], from);
    const float h0 = __shfl_sync(~0u, had[0], from), h1 = __shfl_sync(~0u, had[1], from);
    const float n0 = __shfl_sync(~0u, now[0], from), n1 = __shfl_sync(~0u, now[1], from);
    const float was = hi ? h1 : h0, is = hi ? n1 : n0;
    const bool move = j <= n && (nodes[j <= n ? j : 0] != j || was != is);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (move)
      v = reinterpret_cast<const uint4*>(
          c.pool + c.row(hi ? s1 : s0, kind, h, (int)((base + nodes[j]) % c.tpb)))[lane % vpr];
    __syncwarp();
    if (move) {
      if (was != is) v = rescale_e4m3x16(v, scale_ratio(was, is));
      reinterpret_cast<uint4*>(
          c.pool + c.row(hi ? d1 : d0, kind, h, (int)((base + j) % c.tpb)))[lane % vpr] = v;
    }
    __syncwarp();
  }
}

// CTAs above which one takes all of a block's units (a warp per unit): some
// eight times those that fit the GPU.  64 prompts of 4096 tokens, 8 heads of
// 128: 282 us instead of 417 with blocks of 16 tokens, 280 instead of 291 with
// 32; with the CTA per unit (64 tokens) it is the other way, 300 and 293.
constexpr long kStoreMany = 8l * 152 * 8;

template <class T, int WARPS, int VECS>
int launch_store_as(StoreArgs& a, cudaStream_t st) {
  const long blocks = (long)a.B * a.pages;
  const int groups = ceil_div(2 * a.c.H, kStoreThreads / 32 / WARPS);
  a.split = WARPS == 1 && blocks * groups > kStoreMany ? 1 : groups;
  if (blocks * a.split > INT_MAX) return SPEC_EINVAL;
  store_kernel<T, WARPS, VECS><<<(unsigned)(blocks * a.split), kStoreThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}

// A warp per unit while a block's new rows fit its registers, else the CTA.
// (The CTA for all took 814 us with blocks of 16 tokens and 491 with 32; and
// 105 us for 2048 requests of 4 tokens, now 23.)
template <class T>
int launch_store(StoreArgs& a, cudaStream_t st) {
  const int vecs = min(a.c.tpb, a.W) * a.c.D / 8;
  if (vecs <= 32 * 4) return launch_store_as<T, 1, 4>(a, st);
  if (vecs <= 32 * 8) return launch_store_as<T, 1, 8>(a, st);
  if (vecs <= 32 * 16) return launch_store_as<T, 1, 16>(a, st);
  return launch_store_as<T, 4, 8>(a, st);
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" {

int spec_store_kv(const spec_kv_cache* cache, const void* k, const int64_t* k_strides,
                  const void* v, const int64_t* v_strides, int dtype, const int32_t* seq_lens,
                  const int32_t* window_lens, int B, int W, spec_stream_t stream) {
  StoreArgs a{};
  const int rc = kv_setup(cache, &a.c);
  if (rc != SPEC_OK) return rc;
  if (!kv_strides_ok(k, k_strides) || !kv_strides_ok(v, v_strides) || !seq_lens ||
      (dtype != SPEC_BF16 && dtype != SPEC_F16) || B < 1 || B > SPEC_MAX_BATCH || W < 1 ||
      W > SPEC_MAX_WINDOW)
    return SPEC_EINVAL;
  const void* x[2] = {k, v};
  const int64_t* st[2] = {k_strides, v_strides};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = static_cast<const char*>(x[i]);
    a.sb[i] = st[i][0];
    a.st[i] = st[i][1];
    a.sh[i] = st[i][2];
  }
  a.seq = seq_lens;
  a.win = window_lens;
  a.B = B;
  a.W = W;
  // blocks a window can touch; at most the whole table row
  a.pages = min((W - 2 + a.c.tpb) / a.c.tpb + 1, a.c.max_blocks);
  return dtype == SPEC_BF16 ? launch_store<__nv_bfloat16>(a, (cudaStream_t)stream)
                            : launch_store<__half>(a, (cudaStream_t)stream);
}

int spec_relocate_quantised_kv(const spec_kv_cache* cache, const int32_t* base_lens,
                               const int32_t* accepted_nodes, const int32_t* num_accepted, int B,
                               int L, spec_stream_t stream) {
  MoveArgs a{};
  const int rc = kv_setup(cache, &a.c);
  if (rc != SPEC_OK) return rc;
  if (!base_lens || !accepted_nodes || !num_accepted || B < 1 || B > SPEC_MAX_BATCH || L < 1 ||
      L > SPEC_MAX_PATH_LEN)
    return SPEC_EINVAL;
  a.base = base_lens;
  a.nodes = accepted_nodes;
  a.num_accepted = num_accepted;
  a.B = B;
  a.L = L;
  const long grid = ((long)B * 2 * a.c.H + kMoveWarps - 1) / kMoveWarps;
  move_kernel<<<(unsigned)grid, kMoveWarps * 32, 0, (cudaStream_t)stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}

}  // extern "C"

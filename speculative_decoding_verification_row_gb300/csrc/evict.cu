// Eviction from the 8-bit cache by weight (spec_evict_kv): a selection per
// request and KV head, then the kept rows' move.
//
// Selection: one CTA finds the weight of the last position kept with a radix
// selection over the weights' order keys (11, 11 and 10 bits), and writes the
// kept positions in order in one more pass; equal weights are taken from the
// front.
//
// Move: one CTA per request, KV head and kind.  A kept row never moves up, so
// rows are gathered in order, group by group: all of a group is read before any
// of it is written, and what is written lies below every row still to be read.
#include "kvcache.cuh"

namespace sv {

namespace {

struct EvictArgs {
  KvCache c;
  const float* weights;
  const int32_t* seq;
  const int32_t* held;
  int32_t* new_lens;
  int32_t* kept;
  float* out_weights;
  int32_t* free_blocks;
  int B, T, T_out, keep, first, recent;
};

constexpr int kPickThreads = 1024;
constexpr int kBins = 2048;

// Order key of a weight: NaN below all, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float x) { return x == x ? ord32(x) : 0u; }

// Exclusive sum over the CTA of two small counts of a warp, packed in 16 bits
// each; *total: their sum over all warps.
__device__ __forceinline__ uint32_t before_warp(uint32_t mine, uint32_t* sWarp, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) sWarp[warp] = mine;
  __syncthreads();
  uint32_t x = lane < kPickThreads / 32 ? sWarp[lane] : 0u;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x += y;
  }
  *total = __shfl_sync(~0u, x, 31);
  const uint32_t upto = __shfl_sync(~0u, x, warp);
  __syncthreads();  // sWarp may be written again
  return upto - mine;
}

__global__ void __launch_bounds__(kPickThreads) pick_kernel(const EvictArgs a) {
  __shared__ int sHist[kBins];
  __shared__ uint32_t sWarp[kPickThreads / 32];
  __shared__ int sBin, sAbove;
  const KvCache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = blockIdx.x / c.H;
  const int n = a.seq[b];
  int32_t* kept = a.kept + (size_t)blockIdx.x * a.keep;
  const float* w = a.weights + (size_t)blockIdx.x * a.T;
  float* out = a.out_weights + (size_t)blockIdx.x * a.T_out;
  int bad = n < 0 || n > a.T || (long)n > (long)c.max_blocks * c.tpb;
  if (!bad) {
    const int32_t* table = c.tables + (size_t)b * c.max_blocks;
    for (int i = tid; (long)i * c.tpb < n; i += kPickThreads) bad |= table[i] < 0 || table[i] >= c.num_blocks;
  }
  bad = __syncthreads_or(bad);
  if (bad || n <= a.keep) {
    for (int j = tid; j < a.keep; j += kPickThreads) {
      const bool real = !bad && j < n;
      kept[j] = real ? j : -1;
      if (real) out[j] = w[j];
    }
    return;
  }
  const int lo = a.first, hi = n - a.recent;  // the positions that may go: [lo, hi)
  const int want = a.keep - a.first - a.recent;
  // ---- the key of the last one kept, and how many of that key
  uint32_t top = 0xffffffffu;  // nothing reaches it: NaN has key 0, every number less
  int ties = 0;
  if (want > 0) {
    uint32_t prefix = 0, known = 0;
    int left = want;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass < 2 ? kBins : kBins / 2;
      for (int i = tid; i < kBins; i += kPickThreads) sHist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int t = lo + tid; t < hi; t += kPickThreads) {
        const uint32_t k = weight_key(w[t]);
        if ((k & known) == prefix) atomicAdd(&sHist[k >> shift & (bins - 1)], 1);
      }
      __syncthreads();
      // the highest bin whose sum from the top reaches `left`: two bins a thread, from the top
      const int b0 = bins - 1 - 2 * tid;
      const int h0 = b0 >= 0 ? sHist[b0] : 0, h1 = b0 >= 1 ? sHist[b0 - 1] : 0;
      int incl = h0 + h1;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(~0u, incl, d);
        if (lane >= d) incl += y;
      }
      if (lane == 31) sWarp[warp] = (uint32_t)incl;
      __syncthreads();
      int above = incl - h0 - h1;
      for (int i = 0; i < warp; ++i) above += (int)sWarp[i];
      if (above < left && left <= above + h0) sBin = b0, sAbove = above;
      if (above + h0 < left && left <= above + h0 + h1) sBin = b0 - 1, sAbove = above + h0;
      __syncthreads();
      prefix |= (uint32_t)sBin << shift;
      known |= (uint32_t)(bins - 1) << shift;
      left -= sAbove;
      __syncthreads();
    }
    top = prefix;
    ties = left;
  }
  // ---- the kept positions in order
  int before = 0, equal = 0;  // kept without the ties, and ties, of the tiles before
  for (int t0 = 0; t0 < n; t0 += kPickThreads) {
    const int t = t0 + tid;
    const float x = t < n ? w[t] : 0.f;
    const bool must = t < n && (t < lo || t >= hi);
    const bool may = t >= lo && t < hi;
    const uint32_t k = weight_key(x);
    const bool above = must || (may && want > 0 && k > top), tie = may && want > 0 && k == top;
    const unsigned am = __ballot_sync(~0u, above), tm = __ballot_sync(~0u, tie);
    uint32_t total;
    const uint32_t pre = before_warp((uint32_t)__popc(am) << 16 | (uint32_t)__popc(tm), sWarp, &total);
    const unsigned mask = (1u << lane) - 1;
    const int at = before + (int)(pre >> 16) + __popc(am & mask);
    const int tied = equal + (int)(pre & 0xffffu) + __popc(tm & mask);
    if (above || (tie && tied < ties)) {  // every weight of the tile has been read
      const int j = at + min(tied, ties);
      kept[j] = t;
      out[j] = x;
    }
    before += (int)(total >> 16);
    equal += (int)(total & 0xffffu);
  }
}

constexpr int kGatherThreads = 512;
constexpr int kGatherRows = 512;  // rows read before any of them is written
constexpr int kMostRows = 1024;   // rows of a group: whole blocks, at least one

template <int D>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const EvictArgs a) {
  constexpr int V = D / 16;                                // 16-byte vectors of a row
  constexpr int N = kGatherRows * V / kGatherThreads;      // of a thread and batch
  __shared__ int2 sFrom[kMostRows];                        // a row's block and place in it
  __shared__ float sHad[kMostRows];                        // that block's scale
  __shared__ int sNew[kMostRows / 16];                     // the scales of the blocks written, as bits
  const KvCache& c = a.c;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int kind = blockIdx.x & 1, h = (blockIdx.x >> 1) % c.H, b = (blockIdx.x >> 1) / c.H;
  const int32_t* kept = a.kept + ((size_t)b * c.H + h) * a.keep;
  const int last = kept[a.keep - 1];
  if (kind == 0 && h == 0 && tid == 0) {
    const int n = a.seq[b], now = last >= 0 ? a.keep : n;
    if (a.free_blocks) {
      const bool ok = n == 0 || kept[0] >= 0;
      a.free_blocks[b] = ok ? max(0, a.held[b] - (int)(((long)now + c.tpb - 1) / c.tpb)) : 0;
    }
    a.new_lens[b] = now;
  }
  if (last < a.keep) return;  // at most `keep` positions: nothing moves
  const int32_t* table = c.tables + (size_t)b * c.max_blocks;
  const int group = c.tpb <= kGatherRows ? kGatherRows / c.tpb * c.tpb : c.tpb;
  for (int j0 = 0; j0 < a.keep; j0 += group) {
    const int rows = min(group, a.keep - j0);
    for (int i = tid; i < kMostRows / 16; i += kGatherThreads) sNew[i] = 0;
    __syncthreads();
    for (int r = tid; r < rows; r += kGatherThreads) {
      const int t = kept[j0 + r], col = t / c.tpb;
      const int blk = table[col];
      const float s = c.scales[c.scale_at(blk, kind, h)];
      sFrom[r] = make_int2(blk, t - col * c.tpb);
      sHad[r] = s;
      atomicMax(&sNew[r / c.tpb], __float_as_int(s));  // scales are >= 0: ordered as integers
    }
    __syncthreads();
    for (int r0 = 0; r0 < rows; r0 += kGatherRows) {
      uint4 x[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int v = tid + k * kGatherThreads, r = r0 + v / V;
        if (r < rows) {
          const int2 f = sFrom[r];
          x[k] = reinterpret_cast<const uint4*>(c.pool + c.row(f.x, kind, h, f.y))[v % V];
        }
      }
      __syncthreads();  // all of the batch has been read
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int v = tid + k * kGatherThreads, r = r0 + v / V;
        if (r < rows) {
          const float was = sHad[r], is = __int_as_float(sNew[r / c.tpb]);
          if (was != is) x[k] = rescale_e4m3x16(x[k], scale_ratio(was, is));
          const int j = j0 + r, col = j / c.tpb;
          reinterpret_cast<uint4*>(c.pool + c.row(table[col], kind, h, j - col * c.tpb))[v % V] = x[k];
        }
      }
    }
    for (int i = tid; i * c.tpb < rows; i += kGatherThreads)
      c.scales[c.scale_at(table[j0 / c.tpb + i], kind, h)] = __int_as_float(sNew[i]);
    __syncthreads();
  }
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" int spec_evict_kv(const spec_kv_cache* cache, const spec_evict_params* p, spec_stream_t stream) {
  EvictArgs a{};
  const int rc = kv_setup(cache, &a.c);
  if (rc != SPEC_OK) return rc;
  if (!p || p->size != sizeof(spec_evict_params) || !p->weights || !p->seq_lens || !p->new_lens || !p->kept ||
      !p->out_weights || p->B < 1 || p->B > SPEC_MAX_BATCH || p->T < 1 || p->keep < 1 || p->keep > 1 << 30 ||
      p->first < 0 || p->recent < 0 || (long)p->first + p->recent > p->keep || p->T_out < p->keep ||
      (p->out_weights == p->weights && p->T_out != p->T) || !p->blocks_held != !p->free_blocks ||
      (long)a.c.max_blocks * a.c.tpb > 1l << 30)
    return SPEC_EINVAL;
  a.weights = p->weights;
  a.seq = p->seq_lens;
  a.held = p->blocks_held;
  a.new_lens = p->new_lens;
  a.kept = p->kept;
  a.out_weights = p->out_weights;
  a.free_blocks = p->free_blocks;
  a.B = p->B;
  a.T = p->T;
  a.T_out = p->T_out;
  a.keep = p->keep;
  a.first = p->first;
  a.recent = p->recent;
  const cudaStream_t st = (cudaStream_t)stream;
  const long heads = (long)a.B * a.c.H;
  cudaError_t e = launch_first(pick_kernel, heads, kPickThreads, st, a);
  if (e == cudaSuccess)
    e = a.c.D == 64 ? launch_first(gather_kernel<64>, 2 * heads, kGatherThreads, st, a)
                    : launch_first(gather_kernel<128>, 2 * heads, kGatherThreads, st, a);
  return e == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}

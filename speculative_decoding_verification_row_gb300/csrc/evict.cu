// Eviction from the 8-bit cache by weight (spec_evict_kv): a selection per
// request and KV head, then the kept rows' move.
//
// Selection: one CTA finds the weight of the last position kept with a radix
// selection over the weights' order keys (11, 11 and 10 bits), writes the kept
// positions in order in one more pass, equal weights from the front, and notes
// for the move where each kept row lies, its block's scale and the new scales.
//
// Move: CTAs per request, KV head and kind, each with a slice of the rows'
// bytes (whole rows where there are enough of them to fill the GPU).  A kept
// row never moves up, so a CTA gathers its slice batch by batch: all of a batch
// is read before any of it is written, and what is written lies below every
// row still to be read.
//
// In a graph: 64 requests of up to 8192 positions to 2048, 8 heads of 128, 147 us,
// the selection some 40 (latency of its passes) and the move 105 (0.7 of the
// measured copy rate); one request of 16000 to 4096 32 us.
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
  int2* from;       // scratch [B, H, keep]: a kept row's block and place in it
  float2* had;      // [B, H, keep]: that block's scales of K and V
  int* now;         // [B, H, pages, 2]: the scales of the blocks written, as bits
  int pages;        // blocks of `keep` positions
  unsigned div16;   // x / (tpb / 16) = umulhi(x, div16) for x < 2^26, tpb > 16
  // Block table column of position t (below 2^30).
  __device__ __forceinline__ int col(int t) const {
    return c.tpb == 16 ? t >> 4 : (int)__umulhi((unsigned)t >> 4, div16);
  }
  int B, T, T_out, keep, first, recent;
};

constexpr int kBins = 2048;
constexpr int kHeld = 4;   // tiles of THREADS x kTake weights that stay in registers
constexpr int kTake = 4;   // runs of 32 positions that a warp takes at a time

// Order key of a weight: NaN below all, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float x) { return x == x ? ord32(x) : 0u; }

// Exclusive sum over the CTA of two small counts of a warp, packed in 16 bits
// each; *total: their sum over all warps.
template <int THREADS>
__device__ __forceinline__ uint32_t before_warp(uint32_t mine, uint32_t* sWarp, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) sWarp[warp] = mine;
  __syncthreads();
  uint32_t x = lane < THREADS / 32 ? sWarp[lane] : 0u;
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

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) pick_kernel(const EvictArgs a) {
  __shared__ int sHist[kBins];
  __shared__ uint32_t sWarp[THREADS / 32];
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
    for (int i = tid; (long)i * c.tpb < n; i += THREADS) bad |= table[i] < 0 || table[i] >= c.num_blocks;
  }
  bad = __syncthreads_or(bad);
  if (bad || n <= a.keep) {
    for (int j = tid; j < a.keep; j += THREADS) {
      const bool real = !bad && j < n;
      kept[j] = real ? j : -1;
      if (real) out[j] = w[j];
    }
    return;
  }
  const int lo = a.first, hi = n - a.recent;  // the positions that may go: [lo, hi)
  const int want = a.keep - a.first - a.recent;
  // The weights, a warp's 32 kTake in a row: those of short requests stay in registers.
  constexpr int kTile = THREADS * kTake;
  const int mine = warp * kTake * 32 + lane;
  float x[kHeld][kTake];
  auto load = [&](float (&v)[kTake], int t0) {
#pragma unroll
    for (int y = 0; y < kTake; ++y) {
      const int t = t0 + mine + y * 32;
      v[y] = t < n ? w[t] : 0.f;
    }
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i) load(x[i], i * kTile);
  // f(weights, first position of the tile) in order
  auto tiles = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i * kTile < n) f(x[i], i * kTile);
    for (int t0 = kHeld * kTile; t0 < n; t0 += 2 * kTile) {
      float v[2][kTake];
      load(v[0], t0);
      load(v[1], t0 + kTile);
      f(v[0], t0);
      if (t0 + kTile < n) f(v[1], t0 + kTile);
    }
  };
  // ---- the key of the last one kept, and how many of that key
  uint32_t top = 0xffffffffu;  // nothing reaches it: NaN has key 0, every number less
  int ties = 0;
  if (want > 0) {
    uint32_t prefix = 0, known = 0;
    int left = want;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass < 2 ? kBins : kBins / 2;
      for (int i = tid; i < kBins; i += THREADS) sHist[i] = 0;
      __syncthreads();
      tiles([&](const float (&v)[kTake], int t0) {
#pragma unroll
        for (int y = 0; y < kTake; ++y) {
          const int t = t0 + mine + y * 32;
          const uint32_t k = weight_key(v[y]);
          if (t >= lo && t < hi && (k & known) == prefix) atomicAdd(&sHist[k >> shift & (bins - 1)], 1);
        }
      });
      __syncthreads();
      // the highest bin whose sum from the top reaches `left`: some bins a thread, from the top
      constexpr int kMine = kBins / THREADS;
      const int b0 = bins - 1 - kMine * tid;
      int count[kMine], incl = 0;
#pragma unroll
      for (int i = 0; i < kMine; ++i) incl += count[i] = b0 - i >= 0 ? sHist[b0 - i] : 0;
      const int own = incl;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(~0u, incl, d);
        if (lane >= d) incl += y;
      }
      if (lane == 31) sWarp[warp] = (uint32_t)incl;
      __syncthreads();
      int above = incl - own;
      for (int i = 0; i < warp; ++i) above += (int)sWarp[i];
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        if (above < left && left <= above + count[i]) sBin = b0 - i, sAbove = above;
        above += count[i];
      }
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
  int* now = a.now + (size_t)blockIdx.x * a.pages * 2;
  for (int i = tid; i < 2 * a.pages; i += THREADS) now[i] = 0;
  int before = 0, equal = 0;  // kept without the ties, and ties, of the tiles before
  tiles([&](const float (&v)[kTake], int t0) {
    unsigned am[kTake], tm[kTake];
    uint32_t count = 0;
#pragma unroll
    for (int y = 0; y < kTake; ++y) {
      const int t = t0 + mine + y * 32;
      const bool must = t < n && (t < lo || t >= hi), may = t >= lo && t < hi && want > 0;
      const uint32_t k = weight_key(v[y]);
      am[y] = __ballot_sync(~0u, must || (may && k > top));
      tm[y] = __ballot_sync(~0u, may && k == top);
      count += (uint32_t)__popc(am[y]) << 16 | (uint32_t)__popc(tm[y]);
    }
    uint32_t total;  // at most kTile of each kind
    const uint32_t pre = before_warp<THREADS>(count, sWarp, &total);
    int at = before + (int)(pre >> 16), tied = equal + (int)(pre & 0xffffu);
    const unsigned mask = (1u << lane) - 1;
#pragma unroll
    for (int y = 0; y < kTake; ++y) {
      const int ties_before = tied + __popc(tm[y] & mask);
      if (am[y] >> lane & 1 || (tm[y] >> lane & 1 && ties_before < ties)) {
        const int j = at + __popc(am[y] & mask) + min(ties_before, ties);
        kept[j] = t0 + mine + y * 32;
        out[j] = v[y];  // in place: below every weight still to be read
      }
      at += __popc(am[y]);
      tied += __popc(tm[y]);
    }
    before += (int)(total >> 16);
    equal += (int)(total & 0xffffu);
  });
  // ---- where the kept rows lie, and the scales of the blocks that receive them
  __syncthreads();
  const int32_t* table = c.tables + (size_t)b * c.max_blocks;
  const int h = blockIdx.x - b * c.H;
  int2* from = a.from + (size_t)blockIdx.x * a.keep;
  float2* had = a.had + (size_t)blockIdx.x * a.keep;
#pragma unroll 4
  for (int j0 = warp * 32; j0 < a.keep; j0 += THREADS) {
    const int j = min(j0 + lane, a.keep - 1), t = kept[j], col = a.col(t), blk = table[col];
    const float* s = c.scales + c.scale_at(blk, 0, h);
    const float2 had_j = make_float2(s[0], s[c.H]);
    if (j0 + lane < a.keep) {
      from[j] = make_int2(blk, t - col * c.tpb);
      had[j] = had_j;
    }
    // 16 lanes write to one block: the lanes behind the last row repeat it
    int top_k = __float_as_int(had_j.x), top_v = __float_as_int(had_j.y);  // scales are >= 0: ordered as integers
#pragma unroll
    for (int d = 8; d; d >>= 1) {
      top_k = max(top_k, __shfl_xor_sync(~0u, top_k, d));
      top_v = max(top_v, __shfl_xor_sync(~0u, top_v, d));
    }
    if ((lane & 15) == 0 && j0 + lane < a.keep) {
      int* p = now + a.col(j0 + lane) * 2;
      atomicMax(p, top_k);
      atomicMax(p + 1, top_v);
    }
  }
}

constexpr int kGatherVecs = 4;  // 16-byte vectors of a thread in a batch

// V: 16-byte vectors of a row in a CTA's slice.
template <int V, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) gather_kernel(const EvictArgs a, int slices) {
  const KvCache& c = a.c;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int u = blockIdx.x;
  const int slice = u % slices;
  u /= slices;
  const int kind = u & 1, h = (u >> 1) % c.H, b = (u >> 1) / c.H;
  const size_t head = (size_t)b * c.H + h;
  const int32_t* kept = a.kept + head * a.keep;
  const int last = kept[a.keep - 1];
  if (kind == 0 && h == 0 && slice == 0 && tid == 0) {
    const int n = a.seq[b], now = last >= 0 ? a.keep : n;
    if (a.free_blocks) {
      const bool ok = n == 0 || kept[0] >= 0;
      a.free_blocks[b] = ok ? max(0, a.held[b] - (int)(((long)now + c.tpb - 1) / c.tpb)) : 0;
    }
    a.new_lens[b] = now;
  }
  if (last < a.keep) return;  // at most `keep` positions: nothing moves
  const int32_t* table = c.tables + (size_t)b * c.max_blocks;
  const int2* from = a.from + head * a.keep;
  const float* had = reinterpret_cast<const float*>(a.had + head * a.keep) + kind;
  const float* now = reinterpret_cast<const float*>(a.now + head * a.pages * 2) + kind;
  if (slice == 0)  // the old scales are in `had`
    for (int i = tid; i < a.pages; i += THREADS) c.scales[c.scale_at(table[i], kind, h)] = now[2 * i];
  const int x0 = slice * V + tid % V;  // the thread's vector of its rows
  constexpr int kStep = THREADS / V;
  int2 f[kGatherVecs];  // of the batch to come
  auto places = [&](int j0) {
#pragma unroll
    for (int k = 0; k < kGatherVecs; ++k) f[k] = from[min(j0 + k * kStep, a.keep - 1)];
  };
  places(tid / V);
  for (int j0 = tid / V; j0 - tid / V < a.keep; j0 += kStep * kGatherVecs) {
    uint4 x[kGatherVecs];
    float ratio[kGatherVecs];
    uint8_t* to[kGatherVecs];
#pragma unroll
    for (int k = 0; k < kGatherVecs; ++k) {
      const int j = min(j0 + k * kStep, a.keep - 1), col = a.col(j);
      x[k] = reinterpret_cast<const uint4*>(c.pool + c.row(f[k].x, kind, h, f[k].y))[x0];
      const float was = had[2 * j], is = now[2 * col];
      ratio[k] = was != is ? scale_ratio(was, is) : -1.f;  // -1: the codes stay
      to[k] = c.pool + c.row(table[col], kind, h, j - col * c.tpb) + x0 * 16;
    }
    places(j0 + kStep * kGatherVecs);
    __syncthreads();  // all of the batch has been read
#pragma unroll
    for (int k = 0; k < kGatherVecs; ++k) {
      if (ratio[k] >= 0.f) x[k] = rescale_e4m3x16(x[k], ratio[k]);
      if (j0 + k * kStep < a.keep) *reinterpret_cast<uint4*>(to[k]) = x[k];
    }
  }
}

template <int V, int THREADS>
cudaError_t launch_gather(const EvictArgs& a, long units, cudaStream_t st) {
  const int slices = a.c.D / 16 / V;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * slices));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gather_kernel<V, THREADS>, a, slices);
}

size_t scratch_bytes_of(int B, int kv_heads, int keep, int tpb) {
  const size_t heads = (size_t)B * kv_heads;
  return align256(heads * keep * sizeof(int2)) + align256(heads * keep * sizeof(float2)) +
         align256(heads * ceil_div(keep, tpb) * 2 * sizeof(int));
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_evict_scratch_size(int B, int kv_heads, int keep, int tokens_per_block) {
  if (B < 1 || B > SPEC_MAX_BATCH || kv_heads < 1 || kv_heads > 1024 || keep < 1 || keep > 1 << 30 ||
      tokens_per_block < 16 || tokens_per_block > 1024 || tokens_per_block % 16 != 0)
    return 0;
  return scratch_bytes_of(B, kv_heads, keep, tokens_per_block);
}

int spec_evict_kv(const spec_kv_cache* cache, const spec_evict_params* p, void* scratch, size_t scratch_bytes,
                  spec_stream_t stream) {
  EvictArgs a{};
  const int rc = kv_setup(cache, &a.c);
  if (rc != SPEC_OK) return rc;
  if (!p || p->size != sizeof(spec_evict_params) || !p->weights || !p->seq_lens || !p->new_lens || !p->kept ||
      !p->out_weights || p->B < 1 || p->B > SPEC_MAX_BATCH || p->T < 1 || p->keep < 1 || p->keep > 1 << 30 ||
      p->first < 0 || p->recent < 0 || (long)p->first + p->recent > p->keep || p->T_out < p->keep ||
      (p->out_weights == p->weights && p->T_out != p->T) || !p->blocks_held != !p->free_blocks ||
      (long)a.c.max_blocks * a.c.tpb > 1l << 30)
    return SPEC_EINVAL;
  if (!scratch || reinterpret_cast<uintptr_t>(scratch) % 256 != 0 ||
      scratch_bytes < scratch_bytes_of(p->B, a.c.H, p->keep, a.c.tpb))
    return SPEC_EWORKSPACE;
  const long lens = (long)p->B * sizeof(int32_t), per_row = (long)p->B * a.c.H * sizeof(float);
  Arrays x;
  const int old = x.read(dense(p->weights, per_row * p->T)), seq = x.read(dense(p->seq_lens, lens));
  x.read(dense(p->blocks_held, lens));
  cache_arrays(a.c, p->B, true, &x);
  x.write(dense(p->new_lens, lens), seq);
  x.write(dense(p->kept, per_row * p->keep));
  x.write(dense(p->out_weights, per_row * p->T_out), old);
  x.write(dense(p->free_blocks, lens));
  x.write(dense(scratch, scratch_bytes_of(p->B, a.c.H, p->keep, a.c.tpb)));
  if (!x.apart()) return SPEC_EINVAL;
  const long heads = (long)p->B * a.c.H;
  char* s = static_cast<char*>(scratch);
  a.from = reinterpret_cast<int2*>(s);
  s += align256(heads * p->keep * sizeof(int2));
  a.had = reinterpret_cast<float2*>(s);
  s += align256(heads * p->keep * sizeof(float2));
  a.now = reinterpret_cast<int*>(s);
  a.pages = ceil_div(p->keep, a.c.tpb);
  a.div16 = (unsigned)((1ull << 32) / (a.c.tpb / 16) + ((1ull << 32) % (a.c.tpb / 16) != 0));
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
  // A CTA of 1024 holds 16384 weights in its registers, and there is one for each
  // SM; with more heads two of 512.
  cudaError_t e = heads <= 152 ? launch_first(pick_kernel<1024>, heads, 1024, st, a)
                               : launch_first(pick_kernel<512>, heads, 512, st, a);
  if (e != cudaSuccess) return SPEC_ECUDA;
  // Whole rows where they give every SM several CTAs, else half of them, or 32
  // bytes (a sector) with larger CTAs.  64 requests, 2048 of up to 8192
  // positions kept: 149 us with 4 CTAs of 256 per SM, 158 with 2 of 512; one
  // request, 4096 of 16000: 42 with CTAs of 256, 36 with 512.  The rule's ends, 8 KV
  // heads, 2048 of 8192 kept, the three forms in this order (heads of 64 have no
  // second): 1 request 30, -, 20 with heads of 64 and 44, 30, 20 with 128; 16
  // requests 45, -, 35 and 73, 46, 53; 38 requests 62, -, 69 and 90, 91, 108; 100
  // requests 167, -, 178 and 245, 244, 281.  Between 16 and 38 requests the best form
  // is some 10 percent ahead of the rule's.
  const bool wide = a.c.D == 128;
  if (2 * heads >= 8 * 152)
    e = wide ? launch_gather<8, 256>(a, 2 * heads, st) : launch_gather<4, 256>(a, 2 * heads, st);
  else if (wide && 2 * heads >= 4 * 152)
    e = launch_gather<4, 256>(a, 2 * heads, st);
  else
    e = launch_gather<2, 512>(a, 2 * heads, st);
  return e == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}

}  // extern "C"

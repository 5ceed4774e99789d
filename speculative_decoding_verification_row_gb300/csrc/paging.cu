// Block tables and slot maps of a step's windows (spec_reserve_blocks), the
// way back (spec_release_blocks), and the ancestor masks of a tree
// (spec_tree_masks).
//
// Reserve and release are a prefix sum over at most SPEC_MAX_BATCH = 8192
// requests and a few words for each, so they are bound by latency: a launch,
// the load of the per-request words, the scan, the load of the block id, the
// store.  One launch of one thread-block cluster does it: request r belongs
// to thread r of the cluster (8 CTAs x 1024 threads = 8192), the scan crosses
// the CTAs through distributed shared memory, and the cluster barrier between
// the last read and the first write lets the counters be updated in place
// with no workspace and no second launch.  The sums saturate at 2^31 - 1,
// which no stack reaches: 32-bit shuffles and no 64-bit division.
//
// Reserve and release of a step, in a graph: 6.0 us for 64 requests of 8
// tokens, 11.5 us for 8192 of 4 (eight CTAs, 131 KB of slots), against about
// 2.5 us for each of the two launches.
#include <cooperative_groups.h>

#include "kernels.cuh"

namespace cg = cooperative_groups;

namespace sv {

namespace {

constexpr int kMaxCluster = 8;
constexpr int kPageThreads = 1024;
static_assert(kMaxCluster * kPageThreads >= SPEC_MAX_BATCH, "one thread per request");

struct PageArgs {
  const int32_t* seq;
  const int32_t* win;
  const int32_t* counts;
  int W, tpb, B;
  int32_t* tables;
  int max_blocks;
  int32_t* held;
  int32_t* free_blocks;
  int num_blocks;
  int32_t* free_count;
  int32_t* slots;
  int32_t* granted;
};

__device__ __forceinline__ unsigned sat_add(unsigned a, unsigned b) {
  return min(a + b, 0x7fffffffu);  // both at most 2^31 - 1
}

// Inclusive prefix of x over the cluster's threads in rank order (saturating),
// and the total.  sWarp: 32 words, sTotal: one word that the other CTAs read.
// Ends past a cluster barrier: everything the threads loaded before the call
// has been read by then.
__device__ unsigned cluster_scan(cg::cluster_group& cl, unsigned x, unsigned* sWarp,
                                 unsigned* sTotal, unsigned* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned incl = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned y = __shfl_up_sync(~0u, incl, d);
    if (lane >= d) incl = sat_add(incl, y);
  }
  if (lane == 31) sWarp[warp] = incl;
  __syncthreads();
  unsigned before = 0, all = 0;
  if (blockDim.x > 256 || cl.num_blocks() > 1) {
    if (warp == 0) {
      unsigned w = lane < (int)(blockDim.x >> 5) ? sWarp[lane] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned y = __shfl_up_sync(~0u, w, d);
        if (lane >= d) w = sat_add(w, y);
      }
      sWarp[lane] = w;
      if (lane == 31) *sTotal = w;
    }
    cl.sync();
    const int me = cl.block_rank(), n = cl.num_blocks();
    for (int r = 0; r < n; ++r) {
      const unsigned t = *cl.map_shared_rank(sTotal, r);
      if (r < me) before = sat_add(before, t);
      all = sat_add(all, t);
    }
    if (warp) before = sat_add(before, sWarp[warp - 1]);
  } else {  // few warps of one CTA
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
      if (w < warp) before = sat_add(before, sWarp[w]);
      all = sat_add(all, sWarp[w]);
    }
  }
  *total = all;
  return sat_add(before, incl);
}

// Calls f(r, i, n) for i in [0, n) of every lane's n: each lane serves its
// own first two entries, the whole warp the rest (a prompt's hundreds).
template <class F>
__device__ __forceinline__ void for_entries(int n, F f) {
  const int lane = threadIdx.x & 31;
  if (n > 0) f(lane, 0);
  if (n > 1) f(lane, 1);
  unsigned more = __ballot_sync(~0u, n > 2);
  while (more) {
    const int src = __ffs(more) - 1;
    more &= more - 1;
    const int m = __shfl_sync(~0u, n, src);
    for (int i = 2 + lane; i < m; i += 32) f(src, i);
  }
}

__global__ void __launch_bounds__(kPageThreads) reserve_kernel(const PageArgs a) {
  __shared__ unsigned sWarp[32], sTotal, sUsed;
  __shared__ int sFirst[kPageThreads];  // stack index of the request's first new block
  __shared__ int sSeq[kPageThreads], sHeld[kPageThreads], sGranted[kPageThreads];
  cg::cluster_group cl = cg::this_cluster();
  const int b = cl.block_rank() * blockDim.x + threadIdx.x;
  const int count = *a.free_count;
  int seq = 0, win = 0, held = 0;
  unsigned need = 0;
  bool ok = false;
  if (threadIdx.x == 0) sUsed = 0;
  if (b < a.B) {
    seq = a.seq[b];
    win = a.win ? a.win[b] : a.W;
    held = a.held[b];
    ok = seq >= 0 && win >= 0 && win <= a.W && held >= 0 && held <= a.max_blocks;
    if (ok) {
      const unsigned end = (unsigned)seq + win, tpb = a.tpb;
      const unsigned blocks = end / tpb + (end % tpb != 0);
      ok = blocks <= (unsigned)a.max_blocks;
      need = ok && blocks > (unsigned)held ? blocks - held : 0;
    }
  }
  unsigned total;
  const unsigned upto = cluster_scan(cl, need, sWarp, &sTotal, &total);
  const unsigned avail = count < 0 || count > a.num_blocks ? 0 : count;
  // Requests are served while the running sum fits, so every served request
  // comes before every refused one that needs a block.
  if (ok && need > 0 && upto > avail) ok = false;
  const int take = ok ? (int)need : 0;
  sFirst[threadIdx.x] = (int)(avail - 1 - (upto - need));
  sSeq[threadIdx.x] = seq;
  sHeld[threadIdx.x] = held;
  sGranted[threadIdx.x] = ok ? win : -1;
  // what the stack gave: the running sum at the last served request
  const unsigned used = __reduce_max_sync(~0u, take > 0 ? upto : 0u);
  if ((threadIdx.x & 31) == 0 && used > 0) atomicMax(cl.map_shared_rank(&sUsed, 0), used);
  if (b < a.B) {
    a.granted[b] = ok ? win : -1;
    if (take > 0) a.held[b] = held + take;
  }
  const int b0 = cl.block_rank() * blockDim.x;
  const int w0 = threadIdx.x & ~31;
  __syncthreads();
  for_entries(take, [&](int lane, int i) {
    const int r = w0 + lane;
    a.tables[(size_t)(b0 + r) * a.max_blocks + sHeld[r] + i] = a.free_blocks[sFirst[r] - i];
  });
  if (a.slots) {
    // A block that was just taken is read from the stack again rather than
    // from the table, so the slots need not wait for its stores.
    const unsigned rows = max(0, min((int)blockDim.x, a.B - b0)), n = rows * a.W;  // at most 2^26
    for (unsigned s = threadIdx.x; s < n; s += blockDim.x) {
      const unsigned r = s / (unsigned)a.W, i = s - r * a.W;
      int slot = -1;
      if ((int)i < sGranted[r]) {
        const unsigned t = (unsigned)sSeq[r] + i, col = t / (unsigned)a.tpb;
        const int blk = (int)col < sHeld[r] ? a.tables[(size_t)(b0 + r) * a.max_blocks + col]
                                            : a.free_blocks[sFirst[r] - (int)(col - sHeld[r])];
        if (blk >= 0 && blk < a.num_blocks) slot = blk * a.tpb + (int)(t - col * a.tpb);
      }
      a.slots[(size_t)b0 * a.W + s] = slot;
    }
  }
  cl.sync();  // every CTA has read the totals and stored what it used
  if (b == 0 && sUsed > 0) *a.free_count = count - (int)sUsed;
}

__global__ void __launch_bounds__(kPageThreads) release_kernel(const PageArgs a) {
  __shared__ unsigned sWarp[32], sTotal;
  __shared__ int sTop[kPageThreads];   // stack index the request's first block goes to
  __shared__ int sFrom[kPageThreads];  // table column of that block
  cg::cluster_group cl = cg::this_cluster();
  const int b = cl.block_rank() * blockDim.x + threadIdx.x;
  const int count = *a.free_count;
  int held = 0, n = 0;
  if (b < a.B) {
    held = a.held[b];
    n = a.counts[b];
    if (held < 0 || held > a.max_blocks || n < 0 || n > held) n = 0;
  }
  unsigned total;
  const unsigned upto = cluster_scan(cl, n, sWarp, &sTotal, &total);
  const bool fits = count >= 0 && count <= a.num_blocks && total <= (unsigned)(a.num_blocks - count);
  sTop[threadIdx.x] = (int)(count + total - 1 - (upto - n));
  if (!fits) n = 0;
  sFrom[threadIdx.x] = held - n;
  __syncthreads();  // also: thread 0 stores the count only when all have read it
  if (n > 0) a.held[b] = held - n;
  const int b0 = cl.block_rank() * blockDim.x;
  const int w0 = threadIdx.x & ~31;
  for_entries(n, [&](int lane, int i) {
    const int r = w0 + lane;
    int32_t* entry = a.tables + (size_t)(b0 + r) * a.max_blocks + sFrom[r] + i;
    a.free_blocks[sTop[r] - i] = *entry;
    *entry = -1;
  });
  cl.sync();  // no CTA leaves, and the count stays, while another may still read
  if (b == 0 && fits && total > 0) *a.free_count = count + (int)total;
}

// One CTA builds the mask rows [r0, r0 + kMaskRows) of one request.  The paths
// pass through shared memory in batches, a warp to a path (L <= 64: two nodes
// per lane).  First every node's parent: where a node has one parent on all
// used paths (a tree), its row is its parent's chain up to the root, walked by
// one thread.  Paths that give a node several parents are ORed bit by bit.
// 16 requests of 60 nodes take 3.1 us in a graph, 64 of 509 nodes and 301
// paths of 17 8.7 us: latency again (the passage, the chain of 17 parents, the
// rows).  The latter took 39 us when every path was ORed, its loads waited for
// path by path.
constexpr int kMaskRows = 128;
constexpr int kMaskThreads = 512;
constexpr int kMaskBatch = 4096;  // path entries at a time

__global__ void __launch_bounds__(kMaskThreads) tree_mask_kernel(const int32_t* paths, int P, int L,
                                                                 int N, int32_t* masks) {
  __shared__ int sPath[kMaskBatch];
  __shared__ int sParent[SPEC_MAX_TREE_NODES];
  __shared__ unsigned sBits[kMaskRows * (SPEC_MAX_TREE_NODES / 32 + 1)];
  __shared__ int sBad, sSeveral;
  constexpr int kNone = -2;  // on no used path; -1: the root's parent
  const int words = (N + 31) / 32, pitch = words | 1;
  const int chunks = (N + kMaskRows - 1) / kMaskRows;
  const int b = blockIdx.x / chunks, r0 = blockIdx.x % chunks * kMaskRows;
  const int rows = min(kMaskRows, N - r0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < rows * pitch; i += kMaskThreads) sBits[i] = 0;
  for (int i = threadIdx.x; i < N; i += kMaskThreads) sParent[i] = kNone;
  if (threadIdx.x == 0) sBad = sSeveral = 0;
  const int per = kMaskBatch / L;  // paths of a batch
  // calls f(n0, n1, len) for every used path: the lane's nodes lane and lane + 32
  auto each_path = [&](auto f) {
    for (long p0 = 0; p0 < P; p0 += per) {
      const int np = (int)min((long)per, P - p0);
      const int32_t* src = paths + ((size_t)b * P + p0) * L;
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kMaskBatch / kMaskThreads; ++q) {
        const int i = threadIdx.x + q * kMaskThreads;
        if (i < np * L) sPath[i] = src[i];
      }
      __syncthreads();
      for (int p = warp; p < np; p += kMaskThreads / 32) {
        const int* path = sPath + p * L;
        if (path[0] != 0) continue;  // an unused path
        const int n0 = lane < L ? path[lane] : -1, n1 = lane + 32 < L ? path[lane + 32] : -1;
        const unsigned neg0 = __ballot_sync(~0u, n0 < 0), neg1 = __ballot_sync(~0u, n1 < 0);
        f(path, n0, n1, neg0 ? __ffs(neg0) - 1 : neg1 ? 31 + __ffs(neg1) : 64);
      }
    }
  };
  each_path([&](const int* path, int n0, int n1, int len) {
    auto claim = [&](int d, int node) {
      if (d >= len) return;
      if (node >= N) {
        sBad = 1;
        return;
      }
      const int parent = d ? path[d - 1] : -1, had = atomicCAS(&sParent[node], kNone, parent);
      if (had != kNone && had != parent) sSeveral = 1;
    };
    claim(lane, n0);
    claim(lane + 32, n1);
  });
  __syncthreads();
  if (!sBad && !sSeveral) {
    for (int i = threadIdx.x; i < rows; i += kMaskThreads) {
      // A parent is on a path before its node: the chain ends at the root.
      if (sParent[r0 + i] != kNone)
        for (int node = r0 + i; node >= 0; node = sParent[node])
          sBits[i * pitch + (node >> 5)] |= 1u << (node & 31);
    }
  } else if (!sBad) {
    each_path([&](const int* path, int n0, int n1, int len) {
      for (int d = 0; d < len; ++d) {
        const int row = path[d] - r0;
        if (row < 0 || row >= rows) continue;
        unsigned* bits = sBits + row * pitch;
        if (lane <= d) atomicOr(bits + (n0 >> 5), 1u << (n0 & 31));
        if (lane + 32 <= d) atomicOr(bits + (n1 >> 5), 1u << (n1 & 31));
      }
    });
  }
  __syncthreads();
  int32_t* dst = masks + ((size_t)b * N + r0) * words;
  for (int i = threadIdx.x; i < rows * words; i += kMaskThreads) {
    const int r = (unsigned)i / (unsigned)words;
    dst[i] = (int32_t)sBits[r * pitch + i - r * words];
  }
}

// One cluster that gives every request a thread: a CTA up to 1024 requests,
// with more threads than requests where their slots are many.
template <class Kern>
cudaError_t launch_paged(Kern kernel, const PageArgs& a, long slots, cudaStream_t st) {
  const int ctas = a.B > 4 * kPageThreads ? 8 : a.B > 2 * kPageThreads ? 4 : a.B > kPageThreads ? 2 : 1;
  const int per = max(ceil_div(a.B, ctas), min(kPageThreads, ceil_div(slots, 2L * ctas)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(max(64, (per + 31) / 32 * 32));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" {

int spec_reserve_blocks(const int32_t* seq_lens, const int32_t* window_lens, int W,
                        int tokens_per_block, int B, int32_t* block_tables, int max_blocks,
                        int32_t* blocks_held, const int32_t* free_blocks, int num_blocks,
                        int32_t* free_count, int32_t* slots, int32_t* granted,
                        spec_stream_t stream) {
  if (!seq_lens || !block_tables || !blocks_held || !free_blocks || !free_count || !granted)
    return SPEC_EINVAL;
  if (B < 1 || B > SPEC_MAX_BATCH || W < 1 || W > SPEC_MAX_WINDOW || tokens_per_block < 1 ||
      max_blocks < 1 || num_blocks < 1 ||
      (slots && (long long)num_blocks * tokens_per_block > INT_MAX))
    return SPEC_EINVAL;
  PageArgs a{seq_lens,    window_lens, nullptr,     W,          tokens_per_block,
             B,           block_tables, max_blocks, blocks_held, const_cast<int32_t*>(free_blocks),
             num_blocks,  free_count,  slots,       granted};
  return launch_paged(reserve_kernel, a, slots ? (long)B * W : 0, (cudaStream_t)stream) == cudaSuccess ? SPEC_OK
                                                                              : SPEC_ECUDA;
}

int spec_release_blocks(const int32_t* counts, int B, int32_t* block_tables, int max_blocks,
                        int32_t* blocks_held, int32_t* free_blocks, int num_blocks,
                        int32_t* free_count, spec_stream_t stream) {
  if (!counts || !block_tables || !blocks_held || !free_blocks || !free_count) return SPEC_EINVAL;
  if (B < 1 || B > SPEC_MAX_BATCH || max_blocks < 1 || num_blocks < 1) return SPEC_EINVAL;
  PageArgs a{nullptr,    nullptr,      counts,     0,           1,
             B,          block_tables, max_blocks, blocks_held, free_blocks,
             num_blocks, free_count,   nullptr,    nullptr};
  return launch_paged(release_kernel, a, 0, (cudaStream_t)stream) == cudaSuccess ? SPEC_OK
                                                                              : SPEC_ECUDA;
}

int spec_tree_masks(const int32_t* paths, int B, int P, int L, int N, int32_t* masks,
                    spec_stream_t stream) {
  if (!paths || !masks) return SPEC_EINVAL;
  if (B < 1 || B > SPEC_MAX_BATCH || N < 1 || N > SPEC_MAX_TREE_NODES || P < 1 || L < 1 ||
      L > SPEC_MAX_PATH_LEN)
    return SPEC_EINVAL;
  const int chunks = ceil_div(N, kMaskRows);
  tree_mask_kernel<<<(unsigned)(B * chunks), kMaskThreads, 0, (cudaStream_t)stream>>>(paths, P, L, N,
                                                                                      masks);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}

}  // extern "C"

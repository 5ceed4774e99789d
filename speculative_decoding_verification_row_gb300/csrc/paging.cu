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
// with no workspace and no second launch.
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

// Exclusive prefix of x over the cluster's threads in rank order, and the
// total.  sWarp: 32 words, sTotal: one word that the other CTAs read.  Ends
// past a cluster barrier: everything the threads loaded before the call has
// been read by then.
__device__ long long cluster_scan(cg::cluster_group& cl, long long x, long long* sWarp,
                                  long long* sTotal, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(~0u, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) sWarp[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < (int)(blockDim.x >> 5) ? sWarp[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(~0u, w, d);
      if (lane >= d) w += y;
    }
    sWarp[lane] = w;
    if (lane == 31) *sTotal = w;
  }
  cl.sync();
  long long before = 0, all = 0;
  const int me = cl.block_rank(), n = cl.num_blocks();
  for (int r = 0; r < n; ++r) {
    const long long t = *cl.map_shared_rank(sTotal, r);
    before += r < me ? t : 0;
    all += t;
  }
  *total = all;
  return before + (warp ? sWarp[warp - 1] : 0) + incl - x;
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
  __shared__ long long sWarp[32];
  __shared__ long long sTotal[2];
  __shared__ long long sFirst[kPageThreads];  // stack index of the request's first new block
  __shared__ int sSeq[kPageThreads], sHeld[kPageThreads], sGranted[kPageThreads];
  cg::cluster_group cl = cg::this_cluster();
  const int b = cl.block_rank() * blockDim.x + threadIdx.x;
  const int count = *a.free_count;
  int seq = 0, win = 0, held = 0;
  long long need = 0;
  bool ok = false;
  if (b < a.B) {
    seq = a.seq[b];
    win = a.win ? a.win[b] : a.W;
    held = a.held[b];
    ok = seq >= 0 && win >= 0 && win <= a.W && held >= 0 && held <= a.max_blocks;
    if (ok) {
      const long long blocks = ((long long)seq + win + a.tpb - 1) / a.tpb;
      ok = blocks <= a.max_blocks;
      need = ok && blocks > held ? blocks - held : 0;
    }
  }
  long long total;
  const long long first = cluster_scan(cl, need, sWarp, &sTotal[0], &total);
  const int avail = count < 0 || count > a.num_blocks ? 0 : count;
  // Requests are served while the running sum fits, so every served request
  // comes before every refused one that needs a block.
  if (ok && need > 0 && first + need > avail) ok = false;
  const int take = ok ? (int)need : 0;
  sFirst[threadIdx.x] = avail - 1 - first;
  sSeq[threadIdx.x] = seq;
  sHeld[threadIdx.x] = held;
  sGranted[threadIdx.x] = ok ? win : -1;
  // what the stack gave: the sum up to the first refused request
  long long used;
  __syncthreads();
  cluster_scan(cl, take, sWarp, &sTotal[1], &used);
  if (b < a.B) {
    a.granted[b] = ok ? win : -1;
    if (take > 0) a.held[b] = held + take;
  }
  if (b == 0 && used > 0) *a.free_count = count - (int)used;
  const int b0 = cl.block_rank() * blockDim.x;
  const int w0 = threadIdx.x & ~31;
  for_entries(take, [&](int lane, int i) {
    const int r = w0 + lane;
    a.tables[(size_t)(b0 + r) * a.max_blocks + sHeld[r] + i] = a.free_blocks[sFirst[r] - i];
  });
  if (a.slots) {
    // A block that was just taken is read from the stack again rather than
    // from the table, so the slots need not wait for its stores.
    const int rows = min((int)blockDim.x, a.B - b0);
    const long long n = rows > 0 ? (long long)rows * a.W : 0;
    for (long long s = threadIdx.x; s < n; s += blockDim.x) {
      const int r = (int)(s / a.W), i = (int)(s % a.W);
      int slot = -1;
      if (i < sGranted[r]) {
        const int t = sSeq[r] + i, col = t / a.tpb;
        const int blk = col < sHeld[r] ? a.tables[(size_t)(b0 + r) * a.max_blocks + col]
                                       : a.free_blocks[sFirst[r] - (col - sHeld[r])];
        if (blk >= 0 && blk < a.num_blocks) slot = blk * a.tpb + t % a.tpb;
      }
      a.slots[(size_t)b0 * a.W + s] = slot;
    }
  }
  cl.sync();  // no CTA leaves while another may still read its total
}

__global__ void __launch_bounds__(kPageThreads) release_kernel(const PageArgs a) {
  __shared__ long long sWarp[32];
  __shared__ long long sTotal;
  __shared__ long long sTop[kPageThreads];  // stack index the request's first block goes to
  __shared__ int sFrom[kPageThreads];       // table column of that block
  cg::cluster_group cl = cg::this_cluster();
  const int b = cl.block_rank() * blockDim.x + threadIdx.x;
  const int count = *a.free_count;
  int held = 0, n = 0;
  if (b < a.B) {
    held = a.held[b];
    n = a.counts[b];
    if (held < 0 || held > a.max_blocks || n < 0 || n > held) n = 0;
  }
  long long total;
  const long long first = cluster_scan(cl, n, sWarp, &sTotal, &total);
  const bool fits = count >= 0 && count + total <= a.num_blocks;
  if (!fits) n = 0;
  sTop[threadIdx.x] = count + total - 1 - first;
  sFrom[threadIdx.x] = held - n;
  __syncwarp();
  if (n > 0) a.held[b] = held - n;
  const int b0 = cl.block_rank() * blockDim.x;
  const int w0 = threadIdx.x & ~31;
  for_entries(n, [&](int lane, int i) {
    const int r = w0 + lane;
    int32_t* entry = a.tables + (size_t)(b0 + r) * a.max_blocks + sFrom[r] + i;
    a.free_blocks[sTop[r] - i] = *entry;
    *entry = -1;
  });
  if (b == 0 && fits && total > 0) *a.free_count = count + (int)total;
  cl.sync();
}

// One CTA builds the mask rows [r0, r0 + kMaskRows) of one request in shared
// memory: a warp reads a whole path (L <= 64: two nodes per lane) and sets,
// for every node of the path among its rows, the bits of the nodes up to it.
constexpr int kMaskRows = 64;
constexpr int kMaskThreads = 256;

__global__ void __launch_bounds__(kMaskThreads) tree_mask_kernel(const int32_t* paths, int P, int L,
                                                                 int N, int32_t* masks) {
  __shared__ unsigned sBits[kMaskRows * (SPEC_MAX_TREE_NODES / 32)];
  __shared__ int sBad;
  const int words = (N + 31) / 32;
  const int chunks = (N + kMaskRows - 1) / kMaskRows;
  const int b = blockIdx.x / chunks, r0 = blockIdx.x % chunks * kMaskRows;
  const int rows = min(kMaskRows, N - r0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < rows * words; i += kMaskThreads) sBits[i] = 0;
  if (threadIdx.x == 0) sBad = 0;
  __syncthreads();
  for (int p = warp; p < P; p += kMaskThreads / 32) {
    const int32_t* path = paths + ((size_t)b * P + p) * L;
    const int n0 = lane < L ? path[lane] : -1;
    const int n1 = lane + 32 < L ? path[lane + 32] : -1;
    const unsigned neg0 = __ballot_sync(~0u, n0 < 0), neg1 = __ballot_sync(~0u, n1 < 0);
    if (__shfl_sync(~0u, n0, 0) != 0) continue;  // an unused path
    const int len = neg0 ? __ffs(neg0) - 1 : neg1 ? 31 + __ffs(neg1) : 64;
    if ((lane < len && n0 >= N) || (lane + 32 < len && n1 >= N)) sBad = 1;
    for (int d = 0; d < len; ++d) {
      const int row = __shfl_sync(~0u, d < 32 ? n0 : n1, d & 31) - r0;
      if (row < 0 || row >= rows) continue;
      unsigned* bits = sBits + row * words;
      if (lane <= d && n0 < N) atomicOr(bits + (n0 >> 5), 1u << (n0 & 31));
      if (lane + 32 <= d && n1 < N) atomicOr(bits + (n1 >> 5), 1u << (n1 & 31));
    }
  }
  __syncthreads();
  int32_t* dst = masks + ((size_t)b * N + r0) * words;
  for (int i = threadIdx.x; i < rows * words; i += kMaskThreads)
    dst[i] = sBad ? 0 : (int32_t)sBits[i];
}

// One cluster that gives every request a thread: a CTA up to 1024 requests,
// with more threads than requests where their slots are many.
template <class Kern>
cudaError_t launch_paged(Kern kernel, const PageArgs& a, long slots, cudaStream_t st) {
  const int ctas = a.B > 4 * kPageThreads ? 8 : a.B > 2 * kPageThreads ? 4 : a.B > kPageThreads ? 2 : 1;
  const int per = max(ceil_div(a.B, ctas), min(kPageThreads, ceil_div(slots, 8L * ctas)));
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

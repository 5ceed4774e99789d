// Weighing the cached positions for many rows per KV head (tree windows,
// prompts): bound by the exponentials.
//
// One CTA per SM on tcgen05, 256 keys x 64 rows a step, the keys as the left
// operand: a key is a lane of tensor memory, so each thread adds up the weights
// of its own key and no sum crosses threads.  Warps by role:
//   0-7    weights: a thread per key reads its 64 scores of a step from tensor
//          memory and adds exp(score - lse); writes the sum.
//   8-11   keys: e4m3 rows of the pages as bf16 or fp16 (exact) into tensor
//          memory, a unit ahead.
//   12-14  queries: rows and their lse into shared memory (cp.async, 128-byte
//          swizzle), every warp each third step, two of its steps under way.
//          (Four warps on one step: 88 us for 2 prompt chunks of 2049 tokens, 16/4
//          heads of 64; a division in every copy there: 101.)
//   15     one thread issues the products.  (16 warps in all leave 128 registers,
//          room for a step's 64 scores at once; 17 with 32 at a time: 86.)
// 256 keys share a read of the queries: a step takes 16 KB (D = 128) from L2
// and 16384 exponentials.
//
// A unit is 256 keys of one (request, KV head); its steps are the row tiles
// that see any of them.  The steps of all units form one line that is cut into
// equal shares, one per CTA; a unit that falls to several CTAs is joined by a
// second launch in a fixed order.
//
// What is rounded: a score is one chain of D / 16 products, whose partial sums the
// tensor cores cut off instead of rounding; score - lse and its product with
// log2(e) round to fp32, exp2 is ex2.approx, and a key's rows are summed in fp32,
// 64 of a step on their own and then the steps.  A prompt of 1500 tokens, 8/2 heads
// of 128 in fp16 is 2.2e-7 off (of the weights' norm) and 0.7e-7 with scores that
// are exact, where products, exp and sums in fp32 give 0.6e-7 and 0.5e-7: the chain
// is what is left.  Two chains, as in weigh.cu, would take four buffers of scores;
// tensor memory has two beside the keys.  Weights only rank positions.
//
// In a graph: 2 prompt chunks of 2049 tokens over 0 and 4500, 16/4 heads of 64,
// 80 us; 32/8 heads of 128, 163 us (675 TFLOP/s, 0.36 of the measured dense
// rate); a prompt of 4096 109 us.  A step takes some 1600 clocks, its exponentials
// 512 to 1024, its products 512: the hops scores -> sums -> next products.
#include "tcgen05.cuh"
#include "weigh.cuh"

namespace sv {

namespace {

constexpr int kWKeys = 256;   // keys of a unit: two tiles of 128 lanes
constexpr int kWRows = 64;    // rows of a step
constexpr int kUnitCost = 2;  // cells of a unit besides its steps
constexpr int kLeast = 4;     // cells below which a share is not worth a CTA
constexpr int kSumWarps = 8, kKeyWarps = 4, kRowWarp = kSumWarps + kKeyWarps, kRowWarps = 3,
              kMmaWarp = kRowWarp + kRowWarps;
constexpr int kWThreads = (kMmaWarp + 1) * 32;
constexpr int kStages = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kColA = 0, kColD = 256, kCols = 512;  // keys: two buffers of two tiles; scores likewise

// The line of steps, from a cell on.
struct Line {
  int b, h, j;  // request, KV head, unit of 256 keys
  int seq, w, rows, units;
  int first, steps;  // the unit's first step, and how many it has
  long unit0, at, end;
  int s0, s1;  // the segment found: steps [s0, s1) of the unit

  __device__ __forceinline__ static int all_steps(int rows) { return max(1, (rows + kWRows - 1) / kWRows); }
  __device__ __forceinline__ void request(const WeighArgs& a) {
    Division<1, kWKeys>::lens(a, b, &seq, &w);
    rows = w > 0 ? w * a.G : 0;
    units = w < 0 ? 0 : (min(seq + w, a.T) + kWKeys - 1) / kWKeys;
  }
  // The first step with a row that sees a key of unit `x`.
  __device__ __forceinline__ int first_of(const WeighArgs& a, int x) const {
    return max(0, x * kWKeys - seq) * a.G / kWRows;
  }
  __device__ __forceinline__ void unit(const WeighArgs& a) {
    first = first_of(a, j);
    steps = all_steps(rows) - first;
  }
  // Units that every row sees the first key of: their steps are all.
  __device__ __forceinline__ int whole_units() const { return min(units, seq / kWKeys + 1); }
  // Cells of one KV head of the request.
  __device__ __forceinline__ long cells(const WeighArgs& a) const {
    const int whole = whole_units(), all = all_steps(rows);
    long n = (long)whole * (kUnitCost + all);
    for (int x = whole; x < units; ++x) n += kUnitCost + all - first_of(a, x);
    return n;
  }
  // To the next segment of the share; false at its end.
  __device__ __forceinline__ bool next(const WeighArgs& a) {
    for (;;) {
      if (at >= end) return false;
      const long unit1 = unit0 + kUnitCost + steps;
      if (at == unit1) {
        unit0 = unit1;
        if (++j == units) {
          j = 0;
          if (++h == a.c.H) {
            h = 0;
            do {
              if (++b == a.B) return false;
              request(a);
            } while (units == 0);
          }
        }
        unit(a);
        continue;
      }
      const long stop = min(end, unit1);
      s0 = first + (int)max(0l, at - unit0 - kUnitCost);
      s1 = first + (int)max(0l, stop - unit0 - kUnitCost);
      at = stop;
      if (s1 > s0) return true;
    }
  }
  __device__ __forceinline__ bool whole() const { return s0 == first && s1 == first + steps; }
};

// Sets `line` before the CTA's share (by all threads; one line in shared
// memory).  False: nothing to do.
__device__ __forceinline__ bool share(const WeighArgs& a, Line* line, Shares* shares) {
  __shared__ long long sWarp[kWThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + kWThreads - 1) / kWThreads, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  Line l = {};
  long long mine = 0;
  for (l.b = b0; l.b < b1; ++l.b) {
    l.request(a);
    mine += l.cells(a) * a.c.H;
  }
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(~0u, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) sWarp[warp] = incl;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int i = 0; i < kWThreads / 32; ++i) {
    if (i < warp) incl += sWarp[i];
    total += sWarp[i];
  }
  const long most = quotient(total, kLeast);
  const int ctas = most < 1 ? 1 : most < (long)gridDim.x ? (int)most : (int)gridDim.x;
  if (total == 0 || (int)blockIdx.x >= ctas) return false;
  Shares s;
  s.set(total, ctas);
  const long begin = s.begin(blockIdx.x);
  if (incl - mine <= begin && begin < incl) {  // one thread: its requests hold the share's first cell
    long at = incl - mine, head = 0;
    for (l.b = b0;; ++l.b) {
      l.request(a);
      head = l.cells(a);
      if (begin < at + head * a.c.H) break;
      at += head * a.c.H;
    }
    l.h = (int)quotient(begin - at, head);
    l.unit0 = at + l.h * head;
    const long whole = (long)l.whole_units() * (kUnitCost + Line::all_steps(l.rows));
    if (begin - l.unit0 < whole) {
      l.j = (int)quotient(begin - l.unit0, kUnitCost + Line::all_steps(l.rows));
      l.unit(a);
      l.unit0 += (long)l.j * (kUnitCost + l.steps);
    } else {
      l.unit0 += whole;
      l.j = l.whole_units();
      for (l.unit(a); begin >= l.unit0 + kUnitCost + l.steps; l.unit(a)) l.unit0 += kUnitCost + l.steps, ++l.j;
    }
    l.at = begin;
    l.end = s.begin(blockIdx.x + 1);
    *line = l;
    *shares = s;
  }
  __syncthreads();
  return true;
}

struct Bars {
  unsigned long long q_full[kStages], q_empty[kStages], a_full[2], a_empty[2], d_full[2], d_empty[2], end;
};

__host__ __device__ constexpr uint32_t instr_desc(bool bf16) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (uint32_t)(kWRows >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}

// What a key's position in its request's cache gives: decayed weight plus the window's.
__device__ __forceinline__ void put_sum(const WeighArgs& a, int b, int h, long t, int seq, float x) {
  const size_t at = ((size_t)b * a.c.H + h) * a.T + t;
  if (a.old && t < seq) x = fmaf(a.decay, a.old[at], x);
  a.sum[at] = x;
}

template <class T, int D>
__global__ void __launch_bounds__(kWThreads, 1) weigh_tiles_kernel(const WeighArgs a) {
  constexpr int kStage = kWRows * D * 2;  // bytes of a step's rows
  constexpr bool kBf = sizeof(T) == 2 && !__is_same(T, __half);
  extern __shared__ unsigned char smem_raw[];
  __shared__ Bars bars;
  __shared__ __align__(16) float sNeg[kStages][kWRows];  // -lse, -inf: no weight
  __shared__ int sSome[kStages];                         // some row has no weight
  __shared__ float sScale[2][kWKeys];
  __shared__ long sRow[kRowWarps][kWRows];  // where a step's rows lie, in elements of q; -1: no such row
  __shared__ Line sLine;
  __shared__ Shares sShares;
  __shared__ uint32_t sTmem;
  __shared__ int sDead;
  const KvCache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(&bars.q_full[i], 1);
      bar_init(&bars.q_empty[i], 1 + kSumWarps);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&bars.a_full[i], kKeyWarps);
      bar_init(&bars.a_empty[i], 1 + kSumWarps);
      bar_init(&bars.d_full[i], 1);
      bar_init(&bars.d_empty[i], kSumWarps);
    }
    bar_init(&bars.end, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    sDead = 0;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Tensor memory only now: see attend_tiles.cu.
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sTmem)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid < kDescWords) a.desc[blockIdx.x * kDescWords + tid] = -1;
  const bool work = share(a, &sLine, &sShares);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sTmem);
  volatile int* dead = &sDead;
  unsigned char* rows_s = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  Line v = sLine;
  // `n` counts steps and `seg` segments over the CTA's share.
  uint32_t n = 0, seg = 0;
  if (!work) {
  } else if (warp < kSumWarps) {
    const int key = tid;  // of the unit
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kColD + (warp >> 2) * kWRows;
    for (; v.next(a); ++seg) {
      bar_wait(&bars.a_full[seg & 1], (seg >> 1) & 1, dead);
      const float cs = sScale[seg & 1][key];
      __syncwarp();
      if (lane == 0) bar_arrive(&bars.a_empty[seg & 1]);
      const long t = (long)v.j * kWKeys + key, end = min((long)v.seq + v.w, (long)a.T);
      const long t0 = (long)v.j * kWKeys + (key & 128);  // the tile's first key
      const int from = (int)max(0l, min(t, end) - v.seq) * a.G;             // first row that sees the key,
      const int seen = (int)max(0l, min(t0 + 127, end - 1) - v.seq) * a.G;  // and that sees all of the tile's
      float sum = 0.f;
      for (int s = v.s0; s < v.s1; ++s, ++n) {
        const int st = n % kStages, r0 = s * kWRows;
        bar_wait(&bars.d_full[n & 1], (n >> 1) & 1, dead);
        bar_wait(&bars.q_full[st], (n / kStages) & 1, dead);
        fence_after();
        const bool plain = r0 >= seen && !sSome[st];
        float2 acc = make_float2(0.f, 0.f);  // a step's sum on its own: fewer roundings on the way
        if (t0 < end) {
          float x[kWRows];
          tmem_ld32(x, lanes + (n & 1) * 128);
          tmem_ld32(x + 32, lanes + (n & 1) * 128 + 32);
          tmem_wait_ld();
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&bars.d_empty[n & 1]);
          if (plain) {
            const float2 scale = make_float2(cs, cs), log2e = make_float2(kLog2e, kLog2e);
#pragma unroll
            for (int k = 0; k < kWRows; k += 4) {
              const float4 neg = *reinterpret_cast<const float4*>(&sNeg[st][k]);
              const float2 y = mul2(fma2(make_float2(x[k], x[k + 1]), scale, make_float2(neg.x, neg.y)), log2e);
              const float2 z = mul2(fma2(make_float2(x[k + 2], x[k + 3]), scale, make_float2(neg.z, neg.w)), log2e);
              acc = add2(acc, make_float2(ex2(y.x), ex2(y.y)));
              acc = add2(acc, make_float2(ex2(z.x), ex2(z.y)));
            }
          } else {
#pragma unroll
            for (int k = 0; k < kWRows; ++k) {
              const float neg = sNeg[st][k];
              const float e = ex2(fmaf(x[k], cs, neg) * kLog2e);
              if (r0 + k >= from && neg != -INFINITY) acc.x += e;
            }
          }
        } else {
          __syncwarp();
          if (lane == 0) bar_arrive(&bars.d_empty[n & 1]);
        }
        sum += acc.x + acc.y;
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.q_empty[st]);
      }
      if (cs != cs || *dead) sum = NAN;  // no such block
      if (v.whole()) {
        if (t < end) put_sum(a, v.b, v.h, t, v.seq, sum);
      } else {
        a.part[(2 * (size_t)blockIdx.x + (v.s0 == v.first)) * kWKeys + key] = sum;
        if (v.s0 == v.first && tid == 0) {
          int* d = a.desc + blockIdx.x * kDescWords;
          d[0] = v.b;
          d[1] = v.h;
          d[2] = v.j;
          d[3] = sShares.owner(v.unit0 + kUnitCost + v.steps - 1);
        }
      }
    }
  } else if (warp < kRowWarp) {
    // ---- a lane's two keys, 128 apart
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kColA;
    for (; v.next(a); ++seg) {
      const long end = min((long)v.seq + v.w, (long)a.T);
      const int32_t* table = c.tables + (size_t)v.b * c.max_blocks;
      uint32_t x[D / 4];
#pragma unroll 1
      for (int y = 0; y < kWKeys; y += 128) {
        const int key = y + (warp & 3) * 32 + lane;
        const long t = (long)v.j * kWKeys + key;
        const int col = (int)((unsigned)min(t, end - 1) / (unsigned)c.tpb);
        const int blk = table[col];
        const bool ok = t < end && blk >= 0 && blk < c.num_blocks;
        float scale = t < end ? NAN : 0.f;  // NaN: no such block
#pragma unroll
        for (int k = 0; k < D / 4; ++k) x[k] = 0;
        if (ok) {
          scale = a.scale * c.scales[c.scale_at(blk, 0, v.h)];
          const uint8_t* p = c.pool + c.row(blk, 0, v.h, (int)t - col * c.tpb);
#pragma unroll
          for (int k = 0; k < D / 32; ++k) load32(*reinterpret_cast<uint32_t(*)[8]>(&x[8 * k]), p + 32 * k);
        }
        if (y == 0) {
          bar_wait(&bars.a_empty[seg & 1], ((seg >> 1) & 1) ^ 1, dead);
          fence_after();
        }
        sScale[seg & 1][key] = scale;
#pragma unroll
        for (int k = 0; k < D / 4; k += 8) {
          uint32_t h[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) e4m3x4_to(x[k + e], h[2 * e], h[2 * e + 1], (T*)nullptr);
          tmem_st16(lanes + (seg & 1) * 128 + y / 2 + 2 * k, h);
        }
      }
      tmem_wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&bars.a_full[seg & 1]);
    }
  } else if (warp < kMmaWarp) {
    // ---- a lane: 16-byte vector lane % V of every kPer-th row, and two rows' place and lse
    constexpr int V = D / 8, kPer = 32 / V;
    const int mine = warp - kRowWarp, vec = lane % V, row = lane / V;
    const uint32_t at = smem_u32(rows_s) + (vec >> 3) * (kWRows * 128) + row * 128;
    uint32_t last = 0;  // the warp's step before, and its rows from its first on
    int left = 0;
    bool any = false;
    auto hand = [&]() {  // that step has arrived
      const int st = last % kStages;
      bool none = false;
#pragma unroll
      for (int r = lane; r < kWRows; r += 32) {
        const float l = sNeg[st][r], neg = r < left && l != -INFINITY ? -l : -INFINITY;
        sNeg[st][r] = neg;
        none = none || neg == -INFINITY;
      }
      none = __any_sync(~0u, none);
      if (lane == 0) sSome[st] = none;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive(&bars.q_full[st]);
    };
    for (; v.next(a); ++seg) {
      for (int s = v.s0; s < v.s1; ++s, ++n) {
        if (n % kRowWarps != mine) continue;
        const int st = n % kStages;
        bar_wait(&bars.q_empty[st], ((n / kStages) & 1) ^ 1, dead);
#pragma unroll
        for (int x = lane; x < kWRows; x += 32) {
          const int r = s * kWRows + x;
          const bool real = r < v.rows;
          const int i = real ? (unsigned)r / (unsigned)a.G : 0, g = real ? r - i * a.G : 0;
          sRow[mine][x] = real ? v.b * a.qb + i * a.qt + ((long)v.h * a.G + g) * a.qh : -1;
          cp4(smem_u32(&sNeg[st][x]), a.row_lse + ((size_t)v.b * a.W + i) * a.Hq + (size_t)v.h * a.G + g, real);
        }
        __syncwarp();
#pragma unroll 8
        for (int p = 0; p < kWRows / kPer; ++p) {
          const int r = p * kPer + row;
          const long from = sRow[mine][r];
          cp16(at + st * kStage + p * kPer * 128 + (((vec ^ r) & 7) << 4),
               a.q + (from == -1 ? 0 : 2 * (from + vec * 8)), from != -1);
        }
        __syncwarp();  // the places have been read by every lane: the next step writes them
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (any) {
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          hand();
        }
        any = true;
        last = n;
        left = v.rows - s * kWRows;
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (any) hand();
  } else {
    const uint64_t q_desc = smem_desc(smem_u32(rows_s), 16);
    for (; v.next(a); ++seg) {
      bar_wait(&bars.a_full[seg & 1], (seg >> 1) & 1, dead);
      const long end = min((long)v.seq + v.w, (long)a.T);
      const bool both = (long)v.j * kWKeys + 128 < end;
      for (int s = v.s0; s < v.s1; ++s, ++n) {
        const uint32_t st = n % kStages;
        if (n > 1) bar_wait(&bars.d_empty[n & 1], ((n >> 1) - 1) & 1, dead);
        bar_wait(&bars.q_full[st], (n / kStages) & 1, dead);
        fence_after();
        if (elect() && !*dead) {
          const uint64_t q = q_desc + st * (kStage >> 4);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            if (y && !both) break;
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ts(tmem + kColD + (n & 1) * 128 + y * kWRows, tmem + kColA + (seg & 1) * 128 + y * 64 + k * 8,
                     q + (k / 4) * (kWRows * 128 >> 4) + (k % 4) * (32 >> 4), instr_desc(kBf), k > 0);
          }
          mma_commit(&bars.q_empty[st]);
          mma_commit(&bars.d_full[n & 1]);
          if (s + 1 == v.s1) mma_commit(&bars.a_empty[seg & 1]);
        }
        __syncwarp();
      }
    }
    // every product has finished before tensor memory is given back
    if (elect()) mma_commit(&bars.end);
    __syncwarp();
    const long long begin = clock64();
    while (!bar_try(&bars.end, 0) && clock64() - begin < 4000000000ll) {
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
}

// Adds up the units that several CTAs worked on: CTA i the one that began in CTA i and did not end there.
__global__ void __launch_bounds__(kWKeys) weigh_join_kernel(const WeighArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int4 d = reinterpret_cast<const int4*>(a.desc)[2 * blockIdx.x];
  if (d.x < 0) return;
  int seq, w;
  Division<1, kWKeys>::lens(a, d.x, &seq, &w);
  const long t = (long)d.z * kWKeys + threadIdx.x;
  if (t >= min((long)seq + w, (long)a.T)) return;
  float x = a.part[(2 * (size_t)blockIdx.x + 1) * kWKeys + threadIdx.x];
  for (int i = blockIdx.x + 1; i <= d.w; ++i) x += a.part[2 * (size_t)i * kWKeys + threadIdx.x];
  put_sum(a, d.x, d.y, t, seq, x);
}

template <class T, int D>
cudaError_t launch(const WeighArgs& a, cudaStream_t st) {
  const size_t bytes = kStages * kWRows * D * 2 + 1024;  // 1024: alignment
  const cudaError_t e = cudaFuncSetAttribute(weigh_tiles_kernel<T, D>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  return e != cudaSuccess ? e : launch_first(weigh_tiles_kernel<T, D>, kSms, kWThreads, st, a, bytes);
}

}  // namespace

size_t weigh_tiles_scratch() { return align256((size_t)kSms * kDescWords * 4) + 2 * (size_t)kSms * kWKeys * 4; }

cudaError_t launch_weigh_tiles(WeighArgs& a, int dtype, void* scratch, cudaStream_t st) {
  a.desc = static_cast<int*>(scratch);
  a.part = reinterpret_cast<float*>(static_cast<char*>(scratch) + align256((size_t)kSms * kDescWords * 4));
  cudaError_t e;
  if (dtype == SPEC_BF16)
    e = a.c.D == 64 ? launch<__nv_bfloat16, 64>(a, st) : launch<__nv_bfloat16, 128>(a, st);
  else
    e = a.c.D == 64 ? launch<__half, 64>(a, st) : launch<__half, 128>(a, st);
  return e != cudaSuccess ? e : launch_first(weigh_join_kernel, kSms, kWKeys, st, a);
}

}  // namespace sv

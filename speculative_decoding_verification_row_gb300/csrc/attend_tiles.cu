// Attention for many rows per KV head (tree windows, grouped heads, prompt
// chunks): bound by the tensor cores.
//
// One CTA per SM, 128 rows x 128 keys a step, on tcgen05 (fp16 operands, fp32
// accumulators in tensor memory).  Warps by role:
//   0-7    softmax: two threads per row, one for each half of the tile's
//          keys (and of D).  Reads S from tensor memory, writes the weights P
//          back there as fp16, rescales O when a reference moves, and writes
//          the result.  Loads Q at a unit's start.
//   8      one thread issues S = Q K^T, Q in tensor memory, K in shared memory.
//   9      one thread issues O += P V, P in tensor memory, V in shared memory.
//          (Issuing takes as long as the product: with one warp for both, its
//          waits left the tensor cores idle half of the time.)  The warp also
//          looks up the pages and scales of the tiles to come.
//   10-15  read e4m3 rows of the pages, two tiles ahead in registers, and
//          write them as fp16 (exact) in the 128-byte swizzle.
// With both left operands in tensor memory a step reads 64 KB (D = 128) and
// writes 64 KB of shared memory, as long as its products take (1024 clocks);
// with Q in shared memory it would be 160 KB and shared memory the bound.
// Tensor memory: Q, S (two buffers; the weights replace the scores there), O.
//
// Scales, weights and lazy rescaling are as in attend_rows.cu, but that a V
// scale goes into the exponent whole, as its log2.
//
// Measured with 32 heads over 8 KV heads of 128: 16 trees of 60 tokens over
// 8192 positions 169 us, 770 TFLOP/s (0.40 of the measured dense rate; 16 of
// the 256 rows are empty); over 512 to 8192, 107 us.  A tile takes about 2200
// clocks where its products take 1024: the hops weights -> product -> scores of
// a row's chain, and the conversion of the pages, which the products wait for.
#include "attend.cuh"
#include "tcgen05.cuh"

namespace sv {

namespace {

constexpr int kRows = 128;
constexpr int kKeys = 128;
constexpr int kUnitCost = 4;             // cells of a unit besides its tiles
constexpr int kLeastCells = 4;              // a share below this is not worth a CTA: see attend_rows.cu
constexpr int kSoftWarps = 8, kScoreWarp = 8, kValueWarp = 9, kConvWarp = 10, kConvWarps = 6;
constexpr int kTThreads = (kConvWarp + kConvWarps) * 32;
constexpr int kConvThreads = kConvWarps * 32;
constexpr int kGroups = kKeys / 16;      // scale groups of a tile
constexpr int kRing = 16;                // tiles whose pages and scales are kept
constexpr int kAhead = 8;                // fewer than these are known ahead: more are looked up
constexpr uint32_t kColQ = 0, kColS = 128, kColO = 384, kCols = 512;

template <int D>
struct Tile {
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kBytes = kKeys * D * 2;  // one K (or V) tile as fp16
  static constexpr size_t kSmem = 2 * (size_t)kStages * kBytes + 1024;  // 1024: alignment
};

struct Bars {
  unsigned long long k_full[4], k_empty[4], v_full[4], v_empty[4];
  unsigned long long s_full[2], p_full[2], pv_done[2], q_full, pages[kRing], end;
};

// fp32 accumulator, fp16 operands, M = 128, N columns, B K-major or MN-major.
__host__ __device__ constexpr uint32_t instr_desc(int n, bool b_mn) {
  return 1u << 4 | (b_mn ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(kRows >> 4) << 24;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The two softmax warps of the same rows.
__device__ __forceinline__ void soft_sync() {  // all softmax warps
  asm volatile("barrier.cta.sync 5, %0;" ::"n"(kSoftWarps * 32) : "memory");
}
__device__ __forceinline__ void pair_sync(int warp) {
  asm volatile("barrier.cta.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory");
}

// Keys of a unit, from the first, that each of its rows sees.
__device__ __forceinline__ int seen_by_all(const AttendArgs& a, const Unit& u) {
  return u.seq + (a.masks ? 0 : u.mt * kRows / a.G + 1);
}

// Bit k: the row of window token i sees window place j + k (all of the prefix,
// j + k < 0, is seen).
__device__ __noinline__ unsigned seen_bits(const AttendArgs& a, const Unit& u, int i, long j) {
  if (!a.masks) {
    const long upto = min((long)i, (long)u.w - 1) - j;  // last place seen
    return upto >= 31 ? ~0u : upto < 0 ? 0u : (2u << upto) - 1;
  }
  const int32_t* row = a.masks + ((size_t)u.b * a.W + i) * a.words;
  unsigned bits = j >= 0 ? 0u : j <= -32 ? ~0u : (1u << -j) - 1;
#pragma unroll
  for (int y = 0; y < 2; ++y) {  // the two words that 32 places can straddle
    const long word = (j >> 5) + y;
    if (word < 0 || word * 32 >= u.w) continue;
    const int left = (int)(u.w - word * 32), shift = (int)(word * 32 - j);
    const unsigned m = (unsigned)row[word] & (left < 32 ? (1u << left) - 1 : ~0u);
    bits |= shift >= 32 ? 0u : shift >= 0 ? m << shift : m >> -shift;
  }
  return bits;
}

__device__ __forceinline__ void give_back(uint32_t tmem) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
}

template <class T, int D>
__global__ void __launch_bounds__(kTThreads, 1) attend_tiles_kernel(const AttendArgs a) {
  using TL = Tile<D>;
  constexpr int ST = TL::kStages;
  extern __shared__ unsigned char smem_raw[];
  __shared__ Bars bars;
  // of each 16-key group: K's scale, and log2 of V's
  __shared__ __align__(16) float sK[kRing][kGroups], sLog[kRing][kGroups];
  __shared__ const uint8_t* sPage[kRing][kGroups];  // K rows of each 16-key group
  __shared__ int sKeys[kRing], sPrefix[kRing], sFirst[kRing];  // see the lookup
  // what the two threads of a row tell each other
  __shared__ float2 sTop[2][2][kRows];
  __shared__ float sAux[2][2][kRows];
  // the walk of the softmax warps and that of the lookup; the segment that thread 0 found
  using Walker = Walk<kRows, kKeys, kUnitCost>;
  __shared__ Walker sWalk[2];
  __shared__ struct {
    Unit u;
    int tile0, tile1, whole, last, more;
  } sSeg;
  __shared__ uint32_t sTmem;
  __shared__ int sDead, sNan;
  const KvCache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      bar_init(&bars.k_full[i], kConvWarps);
      bar_init(&bars.v_full[i], kConvWarps);
      bar_init(&bars.k_empty[i], 1);
      bar_init(&bars.v_empty[i], 1);
    }
    bar_init(&bars.s_full[0], 1);
    bar_init(&bars.s_full[1], 1);
    // by a tile's parity: a warp may be a tile ahead of another, or two behind the products
    bar_init(&bars.p_full[0], kSoftWarps);
    bar_init(&bars.p_full[1], kSoftWarps);
    bar_init(&bars.pv_done[0], 1);
    bar_init(&bars.pv_done[1], 1);
    bar_init(&bars.q_full, kSoftWarps);
    for (int i = 0; i < kRing; ++i) bar_init(&bars.pages[i], 1);
    bar_init(&bars.end, 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    sDead = 0;
    sNan = 0;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Tensor memory only now: a kernel before this one that takes some after it has let its
  // dependents start would wait for these columns while the wait above waits for its end.
  if (warp == kScoreWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sTmem)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid < kDescWords) a.desc[blockIdx.x * kDescWords + tid] = -1;
  if (!divide<kRows, kKeys, kUnitCost, kTThreads>(a, kLeastCells, sWalk[0])) {
    if (warp == kScoreWarp) give_back(sTmem);
    return;
  }
  __syncthreads();  // every thread has stored the walk's beginning
  if (tid == 0) sWalk[1] = sWalk[0];
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sTmem);
  unsigned char* tiles = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  volatile int* dead = &sDead;
  using Div = Division<kRows, kKeys>;

  // The addresses are below 2^18: adding to the descriptor's low bits never carries out of them.
  const uint64_t k_desc = smem_desc(smem_u32(tiles), 16);
  const uint64_t v_desc = smem_desc(smem_u32(tiles) + ST * TL::kBytes, kKeys * 128);

  // `n` counts tiles over all segments of the CTA's share.
  uint32_t n = 0;
  if (warp < kSoftWarps) {
    const int half = warp >> 2, r = tid & (kRows - 1);
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    constexpr int HD = D / 2;  // elements of D that this thread serves
    // this thread's row of the segment's unit, and the scale of its scores
    int r0 = 0, rows = 0, i = 0, head = 0;
    float qs = 0.f;
    auto load_q = [&](const Unit& u) {
      r0 = u.mt * kRows;
      rows = min(kRows, (u.w < 0 ? a.W : u.w) * a.G - r0);
      i = r < rows ? (r0 + r) / a.G : 0;
      head = r < rows ? (r0 + r) % a.G : 0;
      if (u.w < 0) return;
      // ---- Q: a power of two per row, rounded to fp16, into tensor memory
      const uint4* qp = reinterpret_cast<const uint4*>(
          a.q + 2 * (u.b * a.qb + i * a.qt + ((long)u.h * a.G + head) * a.qh + half * HD));
      uint4 qv[HD / 8];
      float top = 0.f;
#pragma unroll
      for (int v = 0; v < HD / 8; ++v) qv[v] = r < rows ? qp[v] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int v = 0; v < HD / 8; ++v) {
        const uint32_t e[4] = {qv[v].x, qv[v].y, qv[v].z, qv[v].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = as_float2(e[k], (T*)nullptr);
          top = max3(top, fabsf(f.x), fabsf(f.y));
        }
      }
      sAux[0][half][r] = top;
      pair_sync(warp);
      top = fmaxf(top, sAux[0][half ^ 1][r]);
      int e2;
      frexpf(top, &e2);
      const int up = top > 0.f && top < INFINITY ? min(15 - e2, 126) : 0;
      const float f = copysignf(ldexpf(1.f, up), a.scale_log2);
      qs = fabsf(a.scale_log2) * ldexpf(1.f, -up);  // >= 0: maxima stay maxima
#pragma unroll
      for (int v = 0; v < HD / 32; ++v) {
        uint32_t h[16];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t e[4] = {qv[v * 4 + y].x, qv[v * 4 + y].y, qv[v * 4 + y].z, qv[v * 4 + y].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 p = as_float2(e[k], (T*)nullptr);
            h[y * 4 + k] = half2_of(p.x * f, p.y * f);
          }
        }
        tmem_st16(lanes + kColQ + half * (HD / 2) + v * 16, h);
      }
      tmem_wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&bars.q_full);
    };
    Unit u = {};
    int tile0 = 0, tile1 = 0, last = 0;
    bool whole = false, any = false;
    RowRef ref;
    float l = 0.f;
    auto finish = [&](int my_rows, int my_i, int my_head) {
      bool bad = u.w < 0;
      if (u.w >= 0) {
        if (tile1 == u.tiles) {  // a window block that these rows do not read is checked all the same
          const int32_t* table = c.tables + (size_t)u.b * c.max_blocks;
          bool miss = false;
          for (int x = (int)(u.seq / c.tpb) + lane; (long)x * c.tpb < (long)u.seq + u.w; x += 32)
            miss = miss || table[x] < 0 || table[x] >= c.num_blocks;
          bad = __any_sync(~0u, miss);
        }
        sAux[1][half][r] = l;
        pair_sync(warp);
        l += sAux[1][half ^ 1][r];
        bar_wait(&bars.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, dead);
        fence_after();
      }
      if (bad || *dead) l = NAN;
      // ---- the result, or this CTA's part of it
      const size_t orow = ((size_t)u.b * a.W + my_i) * a.Hq + (size_t)u.h * a.G + my_head;
      float* part = a.part + (2 * (size_t)blockIdx.x + (tile0 == 0)) * part_floats<kRows>(D);
      const float2 f = result_factors(l, ref.r);
      // the window tokens among this segment's keys, for NaN in V
      const long j0 = max(0l, (long)tile0 * kKeys - u.seq);
      const long j1 = sNan ? min((long)u.w, (long)tile1 * kKeys - u.seq) : 0;
#pragma unroll 1
      for (int x = half * HD; x < half * HD + HD; x += 32) {
        float o[32];
        if (u.w >= 0) {
          tmem_ld32(o, lanes + kColO + x);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0.f;
        }
        if (r < my_rows) {
          for (long j = j0; j < j1; ++j) {
            const bool see = a.masks ? a.masks[((size_t)u.b * a.W + my_i) * a.words + (j >> 5)] >> (j & 31) & 1
                                     : j <= my_i;
            const int blk = see ? c.block(u.b, u.seq + j) : -1;
            if (blk < 0) continue;
            const uint32_t* v = reinterpret_cast<const uint32_t*>(
                c.pool + c.row(blk, 1, u.h, (int)((u.seq + j) % c.tpb)) + x);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t nb = nan_bytes(v[k]);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (nb >> (8 * e + 7) & 1) o[k * 4 + e] = NAN;
            }
          }
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + 2 * (orow * D + x));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                y[e] = pack_out(o[k * 8 + e * 2] * f.x * f.y, o[k * 8 + e * 2 + 1] * f.x * f.y, (T*)nullptr);
              dst[k] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 32; k += 8)  // whole sectors: every lane has a row of its own
              asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(part + (size_t)r * D + x + k),
                           "f"(o[k]), "f"(o[k + 1]), "f"(o[k + 2]), "f"(o[k + 3]), "f"(o[k + 4]), "f"(o[k + 5]),
                           "f"(o[k + 6]), "f"(o[k + 7])
                           : "memory");
          }
        }
        __syncwarp();
      }
      if (r < my_rows && half == 0) {
        if (whole) {
          if (a.lse) a.lse[orow] = row_lse(ref.m, l);
        } else {
          part[(size_t)kRows * D + r] = ref.m;
          part[(size_t)kRows * (D + 1) + r] = ref.r;
          part[(size_t)kRows * (D + 2) + r] = l;
        }
      }
      if (!whole && tile0 == 0 && tid == 0) {
        int* d = a.desc + blockIdx.x * kDescWords;
        d[0] = u.b;
        d[1] = u.h;
        d[2] = u.mt;
        d[3] = last;
        d[4] = my_rows;
      }
      fence_before();  // O has been read: the next unit's first product follows this thread's p_full
    };
    // Segment by segment; the next one's Q goes in before this one's result
    // comes out: its first scores are computed meanwhile (all of this one's are
    // done).
    auto find_next = [&]() {
      Walker& v = sWalk[0];
      sSeg.more = v.next(a);
      sSeg.u = v.u;
      sSeg.tile0 = v.tile0;
      sSeg.tile1 = v.tile1;
      sSeg.whole = v.whole();
      sSeg.last = v.tile0 == 0 && !v.whole() && sSeg.more ? v.last_cta() : 0;
    };
    if (tid == 0) find_next();
    for (;;) {
      soft_sync();
      const bool more = sSeg.more;
      const int my_rows = rows, my_i = i, my_head = head;
      if (more) load_q(sSeg.u);
      if (any) finish(my_rows, my_i, my_head);
      if (!more) break;
      u = sSeg.u;
      tile0 = sSeg.tile0, tile1 = sSeg.tile1, last = sSeg.last;
      whole = sSeg.whole;
      any = true;
      soft_sync();  // sSeg has been read
      if (tid == 0) find_next();
      ref = RowRef{}, l = 0.f;
      if (u.w < 0) continue;
      for (int tile = tile0; tile < tile1; ++tile, ++n) {
        const int ring = n % kRing;
        bar_wait(&bars.pages[ring], (n / kRing) & 1, dead);
        const float4 k4 = reinterpret_cast<const float4*>(sK[ring])[half];
        const float4 log4 = reinterpret_cast<const float4*>(sLog[ring])[half];
        float kf[4] = {k4.x * qs, k4.y * qs, k4.z * qs, k4.w * qs};
        const float lv[4] = {log4.x, log4.y, log4.z, log4.w};
#pragma unroll
        for (int y = 0; y < 4; ++y)  // -inf times it stays -inf; NaN (no such block) stays NaN
          kf[y] = kf[y] < 0x1p-120f ? 0x1p-120f : kf[y];
        bar_wait(&bars.s_full[n & 1], (n >> 1) & 1, dead);
        fence_after();
        float s[64];
        tmem_ld32(s, lanes + kColS + (n & 1) * kKeys + half * 64);
        tmem_ld32(s + 32, lanes + kColS + (n & 1) * kKeys + half * 64 + 32);
        tmem_wait_ld();
        const long k0 = (long)tile * kKeys + half * 64 - u.seq;  // window place of s[0]
        if ((tile + 1) * kKeys > seen_by_all(a, u)) {
#pragma unroll
          for (int x = 0; x < 64; x += 32) {
            const unsigned bits = seen_bits(a, u, i, k0 + x);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!(bits >> k & 1)) s[x + k] = -INFINITY;
          }
        }
        float2 top = make_float2(-INFINITY, -INFINITY);  // largest score, and with V's scale
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
          for (int k = 0; k < 16; k += 4) {
            t0 = max3(t0, s[y * 16 + k], s[y * 16 + k + 1]);
            t1 = max3(t1, s[y * 16 + k + 2], s[y * 16 + k + 3]);
          }
          const float t = fmaxf(t0, t1) * kf[y];
          top = make_float2(fmaxf(top.x, t), fmaxf(top.y, t + lv[y]));
        }
        sTop[n & 1][half][r] = top;
        pair_sync(warp);
        const float2 other = sTop[n & 1][half ^ 1][r];
        top = make_float2(fmaxf(top.x, other.x), fmaxf(top.y, other.y));
        if (__any_sync(~0u, top.x > ref.m + kLazy || top.y > ref.m + ref.r + kLazy)) {
          float fl, fo;
          ref.move(top.x, top.y, &fl, &fo);
          l *= fl;
          if (tile > tile0 && __any_sync(~0u, fo != 1.f)) {
            bar_wait(&bars.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, dead);
            fence_after();
#pragma unroll 1
            for (int x = half * HD; x < half * HD + HD; x += 16) {
              uint32_t o[16];
              tmem_ld16(o, lanes + kColO + x);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fo);
              tmem_st16(lanes + kColO + x, o);
            }
          }
        }
        // V's scale goes into the exponent, and out of the sum again
        const float add = kPBits - ref.m;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          uint32_t p[16];
#pragma unroll
          for (int y = 2 * z; y < 2 * z + 2; ++y) {
            const float depth = ref.depth(lv[y]), av = add - depth;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const int x = y * 16 + k;
              float2 e = fma2(make_float2(s[x], s[x + 1]), make_float2(kf[y], kf[y]), make_float2(av, av));
              e = make_float2(ex2(e.x), ex2(e.y));
              sum = add2(sum, e);
              p[(x & 31) / 2] = weights_f16(e.x, e.y);
            }
            l = fmaf(sum.x + sum.y, ex2(depth), l);
          }
          // over this thread's scores, all of which it has read
          tmem_st16(lanes + kColS + (n & 1) * kKeys + half * 64 + z * 16, p);
        }
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.p_full[n & 1]);
      }
    }
  } else if (warp == kScoreWarp) {
    for (uint32_t seg = 0;; ++n) {
      const int at = n % kRing;
      bar_wait(&bars.pages[at], (n / kRing) & 1, dead);
      if (sKeys[at] == 0 || *dead) break;
      if (sFirst[at]) {
        bar_wait(&bars.q_full, seg & 1, dead);
        ++seg;
      }
      // the buffer is free when the product with the weights that lay in it is done
      if (n > 1) bar_wait(&bars.pv_done[n & 1], ((n >> 1) - 1) & 1, dead);
      const uint32_t st = n % ST;
      bar_wait(&bars.k_full[st], (n / ST) & 1, dead);
      fence_after();
      if (elect() && !*dead) {
        const uint32_t d = tmem + kColS + (n & 1) * kKeys;
        const uint64_t b = k_desc + st * (TL::kBytes >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ts(d, tmem + kColQ + k * 8, b + (k / 4) * (kKeys * 128 >> 4) + (k % 4) * (32 >> 4),
                 instr_desc(kKeys, false), k > 0);
        mma_commit(&bars.k_empty[st]);
        mma_commit(&bars.s_full[n & 1]);
      }
      __syncwarp();
    }
  } else if (warp == kValueWarp) {
    // ---- the lookup, up to four tiles of a segment at a time: block ids, then
    // scales, then the ring, a call apart each, so that no use waits for its
    // load.  Lane x: group x % 8 of the batch's tile x / 8.
    // the walk's segment: lane 0 walks, all copy
    Walker& v = sWalk[1];
    Unit u = {};
    int tile = 0, tile0 = 0, tile1 = 0, keys = 0;
    bool more = true;
    const int my_tile = lane >> 3;
    // stage 1: block ids under way
    int blk = 0, grp1 = 0, unit_h = 0, count1 = 0, keys1 = 0, all1 = 0;
    bool first1 = false, keyed1 = false;  // keyed1: the lane's group has keys, blk is a table entry
    // stage 2: scales under way
    const uint8_t* page = nullptr;
    float k_scale = 0.f, v_scale = 0.f;
    int count2 = 0, keys2 = 0, all2 = 0;
    bool first2 = false;
    uint32_t posted = 0;
    bool ended = false;
    auto lookup = [&](bool post) {
      if (post && !ended) {
        float vf;
        const float ve = scale_exponent(v_scale, &vf);
        const int at = (posted + my_tile) % kRing, g = lane & 7;
        if (my_tile < count2) {
          sPage[at][g] = page;
          sK[at][g] = k_scale;
          sLog[at][g] = vf == 1.f ? ve : vf > 0.f ? ve + __log2f(vf) : -150.f;  // 448 * 2^-150 is 0 in any output
        }
        // keys of the tile, those that every row sees, and whether a segment begins;
        // no keys: the share has ended
        if (g == 0 && my_tile < max(count2, 1)) {
          sKeys[at] = count2 == 0 ? 0 : min(kKeys, keys2 - my_tile * kKeys);
          sPrefix[at] = max(0, min(kKeys, all2 - my_tile * kKeys));
          sFirst[at] = first2 && my_tile == 0;
        }
        __syncwarp();
        if (g == 0 && my_tile < max(count2, 1)) bar_arrive(&bars.pages[at]);
        ended = count2 == 0;
        posted += max(count2, 1);
      }
      // a block that does not exist: block 0 is read, and the scores are NaN
      const bool ok = keyed1 && (unsigned)blk < (unsigned)c.num_blocks;
      const int off = ok ? (int)(grp1 - col16(a, grp1) * (c.tpb / 16)) * 16 : 0;
      page = c.pool + ((((size_t)(ok ? blk : 0) * 2) * c.H + unit_h) * c.tpb + off) * D;
      k_scale = keyed1 ? NAN : 0.f;
      v_scale = 0.f;
      if (ok) {
        const float* sp = c.scales + c.scale_at(blk, 0, unit_h);
        k_scale = sp[0];
        v_scale = sp[c.H];
      }
      count2 = count1, keys2 = keys1, all2 = all1, first2 = first1;
      count1 = 0;
      keyed1 = false;
      while (more && tile == tile1) {  // a new segment; those without keys are skipped
        bool left = false;
        if (lane == 0) left = v.next(a);
        more = __shfl_sync(~0u, left, 0);
        __syncwarp();
        u = v.u;
        tile = tile0 = v.tile0;
        tile1 = more && u.w >= 0 ? v.tile1 : tile0;
        keys = (int)Div::seen(a, u.seq, u.w, u.mt);
        __syncwarp();
      }
      if (more) {
        const int k0 = tile * kKeys;
        count1 = min(4, tile1 - tile);
        keys1 = keys - k0;
        all1 = seen_by_all(a, u) - k0;
        first1 = tile == tile0;
        unit_h = u.h;
        grp1 = tile * kGroups + lane;
        keyed1 = my_tile < count1 && grp1 * 16 < keys;
        if (keyed1) blk = c.tables[(size_t)u.b * c.max_blocks + col16(a, grp1)];
        tile += count1;
      }
    };
    // One loop, so that the lookup is in the code once: calls -2 and -1 fill its
    // stages, those up to `ready` the ring, the others go between the products.
    int calls = -2;
    bool ready = false;
    for (;;) {
      if (!ended && posted < n + kAhead) {
        lookup(calls >= 0);  // while the next weights are computed
        ++calls;
        if (!ready) continue;
      }
      ready = true;
      if (sKeys[n % kRing] == 0 || *dead) break;
      const uint32_t st = n % ST;
      bar_wait(&bars.v_full[st], (n / ST) & 1, dead);
      bar_wait(&bars.p_full[n & 1], (n >> 1) & 1, dead);
      fence_after();
      if (elect() && !*dead) {
        const bool add = sFirst[n % kRing] == 0;
        const uint32_t p = tmem + kColS + (n & 1) * kKeys;  // 32 columns, and 32 from the 64th on
        const uint64_t b = v_desc + st * (TL::kBytes >> 4);
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          mma_ts(tmem + kColO, p + k / 4 * 64 + k % 4 * 8, b + k * (2048 >> 4), instr_desc(D, true),
                 add || k > 0);
        mma_commit(&bars.v_empty[st]);
        mma_commit(&bars.pv_done[n & 1]);
      }
      __syncwarp();
      ++n;
    }
  } else {
    // ---- Thread t of the converters: chunk ch (32 bytes) of rows row + kPer p.
    // Eight neighbours hold two chunks of four rows, one atom's, which keeps
    // their 16-byte stores below off each other's banks.
    constexpr int CPR = D / 32, kPer = kConvThreads / CPR, NP = (kKeys + kPer - 1) / kPer;
    static_assert(kConvThreads % CPR == 0 && kPer % 8 == 0, "converter layout");
    const int t = tid - kConvWarp * 32;
    const int ch = D == 128 ? (t & 1) | (t >> 2 & 2) : t & 1;
    const int row = D == 128 ? (t >> 1 & 3) | t >> 4 << 2 : t >> 1;
    const size_t v_off = (size_t)c.H * c.tpb * D;  // from a block's K rows to its V rows
    // the rows of tile `at`; false behind the last
    auto load = [&](uint32_t (&x)[NP][8], uint32_t (&y)[NP][8], uint32_t at) {
      bar_wait(&bars.pages[at % kRing], (at / kRing) & 1, dead);
      if (sKeys[at % kRing] == 0 || *dead) return false;
      const uint8_t* const* page = sPage[at % kRing];
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int r = p * kPer + row;
        if (p * kPer + kPer <= kKeys || r < kKeys) {
          const uint8_t* src = page[r >> 4] + ((r & 15) * D + ch * 32);
          load32(x[p], src);
          load32(y[p], src + v_off);
        }
      }
      return true;
    };
    // places of the four fp16 vectors of row `row` (kPer is a multiple of the swizzle's 8 rows)
    const int atom = (ch >> 1) * (kKeys * 128) + row * 128, c0 = (ch & 1) * 4;
    auto put = [&](const uint32_t (&x)[NP][8], unsigned char* tile) {
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        if (p * kPer + kPer <= kKeys || p * kPer + row < kKeys) {
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint32_t h[4];
            e4m3x4_to_half(x[p][2 * s], h[0], h[1]);
            e4m3x4_to_half(x[p][2 * s + 1], h[2], h[3]);
            *reinterpret_cast<uint4*>(tile + p * kPer * 128 + atom + (((c0 + s) ^ (row & 7)) << 4)) =
                make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    };
    // Writes tile n and starts to load tile n + 2 into the same registers:
    // two tiles are on their way while a third is written.
    auto step = [&](uint32_t (&kr)[NP][8], uint32_t (&vr)[NP][8], bool follows) {
      const uint32_t st = n % ST;
      bar_wait(&bars.k_empty[st], ((n / ST) & 1) ^ 1, dead);
      put(kr, tiles + st * TL::kBytes);
      if (lane == 0) bar_arrive(&bars.k_full[st]);
      const int keys = sKeys[n % kRing], prefix = sPrefix[n % kRing];
      if (prefix < kKeys) {
        // Rows behind the keys hold anything; they are zero here.  NaN in a key
        // that not every row sees: only those that do may get it (see the result).
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int key = p * kPer + row;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t nb = key >= keys ? 0x80808080u : key >= prefix ? nan_bytes(vr[p][k]) : 0u;
            if (nb && key < keys) sNan = 1;
            vr[p][k] &= ~((nb >> 7) * 255u);
          }
        }
      }
      bar_wait(&bars.v_empty[st], ((n / ST) & 1) ^ 1, dead);
      put(vr, tiles + (ST + st) * TL::kBytes);
      if (lane == 0) bar_arrive(&bars.v_full[st]);
      ++n;
      return follows && load(kr, vr, n + 1);
    };
    uint32_t ka[NP][8], va[NP][8], kb[NP][8], vb[NP][8];
    bool in_a = load(ka, va, 0), in_b = in_a && load(kb, vb, 1);
    while (in_a) {
      in_a = step(ka, va, in_b);
      if (!in_b) break;
      in_b = step(kb, vb, in_a);
    }
  }

  // Every product has finished before tensor memory is given back.
  if (warp == kScoreWarp || warp == kValueWarp) {
    if (elect()) mma_commit(&bars.end);
    __syncwarp();
  }
  if (warp == kScoreWarp) {
    const long long begin = clock64();
    while (!bar_try(&bars.end, 0) && clock64() - begin < 4000000000ll) {
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kScoreWarp) give_back(tmem);
}

}  // namespace

size_t attend_tiles_scratch(int D) {
  return align256((size_t)kSms * kDescWords * 4) + 2 * (size_t)kSms * part_floats<kRows>(D) * 4;
}

namespace {

template <class T, int D>
cudaError_t launch_tiles(const AttendArgs& a, cudaStream_t st) {
  const auto kernel = attend_tiles_kernel<T, D>;
  const size_t bytes = Tile<D>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSms);
  cfg.blockDim = dim3(kTThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e != cudaSuccess) return e;
  return launch_join<T, D, kRows>(a, kSms, st);
}

}  // namespace

cudaError_t launch_attend_tiles(AttendArgs& a, int dtype, void* scratch, cudaStream_t st) {
  a.mtiles = ceil_div((long)a.W * a.G, kRows);
  a.desc = static_cast<int*>(scratch);
  a.part = reinterpret_cast<float*>(static_cast<char*>(scratch) + align256((size_t)kSms * kDescWords * 4));
  if (dtype == SPEC_BF16)
    return a.c.D == 64 ? launch_tiles<__nv_bfloat16, 64>(a, st) : launch_tiles<__nv_bfloat16, 128>(a, st);
  return a.c.D == 64 ? launch_tiles<__half, 64>(a, st) : launch_tiles<__half, 128>(a, st);
}

}  // namespace sv

// Attention for many rows per KV head (tree windows, grouped heads, prompt
// chunks): bound by the tensor cores.
//
// One CTA per SM, 128 rows x 128 keys a step, on tcgen05 (fp16 operands, fp32
// accumulators in tensor memory).  Warps by role:
//   0-3    softmax: thread = row.  Reads S from tensor memory, writes the
//          weights P back there as fp16, rescales O when the maximum moves by
//          more than 2^7, and writes the result.  Loads Q at a unit's start.
//   4      one thread issues the products: S = Q K^T with Q in tensor memory,
//          O += P V with P in tensor memory, K and V in shared memory.
//   5-12   read e4m3 rows of the pages, one tile ahead in registers, and
//          write them as fp16 (exact) in the 128-byte swizzle.
// With both left operands in tensor memory a step reads 64 KB (D = 128) and
// writes 64 KB of shared memory, as long as its products take (1024 clocks);
// with Q in shared memory it would be 160 KB and shared memory the bound.
// Tensor memory: Q, P (one buffer), S (two buffers), O: 512 columns, all.
//
// Scales, weights and lazy rescaling are as in attend_rows.cu.
#include "attend.cuh"

namespace sv {

namespace {

constexpr int kRows = 128;
constexpr int kKeys = 128;
constexpr int kLeastTiles = 2;
constexpr int kSoftWarps = 4, kMmaWarp = 4, kConvWarp = 5, kConvWarps = 8;
constexpr int kTThreads = (kConvWarp + kConvWarps) * 32;
constexpr int kConvThreads = kConvWarps * 32;
constexpr int kGroups = kKeys / 16;      // scale groups of a tile
constexpr int kScaleRing = 8;            // tiles whose scales are kept; more than any role runs ahead
using Div = Division<kRows, kKeys>;

constexpr uint32_t kColQ = 0, kColP = 64, kColS = 128, kColO = 384, kCols = 512;

template <int D>
struct Tile {
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kBytes = kKeys * D * 2;  // one K (or V) tile as fp16
  static constexpr size_t kSmem = 2 * (size_t)kStages * kBytes + 1024;  // 1024: alignment
};

struct Bars {
  unsigned long long k_full[4], k_empty[4], v_full[4], v_empty[4];
  unsigned long long s_full[2], p_full, pv_done, q_full, scales[kScaleRing], end;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void bar_init(unsigned long long* b, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(unsigned long long* b) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ bool bar_try(unsigned long long* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the phase, about two seconds at most; after that *dead is set and
// no wait of the CTA waits any longer: it ends, and its rows read NaN.
__device__ __noinline__ void bar_wait_slow(unsigned long long* b, uint32_t parity, volatile int* dead) {
  const long long begin = clock64();
  while (!bar_try(b, parity)) {
    if (*dead) return;
    if (clock64() - begin > 4000000000ll) {
      *dead = 1;
      return;
    }
  }
}
__device__ __forceinline__ void bar_wait(unsigned long long* b, uint32_t parity, volatile int* dead) {
  if (!bar_try(b, parity)) bar_wait_slow(b, parity, dead);
}

__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_commit(unsigned long long* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}

// Shared memory descriptor, 128-byte swizzle.  K-major (K^T): 8 rows of 128
// bytes are an atom, atoms 1024 bytes apart along the keys.  MN-major (V):
// an atom is 64 elements of d by 8 keys, atoms 1024 bytes apart along the
// keys and `lead` bytes along d.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// fp32 accumulator, fp16 operands, M = 128, N columns, B K-major or MN-major.
__host__ __device__ constexpr uint32_t instr_desc(int n, bool b_mn) {
  return 1u << 4 | (b_mn ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(kRows >> 4) << 24;
}

__device__ __forceinline__ void e4m3x4_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t half2_of(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}
__device__ __forceinline__ float2 as_float2(uint32_t w, __nv_bfloat16*) {
  return make_float2(bf16_lo(w), bf16_hi(w));
}
__device__ __forceinline__ float2 as_float2(uint32_t w, __half*) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <class T, int D>
__global__ void __launch_bounds__(kTThreads, 1) attend_tiles_kernel(const AttendArgs a) {
  using TL = Tile<D>;
  constexpr int ST = TL::kStages;
  extern __shared__ unsigned char smem_raw[];
  __shared__ Bars bars;
  __shared__ long long sPre[kTThreads + 1];
  __shared__ float sK[kScaleRing][kGroups], sV[kScaleRing][kGroups];
  __shared__ uint32_t sTmem;
  __shared__ int sDead, sNan;
  const KvCache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid < kDescWords) a.desc[blockIdx.x * kDescWords + tid] = -1;
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      bar_init(&bars.k_full[i], kConvWarps);
      bar_init(&bars.v_full[i], kConvWarps);
      bar_init(&bars.k_empty[i], 1);
      bar_init(&bars.v_empty[i], 1);
    }
    bar_init(&bars.s_full[0], 1);
    bar_init(&bars.s_full[1], 1);
    bar_init(&bars.p_full, kSoftWarps);
    bar_init(&bars.pv_done, 1);
    bar_init(&bars.q_full, kSoftWarps);
    for (int i = 0; i < kScaleRing; ++i) bar_init(&bars.scales[i], 1);
    bar_init(&bars.end, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    sDead = 0;
    sNan = 0;
  }
  Unit u;
  long t0, t1, unit0, total;
  int ctas;
  if (!divide<kRows, kKeys, kTThreads>(a, kLeastTiles, sPre, u, &t0, &t1, &unit0, &total, &ctas))
    return;
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sTmem)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sTmem);
  unsigned char* tiles = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  volatile int* dead = &sDead;

  // Every role walks the same segments; `n` counts tiles over all of them.
  uint32_t n = 0, seg = 0;
  for (long at = t0; at < t1; ++seg) {
    const long stop = min(t1, unit0 + u.tiles);
    const int tile0 = (int)(at - unit0), tile1 = (int)(stop - unit0);
    const long keys = u.w < 0 ? 0 : Div::seen(a, u.seq, u.w, u.mt);

    if (warp < kSoftWarps) {
      const int r0 = u.mt * kRows, r = tid;
      const int w = u.w < 0 ? a.W : u.w;
      const int rows = (int)min((long)kRows, (long)w * a.G - r0);
      const int i = r < rows ? (r0 + r) / a.G : 0, head = r < rows ? (r0 + r) % a.G : 0;
      const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
      float m = -INFINITY, l = 0.f, vref = 0.f;
      bool bad = u.w < 0;
      if (u.w >= 0) {
        // ---- Q: a power of two per row, rounded to fp16, into tensor memory
        const uint4* qp = reinterpret_cast<const uint4*>(
            a.q + 2 * (u.b * a.qb + i * a.qt + ((long)u.h * a.G + head) * a.qh));
        float top = 0.f;
#pragma unroll 4
        for (int v = 0; v < D / 8; ++v) {
          const uint4 x = r < rows ? qp[v] : make_uint4(0, 0, 0, 0);
          const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = as_float2(e[k], (T*)nullptr);
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
        int e2;
        frexpf(top, &e2);
        const int up = top > 0.f && top < INFINITY ? min(15 - e2, 126) : 0;
        const float f = copysignf(ldexpf(1.f, up), a.scale_log2);
        const float qs = fabsf(a.scale_log2) * ldexpf(1.f, -up);  // >= 0: maxima stay maxima
#pragma unroll
        for (int v = 0; v < D / 32; ++v) {
          uint32_t h[16];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint4 x = r < rows ? qp[v * 4 + y] : make_uint4(0, 0, 0, 0);
            const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 p = as_float2(e[k], (T*)nullptr);
              h[y * 4 + k] = half2_of(p.x * f, p.y * f);
            }
          }
          tmem_st16(lanes + kColQ + v * 16, h);
        }
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.q_full);

        for (int tile = tile0; tile < tile1; ++tile, ++n) {
          const int ring = n % kScaleRing;
          bar_wait(&bars.scales[ring], (n / kScaleRing) & 1, dead);
          const uint32_t s_addr = lanes + kColS + (n & 1) * kKeys;
          bar_wait(&bars.s_full[n & 1], (n >> 1) & 1, dead);
          fence_after();
          const long k0 = (long)tile * kKeys;
          const bool edge = k0 + kKeys > u.seq;
          // the window tokens that this row sees among keys [x, x + 32) of the tile
          auto seen32 = [&](int x) {
            const long j = k0 + x - u.seq;  // window place of key x
            unsigned bits = 0;
            if (a.masks) {
              const int32_t* row = a.masks + ((size_t)u.b * a.W + i) * a.words;
              const int left = u.w;
#pragma unroll
              for (int y = 0; y < 2; ++y) {  // the two words that the 32 places can straddle
                const long wd = (j >> 5) + y;
                if (wd >= 0 && wd * 32 < left) {
                  unsigned m32 = (unsigned)row[wd];
                  if (left - wd * 32 < 32) m32 &= (1u << (left - wd * 32)) - 1;
                  const int sh = (int)(wd * 32 - j);  // place of the word's bit 0
                  bits |= sh >= 32 ? 0u : sh >= 0 ? m32 << sh : m32 >> -sh;
                }
              }
              if (j < 0) bits |= j <= -32 ? ~0u : (1u << -j) - 1;
            } else {
              const long upto = min((long)i, (long)u.w - 1) - j;  // last place seen
              bits = upto >= 31 ? ~0u : upto < 0 ? 0u : (2u << upto) - 1;
            }
            return bits;
          };
          // ---- the tile's largest score, V scale
          float top = -INFINITY, vmax = 0.f;
#pragma unroll
          for (int x = 0; x < kKeys; x += 32) {
            uint32_t s[32];
            tmem_ld32(s, s_addr + x);
            tmem_wait_ld();
            if (edge) {
              const unsigned bits = seen32(x);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(bits >> k & 1)) s[k] = 0xff800000u;
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float t = -INFINITY;
#pragma unroll
              for (int k = 0; k < 16; ++k) t = fmaxf(t, __uint_as_float(s[y * 16 + k]));
              const int grp = x / 16 + y;
              vmax = fmaxf(vmax, sV[ring][grp]);
              const float kf = qs * sK[ring][grp];
              if (t > -INFINITY) top = fmaxf(top, t * kf);
            }
          }
          const bool move = top > m + kLazy;
          const bool wide = vmax > vref;
          if (__any_sync(~0u, move || wide)) {
            const float now = move ? top : m;
            const float al = move ? ex2(m - now) : 1.f;
            const float ar = al * (wide ? vref / vmax : 1.f);
            m = now;
            l *= al;
            if (wide) vref = vmax;
            if (tile > tile0) {
              bar_wait(&bars.pv_done, (n - 1) & 1, dead);
              fence_after();
#pragma unroll 1
              for (int x = 0; x < D; x += 32) {
                uint32_t o[32];
                tmem_ld32(o, lanes + kColO + x);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * ar);
                tmem_st32(lanes + kColO + x, o);
              }
            }
          }
          const float sub = m == -INFINITY ? 0.f : m - kPBits;
          const float inv_vref = vref > 0.f ? 1.f / vref : 0.f;
          // P has one buffer: the last tile's product has read it
          if (n > 0) bar_wait(&bars.pv_done, (n - 1) & 1, dead);
          fence_after();
#pragma unroll
          for (int x = 0; x < kKeys; x += 32) {
            uint32_t s[32], p[16];
            tmem_ld32(s, s_addr + x);
            tmem_wait_ld();
            if (edge) {
              const unsigned bits = seen32(x);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(bits >> k & 1)) s[k] = 0xff800000u;
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int grp = x / 16 + y;
              const float kf = qs * sK[ring][grp];
              const float vr = sV[ring][grp] * inv_vref;
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                const float s0 = __uint_as_float(s[y * 16 + k]), s1 = __uint_as_float(s[y * 16 + k + 1]);
                // a masked score stays -inf under a scale of zero
                const float e0 = ex2(s0 == -INFINITY ? s0 : fmaf(s0, kf, -sub));
                const float e1 = ex2(s1 == -INFINITY ? s1 : fmaf(s1, kf, -sub));
                l += e0 + e1;
                p[y * 8 + k / 2] = half2_of(e0 * vr, e1 * vr);
              }
            }
            tmem_st16(lanes + kColP + x / 2, p);
          }
          tmem_wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&bars.p_full);
        }
        if (tile1 == u.tiles) {  // a window block that these rows do not read is checked all the same
          const int32_t* table = c.tables + (size_t)u.b * c.max_blocks;
          bool miss = false;
          for (int x = (int)(u.seq / c.tpb) + lane; (long)x * c.tpb < u.seq + u.w; x += 32)
            miss = miss || table[x] < 0 || table[x] >= c.num_blocks;
          bad = __any_sync(~0u, miss);
        }
        bar_wait(&bars.pv_done, (n - 1) & 1, dead);
        fence_after();
      }
      if (bad || *dead) l = NAN;
      // ---- the result, or this CTA's part of it
      const bool whole = tile0 == 0 && tile1 == u.tiles;
      const size_t orow = ((size_t)u.b * a.W + i) * a.Hq + (size_t)u.h * a.G + head;
      float* part = a.part + (2 * (size_t)blockIdx.x + (tile0 == 0)) * part_floats<kRows>(D);
      const float f = whole ? (l == 0.f ? 0.f : vref / l) : vref;
      // the window tokens among this segment's keys, for NaN in V
      const long j0 = max(0l, (long)tile0 * kKeys - u.seq);
      const long j1 = sNan ? min((long)u.w, (long)tile1 * kKeys - u.seq) : 0;
#pragma unroll 1
      for (int x = 0; x < D; x += 32) {
        uint32_t o[32];
        if (u.w >= 0) {
          tmem_ld32(o, lanes + kColO + x);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0;
        }
        if (r < rows) {
          for (long j = j0; j < j1; ++j) {
            const bool see = a.masks ? a.masks[((size_t)u.b * a.W + i) * a.words + (j >> 5)] >> (j & 31) & 1
                                     : j <= i;
            const int blk = see ? c.block(u.b, u.seq + j) : -1;
            if (blk < 0) continue;
            const uint32_t* v = reinterpret_cast<const uint32_t*>(
                c.pool + c.row(blk, 1, u.h, (int)((u.seq + j) % c.tpb)) + x);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t nb = nan_bytes(v[k]);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (nb >> (8 * e + 7) & 1) o[k * 4 + e] = 0x7fc00000u;
            }
          }
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + 2 * (orow * D + x));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                y[e] = pack_out(__uint_as_float(o[k * 8 + e * 2]) * f,
                                __uint_as_float(o[k * 8 + e * 2 + 1]) * f, (T*)nullptr);
              dst[k] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<float4*>(part + (size_t)r * D + x + 4 * k) = make_float4(
                  __uint_as_float(o[4 * k]) * f, __uint_as_float(o[4 * k + 1]) * f,
                  __uint_as_float(o[4 * k + 2]) * f, __uint_as_float(o[4 * k + 3]) * f);
          }
        }
        __syncwarp();
      }
      if (r < rows) {
        if (whole) {
          if (a.lse) a.lse[orow] = row_lse(m, l);
        } else {
          part[(size_t)kRows * D + r] = m;
          part[(size_t)kRows * D + kRows + r] = l;
        }
      }
      if (!whole && tile0 == 0 && tid == 0) {
        int* d = a.desc + blockIdx.x * kDescWords;
        d[0] = u.b;
        d[1] = u.h;
        d[2] = u.mt;
        d[3] = share_owner(total, unit0 + u.tiles - 1, ctas);
      }
      fence_before();  // O has been read: the next unit's first product may follow its q_full, p_full
    } else if (warp == kMmaWarp) {
      if (u.w >= 0) {
        bar_wait(&bars.q_full, seg & 1, dead);
        fence_after();
        const uint32_t base = smem_u32(tiles);
        auto scores = [&](uint32_t t) {
          const int st = t % ST;
          bar_wait(&bars.k_full[st], (t / ST) & 1, dead);
          fence_after();
          if (lane == 0 && !*dead) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ts(tmem + kColS + (t & 1) * kKeys, tmem + kColQ + k * 8,
                     smem_desc(base + st * TL::kBytes + (k / 4) * (kKeys * 128) + (k % 4) * 32, 16),
                     instr_desc(kKeys, false), k > 0);
            mma_commit(&bars.k_empty[st]);
            mma_commit(&bars.s_full[t & 1]);
          }
          __syncwarp();
        };
        scores(n);
        for (int tile = tile0; tile < tile1; ++tile, ++n) {
          if (tile + 1 < tile1) scores(n + 1);
          const int st = n % ST;
          bar_wait(&bars.v_full[st], (n / ST) & 1, dead);
          bar_wait(&bars.p_full, n & 1, dead);
          fence_after();
          if (lane == 0 && !*dead) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              mma_ts(tmem + kColO, tmem + kColP + k * 8,
                     smem_desc(base + (ST + st) * TL::kBytes + k * 2048, kKeys * 128),
                     instr_desc(D, true), tile > tile0 || k > 0);
            mma_commit(&bars.v_empty[st]);
            mma_commit(&bars.pv_done);
          }
          __syncwarp();
        }
      }
    } else {
      if (u.w >= 0) {
        // Thread t of the converters: chunk t % (D / 16) of rows t / (D / 16) + kPer p.
        constexpr int CPR = D / 16, kPer = kConvThreads / CPR, NP = kKeys / kPer;
        const int t = tid - kConvWarp * 32, ch = t % CPR, row = t / CPR;
        const int tpb16 = c.tpb / 16;
        const int32_t* table = c.tables + (size_t)u.b * c.max_blocks;
        const size_t v_off = (size_t)c.H * c.tpb * D;
        uint4 kr[NP], vr[NP];
        const uint8_t* src[NP];
        auto locate = [&](int tile) {  // where this thread's rows of a tile are (null: no such row)
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const long key = (long)tile * kKeys + p * kPer + row;
            src[p] = nullptr;
            if (key < keys) {
              const int grp = (int)(key >> 4), col = grp / tpb16;
              const int blk = table[col];
              if (blk >= 0 && blk < c.num_blocks)
                src[p] = c.pool + c.row(blk, 0, u.h, (grp - col * tpb16) * 16 + (int)(key & 15)) + ch * 16;
            }
          }
        };
        auto load = [&](uint4 (&x)[NP], size_t off) {
#pragma unroll
          for (int p = 0; p < NP; ++p)
            x[p] = src[p] ? *reinterpret_cast<const uint4*>(src[p] + off) : make_uint4(0, 0, 0, 0);
        };
        auto put = [&](const uint4 (&x)[NP], unsigned char* tile) {
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const int key = p * kPer + row;
            const uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
            uint32_t h[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) e4m3x4_to_half(w[k], h[2 * k], h[2 * k + 1]);
            unsigned char* at16 = tile + (ch >> 2) * (kKeys * 128) + key * 128;
            const int c0 = (ch & 3) * 2;
            // half of the threads write their second 16 bytes first: no bank conflicts
            const int first = D == 128 ? ch >> 2 : 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int s = k ^ first;
              *reinterpret_cast<uint4*>(at16 + (((c0 + s) ^ (key & 7)) << 4)) =
                  s ? make_uint4(h[4], h[5], h[6], h[7]) : make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        };
        locate(tile0);
        load(kr, 0);
        load(vr, v_off);
        for (int tile = tile0; tile < tile1; ++tile, ++n) {
          const int st = n % ST, ring = n % kScaleRing;
          if (warp == kConvWarp) {  // the tile's scales
            const int grp = tile * kGroups + (lane & 7), col = grp / tpb16;
            float s = 0.f;
            if (lane < 16 && (long)grp * 16 < keys) {
              const int blk = table[col];
              // a block that does not exist makes the scores NaN
              s = blk >= 0 && blk < c.num_blocks ? c.scales[c.scale_at(blk, lane >> 3, u.h)]
                                                 : lane < 8 ? NAN : 0.f;
            }
            if (lane < 8) sK[ring][lane] = s;
            else if (lane < 16) sV[ring][lane - 8] = s;
            __syncwarp();
            if (lane == 0) bar_arrive(&bars.scales[ring]);
          }
          bar_wait(&bars.k_empty[st], ((n / ST) & 1) ^ 1, dead);
          put(kr, tiles + st * TL::kBytes);
          if (lane == 0) bar_arrive(&bars.k_full[st]);
          if ((long)(tile + 1) * kKeys > u.seq) {
            // NaN in a window row of V: only the rows that see it may get it
#pragma unroll
            for (int p = 0; p < NP; ++p) {
              uint32_t w[4] = {vr[p].x, vr[p].y, vr[p].z, vr[p].w};
              if ((long)tile * kKeys + p * kPer + row >= u.seq) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const uint32_t nb = nan_bytes(w[k]);
                  if (nb) sNan = 1;
                  w[k] &= ~((nb >> 7) * 255u);
                }
                vr[p] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
          if (tile + 1 < tile1) {
            locate(tile + 1);
            load(kr, 0);
          }
          bar_wait(&bars.v_empty[st], ((n / ST) & 1) ^ 1, dead);
          put(vr, tiles + (ST + st) * TL::kBytes);
          if (lane == 0) bar_arrive(&bars.v_full[st]);
          if (tile + 1 < tile1) load(vr, v_off);
        }
      }
    }
    at = stop;
    unit0 += u.tiles;
    if (u.w < 0) --seg;  // no Q was loaded for it
    if (at < t1 && !Div::next(a, u)) break;
  }

  // Every product has finished before tensor memory is given back.
  if (warp == kMmaWarp) {
    if (lane == 0) mma_commit(&bars.end);
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
  return launch_join<T, D, kRows, kKeys>(a, kSms, st);
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

// Attention for few rows per KV head (a token, a short window): bound by the
// bytes of the cache.
//
// Tensor cores through mma.sync m16n8k16 (fp16 operands, fp32 sums): with at
// most 16 rows per KV head each cache byte meets 16 multiply-adds, which is
// far below what the legacy path sustains, and it takes its operands from
// registers, so that an e4m3 byte goes global -> shared (cp.async) ->
// register -> two fp16 values -> mma with no second pass through shared
// memory, which tcgen05 would need.
//
// e4m3 -> fp16 is exact.  Q is scaled by a power of two per row to a largest
// magnitude in [2^14, 2^15) and rounded to fp16: exact for bf16 and fp16
// elements down to 2^-28 of the row's largest.  The scale of a key's block
// multiplies the score.  The weights are those of RowRef: a power of two of the
// score and of the exponent of their block's V scale, rounded to fp16 (11 bits;
// below 2^-22 of the row's largest in steps of 2^-32).  The references move
// only when a key exceeds them by more than 7, so that the sums are rarely
// rescaled.
//
// Measured in a graph with 32 heads over 8 KV heads of 128 and windows of 4
// tokens: 256 requests of 8192 positions 682 us, 6.3 TB/s (0.93 of the measured
// copy rate); 256 of 512 to 8192, 393 us, 5.8 TB/s (0.86).  One token of one
// request over 1000 positions takes 12.6 us, both launches: latency (the
// shares, the table, the rows, the four warps' merge, the join).
#include "attend.cuh"

namespace sv {

namespace {

constexpr int kRows = 16;
constexpr int kStep = 16;                 // keys of one warp step
constexpr int kRWarps = 4;
constexpr int kRThreads = kRWarps * 32;
constexpr int kKeys = kStep * kRWarps;    // keys of a tile: one step of every warp
constexpr int kStages = 4;
// Cells of a unit besides its tiles: what its start and its result take.  256
// requests of 512 to 8192 positions, 1 to 4 tokens each: 413 us with 2, 403 with
// 4, 390 with 6, 384 with 8 (eager); 512 of 4 tokens over 100 to 900: 187, 169,
// 162, 162 (160 now); one token of one request over 4000 positions: 14.8, 14.5,
// 14.2, 16.3 (14.6 now).
constexpr int kUnitCost = 6;
// Cells below which a share is not worth a CTA.  One request, one token, 8 KV
// heads, 100 / 1000 / 30000 positions: 10.5 / 12.3 / 34.7 us with 3 cells, 9.5
// / 12.5 / 34.4 with 4, 15.7 / 13.4 / 34.4 with 6, 25.4 / 19.5 / 33.1 with 12
// (with the join of that time; 10.0 / 12.4 / 24.5 now).
constexpr int kLeastCells = 4;
constexpr int kCtas = 3 * kSms;           // resident at 168 registers and 66 KB of shared memory
using Div = Division<kRows, kKeys>;

template <int D>
struct Ring {
  static constexpr int kHalf = kStep * D;            // bytes of K (and of V) in a stage
  static constexpr int kStage = 2 * kHalf + 16;      // and the two scales
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kPitch = D + 4;               // floats of a row in the join
  static constexpr size_t kJoin = (size_t)kRWarps * kRows * kPitch * 4;
  static constexpr size_t kBytes = kWarp * kRWarps > kJoin ? kWarp * kRWarps : kJoin;
  // Byte of 16-byte chunk ch of key row r.  Fragments read K as row = lane / 4,
  // chunk = lane % 4 (+ 4) and V as row = 2 (lane % 4) (+ 1), chunk (or half a
  // chunk) = lane / 4: these places keep both free of bank conflicts.
  static __device__ __forceinline__ int k_at(int r, int ch) {
    return D == 128 ? r * 128 + ((ch ^ ((r & 1) << 2)) << 4) : r * 64 + (ch << 4);
  }
  static __device__ __forceinline__ int v_at(int r, int ch) {
    if (D == 128) return r * 128 + ((ch ^ (r & 6)) << 4);
    return (r >> 1) * 128 + (((r ^ (r >> 2)) & 1) << 6) + ((ch ^ (r & 2)) << 4);
  }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <class T, int D>
__global__ void __launch_bounds__(kRThreads, 3) attend_rows_kernel(const AttendArgs a) {
  using R = Ring<D>;
  constexpr int U = D / 64;   // 16-byte K chunks per thread and key
  constexpr int NT = D / 8;   // mma tiles along D
  constexpr int VW = D / 32;  // 32-bit words of V per thread and key
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float sM[kRWarps][kRows], sR[kRWarps][kRows], sL[kRWarps][kRows];
  __shared__ int sBad;
  const KvCache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, cc = lane & 3;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the walk lies in shared memory: its 20 words are needed between segments only
  __shared__ Walk<kRows, kKeys, kUnitCost> v;
  __shared__ int sMore;
  if (tid < kDescWords) a.desc[blockIdx.x * kDescWords + tid] = -1;
  if (!divide<kRows, kKeys, kUnitCost, kRThreads>(a, kLeastCells, v)) return;
  __syncthreads();  // every thread has stored the walk's beginning
  unsigned char* ring = smem + warp * R::kWarp;
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
  const int tpb16 = c.tpb / kStep;
  const size_t v_off = (size_t)c.H * c.tpb * D;  // from a block's K rows to its V rows

  for (;;) {
    if (tid == 0) sMore = v.next(a);
    __syncthreads();
    if (!sMore) break;
    const Unit u = v.u;
    const int tile0 = v.tile0, tile1 = v.tile1;
    const int r0 = u.mt * kRows;
    const int w = u.w < 0 ? a.W : u.w;
    const int rows = min((long)kRows, (long)w * a.G - r0);
    if (tid == 0) sBad = u.w < 0;
    __syncthreads();
    float o[NT][4];
    RowRef ref[2];
    float l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    if (u.w >= 0) {
      const int32_t* table = c.tables + (size_t)u.b * c.max_blocks;
      const long keys = Div::seen(a, u.seq, u.w, u.mt);
      const int steps = (int)min((long)tile1 * kRWarps, (keys + kStep - 1) / kStep);
      if (tile1 == u.tiles)  // a window block that no row of this tile reads is checked all the same
        for (int i = (int)(u.seq / c.tpb) + tid; (long)i * c.tpb < (long)u.seq + u.w; i += kRThreads)
          if (table[i] < 0 || table[i] >= c.num_blocks) sBad = 1;

      // ---- the ring: step st of the unit = keys [16 st, 16 st + 16)
      int fst = tile0 * kRWarps + warp;               // next step to fetch
      int fcol = fst / tpb16, foff = fst % tpb16;     // its block table column and place there
      int fblk = fst < steps ? table[fcol] : 0;       // its block, loaded one fetch ahead ...
      const int dcol = kRWarps / tpb16, doff = kRWarps % tpb16;
      int stage = 0;
      int early[kStages - 1];  // ... but for the first fetches, whose blocks are loaded together
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) {
        const int st = fst + (i + 1) * kRWarps;
        early[i] = st < steps ? table[st / tpb16] : 0;
      }
      auto fetch = [&](int n) {
        if (fst < steps) {
          const bool ok = fblk >= 0 && fblk < c.num_blocks;
          if (!ok) sBad = 1;
          const uint8_t* kp = c.pool + c.row(ok ? fblk : 0, 0, u.h, foff * kStep);
          const float* sp = c.scales + c.scale_at(ok ? fblk : 0, 0, u.h);
          const uint32_t dst = ring_s + stage * R::kStage;
          const int left = (int)min((long)kStep, keys - (long)fst * kStep);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const int q = lane + 32 * i, r = q / (D / 16), ch = q % (D / 16);
            // rows past the keys are zeroed: what lies there may be NaN
            cp16(dst + R::k_at(r, ch), kp + q * 16, ok && r < left);
            cp16(dst + R::kHalf + R::v_at(r, ch), kp + v_off + q * 16, ok && r < left);
          }
          if (lane < 2) cp4(dst + 2 * R::kHalf + 4 * lane, sp + lane * c.H, ok);
          fst += kRWarps;
          fcol += dcol;
          foff += doff;
          if (foff >= tpb16) foff -= tpb16, ++fcol;
          if (n < kStages - 1)
            fblk = early[n];
          else if (fst < steps)
            fblk = table[fcol];
        }
        cp_commit();
        stage = stage + 1 == kStages ? 0 : stage + 1;
      };
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) fetch(i);

      // ---- Q fragments: thread (g, cc) holds elements 16 (cc + 4 x) .. + 15 of rows g and g + 8
      uint32_t qf[U * 4][4];
      float qs[2];   // scale * log2(e) over the row's power of two
      int qi[2];     // the rows' window tokens
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = g + 8 * k;
        const bool real = r < rows;
        const int i = real ? (r0 + r) / a.G : 0, head = real ? (r0 + r) % a.G : 0;
        qi[k] = i;
        const uint4* qp = reinterpret_cast<const uint4*>(
            a.q + 2 * (u.b * a.qb + i * a.qt + (u.h * a.G + head) * a.qh));
        uint32_t x[U * 8];
#pragma unroll
        for (int y = 0; y < U; ++y)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const uint4 v = real ? qp[(cc + 4 * y) * 2 + z] : make_uint4(0, 0, 0, 0);
            x[y * 8 + z * 4] = v.x, x[y * 8 + z * 4 + 1] = v.y;
            x[y * 8 + z * 4 + 2] = v.z, x[y * 8 + z * 4 + 3] = v.w;
          }
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < U * 8; ++e) {
          const float2 f = as_float2(x[e], (T*)nullptr);
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        int e;
        frexpf(top, &e);  // top < 2^e
        const int up = top > 0.f && top < INFINITY ? min(15 - e, 126) : 0;
        const float f = ldexpf(1.f, up);
        qs[k] = a.scale_log2 * ldexpf(1.f, -up);
#pragma unroll
        for (int y = 0; y < U * 4; ++y) {
          const float2 p0 = as_float2(x[y * 2], (T*)nullptr);
          const float2 p1 = as_float2(x[y * 2 + 1], (T*)nullptr);
          qf[y][k] = half2_of(p0.x * f, p0.y * f);
          qf[y][2 + k] = half2_of(p1.x * f, p1.y * f);
        }
      }

      int cst = 0;  // stage to compute
      for (int st = tile0 * kRWarps + warp; st < steps; st += kRWarps) {
        cp_wait<kStages - 2>();
        __syncwarp();
        const unsigned char* sp = ring + cst * R::kStage;
        cst = cst + 1 == kStages ? 0 : cst + 1;
        // ---- scores of 16 keys: two tiles of 8
        float s[2][4] = {};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int y = 0; y < U; ++y) {
            const uint4 kv = *reinterpret_cast<const uint4*>(sp + R::k_at(n * 8 + g, cc + 4 * y));
            const uint32_t kw[4] = {kv.x, kv.y, kv.z, kv.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t b0, b1;
              e4m3x4_to_half(kw[x], b0, b1);
              mma16816(s[n], qf[y * 4 + x], b0, b1);
            }
          }
        const float2 scales = *reinterpret_cast<const float2*>(sp + 2 * R::kHalf);
        const long j0 = (long)st * kStep - u.seq;  // the window's place of key 0
        // ---- t = score in log2 units; element e of tile n: row e / 2, key 8 n + 2 cc + e % 2
        unsigned seen = 0xff;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] *= qs[e >> 1] * scales.x;
        if (j0 + kStep > 0) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = qi[e >> 1];
              const long j = j0 + 8 * n + 2 * cc + (e & 1);
              bool see = j < u.w;
              if (j >= 0 && see) {
                if (a.masks)
                  see = a.masks[((size_t)u.b * a.W + i) * a.words + (j >> 5)] >> (j & 31) & 1;
                else
                  see = j <= i;
              }
              if (!see) s[n][e] = -INFINITY, seen &= ~(1u << (n * 4 + e));
            }
        }
        float top[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          top[k] = fmaxf(fmaxf(s[0][2 * k], s[0][2 * k + 1]), fmaxf(s[1][2 * k], s[1][2 * k + 1]));
        float vf;  // V's scale is vf * 2^ve
        const float ve = scale_exponent(scales.y, &vf);
        float depth[2] = {ref[0].r - ve, ref[1].r - ve};
        const bool up = top[0] > ref[0].m + kLazy + fminf(depth[0], 0.f) ||
                        top[1] > ref[1].m + kLazy + fminf(depth[1], 0.f);
        if (__any_sync(~0u, up)) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            top[k] = fmaxf(top[k], __shfl_xor_sync(~0u, top[k], 1));
            top[k] = fmaxf(top[k], __shfl_xor_sync(~0u, top[k], 2));
            float fl, fo;
            ref[k].move(top[k], top[k] + ve, &fl, &fo);
            depth[k] = ref[k].r - ve;
            l[k] *= fl;
#pragma unroll
            for (int j = 0; j < NT; ++j) o[j][2 * k] *= fo, o[j][2 * k + 1] *= fo;
          }
        }
        // ---- weights
        float p[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          depth[k] = fminf(depth[k], kDeep);
          const float sub = ref[k].m - kPBits + depth[k];
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              p[n][2 * k + e] = ex2(s[n][2 * k + e] - sub);
              sum += p[n][2 * k + e];
            }
          l[k] = fmaf(sum, ex2(depth[k]), l[k]);
        }
        if (vf != 1.f) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) p[n][e] *= vf;
        }
        const uint32_t pa[4] = {weights_f16(p[0][0], p[0][1]), weights_f16(p[0][2], p[0][3]),
                                weights_f16(p[1][0], p[1][1]), weights_f16(p[1][2], p[1][3])};
        // ---- weighted V: keys 2 cc, 2 cc + 1 (tile 0) and 8 + 2 cc, 8 + 2 cc + 1 (tile 1);
        // mma tile j holds d = (D / 8) g + j
        const unsigned char* vp = sp + R::kHalf;
        uint32_t vw[4][VW];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = (k >> 1) * 8 + 2 * cc + (k & 1);
          if (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(vp + R::v_at(r, g));
            vw[k][0] = v.x, vw[k][1] = v.y, vw[k][VW - 2] = v.z, vw[k][VW - 1] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(vp + R::v_at(r, g >> 1) + (g & 1) * 8);
            vw[k][0] = v.x, vw[k][1] = v.y;
          }
        }
        if (j0 + kStep > 0) {
          // NaN in a window row: only the rows that see it may get it, and a
          // weight of 0 times NaN is NaN.  Zero it here and count, with a
          // product of ones, the NaN that each row sees.
          uint32_t bad[4][VW], any = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int x = 0; x < VW; ++x) any |= bad[k][x] = nan_bytes(vw[k][x]);
          if (__any_sync(~0u, any != 0)) {
            uint32_t ones[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              // pa[q]: row q % 2, tile q / 2
              const int n = q >> 1, e = (q & 1) * 2;
              ones[q] = ((seen >> (n * 4 + e)) & 1 ? 0x3c00u : 0u) |
                        ((seen >> (n * 4 + e + 1)) & 1 ? 0x3c000000u : 0u);
            }
#pragma unroll
            for (int x = 0; x < VW; ++x)
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                uint32_t b[2];
#pragma unroll
                for (int q = 0; q < 2; ++q)
                  b[q] = ((bad[2 * q][x] >> (8 * d + 7)) & 1 ? 0x3c00u : 0u) |
                         ((bad[2 * q + 1][x] >> (8 * d + 7)) & 1 ? 0x3c000000u : 0u);
                float cnt[4] = {};
                mma16816(cnt, ones, b[0], b[1]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (cnt[e] > 0.f) o[x * 4 + d][e] = NAN;
              }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int x = 0; x < VW; ++x) vw[k][x] &= ~((bad[k][x] >> 7) * 255u);
          }
        }
#pragma unroll
        for (int x = 0; x < VW; ++x) {
          uint32_t b[2][4];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            e4m3x4_to_half(__byte_perm(vw[2 * q][x], vw[2 * q + 1][x], 0x5140), b[q][0], b[q][1]);
            e4m3x4_to_half(__byte_perm(vw[2 * q][x], vw[2 * q + 1][x], 0x7362), b[q][2], b[q][3]);
          }
#pragma unroll
          for (int d = 0; d < 4; ++d) mma16816(o[x * 4 + d], pa, b[0][d], b[1][d]);
        }
        __syncwarp();  // every lane has read the stage that the next fetch may reuse
        fetch(kStages);
      }
      cp_wait<0>();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        l[k] += __shfl_xor_sync(~0u, l[k], 1);
        l[k] += __shfl_xor_sync(~0u, l[k], 2);
      }
    }
    // ---- join the four warps
    __syncthreads();
    float* join = reinterpret_cast<float*>(smem) + (size_t)warp * kRows * R::kPitch;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float* row = join + (g + 8 * k) * R::kPitch + 2 * cc * NT;
#pragma unroll
      for (int j = 0; j < NT; j += 4) {
        *reinterpret_cast<float4*>(row + j) =
            make_float4(o[j][2 * k], o[j + 1][2 * k], o[j + 2][2 * k], o[j + 3][2 * k]);
        *reinterpret_cast<float4*>(row + NT + j) = make_float4(
            o[j][2 * k + 1], o[j + 1][2 * k + 1], o[j + 2][2 * k + 1], o[j + 3][2 * k + 1]);
      }
      if (cc == 0) sM[warp][g + 8 * k] = ref[k].m, sR[warp][g + 8 * k] = ref[k].r, sL[warp][g + 8 * k] = l[k];
    }
    __syncthreads();
    {
      const int r = tid >> 3, part = tid & 7;  // 8 threads per row, D / 8 elements each
      float M = kNone, R = kNone, L = 0.f, f[kRWarps];
#pragma unroll
      for (int k = 0; k < kRWarps; ++k) M = fmaxf(M, sM[k][r]);
#pragma unroll
      for (int k = 0; k < kRWarps; ++k) R = fmaxf(R, sM[k][r] - M + sR[k][r]);
      R = floorf(R);
#pragma unroll
      for (int k = 0; k < kRWarps; ++k) {
        const float d = sM[k][r] - M;
        f[k] = ex2(d + (sR[k][r] - R));
        L = fmaf(sL[k][r], ex2(d), L);
      }
      if (sBad) L = NAN;
      float x[NT];
#pragma unroll
      for (int j = 0; j < NT; j += 4) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kRWarps; ++k) {
          const float4 z = *reinterpret_cast<const float4*>(
              reinterpret_cast<float*>(smem) + ((size_t)k * kRows + r) * R::kPitch + part * NT + j);
          y.x += z.x * f[k], y.y += z.y * f[k], y.z += z.z * f[k], y.w += z.w * f[k];
        }
        x[j] = y.x, x[j + 1] = y.y, x[j + 2] = y.z, x[j + 3] = y.w;
      }
      const bool whole = v.whole();
      if (r < rows) {
        if (whole) {
          const int i = (r0 + r) / a.G, head = u.h * a.G + (r0 + r) % a.G;
          const size_t orow = ((size_t)u.b * a.W + i) * a.Hq + head;
          const float2 out = result_factors(L, R);
          uint32_t y[NT / 2];
#pragma unroll
          for (int j = 0; j < NT; j += 2)
            y[j / 2] = pack_out(x[j] * out.x * out.y, x[j + 1] * out.x * out.y, (T*)nullptr);
          uint4* dst = reinterpret_cast<uint4*>(a.out + 2 * (orow * D + part * NT));
#pragma unroll
          for (int j = 0; j < NT / 8; ++j)
            dst[j] = make_uint4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
          if (a.lse && part == 0) a.lse[orow] = row_lse(M, L);
        } else {
          const size_t slot = 2 * (size_t)blockIdx.x + (tile0 == 0);
          float* dst = a.part + slot * part_floats<kRows>(D);
#pragma unroll
          for (int j = 0; j < NT; j += 4)
            *reinterpret_cast<float4*>(dst + r * D + part * NT + j) =
                make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
          if (part == 0) dst[kRows * D + r] = M, dst[kRows * (D + 1) + r] = R, dst[kRows * (D + 2) + r] = L;
        }
      }
      if (!whole && tile0 == 0 && tid == 0) {
        int* d = a.desc + blockIdx.x * kDescWords;
        d[0] = u.b;
        d[1] = u.h;
        d[2] = u.mt;
        d[3] = v.last_cta();
        d[4] = rows;
      }
    }
    __syncthreads();
  }
}

}  // namespace

size_t attend_rows_scratch(int D) {
  return align256((size_t)kCtas * kDescWords * 4) + 2 * (size_t)kCtas * part_floats<kRows>(D) * 4;
}

namespace {

template <class T, int D>
cudaError_t launch_rows(const AttendArgs& a, cudaStream_t st) {
  const auto kernel = attend_rows_kernel<T, D>;
  const size_t bytes = Ring<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCtas);
  cfg.blockDim = dim3(kRThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e != cudaSuccess) return e;
  return launch_join<T, D, kRows>(a, kCtas, st);
}

}  // namespace

cudaError_t launch_attend_rows(AttendArgs& a, int dtype, void* scratch, cudaStream_t st) {
  a.mtiles = ceil_div((long)a.W * a.G, kRows);
  a.desc = static_cast<int*>(scratch);
  a.part = reinterpret_cast<float*>(static_cast<char*>(scratch) + align256((size_t)kCtas * kDescWords * 4));
  if (dtype == SPEC_BF16)
    return a.c.D == 64 ? launch_rows<__nv_bfloat16, 64>(a, st)
                       : launch_rows<__nv_bfloat16, 128>(a, st);
  return a.c.D == 64 ? launch_rows<__half, 64>(a, st) : launch_rows<__half, 128>(a, st);
}

}  // namespace sv

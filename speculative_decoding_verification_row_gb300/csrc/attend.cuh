// Arguments and work division of the attention kernels over the 8-bit paged
// cache (internal).
#pragma once

#include "kvcache.cuh"

namespace sv {

struct AttendArgs {
  KvCache c;
  const char* q;
  long qb, qt, qh;  // strides in elements
  int B, W, Hq, G;  // G = Hq / H query heads per KV head
  const int32_t* seq;
  const int32_t* win;
  const int32_t* masks;
  int words;        // mask words per row
  float scale_log2; // scale * log2(e)
  char* out;
  float* lse;
  int mtiles;       // row tiles of a full window
  unsigned tpb16_div;  // x / (tpb / 16) = umulhi(x, tpb16_div) for x < 2^26, tpb > 16
  int* desc;        // scratch: per CTA, where a unit begins that other CTAs end
  float* part;      // scratch: two partial results per CTA
};

// Block table column of 16-key group x.  ceil(2^32 / d) * d - 2^32 < d <= 64, so
// the quotient is exact for x < 2^26, the limit of kMaxPositions.
__device__ __forceinline__ unsigned col16(const AttendArgs& a, unsigned x) {
  return a.c.tpb == 16 ? x : __umulhi(x, a.tpb16_div);
}
constexpr long kMaxPositions = 1l << 30;
// Most rows (tokens times query heads) of a call: its outputs would be 128 GB, 256 with D = 128.
constexpr long kMaxRows = 1l << 30;

// Rows of one request and KV head are numbered r = i * G + g (window token i,
// query head g of the group) and cut into tiles of ROWS; a "unit" is one such
// tile of one (request, KV head).  Its keys are cut into tiles of KEYS.  The
// key tiles of all units, ordered by request, row tile and head, form one
// line that is cut into equal shares, one per CTA (see Walk), so a ragged
// batch keeps every SM equally busy and a long prefix spreads over all.  A unit
// whose tiles fall to several CTAs is joined afterwards from the (max, sum,
// weighted V) of each.
struct Unit {
  int b, h, mt;
  int seq;
  int w;        // window length; -1: the request's lengths are out of range
  int tiles;    // key tiles of the unit
};

template <int ROWS, int KEYS>
struct Division {
  static __device__ __forceinline__ void lens(const AttendArgs& a, int b, int* seq, int* w) {
    *seq = a.seq[b];
    *w = a.win ? a.win[b] : a.W;
    if (*seq < 0 || *w < 0 || *w > a.W || (long)*seq + *w > (long)a.c.max_blocks * a.c.tpb) *w = -1;
  }
  // Keys that some row of tile mt sees, at most (0: the tile has no rows).
  static __device__ __forceinline__ unsigned seen(const AttendArgs& a, int seq, int w, int mt) {
    const int r0 = mt * ROWS, rows = w * a.G;  // at most 2^30: 65536 tokens, 16384 heads
    if (r0 >= rows) return 0;
    if (a.masks) return (unsigned)seq + w;
    return (unsigned)seq + (unsigned)(min(r0 + ROWS, rows) - 1) / (unsigned)a.G + 1;
  }
  static __device__ __forceinline__ int tiles(const AttendArgs& a, int seq, int w, int mt) {
    if (w < 0) return mt * ROWS < a.W * a.G ? 1 : 0;  // its rows are written all the same
    return (int)((seen(a, seq, w, mt) + KEYS - 1) / KEYS);
  }
  // Moves u to the next unit that has tiles, if any.
  static __device__ __forceinline__ bool next(const AttendArgs& a, Unit& u) {
    if (++u.h < a.c.H) return true;
    u.h = 0;
    for (;;) {
      if (++u.mt == a.mtiles) {
        u.mt = 0;
        if (++u.b == a.B) return false;
        lens(a, u.b, &u.seq, &u.w);
      }
      u.tiles = tiles(a, u.seq, u.w, u.mt);
      if (u.tiles > 0) return true;
    }
  }
};

// x / n: 32-bit arithmetic where it suffices (a 64-bit division takes hundreds of clocks).
static __device__ __noinline__ long quotient(long x, long n) {
  return (x | n) >> 31 ? x / n : (long)((unsigned)x / (unsigned)n);
}
// A line of `total` cells in n shares: the first `more` of them hold one cell
// more than `each`.
struct Shares {
  long total, each;
  int n, more;
  __device__ __forceinline__ void set(long cells, int shares) {
    total = cells;
    n = shares;
    each = quotient(cells, shares);
    more = (int)(cells - each * shares);
  }
  __device__ __forceinline__ long begin(int i) const { return each * i + min(i, more); }
  // The share that holds a cell.
  __device__ __forceinline__ int owner(long cell) const {
    const long wide = (each + 1) * more;  // cells of the longer shares
    return cell < wide ? (int)quotient(cell, each + 1) : more + (int)quotient(cell - wide, each);
  }
};

// A CTA's share of the line.  A unit takes COST cells (for loading its rows
// and writing its result) and one for each of its key tiles; the tiles of a
// unit that fall into the share are a segment.
template <int ROWS, int KEYS, int COST>
struct Walk {
  Unit u;
  long at, end;      // the share's cells not yet walked
  long unit0;        // first cell of u
  Shares shares;
  int tile0, tile1;  // the segment
  // To the next segment; false at the share's end.  For one thread, on a walk
  // in shared memory; not inlined: the kernels' code has to stay in the
  // instruction caches.
  __device__ __noinline__ bool next(const AttendArgs& a) {
    for (;;) {
      if (at >= end) return false;
      const long unit1 = unit0 + COST + u.tiles;
      if (at == unit1) {
        unit0 = unit1;
        Unit n = u;
        if (!Division<ROWS, KEYS>::next(a, n)) return false;
        u = n;
        continue;
      }
      const long stop = min(end, unit1);
      tile0 = (int)max(0l, at - unit0 - COST);
      tile1 = (int)max(0l, stop - unit0 - COST);
      at = stop;
      if (tile1 > tile0) return true;
    }
  }
  __device__ __forceinline__ bool whole() const { return tile0 == 0 && tile1 == u.tiles; }
  // The CTA that holds the unit's last tile.
  __device__ __forceinline__ int last_cta() const {
    return shares.owner(unit0 + COST + u.tiles - 1);
  }
};

// Sets a CTA of THREADS threads before the first segment of its share.
// False: nothing to do.  `least`: cells below which a share is not worth a
// CTA.  Every CTA sums the line anew, (request, row
// tile) pairs over its threads: no state between launches and none to clear.
template <int ROWS, int KEYS, int COST, int THREADS>
__device__ __forceinline__ bool divide(const AttendArgs& a, int least, Walk<ROWS, KEYS, COST>& v) {
  using Div = Division<ROWS, KEYS>;
  __shared__ long long sWarp[THREADS / 32];
  __shared__ int sFind[6];
  __shared__ long long sUnit0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int items = a.B * a.mtiles;  // fits: see kMaxRows
  const int per = (unsigned)(items + THREADS - 1) / (unsigned)THREADS;
  const int x0 = min(items, tid * per), x1 = min(items, x0 + per);
  // calls f(b, mt, seq, w, tiles) for this thread's pairs until f returns false
  auto pairs = [&](auto f) {
    int b = (unsigned)x0 / (unsigned)a.mtiles, mt = x0 - b * a.mtiles, seq = 0, w = 0;
    for (int x = x0; x < x1; ++x) {
      if (x == x0 || mt == 0) Div::lens(a, b, &seq, &w);
      if (!f(b, mt, seq, w, Div::tiles(a, seq, w, mt))) return;
      if (++mt == a.mtiles) mt = 0, ++b;
    }
  };
  long long mine = 0;
  pairs([&](int, int, int, int, int n) { return mine += n > 0 ? n + COST : 0, true; });
  mine *= a.c.H;
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
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < warp) incl += sWarp[i];
    total += sWarp[i];
  }
  const long most = quotient(total, least);
  const int ctas = most < 1 ? 1 : most < (long)gridDim.x ? (int)most : (int)gridDim.x;
  if (total == 0 || (int)blockIdx.x >= ctas) return false;
  Shares s;
  s.set(total, ctas);
  const long begin = s.begin(blockIdx.x);
  if (incl - mine <= begin && begin < incl) {  // one thread: its pairs hold the share's first cell
    long at = incl - mine;
    pairs([&](int b, int mt, int seq, int w, int n) {
      const int cells = n > 0 ? n + COST : 0;
      if (begin >= at + (long)cells * a.c.H) return at += (long)cells * a.c.H, true;
      const int h = (int)quotient(begin - at, cells);
      sFind[0] = b;
      sFind[1] = h;
      sFind[2] = mt;
      sFind[3] = seq;
      sFind[4] = w;
      sFind[5] = n;
      sUnit0 = at + (long)h * cells;
      return false;
    });
  }
  __syncthreads();
  v.shares = s;  // every thread stores the same
  v.at = begin;
  v.end = s.begin(blockIdx.x + 1);
  v.unit0 = sUnit0;
  v.u = Unit{sFind[0], sFind[1], sFind[2], sFind[3], sFind[4], sFind[5]};
  return true;
}

// The sums of a row, over the positions t that it sees (scores in log2 units,
// V = 2^v times its code):
//   l = sum 2^(t - m + 8)             m follows the largest t,
//   o = sum 2^(t + v - m - r + 8) code    m + r follows the largest t + v;
// out = 2^r o / l.  Each reference moves only when a position exceeds it by
// more than 7, and stays at or below the largest: the weights of o, which are
// rounded to fp16, reach 2^8 and stay at or below 2^15.  Both references are
// the row's own, so a position that it does not see takes none of its bits, and
// no sum leaves fp32's range whatever V's scales are.  r is an integer: with
// scales that are powers of two r - v is exact.  v is taken as at least r - 64:
// with t <= m + 7 such a position adds at most 2^-57 of the largest, and
// 2^(r - v) in l stays finite.  Before the first position m is the least float:
// every sum is 0 then, and no difference is NaN.
constexpr float kPBits = 8.f;
constexpr float kLazy = 7.f;
constexpr float kDeep = 64.f;
constexpr float kNone = -3.402823466e38f;

struct RowRef {
  float m = kNone, r = 0.f;
  // Moves to the largest t and t + v of some positions; *fl and *fo: what l and o are to be multiplied by.
  __device__ __forceinline__ void move(float t, float tv, float* fl, float* fo) {
    const float now = t > m + kLazy ? t : m, at = m + r;
    // rounding r down lowers m + r by less than 1: one less of slack keeps the weights below 2^15
    const float rn = floorf((tv > at + (kLazy - 1.f) ? tv : at) - now);
    *fl = ex2(m - now);
    *fo = ex2((m - now) + (r - rn));
    m = now;
    r = rn;
  }
  // r - v, v not below r - 64.
  __device__ __forceinline__ float depth(float v) const { return fminf(r - v, kDeep); }
};

// Two weights as fp16.  With scores beyond 2^24, whose rounding exceeds the
// references' slack, a weight may pass fp16's largest: it is cut off there.
__device__ __forceinline__ uint32_t weights_f16(float x, float y) {
  uint32_t w;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(y), "f"(x));
  return w;
}

// s = f * 2^e with f in (1/2, 1]; f is smaller below 2^-126, and 0 for s = 0.
__device__ __forceinline__ float scale_exponent(float s, float* f) {
  const uint32_t bits = __float_as_uint(s), frac = bits & 0x7fffffu;
  const int field = (int)(bits >> 23 & 255u);  // without the sign: -0 is 0
  if (field == 0) {
    *f = s * 0x1p126f;
    return -126.f;
  }
  *f = frac ? __uint_as_float(126u << 23 | frac) : 1.f;
  return (float)(field - 127 + (frac != 0));
}

// 2^r / l as two factors that are in range one by one (|r| < 200); both 0 for l = 0.
__device__ __forceinline__ float2 result_factors(float l, float r) {
  const float lo = floorf(0.5f * r);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  return make_float2(inv * __uint_as_float((uint32_t)((int)lo + 127) << 23),
                     __uint_as_float((uint32_t)((int)(r - lo) + 127) << 23));
}

// Partial result slots: floats of one (ROWS x D of o, then m, r and l).
template <int ROWS>
__host__ __device__ constexpr size_t part_floats(int D) { return (size_t)ROWS * (D + 3); }

// desc words per CTA: {request, head, row tile, last CTA of the unit, its rows}; -1: none.
constexpr int kDescWords = 8;

// Four e4m3 bytes as two fp16 pairs.
__device__ __forceinline__ void e4m3x4_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Two of Q's elements as fp16.
__device__ __forceinline__ uint32_t half2_of(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Bytes of w that are NaN codes, as bit 7 of each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

__device__ __forceinline__ float2 as_float2(uint32_t w, __nv_bfloat16*) {
  return make_float2(bf16_lo(w), bf16_hi(w));
}
__device__ __forceinline__ float2 as_float2(uint32_t w, __half*) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ uint32_t pack_out(float x, float y, __nv_bfloat16*) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_out(float x, float y, __half*) {
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// lse of a row from its maximum (log2 units) and sum (times 2^kPBits).
__device__ __forceinline__ float row_lse(float M, float L) {
  return L == 0.f ? -INFINITY : (M + log2f(L) - kPBits) * 0.69314718055994531f;
}

// Joins the units that several CTAs worked on: CTA (i, y) serves rows
// [16 y, 16 y + 16) of the unit that began in CTA i and did not end there.  A
// warp per row, or 2, 4 or 8 where the unit has few: these take turns at the
// parts, kJoinBatch parts' loads in flight together, and are joined in the
// end, in an order that depends on the division alone, so the result does not
// depend on timing.
constexpr int kJoinRows = 16;
constexpr int kJoinBatch = 3;  // 6 spill: one token over 30000 positions 27.5 us instead of 26.4
constexpr int kJoinThreads = kJoinRows * 32;

// A row's partial result: its references, l and the E elements of o of a lane.
template <int E>
struct Part {
  float m, r, l, x[E];
};

// Adds N parts to one: their references first, so that no part waits for another's factors.
template <int E, int N>
__device__ __forceinline__ void add_parts(Part<E>& s, const Part<E> (&p)[N]) {
  float now = s.m;
#pragma unroll
  for (int k = 0; k < N; ++k) now = fmaxf(now, p[k].m);
  float rn = s.m - now + s.r;
#pragma unroll
  for (int k = 0; k < N; ++k) rn = fmaxf(rn, p[k].m - now + p[k].r);
  rn = floorf(rn);
  const float fl = ex2(s.m - now), fo = ex2((s.m - now) + (s.r - rn));
  s.m = now;
  s.r = rn;
  s.l *= fl;
#pragma unroll
  for (int e = 0; e < E; ++e) s.x[e] *= fo;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float d = p[k].m - now, f = ex2(d + (p[k].r - rn));
    s.l = fmaf(p[k].l, ex2(d), s.l);
#pragma unroll
    for (int e = 0; e < E; ++e) s.x[e] = fmaf(p[k].x[e], f, s.x[e]);
  }
}

template <class T, int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads, 2) attend_join_kernel(const AttendArgs a) {
  constexpr int E = D / 32;  // elements of a lane: 2 or 4
  __shared__ Part<E> sPart[kJoinRows][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int first = blockIdx.x;
  const int4 d = reinterpret_cast<const int4*>(a.desc)[2 * first];
  const int rows = reinterpret_cast<const int*>(a.desc)[8 * first + 4];
  if (d.x < 0) return;
  const int last = d.w, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int mine = min(rows - (int)blockIdx.y * kJoinRows, kJoinRows);  // this CTA's rows
  if (mine <= 0) return;
  const int sets = mine > 8 ? 1 : mine > 4 ? 2 : mine > 2 ? 4 : 8;
  const int set = warp % sets, r = blockIdx.y * kJoinRows + warp / sets;
  const bool real = warp / sets < mine;
  Part<E> sum{kNone, 0.f, 0.f, {}};
  if (real) {
    for (int i = first + set; i <= last; i += sets * kJoinBatch) {
      Part<E> part[kJoinBatch];
#pragma unroll
      for (int k = 0; k < kJoinBatch; ++k) {
        const int at = i + k * sets;
        const float* p = a.part + (2 * (size_t)at + (at == first)) * part_floats<ROWS>(D);
        part[k] = Part<E>{kNone, 0.f, 0.f, {}};
        if (at <= last) {
          part[k].m = p[ROWS * D + r];
          part[k].r = p[ROWS * (D + 1) + r];
          part[k].l = p[ROWS * (D + 2) + r];
          if (E == 4) {
            const float4 z = reinterpret_cast<const float4*>(p + r * D)[lane];
            part[k].x[0] = z.x, part[k].x[1] = z.y, part[k].x[E - 2] = z.z, part[k].x[E - 1] = z.w;
          } else {
            const float2 z = reinterpret_cast<const float2*>(p + r * D)[lane];
            part[k].x[0] = z.x, part[k].x[1] = z.y;
          }
        }
      }
      add_parts(sum, part);
    }
  }
  if (sets > 1) {
    if (set) sPart[warp][lane] = sum;
    __syncthreads();
    if (!set)
      for (int k = 1; k < sets; ++k) {
        const Part<E> part[1] = {sPart[warp + k][lane]};
        add_parts(sum, part);
      }
  }
  if (set || !real) return;
  const long row = (long)d.z * ROWS + r;
  const int i = (int)(row / a.G), head = d.y * a.G + (int)(row % a.G);
  const size_t orow = ((size_t)d.x * a.W + i) * a.Hq + head;
  const float2 f = result_factors(sum.l, sum.r);
  uint32_t y[E / 2];
#pragma unroll
  for (int e = 0; e < E; e += 2)
    y[e / 2] = pack_out(sum.x[e] * f.x * f.y, sum.x[e + 1] * f.x * f.y, (T*)nullptr);
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + 2 * (orow * D + lane * E));
  if (E == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[E / 2 - 1]);
  else
    dst[0] = y[0];
  if (a.lse && lane == 0) a.lse[orow] = row_lse(sum.m, sum.l);
}

template <class T, int D, int ROWS>
cudaError_t launch_join(const AttendArgs& a, int ctas, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, min(ROWS, ceil_div((long)a.W * a.G, 16) * 16) / kJoinRows);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_join_kernel<T, D, ROWS>, a);
}

constexpr int kSms = 152;

// attend_rows.cu: few rows per KV head.
size_t attend_rows_scratch(int D);
cudaError_t launch_attend_rows(AttendArgs& a, int dtype, void* scratch, cudaStream_t st);
// attend_tiles.cu: many rows per KV head.
size_t attend_tiles_scratch(int D);
cudaError_t launch_attend_tiles(AttendArgs& a, int dtype, void* scratch, cudaStream_t st);

}  // namespace sv

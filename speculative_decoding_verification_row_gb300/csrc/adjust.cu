// Penalties, biases and grammar masks on the logits of a window's rows
// (spec_adjust_logits).
//
// A CTA takes a segment of one request's vocabulary and a run of its rows.  It
// counts the request's tokens that fall into the segment in shared memory (the
// history is read again for every segment: some KB from L2 beside the
// segment's rows, and no counts to keep, clear or roll back between calls) and
// lists the tokens that change; meanwhile its other half copies the rows as
// 16-byte vectors (in place: touches them only where a grammar bans something).
// Then the listed tokens of every row, one by one, over what was copied.  (One
// pass that looked for them in every vector was bound by instructions: 149 us
// for 64 x 8 rows of 128256; counting before copying took 90.)
//
// In a graph: 64 x 8 rows of 128256 (bf16) with 4096 tokens and 16 biases each
// 58 us, 4.5 TB/s (0.66 of the measured copy rate), with 60000 tokens each, which
// every segment reads, 197; 16 trees of 60 rows of
// 151936 under 40 grammars 122 us; a grammar in place on 256 x 4 rows of 129280
// 60 us; one row of 32000 (fp32) 5.6 us, latency.
#include <cuda_bf16.h>

#include "kernels.cuh"

namespace sv {

namespace {

struct AdjustArgs {
  const char* in;
  char* out;
  int B, R, V;
  const int32_t* tokens;  // null: nothing is counted
  const int32_t* token_lens;
  const int32_t* prompt_lens;
  int T;
  const int32_t* drafts;  // null: none, or nothing is counted
  int M;                  // window tokens of a request
  const int32_t* masks;
  const int32_t* draft_lens;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_ids;
  const float* bias_values;
  int bias;
  const int32_t* allowed;
  const int32_t* allowed_rows;
  int num_allowed;
  int segs, splits, rows;  // segments of V, runs of rows, rows of a run
};

constexpr int kSeg = 4096;  // tokens of a segment
constexpr int kBuilders = kThreads / 2;  // threads that count; the others begin with the rows
// A token's word: it stands in the prompt, in the window, it has a bias; and its times in the output.
constexpr uint32_t kPrompt = 1u << 31, kDraft = 1u << 30, kBiased = 1u << 29, kTimes = kBiased - 1;

// Eight bits from bit t on of n words; clear behind them.
__device__ __forceinline__ uint32_t bits8(const int32_t* words, int n, int t) {
  const int w = t >> 5;
  const uint32_t lo = (uint32_t)words[w];
  const uint32_t hi = (t & 31) > 24 && w + 1 < n ? (uint32_t)words[w + 1] : 0u;
  return __funnelshift_r(lo, hi, t & 31) & 255u;
}

// DT: SPEC_F32 or SPEC_BF16.  VEC: 16-byte vectors (the rows of in and out lie
// alike in them, wherever they begin), else single elements.  SAME: in place.
// BAN: there are grammars.
template <int DT, bool VEC, bool SAME, bool BAN>
__global__ void __launch_bounds__(kThreads, 6) adjust_kernel(const AdjustArgs a) {
  using Vec = Io<DT, VEC>;
  constexpr int E = Vec::EPV, ES = Vec::ES;
  constexpr int U = 4;  // vectors in flight per thread
  constexpr uint32_t kAll = (1u << E) - 1;
  extern __shared__ __align__(16) uint32_t smem[];  // cleared as 16-byte vectors
  __shared__ int sListed, sDrafts, sBiased, sNext;
  int* masked = reinterpret_cast<int*>(smem);                   // rows' grammars
  uint32_t* count = smem + (BAN ? (a.rows + 3) & ~3 : 0);       // [kSeg] tokens' words
  uint32_t* draft = count + kSeg;                               // the window's: number << 16 | place
  uint32_t* biased = draft + (a.drafts ? a.M : 0);              // biased places
  float* bias = reinterpret_cast<float*>(biased + a.bias);      // and their biases
  uint16_t* list = reinterpret_cast<uint16_t*>(bias + a.bias);  // places whose word is not 0
  const int tid = threadIdx.x, lane = tid & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int u = blockIdx.x;
  const int seg = u % a.segs;
  u /= a.segs;
  const int b = u / a.splits, r0 = u % a.splits * a.rows;
  int rows = min(a.rows, a.R - r0);
  if (a.draft_lens) {
    const int kb = a.draft_lens[b];
    if (kb < 0 || kb >= a.R) return;
    rows = min(rows, kb + 1 - r0);
  }
  if (rows <= 0) return;
  const int s0 = seg * kSeg, len = min(kSeg, a.V - s0);
  const size_t row0 = (size_t)b * a.R + r0;
  const int words = (a.V + 31) >> 5;
  const bool changes = a.tokens || a.drafts || a.bias;
  if (tid == 0) sListed = sDrafts = sBiased = sNext = 0;
  if (BAN)
    for (int r = tid; r < rows; r += kThreads) masked[r] = a.allowed_rows ? a.allowed_rows[row0 + r] : (int)(row0 + r);
  __syncthreads();

  // ---- the tokens that change
  if (changes && tid < kBuilders) {
    for (int i = tid; i < kSeg / 4; i += kBuilders) reinterpret_cast<uint4*>(count)[i] = make_uint4(0, 0, 0, 0);
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(kBuilders) : "memory");
    auto enlist = [&](int o, uint32_t before) {
      if (before == 0) list[atomicAdd(&sListed, 1)] = (uint16_t)o;
    };
    if (a.tokens) {
      const int n = a.token_lens ? min(max(a.token_lens[b], 0), a.T) : a.T;
      const int p = a.prompt_lens ? min(max(a.prompt_lens[b], 0), n) : 0;
      const int32_t* tokens = a.tokens + (size_t)b * a.T;
      constexpr int N = 16;  // loads in flight: the atomics below keep the compiler from gathering them
      for (int i0 = tid; i0 < n; i0 += kBuilders * N) {
        int t[N];
#pragma unroll
        for (int y = 0; y < N; ++y) t[y] = i0 + y * kBuilders < n ? tokens[i0 + y * kBuilders] : -1;
#pragma unroll
        for (int y = 0; y < N; ++y) {
          const int o = t[y] - s0;
          if (t[y] >= 0 && (unsigned)o < (unsigned)len)
            enlist(o, i0 + y * kBuilders < p ? atomicOr(&count[o], kPrompt) : atomicAdd(&count[o], 1u));
        }
      }
    }
    if (a.drafts)
      for (int m = tid; m < a.M; m += kBuilders) {
        const int t = a.drafts[(size_t)b * a.M + m], o = t - s0;
        if (t >= 0 && (unsigned)o < (unsigned)len) {
          draft[atomicAdd(&sDrafts, 1)] = (uint32_t)m << 16 | (uint32_t)o;
          enlist(o, atomicOr(&count[o], kDraft));
        }
      }
    const int32_t* ids = a.bias_ids + (size_t)b * a.bias;
    for (int i = tid; i < a.bias; i += kBuilders) {
      const int t = ids[i], o = t - s0;
      if (t < 0 || (unsigned)o >= (unsigned)len) continue;
      bool first = true;  // the first entry of an id adds up all of them
      for (int j = 0; j < i; ++j) first = first && ids[j] != t;
      if (!first) continue;
      float sum = 0.f;
      for (int j = i; j < a.bias; ++j)
        if (ids[j] == t) sum += a.bias_values[(size_t)b * a.bias + j];
      const int at = atomicAdd(&sBiased, 1);
      biased[at] = (uint32_t)o;
      bias[at] = sum;
      enlist(o, atomicOr(&count[o], kBiased));
    }
  }

  // Tokens t, t + 1, ... that the grammar of row r bans, of the bits in `valid`.
  auto banned = [&](int r, int t, uint32_t valid) {
    const int x = masked[r];
    if (x < 0) return 0u;
    if (x >= a.num_allowed) return valid;
    return ~bits8(a.allowed + (size_t)x * words, words, t) & valid;
  };

  // ---- the rows: whole vectors, 32 U of a row to a warp, and the few elements around them
  if (!SAME || BAN) {
    constexpr int kParts = kSeg / E / (32 * U);
    // The first of the segment's tokens at a vector's beginning, in row r.
    auto begin = [&](int r) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(a.in) + ((row0 + r) * a.V + s0) * ES;
      return VEC ? (int)((16 - (at & 15)) & 15) / ES : 0;
    };
    for (;;) {
      int x = 0;
      if (lane == 0) x = atomicAdd(&sNext, 1);
      x = __shfl_sync(~0u, x, 0);
      if (x >= rows * kParts) break;
      const int r = x / kParts, v0 = x % kParts * (32 * U) + lane, head = begin(r);
      const int vecs = (len - head) / E;
      const size_t at = ((row0 + r) * a.V + s0 + head) * ES + (size_t)v0 * (E * ES);
      const char* in = a.in + at;
      char* out = a.out + at;
      uint32_t bans[U];
#pragma unroll
      for (int y = 0; y < U; ++y)
        bans[y] = BAN && v0 + 32 * y < vecs ? banned(r, s0 + head + (v0 + 32 * y) * E, kAll) : 0u;
      uint32_t w[U][Vec::NW];
#pragma unroll
      for (int y = 0; y < U; ++y) {
        if (v0 + 32 * y >= vecs || (BAN && bans[y] == kAll) || (SAME && bans[y] == 0)) continue;
        const char* p = in + 32 * y * E * ES;
        if constexpr (SAME && VEC) {  // not through the read-only path: this kernel writes it
          const uint4 z = *reinterpret_cast<const uint4*>(p);
          w[y][0] = z.x, w[y][1] = z.y, w[y][2] = z.z, w[y][3] = z.w;
        } else {
          Vec::load(p, 0, w[y]);
        }
      }
#pragma unroll
      for (int y = 0; y < U; ++y) {
        if (v0 + 32 * y >= vecs || (SAME && bans[y] == 0)) continue;
        if (BAN && bans[y]) {
          if constexpr (DT == SPEC_F32) {
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (bans[y] >> e & 1) w[y][e] = 0xff800000u;
          } else if constexpr (VEC) {
#pragma unroll
            for (int e = 0; e < E; e += 2) {  // -inf is 0xff80
              const uint32_t m = (bans[y] >> e & 1 ? 0xffffu : 0u) | (bans[y] >> e & 2 ? 0xffff0000u : 0u);
              w[y][e / 2] = (w[y][e / 2] & ~m) | (0xff80ff80u & m);
            }
          } else {
            w[y][0] = 0xff800000u;
          }
        }
        char* p = out + 32 * y * E * ES;
        if constexpr (VEC)
          *reinterpret_cast<uint4*>(p) = make_uint4(w[y][0], w[y][1], w[y][2], w[y][3]);
        else if constexpr (DT == SPEC_BF16)
          *reinterpret_cast<unsigned short*>(p) = (unsigned short)(w[y][0] >> 16);
        else
          *reinterpret_cast<uint32_t*>(p) = w[y][0];
      }
    }
    if (VEC)
      for (int x = tid; x < rows * 2 * E; x += kThreads) {
        const int r = x / (2 * E), e = x % (2 * E), head = begin(r);
        // the first E of a row stand for its head, the others for its tail
        const int o = e < E ? e : head + max(0, (len - head) / E * E) + e - E;
        if (e < E ? e >= min(head, len) : o >= len || head >= len) continue;
        const size_t at = ((row0 + r) * a.V + s0 + o) * ES;
        const bool ban = BAN && banned(r, s0 + o, 1u);
        if (SAME && !ban) continue;
        const float z = ban ? -INFINITY : load_logit<DT>(a.in + at, 0);
        if (DT == SPEC_BF16)
          *reinterpret_cast<unsigned short*>(a.out + at) = (unsigned short)(__float_as_uint(z) >> 16);
        else
          *reinterpret_cast<float*>(a.out + at) = z;
      }
  }
  if (!changes) return;

  // ---- the listed tokens of every row, over what was written above
  const float rep = a.repetition ? a.repetition[b] : 1.f;
  const float freq = a.frequency ? a.frequency[b] : 0.f;
  const float pres = a.presence ? a.presence[b] : 0.f;
  __syncthreads();
  const int listed = sListed, all = rows * listed;
  constexpr int N = 2;  // in flight per thread
  for (int x0 = tid; x0 < all; x0 += kThreads * N) {
    float z[N];
    int o[N];
    size_t row[N];
#pragma unroll
    for (int y = 0; y < N; ++y) {
      const int x = min(x0 + y * kThreads, all - 1), r = (unsigned)x / (unsigned)listed;
      o[y] = list[x - r * listed];
      row[y] = row0 + r;
      z[y] = load_logit<DT>(a.in + (row[y] * a.V + s0) * ES, o[y]);
    }
#pragma unroll
    for (int y = 0; y < N; ++y) {
      if (x0 + y * kThreads >= all) break;
      if (BAN && banned((int)(row[y] - row0), s0 + o[y], 1u)) continue;
      const uint32_t w = count[o[y]];
      int c = (int)(w & kTimes);
      if (w & kDraft) {
        const int32_t* tree = a.masks ? a.masks + row[y] * ((a.R + 31) >> 5) : nullptr;
        const int r = (int)(row[y] - (size_t)b * a.R);
        for (int i = 0; i < sDrafts; ++i) {
          const int m = (int)(draft[i] >> 16);
          if ((int)(draft[i] & 0xffffu) == o[y]) c += tree ? m > 0 && tree[m >> 5] >> (m & 31) & 1 : m < r;
        }
      }
      float x = z[y];
      if (c > 0 || w & kPrompt) x = x > 0.f ? x / rep : x * rep;
      if (c > 0) x = x - freq * (float)c - pres;
      if (w & kBiased) {
        int i = 0;
        while ((int)biased[i] != o[y]) ++i;
        x += bias[i];
      }
      char* out = a.out + (row[y] * a.V + s0 + o[y]) * ES;
      if (DT == SPEC_BF16)
        *reinterpret_cast<__nv_bfloat16*>(out) = __float2bfloat16_rn(x);
      else
        *reinterpret_cast<float*>(out) = x;
    }
  }
}

template <int DT, bool VEC, bool SAME>
cudaError_t launch_as(const AdjustArgs& a, long grid, size_t smem, cudaStream_t st) {
  return a.allowed ? launch_first(adjust_kernel<DT, VEC, SAME, true>, grid, kThreads, st, a, smem)
                   : launch_first(adjust_kernel<DT, VEC, SAME, false>, grid, kThreads, st, a, smem);
}

template <int DT>
cudaError_t launch(const AdjustArgs& a, bool vec, long grid, size_t smem, cudaStream_t st) {
  if (a.in == a.out) return launch_as<DT, true, true>(a, grid, smem, st);
  return vec ? launch_as<DT, true, false>(a, grid, smem, st) : launch_as<DT, false, false>(a, grid, smem, st);
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" int spec_adjust_logits(const spec_adjust_params* p, spec_stream_t stream) {
  if (!p || p->size != sizeof(spec_adjust_params) || !p->logits || !p->out ||
      (p->dtype != SPEC_F32 && p->dtype != SPEC_BF16) || p->B < 1 || p->B > SPEC_MAX_BATCH || p->R < 1 ||
      p->R > SPEC_MAX_TREE_NODES || p->V < 2 || p->V > INT_MAX - kSeg)
    return SPEC_EINVAL;
  const size_t es = p->dtype == SPEC_F32 ? 4 : 2;
  const uintptr_t in = reinterpret_cast<uintptr_t>(p->logits), out = reinterpret_cast<uintptr_t>(p->out);
  const size_t bytes = (size_t)p->B * p->R * p->V * es;
  if (in % es || out % es || (in != out && in < out + bytes && out < in + bytes)) return SPEC_EINVAL;
  if ((p->tokens && (p->T < 1 || p->T >= 1 << 29)) || (p->masks && (!p->draft_tokens || p->draft_lens)) ||
      (p->bias_ids && (!p->bias_values || p->num_bias < 1 || p->num_bias > SPEC_MAX_BIAS)) ||
      (p->allowed && p->num_allowed < 1) || (!p->allowed && p->allowed_rows) ||
      (p->allowed && !p->allowed_rows && p->num_allowed != (long)p->B * p->R))
    return SPEC_EINVAL;
  AdjustArgs a{};
  a.in = static_cast<const char*>(p->logits);
  a.out = static_cast<char*>(p->out);
  a.B = p->B;
  a.R = p->R;
  a.V = p->V;
  if (p->repetition || p->frequency || p->presence) {  // else the tokens change nothing
    a.tokens = p->tokens;
    a.T = p->T;
    a.M = p->masks ? p->R : p->R - 1;
    a.drafts = a.M ? p->draft_tokens : nullptr;
  }
  a.token_lens = p->token_lens;
  a.prompt_lens = p->prompt_lens;
  a.masks = p->masks;
  a.draft_lens = p->draft_lens;
  a.repetition = p->repetition;
  a.frequency = p->frequency;
  a.presence = p->presence;
  a.bias_ids = p->bias_ids;
  a.bias_values = p->bias_values;
  a.bias = p->bias_ids ? p->num_bias : 0;
  a.allowed = p->allowed;
  a.allowed_rows = p->allowed_rows;
  a.num_allowed = p->num_allowed;
  a.segs = ceil_div(a.V, kSeg);
  const long units = (long)a.B * a.segs;
  a.rows = ceil_div(a.R, min((long)a.R, max(1l, 8l * 152 / units)));
  a.splits = ceil_div(a.R, a.rows);
  if (units * a.splits > INT_MAX) return SPEC_EINVAL;
  const bool changes = a.tokens || a.drafts || a.bias_ids;
  const size_t smem = (changes ? kSeg * 6 + ((a.drafts ? a.M : 0) + 2 * a.bias) * 4 : 0) +
                      (a.allowed ? (a.rows + 3) / 4 * 16 : 0);
  const bool vec = (in - out) % 16 == 0;
  const cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = p->dtype == SPEC_F32 ? launch<SPEC_F32>(a, vec, units * a.splits, smem, st)
                                             : launch<SPEC_BF16>(a, vec, units * a.splits, smem, st);
  return e == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}

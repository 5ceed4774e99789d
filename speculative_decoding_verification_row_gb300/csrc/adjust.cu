// Penalties, biases and grammar masks on the logits of a window's rows
// (spec_adjust_logits).
//
// One pass over the logits.  A CTA takes a segment of one request's
// vocabulary and a run of its rows: it counts the request's tokens that fall
// into the segment in shared memory (the history is read again for every
// segment: some KB from L2 beside the segment's rows, and no counts to keep,
// clear or roll back between calls), and marks in a bitmap every token that
// some row changes.  A vector of logits without a mark and without a banned
// token is copied, or in place not read at all; one whose tokens are all
// banned is not read either.
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
// A token's word: it stands in the prompt, in the window, and its times in the output.
constexpr uint32_t kPrompt = 1u << 31, kDraft = 1u << 30;

// Eight bits from bit t (above -8) of n words; clear outside them.
__device__ __forceinline__ uint32_t bits8(const int32_t* words, int n, int t) {
  if (t < 0) return n > 0 ? (uint32_t)words[0] << -t & 255u : 0u;
  const int w = t >> 5;
  const uint32_t lo = w < n ? (uint32_t)words[w] : 0u;
  const uint32_t hi = (t & 31) > 24 && w + 1 < n ? (uint32_t)words[w + 1] : 0u;
  return __funnelshift_r(lo, hi, t & 31) & 255u;
}

__device__ __forceinline__ uint32_t to_bf16(float x) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// DT: SPEC_F32 or SPEC_BF16.  VEC: 16-byte vectors (the rows of in and out lie
// alike in them, wherever they begin), else single elements.  SAME: in place.
template <int DT, bool VEC, bool SAME>
__global__ void __launch_bounds__(kThreads) adjust_kernel(const AdjustArgs a) {
  using Vec = Io<DT, VEC>;
  constexpr int E = Vec::EPV, ES = Vec::ES;
  constexpr int U = kSeg / kThreads / E < 4 ? kSeg / kThreads / E : 4;  // vectors in flight per thread
  constexpr uint32_t kAll = (1u << E) - 1;
  extern __shared__ uint32_t smem[];
  __shared__ int32_t sMark[kSeg / 32];
  __shared__ uint32_t sDraft[SPEC_MAX_TREE_NODES];  // window tokens of the segment: number << 16 | place
  __shared__ int sDrafts;
  uint32_t* count = smem;  // [kSeg] where tokens are counted
  const bool counts = a.tokens || a.drafts;
  float* bias = reinterpret_cast<float*>(smem + (counts ? kSeg : 0));  // [kSeg] where there are biases
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int u = blockIdx.x;
  const int seg = u % a.segs;
  u /= a.segs;
  const int b = u / a.splits, r0 = u % a.splits * a.rows;
  int r1 = min(a.R, r0 + a.rows);
  if (a.draft_lens) {
    const int kb = a.draft_lens[b];
    if (kb < 0 || kb >= a.R) return;
    r1 = min(r1, kb + 1);
  }
  if (r0 >= r1) return;
  const int s0 = seg * kSeg, len = min(kSeg, a.V - s0);

  // ---- what the segment's rows change
  for (int i = tid; i < kSeg / 32; i += kThreads) sMark[i] = 0;
  if (tid == 0) sDrafts = 0;
  if (counts)
    for (int i = tid; i < kSeg / 4; i += kThreads) reinterpret_cast<uint4*>(count)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  auto mark = [&](int o) { atomicOr(&sMark[o >> 5], (int)(1u << (o & 31))); };
  if (a.tokens) {
    const int n = a.token_lens ? min(max(a.token_lens[b], 0), a.T) : a.T;
    const int p = a.prompt_lens ? min(max(a.prompt_lens[b], 0), n) : 0;
    const int32_t* tokens = a.tokens + (size_t)b * a.T;
#pragma unroll 4
    for (int i = tid; i < n; i += kThreads) {
      const int o = tokens[i] - s0;
      if (tokens[i] >= 0 && (unsigned)o < (unsigned)len) {
        if (i < p)
          atomicOr(&count[o], kPrompt);
        else
          atomicAdd(&count[o], 1u);
        mark(o);
      }
    }
  }
  if (a.drafts)
    for (int m = tid; m < a.M; m += kThreads) {
      const int t = a.drafts[(size_t)b * a.M + m], o = t - s0;
      if (t >= 0 && (unsigned)o < (unsigned)len) {
        atomicOr(&count[o], kDraft);
        sDraft[atomicAdd(&sDrafts, 1)] = (uint32_t)m << 16 | (uint32_t)o;
        mark(o);
      }
    }
  if (a.bias_ids) {
    const int32_t* ids = a.bias_ids + (size_t)b * a.bias;
    for (int i = tid; i < kSeg; i += kThreads) bias[i] = 0.f;
    __syncthreads();
    for (int i = tid; i < a.bias; i += kThreads) {
      const int t = ids[i], o = t - s0;
      if (t < 0 || (unsigned)o >= (unsigned)len) continue;
      bool first = true;  // the first entry of an id adds up all of them
      for (int j = 0; j < i; ++j) first = first && ids[j] != t;
      if (!first) continue;
      float sum = 0.f;
      for (int j = i; j < a.bias; ++j)
        if (ids[j] == t) sum += a.bias_values[(size_t)b * a.bias + j];
      bias[o] = sum;
      mark(o);
    }
  }
  __syncthreads();
  const float rep = a.repetition ? a.repetition[b] : 1.f;
  const float freq = a.frequency ? a.frequency[b] : 0.f;
  const float pres = a.presence ? a.presence[b] : 0.f;
  const int words = (a.V + 31) >> 5;

  for (int r = r0; r < r1; ++r) {
    const size_t row = (size_t)b * a.R + r, at = (row * a.V + s0) * ES;
    const char* in = a.in + at;
    const int shift = VEC ? (int)(reinterpret_cast<uintptr_t>(in) & 15) / ES : 0;
    in -= shift * ES;
    char* out = a.out + at - shift * ES;
    const int nvec = (len + shift + E - 1) / E;
    const int32_t* allowed = nullptr;
    int have = words;  // words of the mask; 0: everything is banned
    if (a.allowed) {
      const int x = a.allowed_rows ? a.allowed_rows[row] : (int)row;
      if (x >= 0) allowed = a.allowed + (x < a.num_allowed ? (size_t)x * words : 0);
      if (x >= a.num_allowed) have = 0;
    }
    const int32_t* tree = a.masks ? a.masks + row * ((a.R + 31) >> 5) : nullptr;
    auto change = [&](float x, int o) {
      if (counts) {
        const uint32_t w = count[o];
        int c = (int)(w & (kDraft - 1));
        if (w & kDraft)
          for (int i = 0; i < sDrafts; ++i) {
            const int m = (int)(sDraft[i] >> 16);
            if ((int)(sDraft[i] & 0xffffu) == o) c += tree ? m > 0 && tree[m >> 5] >> (m & 31) & 1 : m < r;
          }
        if (c > 0 || w & kPrompt) x = x > 0.f ? x / rep : x * rep;
        if (c > 0) x = x - freq * (float)c - pres;
      }
      return a.bias_ids ? x + bias[o] : x;
    };
    for (int v0 = tid; v0 < nvec; v0 += kThreads * U) {
      uint32_t w[U][Vec::NW], marks[U], bans[U], valid[U];
#pragma unroll
      for (int y = 0; y < U; ++y) {
        const int v = v0 + y * kThreads, o = v * E - shift;
        valid[y] = v < nvec ? kAll : 0u;
        if (o < 0) valid[y] &= kAll << -o;
        if (o + E > len) valid[y] &= len > o ? kAll >> (o + E - len) : 0u;
        marks[y] = bans[y] = 0;
        if (valid[y]) {
          marks[y] = bits8(sMark, kSeg / 32, o) & valid[y];
          if (allowed) bans[y] = ~bits8(allowed, have, s0 + o) & valid[y];
        }
        marks[y] &= ~bans[y];
        const bool all = bans[y] == kAll;
        if (valid[y] == kAll && !all && (!SAME || (marks[y] | bans[y]))) {
          if constexpr (SAME && VEC) {  // not through the read-only path: this kernel writes it
            const uint4 z = *reinterpret_cast<const uint4*>(in + (size_t)v * 16);
            w[y][0] = z.x, w[y][1] = z.y, w[y][2] = z.z, w[y][3] = z.w;
          } else if constexpr (SAME) {
            w[y][0] = __float_as_uint(load_logit<DT>(in, v));
          } else {
            Vec::load(in, v, w[y]);
          }
        }
      }
#pragma unroll
      for (int y = 0; y < U; ++y) {
        const int v = v0 + y * kThreads, o = v * E - shift;
        if (valid[y] == 0 || (SAME && !(marks[y] | bans[y]))) continue;
        if (valid[y] != kAll) {  // a row's or segment's edge inside a vector
          for (int e = 0; e < E; ++e) {
            if (!(valid[y] >> e & 1)) continue;
            float x = load_logit<DT>(in, v * E + e);
            if (marks[y] >> e & 1) x = change(x, o + e);
            if (bans[y] >> e & 1) x = -INFINITY;
            if (DT == SPEC_BF16)
              reinterpret_cast<unsigned short*>(out)[v * E + e] = (unsigned short)to_bf16(x);
            else
              reinterpret_cast<float*>(out)[v * E + e] = x;
          }
          continue;
        }
        float x[E];
        if (marks[y] | bans[y]) {
          if (bans[y] != kAll) Vec::unpack(w[y], x);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (marks[y] >> e & 1) x[e] = change(x[e], o + e);
            if (bans[y] >> e & 1) x[e] = -INFINITY;
          }
          if constexpr (DT == SPEC_F32) {
#pragma unroll
            for (int e = 0; e < E; ++e) w[y][e] = __float_as_uint(x[e]);
          } else if constexpr (VEC) {
#pragma unroll
            for (int e = 0; e < E; e += 2) w[y][e / 2] = to_bf16(x[e]) | to_bf16(x[e + 1]) << 16;
          } else {
            w[y][0] = to_bf16(x[0]) << 16;
          }
        }
        if constexpr (VEC)
          *reinterpret_cast<uint4*>(out + (size_t)v * 16) = make_uint4(w[y][0], w[y][1], w[y][2], w[y][3]);
        else if constexpr (DT == SPEC_BF16)
          reinterpret_cast<unsigned short*>(out)[v] = (unsigned short)(w[y][0] >> 16);
        else
          reinterpret_cast<uint32_t*>(out)[v] = w[y][0];
      }
    }
  }
}

template <int DT, bool VEC>
cudaError_t launch(const AdjustArgs& a, long grid, size_t smem, cudaStream_t st) {
  return a.in == a.out ? launch_first(adjust_kernel<DT, VEC, true>, grid, kThreads, st, a, smem)
                       : launch_first(adjust_kernel<DT, VEC, false>, grid, kThreads, st, a, smem);
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
  if ((p->tokens && (p->T < 1 || p->T >= 1 << 30)) || (p->masks && (!p->draft_tokens || p->draft_lens)) ||
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
  a.bias = p->num_bias;
  a.allowed = p->allowed;
  a.allowed_rows = p->allowed_rows;
  a.num_allowed = p->num_allowed;
  a.segs = ceil_div(a.V, kSeg);
  const long units = (long)a.B * a.segs;
  a.rows = ceil_div(a.R, min((long)a.R, max(1l, 8l * 152 / units)));
  a.splits = ceil_div(a.R, a.rows);
  if (units * a.splits > INT_MAX) return SPEC_EINVAL;
  const size_t smem = ((a.tokens || a.drafts ? kSeg : 0) + (a.bias_ids ? kSeg : 0)) * 4;
  const bool vec = (in - out) % 16 == 0;
  const cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = p->dtype == SPEC_F32
                            ? (vec ? launch<SPEC_F32, true>(a, units * a.splits, smem, st)
                                   : launch<SPEC_F32, false>(a, units * a.splits, smem, st))
                            : (vec ? launch<SPEC_BF16, true>(a, units * a.splits, smem, st)
                                   : launch<SPEC_BF16, false>(a, units * a.splits, smem, st));
  return e == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}

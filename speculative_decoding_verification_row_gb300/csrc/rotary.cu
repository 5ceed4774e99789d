// Rotary positions of a window's queries and keys (spec_rotate_qk).
//
// Bound by the bytes of the rows; at a step's sizes by latency.  A CTA takes
// one token.  An angle is reduced modulo a turn in 64-bit integers (turns_of),
// so a far position costs no precision and no arithmetic in 64-bit floats.
// In a graph: 128032 tokens, 40 heads of 128, 377 us, 7.0 TB/s (as fast as the
// measured copy); 4 x 4001 tokens, 36 heads, 46 us; 64 x 8 tokens, 5.2 us.
#include "rotary.cuh"

namespace sv {

namespace {

template <class T, bool INTER>
__global__ void __launch_bounds__(kTurnThreads) rotate_kernel(const RotateArgs a) {
  __shared__ float2 cs[kMaxPairs];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = blockIdx.x / a.W;
  rotate_token<T, INTER>(a, b, blockIdx.x - b * a.W, cs);
}

template <class T>
cudaError_t launch(const RotateArgs& a, cudaStream_t st) {
  const long grid = (long)a.B * a.W;
  return a.interleaved ? launch_first(rotate_kernel<T, true>, grid, kTurnThreads, st, a)
                       : launch_first(rotate_kernel<T, false>, grid, kTurnThreads, st, a);
}

}  // namespace

int rotate_setup(const spec_rotate_params* p, RotateArgs* a) {
  if (!p || p->size != sizeof(spec_rotate_params) || (p->dtype != SPEC_BF16 && p->dtype != SPEC_F16) ||
      p->B < 1 || p->B > SPEC_MAX_BATCH || p->W < 1 || p->W > SPEC_MAX_WINDOW || p->head_dim < 16 ||
      p->head_dim > 512 || p->head_dim % 16 != 0 || p->pairs < 8 || p->pairs % 8 != 0 ||
      2 * p->pairs > p->head_dim || !p->starts || !p->inv_freq || !isfinite(p->gain) ||
      (p->masks && p->W > SPEC_MAX_TREE_NODES))
    return SPEC_EINVAL;
  const void* in[2] = {p->q, p->k};
  void* out[2] = {p->out_q, p->out_k};
  const int64_t* is[2] = {p->q_strides, p->k_strides};
  const int64_t* os[2] = {p->out_q_strides, p->out_k_strides};
  const int heads[2] = {p->q_heads, p->k_heads};
  for (int x = 0; x < 2; ++x) {
    if (heads[x] < 0 || heads[x] > 16384 || (heads[x] > 0) != (in[x] != nullptr)) return SPEC_EINVAL;
    if (in[x] && !kv_strides_ok(in[x], is[x])) return SPEC_EINVAL;
    if (out[x] && !kv_strides_ok(out[x], os[x])) return SPEC_EINVAL;
    const int n[3] = {p->B, p->W, heads[x]};
    if (in[x] == out[x] && in[x])
      for (int d = 0; d < 3; ++d)
        if (n[d] > 1 && is[x][d] != os[x][d]) return SPEC_EINVAL;  // the stride of an axis of one element is never used
    a->x[x] = RotateRows{static_cast<const char*>(in[x]), static_cast<char*>(out[x]), is[x][0], is[x][1],
                         is[x][2], os[x][0], os[x][1], os[x][2], heads[x]};
  }
  a->B = p->B;
  a->W = p->W;
  a->D = p->head_dim;
  a->starts = p->starts;
  a->win = p->window_lens;
  a->masks = p->masks;
  a->inv_freq = p->inv_freq;
  a->pairs = p->pairs;
  a->interleaved = p->interleaved;
  a->gain = p->gain;
  return SPEC_OK;
}

void rotate_arrays(const spec_rotate_params* p, Arrays* x) {
  const int B = p->B, W = p->W, D = p->head_dim;
  const int q = x->read(strided(p->q, p->q_strides, B, W, p->q_heads, D, 2));
  const int k = x->read(strided(p->k, p->k_strides, B, W, p->k_heads, D, 2));
  x->read(dense(p->starts, (long)B * sizeof(int32_t)));
  x->read(dense(p->window_lens, (long)B * sizeof(int32_t)));
  x->read(dense(p->masks, (long)B * W * ceil_div(W, 32) * sizeof(int32_t)));
  x->read(dense(p->inv_freq, (long)p->pairs * sizeof(double)));
  x->write(strided(p->out_q, p->out_q_strides, B, W, p->q_heads, D, 2), q);
  x->write(strided(p->out_k, p->out_k_strides, B, W, p->k_heads, D, 2), k);
}

cudaError_t launch_rotate(const RotateArgs& a, int dtype, cudaStream_t st) {
  return dtype == SPEC_BF16 ? launch<__nv_bfloat16>(a, st) : launch<__half>(a, st);
}

}  // namespace sv

using namespace sv;

extern "C" int spec_rotate_qk(const spec_rotate_params* p, spec_stream_t stream) {
  RotateArgs a{};
  const int rc = rotate_setup(p, &a);
  if (rc != SPEC_OK) return rc;
  if ((!a.x[0].in && !a.x[1].in) || !a.x[0].in != !a.x[0].out || !a.x[1].in != !a.x[1].out) return SPEC_EINVAL;
  Arrays x;
  rotate_arrays(p, &x);
  if (!x.apart()) return SPEC_EINVAL;
  const cudaError_t e = launch_rotate(a, p->dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}

// Attention of a window's rows over the paged 8-bit cache (spec_attend_kv):
// argument checks and the choice of the kernel.
#include "attend.cuh"

using namespace sv;

namespace {

// Whether attend_rows.cu serves this many rows per KV head; else attend_tiles.cu.
// The first reads the cache once for every 16 rows, the second once for 128 at
// a step's fixed cost.  Measured with 64 requests of 4096 cached positions and
// 8 KV heads: D = 128, rows 106 us for 16 rows and 190 for 20, tiles 169 for
// both; D = 64, rows 68 us for 16 and 120 for 32, tiles 138 (and 224 against
// 141 for 64).  With 4 requests of 30000 and D = 128: rows 59 us for 16 and 91
// for 32, tiles 77.
bool few_rows(int W, int G, int D) { return (long)W * G <= (D == 64 ? 32 : 16); }

}  // namespace

extern "C" {

size_t spec_attend_scratch_size(int B, int W, int q_heads, int kv_heads, int head_dim) {
  if (B < 1 || B > SPEC_MAX_BATCH || W < 1 || W > SPEC_MAX_WINDOW || kv_heads < 1 ||
      kv_heads > 1024 || q_heads < 1 || q_heads > 16384 || q_heads % kv_heads != 0 ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return few_rows(W, q_heads / kv_heads, head_dim) ? attend_rows_scratch(head_dim)
                                         : attend_tiles_scratch(head_dim);
}

int spec_attend_kv(const spec_kv_cache* cache, const spec_attend_params* p, void* scratch,
                   size_t scratch_bytes, spec_stream_t stream) {
  constexpr double kLog2e = 1.4426950408889634073599246810019;
  AttendArgs a{};
  const int rc = kv_setup(cache, &a.c);
  if (rc != SPEC_OK) return rc;
  if (!p || p->size != sizeof(spec_attend_params) || !kv_strides_ok(p->q, p->q_strides) ||
      (p->dtype != SPEC_BF16 && p->dtype != SPEC_F16) || !p->seq_lens || !p->out ||
      reinterpret_cast<uintptr_t>(p->out) % 16 != 0 || !isfinite((float)(p->scale * kLog2e)) ||
      (p->masks && p->W > SPEC_MAX_TREE_NODES) ||
      (long)a.c.max_blocks * a.c.tpb > kMaxPositions ||
      (long)p->B * p->W * p->q_heads > kMaxRows)
    return SPEC_EINVAL;
  const size_t need = spec_attend_scratch_size(p->B, p->W, p->q_heads, a.c.H, a.c.D);
  if (need == 0) return SPEC_EINVAL;
  if (!scratch || reinterpret_cast<uintptr_t>(scratch) % 256 != 0 || scratch_bytes < need)
    return SPEC_EWORKSPACE;
  a.q = static_cast<const char*>(p->q);
  a.qb = p->q_strides[0];
  a.qt = p->q_strides[1];
  a.qh = p->q_strides[2];
  a.B = p->B;
  a.W = p->W;
  a.Hq = p->q_heads;
  a.G = p->q_heads / a.c.H;
  a.seq = p->seq_lens;
  a.win = p->window_lens;
  a.masks = p->masks;
  a.words = (p->W + 31) / 32;
  a.tpb16_div = (unsigned)((1ull << 32) / (a.c.tpb / 16) + ((1ull << 32) % (a.c.tpb / 16) != 0));
  a.scale_log2 = (float)(p->scale * kLog2e);
  a.out = static_cast<char*>(p->out);
  a.lse = p->out_lse;
  const cudaError_t e = few_rows(a.W, a.G, a.c.D)
                            ? launch_attend_rows(a, p->dtype, scratch, (cudaStream_t)stream)
                            : launch_attend_tiles(a, p->dtype, scratch, (cudaStream_t)stream);
  return e == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}

}  // extern "C"

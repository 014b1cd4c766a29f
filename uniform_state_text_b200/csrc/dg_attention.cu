// Attention of a block of new tokens over a paged key/value cache
// (dg_cache_attention).
//
// For one query row, over the keys j it sees, with t_j = scale log2(e) q.k_j:
//   m = max t_j,  l = sum 2^(t_j - m),  out = sum 2^(t_j - m) v_j / l,
//   lse = (m + log2 l) ln 2
// in one pass over the keys: a larger maximum rescales l and the running sum.
#include <cmath>

#include "dg.h"
#include "dg_cache.cuh"
#include "dg_fp8.cuh"

namespace dg {
void set_last_error(const char* msg);
int kv_check(const dg_kv_cache* c, const dg_kv_batch* b);
int kv_row_args(const void* p, int64_t ts, int64_t hs);
int kv_launched(cudaError_t e);

namespace attn {

struct Args {
  KvView w;
  const __nv_bfloat16* q;
  int64_t q_ts, q_hs;
  int q_heads;
  float scale_log2;            // scale log2(e)
  int mask;
  const uint32_t* tree;
  int words;
  __nv_bfloat16* out;
  float* lse;
};

// One warp per (token, query head), 8 elements of head_dim to a lane.
template <bool F8>
__global__ void __launch_bounds__(256) k_attend_rows(const __grid_constant__ Args a) {
  const KvView& w = a.w;
  const int64_t unit = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 32;
  const int lane = threadIdx.x & 31;
  if (unit >= (int64_t)w.b.tokens * a.q_heads) return;
  const int token = (int)(unit / a.q_heads), h = (int)(unit % a.q_heads);
  const int b = kv_sequence(w, token);
  if (b < 0) return;
  int t0;
  const int n = kv_new(w, b, &t0);
  const int i = token - t0, D = w.c.head_dim, kh = h / (a.q_heads / w.c.kv_heads);
  const int64_t past = kv_past(w, b, n);
  const int32_t* table = w.b.page_table + (int64_t)b * w.b.table_stride;
  const int x0 = lane * 8;
  float q[8] = {0, 0, 0, 0, 0, 0, 0, 0}, o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (x0 < D)
    for (int j = 0; j < 8; ++j) q[j] = to_f32(a.q[token * a.q_ts + h * a.q_hs + x0 + j]);
  float m = -INFINITY, l = 0.f;
  for (int64_t p = 0; p < past + n; ++p) {
    if (p >= past) {
      const int node = (int)(p - past);
      if (a.mask == DG_MASK_CAUSAL && node > i) break;
      if (a.mask == DG_MASK_TREE &&
          (node / 32 >= a.words || !(a.tree[(int64_t)token * a.words + node / 32] >> (node % 32) & 1)))
        continue;
    }
    const int row = kv_row(w, table, p, kh);
    float k[8] = {0, 0, 0, 0, 0, 0, 0, 0}, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (row >= 0 && x0 < D) {
      const int64_t at = (int64_t)row * D + x0;
      for (int j = 0; j < 8; ++j) {
        if (F8) {
          k[j] = ldexpf(e4m3_to_f32(static_cast<const uint8_t*>(w.c.k)[at + j]), w.c.k_exp[row] - 127);
          v[j] = ldexpf(e4m3_to_f32(static_cast<const uint8_t*>(w.c.v)[at + j]), w.c.v_exp[row] - 127);
        } else {
          k[j] = to_f32(static_cast<const __nv_bfloat16*>(w.c.k)[at + j]);
          v[j] = to_f32(static_cast<const __nv_bfloat16*>(w.c.v)[at + j]);
        }
      }
    }
    float s = 0.f;
    for (int j = 0; j < 8; ++j) s = fmaf(q[j], k[j], s);
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float t = s * a.scale_log2;
    const float mn = fmaxf(m, t);
    const float c = exp2f(m - mn), e = exp2f(t - mn);
    m = mn;
    l = l * c + e;
    for (int j = 0; j < 8; ++j) o[j] = fmaf(e, v[j], o[j] * c);
  }
  const float r = l > 0.f ? 1.f / l : 0.f;
  if (x0 < D)
    for (int j = 0; j < 8; ++j)
      a.out[unit * D + x0 + j] = __float2bfloat16_rn(l == l ? o[j] * r : l);
  if (a.lse && lane == 0) a.lse[unit] = (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace attn

namespace {
int fail(int code, const char* msg) {
  set_last_error(msg);
  return code;
}
bool off16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }
}  // namespace

}  // namespace dg

using namespace dg;

extern "C" size_t dg_cache_attention_scratch_bytes(const dg_kv_cache* cache, const dg_kv_batch* batch,
                                                   int32_t q_heads) {
  if (kv_check(cache, batch) || q_heads < 1 || q_heads % cache->kv_heads) return 0;
  return 256;
}

extern "C" int dg_cache_attention(const dg_kv_cache* cache, const dg_kv_batch* batch, int32_t q_heads,
                                  const void* q, int64_t q_ts, int64_t q_hs, float scale, int32_t mask,
                                  const uint32_t* tree_mask, int32_t mask_words, void* out, float* lse,
                                  void* scratch, size_t scratch_bytes, void* stream) {
  int rc = kv_check(cache, batch);
  if (rc) return rc;
  if (q_heads < 1 || q_heads % cache->kv_heads) return fail(DG_EINVAL, "q_heads must be a multiple of kv_heads");
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(DG_EINVAL, "scale must be positive and finite");
  if (mask < DG_MASK_FULL || mask > DG_MASK_TREE) return fail(DG_EINVAL, "mask must be one of DG_MASK_*");
  if (mask == DG_MASK_TREE && (mask_words < 0 || (mask_words && !tree_mask)))
    return fail(DG_EINVAL, "DG_MASK_TREE needs tree_mask and mask_words >= 0");
  if (batch->tokens == 0 || batch->batch == 0) return DG_OK;
  if ((rc = kv_row_args(q, q_ts, q_hs))) return rc;
  if (!out || off16(out)) return fail(DG_EINVAL, "out must be 16-byte aligned and not NULL");
  if (!scratch || reinterpret_cast<uintptr_t>(scratch) % 256) return fail(DG_EINVAL, "scratch must be 256-byte aligned and not NULL");
  if (scratch_bytes < dg_cache_attention_scratch_bytes(cache, batch, q_heads))
    return fail(DG_ENOMEM, "scratch is smaller than dg_cache_attention_scratch_bytes()");
  const attn::Args a{{*cache, *batch}, static_cast<const __nv_bfloat16*>(q), q_ts, q_hs, q_heads,
                     scale * 1.4426950408889634f, mask, tree_mask, mask_words,
                     static_cast<__nv_bfloat16*>(out), lse};
  const int64_t grid = ((int64_t)batch->tokens * q_heads + 7) / 8;
  if (grid > 0x7fffffff) return fail(DG_EUNSUPPORTED, "too many rows");
  if (cache->format == DG_KV_E4M3) attn::k_attend_rows<true><<<(unsigned)grid, 256, 0, (cudaStream_t)stream>>>(a);
  else attn::k_attend_rows<false><<<(unsigned)grid, 256, 0, (cudaStream_t)stream>>>(a);
  return kv_launched(cudaGetLastError());
}

// Row operators of an attention layer: per-head norms with rotation
// (dg_qk_norm_rope), and the paged key/value cache's write and read
// (dg_cache_write, dg_cache_read).
//
// Each element is read once and written once, with a few operations between:
// write and read are bound by memory, the norm by the instructions of its rows. A
// row (one token, one head) belongs to a group of 8, 16 or 32 lanes (head_dim up
// to 64, 128, 256), 8 elements to a lane, so that a row is one fully used memory
// transaction per lane and its sums and maxima are a few shuffles; only the norm's
// weights, cosines and sines pass through shared memory.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "dg.h"
#include "dg_cache.cuh"
#include "dg_fp8.cuh"

namespace dg {
void set_last_error(const char* msg);   // dg_api.cu: the message dg_last_error(NULL) returns
}

namespace dg {
namespace rows {

constexpr int THREADS = 256;

// 4 and 8 elements as fp32.
template <typename T> __device__ __forceinline__ void load4(const T* p, float* v);
template <> __device__ __forceinline__ void load4<float>(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
template <> __device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float* v) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(u.x << 16);
  v[1] = __uint_as_float(u.x & 0xFFFF0000u);
  v[2] = __uint_as_float(u.y << 16);
  v[3] = __uint_as_float(u.y & 0xFFFF0000u);
}
template <typename T> __device__ __forceinline__ void store4(T* p, const float* v);
template <> __device__ __forceinline__ void store4<float>(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* p, const float* v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
template <typename T> __device__ __forceinline__ void load8(const T* p, float* v);
template <> __device__ __forceinline__ void load8<float>(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <> __device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float* v) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
template <typename T> __device__ __forceinline__ void store8(T* p, const float* v);
template <> __device__ __forceinline__ void store8<float>(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
template <> __device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------------------
// Norm and rotation.
// ---------------------------------------------------------------------------
struct NormArgs {
  const void *q, *k, *wq, *wk;
  void *qo, *ko;
  int64_t q_ts, q_hs, k_ts, k_hs;
  const int32_t* pos;
  const double* freq;
  int tokens, qh, kh, D, rot;
  int tpb, hpb;                // tokens and heads per block
  float off, eps;
};

// The fraction of a turn per position as a 64-bit fixed-point number: its
// product with an integer position, mod 2^64, is the phase itself, with no
// range reduction. 1 / (2 pi) is taken in two doubles and the product's
// rounding is kept, so that the fraction is right to 2^-63 turns and the phase
// to 2^-32 turns at any int32 position. (Of the magnitude: hi - floor(hi) is
// exact for hi >= 0, but would round for a small negative one. The sign is then
// exact mod 2^64.)
__device__ __forceinline__ uint64_t turns_per_position(double radians) {
  const double r = fabs(radians);
  const double hi = r * 0.15915494309189535;
  const double lo = fma(r, 0.15915494309189535, -hi) + r * -9.839338337591243e-18;
  const double t = hi - floor(hi);
  const uint64_t turns = (uint64_t)(t * 18446744073709551616.0) + (uint64_t)(int64_t)(lo * 18446744073709551616.0);
  return radians < 0.0 ? 0 - turns : turns;
}
__device__ __forceinline__ void sincos_turns(uint64_t phase, float* s, float* c) {
  // the top 32 bits, signed, as multiples of pi in [-1, 1); the rounding to
  // fp32 moves the angle by at most pi 2^-25
  sincospif((float)(int32_t)(uint32_t)(phase >> 32) * 4.656612873077392578125e-10f, s, c);
}

constexpr float kLeast = 0x1p-100f, kMost = 0x1p120f;   // mean squares between them are right in fp32

// Over the LPR lanes of each row, the same in all of them.
template <int LPR>
__device__ __forceinline__ float sum_of_squares(const float* v) {
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
#pragma unroll
  for (int m = LPR / 2; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
  return ss;
}

// Where a lane's 8 elements of a row lie: 4 pairs of the rotation, (4 l, 4 l + half)
// or 8 neighbours, or else 8 elements behind rot, so that none changes lanes.
template <bool INTERLEAVED>
struct Place {
  int sub, x0, x1;             // the lane within its row's; elements x0 .. + 3 and x1 .. + 3
  bool turn, in;
  __device__ __forceinline__ Place(const NormArgs& a, int lpr) {
    sub = threadIdx.x % lpr;
    turn = sub * 8 < a.rot;
    in = sub * 8 < a.D;
    x0 = !INTERLEAVED && turn ? sub * 4 : sub * 8;
    x1 = !INTERLEAVED && turn ? a.rot / 2 + sub * 4 : x0 + 4;
  }
};

template <typename T, bool I>
__device__ __forceinline__ void load_row(const NormArgs& a, const Place<I>& at, int t, int h, float* v) {
  const T* src = h < a.qh ? static_cast<const T*>(a.q) + t * a.q_ts + h * a.q_hs
                          : static_cast<const T*>(a.k) + t * a.k_ts + (h - a.qh) * a.k_hs;
  load4(src + at.x0, v);
  load4(src + at.x1, v + 4);
}

// v rs weight, rotated, to the output. sh: weights of q and k, cosines, sines; tok:
// the token within the block's.
template <typename T, bool I>
__device__ __forceinline__ void finish_row(const NormArgs& a, const Place<I>& at, const float* sh, int t, int tok, int h,
                                           const float* v, float rs) {
  const bool is_q = h < a.qh;
  const int half = a.rot / 2;
  const float* w = is_q ? sh : sh + a.D;
  const float* cs = sh + 2 * a.D;
  const float* sn = cs + a.tpb * half;
  const float4 w0 = *reinterpret_cast<const float4*>(w + at.x0), w1 = *reinterpret_cast<const float4*>(w + at.x1);
  float y[8] = {v[0] * rs * w0.x, v[1] * rs * w0.y, v[2] * rs * w0.z, v[3] * rs * w0.w,
                v[4] * rs * w1.x, v[5] * rs * w1.y, v[6] * rs * w1.z, v[7] * rs * w1.w};
  if (at.turn) {
    const float4 c = *reinterpret_cast<const float4*>(cs + tok * half + at.sub * 4);
    const float4 s = *reinterpret_cast<const float4*>(sn + tok * half + at.sub * 4);
    const float cc[4] = {c.x, c.y, c.z, c.w}, sc[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float& ya = y[I ? 2 * j : j];
      float& yb = y[I ? 2 * j + 1 : j + 4];
      const float p = ya * cc[j] - yb * sc[j];
      yb = yb * cc[j] + ya * sc[j];
      ya = p;
    }
  }
  T* dst = is_q ? static_cast<T*>(a.qo) + ((int64_t)t * a.qh + h) * a.D
                : static_cast<T*>(a.ko) + ((int64_t)t * a.kh + h - a.qh) * a.D;
  store4(dst + at.x0, y);
  store4(dst + at.x1, y + 4);
}

// A block takes `hpb` heads of `tpb` tokens. Their cosines and sines, which cost
// as much as the rest of several heads, are worked out once into shared memory,
// and so are the weights in fp32; then a group of LPR lanes takes a row at a
// time.
//
// 16384 tokens of 24 heads of 128, bf16: 52 us, 3.9 TB/s; bound by the
// instructions of a row (about 115 of a warp for 512 bytes in and out). Two rows
// in flight took 62 us (fewer warps fit), the sines of a lane's own heads in
// registers 88. The second pass and the test for it cost 1.2 us.
template <typename T, int LPR, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) k_norm_rope(const __grid_constant__ NormArgs a) {
  extern __shared__ float sh[];                     // weights [2][D], cosines [tpb][half], sines
  constexpr int GROUPS = THREADS / LPR;
  const int half = a.rot / 2;
  const int t0 = blockIdx.x * a.tpb, nt = min(a.tpb, a.tokens - t0);
  const int h0 = blockIdx.y * a.hpb, nh = min(a.hpb, a.qh + a.kh - h0);
  const Place<INTERLEAVED> at(a, LPR);
  const int nr = nt * nh;
  const uint32_t mul = nh > 1 ? 0xffffffffu / (uint32_t)nh + 1 : 0; // r / nh by the high half, exact for r < 2^16
  for (int x = threadIdx.x; x < 2 * a.D; x += THREADS) {
    const T* w = static_cast<const T*>(x < a.D ? a.wq : a.wk);
    sh[x] = (w ? to_f32(w[x < a.D ? x : x - a.D]) : 1.0f) + a.off;
  }
  float* cs = sh + 2 * a.D;
  for (int x = threadIdx.x; x < nt * half; x += THREADS) {
    const int t = x / half, p = x - t * half;
    sincos_turns((uint64_t)(int64_t)__ldg(a.pos + t0 + t) * turns_per_position(__ldg(a.freq + p)), &cs[a.tpb * half + x], &cs[x]);
  }
  __syncthreads();
  const float per = 1.0f / (float)a.D;
  uint32_t far = 0;                                 // a bit for each of the (at most eight) rounds
  for (int r0 = 0; r0 < nr; r0 += GROUPS) {         // every lane of the block runs every round
    const int r = r0 + threadIdx.x / LPR;
    const int tok = nh > 1 ? (int)__umulhi((uint32_t)r, mul) : r;
    const int h = h0 + r - tok * nh, t = t0 + tok;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const bool on = r < nr && at.in;
    if (on) load_row<T>(a, at, t, h, v);
    const float mean = fmaf(sum_of_squares<LPR>(v), per, a.eps);
    if (!on) continue;
    if (mean > kLeast && mean < kMost) finish_row<T>(a, at, sh, t, tok, h, v, rsqrtf(mean));   // (rsqrtf: 2 ulp)
    else far |= 1u << (r0 / GROUPS);
  }
  // Rows whose mean square (and eps) lies where squares or their sum may have left
  // fp32's range: again with the row times a power of two, which a small row keeps
  // and a large one gives back after its division. (A row with infinities or NaN, and
  // one of zeros without eps, come out as by the formula.)
  if (!__any_sync(0xffffffffu, far)) return;
#pragma unroll 1
  for (int r0 = 0; r0 < nr; r0 += GROUPS) {
    const bool on = far >> (r0 / GROUPS) & 1;
    const int r = r0 + threadIdx.x / LPR, tok = r / nh, h = h0 + r - tok * nh, t = t0 + tok;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (on) load_row<T>(a, at, t, h, v);
    const bool small = fmaf(sum_of_squares<LPR>(v), per, a.eps) <= kLeast;
    const float s = small ? 0x1p100f : 0x1p-70f;
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = v[j] * s;
    const float rs = rsqrtf(fmaf(sum_of_squares<LPR>(u), per, a.eps * s * s));
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = small ? u[j] : v[j] * rs * s;
    if (on) finish_row<T>(a, at, sh, t, tok, h, v, small ? rs : 1.f);
  }
}

// ---------------------------------------------------------------------------
// Cache write and read.
// ---------------------------------------------------------------------------
struct WriteArgs {
  KvView w;
  const void *k, *v;
  int64_t k_ts, k_hs, v_ts, v_hs;
};

// Exponent of a row whose largest finite magnitude is amax (0 for a row of
// zeros), held to a range in which 2^e, its inverse and every dequantised code
// are normal numbers of fp32 and of bf16.
__device__ __forceinline__ int kv_exponent(float amax) {
  return max(-100, min(119, e4m3_row_exponent(amax)));
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <typename T, int LPR, bool F8>
__device__ __forceinline__ void write_row(const T* src, void* pages, uint8_t* exps, int row, int D,
                                          int x0) {
  const bool on = row >= 0 && x0 < D;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (on) load8(src + x0, v);
  if constexpr (F8) {
    float amax = 0.f;                                // (fmaxf passes over NaN)
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
    if (amax == INFINITY) {                          // infinities do not scale the row, and become NaN
      amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (fabsf(v[j]) == INFINITY) v[j] = NAN;
        else amax = fmaxf(amax, fabsf(v[j]));
      }
    }
#pragma unroll
    for (int m = LPR / 2; m; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    const int e = kv_exponent(amax);
    const float s = pow2(-e);
    uint32_t c[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      c[j] = f32x2_to_e4m3(v[4 * j] * s, v[4 * j + 1] * s) | ((uint32_t)f32x2_to_e4m3(v[4 * j + 2] * s, v[4 * j + 3] * s) << 16);
    if (on) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pages) + (int64_t)row * D + x0) = make_uint2(c[0], c[1]);
      if (x0 == 0) exps[row] = (uint8_t)(e + 127);
    }
  } else {
    if (on) store8(static_cast<__nv_bfloat16*>(pages) + (int64_t)row * D + x0, v);
  }
}

// A group of LPR lanes per (token, head): its key row and its value row. 22576
// tokens of 4 heads of 256, fp32 to e4m3: 42 us, 5.5 TB/s (called one by one 46);
// bf16 to bf16 37 us, 5.0 TB/s.
template <typename T, int LPR, bool F8>
__global__ void __launch_bounds__(THREADS) k_cache_write(const __grid_constant__ WriteArgs a) {
  const KvView& w = a.w;
  const int64_t unit = ((int64_t)blockIdx.x * THREADS + threadIdx.x) / LPR;
  const int token = (int)(unit / w.c.kv_heads), head = (int)(unit % w.c.kv_heads);
  const int x0 = (threadIdx.x % LPR) * 8;
  int row = -1;
  if (unit < (int64_t)w.b.tokens * w.c.kv_heads) {
    const int b = kv_sequence(w, token);
    if (b >= 0)
      row = kv_row(w, w.b.page_table + (int64_t)b * w.b.table_stride,
                   (int64_t)__ldg(w.b.past + b) + (token - __ldg(w.b.first + b)), head);
  }
  write_row<T, LPR, F8>(static_cast<const T*>(a.k) + token * a.k_ts + head * a.k_hs, w.c.k, w.c.k_exp,
                        row, w.c.head_dim, x0);
  write_row<T, LPR, F8>(static_cast<const T*>(a.v) + token * a.v_ts + head * a.v_hs, w.c.v, w.c.v_exp,
                        row, w.c.head_dim, x0);
}

struct ReadArgs {
  KvView w;
  void *k, *v;
};

template <typename T, bool F8>
__device__ __forceinline__ void read_row(const void* pages, const uint8_t* exps, int row, int D, int x0,
                                         T* dst) {
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (row >= 0) {
    if constexpr (F8) {
      const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pages) + (int64_t)row * D + x0);
      // any byte is a power of two that fp32 holds, also in rows never written
      const float s = pow2(max(-126, min(127, (int)exps[row] - 127)));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((j < 2 ? c.x : c.y) >> (16 * (j & 1))), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[2 * j] = f.x * s;
        v[2 * j + 1] = f.y * s;
      }
    } else {
      load8(static_cast<const __nv_bfloat16*>(pages) + (int64_t)row * D + x0, v);
    }
  }
  store8(dst + x0, v);
}

// A group of LPR lanes per head and TOK neighbouring tokens, whose rows lie
// together in their page: one search for the sequence, and 2 TOK rows in flight.
// 103000 tokens of 8 heads of 128, e4m3 to bf16: 133 us, 4.8 TB/s (1 token to a
// group: 142; 8: 173), to fp32 177 us, 6.0 TB/s (187; 218); from a bf16 cache 156
// us, 5.4 TB/s (150; 172).
template <typename T, int LPR, bool F8, int TOK>
__global__ void __launch_bounds__(THREADS) k_cache_read(const __grid_constant__ ReadArgs a) {
  const KvView& w = a.w;
  const int64_t unit = ((int64_t)blockIdx.x * THREADS + threadIdx.x) / LPR;
  const int head = (int)(unit % w.c.kv_heads), x0 = (threadIdx.x % LPR) * 8;
  const int64_t t0 = unit / w.c.kv_heads * TOK;
  if (t0 >= w.b.tokens || x0 >= w.c.head_dim) return;
  int b = -1, row[TOK], end = 0;
  int64_t shift = 0;                               // position less token
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    const int token = (int)t0 + i;
    row[i] = -2;
    if (t0 + i >= w.b.tokens) continue;
    if (i == 0 || token >= end) {
      b = kv_sequence(w, token);
      if (b >= 0) {
        end = __ldg(w.b.first + b + 1);
        shift = (int64_t)__ldg(w.b.past + b) - __ldg(w.b.first + b);
      }
    }
    if (b >= 0) row[i] = kv_row(w, w.b.page_table + (int64_t)b * w.b.table_stride, token + shift, head);
  }
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    if (row[i] == -2) continue;                    // padding
    const int64_t o = ((t0 + i) * w.c.kv_heads + head) * w.c.head_dim;
    read_row<T, F8>(w.c.k, w.c.k_exp, row[i], w.c.head_dim, x0, static_cast<T*>(a.k) + o);
    read_row<T, F8>(w.c.v, w.c.v_exp, row[i], w.c.head_dim, x0, static_cast<T*>(a.v) + o);
  }
}

// ---------------------------------------------------------------------------
// Launches. The functors pick the template by type, lanes per row and format.
// ---------------------------------------------------------------------------
template <typename F> cudaError_t by_lanes(int D, F f) {
  if (D <= 64) return f(std::integral_constant<int, 8>());
  if (D <= 128) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}
template <typename F> cudaError_t by_type(int dtype, F f) {
  return dtype == DG_BF16 ? f(__nv_bfloat16()) : f(float());
}

// Blocks for n groups of lpr lanes; 0 if the grid would not fit.
unsigned blocks(int64_t n, int lpr) {
  const int64_t b = (n * lpr + THREADS - 1) / THREADS;
  return b > 0x7fffffff ? 0u : (unsigned)b;
}

}  // namespace rows

namespace {
int fail(int code, const char* msg) {
  set_last_error(msg);
  return code;
}
bool off16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }
}  // namespace

// Host checks of a cache and a batch, for the cache and attention calls; a
// message in dg_last_error(NULL) and a code, or DG_OK.
int kv_check(const dg_kv_cache* c, const dg_kv_batch* b) {
  if (!c || !b) return fail(DG_EINVAL, "NULL cache or batch");
  if (c->format != DG_KV_BF16 && c->format != DG_KV_E4M3) return fail(DG_EINVAL, "format must be DG_KV_BF16 or DG_KV_E4M3");
  if (c->pages < 0 || c->page_size < 1 || c->kv_heads < 1) return fail(DG_EINVAL, "need pages >= 0, page_size >= 1, kv_heads >= 1");
  if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16)
    return fail(DG_EUNSUPPORTED, "head_dim must be a multiple of 16, 16..256");
  // page_size and kv_heads < 2^31: their product and then the whole fit 64 and 96 bits
  const int64_t per_page = (int64_t)c->page_size * c->kv_heads;
  if (per_page >= (1ll << 31) || (c->pages && per_page > ((1ll << 31) - 1) / c->pages))
    return fail(DG_EUNSUPPORTED, "the cache must have fewer than 2^31 rows (pages x kv_heads x page_size)");
  if (b->batch < 0 || b->tokens < 0 || b->table_stride < 0) return fail(DG_EINVAL, "batch, tokens and table_stride must be >= 0");
  if (b->batch > kMaxBatch) return fail(DG_EUNSUPPORTED, "batch must be at most 1024");
  if ((int64_t)b->table_stride * c->page_size >= (1ll << 31))
    return fail(DG_EUNSUPPORTED, "table_stride x page_size must be below 2^31");
  if (b->batch == 0 || b->tokens == 0) return DG_OK;
  if (!c->status || !b->first || !b->past) return fail(DG_EINVAL, "NULL status, first or past");
  if (b->table_stride && !b->page_table) return fail(DG_EINVAL, "NULL page_table");
  if (c->pages) {
    if (!c->k || !c->v) return fail(DG_EINVAL, "NULL cache pages");
    if (c->format == DG_KV_E4M3 && (!c->k_exp || !c->v_exp)) return fail(DG_EINVAL, "an e4m3 cache needs k_exp and v_exp");
    if (off16(c->k) || off16(c->v)) return fail(DG_EINVAL, "cache pages must be 16-byte aligned");
  }
  return DG_OK;
}

int kv_row_args(const void* p, int64_t ts, int64_t hs) {
  if (!p) return fail(DG_EINVAL, "NULL input");
  if (off16(p) || ts % 8 || hs % 8) return fail(DG_EINVAL, "inputs must be 16-byte aligned, strides multiples of 8 elements");
  return DG_OK;
}

int kv_launched(cudaError_t e) {
  if (e == cudaSuccess) return DG_OK;
  return fail(DG_ECUDA, cudaGetErrorString(e));
}

}  // namespace dg

using namespace dg;

extern "C" int dg_qk_norm_rope(int32_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim,
                               int32_t rot_dim, int32_t interleaved, int32_t dtype, const void* q,
                               int64_t q_ts, int64_t q_hs, const void* k, int64_t k_ts, int64_t k_hs,
                               const void* q_weight, const void* k_weight, float weight_offset,
                               float eps, const int32_t* positions, const double* inv_freq,
                               void* q_out, void* k_out, void* stream) {
  using namespace rows;
  if (tokens < 0 || q_heads < 0 || k_heads < 0) return fail(DG_EINVAL, "tokens and heads must be >= 0");
  if (head_dim < 8 || head_dim > 256 || head_dim % 8) return fail(DG_EUNSUPPORTED, "head_dim must be a multiple of 8, 8..256");
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16) return fail(DG_EUNSUPPORTED, "rot_dim must be a multiple of 16, 0..head_dim");
  if (dtype != DG_F32 && dtype != DG_BF16) return fail(DG_EINVAL, "dtype must be DG_F32 or DG_BF16");
  if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(weight_offset)) return fail(DG_EINVAL, "need eps >= 0 and a finite weight_offset");
  const int64_t heads = (int64_t)q_heads + k_heads;
  if (tokens == 0 || heads == 0) return DG_OK;
  if (heads > (1 << 20)) return fail(DG_EUNSUPPORTED, "too many heads");
  int rc;
  if (q_heads && (rc = kv_row_args(q, q_ts, q_hs))) return rc;
  if (k_heads && (rc = kv_row_args(k, k_ts, k_hs))) return rc;
  if ((q_heads && (!q_out || off16(q_out))) || (k_heads && (!k_out || off16(k_out))))
    return fail(DG_EINVAL, "outputs must be 16-byte aligned and not NULL");
  if (off16(q_weight) || off16(k_weight)) return fail(DG_EINVAL, "weights must be 16-byte aligned");
  if (rot_dim && (!positions || !inv_freq)) return fail(DG_EINVAL, "a rotation needs positions and inv_freq");
  NormArgs a{q, k, q_weight, k_weight, q_out, k_out, q_ts, q_hs, k_ts, k_hs, positions, inv_freq,
             tokens, q_heads, k_heads, head_dim, rot_dim, 1, 1, weight_offset, eps};
  const cudaError_t e = by_lanes(head_dim, [&](auto lpr) {
    constexpr int L = decltype(lpr)::value;
    // A block has about eight rounds of rows, so that the sines are shared by many
    // rows (four: 55.7 us for 52.1 on the prompt above); with few tokens one or two,
    // to fill the SMs.
    const int64_t round = THREADS / L, rows = (int64_t)tokens * heads;
    const int64_t want = rows >= 148 * 8 * round ? 8 * round : 2 * round;
    a.hpb = (int)std::min<int64_t>(heads, want);
    a.tpb = (int)std::min<int64_t>(std::max<int64_t>(1, want / heads), tokens);
    a.tpb = std::min(a.tpb, 32);
    const dim3 grid((unsigned)(((int64_t)tokens + a.tpb - 1) / a.tpb), (unsigned)((heads + a.hpb - 1) / a.hpb));
    const size_t smem = sizeof(float) * (2 * head_dim + a.tpb * rot_dim);   // at most 34 KB
    return by_type(dtype, [&](auto t) {
      using T = decltype(t);
      if (interleaved) k_norm_rope<T, L, true><<<grid, THREADS, smem, (cudaStream_t)stream>>>(a);
      else k_norm_rope<T, L, false><<<grid, THREADS, smem, (cudaStream_t)stream>>>(a);
      return cudaGetLastError();
    });
  });
  return kv_launched(e);
}

extern "C" int dg_cache_write(const dg_kv_cache* cache, const dg_kv_batch* batch, int32_t dtype,
                              const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts,
                              int64_t v_hs, void* stream) {
  using namespace rows;
  int rc = kv_check(cache, batch);
  if (rc) return rc;
  if (dtype != DG_F32 && dtype != DG_BF16) return fail(DG_EINVAL, "dtype must be DG_F32 or DG_BF16");
  if (batch->tokens == 0 || batch->batch == 0) return DG_OK;
  if ((rc = kv_row_args(k, k_ts, k_hs)) || (rc = kv_row_args(v, v_ts, v_hs))) return rc;
  const WriteArgs a{{*cache, *batch}, k, v, k_ts, k_hs, v_ts, v_hs};
  const int64_t n = (int64_t)batch->tokens * cache->kv_heads;
  return kv_launched(by_lanes(cache->head_dim, [&](auto lpr) {
    constexpr int L = decltype(lpr)::value;
    const unsigned grid = blocks(n, L);
    if (!grid) return cudaErrorInvalidConfiguration;
    return by_type(dtype, [&](auto t) {
      using T = decltype(t);
      if (cache->format == DG_KV_E4M3) k_cache_write<T, L, true><<<grid, THREADS, 0, (cudaStream_t)stream>>>(a);
      else k_cache_write<T, L, false><<<grid, THREADS, 0, (cudaStream_t)stream>>>(a);
      return cudaGetLastError();
    });
  }));
}

extern "C" int dg_cache_read(const dg_kv_cache* cache, const dg_kv_batch* batch, int32_t dtype,
                             void* k_out, void* v_out, void* stream) {
  using namespace rows;
  int rc = kv_check(cache, batch);
  if (rc) return rc;
  if (dtype != DG_F32 && dtype != DG_BF16) return fail(DG_EINVAL, "dtype must be DG_F32 or DG_BF16");
  if (batch->tokens == 0 || batch->batch == 0) return DG_OK;
  if (!k_out || !v_out || off16(k_out) || off16(v_out)) return fail(DG_EINVAL, "outputs must be 16-byte aligned and not NULL");
  const ReadArgs a{{*cache, *batch}, k_out, v_out};
  const int64_t n = (int64_t)batch->tokens * cache->kv_heads;
  return kv_launched(by_lanes(cache->head_dim, [&](auto lpr) {
    constexpr int L = decltype(lpr)::value;
    const unsigned grid = blocks(n, L);
    if (!grid) return cudaErrorInvalidConfiguration;
    // four tokens to a group once that still fills every SM
    const bool many = n * L >= 4 * 148 * 2048;
    const unsigned grid4 = blocks(((int64_t)batch->tokens + 3) / 4 * cache->kv_heads, L);
    return by_type(dtype, [&](auto t) {
      using T = decltype(t);
      cudaStream_t s = (cudaStream_t)stream;
      if (cache->format == DG_KV_E4M3) {
        if (many) k_cache_read<T, L, true, 4><<<grid4, THREADS, 0, s>>>(a);
        else k_cache_read<T, L, true, 1><<<grid, THREADS, 0, s>>>(a);
      } else {
        if (many) k_cache_read<T, L, false, 4><<<grid4, THREADS, 0, s>>>(a);
        else k_cache_read<T, L, false, 1><<<grid, THREADS, 0, s>>>(a);
      }
      return cudaGetLastError();
    });
  }));
}

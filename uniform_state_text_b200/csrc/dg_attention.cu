// Attention of a block of new tokens over a paged key/value cache
// (dg_cache_attention).
//
// For one query row, over the keys j it sees, with t_j = scale log2(e) q.k_j:
//   m = max t_j,  l = sum 2^(t_j - m),  out = sum 2^(t_j - m) v_j / l,
//   lse = (m + log2 l) ln 2
// in one pass over the keys: a larger maximum rescales l and the running sum. (m
// is kept before the scale, where it is one of the logits to the bit, so that
// differences from it stay differences however large the logits are.)
//
// Rows. The query heads of one key/value head and the tokens of one sequence
// are packed into one matrix, row r = token r / G, head r % G (G query heads
// per key/value head), so that every key and value row is read once per
// matrix and not once per query head. A tile has 128 such rows (the MMA's M,
// one TMEM lane each); an item is NT tiles of one sequence and head.
//
// Work split. An item's keys come in tiles of BN. All items' key tiles, in
// order (sequence, head, item), form one list, with kItem empty places before
// each item that stand for its queries, first products and result; CTA c of a
// persistent grid takes a contiguous share of it: whatever the batch's lengths,
// every SM has the same work and there is one wave. A share may begin or end
// inside an item; such pieces go to scratch with their m and l, and a second
// launch joins them in the order of the list. Lengths are read on the device,
// so a captured graph follows them.
//
// A CTA's warps:
//   softmax   NT x 4 warps: TMEM lane = row; S from TMEM, P = 2^(t - m) back
//             to TMEM as bf16, the running m and l in registers
//   loads     bf16: one warp per slot of the ring of key and value tiles; runs
//             of rows that lie together in a page come by TMA, single rows by
//             16-byte cp.async, into the 128-byte swizzle that the MMA reads.
//             e4m3: two warps bring the codes ahead of their use, others convert
//             them to bf16, which holds code x 2^e exactly. The item's query
//             rows come by TMA where a head's group is a power of two
//   MMA       one warp, one elected lane issuing: S = Q K^T (both from shared
//             memory), O += P V (P from TMEM, V as it lies, keys along K),
//             accumulators in TMEM
// With NT = 2 the two tiles share each key and value tile and alternate, so
// that one tile's softmax runs under the other's products; with NT = 1 there
// are two S buffers and S of the next keys is issued before P V of these. (With
// two buffers for each of two tiles, TMEM has room for 64 keys to a tile only:
// the prompt below, when it took 347 us, then took 456, a tile's hand-overs
// costing as much as with 128.)
//
// O is rescaled only when a row's maximum has grown by more than 2^8 over the
// one in use (P then stays below 2^8, harmless in bf16 and fp32): the wait for
// the previous P V and the pass over O are rare. Without that the prompt takes
// 359 us for 327, the canvases 144 for 136.
//
// Rounding: keys, values and queries enter the products as they are; P is
// rounded to bf16, the tensor cores' operand type with V's range (2^-8 relative
// at most, independent from key to key); S, m, l and O stay in fp32; the output
// is rounded once.
//
// Measured on B200 (replays of a captured graph, two sets of inputs in turn;
// called one by one with inputs of their own each, the long sequence takes 106 us
// and the prompt up to 338, the others as here):
//   one token, 131072 bf16 keys, 8 x 2 heads of 128: 95 us, 5.6 TB/s of the 6.55
//     that a copy reaches; bound by memory
//   33 tokens, 2000 to 8000 e4m3 keys each, 8 x 4 heads of 128: 124 us, 2.3
//     TB/s; bound by hand-overs between the warps, tile by tile
//   4 canvases of 256, 8448 e4m3 keys, 4 x 2 heads of 256: 137 us, 518 TFLOP/s;
//     8 x 2 heads of 128: 117 us, over bf16 keys 95 (605 and 743 TFLOP/s)
//   a prompt of 8192, 8 x 2 heads of 128: 327 us, 842 TFLOP/s (e4m3 keys 373);
//     bound by the chain softmax - P V - S of each tile: S is read from TMEM
//     twice, a row's 128 logits not fitting the registers of a softmax thread,
//     and the tensor cores are busy half the time
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "dg.h"
#include "dg_cache.cuh"
#include "dg_fp8.cuh"
#include "dg_tc.h"
#include "dg_tcgen05.cuh"

namespace dg {
void set_last_error(const char* msg);
int kv_check(const dg_kv_cache* c, const dg_kv_batch* b);
int kv_row_args(const void* p, int64_t ts, int64_t hs);
int kv_launched(cudaError_t e);

namespace attn {

using namespace tc;

constexpr int kMaxCtas = 148;                 // scratch is laid out for at most this many
constexpr int TMEM_COLS = 512;
// An item's cost beside its key tiles, in key tiles. (With 0 the prompt takes 351 us
// for 322 and the single tokens 130 for 123, with 6 324 and 128; a single canvas,
// where shares are of a tile or two, 22.5 for 23.6 with 0.)
constexpr int kItem = 3;
constexpr float kGrow = 8.0f;                 // log2 growth of a maximum that rescales O
constexpr float kLarge = 16777216.0f;         // scaled logits of this size have steps of one and more
constexpr unsigned long long kWaitNs = 2000000000ull;   // a wait's limit by default
constexpr float kLn2 = 0.6931471805599453f;

struct Args {
  KvView w;
  const __nv_bfloat16* q;
  int64_t q_ts, q_hs;
  int q_heads, G;              // G query heads per key/value head
  // r / G and position / page_size as products, exact below 2^31 (a division for
  // every tile and row had cost more than the tile's copies)
  uint32_t g_mul, ps_mul;
  int g_shift, ps_shift;
  float scale_log2;            // scale log2(e)
  int mask;
  const uint32_t* tree;
  int words;
  __nv_bfloat16* out;
  float* lse;
  // scratch
  float* part_o;               // [CTAs][2][rows][DP] unnormalised sums
  float2* part_ml;             // [CTAs][2][rows] their m (unscaled) and l
  struct Open* open;           // [CTAs] the item a CTA begins and does not finish
  int rows;                    // rows kept per piece
  int box;                     // rows per TMA copy: a power of two that divides page_size; 0: no TMA
  int q_box;                   // queries by TMA, 32 rows (32 / G tokens of G heads) at a time
  // failure-path testing
  unsigned long long wait_ns;  // the limit of every wait
  uint32_t stall;              // > 0: the softmax does not announce each CTA's key tile of this number, from 1

  __device__ __forceinline__ uint32_t over_g(uint32_t r) const {
    return (uint32_t)(((uint64_t)r * g_mul) >> g_shift);
  }
  __device__ __forceinline__ uint32_t over_page(uint32_t pos) const {
    return (uint32_t)(((uint64_t)pos * ps_mul) >> ps_shift);
  }
};

// The item that a CTA's share ends inside, if it also begins there: rows (0:
// none), the CTAs it lies in, the sequence's first token, head and item index.
struct Open {
  int rows, pieces, t0, h, m;
};

template <int DP_, int NT_, bool F8_>
struct Shape {
  static constexpr bool F8 = F8_;                      // e4m3 cache
  static constexpr int DP = DP_;                       // head_dim padded to 64, 128 or 256
  static constexpr int NT = NT_;
  static constexpr int BN = DP == 256 ? 64 : 128;      // keys per tile
  static constexpr int SLOT = BN * DP * 2;
  static constexpr int QTILE = 128 * DP * 2;
  static constexpr int SL = F8 ? (DP == 64 ? 6 : 4) : DP == 256 ? 4 : DP == 128 ? 5 : (NT == 2 ? 6 : 8);   // ring slots
  // Load warps. bf16: one per slot. e4m3: CW that convert, several to a tile, so
  // that a slot is not held longer than its share of the time, and two that
  // bring the codes AHEAD tiles before. Eight warps pay where rows are of 256
  // codes only (the canvases 136 us, with 4 146). Up to 128 they cost registers:
  // with 4 and 8 the single tokens take 123 and 125 us, canvases of heads of 128
  // 116 and 125, of 64 87 and 94, an e4m3 prompt 366 and 415. AHEAD is what
  // shared memory leaves: 2 instead of 4 costs the single tokens 165 us for 123.
  static constexpr int CW = F8 ? (DP == 256 ? 8 : 4) : 0;
  static constexpr int TEAM = F8 ? CW / 2 : 1;         // half convert keys, half values
  static constexpr int N_LOAD = F8 ? CW : SL;
  static constexpr int AHEAD = F8 ? (DP == 64 || (DP == 128 && NT == 1) ? 4 : 2) : 0;
  static_assert(AHEAD % 2 == 0, "keys and values have buffers of their own: each is then used by one fetching warp and one team, in order");
  static constexpr int RAW = BN * DP;                  // bytes of a tile's codes
  static constexpr int W_LOAD = NT * 4, W_FETCH = W_LOAD + N_LOAD, W_MMA = W_FETCH + (F8 ? 2 : 0);
  static constexpr int THREADS = (W_MMA + 1) * 32;
  // TMEM: two S buffers, tile x's (NT = 2) or key tile k's (NT = 1, k mod 2); then O
  static constexpr int T_O = 2 * BN;
  static constexpr size_t SMEM = 1024 + (size_t)NT * QTILE + (size_t)SL * SLOT + (size_t)AHEAD * RAW + 1024;
  static_assert(8 * (kMaxBatch + 1) <= SL * SLOT, "the plan's sums lie in the ring before it is used");
  static_assert(T_O + NT * DP <= TMEM_COLS, "TMEM");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// ---------------------------------------------------------------------------
// The list of key tiles.
// ---------------------------------------------------------------------------
template <int ROWS, int BN>
struct Walk {
  const Args& a;
  int b, h, m;                 // sequence, key/value head, item of the pair
  int n, past, t0;             // the sequence's new tokens, cached positions, first row
  int tb, te, T;               // this segment's key tiles [tb, te) of the item's T
  int64_t at, lo, hi;          // the item's first place in the list; the CTA's share

  __device__ __forceinline__ Walk(const Args& a_) : a(a_) {}
  __device__ __forceinline__ void sequence(int b_) {
    b = b_;
    n = kv_new(a.w, b, &t0);
    past = kv_past(a.w, b, n);
  }
  // (Rows and positions are below 2^31, so that 32-bit arithmetic serves: a
  // 64-bit division here and in the query loads had cost more than the tiles.)
  __device__ __forceinline__ int items() const { return (int)(((uint32_t)n * (uint32_t)a.G + ROWS - 1) / ROWS); }
  // Key tiles of item x: up to its last row's token under a causal mask, else all; at least one.
  __device__ __forceinline__ int tiles(int x) const {
    uint32_t e = (uint32_t)n;
    if (a.mask == DG_MASK_CAUSAL) e = min(e, a.over_g((uint32_t)(x + 1) * ROWS + (uint32_t)a.G - 1));
    return (int)max(1u, ((uint32_t)past + e + BN - 1) / BN);
  }
  __device__ __forceinline__ int64_t keys() const { return (int64_t)past + n; }
  // First position that some row of the item may not see.
  __device__ __forceinline__ int64_t clear() const {
    return a.mask == DG_MASK_FULL ? keys() : a.mask == DG_MASK_TREE ? past : (int64_t)past + a.over_g((uint32_t)m * ROWS) + 1;
  }
  // (A share that ends within an item's empty places leaves the item alone.)
  __device__ __forceinline__ bool more() const { return te > tb; }
  __device__ __forceinline__ void segment() {
    T = tiles(m);
    const int64_t first = at + kItem;
    tb = lo > first ? (int)(lo - first) : 0;
    te = hi - first < T ? (int)(hi - first) : T;
  }
  __device__ __forceinline__ void next() {
    at += kItem + T;
    te = tb;
    if (at >= hi) return;
    if (++m == items()) {
      m = 0;
      if (++h == a.w.c.kv_heads) {
        h = 0;
        do { sequence(b + 1); } while (n == 0);       // the list ends before the batch does
      }
    }
    segment();
  }
  __device__ __forceinline__ int rows() const {
    return min(n * a.G - m * ROWS, ROWS);
  }
};

// Where a CTA's share begins; worked out once per CTA.
struct Start {
  int64_t lo, hi, share, at;
  int b, h, m;
};

// The whole CTA: tiles per head of every sequence, their prefix sums (in
// shared memory, pref[batch + 1]), and this CTA's share. The sums lie where the
// first tiles are copied to by TMA: every thread fences its ordinary accesses to
// them before the last barrier, since a barrier alone does not order those
// before accesses of the asynchronous proxy.
template <int ROWS, int BN>
__device__ __forceinline__ void plan(const Args& a, int64_t* pref, Start* st) {
  const int B = a.w.b.batch;
  Walk<ROWS, BN> w(a);
  constexpr int kAlone = 16;                          // items that one thread adds up by itself
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    w.sequence(b);
    const int it = w.items();
    int64_t u = 0;
    if (a.mask != DG_MASK_CAUSAL) u = it ? (int64_t)it * (w.tiles(0) + kItem) : 0;
    else if (it > kAlone) u = -1;
    else for (int x = 0; x < it; ++x) u += w.tiles(x) + kItem;
    pref[b + 1] = u;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int b = warp; b < B; b += blockDim.x >> 5) {
    if (pref[b + 1] >= 0) continue;
    w.sequence(b);
    int64_t u = 0;
    for (int x = lane, it = w.items(); x < it; x += 32) u += w.tiles(x) + kItem;
#pragma unroll
    for (int d = 16; d; d >>= 1) u += __shfl_xor_sync(0xffffffffu, u, d);
    __syncwarp();
    if (lane == 0) pref[b + 1] = u;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t run = 0;
    if (lane == 0) pref[0] = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      int64_t u = b0 + lane < B ? pref[b0 + lane + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, u, d);
        if (lane >= d) u += o;
      }
      if (b0 + lane < B) pref[b0 + lane + 1] = run + u;
      run += __shfl_sync(0xffffffffu, u, 31);
    }
    __syncwarp();
    if (lane == 0) {
      const int H = a.w.c.kv_heads;
      const int64_t total = run * H;
      const int64_t share = (total + gridDim.x - 1) / gridDim.x;
      st->share = share;
      st->lo = min(total, share * (int64_t)blockIdx.x);
      st->hi = min(total, st->lo + share);
      if (st->lo < st->hi) {
        int l = 0, r = B;                             // H pref[l] <= lo < H pref[r]
        while (r - l > 1) {
          const int mid = (l + r) >> 1;
          if (pref[mid] * H <= st->lo) l = mid;
          else r = mid;
        }
        w.sequence(l);
        const int64_t per = pref[l + 1] - pref[l];
        int64_t rest = st->lo - pref[l] * H;
        st->b = l;
        st->h = (int)(rest / per);
        rest -= st->h * per;
        int x = 0;
        if (a.mask != DG_MASK_CAUSAL) {
          x = (int)(rest / (w.tiles(0) + kItem));
          rest -= (int64_t)x * (w.tiles(0) + kItem);
        } else {
          for (int t; rest >= (t = w.tiles(x) + kItem); ++x) rest -= t;
        }
        st->m = x;
        st->at = st->lo - rest;
      }
    }
  }
  fence_proxy_async_shared();
  __syncthreads();
}

template <int ROWS, int BN>
__device__ __forceinline__ void begin(Walk<ROWS, BN>& w, const Start& st) {
  w.lo = st.lo;
  w.hi = st.hi;
  w.tb = w.te = 0;
  if (st.lo >= st.hi) return;
  w.sequence(st.b);
  w.h = st.h;
  w.m = st.m;
  w.at = st.at;
  w.segment();
}

// ---------------------------------------------------------------------------
// Small pieces.
// ---------------------------------------------------------------------------
struct Sync {
  // Barriers of a key tile k lie at k mod 4, with phase k / 4: whoever waits may
  // then be up to four tiles behind (a parity wait on a barrier that has gone on
  // by two phases, or not yet reached the one before, answers for another phase).
  uint64_t full[8];                // ring slots
  uint64_t s_full[8], p_full[8];   // 4 x + k mod 4: S ready (the keys' slot is free after the last x), P stored
  uint64_t o_done[8], o_free[2];   // P V done (the values' slot is free after the last x); O read
  uint64_t q_full, q_free, fin;
  uint64_t raw[8], taken[4];       // e4m3: a tile's codes have landed, and have been converted (bf16: a value
                                   // tile to be cleaned has landed)
  uint8_t exps[4][128];            // their rows' exponents
  uint64_t busy;                   // when the search for infinities last said that it goes on
  uint32_t tmem;
  int abort, nonfinite;
  Start start;
};

// A CTA's shared memory, aligned: query tiles, ring, codes; then its Sync.
__device__ __forceinline__ unsigned char* tiles() {
  extern __shared__ unsigned char smem_raw[];
  return reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
}
template <class S>
__device__ __forceinline__ Sync& sync_of() {
  return *reinterpret_cast<Sync*>(tiles() + S::NT * S::QTILE + S::SL * S::SLOT + S::AHEAD * S::RAW);
}

// Bounded wait on an mbarrier phase; gives up on the CTA's abort flag or after
// limit_ns in which nothing was said to go on (then raises DG_ETIMEOUT).
// check_abort = false: time limit only.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, Sync& sy, int* status,
                                       unsigned long long limit_ns, bool check_abort) {
  const uint64_t t0 = gtimer();
  for (uint32_t k = 1;; ++k) {
    if (mbar_try(bar, parity)) return true;
    if ((k & 63) == 0) {
      if (check_abort && *(volatile int*)&sy.abort) return false;
      const uint64_t since = max(t0, *(volatile uint64_t*)&sy.busy);   // (may be later than this thread's clock)
      if ((int64_t)(gtimer() - since) > (int64_t)limit_ns) {
        *(volatile int*)&sy.abort = 1;
        raise_status(status, DG_ETIMEOUT);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Sync& sy, const Args& a,
                                     bool check_abort = true) {
  return mbar_try(bar, parity) || wait_slow(bar, parity, sy, a.w.c.status, a.wait_ns, check_abort);
}

// A whole warp waits, every lane for itself: with one lane waiting and the others
// held until it had, each hand-over took several times as long (the whole kernel
// up to twice), so no role waits in a divergent warp.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Sync& sy, const Args& a) {
  return __all_sync(0xffffffffu, wait(bar, parity, sy, a)) != 0;
}

// A value that is the same in every lane, made visibly so.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// D (TMEM) += A (TMEM, bf16) B (shared memory).
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 16 columns of TMEM to each lane, in two halves: the issue (its registers are
// not to be read yet), and the wait, which names them so that no read moves above it.
__device__ __forceinline__ void tmem_ld16_issue(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
// 8 registers of each lane to 8 columns of TMEM.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 16 registers of each lane to 16 columns of TMEM.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 16 bytes into shared memory, or zeros where `bytes` is 0.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_landed() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void st_shared(uint32_t dst, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(src) : "memory");
  return v;
}
// Pairs of floats in one register pair, and the instructions that work on both.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float lo2(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {   // NaN if one of them is
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint64_t exp2_mufu2(uint64_t x) { return pack2(ex2(lo2(x)), ex2(hi2(x))); }
// 2^x without the special-function unit, of which an SM has 16 lanes to 128 for
// arithmetic: x = n + f with n the nearest whole number (by adding 1.5 2^23),
// 2^f on [-1/2, 1/2] by the polynomial of degree 5 through 2^f at the Chebyshev
// points (relative error 2.1e-7 in fp32), n added to the exponent. For x up to
// 127, not NaN; below -126.5 the result is a denormal number, and below -127, minus
// infinity included, 2^-149, which is zero in bf16.
__device__ __forceinline__ uint64_t exp2_poly2(uint64_t x) {
  constexpr float kMagic = 12582912.0f;
  x = pack2(fmaxf(lo2(x), -127.0f), fmaxf(hi2(x), -127.0f));
  const uint64_t r = add2(x, pack2(kMagic, kMagic));
  const uint64_t f = fma2(add2(r, pack2(-kMagic, -kMagic)), pack2(-1.f, -1.f), x);
  uint64_t p = pack2(0.00133908633f, 0.00133908633f);
  p = fma2(p, f, pack2(0.00967603177f, 0.00967603177f));
  p = fma2(p, f, pack2(0.0555035695f, 0.0555035695f));
  p = fma2(p, f, pack2(0.240221068f, 0.240221068f));
  p = fma2(p, f, pack2(0.693147182f, 0.693147182f));
  p = fma2(p, f, pack2(1.00000012f, 1.00000012f));
  return pack2(__uint_as_float((uint32_t)p + ((uint32_t)r << 23)),
               __uint_as_float((uint32_t)(p >> 32) + ((uint32_t)(r >> 32) << 23)));
}
// Byte offset of 16-byte chunk c (8 bf16 columns) of row r in an operand tile of
// `rows` rows: blocks of 64 columns, 128-byte rows, the chunk index xored with r % 8.
__device__ __forceinline__ uint32_t swizzled(int r, int c, int rows) {
  return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// The lowest k bits (none for k <= 0, all for k >= 32).
__device__ __forceinline__ uint32_t low_bits(int64_t k) {
  return k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << (int)k) - 1u;
}
// 32 bits of a bit row from bit `at` on (may be negative); words beyond the row are zero.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* row, int words, int64_t at) {
  if (at <= -32 || at >= (int64_t)words * 32) return 0;
  const int64_t x = at >= 0 ? at >> 5 : -1;
  const uint32_t lo = x >= 0 ? __ldg(row + x) : 0u;
  const uint32_t hi = x + 1 < words ? __ldg(row + x + 1) : 0u;
  return __funnelshift_r(lo, hi, (uint32_t)(at & 31));
}
// Which of 32 positions from `at` on token i of the sequence sees.
template <typename W>
__device__ __forceinline__ uint32_t seen(const W& w, const uint32_t* tree, int i, int64_t at) {
  if (w.a.mask == DG_MASK_CAUSAL) return low_bits((int64_t)w.past + i + 1 - at);
  const uint32_t in = low_bits(w.keys() - at);
  if (w.a.mask == DG_MASK_FULL) return in;
  return in & (low_bits(w.past - at) | bits_at(tree, w.a.words, at - w.past));
}
__device__ __forceinline__ bool finite_bf16(uint32_t half) { return (half & 0x7f80u) != 0x7f80u; }
// A pair of bf16 with what is not finite replaced by zero.
__device__ __forceinline__ uint32_t only_finite(uint32_t x) {
  if (!finite_bf16(x)) x &= 0xffff0000u;
  if (!finite_bf16(x >> 16)) x &= 0x0000ffffu;
  return x;
}

// ---------------------------------------------------------------------------
// Loads.
// ---------------------------------------------------------------------------
// Two e4m3 codes to bf16 x 2^e; exact (4 significant bits, and the exponents
// of a written cache keep code and product normal).
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t pair, float scale) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16(f.x * scale, f.y * scale);
}
// 2^(e - 127) for a row's exponent byte; any byte is one that fp32 holds, also in
// rows never written. (A code that it takes beyond bf16 enters as an infinity.)
__device__ __forceinline__ float exponent_scale(uint8_t e) {
  return __uint_as_float(max(1u, min(254u, (uint32_t)e)) << 23);
}
// kv_row() with the division as a product.
__device__ __forceinline__ int cache_row(const Args& a, const int32_t* table, int64_t pos, int head) {
  const dg_kv_cache& c = a.w.c;
  if (pos >= 0 && pos <= 0x7fffffff) {
    const uint32_t at = a.over_page((uint32_t)pos);
    if (at < (uint32_t)a.w.b.table_stride) {
      const int page = __ldg(table + at);
      if (page >= 0 && page < c.pages)
        return (page * c.kv_heads + head) * c.page_size + (int)((uint32_t)pos - at * (uint32_t)c.page_size);
    }
  }
  raise_status(c.status, DG_EINVAL);
  return -1;
}

// The cache rows of a key tile: rows lane, lane + 32, ... from position j0 on; -1
// beyond the sequence or without a page.
template <class S, typename W>
__device__ __forceinline__ void find_rows(const W& w, int64_t j0, int* row) {
  const int32_t* table = w.a.w.b.page_table + (int64_t)w.b * w.a.w.b.table_stride;
  const int64_t L = w.keys();
#pragma unroll
  for (int p = 0; p < S::BN / 32; ++p) {
    const int64_t j = j0 + p * 32 + (threadIdx.x & 31);
    row[p] = j < L ? cache_row(w.a, table, j, w.h) : -1;
  }
}
// 32 entries of a sequence's page table in the lanes of a warp: a look-up per tile
// had cost more than the tile's copies.
struct Pages {
  int b = -1, base = 0, page = 0;
};
// The same for TMA, by eights (a.box != 0: page_size is a multiple of 8): lane l
// gets the cache row of position j0 + 8 l, l < BN / 8 (behind the sequence's end
// any row: the keys there are masked, the values set to zero); whether all rows
// up to the end have pages.
template <class S, typename W>
__device__ __forceinline__ bool find_eights(const W& w, Pages& pg, int64_t j0, int* eight) {
  *eight = -1;
  if (w.a.box == 0 || j0 >= w.keys()) return false;
  const dg_kv_cache& c = w.a.w.c;
  const int lane = threadIdx.x & 31;
  const uint32_t ps = (uint32_t)c.page_size, lo = w.a.over_page((uint32_t)j0);
  const uint32_t j = (int64_t)j0 + lane * 8 < w.keys() ? (uint32_t)j0 + lane * 8 : (uint32_t)j0, at = w.a.over_page(j);
  if (pg.b != w.b || (int)lo < pg.base || (int)w.a.over_page((uint32_t)j0 + S::BN - 8) >= pg.base + 32) {
    pg.b = w.b;
    pg.base = (int)lo;
    const int64_t t = (int64_t)lo + lane;
    pg.page = t < w.a.w.b.table_stride ? __ldg(w.a.w.b.page_table + (int64_t)w.b * w.a.w.b.table_stride + t) : -1;
  }
  const int page = __shfl_sync(0xffffffffu, pg.page, (int)at - pg.base);
  if (lane < S::BN / 8 && page >= 0 && page < c.pages)
    *eight = (page * c.kv_heads + w.h) * c.page_size + (int)(j - at * ps);
  return __all_sync(0xffffffffu, *eight >= 0 || lane >= S::BN / 8) != 0;
}

// Single rows. One warp copies a key tile (zeros for a row of -1): bf16 to a ring
// slot, e4m3 codes to their buffer, rows of DP bytes.
template <class S>
__device__ __forceinline__ void copy_rows(const Args& a, const void* pages, const int* row, uint32_t dst) {
  const int lane = threadIdx.x & 31, D = a.w.c.head_dim;
  auto pick = [&](int p) {                         // row[p], by selects
    int x = row[0];
#pragma unroll
    for (int t = 1; t < S::BN / 32; ++t) x = p == t ? row[t] : x;
    return x;
  };
  if constexpr (!S::F8) {
    constexpr int CPR = S::DP / 8, RPI = 32 / CPR; // chunks per row, rows per instruction
    const int c = lane % CPR;
    const bool in = c * 8 < D;
    const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(pages) + c * 8;
#pragma unroll 1
    for (int p = 0; p < S::BN / 32; ++p) {
      const int mine = pick(p);
#pragma unroll 8
      for (int it = 0; it < 32 / RPI; ++it) {
        const int r = it * RPI + lane / CPR;
        const int cr = __shfl_sync(0xffffffffu, mine, r);
        const bool on = in && cr >= 0;
        copy16(dst + swizzled(p * 32 + r, c, S::BN), on ? base + (int64_t)cr * D : a.q, on ? 16 : 0);
      }
    }
  } else {
    constexpr int CPR = S::DP / 16, RPI = 32 / CPR;
    const int c = lane % CPR;
    const bool in = c * 16 < D;
    const uint8_t* base = static_cast<const uint8_t*>(pages) + c * 16;
#pragma unroll 1
    for (int p = 0; p < S::BN / 32; ++p) {
      const int mine = pick(p);
#pragma unroll 8
      for (int it = 0; it < 32 / RPI; ++it) {
        const int r = it * RPI + lane / CPR;
        const int cr = __shfl_sync(0xffffffffu, mine, r);
        const bool on = in && cr >= 0;
        copy16(dst + (p * 32 + r) * S::DP + c * 16, on ? base + (int64_t)cr * D : (const void*)a.q, on ? 16 : 0);
      }
    }
  }
}

// Runs of rows: the lanes' TMA copies of a key tile, counted on `bar`. (Whoever
// last used the buffer has fenced its ordinary accesses.)
template <class S>
__device__ __forceinline__ void copy_boxes(const Args& a, const CUtensorMap* map, int eight, uint32_t dst, uint64_t* bar) {
  constexpr int NB = S::F8 ? 1 : S::DP / 64;       // copies side by side: 64 columns of bf16, whole rows of codes
  const int lane = threadIdx.x & 31;
  const int run = lane / NB * a.box, cb = lane % NB;            // the lane's rows and columns
  const int first = __shfl_sync(0xffffffffu, eight, (run >> 3) & 31);   // (a run lies in one page, its head before the end)
  if (lane == 0) mbar_expect_tx(bar, S::BN * S::DP * (S::F8 ? 1 : 2));
  __syncwarp();
  if (run < S::BN)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            S::F8 ? dst + run * S::DP : dst + (cb * S::BN + run) * 128),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(cb * 64), "r"(first)
        : "memory");
  __syncwarp();
}

// Warp `part` of N_LOAD brings its share of the item's query rows.
template <class S, typename W>
__device__ __forceinline__ void load_queries(const W& w, int part, uint32_t dst) {
  constexpr int CPR = S::DP / 8, RPI = 32 / CPR, ROWS = S::NT * 128;
  const Args& a = w.a;
  const int lane = threadIdx.x & 31, c = lane % CPR, rows = w.rows();
#pragma unroll 4
  for (int r0 = part * RPI; r0 < rows; r0 += S::N_LOAD * RPI) {
    const int r = r0 + lane / CPR;
    const uint32_t rid = (uint32_t)w.m * ROWS + (r < rows ? r : 0);
    const uint32_t i = a.over_g(rid), g = rid - i * (uint32_t)a.G;
    const bool on = r < rows && c * 8 < a.w.c.head_dim;
    const __nv_bfloat16* src = on ? a.q + (int64_t)(w.t0 + i) * a.q_ts + (int64_t)(w.h * a.G + g) * a.q_hs + c * 8 : a.q;
    copy16(dst + (r >> 7) * S::QTILE + swizzled(r & 127, c, 128), src, on ? 16 : 0);
  }
  copies_landed();
}

// The same by TMA, one warp for all: a row r of an item is token r / G, head
// r % G, so that G heads of 32 / G tokens, as a box takes them, are 32 rows in
// order. (Rows behind the sequence's last hold the next one's, or zeros; no
// other row's result depends on them.)
template <class S, typename W>
__device__ __forceinline__ void query_boxes(const W& w, const CUtensorMap* map, uint32_t dst, uint64_t* bar) {
  constexpr int NB = S::DP / 64, ROWS = S::NT * 128;
  const int lane = threadIdx.x & 31, rows = w.rows();
  const int group = lane / NB, cb = lane % NB, n = (rows + 31) / 32;   // groups of 32 rows
  if (lane == 0) mbar_expect_tx(bar, n * NB * 32 * 128);
  __syncwarp();
  if (group < n) {
    const uint32_t i = w.a.over_g((uint32_t)w.m * ROWS + group * 32);
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            dst + (group >> 2) * S::QTILE + cb * (128 * 128) + (group & 3) * (32 * 128)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(cb * 64), "r"(w.h * w.a.G), "r"(w.t0 + (int)i)
        : "memory");
  }
  __syncwarp();
}

// e4m3: rows r0 to r0 + BN / TEAM of a tile of codes to bf16 in a ring slot. (The
// same by moving the codes' bits and one packed product took as long: 48
// conversions and products or 60 integer instructions for 16 codes.)
template <class S>
__device__ __forceinline__ void convert(const uint8_t* exps, int r0, uint32_t src, uint32_t slot) {
  constexpr int CPR = S::DP / 16, RPI = 32 / CPR, N = S::BN / S::TEAM / RPI;   // 16-code chunks of a row, rows at a time
  constexpr int K = N < 4 ? N : 4;
  const int lane = threadIdx.x & 31, q = lane % CPR, cb = q >> 2;
#pragma unroll 1
  for (int n = 0; n < N; n += K) {
    const int r = r0 + n * RPI + lane / CPR;
    uint4 v[K];
    float scale[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = ld_shared(src + (r + k * RPI) * S::DP + q * 16);
      scale[k] = exponent_scale(exps[r + k * RPI]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t x[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      uint32_t o[8];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        o[2 * t] = codes_to_bf16(x[t], scale[k]);
        o[2 * t + 1] = codes_to_bf16(x[t] >> 16, scale[k]);
      }
      // 8 neighbouring lanes write all 8 chunks' places of the swizzle: lanes of an
      // odd block take their second chunk first
      const uint32_t to = slot + cb * (S::BN * 128) + (r + k * RPI) * 128;
      const uint32_t c0 = 2 * (q & 3), sw = (r + k * RPI) & 7;
      const bool odd = cb & 1;
      const uint4 a0 = make_uint4(o[0], o[1], o[2], o[3]), a1 = make_uint4(o[4], o[5], o[6], o[7]);
      st_shared(to + (((c0 + (odd ? 1 : 0)) ^ sw) << 4), odd ? a1 : a0);
      st_shared(to + (((c0 + (odd ? 0 : 1)) ^ sw) << 4), odd ? a0 : a1);
    }
  }
}

// Rows r0 to r0 + RW of a value tile in its slot: those from `live` on, behind
// the sequence's end, become zeros; with `scrub`, what is not finite in the
// others too, and is noted. For tiles that hold positions which a query row of
// the item may not see: 0 x NaN in the second product would reach every row.
template <class S, int RW>
__device__ __forceinline__ void clean_rows(uint32_t slot, int r0, int live, bool scrub, Sync& sy) {
  constexpr int CPR = S::DP / 8, RPI = 32 / CPR, N = RW / RPI;
  const int lane = threadIdx.x & 31, c = lane % CPR;
  bool dirty = false;
  __syncwarp();
#pragma unroll 4
  for (int it = 0; it < N; ++it) {
    const int r = r0 + it * RPI + lane / CPR;
    const uint32_t at = slot + swizzled(r, c, S::BN);
    if (r >= live) {
      st_shared(at, make_uint4(0, 0, 0, 0));
    } else if (scrub) {
      const uint4 v = ld_shared(at);
      // an exponent of all ones carries into the sign's place
      const uint32_t t = ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
                         ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
      if (t & 0x80008000u) {
        st_shared(at, make_uint4(only_finite(v.x), only_finite(v.y), only_finite(v.z), only_finite(v.w)));
        dirty = true;
      }
    }
  }
  if (dirty) *(volatile int*)&sy.nonfinite = 1;
}

// Logit of a query row (head_dim bf16) and a cache row, as the products have it up
// to the order of its sum. For rows whose value is not finite only.
template <class S>
__device__ __forceinline__ float logit_of(const Args& a, const __nv_bfloat16* q, int row) {
  float z = 0.f;
  for (int d = 0; d < a.w.c.head_dim; ++d) {
    const int64_t at = (int64_t)row * a.w.c.head_dim + d;
    uint32_t k;
    if constexpr (S::F8)
      k = codes_to_bf16(static_cast<const uint8_t*>(a.w.c.k)[at], exponent_scale(a.w.c.k_exp[row]));
    else
      k = static_cast<const uint16_t*>(a.w.c.k)[at];
    z = fmaf(to_f32(q[d]), __uint_as_float(k << 16), z);
  }
  return z * a.scale_log2;
}

// Adds to a warp's rows of O (in TMEM; orow: a lane's output row, one of the
// sequence's, or -1) the infinities and NaN among the values that each sees in the
// segment's keys from position `from` on, where clean_rows has left them out. They
// are added as they are, whatever their positive weight; times a weight of zero (a
// logit of minus infinity) an infinity is NaN. (A long tree's search can outlast
// the limit of the waits behind it, so it says that it goes on.)
template <class S, typename W>
__device__ __noinline__ void add_not_finite(const W w, int orow, int64_t from, uint32_t t_o) {
  const Args& a = w.a;
  const int D = a.w.c.head_dim, token = orow / a.q_heads, i = token - w.t0;
  const uint32_t* tree = a.mask == DG_MASK_TREE ? a.tree + (int64_t)token * a.words : nullptr;
  const __nv_bfloat16* q = a.q + (int64_t)token * a.q_ts + (int64_t)(orow - token * a.q_heads) * a.q_hs;
  const int64_t end = min(w.keys(), (int64_t)w.te * S::BN);
  for (int d = 0; d < D; d += 16) {                  // (head_dim is a multiple of 16)
    uint32_t o[16];
    __syncwarp();
    tmem_ld16_issue(t_o + d, o);
    tmem_ld16_wait(o);
    float x[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = 0.f;
    for (int64_t j = orow < 0 ? end : max(from, (int64_t)w.tb * S::BN); j < end; ++j) {
      if ((j & 63) == 0) *(volatile uint64_t*)&sync_of<S>().busy = gtimer();
      if (!(seen(w, tree, i, j) & 1)) continue;
      const int row = cache_row(a, a.w.b.page_table + (int64_t)w.b * a.w.b.table_stride, j, w.h);
      if (row < 0) continue;
      const int64_t at = (int64_t)row * D + d;
      uint32_t c[8];                                 // the values as they enter the products
      if constexpr (S::F8) {
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.w.c.v) + at);
        const uint32_t codes[4] = {v.x, v.y, v.z, v.w};
        const float scale = exponent_scale(a.w.c.v_exp[row]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          c[2 * k] = codes_to_bf16(codes[k], scale);
          c[2 * k + 1] = codes_to_bf16(codes[k] >> 16, scale);
        }
      } else {
        const uint4* v = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.w.c.v) + at);
        const uint4 v0 = v[0], v1 = v[1];
        c[0] = v0.x; c[1] = v0.y; c[2] = v0.z; c[3] = v0.w;
        c[4] = v1.x; c[5] = v1.y; c[6] = v1.z; c[7] = v1.w;
      }
      bool fine = true;
#pragma unroll
      for (int k = 0; k < 8; ++k) fine = fine && only_finite(c[k]) == c[k];
      if (fine) continue;
      const bool zero = logit_of<S>(a, q, row) == -INFINITY;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const uint32_t half = c[k >> 1] >> (16 * (k & 1)) & 0xffffu;
        if (!finite_bf16(half)) x[k] += zero ? NAN : __uint_as_float(half << 16);
      }
    }
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (x[k] != 0.f) o[k] = __float_as_uint(__uint_as_float(o[k]) + x[k]);
    __syncwarp();
    tmem_st16(t_o + d, o);
  }
  tmem_st_wait();
}

// A 4 x 4 transposition of 16-byte pieces over each four lanes: lane q of four
// leaves with piece q of the four lanes' rows.
__device__ __forceinline__ void transpose4(uint4* v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & d) continue;
      uint4 t = up ? v[i] : v[i | d];
      t.x = __shfl_xor_sync(0xffffffffu, t.x, d);
      t.y = __shfl_xor_sync(0xffffffffu, t.y, d);
      t.z = __shfl_xor_sync(0xffffffffu, t.z, d);
      t.w = __shfl_xor_sync(0xffffffffu, t.w, d);
      if (up) v[i] = t;
      else v[i | d] = t;
    }
  }
}

// ---------------------------------------------------------------------------
// The kernel.
// ---------------------------------------------------------------------------
template <class S>
__global__ void __launch_bounds__(S::THREADS, 1) k_attend(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap k_map,
                                                           const __grid_constant__ CUtensorMap v_map,
                                                           const __grid_constant__ CUtensorMap q_map) {
  unsigned char* smem = tiles();
  unsigned char* ring = smem + S::NT * S::QTILE;
  unsigned char* codes = ring + S::SL * S::SLOT;
  Sync& sy = sync_of<S>();
  static_assert(sizeof(Sync) <= 1024 && S::SL <= 8 && S::N_LOAD <= 8 && S::AHEAD <= 4, "barriers");
  int64_t* pref = reinterpret_cast<int64_t*>(ring);
  constexpr int ROWS = S::NT * 128, BN = S::BN;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::SL; ++s) mbar_init(&sy.full[s], S::F8 ? S::TEAM : 1);
    for (int x = 0; x < 8; ++x) {
      mbar_init(&sy.s_full[x], 1);
      mbar_init(&sy.p_full[x], 4);
      mbar_init(&sy.o_done[x], 1);
      if (x < 2) mbar_init(&sy.o_free[x], 4);
    }
    mbar_init(&sy.q_full, a.q_box ? 1 : S::N_LOAD);
    mbar_init(&sy.q_free, 1);
    mbar_init(&sy.fin, 1);
    for (int x = 0; x < 8; ++x) mbar_init(&sy.raw[x], S::F8 ? 1 + BN / 8 : 1);
    for (int x = 0; x < S::AHEAD; ++x) mbar_init(&sy.taken[x], S::TEAM);
    sy.abort = 0;
    sy.busy = 0;
    sy.nonfinite = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == S::W_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::
                     "r"(smem_u32(&sy.tmem)), "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  plan<ROWS, BN>(a, pref, &sy.start);                 // ends with a block barrier
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = *(volatile uint32_t*)&sy.tmem;
  Walk<ROWS, BN> w(a);
  begin(w, sy.start);

  if (warp < S::W_LOAD) {
    // ---------------------------------------------------------------- softmax
    const int x = warp >> 2;                          // row tile
    const int quarter = warp & 3;
    const int r = x * 128 + quarter * 32 + lane;      // row of the tiles
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t t_o = tmem + S::T_O + x * S::DP + lanes;
    bool ok = true;
    uint32_t gt = 0;                                  // key tiles done by this CTA
    auto pv_done = [&](uint32_t k) { return wait_warp(&sy.o_done[4 * x + (k & 3)], (k >> 2) & 1, sy, a); };
    Open open{0, 0, 0, 0, 0};                         // an item begun and not finished
    for (; w.more() && ok; w.next()) {
      const int rows = w.rows();
      const bool any = x * 128 + quarter * 32 < rows; // warp-uniform
      const bool valid = r < rows;
      const uint32_t rid = (uint32_t)w.m * ROWS + (valid ? r : 0);
      const int i = (int)a.over_g(rid), g = (int)(rid - (uint32_t)i * a.G);
      const uint32_t* tree = a.mask == DG_MASK_TREE ? a.tree + (int64_t)(w.t0 + i) * a.words : nullptr;
      // tiles that reach beyond this position hold some that the row may not see
      const int64_t clear = a.mask == DG_MASK_FULL ? w.keys() : a.mask == DG_MASK_CAUSAL ? (int64_t)w.past + i + 1 : w.past;
      float m = -INFINITY, l = 0.f;                   // m unscaled
      for (int t = w.tb; t < w.te; ++t, ++gt) {
        const int bar = 4 * x + (int)(gt & 3);
        if (!wait_warp(&sy.s_full[bar], (gt >> 2) & 1, sy, a)) { ok = false; break; }
        if (any) {
          tc_fence_after();
          const uint32_t t_s = tmem + (S::NT == 2 ? x : (int)(gt & 1)) * BN + lanes;
          const int64_t j0 = (int64_t)t * BN;
          const bool masked = __any_sync(0xffffffffu, j0 + BN > clear);
          // The usual tile, all columns seen: straight code, the next 16 columns on
          // their way from TMEM while one chunk is worked on.
          bool plain = !masked;
          uint32_t ra[16], rb[16];
          float top = -INFINITY;
          if (plain) {
            tmem_ld16_issue(t_s, ra);
#pragma unroll
            for (int c = 0; c < BN / 16; ++c) {
              uint32_t* r = c & 1 ? rb : ra;
              tmem_ld16_wait(r);
              if (c + 1 < BN / 16) tmem_ld16_issue(t_s + (c + 1) * 16, c & 1 ? ra : rb);
              float u0 = top, u1 = __uint_as_float(r[15]);
#pragma unroll
              for (int j = 0; j < 14; j += 4) {
                u0 = max3_nan(u0, __uint_as_float(r[j]), __uint_as_float(r[j + 1]));
                if (j + 3 < 15) u1 = max3_nan(u1, __uint_as_float(r[j + 2]), __uint_as_float(r[j + 3]));
                else u1 = max3_nan(u1, __uint_as_float(r[j + 2]), u1);
              }
              top = max3_nan(u0, u1, u1);
            }
            // a maximum that is NaN, infinite or very large: below, with differences of
            // unscaled logits (here the maximum's rounding would be one of the exponent)
            plain = !__any_sync(0xffffffffu, valid && !(fabsf(top * a.scale_log2) < kLarge));
          }
          // others: 32 columns at a time
          const int chunks = plain ? 0 : BN / 32;
          float s[32];
          if (!plain) top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            tmem_ld32(t_s + c * 32, s);
            if (masked) {
              const uint32_t word = seen(w, tree, i, j0 + c * 32);
#pragma unroll
              for (int j = 0; j < 32; ++j) s[j] = (word >> j) & 1 ? s[j] : -INFINITY;
            }
            float u0 = -INFINITY, u1 = -INFINITY;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              u0 = fmaxf(u0, fmaxf(s[j], s[j + 1]));
              u1 = fmaxf(u1, fmaxf(s[j + 2], s[j + 3]));
            }
            top = fmaxf(top, fmaxf(u0, u1));
          }
          // the maximum in use moves at the first tile and when it has grown by kGrow
          // (two of -infinity: NaN, no move)
          const bool first = t == w.tb;
          const bool move = (top - m) * a.scale_log2 > kGrow;
          if (!first && __any_sync(0xffffffffu, move && valid)) {
            if (!pv_done(gt - 1)) { ok = false; break; }
            tc_fence_after();
            const float f = move ? ex2((m - top) * a.scale_log2) : 1.f;
            l *= f;
#pragma unroll 1
            for (int c = 0; c < S::DP / 32; ++c) {
              float o[32];
              tmem_ld32(t_o + c * 32, o);
              uint32_t p[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) p[j] = __float_as_uint(o[j] * f);
              tmem_st16(t_o + c * 32, p);
              tmem_st16(t_o + c * 32 + 16, p + 16);
            }
            tmem_st_wait();
          }
          if (move) m = top;
          const float sub = m == -INFINITY ? 0.f : m;  // a row that has seen nothing yet: P = 0
          float l0 = 0.f, l1 = 0.f;
          if (plain) {
            const float to = -sub * a.scale_log2;
            const uint64_t sc = pack2(a.scale_log2, a.scale_log2), ns = pack2(to, to);
            uint64_t ls = pack2(0.f, 0.f);
            tmem_ld16_issue(t_s, ra);
#pragma unroll
            for (int c = 0; c < BN / 16; ++c) {
              uint32_t* r = c & 1 ? rb : ra;
              tmem_ld16_wait(r);
              if (c + 1 < BN / 16) tmem_ld16_issue(t_s + (c + 1) * 16, c & 1 ? ra : rb);
              uint32_t p[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const uint64_t x = fma2(pack2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), sc, ns);
                const uint64_t e = S::NT == 2 && (j & 3) == 3 ? exp2_poly2(x) : exp2_mufu2(x);
                ls = add2(ls, e);
                p[j] = pack_bf16(lo2(e), hi2(e));
              }
              tmem_st8(t_s + c * 8, p);
            }
            l0 = lo2(ls);
            l1 = hi2(ls);
          }
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            tmem_ld32(t_s + c * 32, s);
            if (masked) {
              const uint32_t word = seen(w, tree, i, j0 + c * 32);
#pragma unroll
              for (int j = 0; j < 32; ++j) s[j] = (word >> j) & 1 ? s[j] : -INFINITY;
            }
            uint32_t p[16];
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float e0 = ex2((s[j] - sub) * a.scale_log2);
              const float e1 = ex2((s[j + 1] - sub) * a.scale_log2);
              l0 += e0;
              l1 += e1;
              p[j >> 1] = pack_bf16(e0, e1);
            }
            tmem_st16(t_s + c * 16, p);
          }
          l += l0 + l1;
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0 && gt + 1 != a.stall) mbar_arrive(&sy.p_full[bar]);
      }
      if (!ok) break;
      // ---------------------------------------------------------- the segment's result
      if (!pv_done(gt - 1)) { ok = false; break; }
      const bool whole = w.tb == 0 && w.te == w.T;
      const bool fix = a.mask != DG_MASK_FULL && __any_sync(0xffffffffu, *(volatile int*)&sy.nonfinite);
      const int piece = blockIdx.x * 2 + (w.tb == 0 ? 1 : 0);
      const int orow = (w.t0 + i) * a.q_heads + w.h * a.G + g;
      const int64_t prow = (int64_t)piece * a.rows + r;
      tc_fence_after();
      if (any) {
        if (fix) add_not_finite<S>(w, valid ? orow : -1, w.clear() / BN * BN, t_o);
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
        // stores by fours of lanes, 64 contiguous bytes of a row each
        const int four = lane & ~3, q = lane & 3;
#pragma unroll 1
        for (int c = 0; c < S::DP / 32; ++c) {
          float o[32];
          __syncwarp();                               // the lanes part below; TMEM loads take all of them
          tmem_ld32(t_o + c * 32, o);
          if (whole) {
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              v[k] = make_uint4(pack_bf16(o[8 * k] * inv, o[8 * k + 1] * inv),
                                pack_bf16(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                                pack_bf16(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                                pack_bf16(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
            transpose4(v);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int to = __shfl_sync(0xffffffffu, valid ? orow : -1, four + k);
              if (to >= 0 && c * 32 + q * 8 < a.w.c.head_dim)
                *reinterpret_cast<uint4*>(a.out + (int64_t)to * a.w.c.head_dim + c * 32 + q * 8) = v[k];
            }
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint4 v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                v[k] = make_uint4(__float_as_uint(o[16 * h + 4 * k]), __float_as_uint(o[16 * h + 4 * k + 1]),
                                  __float_as_uint(o[16 * h + 4 * k + 2]), __float_as_uint(o[16 * h + 4 * k + 3]));
              transpose4(v);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (r - q + k < rows)
                  *reinterpret_cast<uint4*>(a.part_o + (prow - q + k) * S::DP + c * 32 + h * 16 + q * 4) = v[k];
            }
          }
        }
        if (valid && whole && a.lse) a.lse[orow] = l == 0.f ? -INFINITY : fmaf(m, a.scale_log2, log2f(l)) * kLn2;
        if (valid && !whole) a.part_ml[prow] = make_float2(m, l);
      }
      __syncwarp();
      tc_fence_before();
      if (w.tb == 0 && w.te < w.T)
        open = Open{rows, (int)((w.at + kItem + w.T - 1) / sy.start.share) - (int)blockIdx.x + 1, w.t0, w.h, w.m};
      __syncwarp();
      if (lane == 0) mbar_arrive(&sy.o_free[x]);
    }
    if (threadIdx.x == 0) {
      if (!ok) open.rows = 0;
      a.open[blockIdx.x] = open;
    }
  } else if (warp < S::W_MMA) {
    // ---------------------------------------------------------------- key and value loads
    const int part = warp - S::W_LOAD;
    const uint32_t ring0 = smem_u32(ring), codes0 = smem_u32(codes);
    bool ok = true;
    Pages pages;
    uint32_t e = 0, e0 = 0, seg = 0;                  // ring entry; the segment's first, tile tb's keys; segments
    bool q_landing = false;                           // this warp brings the queries by TMA; the last copy's phase
    uint32_t q_phase = 0;
    auto queries = [&]() {
      if (a.q_box && part) return true;
      if (seg && !wait_warp(&sy.q_free, (seg - 1) & 1, sy, a)) return false;
      if (a.q_box) {
        query_boxes<S>(w, &q_map, smem_u32(smem), &sy.q_full);
        q_landing = true;
        q_phase = seg & 1;
        return true;
      }
      load_queries<S>(w, part, smem_u32(smem));
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sy.q_full);
      return true;
    };
    // a CTA that gives up still waits for its last copies
    auto drain_queries = [&]() {
      if (q_landing) wait(&sy.q_full, q_phase, sy, a, false);
    };
    // the slot of ring entry e is free: entry e - SL, a key tile's keys or values, has been taken
    auto released = [&]() {
      if (e < S::SL) return true;
      const uint32_t k = (e - S::SL) >> 1, bar = 4 * (S::NT - 1) + (k & 3);
      return wait_warp((e - S::SL) & 1 ? &sy.o_done[bar] : &sy.s_full[bar], (k >> 2) & 1, sy, a);
    };
    auto position = [&]() { return (int64_t)(w.tb + (int)((e - e0) >> 1)) * BN; };
    // of entry e: its rows before the sequence's end; whether it holds values that not every row of the item sees
    auto live_rows = [&]() { return (int)min((int64_t)BN, w.keys() - position()); };
    // (not behind the end: a single token's last tile has none)
    auto to_scrub = [&]() { return ((e - e0) & 1) && min(position() + BN, w.keys()) > w.clear(); };
    if constexpr (!S::F8) {
      // one warp per slot, entries SL apart
      bool landing = false;                           // the slot's last copy is by TMA, and has not been waited for
      uint32_t raws = 0;
      e = part;
      for (; w.more() && ok; w.next(), ++seg) {
        const uint32_t n = 2 * (uint32_t)(w.te - w.tb);
        bool q_due = true;
        for (;; e += S::SL) {
          // the queries: after an entry whose slot waits for the segment before
          if (q_due && (e - e0 >= n || e >= e0 + S::SL)) {
            q_due = false;
            if (!queries()) { ok = false; break; }
          }
          if (e - e0 >= n) break;
          const bool kv = (e - e0) & 1, scrub = to_scrub();
          const int live = live_rows();
          const bool clean = scrub || (kv && live < BN);
          const uint32_t dst = ring0 + part * S::SLOT;
          int eight, row[BN / 32];
          const bool boxes = find_eights<S>(w, pages, position(), &eight);    // under the wait for the slot
          if (!boxes) find_rows<S>(w, position(), row);
          if (!released()) { ok = false; break; }
          landing = boxes && !clean;
          if (landing) {                              // the copies arrive on `full` themselves
            copy_boxes<S>(a, kv ? &v_map : &k_map, eight, dst, &sy.full[part]);
            continue;
          }
          if (boxes) {
            copy_boxes<S>(a, &v_map, eight, dst, &sy.raw[part]);
            if (!wait_warp(&sy.raw[part], raws++ & 1, sy, a)) {
              wait(&sy.raw[part], (raws - 1) & 1, sy, a, false);
              ok = false;
              break;
            }
          } else {
            copy_rows<S>(a, kv ? a.w.c.v : a.w.c.k, row, dst);
            copies_landed();
          }
          if (clean) clean_rows<S, BN>(dst, 0, live, scrub, sy);
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sy.full[part]);
        }
        e0 += n;
      }
      drain_queries();
      if (landing) wait(&sy.full[part], (e / S::SL - 1) & 1, sy, a, false);
    } else if (warp >= S::W_FETCH) {
      // codes and exponents, AHEAD tiles before they are converted: a warp for the keys', one for the values'
      const uint32_t mine = warp - S::W_FETCH;
      for (; w.more() && ok; w.next()) {
        const uint32_t n = 2 * (uint32_t)(w.te - w.tb);
        for (e = e0 + mine; e - e0 < n; e += 2) {
          const uint32_t at = e % S::AHEAD, dst = codes0 + at * S::RAW;
          const bool kv = (e - e0) & 1;
          const uint8_t* exps = kv ? a.w.c.v_exp : a.w.c.k_exp;
          int eight, row[BN / 32];
          const bool boxes = find_eights<S>(w, pages, position(), &eight);    // under the wait for the buffer
          if (!boxes) find_rows<S>(w, position(), row);
          if (!wait_warp(&sy.taken[at], ((e / S::AHEAD) & 1) ^ 1, sy, a)) { ok = false; break; }
          if (boxes) {
            copy_boxes<S>(a, kv ? &v_map : &k_map, eight, dst, &sy.raw[at]);
            // an arrival of each of these lanes when its eight exponents have landed
            if (lane < BN / 8)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n\t"
                           "cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%2];" ::"r"(smem_u32(&sy.exps[at][lane * 8])),
                           "l"(exps + eight), "r"(smem_u32(&sy.raw[at]))
                           : "memory");
          } else {
            copy_rows<S>(a, kv ? a.w.c.v : a.w.c.k, row, dst);
#pragma unroll
            for (int p = 0; p < BN / 32; ++p)
              sy.exps[at][p * 32 + lane] = row[p] >= 0 ? __ldg(exps + row[p]) : (uint8_t)127;
            copies_landed();
            __syncwarp();
            if (lane <= BN / 8) mbar_arrive(&sy.raw[at]);
          }
        }
        e0 += n;
      }
      // as above: of the last AHEAD tiles
      for (uint32_t x = e > S::AHEAD ? e - S::AHEAD : 0; x < e; ++x)
        if ((x & 1) == mine) wait(&sy.raw[x % S::AHEAD], (x / S::AHEAD) & 1, sy, a, false);
    } else {
      // half of the warps on the keys, half on the values, each its own rows
      constexpr int RW = BN / S::TEAM;
      const uint32_t team = part / S::TEAM;
      const int r0 = part % S::TEAM * RW;
      for (; w.more() && ok; w.next(), ++seg) {
        const uint32_t n = 2 * (uint32_t)(w.te - w.tb);
        for (e = e0 + team; e - e0 < n; e += 2) {
          const uint32_t at = e % S::AHEAD, slot = e % S::SL, dst = ring0 + slot * S::SLOT;
          if (!wait_warp(&sy.raw[at], (e / S::AHEAD) & 1, sy, a) ||
              !released()) { ok = false; break; }
          convert<S>(sy.exps[at], r0, codes0 + at * S::RAW, dst);
          const bool scrub = to_scrub();
          const int live = live_rows();
          if (scrub || (((e - e0) & 1) && live < r0 + RW)) clean_rows<S, RW>(dst, r0, live, scrub, sy);
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sy.full[slot]);
            mbar_arrive(&sy.taken[at]);
          }
          // the queries, once the first entry is on its way
          if (e - e0 < 2 && !queries()) { ok = false; break; }
        }
        e0 += n;
      }
      drain_queries();
    }
  } else {
    // ---------------------------------------------------------------- MMA
    // (the warp waits together, one elected lane issues)
    constexpr uint32_t id_s = idesc_bf16(128, BN, 0), id_o = idesc_bf16(128, S::DP, 1);
    const uint32_t q0 = smem_u32(smem), ring0 = smem_u32(ring);
    uint32_t gt = 0, seg = 0;                         // key tiles and segments so far; tile k's keys and values
                                                      // are ring entries 2 k and 2 k + 1
    bool ok = true;
    auto slot_full = [&](uint32_t entry) { return wait_warp(&sy.full[entry % S::SL], (entry / S::SL) & 1, sy, a); };
    // Addresses and descriptors are made the same in every lane, in a form the
    // compiler can see (uniform registers are what the MMA takes), once for each
    // product, and one elected lane issues: building them in a divergent lane for
    // each instruction cost more than the MMA's own time.
    const uint32_t tm = uniform(tmem);
    const uint64_t qd = sdesc(uniform(q0), 16, 1024);
    const uint64_t kd = sdesc(uniform(ring0), 16, 1024), vd = sdesc(uniform(ring0), BN * 128, 1024);
    // Products run in the order of their issue only where accumulator and shape are
    // the same. S of a key tile goes where P of an earlier one lies, so it is issued
    // when that tile's P V, which reads it, is done (by issue order alone the prompt
    // took 322 us for 326, canvases over a bf16 cache 92 for 95; one row tile, whose
    // buffers alternate, no less).
    auto pv_done = [&](uint32_t k, int x) { return wait_warp(&sy.o_done[4 * x + (k & 3)], (k >> 2) & 1, sy, a); };
    auto scores = [&](uint32_t k, int x, bool last) {   // S = Q(x) K^T of key tile k; the last of a segment frees Q
      tc_fence_after();
      const uint64_t b = kd + uniform((2 * k) % S::SL) * (uint64_t)(S::SLOT / 16);
      const uint32_t d = tm + uniform(S::NT == 2 ? x : (int)(k & 1)) * BN;
      uint64_t* bar = &sy.s_full[uniform(4 * x + (k & 3))];
      if (elected()) {
#pragma unroll
        for (int c = 0; c < S::DP / 16; ++c)
          mma_bf16(d, qd + (x * S::QTILE + (c >> 2) * (128 * 128) + (c & 3) * 32) / 16,
                   b + ((c >> 2) * (BN * 128) + (c & 3) * 32) / 16, id_s, c ? 1u : 0u);
        mma_commit(bar);
        if (last && x == S::NT - 1) mma_commit(&sy.q_free);
      }
      __syncwarp();
    };
    auto sums = [&](uint32_t k, int x, bool first) {    // O(x) += P V
      tc_fence_after();
      const uint64_t b = vd + uniform((2 * k + 1) % S::SL) * (uint64_t)(S::SLOT / 16);
      const uint32_t p = tm + uniform(S::NT == 2 ? x : (int)(k & 1)) * BN;
      uint64_t* bar = &sy.o_done[uniform(4 * x + (k & 3))];
      const uint32_t add = uniform(first ? 0u : 1u);
      if (elected()) {
#pragma unroll
        for (int c = 0; c < BN / 16; ++c)
          mma_bf16_ts(tm + S::T_O + x * S::DP, p + c * 8, b + c * (2048 / 16), id_o, c ? 1u : add);
        mma_commit(bar);
      }
      __syncwarp();
    };
    constexpr uint32_t kBack = S::NT == 2 ? 1 : 2;    // key tiles since an S buffer was last used
    for (; w.more() && ok; w.next(), ++seg) {
      if (!wait_warp(&sy.q_full, seg & 1, sy, a) || !slot_full(2 * gt)) { ok = false; break; }
      const int n = w.te - w.tb;
#pragma unroll
      for (int x = 0; x < S::NT; ++x) {
        if (gt >= kBack && !pv_done(gt - kBack, x)) { ok = false; break; }
        scores(gt, x, n == 1);
      }
      if (!ok) break;
      for (int t = 0; t < n && ok; ++t, ++gt) {
        if (S::NT == 1 && t + 1 < n) {                  // the next S has a buffer of its own
          if ((gt + 1 >= kBack && !pv_done(gt + 1 - kBack, 0)) || !slot_full(2 * gt + 2)) { ok = false; break; }
          scores(gt + 1, 0, t + 2 == n);
        }
#pragma unroll
        for (int x = 0; x < S::NT; ++x) {
          if (!wait_warp(&sy.p_full[4 * x + (gt & 3)], (gt >> 2) & 1, sy, a) ||
              (t == 0 && seg && !wait_warp(&sy.o_free[x], (seg - 1) & 1, sy, a)) || (x == 0 && !slot_full(2 * gt + 1))) {
            ok = false;
            break;
          }
          sums(gt, x, t == 0);
          if (S::NT == 2 && t + 1 < n) {
            if ((x == 0 && !slot_full(2 * gt + 2)) || !pv_done(gt, x)) { ok = false; break; }
            scores(gt + 1, x, t + 2 == n);
          }
        }
      }
    }
    // every MMA issued has completed before TMEM is released and the CTA exits
    if (elected()) mma_commit(&sy.fin);
    __syncwarp();
    wait(&sy.fin, 0, sy, a, false);
    __syncwarp();
  }
  copies_landed();
  __syncthreads();
  if (warp == S::W_MMA) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS)
                 : "memory");
  }
}

// Joins the pieces of the items that lie in more than one CTA's share. The
// rows of all such items form one list that the blocks take turns at: a warp per
// row, or all eight where a row has more than kFewPieces. A row's pieces are
// added in a fixed order, so that the result does not depend on timing. Bound by
// the latency of three dependent loads (which item, its maxima, its sums); a
// block per row and piece, as it first was, took three times as long.
constexpr int kFewPieces = 16;

template <class S>
__global__ void __launch_bounds__(256) k_join(const __grid_constant__ Args a, int ctas) {
  constexpr int V = S::DP / 32;                       // columns per lane
  __shared__ float o_s[8][S::DP];
  __shared__ float m_s[8], l_s[8];
  __shared__ Open open_s[kMaxCtas];
  __shared__ int upto[kMaxCtas + 1];                  // units before each item
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x < ctas) open_s[threadIdx.x] = a.open[threadIdx.x];
  __syncthreads();
  if (warp == 0) {
    int run = 0;
    for (int b0 = 0; b0 < ctas; b0 += 32) {
      const int at = b0 + lane;
      int u = 0;
      if (at < ctas) u = open_s[at].pieces > kFewPieces ? open_s[at].rows : (open_s[at].rows + 7) / 8;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, u, d);
        if (lane >= d) u += o;
      }
      if (at < ctas) upto[at + 1] = run + u;
      run += __shfl_sync(0xffffffffu, u, 31);
    }
    if (lane == 0) upto[0] = 0;
  }
  __syncthreads();
  for (int unit = blockIdx.x; unit < upto[ctas]; unit += gridDim.x) {
    int lo = 0, hi = ctas;                            // upto[lo] <= unit < upto[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (upto[mid] <= unit) lo = mid;
      else hi = mid;
    }
    const Open op = open_s[lo];
    const bool few = op.pieces <= kFewPieces;         // the same for the whole block
    const int r = (unit - upto[lo]) * (few ? 8 : 1) + (few ? warp : 0);
    const int first = few ? 0 : warp, step = few ? 1 : 8;
    const int n = r < op.rows ? (op.pieces - first + step - 1) / step : 0;   // this warp's pieces, at most 19
    auto place = [&](int k) {                         // of its k-th
      const int p = first + k * step;
      return (int64_t)((lo + p) * 2 + (p == 0 ? 1 : 0)) * a.rows + r;
    };
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < n) ml = a.part_ml[place(lane)];
    float m = ml.x;
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float f = ex2((ml.x - (m == -INFINITY ? 0.f : m)) * a.scale_log2);
    float l = lane < n ? f * ml.y : 0.f;
#pragma unroll
    for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    float o[V];
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = 0.f;
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float* src = a.part_o + place(k) * S::DP + lane * V;
      const float g = __shfl_sync(0xffffffffu, f, k);
#pragma unroll
      for (int c = 0; c < V; c += 2) {
        const float2 x = *reinterpret_cast<const float2*>(src + c);
        o[c] = fmaf(x.x, g, o[c]);
        o[c + 1] = fmaf(x.y, g, o[c + 1]);
      }
    }
    if (!few) {
#pragma unroll
      for (int k = 0; k < V; ++k) o_s[warp][lane * V + k] = o[k];
      if (lane == 0) { m_s[warp] = m; l_s[warp] = l; }
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int p = 1; p < 8; ++p) m = fmaxf(m, m_s[p]);
        const float base = m == -INFINITY ? 0.f : m;
        l = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = 0.f;
        for (int p = 0; p < 8; ++p) {
          const float g = ex2((m_s[p] - base) * a.scale_log2);
          l += g * l_s[p];
#pragma unroll
          for (int k = 0; k < V; ++k) o[k] = fmaf(o_s[p][lane * V + k], g, o[k]);
        }
      }
      __syncthreads();
      if (warp) continue;
    }
    if (n == 0) continue;
    const uint32_t rid = (uint32_t)op.m * (S::NT * 128) + r;
    const uint32_t i = a.over_g(rid), g = rid - i * (uint32_t)a.G;
    const int64_t orow = (int64_t)(op.t0 + i) * a.q_heads + op.h * a.G + g;
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
#pragma unroll
    for (int k = 0; k < V; k += 2)
      if (lane * V + k < a.w.c.head_dim)
        *reinterpret_cast<uint32_t*>(a.out + orow * a.w.c.head_dim + lane * V + k) = pack_bf16(o[k] * inv, o[k + 1] * inv);
    if (lane == 0 && a.lse) a.lse[orow] = l == 0.f ? -INFINITY : fmaf(m, a.scale_log2, log2f(l)) * kLn2;
  }
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------
size_t al(size_t x) { return (x + 255) / 256 * 256; }

// Failure-path testing, for every later call of the process.
std::atomic<unsigned long long> wait_ns{kWaitNs};
std::atomic<uint32_t> stall{0};

struct Plan {
  int dp, nt, rows;            // padded head_dim, row tiles per item, rows kept per piece
  size_t o, ml, open, total;   // scratch offsets and size
};

// NT = 2 shares every key and value tile between two row tiles and needs more
// than 128 rows to have a second one (the prompt above: 327 us, with NT = 1 370;
// the canvases of heads of 128: 95 and 105, over e4m3 keys 117 and 128). Where a
// CTA has a few tiles only, the two are close: one canvas over 2304 keys 23.8 and
// 22.2, draft trees of 504 rows 31.7 and 30.4. head_dim above 128 leaves TMEM and
// shared memory for one. The lengths are device data, so the rule goes by the
// batch's average.
Plan make_plan(const dg_kv_cache& c, const dg_kv_batch& b, int q_heads) {
  Plan p;
  p.dp = c.head_dim <= 64 ? 64 : c.head_dim <= 128 ? 128 : 256;
  const int64_t rows = (int64_t)b.tokens * (q_heads / c.kv_heads);
  p.nt = p.dp <= 128 && rows > 128ll * b.batch ? 2 : 1;
  p.rows = (int)std::min<int64_t>(128 * p.nt, (rows + 7) / 8 * 8);
  const size_t pieces = 2 * (size_t)kMaxCtas * p.rows;
  p.o = 0;
  p.ml = al(pieces * p.dp * 4);
  p.open = p.ml + al(pieces * 8);
  p.total = p.open + al(sizeof(Open) * kMaxCtas);
  return p;
}

template <class S>
cudaError_t launch(Args a, int dev, int ctas, cudaStream_t s) {
  // TMA copies take runs of rows that lie together: a power of two that divides
  // page_size, at least 8 (one swizzle pattern, and the exponents' 8 bytes). Rows
  // one by one instead: long sequence 147 us for 95, prompt 376 for 327
  const dg_kv_cache& c = a.w.c;
  a.box = std::min(c.page_size & -c.page_size, S::BN);
  if (a.box < 8 || c.head_dim < 64 || c.pages == 0) a.box = 0;
  if (S::F8 && (reinterpret_cast<uintptr_t>(c.k_exp) | reinterpret_cast<uintptr_t>(c.v_exp)) % 8) a.box = 0;
  alignas(64) CUtensorMap maps[2] = {};
  const uint64_t rows = (uint64_t)c.pages * c.kv_heads * c.page_size;
  if (a.box && (!tc_encode_2d_rows(&maps[0], c.k, c.head_dim, rows, S::F8 ? S::DP : 64, a.box, S::F8) ||
                !tc_encode_2d_rows(&maps[1], c.v, c.head_dim, rows, S::F8 ? S::DP : 64, a.box, S::F8)))
    return cudaErrorInvalidValue;
  // queries: dimensions (column, head, token); a dimension of one takes any stride.
  // (Row by row: prompt 342 us for 327, one canvas 25.6 for 23.8.)
  const int64_t hs = a.q_heads > 1 ? a.q_hs : c.head_dim, ts = a.w.b.tokens > 1 ? a.q_ts : a.q_heads * hs;
  a.q_box = a.G <= 32 && !(a.G & (a.G - 1)) && c.head_dim >= 64 && hs > 0 && ts > 0 && hs < (1ll << 38) && ts < (1ll << 38);
  alignas(64) CUtensorMap q_map = {};
  if (a.q_box) {
    const uint64_t dims[3] = {(uint64_t)c.head_dim, (uint64_t)a.q_heads, (uint64_t)a.w.b.tokens};
    const uint64_t strides[2] = {2 * (uint64_t)hs, 2 * (uint64_t)ts};
    const uint32_t box[3] = {64, (uint32_t)a.G, 32 / (uint32_t)a.G};
    if (!tc_encode_3d_bf16(&q_map, a.q, dims, strides, box)) return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaSuccess;
  static std::atomic<uint64_t> ready{0};                // devices whose kernel may take this much shared memory
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(k_attend<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  k_attend<S><<<ctas, S::THREADS, S::SMEM, s>>>(a, maps[0], maps[1], q_map);
  if ((e = cudaGetLastError()) != cudaSuccess || ctas == 1) return e;
  // the join's launch overlaps the kernel's end; it waits for it on the device
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // no more than ctas - 1 items are cut, whatever the lengths; as many blocks as fit at once
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(6ll * ctas, (int64_t)(ctas - 1) * ((a.rows + 7) / 8)));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_join<S>, a, ctas);
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
  if (kv_check(cache, batch)) return 0;
  if (q_heads < 1 || q_heads % cache->kv_heads) {
    fail(DG_EINVAL, "q_heads must be a multiple of kv_heads");
    return 0;
  }
  if ((int64_t)batch->tokens * q_heads > (1 << 30)) {
    fail(DG_EUNSUPPORTED, "tokens x q_heads must be at most 2^30");
    return 0;
  }
  return attn::make_plan(*cache, *batch, q_heads).total;
}

extern "C" int dg_cache_attention_inject_stall(int64_t wait_limit_ns, int32_t stall) {
  if (wait_limit_ns < 0 || wait_limit_ns > 60ll * 1000000000ll || stall < 0)
    return fail(DG_EINVAL, "wait limit must lie in [0, 60 s] and stall be >= 0");
  attn::wait_ns = wait_limit_ns ? (unsigned long long)wait_limit_ns : attn::kWaitNs;
  attn::stall = (uint32_t)stall;
  return DG_OK;
}

extern "C" int dg_cache_attention(const dg_kv_cache* cache, const dg_kv_batch* batch, int32_t q_heads,
                                  const void* q, int64_t q_ts, int64_t q_hs, float scale, int32_t mask,
                                  const uint32_t* tree_mask, int32_t mask_words, void* out, float* lse,
                                  void* scratch, size_t scratch_bytes, void* stream) {
  using namespace attn;
  int rc = kv_check(cache, batch);
  if (rc) return rc;
  if (q_heads < 1 || q_heads % cache->kv_heads) return fail(DG_EINVAL, "q_heads must be a multiple of kv_heads");
  if (!(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f)) return fail(DG_EINVAL, "scale must be positive and finite");
  if (mask < DG_MASK_FULL || mask > DG_MASK_TREE) return fail(DG_EINVAL, "mask must be one of DG_MASK_*");
  if (mask == DG_MASK_TREE && (mask_words < 0 || (mask_words && !tree_mask)))
    return fail(DG_EINVAL, "DG_MASK_TREE needs tree_mask and mask_words >= 0");
  if (batch->tokens == 0 || batch->batch == 0) return DG_OK;
  if ((int64_t)batch->tokens * q_heads > (1 << 30)) return fail(DG_EUNSUPPORTED, "tokens x q_heads must be at most 2^30");
  if ((rc = kv_row_args(q, q_ts, q_hs))) return rc;
  if (!out || off16(out)) return fail(DG_EINVAL, "out must be 16-byte aligned and not NULL");
  if (!scratch || reinterpret_cast<uintptr_t>(scratch) % 256) return fail(DG_EINVAL, "scratch must be 256-byte aligned and not NULL");
  const Plan p = make_plan(*cache, *batch, q_heads);
  if (scratch_bytes < p.total) return fail(DG_ENOMEM, "scratch is smaller than dg_cache_attention_scratch_bytes()");
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return kv_launched(e);
  char* sc = static_cast<char*>(scratch);
  const uint32_t G = (uint32_t)(q_heads / cache->kv_heads), ps = (uint32_t)cache->page_size;
  // r / n for r < 2^31: 2^log >= n, the multiplier rounded up
  auto log_of = [](uint32_t n) { int log = 0; while ((1ull << log) < n) ++log; return log; };
  auto mul_of = [&](uint32_t n) { return (uint32_t)(((1ull << (31 + log_of(n))) + n - 1) / n); };
  const Args a{{*cache, *batch}, static_cast<const __nv_bfloat16*>(q), q_ts, q_hs, q_heads,
               (int)G, mul_of(G), mul_of(ps), 31 + log_of(G), 31 + log_of(ps), scale * 1.4426950408889634f, mask, tree_mask, mask_words,
               static_cast<__nv_bfloat16*>(out), lse, reinterpret_cast<float*>(sc + p.o),
               reinterpret_cast<float2*>(sc + p.ml), reinterpret_cast<Open*>(sc + p.open), p.rows, 0, 0,
               wait_ns.load(std::memory_order_relaxed), stall.load(std::memory_order_relaxed)};
  const int ctas = std::min(sms, kMaxCtas);
  const bool f8 = cache->format == DG_KV_E4M3;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto go = [&](auto dp, auto nt) {
    constexpr int DP = decltype(dp)::value, NT = decltype(nt)::value;
    return f8 ? launch<Shape<DP, NT, true>>(a, dev, ctas, s) : launch<Shape<DP, NT, false>>(a, dev, ctas, s);
  };
  using std::integral_constant;
  const integral_constant<int, 1> one;
  const integral_constant<int, 2> two;
  if (p.dp == 256) e = go(integral_constant<int, 256>(), one);
  else if (p.dp == 128) e = p.nt == 2 ? go(integral_constant<int, 128>(), two) : go(integral_constant<int, 128>(), one);
  else e = p.nt == 2 ? go(integral_constant<int, 64>(), two) : go(integral_constant<int, 64>(), one);
  return kv_launched(e);
}

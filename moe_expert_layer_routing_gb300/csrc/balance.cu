// Router forward (top-K selection) with the load-balance and z losses, and the losses' gradient.
//
//   p_t = softmax(l_t) over all E logits,  lse_t = log sum exp l_t
//   sequences s of n_s tokens, n = sum_s n_s,  c_se = slots of s routed to e,  P_se = sum_{t in s} p_te
//   L_bal = alpha sum_s (n_s / n) sum_e (E c_se / (K n_s)) (P_se / n_s)
//   L_z   = beta / n sum_t lse_t^2
//   dL_bal / dl_tj = alpha E / (K n n_s) p_tj (c_sj - sum_e c_se p_te),   dL_z / dl_tj = 2 beta / n lse_t p_tj
//
// The counts are constants of the gradient.  A logit of -inf is a masked expert (p = 0); a token with none
// left has p = 0, lse = -inf and no gradient.  NaN and +inf reach the token's scores and the losses.
//
// Work split: the tokens are cut at every multiple of C (a chunk) and at every sequence boundary.  Walking
// along the tokens, each step enters the next chunk or the next sequence, so the piece (chunk c, sequence i)
// has the number c + i of its own, at most chunks + sequences of them, and one CTA per number finds its piece
// by a binary search over the offsets.  No CTA's tokens lie in two sequences: its column sums of p and its
// counts are one partial row, which a second kernel adds per sequence in a fixed order.
//
// The gradient is bound by HBM: 131072 x 256 with `add` moves 403 MB, 59 us at the measured copy rate; measured 62.4 us
// (6.5 TB/s).  The forward reads 34 MB at 65536 x 128 (5.6 us) and takes 23 us with the losses (top-8), 10 us with the ids
// given, and 5 us for the reduction, whose chain of dependent steps is all latency.  It is bound by the selection: about
// 230 warp instructions a token, half of them minima, maxima and logic on the half-rate ALU pipe.  Neither that pipe (busy
// 48% of the time) nor the issue slots (61%) are full: with 80 registers three blocks are resident, 29% of an SM's warps,
// and the dependent steps of a token's merges wait for one another.  Top-16 and top-32 in rounds: 56 and 137 us a call.
//
// Exponentials and quotients are the approximate instructions (2^-22 of the value): scores, sums and losses come out 6e-8
// to 7e-8 from float64, where expf and a division give 5e-8 to 6e-8.
#include <cuda_runtime.h>

#include <algorithm>

#include "moebwd_internal.h"
#include "mx_device.cuh"
#include "ptx.cuh"

namespace moebwd {

constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalStages = 2, kBalBwdStages = 2;

struct BalanceArgs {
  const float* logits;
  int64_t ld;
  int T, K, E;
  const int32_t* off;  // [S + 1] sequence offsets, or null: one sequence of all T tokens
  int S, C;            // sequences; tokens per chunk
  int pieces;          // chunks + S + 1: numbers c + i of the pieces (padding before, S sequences, padding behind)
  float alpha, beta;
  // forward
  int mode, renorm;
  float* scores;
  int32_t* ids;           // written by the top-K, else read
  float* lse;             // [T]
  int32_t* part_c;        // [pieces][E]
  float* part_p;          // [pieces][E]
  float* part_z;          // [pieces]
  float* part_l;          // [S][column tiles + 1]
  unsigned* ticket;
  int32_t* counts;        // [S][E]
  float* prob_sum;        // [S][E]
  float* loss;            // [2]
  int32_t* status;
  // backward
  const float* dloss;     // [2] or null (ones)
  const float* add;       // [T, E] or null
  int64_t ld_add;
  float* dlogits;
};

// Start of segment i of the S + 2: padding before the sequences, the sequences, padding behind them.
__device__ __forceinline__ int seg_start(const BalanceArgs& a, int i) {
  if (i == 0) return 0;
  if (i > a.S + 1) return a.T;
  if (!a.off) return i == 1 ? 0 : a.T;
  return min(max(a.off[i - 1], 0), a.T);
}

// Segment and tokens [lo, hi) of piece p; false when the piece is empty.  Every warp finds them with its 32 lanes, in two
// rounds up to 1023 sequences (a binary search by every thread: gradient over 61 sequences 63.6 instead of 62.4 us).
__device__ __forceinline__ bool find_piece(const BalanceArgs& a, int p, int& seg, int& lo, int& hi) {
  int l = 0, h = a.S + 1;  // the last segment i whose first piece, start / C + i, is not behind p
  while (l < h) {
    const int step = (h - l + 31) >> 5, m = l + ((int)(threadIdx.x & 31) + 1) * step;
    const int c = __popc(__ballot_sync(0xffffffffu, m <= h && seg_start(a, m) / a.C + m <= p));
    h = min(h, l + (c + 1) * step - 1);
    l = min(l + c * step, h);
  }
  seg = l;
  const int64_t c0 = (int64_t)(p - l) * a.C;
  lo = (int)max((int64_t)seg_start(a, l), min(c0, (int64_t)a.T));
  hi = (int)min((int64_t)seg_start(a, l + 1), min(c0 + a.C, (int64_t)a.T));
  return lo < hi;
}

// The status word, from the first block: the offsets have to lie in [0, T] and not decrease.
__device__ __forceinline__ void check_offsets(const BalanceArgs& a) {
  if (!a.status || blockIdx.x) return;
  int bad = 0;
  for (int i = threadIdx.x; a.off && i <= a.S; i += kBalThreads)
    bad |= a.off[i] < 0 || a.off[i] > a.T || (i && a.off[i] < a.off[i - 1]);
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *a.status = bad ? MOE_STATUS_BAD_SEGMENTS : 0;
}

template <int LANES>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ float lane_max(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// e^(x - base): the difference first, so that logits of any magnitude keep it (a row of the type's lowest values
// is a row of equal ones); results below 2^-126 are 0.
__device__ __forceinline__ float exp_from(float x, float base) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"((x - base) * 1.4426950408889634f));
  return e;
}

// Lane sl of a token's LANES lanes holds its logits 4 (LANES j + sl) .. + 3, j < NV, -inf past E.
template <int NV, int LANES, bool VEC>
__device__ __forceinline__ void load_row(const float* row, int E, int sl, bool live, float (&v)[4 * NV]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = 4 * (LANES * j + sl);
    if constexpr (VEC) {
      const float4 f = live && c < E ? *reinterpret_cast<const float4*>(row + c)
                                     : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      v[4 * j] = f.x;
      v[4 * j + 1] = f.y;
      v[4 * j + 2] = f.z;
      v[4 * j + 3] = f.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * j + i] = live && c + i < E ? row[c + i] : -INFINITY;
    }
  }
}

// 32-bit keys in the order of the values: -inf below every number, +inf, then every NaN; -0 equals +0.
// 0 is below them all (no value has it).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  const uint32_t k = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return x != x ? 0xffffffffu : k;
}

// The K selected logits of a token, slot k held by lane k % LANES (as col[k / LANES]; K <= 64 at 32 lanes), by exact
// keys: K rounds of the largest key left, its lowest column, and that one taken out.
template <int NV, int LANES, bool VEC, int SLOTS>
__device__ __noinline__ void topk_exact(const float* row, int E, int K, int sl, bool live, int (&col)[SLOTS]) {
  constexpr int N = 4 * NV;
  uint32_t key[N];
  {
    float v[N];
    load_row<NV, LANES, VEC>(row, E, sl, live, v);
#pragma unroll
    for (int j = 0; j < N; ++j) key[j] = 4 * (LANES * (j >> 2) + sl) + (j & 3) < E ? order_key(v[j]) : 0u;
  }
  for (int r = 0; r < K; ++r) {
    uint32_t g = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) g = max(g, key[j]);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) g = max(g, __shfl_xor_sync(0xffffffffu, g, o));
    int c = 1 << 30;
#pragma unroll
    for (int j = N - 1; j >= 0; --j) c = key[j] == g ? 4 * (LANES * (j >> 2) + sl) + (j & 3) : c;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) c = min(c, __shfl_xor_sync(0xffffffffu, c, o));
#pragma unroll
    for (int j = 0; j < N; ++j) key[j] = c == 4 * (LANES * (j >> 2) + sl) + (j & 3) ? 0u : key[j];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
      if (r == s * LANES + sl) col[s] = c;
  }
}

// The same with unique keys of 32 bits (31 in rounds): a value's leading bits, then its column counted backwards, so
// that the larger key is the value to take and no search for columns follows.  True marks rows that need exact keys all
// the same: values that differ in the dropped bits alone and came out of order, or might have at the end.
//
// Measured at 65536 x 128 with the losses: exact keys with a search per round 42 us, rounds of packed keys 30 us, sorted
// lists 26 us, 24 us with the logits a pass ahead in shared memory and read again after the selection, 23 us with the
// softmax and its column sums in paired arithmetic.
//
// K <= 8 (LIST): a sorted list of the eight largest per lane (a sorting network of 19 comparators in six layers per 8
// values, the fewest there can be: Knuth, The Art of Computer Programming, volume 3, section 5.3.4), then merged with the
// lists of the lanes 1, 2, 4, ... away: max(a_i, b_7-i) holds the eight largest of both and is bitonic, and the twelve
// comparators of Batcher's bitonic merge sort it.  log2(LANES) dependent shuffle steps, all comparators of a level independent.
// K > 8: rounds of one maximum.  "Smaller than the last" is a subtraction: key - m as unsigned is 2^31 or more
// exactly for the keys below m.
__device__ __forceinline__ void sort_desc(uint32_t& a, uint32_t& b) {
  const uint32_t h = max(a, b);
  b = min(a, b);
  a = h;
}
__device__ __forceinline__ void sort8(uint32_t (&a)[8]) {
  sort_desc(a[0], a[2]); sort_desc(a[1], a[3]); sort_desc(a[4], a[6]); sort_desc(a[5], a[7]);
  sort_desc(a[0], a[4]); sort_desc(a[1], a[5]); sort_desc(a[2], a[6]); sort_desc(a[3], a[7]);
  sort_desc(a[0], a[1]); sort_desc(a[2], a[3]); sort_desc(a[4], a[5]); sort_desc(a[6], a[7]);
  sort_desc(a[2], a[4]); sort_desc(a[3], a[5]);
  sort_desc(a[1], a[4]); sort_desc(a[3], a[6]);
  sort_desc(a[1], a[2]); sort_desc(a[3], a[4]); sort_desc(a[5], a[6]);
}
// a bitonic list into descending order
__device__ __forceinline__ void merge8(uint32_t (&a)[8]) {
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) sort_desc(a[i], a[i + d]);
}

template <int NV, int LANES, int SLOTS, bool LIST, typename Logit>
__device__ __forceinline__ bool topk_packed(const float (&v)[4 * NV], Logit logit, int E, int K, int sl, bool live,
                                            int (&col)[SLOTS]) {
  constexpr int N = 4 * NV;
  constexpr int CAP = N * LANES;  // columns
  constexpr uint32_t CM = CAP - 1;
  static_assert((CAP & (CAP - 1)) == 0, "column bits");
  uint32_t key[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int c = 4 * (LANES * (j >> 2) + sl) + (j & 3);
    const int b = __float_as_int(v[j] + 0.f);
    // columns past E hold -inf, behind every logit: they are taken last (K <= E), or in a row with a NaN of negative
    // sign, which is done over
    key[j] = ((uint32_t)(b ^ (b >> 31 | (int)0x80000000)) >> (LIST ? 0 : 1) & ~CM) | (CM - (uint32_t)c);
  }
  uint32_t mk[SLOTS] = {}, next[SLOTS] = {};
  uint32_t last, behind;  // the K-th key, and the largest of this lane's (LIST) or of all below it
  if constexpr (LIST) {
    uint32_t top[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) top[j] = j < N ? key[j] : 0u;
    sort8(top);
#pragma unroll
    for (int g = 8; g < N; g += 8) {
      uint32_t more[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) more[j] = key[g + j];
      sort8(more);
#pragma unroll
      for (int j = 0; j < 8; ++j) top[j] = max(top[j], more[7 - j]);
      merge8(top);
    }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
      uint32_t other[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) other[j] = __shfl_xor_sync(0xffffffffu, top[7 - j], o);
#pragma unroll
      for (int j = 0; j < 8; ++j) top[j] = max(top[j], other[j]);
      merge8(top);
    }
    // slot sl, by the bits of sl
    const uint32_t h0 = sl & 4 ? top[4] : top[0], h1 = sl & 4 ? top[5] : top[1], h2 = sl & 4 ? top[6] : top[2],
                   h3 = sl & 4 ? top[7] : top[3];
    const uint32_t q0 = sl & 2 ? h2 : h0, q1 = sl & 2 ? h3 : h1;
    mk[0] = sl & 1 ? q1 : q0;
    next[0] = __shfl_down_sync(0xffffffffu, mk[0], 1, LANES);
    last = __shfl_sync(0xffffffffu, mk[0], K - 1, LANES);
    // the least last - 1 - key: as unsigned, keys from last on are far above those in the same leading bits, but where
    // last itself has none of them set (a NaN of negative sign): there every key is looked at
    uint32_t below = 0xffffffffu;
#pragma unroll
    for (int j = 0; j < N; j += 2) below = __vimin3_u32(below, last - 1u - key[j], last - 1u - key[j + 1]);
    behind = last <= CM ? last : below <= CM ? last - 1u - below : 0u;
  } else {
    uint32_t m = 0x80000000u;
    last = 0;
    for (int r = 0; r <= K; ++r) {
      uint32_t d = 0;
#pragma unroll
      for (int j = 0; j < N; j += 2) d = __vimax3_u32(d, key[j] - m, key[j + 1] - m);
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) d = max(d, __shfl_xor_sync(0xffffffffu, d, o));
      m = d < 0x80000000u ? 0u : m + d;  // 0: none is left (K = E)
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        if (r == s * LANES + sl) mk[s] = m;
        if (r == s * LANES + sl + 1) next[s] = m;
      }
      if (r == K - 1) last = m;
    }
    behind = m;
  }
  // exact keys of the slot and of the one behind it
  bool odd = false;
  uint32_t ek = 0;  // exact key of slot K - 1, in the lane that holds it
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    const int k = s * LANES + sl;
    col[s] = min((int)(CM - (mk[s] & CM)), E - 1);
    if (live && k < K && (k + 1 == K || (mk[s] ^ next[s]) <= CM)) {  // the same leading bits
      const uint32_t exact = order_key(logit(col[s]));
      if (k + 1 < K)
        odd |= exact < order_key(logit(min((int)(CM - (next[s] & CM)), E - 1)));
      else
        ek = exact;
    }
  }
  // at the end: a value left out may be larger in the dropped bits than the last one taken
  const bool tie = live && behind != 0 && (last ^ behind) <= CM;
  if (__any_sync(0xffffffffu, tie)) {
    ek = __shfl_sync(0xffffffffu, ek, (K - 1) % LANES, LANES);
#pragma unroll
    for (int j = 0; j < N; ++j) odd |= tie && key[j] < last && (key[j] ^ last) <= CM &&
             order_key(logit(min((int)(CM - (key[j] & CM)), E - 1))) > ek;
  }
  return odd;
}

// Selects and writes scores and ids (else reads ids).  One token per LANES lanes.
enum TopK { kIdsGiven = 0, kTopKList = 1, kTopKRounds = 2 };
template <int NV, int LANES, bool VEC, int HOW>
__global__ void __launch_bounds__(kBalThreads, NV <= 4 ? 3 : 1) router_fwd_kernel(const BalanceArgs a) {
  constexpr int SEGS = 32 / LANES, N = 4 * NV;
  constexpr bool TOPK = HOW != kIdsGiven;
  constexpr int SLOTS = LANES == 32 && HOW == kTopKRounds ? 2 : 1;  // slots a lane holds (K <= 64 at 32 lanes)
  // VEC: a ring of kBalStages rows per segment, filled by 16-byte asynchronous copies a pass ahead; then [kBalWarps][E]
  // partial sums of p, [E] counts, [kBalWarps] z
  extern __shared__ float4 ring[];
  float* sm = reinterpret_cast<float*>(ring + (VEC ? kBalStages * NV * kBalThreads : 0));
  int* hist = reinterpret_cast<int*>(sm + kBalWarps * a.E);
  float* zs = sm + (kBalWarps + 1) * a.E;
  pdl_wait();
  pdl_trigger();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, seg = lane / LANES, sl = lane % LANES;
  const bool stats = a.part_p != nullptr;
  check_offsets(a);
  if (stats && blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  int which, lo, hi;
  if (!find_piece(a, blockIdx.x, which, lo, hi)) return;
  if (which == 0 || which == a.S + 1) {  // padding tokens: no slot is used
    for (int64_t i = (int64_t)lo * a.K + threadIdx.x; TOPK && i < (int64_t)hi * a.K; i += kBalThreads) {
      a.ids[i] = -1;
      a.scores[i] = 0.f;
    }
    for (int t = lo + threadIdx.x; a.lse && t < hi; t += kBalThreads) a.lse[t] = -INFINITY;
    return;
  }
  if (stats)
    for (int i = threadIdx.x; i < a.E; i += kBalThreads) hist[i] = 0;
  __syncthreads();
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.f;
  float z = 0.f;
  auto slot = [&](int stage, int j) { return ring + (stage * NV + j) * kBalThreads + threadIdx.x; };
  auto fetch = [&](int t, int stage) {
    if constexpr (VEC) {
      if (t < hi) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = 4 * (LANES * j + sl);
          if (c < a.E) cp_async_16(smem_u32(slot(stage, j)), a.logits + (int64_t)t * a.ld + c);
        }
      }
      cp_async_commit();
    }
  };
#pragma unroll
  for (int s = 0; s < kBalStages - 1; ++s) fetch(lo + (w + s * kBalWarps) * SEGS + seg, s);
  int stage = 0;
  for (int tb = lo + w * SEGS; tb < hi; tb += kBalWarps * SEGS) {
    const int t = tb + seg;
    const bool live = t < hi;
    const float* row = a.logits + (int64_t)t * a.ld;
    float v[N];
    auto read = [&](float (&u)[N]) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const float4 f = live && 4 * (LANES * j + sl) < a.E ? *slot(stage, j)
                                                            : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        u[4 * j] = f.x;
        u[4 * j + 1] = f.y;
        u[4 * j + 2] = f.z;
        u[4 * j + 3] = f.w;
      }
    };
    if constexpr (VEC) {
      __syncwarp();  // the slot filled next was read by the whole segment
      fetch(t + (kBalStages - 1) * kBalWarps * SEGS, stage == 0 ? kBalStages - 1 : stage - 1);
      cp_async_wait<kBalStages - 1>();
      __syncwarp();
      read(v);
    } else {
      load_row<NV, LANES, VEC>(row, a.E, sl, live, v);
    }
    // one logit of the row: from the lane that copied it
    auto logit = [&](int c) {
      if constexpr (VEC)
        return reinterpret_cast<const float*>(ring + (stage * NV + c / (4 * LANES)) * kBalThreads + threadIdx.x - sl +
                                              (c >> 2) % LANES)[c & 3];
      else
        return row[c];
    };
    int col[SLOTS];
    bool odd = false;
    // the tokens that need exact keys, done over
    auto settle = [&]() {
      const unsigned which_lanes = __ballot_sync(0xffffffffu, odd);
      if (!which_lanes) return;
      int ex[SLOTS];
      topk_exact<NV, LANES, VEC, SLOTS>(row, a.E, a.K, sl, live, ex);
      const unsigned mine = (LANES == 32 ? 0xffffffffu : ((1u << (LANES & 31)) - 1u)) << (LANES * seg);
      if (which_lanes & mine) {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) col[s] = ex[s];
      }
    };
    float m = -INFINITY;  // the row's maximum
    if constexpr (TOPK) {
      odd = topk_packed<NV, LANES, SLOTS, HOW == kTopKList>(v, logit, a.E, a.K, sl, live, col);
      settle();
      if (live && sl == 0) m = logit(col[0]);
      m = __shfl_sync(0xffffffffu, m, 0, LANES);
      if constexpr (VEC) {  // read again rather than kept through the selection: registers
        asm volatile("" ::: "memory");
        read(v);
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) m = fmaxf(m, v[j]);
      m = lane_max<LANES>(m);
    }
    const float base = m == -INFINITY ? 0.f : m;
    const uint64_t nbase = f2_splat(-base), l2e = f2_splat(1.4426950408889634f);
    uint64_t total2 = f2_splat(0.f);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      float x0, x1;
      f2_unpack(f2_mul(f2_add(f2_pack(v[j], v[j + 1]), nbase), l2e), x0, x1);
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v[j]) : "f"(x0));
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v[j + 1]) : "f"(x1));
      total2 = f2_add(total2, f2_pack(v[j], v[j + 1]));
    }
    float total, total_hi;
    f2_unpack(total2, total, total_hi);
    total = lane_sum<LANES>(total + total_hi);
    const float inv = total != 0.f ? __fdividef(1.f, total) : 0.f;  // 0: every expert masked (or no token here)
    const float lse = base + logf(total);
    const uint64_t inv2 = f2_splat(inv);
#pragma unroll
    for (int j = 0; j < N; j += 2)
      f2_unpack(f2_fma(f2_pack(v[j], v[j + 1]), inv2, f2_pack(acc[j], acc[j + 1])), acc[j], acc[j + 1]);
    if (sl == 0 && live) {
      if (a.lse) a.lse[t] = lse;
      if (total != 0.f) z = fmaf(lse, lse, z);
    }
    if constexpr (TOPK) {
      odd = total != total;  // NaN or +inf among the logits
      settle();
      float x[SLOTS], e[SLOTS], sum = 0.f;
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        x[s] = live && s * LANES + sl < a.K ? logit(col[s]) : -INFINITY;
        if (x[s] == -INFINITY) col[s] = -1;  // a masked expert takes no slot
        e[s] = exp_from(x[s], base);
        sum += e[s];
      }
      sum = lane_sum<LANES>(sum);
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        const int k = s * LANES + sl;
        if (live && k < a.K) {
          float sc = 0.f;
          if (col[s] >= 0)
            sc = a.mode == MOE_ROUTER_TOPK ? x[s]
                 : a.mode == MOE_ROUTER_TOPK_OVER_SOFTMAX && !a.renorm ? e[s] * inv
                                                                       : __fdividef(e[s], sum);
          a.scores[(int64_t)t * a.K + k] = sc;
          a.ids[(int64_t)t * a.K + k] = col[s];
          if (stats && col[s] >= 0) atomicAdd(&hist[col[s]], 1);  // integers: any order gives the same counts
        }
      }
    } else {
      for (int k = sl; live && k < a.K; k += LANES) {
        const int id = a.ids[(int64_t)t * a.K + k];
        if (id >= 0 && id < a.E) atomicAdd(&hist[id], 1);
      }
    }
    stage = stage + 1 == kBalStages ? 0 : stage + 1;
  }
  if (!stats) return;
  // the warp's tokens, then the warps, in a fixed order
#pragma unroll
  for (int j = 0; j < N; ++j) {
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
    const int c = 4 * (LANES * (j >> 2) + sl) + (j & 3);
    if (seg == 0 && c < a.E) sm[w * a.E + c] = acc[j];
  }
  z = lane_sum<32>(z);
  if (lane == 0) zs[w] = z;
  __syncthreads();
  const int64_t row = (int64_t)blockIdx.x * a.E;
  for (int i = threadIdx.x; i < a.E; i += kBalThreads) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kBalWarps; ++k) s += sm[k * a.E + i];
    a.part_p[row + i] = s;
    a.part_c[row + i] = hist[i];
  }
  if (threadIdx.x == 0) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kBalWarps; ++k) s += zs[k];
    a.part_z[blockIdx.x] = s;
  }
}

// counts and prob_sum of sequence blockIdx.x, columns blockIdx.y * 32 .. + 31, from its pieces; each block's
// share of the losses, which the block that comes last adds up in a fixed order.
__global__ void __launch_bounds__(kBalThreads) balance_reduce_kernel(const BalanceArgs a) {
  __shared__ float sp[kBalWarps][32], sz[kBalWarps];
  __shared__ int sc[kBalWarps][32];
  __shared__ bool last;
  pdl_wait();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.x, col = blockIdx.y * 32 + lane, tiles = gridDim.y;
  const int b0 = seg_start(a, s + 1), b1 = seg_start(a, s + 2);
  const int p0 = b0 / a.C + s + 1, p1 = b1 > b0 ? min((b1 - 1) / a.C + s + 2, a.pieces) : p0;
  float p = 0.f, z = 0.f;
  int c = 0;
  if (col < a.E)
    for (int i = p0 + w; i < p1; i += kBalWarps) {
      p += a.part_p[(int64_t)i * a.E + col];
      c += a.part_c[(int64_t)i * a.E + col];
    }
  if (blockIdx.y == 0)
    for (int i = p0 + (int)threadIdx.x; i < p1; i += kBalThreads) z += a.part_z[i];
  sp[w][lane] = p;
  sc[w][lane] = c;
  z = lane_sum<32>(z);
  if (lane == 0) sz[w] = z;
  __syncthreads();
  if (w == 0) {
    p = 0.f;
    c = 0;
    z = 0.f;
#pragma unroll
    for (int k = 0; k < kBalWarps; ++k) {
      p += sp[k][lane];
      c += sc[k][lane];
      z += sz[k];
    }
    float l = 0.f;
    if (col < a.E) {
      a.counts[(int64_t)s * a.E + col] = c;
      a.prob_sum[(int64_t)s * a.E + col] = p;
      l = b1 > b0 ? (float)c * p / (float)(b1 - b0) : 0.f;
    }
    l = lane_sum<32>(l);
    if (lane == 0) {
      a.part_l[(int64_t)s * (tiles + 1) + blockIdx.y] = l;
      if (blockIdx.y == 0) a.part_l[(int64_t)s * (tiles + 1) + tiles] = z;
      __threadfence();
      last = atomicAdd(a.ticket, 1u) == gridDim.x * gridDim.y - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  float lb = 0.f, lz = 0.f;
  for (int i = threadIdx.x; i < a.S * (tiles + 1); i += kBalThreads) {
    const float v = __ldcg(a.part_l + i);
    if (i % (tiles + 1) == tiles)
      lz += v;
    else
      lb += v;
  }
  lb = lane_sum<32>(lb);
  lz = lane_sum<32>(lz);
  __syncthreads();
  if (lane == 0) {
    sp[0][w] = lb;
    sz[w] = lz;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    lb = lz = 0.f;
    for (int k = 0; k < kBalWarps; ++k) {
      lb += sp[0][k];
      lz += sz[k];
    }
    const float n = (float)max(seg_start(a, a.S + 1) - seg_start(a, 1), 1);
    a.loss[0] = a.alpha * (float)a.E / ((float)a.K * n) * lb;
    a.loss[1] = a.beta != 0.f ? a.beta / n * lz : 0.f;  // (lse^2 may be infinite)
  }
}

template <int NV, int LANES, bool VEC>
__global__ void __launch_bounds__(kBalThreads) balance_bwd_kernel(const BalanceArgs a) {
  constexpr int SEGS = 32 / LANES, N = 4 * NV;
  pdl_wait();
  pdl_trigger();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, seg = lane / LANES, sl = lane % LANES;
  check_offsets(a);
  int which, lo, hi;
  if (!find_piece(a, blockIdx.x, which, lo, hi)) return;
  const bool pad = which == 0 || which == a.S + 1;
  const float n = (float)max(seg_start(a, a.S + 1) - seg_start(a, 1), 1);
  const float n_s = (float)(seg_start(a, which + 1) - seg_start(a, which));
  const float wb = (a.dloss ? a.dloss[0] : 1.f) * a.alpha * (float)a.E / ((float)a.K * n * n_s);
  const float wz = (a.dloss ? a.dloss[1] : 1.f) * 2.f * a.beta / n;
  float cnt[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int c = 4 * (LANES * (j >> 2) + sl) + (j & 3);
    cnt[j] = !pad && c < a.E ? (float)a.counts[(int64_t)(which - 1) * a.E + c] : 0.f;
  }
  // VEC: logits and `add` come through a ring of rows by 16-byte asynchronous copies, each lane's own
  extern __shared__ float4 ring[];
  auto slot = [&](int stage, int tensor, int j) { return ring + ((stage * 2 + tensor) * NV + j) * kBalThreads + threadIdx.x; };
  auto fetch = [&](int t, int stage) {
    if constexpr (VEC) {
      if (t < hi) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = 4 * (LANES * j + sl);
          if (c < a.E) {
            if (!pad) cp_async_16(smem_u32(slot(stage, 0, j)), a.logits + (int64_t)t * a.ld + c);
            if (a.add) cp_async_16(smem_u32(slot(stage, 1, j)), a.add + (int64_t)t * a.ld_add + c);
          }
        }
      }
      cp_async_commit();
    }
  };
#pragma unroll
  for (int s = 0; s < kBalBwdStages - 1; ++s) fetch(lo + (w + s * kBalWarps) * SEGS + seg, s);
  float ahead = -INFINITY;  // lse of the next pass's token
  {
    const int t = lo + w * SEGS + seg;
    if (t < hi && !pad) ahead = a.lse[t];
  }
  int stage = 0;
  for (int tb = lo + w * SEGS; tb < hi; tb += kBalWarps * SEGS) {
    const int t = tb + seg;
    const bool live = t < hi;
    float v[N], b[N];
    const float lse = ahead;
    {
      const int n = t + kBalWarps * SEGS;
      ahead = n < hi && !pad ? a.lse[n] : -INFINITY;
    }
    if constexpr (VEC) {
      fetch(t + (kBalBwdStages - 1) * kBalWarps * SEGS, stage == 0 ? kBalBwdStages - 1 : stage - 1);
      cp_async_wait<kBalBwdStages - 1>();
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const bool in = live && 4 * (LANES * j + sl) < a.E;
        const float4 f = in && !pad ? *slot(stage, 0, j) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        const float4 g = in && a.add ? *slot(stage, 1, j) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[4 * j] = f.x; v[4 * j + 1] = f.y; v[4 * j + 2] = f.z; v[4 * j + 3] = f.w;
        b[4 * j] = g.x; b[4 * j + 1] = g.y; b[4 * j + 2] = g.z; b[4 * j + 3] = g.w;
      }
      stage = stage + 1 == kBalBwdStages ? 0 : stage + 1;
    } else {
      load_row<NV, LANES, VEC>(a.logits + (int64_t)t * a.ld, a.E, sl, live && !pad, v);
      if (a.add) {
        load_row<NV, LANES, VEC>(a.add + (int64_t)t * a.ld_add, a.E, sl, live, b);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) b[j] = 0.f;
      }
    }
    const bool none = lse == -INFINITY;  // nothing left by the mask, or a padding token
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = none ? 0.f : exp_from(v[j], lse);
    // p = e^(l - lse) sums to 1 within lse's rounding, 2^-24 |lse|; where that shows, p is divided by its sum (finite
    // masks in a whole row lose all of lse's fraction)
    if (__any_sync(0xffffffffu, !none && !(fabsf(lse) < 16.f))) {
      float total = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) total += v[j];
      total = lane_sum<LANES>(total);
      const float inv = none ? 0.f : __fdividef(1.f, total);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] *= inv;
    }
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) dot = fmaf(cnt[j], v[j], dot);
    dot = lane_sum<LANES>(dot);
    const float wt = none ? 0.f : wb, zt = none ? 0.f : wz * lse;  // (the loss's gradient may be infinite)
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = fmaf(v[j], fmaf(wt, cnt[j] - dot, zt), b[j]);
    if (!live) continue;
    float* out = a.dlogits + (int64_t)t * a.E;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 4 * (LANES * j + sl);
      if constexpr (VEC) {
        if (c < a.E) *reinterpret_cast<float4*>(out + c) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i < a.E) out[c + i] = v[4 * j + i];
      }
    }
  }
}

// Lanes per token: 8 for up to 128 experts and K <= 8, 16 for up to 256 and K <= 16, else a warp (16 logits a lane;
// 32 above 512 experts).
static int bal_lanes(int K, int E) { return E <= 128 && K <= 8 ? 8 : E <= 256 && K <= 16 ? 16 : 32; }
// The gradient keeps no slots.
static int bal_bwd_lanes(int E) { return E <= 128 ? 8 : E <= 256 ? 16 : 32; }

// Tokens per chunk, in passes of a CTA's warps.  Forward: one pass, more where the CTAs would not all be resident at
// once (three on an SM): a CTA leaves E partial sums.  Gradient: two passes, more where the CTAs would be over three
// times that (131072 x 256: 63.8 us, 66.7 us resident at once).  8 blocks of each wave on 152 SMs (24 of three) are left
// for what cutting at sequence boundaries adds: there are up to S + 1 more pieces than chunks.
static int64_t bal_passes(int T, int lanes, int64_t most) {
  const int step = kBalThreads / lanes;
  return std::max<int64_t>(1, (((int64_t)T + step - 1) / step + most - 1) / most);  // (no tokens: a chunk has a size)
}
static int bal_chunk(int T, int lanes) { return (int)bal_passes(T, lanes, 3 * 152 - 8) * (kBalThreads / lanes); }
static int bal_bwd_chunk(int T, int lanes) {
  return (int)std::max(bal_passes(T, lanes, 9 * 152 - 24), std::min<int64_t>(2, bal_passes(T, lanes, 3 * 152 - 8))) *
         (kBalThreads / lanes);
}

static int bal_pieces(int T, int C, int S) { return (int)(((int64_t)T + C - 1) / C) + S + 1; }

struct BalLayout {
  size_t c, p, z, l, ticket, total;
  int C, pieces;
};

static BalLayout bal_layout(int T, int K, int E, int S) {
  BalLayout L{};
  L.C = bal_chunk(T, bal_lanes(K, E));
  L.pieces = bal_pieces(T, L.C, S);
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t at = off;
    off = align_up(off + n, 256);
    return at;
  };
  L.c = take(sizeof(int32_t) * (size_t)L.pieces * E);
  L.p = take(sizeof(float) * (size_t)L.pieces * E);
  L.z = take(sizeof(float) * (size_t)L.pieces);
  L.l = take(sizeof(float) * (size_t)S * ((E + 31) / 32 + 1));
  L.ticket = take(sizeof(unsigned));
  L.total = off;
  return L;
}

static int bal_check(const char* who, int T, int K, int E, int S) {
  if (T < 0 || K <= 0 || E <= 0 || K > E || S < 1) return fail(MOE_ERR_INVALID, "%s: bad sizes (need 1 <= K <= E, T >= 0, num_seq >= 1)", who);
  if (E > kMaxExperts || K > 64) return fail(MOE_ERR_UNSUPPORTED, "%s: E above %d or K above 64", who, kMaxExperts);
  if (T > INT32_MAX - (1 << 20) || S > (1 << 20)) return fail(MOE_ERR_UNSUPPORTED, "%s: too many tokens or sequences", who);
  return MOE_OK;
}

typedef void (*BalKernel)(const BalanceArgs);

// Instances by lanes per token and float4 groups a lane; only what bal_lanes and bal_bwd_lanes ask for.
template <bool VEC>
static BalKernel fwd_kernel(int lanes, int nv, int how) {
  if (how == kTopKList) {
    if (lanes == 8)
      return nv <= 1   ? router_fwd_kernel<1, 8, VEC, kTopKList>
             : nv <= 2 ? router_fwd_kernel<2, 8, VEC, kTopKList>
                       : router_fwd_kernel<4, 8, VEC, kTopKList>;
    if (lanes == 16) return router_fwd_kernel<4, 16, VEC, kTopKList>;  // above 128 experts
    return nv <= 4 ? router_fwd_kernel<4, 32, VEC, kTopKList> : router_fwd_kernel<8, 32, VEC, kTopKList>;
  }
  if (how == kTopKRounds) {
    if (lanes == 16)
      return nv <= 1   ? router_fwd_kernel<1, 16, VEC, kTopKRounds>
             : nv <= 2 ? router_fwd_kernel<2, 16, VEC, kTopKRounds>
                       : router_fwd_kernel<4, 16, VEC, kTopKRounds>;
    return nv <= 1   ? router_fwd_kernel<1, 32, VEC, kTopKRounds>
           : nv <= 2 ? router_fwd_kernel<2, 32, VEC, kTopKRounds>
           : nv <= 4 ? router_fwd_kernel<4, 32, VEC, kTopKRounds>
                     : router_fwd_kernel<8, 32, VEC, kTopKRounds>;
  }
  if (lanes == 8)
    return nv <= 1   ? router_fwd_kernel<1, 8, VEC, kIdsGiven>
           : nv <= 2 ? router_fwd_kernel<2, 8, VEC, kIdsGiven>
                     : router_fwd_kernel<4, 8, VEC, kIdsGiven>;
  if (lanes == 16)
    return nv <= 1   ? router_fwd_kernel<1, 16, VEC, kIdsGiven>
           : nv <= 2 ? router_fwd_kernel<2, 16, VEC, kIdsGiven>
                     : router_fwd_kernel<4, 16, VEC, kIdsGiven>;
  return nv <= 1   ? router_fwd_kernel<1, 32, VEC, kIdsGiven>
         : nv <= 2 ? router_fwd_kernel<2, 32, VEC, kIdsGiven>
         : nv <= 4 ? router_fwd_kernel<4, 32, VEC, kIdsGiven>
                   : router_fwd_kernel<8, 32, VEC, kIdsGiven>;
}

template <bool VEC>
static BalKernel bwd_kernel(int lanes, int nv) {
  if (lanes == 8)
    return nv <= 1   ? balance_bwd_kernel<1, 8, VEC>
           : nv <= 2 ? balance_bwd_kernel<2, 8, VEC>
                     : balance_bwd_kernel<4, 8, VEC>;
  return lanes == 16 ? balance_bwd_kernel<4, 16, VEC> : nv <= 4 ? balance_bwd_kernel<4, 32, VEC> : balance_bwd_kernel<8, 32, VEC>;
}

// Both forward entry points: the top-K (scores given) or the caller's ids, with or without the losses.
static int launch_router(BalanceArgs a, bool topk, bool stats, const BalLayout& L, void* workspace, cudaStream_t st) {
  char* ws = static_cast<char*>(workspace);
  a.C = L.C;
  a.pieces = L.pieces;
  if (stats) {
    a.part_c = reinterpret_cast<int32_t*>(ws + L.c);
    a.part_p = reinterpret_cast<float*>(ws + L.p);
    a.part_z = reinterpret_cast<float*>(ws + L.z);
    a.part_l = reinterpret_cast<float*>(ws + L.l);
    a.ticket = reinterpret_cast<unsigned*>(ws + L.ticket);
  }
  const int lanes = bal_lanes(a.K, a.E), nv = (a.E + 4 * lanes - 1) / (4 * lanes);
  const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0;
  const int groups = nv <= 1 ? 1 : nv <= 2 ? 2 : nv <= 4 ? 4 : 8;
  const size_t smem = sizeof(float) * ((size_t)(kBalWarps + 1) * a.E + kBalWarps) +
                      (vec ? sizeof(float4) * kBalStages * groups * kBalThreads : 0);
  const int how = !topk ? kIdsGiven : a.K <= 8 ? kTopKList : kTopKRounds;
  const BalKernel kern = vec ? fwd_kernel<true>(lanes, groups, how) : fwd_kernel<false>(lanes, groups, how);
  const int rc = launch_pdl(kern, dim3(a.pieces), dim3(kBalThreads), smem, st, "router_fwd", a);
  if (rc || !stats) return rc;
  return launch_pdl(balance_reduce_kernel, dim3(a.S, (a.E + 31) / 32), dim3(kBalThreads), 0, st, "balance_reduce", a);
}

// T = 0: no counts, no probabilities, no loss
static int balance_empty(int E, int S, int32_t* counts, float* prob_sum, float* loss, cudaStream_t st) {
  int rc = cuda_check(cudaMemsetAsync(counts, 0, sizeof(int32_t) * (size_t)S * E, st), "memset counts");
  if (!rc) rc = cuda_check(cudaMemsetAsync(prob_sum, 0, sizeof(float) * (size_t)S * E, st), "memset prob_sum");
  if (!rc) rc = cuda_check(cudaMemsetAsync(loss, 0, 2 * sizeof(float), st), "memset loss");
  return rc;
}

}  // namespace moebwd

using namespace moebwd;

extern "C" size_t moe_balance_workspace_size(int T, int K, int E, int num_seq) {
  if (bal_check("moe_balance_workspace_size", T, K, E, num_seq) != MOE_OK) return 0;
  return bal_layout(T, K, E, num_seq).total;
}

static int router_entry(const char* who, bool topk, int mode, int renorm, const float* logits, int64_t ld_logits, int T,
                        int K, int E, const int32_t* seg_offsets, int num_seq, float alpha, float beta, float* scores,
                        int32_t* ids, float* lse, int32_t* counts, float* prob_sum, float* loss, int32_t* status_dev,
                        void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  clear_error();
  int rc = bal_check(who, T, K, E, num_seq);
  if (rc) return rc;
  if (topk && mode != MOE_ROUTER_SOFTMAX_OVER_TOPK && mode != MOE_ROUTER_TOPK_OVER_SOFTMAX && mode != MOE_ROUTER_TOPK)
    return fail(MOE_ERR_INVALID, "%s: bad mode", who);
  if (!seg_offsets && num_seq != 1) return fail(MOE_ERR_INVALID, "%s: several sequences need seg_offsets", who);
  const int given = (counts != nullptr) + (prob_sum != nullptr) + (loss != nullptr);
  if (given != 3 && (given != 0 || !topk))
    return fail(MOE_ERR_INVALID, "%s: counts, prob_sum and loss come together", who);
  const bool stats = given == 3;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0 && status_dev && (rc = cuda_check(cudaMemsetAsync(status_dev, 0, sizeof(int32_t), st), "memset status"))) return rc;
  if (T == 0) return stats ? balance_empty(E, num_seq, counts, prob_sum, loss, st) : MOE_OK;
  if (!logits || !ids || (topk && !scores)) return fail(MOE_ERR_INVALID, "%s: null pointer", who);
  if (ld_logits < E) return fail(MOE_ERR_INVALID, "%s: row stride below E", who);
  for (const void* p : {static_cast<const void*>(logits), static_cast<const void*>(seg_offsets),
                        static_cast<const void*>(scores), static_cast<const void*>(ids), static_cast<const void*>(lse),
                        static_cast<const void*>(counts), static_cast<const void*>(prob_sum),
                        static_cast<const void*>(loss), static_cast<const void*>(status_dev)})
    if (reinterpret_cast<uintptr_t>(p) & 3) return fail(MOE_ERR_INVALID, "%s: tensors must be 4-byte aligned", who);
  const BalLayout L = bal_layout(T, K, E, num_seq);
  if (stats) {
    if (!workspace) return fail(MOE_ERR_INVALID, "%s: null pointer", who);
    if (reinterpret_cast<uintptr_t>(workspace) & 255)
      return fail(MOE_ERR_INVALID, "%s: workspace must be 256-byte aligned", who);
    if (workspace_bytes < L.total)
      return fail(MOE_ERR_INVALID, "%s: workspace too small (%zu < %zu)", who, workspace_bytes, L.total);
  }
  BalanceArgs a{};
  a.logits = logits;
  a.ld = ld_logits;
  a.T = T;
  a.K = K;
  a.E = E;
  a.off = seg_offsets;
  a.S = num_seq;
  a.alpha = alpha;
  a.beta = beta;
  a.mode = mode;
  a.renorm = renorm;
  a.scores = scores;
  a.ids = ids;
  a.lse = lse;
  a.counts = counts;
  a.prob_sum = prob_sum;
  a.loss = loss;
  a.status = status_dev;
  return launch_router(a, topk, stats, L, workspace, st);
}

extern "C" int moe_router_fwd(int mode, int renorm, const float* logits, int64_t ld_logits, int T, int K, int E,
                              const int32_t* seg_offsets, int num_seq, float alpha, float beta, float* scores,
                              int32_t* ids, float* lse, int32_t* counts, float* prob_sum, float* loss,
                              int32_t* status_dev, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  return router_entry("moe_router_fwd", true, mode, renorm, logits, ld_logits, T, K, E, seg_offsets, num_seq, alpha,
                      beta, scores, ids, lse, counts, prob_sum, loss, status_dev, workspace, workspace_bytes, stream);
}

extern "C" int moe_balance_fwd(const float* logits, int64_t ld_logits, const int32_t* ids, int T, int K, int E,
                               const int32_t* seg_offsets, int num_seq, float alpha, float beta, float* lse,
                               int32_t* counts, float* prob_sum, float* loss, int32_t* status_dev, void* workspace,
                               size_t workspace_bytes, moe_stream_t stream) {
  return router_entry("moe_balance_fwd", false, MOE_ROUTER_TOPK, 0, logits, ld_logits, T, K, E, seg_offsets, num_seq,
                      alpha, beta, nullptr, const_cast<int32_t*>(ids), lse, counts, prob_sum, loss, status_dev,
                      workspace, workspace_bytes, stream);
}

extern "C" int moe_balance_bwd(const float* logits, int64_t ld_logits, const float* lse, const int32_t* counts, int T,
                               int K, int E, const int32_t* seg_offsets, int num_seq, float alpha, float beta,
                               const float* dloss, const float* add, int64_t ld_add, float* dlogits,
                               int32_t* status_dev, moe_stream_t stream) {
  clear_error();
  int rc = bal_check("moe_balance_bwd", T, K, E, num_seq);
  if (rc) return rc;
  if (!seg_offsets && num_seq != 1) return fail(MOE_ERR_INVALID, "moe_balance_bwd: several sequences need seg_offsets");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) return status_dev ? cuda_check(cudaMemsetAsync(status_dev, 0, sizeof(int32_t), st), "memset status") : MOE_OK;
  if (!logits || !lse || !counts || !dlogits) return fail(MOE_ERR_INVALID, "moe_balance_bwd: null pointer");
  if (ld_logits < E || (add && ld_add < E)) return fail(MOE_ERR_INVALID, "moe_balance_bwd: row stride below E");
  for (const void* p : {static_cast<const void*>(logits), static_cast<const void*>(lse), static_cast<const void*>(counts),
                        static_cast<const void*>(seg_offsets), static_cast<const void*>(dloss),
                        static_cast<const void*>(add), static_cast<const void*>(dlogits),
                        static_cast<const void*>(status_dev)})
    if (reinterpret_cast<uintptr_t>(p) & 3)
      return fail(MOE_ERR_INVALID, "moe_balance_bwd: tensors must be 4-byte aligned");
  const int lanes = bal_bwd_lanes(E), nv = (E + 4 * lanes - 1) / (4 * lanes);
  BalanceArgs a{};
  a.logits = logits;
  a.ld = ld_logits;
  a.T = T;
  a.K = K;
  a.E = E;
  a.off = seg_offsets;
  a.S = num_seq;
  a.C = bal_bwd_chunk(T, lanes);
  a.pieces = bal_pieces(T, a.C, num_seq);
  a.alpha = alpha;
  a.beta = beta;
  a.lse = const_cast<float*>(lse);
  a.counts = const_cast<int32_t*>(counts);
  a.dloss = dloss;
  a.add = add;
  a.ld_add = ld_add;
  a.dlogits = dlogits;
  a.status = status_dev;
  const bool vec = E % 4 == 0 && ld_logits % 4 == 0 && (!add || ld_add % 4 == 0) &&
                   ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(add) |
                     reinterpret_cast<uintptr_t>(dlogits)) & 15) == 0;
  const BalKernel kern = vec ? bwd_kernel<true>(lanes, nv) : bwd_kernel<false>(lanes, nv);
  const int groups = nv <= 1 ? 1 : nv <= 2 && lanes == 8 ? 2 : nv <= 4 ? 4 : 8;
  const size_t smem = vec ? sizeof(float4) * kBalBwdStages * 2 * groups * kBalThreads : 0;
  return launch_pdl(kern, dim3(a.pieces), dim3(kBalThreads), smem, st, "balance_bwd", a);
}

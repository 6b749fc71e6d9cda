// Routing of tokens to experts (gemm_route_*): scores, the choice of top_k experts
// inside the kept groups, their weights, and the tokens' slots ordered by expert.
//
// With l a token's logits, its scores are s = softmax(l) or 1 / (1 + exp(-l)) and its
// choices c = s + bias (without a bias experts rank by l, which orders them as s does).
// A group's score is the sum of its `group_best` largest choices.
//
// Exact choices from fp32 arithmetic.  Which expert is ahead is defined by c in 64 bits,
// so that a reader's own arithmetic gives the same experts.  The kernel computes c in
// fp32, and looks at the gap between each two neighbours of the ranking, the last of the
// kept and the first of the others included: where a gap is larger than what both
// roundings can make, the order is that of 64 bits.  Experts with a smaller gap (of one
// token in a thousand with sigmoid scores and biases) are ranked again in fp64; equal logits
// with equal biases are no gap but a tie, which goes to the lowest index in both.  Where the
// last kept group and the first left out have a smaller gap, the whole token is done again by
// its block, at about 15 us: a call of 16384 x 256 in 8 groups of which 4 are kept takes 39 us
// with sigmoid scores and biases, 48 with softmax and biases, and 250 with sigmoid scores alone of
// logits of deviation 6, whose largest are all next to 1.
//
// Layout: a warp a token.  Lane i holds the experts i*PER .. i*PER+PER-1, so that the
// lowest lane with the largest key has the lowest index, and a round of the ranking is
// one redux, one ballot and one shuffle.  Per token the kernel reads its logits once:
// 4 E bytes against some 800 warp instructions at E = 256, k = 8 and 8 groups (many of them
// in the half-rate integer pipe), so issue bounds it, not HBM: 16384 tokens take 39 us, 9
// of them for the order by expert, against 3 us for the bytes.
//
// Order by expert without atomics whose order shows: blocks take consecutive tokens and
// count them by expert; a second kernel adds the counts of the blocks before its own,
// and gives each slot its place by its rank among equal experts of its warp
// (match_any), of the warps before it, and of the blocks before it.  One block does
// both where there are few tokens.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "plan.h"
#include "ptx.cuh"

namespace g3 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kPlaceWarps = 8;                 // segments of a block's slots in place_slots

template <typename T>
__device__ __forceinline__ float route_f32(T v);
template <>
__device__ __forceinline__ float route_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float route_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Logits as the scores see them: NaN counts as -inf.
__device__ __forceinline__ float clean(float l) { return fmaxf(l, -INFINITY); }

// A whole number that orders as the float does (-0 as +0); 0 is below every float's.
__device__ __forceinline__ uint32_t key_of(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// The same of a double; compared as a whole number (a handful of cycles, where the few
// fp64 units take tens).
__device__ __forceinline__ uint64_t key_of(double f) {
  const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(kFull, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(kFull, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
  return v;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

// One term of a softmax's sum; m the row's largest logit.  Where some logits are +inf
// they alone have weight, and a row of -inf alone has none.
template <typename F>
__device__ __forceinline__ F soft_term(float l, float m) {
  if (m == INFINITY) return l == INFINITY ? (F)1 : (F)0;
  if (l == -INFINITY) return (F)0;
  return exp((F)l - (F)m);
}
template <typename F>
__device__ __forceinline__ F score_of(bool softmax, float l, float m, F sum) {
  if (softmax) return sum > (F)0 ? soft_term<F>(l, m) / sum : (F)0;
  return (F)1 / ((F)1 + exp(-(F)l));
}

// exp and 1/x a few units of 2^-24 off (exp by one more for each unit of |x|, as its
// argument is rounded); what is below 2^-126 is 0
__device__ __forceinline__ float exp_near(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * 1.4426950408889634f));
  return e;
}
__device__ __forceinline__ float rcp_near(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sigmoid_near(float l) { return rcp_near(1.f + exp_near(-l)); }

// How far apart two choices in 64 bits may be whose fp32 forms are equal, for a score s
// and a choice c: 128 units of the last place of s cover expf of arguments down to its
// underflow and the sum of 1024 terms; a sigmoid is off by at most 3 * 2^-24; and the
// sum with the bias by half a unit of c.  Denormal numbers are whole steps of 2^-149, of which
// a score of softmax is off by four at most (exp by two, its product with 1/sum by a half,
// what that is off by the rest): 2^-140 is 512 of them.  A sigmoid below 2^-126 may come as 0.
__device__ __forceinline__ float slack(bool softmax, float s, float c) {
  const float of_s = softmax ? 0x1p-16f * s + 0x1p-140f : fminf(0x1p-16f * s, 0x1p-20f) + 0x1p-125f;
  return of_s + 0x1p-22f * fabsf(c);
}

// fp64 scores, out of line: the code of the rare paths is read from L2 when it is met, and
// every kilobyte of it costs about a microsecond.
__device__ __noinline__ double score_64(bool softmax, float l, float m, double sum) {
  return score_of<double>(softmax, l, m, sum);
}

// A token done again in fp64 by its block (all threads call it): an expert a thread, so
// that the scores take one fp64 latency, then one warp ranks.  ch: E values of shared
// memory.
template <typename T>
__device__ __noinline__ void route_exactly(const RouteArgs& a, long long t, double* ch, int* hist) {
  __shared__ double all;
  const T* logits = static_cast<const T*>(a.logits) + t * a.ld;
  const int E = a.experts, lane = threadIdx.x % 32;
  float m = -INFINITY;
  if (a.softmax) {
    for (int e = lane; e < E; e += 32) m = fmaxf(m, clean(route_f32(logits[e])));
    m = warp_max(m);
#pragma unroll 1
    for (int e = threadIdx.x; e < E; e += blockDim.x) ch[e] = score_64(true, clean(route_f32(logits[e])), m, 1.0);
    __syncthreads();
    if (threadIdx.x < 32) {
      double sum = 0.0;
      for (int e = lane; e < E; e += 32) sum += ch[e];
      sum = warp_sum(sum);
      if (lane == 0) all = sum;
    }
    __syncthreads();
  }
  const double sum = a.softmax ? all : 0.0;
#pragma unroll 1
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    double c = a.softmax ? (sum > 0.0 ? ch[e] / sum : 0.0) : score_64(false, clean(route_f32(logits[e])), m, sum);
    if (a.bias != nullptr) {
      const float b = a.bias[e];
      c = b < INFINITY ? c + (double)b : -INFINITY;      // NaN and +inf too: such an expert comes last
    }
    ch[e] = c;
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  uint32_t kept = kFull;
  const int G = a.groups, S = a.group_size;
  if (G > 1) {
    uint64_t g = 0;
    if (lane < G) {
      uint64_t b1 = 0, b2 = 0;
      double v1 = -INFINITY, v2 = -INFINITY;
#pragma unroll 1
      for (int i = 0; i < S; ++i) {
        const double c = ch[lane * S + i];
        const uint64_t k = key_of(c);
        if (k > b1) { b2 = b1; v2 = v1; b1 = k; v1 = c; } else if (k > b2) { b2 = k; v2 = c; }
      }
      g = key_of(a.group_best == 2 && S > 1 ? v1 + v2 : v1);
    }
    int ahead = 0;
#pragma unroll 1
    for (int o = 0; o < G; ++o) {
      const uint64_t v = __shfl_sync(kFull, g, o);
      ahead += v > g || (v == g && o < lane);
    }
    kept = __ballot_sync(kFull, lane < G && ahead < a.top_groups);
  }
  // keys in the choices' place; without a bias experts rank by their logits
  uint64_t* key = reinterpret_cast<uint64_t*>(ch);
  __syncwarp();
#pragma unroll 1
  for (int e = lane; e < E; e += 32) {
    const double c = a.bias != nullptr ? ch[e] : (double)clean(route_f32(logits[e]));
    key[e] = G == 1 || ((kept >> (e / S)) & 1u) ? key_of(c) : 0ull;
  }
  int id = 0;
#pragma unroll 1
  for (int j = 0; j < a.top_k; ++j) {
    uint64_t best = 0;
    int at = lane;
#pragma unroll 1
    for (int e = lane; e < E; e += 32)
      if (key[e] > best) { best = key[e]; at = e; }
    const uint64_t top = warp_max(best);
    // of the lanes that have it the one with the lowest expert
    const uint32_t e = __reduce_min_sync(kFull, best == top ? (uint32_t)at : 0xffffffffu);
    if (lane == j) id = (int)e;
    if ((uint32_t)at == e && best == top) key[e] = 0;
  }
  double w = lane < a.top_k ? score_64(a.softmax, clean(route_f32(logits[id])), m, sum) : 0.0;
  if (a.renormalise) {
    const double total = warp_sum(w);
    w = total > 0.0 ? w / total : 0.0;
  }
  if (lane < a.top_k) {
    a.ids[t * a.top_k + lane] = id;
    a.weights[t * a.top_k + lane] = (float)w * a.scale;
    if (hist != nullptr) atomicAdd(hist + id, 1);
  }
}

// The ranking of one token in fp32.  key[i]: lane's experts, 0 where there is none.
// Lane j returns the j-th expert.  Where fp32 cannot tell two neighbours apart, the
// experts down to the first that is clearly behind the last rank (32 at most) are ranked
// again by their choices in fp64, a lane each; *close is set where that does not do.
template <typename T, int PER>
__device__ __forceinline__ int rank_keys(const RouteArgs& a, const T* logits, uint32_t (&key)[PER], float m, float sum,
                                         int lane, bool* close) {
  uint32_t best = 0;
  int at = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (key[i] > best) { best = key[i]; at = i; }
  int mine = 0, prev = -1, ranked = 0;
  float prev_c = 0.f, last_c = 0.f;
  bool unsure = false;
  for (int j = 0;; ++j) {
    if (j >= a.top_k && a.bias == nullptr) break;       // ranks of logits are exact
    const uint32_t k = __reduce_max_sync(kFull, best);
    if (k == 0) break;                                  // none is left
    const int w = __ffs(__ballot_sync(kFull, best == k)) - 1;
    const int e = __shfl_sync(kFull, lane * PER + at, w);
    if (a.bias != nullptr) {
      const float c = of_key(k);
      bool tie = false;
      if (j > 0 && !(prev_c - c > 0x1p-15f * (1.f + fabsf(c)))) {   // also where both are -inf
        const float lp = clean(route_f32(logits[prev])), le = clean(route_f32(logits[e]));
        const float bp = a.bias[prev], be = a.bias[e];
        tie = (lp == le && bp == be) || (c == -INFINITY && prev_c == -INFINITY);
        const float s = fmaxf(score_of<float>(a.softmax, lp, m, sum), score_of<float>(a.softmax, le, m, sum));
        if (!tie && !(prev_c - c > slack(a.softmax, s, fmaxf(fabsf(c), fabsf(prev_c))))) unsure = true;
      }
      // past the last rank: on while it may still belong before it
      if (j >= a.top_k && !tie && !(unsure && !(last_c - c > 0x1p-15f * (1.f + fabsf(c))))) break;
      if (j == a.top_k - 1) last_c = c;
      if (j == 32) {                                    // no lane is left for the next
        *close = true;
        break;
      }
      prev = e;
      prev_c = c;
    }
    if (lane == j) mine = e;
    ranked = j + 1;
    if (lane == w) {
      best = 0;
      const int gone = at;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (i == gone) key[i] = 0;
        if (key[i] > best) { best = key[i]; at = i; }
      }
    }
  }
  if (unsure && !*close) {
    double all = 0.0;
    if (a.softmax) {
#pragma unroll 1
      for (int e = lane; e < a.experts; e += 32) all += score_64(true, clean(route_f32(logits[e])), m, 1.0);
      all = warp_sum(all);
    }
    uint64_t c = 0;
    if (lane < ranked) {
      const float b = a.bias[mine];
      c = key_of(b < INFINITY ? score_64(a.softmax, clean(route_f32(logits[mine])), m, all) + (double)b : -INFINITY);
    }
    int rank = 0;
    for (int o = 0; o < ranked; ++o) {
      const uint64_t v = __shfl_sync(kFull, c, o);
      const int e = __shfl_sync(kFull, mine, o);
      rank += v > c || (v == c && e < mine);
    }
    int sorted = 0;
    for (int o = 0; o < ranked; ++o) {
      const int e = __shfl_sync(kFull, mine, o);
      if (__shfl_sync(kFull, rank, o) == lane) sorted = e;
    }
    mine = sorted;
  }
  return mine;
}

// The same for up to 256 experts, with keys whose last 8 bits are the expert's number
// (inverted: of equal ones the lowest is largest), so that one redux gives a rank.  Each
// lane's keys are sorted once, and a lane that won moves its keys up.  24 bits of a choice
// tell most neighbours apart (of sigmoid scores near 1 two tokens in three); where they
// tell the last rank from the next one at least, the chosen are put in order by their
// choices in fp32, a lane each: 100 instructions in place of rank_keys' 500.  *unsure is
// set where that does not do either, and rank_keys decides.
template <typename T, int PER>
__device__ __forceinline__ int rank_packed(const RouteArgs& a, const T* logits, const uint32_t (&key)[PER], float m, float sum,
                                           int lane, bool* unsure) {
  uint32_t q[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) q[i] = (key[i] & ~0xffu) | (0xffu - (uint32_t)(lane * PER + i));   // below 256: none
  auto order = [&](int i, int j) {
    const uint32_t hi = max(q[i], q[j]), lo = min(q[i], q[j]);
    q[i] = hi;
    q[j] = lo;
  };
  if constexpr (PER == 2) {
    order(0, 1);
  } else if constexpr (PER >= 4) {
#pragma unroll
    for (int h = 0; h < PER; h += 4) {                  // networks of 5 and of 19 comparators
      order(h, h + 1); order(h + 2, h + 3); order(h, h + 2); order(h + 1, h + 3); order(h + 1, h + 2);
    }
    if constexpr (PER == 8) {
      order(0, 4); order(1, 5); order(2, 6); order(3, 7); order(2, 4); order(3, 5); order(1, 2); order(3, 4); order(5, 6);
    }
  }
  uint32_t mine = 0;                                    // lane j: the j-th key
  for (int j = 0; j <= a.top_k; ++j) {
    const uint32_t k = __reduce_max_sync(kFull, q[0]);
    if (lane == j) mine = k;
    const bool won = q[0] == k;
#pragma unroll
    for (int i = 0; i + 1 < PER; ++i) q[i] = won ? q[i + 1] : q[i];
    q[PER - 1] = won ? 0u : q[PER - 1];
  }
  // neighbours.  24 bits hold a bf16 logit whole, and order fp32 logits
  // where they differ
  const uint32_t before = __shfl_up_sync(kFull, mine, 1);
  bool near = false;
  if (lane > 0 && lane <= a.top_k && mine > 0xffu) {
    if (a.bias == nullptr) {
      near = !a.bf16 && (before >> 8) == (mine >> 8);
    } else {
      const float hi = of_key(before & ~0xffu), lo = of_key(mine | 0xffu);
      near = !(hi - lo > 0x1p-15f * (1.f + fabsf(lo)));               // well above slack()
    }
  }
  const int id = (int)(0xffu - (mine & 0xffu));
  const uint32_t some = __ballot_sync(kFull, near);
  *unsure = a.top_k == 32 || ((some >> a.top_k) & 1u);   // of 33 ranks the last has no lane
  if (some == 0 || *unsure) return id;
  const bool in = lane < a.top_k;
  const float l = in ? clean(route_f32(logits[id])) : 0.f;
  const float b = in && a.bias != nullptr ? a.bias[id] : 0.f;
  float s = 0.f, v = l;
  if (a.bias != nullptr) {
    s = score_of<float>(a.softmax, l, m, sum);
    v = b < INFINITY ? s + b : -INFINITY;
  }
  const uint32_t k = key_of(v);
  int rank = 0, from = 0;
  for (int o = 0; o < a.top_k; ++o) {
    const uint32_t ko = __shfl_sync(kFull, k, o);
    const int e = __shfl_sync(kFull, id, o);
    rank += ko > k || (ko == k && e < id);
  }
  for (int o = 0; o < a.top_k; ++o)
    if (__shfl_sync(kFull, rank, o) == lane) from = o;
  const int sorted = __shfl_sync(kFull, id, from);
  if (a.bias != nullptr) {
    const float v1 = __shfl_sync(kFull, v, from), s1 = __shfl_sync(kFull, s, from);
    const float l1 = __shfl_sync(kFull, l, from), b1 = __shfl_sync(kFull, b, from);
    const float v0 = __shfl_up_sync(kFull, v1, 1), s0 = __shfl_up_sync(kFull, s1, 1);
    const float l0 = __shfl_up_sync(kFull, l1, 1), b0 = __shfl_up_sync(kFull, b1, 1);
    // what was last has nothing near it behind it, whichever of the chosen it was
    const bool apart = (l0 == l1 && b0 == b1) || v1 == -INFINITY ||
                       v0 - v1 > slack(a.softmax, fmaxf(s0, s1), fmaxf(fabsf(v0), fabsf(v1)));
    *unsure = __any_sync(kFull, in && lane > 0 && !apart);
  }
  return sorted;
}

// The two largest of this lane's and the others' (lanes that differ in bits below `span`).
__device__ __forceinline__ void best_two(float& b1, float& b2, int span) {
  for (int d = span >> 1; d; d >>= 1) {
    const float o1 = __shfl_xor_sync(kFull, b1, d), o2 = __shfl_xor_sync(kFull, b2, d);
    b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
    b1 = fmaxf(b1, o1);
  }
}

// Which groups are kept, as bits.  c: this lane's choices (-inf where there is no expert);
// ch: E floats of shared memory.  *close is set where fp32 cannot tell the last kept group
// from the first left out.
template <int PER>
__device__ __forceinline__ uint32_t keep_groups(const RouteArgs& a, const float (&c)[PER], float* ch, int lane, bool* close) {
  const int G = a.groups, S = a.group_size;
  int per = a.group_lanes;             // lanes of a group, a power of two
  float b1 = -INFINITY, b2 = -INFINITY;
  if (a.group_whole) {                 // each group is whole lanes: all in registers
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      b2 = fmaxf(b2, fminf(b1, c[i]));
      b1 = fmaxf(b1, c[i]);
    }
  } else {
    const int e0 = lane * PER;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e0 + i < a.experts) ch[e0 + i] = c[i];
    __syncwarp();
    const int group = lane / per, part = lane % per;
    if (group < G)
      for (int i = part; i < S; i += per) {
        const float v = ch[group * S + i];
        b2 = fmaxf(b2, fminf(b1, v));
        b1 = fmaxf(b1, v);
      }
    __syncwarp();
  }
  best_two(b1, b2, per);
  const float g = a.group_best == 2 && S > 1 ? b1 + b2 : b1;
  // ranks of the groups: lane i < G looks at group i
  const float mine = __shfl_sync(kFull, g, min(lane * per, 31));
  const uint32_t k = key_of(mine);
  int ahead = 0;
  for (int o = 0; o < G; ++o) ahead += __shfl_sync(kFull, k, o) >= k + (o >= lane);
  const uint32_t kept = __ballot_sync(kFull, lane < G && ahead < a.top_groups);
  if (a.top_groups < G) {
    const float in = __shfl_sync(kFull, mine, __ffs(__ballot_sync(kFull, lane < G && ahead == a.top_groups - 1)) - 1);
    const float out = __shfl_sync(kFull, mine, __ffs(__ballot_sync(kFull, lane < G && ahead == a.top_groups)) - 1);
    // two softmax scores are at most 1 together, and relative to themselves without a bias
    const float s = a.softmax ? (a.bias != nullptr ? 1.f : fabsf(in)) : 2.f;
    bool sure;
    if (out == -INFINITY)      // such groups are behind all others and by index, but for sums of finite
                               // choices that fp32 does not hold
      sure = !__any_sync(kFull, g == -INFINITY && a.group_best == 2 && S > 1 && b2 > -INFINITY && lane / per < G);
    else
      sure = in - out > slack(a.softmax, s, fmaxf(fabsf(in), fabsf(out))) * 2.f;
    if (!sure) *close = true;
  }
  return kept;
}

// Rows of padding: where all logits are one number, and all biases, all choices are equal in
// 64 bits as well, and the ranking by index stands (16384 x 256 of them in fp64: 1600 us).
template <typename T>
__device__ __noinline__ bool all_equal(const RouteArgs& a, const T* logits, int lane) {
  const float l0 = clean(route_f32(logits[0])), b0 = a.bias != nullptr ? a.bias[0] : 0.f;
  bool same = true;
#pragma unroll 1
  for (int e = lane; e < a.experts; e += 32)
    same = same && clean(route_f32(logits[e])) == l0 && (a.bias == nullptr || a.bias[e] == b0);
  return __all_sync(kFull, same) != 0;
}

// bias: this lane's experts' (0 without one, -inf where there is no expert); ch: E floats of the warp's own, where groups
// are not whole lanes.  A token that fp32 cannot route is marked by ids of -1 and counted
// in *slow.
template <typename T, int PER>
__device__ __forceinline__ void route_token(const RouteArgs& a, long long t, const float (&bias)[PER], float* ch, int* hist,
                                            int* slow, int lane) {
  const T* logits = static_cast<const T*>(a.logits) + t * a.ld;
  const int E = a.experts;
  float l[PER];
  const int e0 = lane * PER;
  if (a.vec && e0 + PER <= E) {          // rows of whole, aligned vectors
    constexpr int BYTES = PER * (int)sizeof(T);
    if constexpr (BYTES % 16 == 0) {
#pragma unroll
      for (int q = 0; q < BYTES / 16; ++q) {
        const uint4 v = reinterpret_cast<const uint4*>(logits + e0)[q];
        alignas(16) T part[16 / sizeof(T)];
        *reinterpret_cast<uint4*>(part) = v;
#pragma unroll
        for (int i = 0; i < (int)(16 / sizeof(T)); ++i) l[q * (int)(16 / sizeof(T)) + i] = clean(route_f32(part[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) l[i] = clean(route_f32(logits[e0 + i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = e0 + i < E ? clean(route_f32(logits[e0 + i])) : -INFINITY;
  }
  float m = 0.f, sum = 0.f;
  float c[PER];
  if (a.softmax) {
    m = l[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      c[i] = soft_term<float>(l[i], m);                  // 0 where there is no expert
      sum += c[i];
    }
    sum = warp_sum(sum);
  }
  uint32_t key[PER];
  bool close = false;
  if (a.choices) {
    const float r = a.softmax && sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      // the approximate operations and the product with 1/sum stay inside slack()'s units
      float s = a.softmax ? c[i] * r : sigmoid_near(l[i]);
      s += bias[i];                                      // -inf: the expert comes last, or there is none
      c[i] = s;
      key[i] = key_of(a.bias != nullptr ? s : l[i]);
    }
    if (a.groups > 1) {
      const uint32_t kept = keep_groups<PER>(a, c, ch, lane, &close);
      if (close) close = !all_equal<T>(a, logits, lane);
      if (a.group_whole) {
        if (!((kept >> ((lane / a.group_lanes) & 31)) & 1u)) {
#pragma unroll
          for (int i = 0; i < PER; ++i) key[i] = 0u;
        }
      } else {
        const int S = a.group_size;
        int g = e0 / S, left = S - e0 % S;     // this lane's experts run through the groups in order
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          if (!((kept >> (g & 31)) & 1u)) key[i] = 0u;
          if (--left == 0) { ++g; left = S; }
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = key_of(l[i]);
  }
  if (E < 32 * PER) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e0 + i >= E) key[i] = 0u;
  }
  int id = 0;
  bool unsure = true;
  if (!close) {
    if constexpr (PER <= 8) id = rank_packed<T, PER>(a, logits, key, m, sum, lane, &unsure);
    if (PER > 8 || (unsure && !all_equal<T>(a, logits, lane))) {
      id = rank_keys<T, PER>(a, logits, key, m, sum, lane, &close);
      if (PER > 8 && close) close = !all_equal<T>(a, logits, lane);
    }
  }
  if (close) {
    if (lane == 0) {
      a.ids[t * a.top_k] = -1;
      atomicAdd(slow, 1);
    }
    return;
  }
  // weights of the chosen, from their logits again
  const bool mine = lane < a.top_k;
  const float lw = mine ? clean(route_f32(logits[id])) : 0.f;
  float w = 0.f;
  if (mine) {
    if (a.softmax) w = sum > 0.f && m < INFINITY ? exp_near(lw - m) * rcp_near(sum) : score_of<float>(true, lw, m, sum);
    else w = rcp_near(1.f + exp_near(-lw));
  }
  // scores so small that the fast operations lose them: the others' way
  if (__any_sync(kFull, mine && !(w > 0x1p-100f)) && mine) w = score_of<float>(a.softmax, lw, m, sum);
  if (a.renormalise) {
    const float all = warp_sum(w);
    if (all > 0x1p-100f) {
      w *= rcp_near(all);
    } else {                             // scores that fp32 holds in a few bits or not at all
      const double v = mine ? score_64(a.softmax, lw, m, (double)sum) : 0.0, total = warp_sum(v);
      w = total > 0.0 ? (float)(v / total) : 0.f;
    }
  }
  if (mine) {
    a.ids[t * a.top_k + lane] = id;
    a.weights[t * a.top_k + lane] = w * a.scale;
    if (hist != nullptr) atomicAdd(hist + id, 1);
  }
}

// Exclusive sums of total[0..E-1] into base[0..E-1] (in place allowed), by one warp;
// returns the sum of all.
__device__ __forceinline__ int warp_scan(const int* total, int* base, int E, int lane) {
  int run = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int v = e0 + lane < E ? total[e0 + lane] : 0;
    int s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kFull, s, d);
      if (lane >= d) s += o;
    }
    if (e0 + lane < E) base[e0 + lane] = run + s - v;
    run += __shfl_sync(kFull, s, 31);
  }
  return run;
}

// Places the slots [s0, s1) whose experts are in ids, by the first kPlaceWarps warps of
// the block.  at[w * E + e]: zero on entry; base[e]: where the block's first slot of
// expert e goes.
__device__ __forceinline__ void place_slots(const RouteArgs& a, long long s0, long long s1, const int* base, int* at) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, E = a.experts;
  const long long each = ((s1 - s0 + kPlaceWarps - 1) / kPlaceWarps + 31) / 32 * 32;
  const long long b = s0 + warp * each, e = b + each < s1 ? b + each : s1;
  constexpr int U = 4;                   // loads in flight
  if (warp < kPlaceWarps)
    for (long long s = b; s < e; s += 32 * U) {
      int id[U];
#pragma unroll
      for (int u = 0; u < U; ++u) id[u] = s + u * 32 + lane < e ? a.ids[s + u * 32 + lane] : -1;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t same = __match_any_sync(kFull, id[u]);
        if (id[u] >= 0 && (same & ((1u << lane) - 1u)) == 0) at[warp * E + id[u]] += __popc(same);
        __syncwarp();
      }
    }
  __syncthreads();
  for (int x = threadIdx.x; x < E; x += blockDim.x) {
    int run = base[x];
#pragma unroll
    for (int w = 0; w < kPlaceWarps; ++w) {
      const int n = at[w * E + x];
      at[w * E + x] = run;
      run += n;
    }
  }
  __syncthreads();
  if (warp < kPlaceWarps)
    for (long long s = b; s < e; s += 32 * U) {
      int id[U];
#pragma unroll
      for (int u = 0; u < U; ++u) id[u] = s + u * 32 + lane < e ? a.ids[s + u * 32 + lane] : -1;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t same = __match_any_sync(kFull, id[u]);
        const uint32_t before = same & ((1u << lane) - 1u);
        int first = 0;
        if (id[u] >= 0) first = at[warp * E + id[u]];
        __syncwarp();
        if (id[u] >= 0) {
          a.order[first + __popc(before)] = (int)(s + u * 32 + lane);
          if (before == 0) at[warp * E + id[u]] = first + __popc(same);
        }
        __syncwarp();
      }
    }
}

// Counts of a block: rows of whole 16-byte vectors
__host__ __device__ constexpr int count_stride(int experts) { return (experts + 3) / 4 * 4; }

// Doubles of shared memory for choices: a token's in fp64, and a row of floats for each warp
__host__ __device__ inline int route_smem_choices(const RouteArgs& a, int warps) {
  return a.choices ? a.experts + (a.groups > 1 && !a.group_whole ? (warps * a.experts + 1) / 2 : 0) : 0;
}

template <int PER>
constexpr int route_threads() { return PER <= 8 ? 1024 : 256; }

// Block b routes tokens [b*chunk, (b+1)*chunk).  One block alone also places them.
template <typename T, int PER>
__global__ void __launch_bounds__(route_threads<PER>()) route_kernel(const __grid_constant__ RouteArgs a, int chunk) {
  extern __shared__ double route_smem[];
  __shared__ int slow, next, list[route_threads<PER>()];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32, E = a.experts;
  double* exact = route_smem;                            // E choices in fp64, of one token at a time
  float* ch = reinterpret_cast<float*>(exact + (a.choices ? E : 0)) + (a.groups > 1 && !a.group_whole ? warp * E : 0);
  int* hist = reinterpret_cast<int*>(route_smem + route_smem_choices(a, warps));
  const bool plan = a.offsets != nullptr;
  if (threadIdx.x == 0) {
    slow = 0;
    next = warps;
  }
  if (plan)
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  griddep_wait();
  __syncthreads();
  const long long t0 = (long long)blockIdx.x * chunk;
  const long long t1 = t0 + chunk < a.tokens ? t0 + chunk : a.tokens;
  float bias[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    const float b = e >= E ? -INFINITY : a.bias != nullptr ? a.bias[e] : 0.f;
    bias[i] = b < INFINITY ? b : -INFINITY;              // NaN and +inf too: such an expert comes last
  }
  // tokens take unlike times: a warp takes the next that none has
  for (long long t = t0 + warp; t < t1;) {
    route_token<T, PER>(a, t, bias, ch, plan ? hist : nullptr, &slow, lane);
    int n = 0;
    if (lane == 0) n = atomicAdd(&next, 1);
    t = t0 + __shfl_sync(kFull, n, 0);
  }
  __syncthreads();
  if (slow > 0) {                                        // marked by warps of this block: a list, then one by one
    __syncthreads();
    for (long long at = t0; at < t1; at += blockDim.x) {
      if (threadIdx.x == 0) slow = 0;
      __syncthreads();
      const long long t = at + threadIdx.x;
      if (t < t1 && a.ids[t * a.top_k] < 0) list[atomicAdd(&slow, 1)] = (int)(t - at);
      __syncthreads();
      const int n = slow;
      for (int i = 0; i < n; ++i) {
        route_exactly<T>(a, at + list[i], exact, plan ? hist : nullptr);
        __syncthreads();
      }
    }
  }
  if (!plan) return;
  if (gridDim.x > 1) {
    griddep_launch_dependents();
    if (a.counts == nullptr) return;                     // route_order_kernel counts ids
    for (int e = threadIdx.x; e < E; e += blockDim.x) a.counts[(size_t)blockIdx.x * count_stride(E) + e] = hist[e];
    return;
  }
  // ids written by this block's other warps are read back below: __syncthreads orders them
  int* at = hist + E;
  for (int x = threadIdx.x; x < kPlaceWarps * E; x += blockDim.x) at[x] = 0;
  if (warp == 0) {
    const int all = warp_scan(hist, hist, E, lane);
    for (int e = lane; e < E; e += 32) a.offsets[e] = hist[e];
    if (lane == 0) a.offsets[E] = all;
  }
  __syncthreads();
  place_slots(a, t0 * a.top_k, t1 * a.top_k, hist, at);
}

constexpr int kPlaceKernelThreads = 1024;
// The sum of all values before this thread's (an expert a thread, 0 behind the last), by the
// whole block.
__device__ __forceinline__ int block_scan(int v) {
  __shared__ int sums[kPlaceKernelThreads / 32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  auto scan = [&](int x) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kFull, x, d);
      if (lane >= d) x += o;
    }
    return x;
  };
  const int s = scan(v);
  if (lane == 31) sums[warp] = s;
  __syncthreads();
  const int w = sums[lane], all = scan(w);             // every warp for itself
  return __shfl_sync(kFull, all - w, warp) + s - v;
}
static_assert(kPlaceKernelThreads == 1024 && kRouteMaxExperts <= kPlaceKernelThreads, "a warp a lane, an expert a thread");

// The same blocks' slots, placed: counts of all blocks and of those before.  A thread
// adds four experts' counts of some of the blocks, eight rows in flight at a time.
__global__ void __launch_bounds__(kPlaceKernelThreads) route_place_kernel(const __grid_constant__ RouteArgs a, int chunk) {
  extern __shared__ int place_smem[];
  const int E = a.experts, x = threadIdx.x;
  int *total = place_smem, *before = total + E, *at = before + E;
  for (int i = x; i < (2 + kPlaceWarps) * E; i += blockDim.x) place_smem[i] = 0;
  griddep_wait();
  __syncthreads();
  const int stride4 = count_stride(E) / 4, blocks = gridDim.x;
  const int parts = kPlaceKernelThreads / stride4;       // at least 4: E is 1024 at most
  const int part = threadIdx.x / stride4, e4 = threadIdx.x % stride4;
  if (part < parts) {
    const int4* rows = reinterpret_cast<const int4*>(a.counts) + e4;
    int all[4] = {0, 0, 0, 0}, mine[4] = {0, 0, 0, 0};
    for (int b0 = part; b0 < blocks; b0 += 8 * parts) {
      int4 n[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int b = b0 + u * parts;
        n[u] = b < blocks ? rows[(size_t)b * stride4] : make_int4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const bool earlier = b0 + u * parts < (int)blockIdx.x;
        const int v[4] = {n[u].x, n[u].y, n[u].z, n[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          all[i] += v[i];
          mine[i] += earlier ? v[i] : 0;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e4 * 4 + i < E) {                  // whole numbers: any order gives the same sum
        atomicAdd(total + e4 * 4 + i, all[i]);
        atomicAdd(before + e4 * 4 + i, mine[i]);
      }
  }
  __syncthreads();
  const int n = x < E ? total[x] : 0, first = block_scan(n);
  if (x < E) before[x] += first;
  if (blockIdx.x == 0 && x < E) a.offsets[x] = first;
  if (blockIdx.x == 0 && x == E - 1) a.offsets[E] = first + n;
  __syncthreads();
  const long long t0 = (long long)blockIdx.x * chunk;
  const long long t1 = t0 + chunk < a.tokens ? t0 + chunk : a.tokens;
  place_slots(a, t0 * a.top_k, t1 * a.top_k, before, at);
}

// All slots of a call by one block, from their ids alone.
__global__ void __launch_bounds__(kPlaceKernelThreads) route_order_kernel(const __grid_constant__ RouteArgs a) {
  extern __shared__ int place_smem[];
  const int E = a.experts, x = threadIdx.x, slots = a.tokens * a.top_k;
  int *total = place_smem, *at = total + E;
  for (int i = x; i < (1 + kPlaceWarps) * E; i += blockDim.x) place_smem[i] = 0;
  griddep_wait();
  __syncthreads();
  for (int s = threadIdx.x; s < slots; s += blockDim.x) atomicAdd(total + a.ids[s], 1);
  __syncthreads();
  const int n = x < E ? total[x] : 0, first = block_scan(n);
  if (x < E) total[x] = a.offsets[x] = first;
  if (x == E - 1) a.offsets[E] = first + n;
  __syncthreads();
  place_slots(a, 0, slots, total, at);
}

template <typename T, int PER>
int launch_impl(const RouteArgs& a, int num_sms, cudaStream_t s) {
  const plan::RoutePlan p = plan::route_plan(a.tokens, a.experts, num_sms);
  const int threads = p.warps * 32;
  const size_t smem = (size_t)route_smem_choices(a, p.warps) * sizeof(double) +
                      (size_t)a.experts * (1 + kPlaceWarps) * sizeof(int);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_smem_once(done, route_kernel<T, PER>,
                                (int)((route_threads<PER>() / 64 + 1) * 32 * PER * sizeof(double) + 32 * PER * (1 + kPlaceWarps) * sizeof(int)));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.blocks, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, route_kernel<T, PER>, a, p.chunk);
  if (e != cudaSuccess || p.blocks == 1 || a.offsets == nullptr) return e;
  if (a.counts == nullptr) {
    cfg.gridDim = dim3(1, 1, 1);
    cfg.blockDim = dim3(kPlaceKernelThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)a.experts * (1 + kPlaceWarps) * sizeof(int);
    return cudaLaunchKernelEx(&cfg, route_order_kernel, a);
  }
  cfg.blockDim = dim3(kPlaceKernelThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)a.experts * (2 + kPlaceWarps) * sizeof(int);
  return cudaLaunchKernelEx(&cfg, route_place_kernel, a, p.chunk);
}

template <typename T>
int launch_type(const RouteArgs& a, int num_sms, cudaStream_t s) {
  switch (route_experts_per_lane(a.experts)) {
    case 1: return launch_impl<T, 1>(a, num_sms, s);
    case 2: return launch_impl<T, 2>(a, num_sms, s);
    case 4: return launch_impl<T, 4>(a, num_sms, s);
    case 8: return launch_impl<T, 8>(a, num_sms, s);
    case 16: return launch_impl<T, 16>(a, num_sms, s);
  }
  return launch_impl<T, 32>(a, num_sms, s);
}

}  // namespace

size_t route_ws_bytes(int tokens, int experts) {
  const plan::RoutePlan p = plan::route_plan(tokens, experts, plan::kRouteMaxBlocks);
  return p.blocks > 1 && !p.few ? (size_t)p.blocks * count_stride(experts) * sizeof(int) : 0;
}

int launch_route(const RouteArgs& a, int num_sms, cudaStream_t s) {
  return a.bf16 ? launch_type<__nv_bfloat16>(a, num_sms, s) : launch_type<float>(a, num_sms, s);
}

}  // namespace g3

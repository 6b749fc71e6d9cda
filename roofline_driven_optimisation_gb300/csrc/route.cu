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
// roundings can make, the order is that of 64 bits.  A token with a smaller gap (one in a
// thousand of sigmoid scores) is done again in fp64; equal logits with equal biases are
// no gap but a tie, which goes to the lowest index in both.
//
// Layout: a warp a token.  Lane i holds the experts i*PER .. i*PER+PER-1, so that the
// lowest lane with the largest key has the lowest index, and a round of the ranking is
// one redux, one ballot and one shuffle.  Per token the kernel reads its logits once:
// 4 E bytes against some 250 warp instructions at E = 256, k = 8, so issue and the chain
// of dependent rounds bound it, not HBM.
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
#include "ptx.cuh"

namespace g3 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kPlaceWarps = 8;                 // segments of a block's slots in place_slots
constexpr int kPlaceThreads = kPlaceWarps * 32;

template <typename T>
__device__ __forceinline__ float route_f32(T v);
template <>
__device__ __forceinline__ float route_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float route_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Logits as the scores see them: NaN counts as -inf.
__device__ __forceinline__ float clean(float l) { return l == l ? l : -INFINITY; }

// A whole number that orders as the float does (-0 as +0); 0 is below every float's.
__device__ __forceinline__ uint32_t key_of(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
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

// How far apart two choices in 64 bits may be whose fp32 forms are equal, for a score s
// and a choice c: 128 units of the last place of s cover expf of arguments down to its
// underflow and the sum of 1024 terms; a sigmoid is off by at most 3 * 2^-24; and the
// sum with the bias by half a unit of c.
__device__ __forceinline__ float slack(bool softmax, float s, float c) {
  const float of_s = softmax ? 0x1p-16f * s : fminf(0x1p-16f * s, 0x1p-20f);
  return of_s + 0x1p-22f * fabsf(c);
}

// A token done again in fp64 by its warp: choices in `ch` (E values of shared memory),
// winners to lane j's return value.  `bias` may be null (groups alone decide by sums).
template <typename T>
__device__ __noinline__ int route_exactly(const RouteArgs& a, const T* logits, double* ch, float m, int lane) {
  const int E = a.experts;
  double sum = 0.0;
  if (a.softmax) {
    for (int e = lane; e < E; e += 32) sum += soft_term<double>(clean(route_f32(logits[e])), m);
    sum = warp_sum(sum);
  }
  for (int e = lane; e < E; e += 32) {
    double c = score_of<double>(a.softmax, clean(route_f32(logits[e])), m, sum);
    if (a.bias != nullptr) {
      const float b = a.bias[e];
      c = b < INFINITY ? c + (double)b : -INFINITY;
    }
    ch[e] = c;
  }
  __syncwarp();
  uint32_t kept = kFull;
  const int G = a.groups, S = E / G;
  if (G > 1) {
    double g = -INFINITY;
    if (lane < G) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int i = 0; i < S; ++i) {
        const double c = ch[lane * S + i];
        if (c > b1) { b2 = b1; b1 = c; } else if (c > b2) { b2 = c; }
      }
      g = a.group_best == 2 && S > 1 ? b1 + b2 : b1;
    }
    int ahead = 0;
    for (int o = 0; o < G; ++o) {
      const double v = __shfl_sync(kFull, g, o);
      ahead += v > g || (v == g && o < lane);
    }
    kept = __ballot_sync(kFull, lane < G && ahead < a.top_groups);
  }
  // without a bias experts rank by their logits
  int mine = 0;
  double last = INFINITY;
  int last_e = -1;                       // ranks so far end at (last, last_e)
  for (int j = 0; j < a.top_k; ++j) {
    double best = 0.0;
    int at = E;
    for (int e = lane; e < E; e += 32) {
      if (G > 1 && !((kept >> (e / S)) & 1u)) continue;
      const double c = a.bias != nullptr ? ch[e] : (double)clean(route_f32(logits[e]));
      if (j > 0 && !(c < last || (c == last && e > last_e))) continue;
      if (at == E || c > best) { best = c; at = e; }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const double ob = __shfl_xor_sync(kFull, best, d);
      const int oe = __shfl_xor_sync(kFull, at, d);
      if (oe < E && (at == E || ob > best || (ob == best && oe < at))) { best = ob; at = oe; }
    }
    last = best;
    last_e = at;
    if (lane == j) mine = at;
  }
  return mine;
}

// The ranking of one token in fp32.  key[i]: lane's experts, 0 where there is none.
// Lane j returns the j-th expert; *close is set where fp32 cannot tell.
template <typename T, int PER>
__device__ __forceinline__ int rank_keys(const RouteArgs& a, const T* logits, uint32_t (&key)[PER], float m, float sum,
                                         int lane, bool* close) {
  uint32_t best = 0;
  int at = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (key[i] > best) { best = key[i]; at = i; }
  int mine = 0, prev = -1;
  float prev_c = 0.f;
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
        if (!tie && !(prev_c - c > slack(a.softmax, s, fmaxf(fabsf(c), fabsf(prev_c))))) {
          *close = true;
          break;
        }
      }
      if (j >= a.top_k && !tie) break;
      prev = e;
      prev_c = c;
    }
    if (lane == j) mine = e;
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
  return mine;
}

// Groups: choices are in ch (E floats of shared memory).  Returns the kept groups as
// bits; *close is set where fp32 cannot tell the last kept from the first left out.
__device__ __forceinline__ uint32_t keep_groups(const RouteArgs& a, const float* ch, int lane, bool* close) {
  const int G = a.groups, S = a.experts / G;
  // lanes of a group: the largest power of two that all groups can have
  int per = 32;
  while (per * G > 32) per >>= 1;
  const int group = lane / per, part = lane % per;
  float b1 = -INFINITY, b2 = -INFINITY;
  if (group < G)
    for (int i = part; i < S; i += per) {
      const float c = ch[group * S + i];
      b2 = fmaxf(b2, fminf(b1, c));
      b1 = fmaxf(b1, c);
    }
  for (int d = per >> 1; d; d >>= 1) {
    const float o1 = __shfl_xor_sync(kFull, b1, d), o2 = __shfl_xor_sync(kFull, b2, d);
    b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
    b1 = fmaxf(b1, o1);
  }
  const float g = a.group_best == 2 && S > 1 ? b1 + b2 : b1;
  // ranks of the groups: lane i < G looks at group i
  const float mine = __shfl_sync(kFull, g, min(lane * per, 31));
  int ahead = 0;
  for (int o = 0; o < G; ++o) {
    const float v = __shfl_sync(kFull, mine, o);
    ahead += v > mine || (v == mine && o < lane);
  }
  const uint32_t kept = __ballot_sync(kFull, lane < G && ahead < a.top_groups);
  if (a.top_groups < G) {
    const float in = __shfl_sync(kFull, mine, __ffs(__ballot_sync(kFull, lane < G && ahead == a.top_groups - 1)) - 1);
    const float out = __shfl_sync(kFull, mine, __ffs(__ballot_sync(kFull, lane < G && ahead == a.top_groups)) - 1);
    // two softmax scores are at most 1 together, and relative to themselves without a bias
    const float s = a.softmax ? (a.bias != nullptr ? 1.f : fabsf(in)) : 2.f;
    if (!(in - out > slack(a.softmax, s, fmaxf(fabsf(in), fabsf(out))) * 2.f) && in != -INFINITY) *close = true;
  }
  return kept;
}

// Shared memory of a block: E counts, then per warp E choices of 8 bytes (fp64 path; as
// floats for the groups).
template <typename T, int PER>
__device__ __forceinline__ void route_token(const RouteArgs& a, long long t, double* ch, int* hist, int lane) {
  const T* logits = static_cast<const T*>(a.logits) + t * a.ld;
  const int E = a.experts;
  float l[PER];
  const int e0 = lane * PER;
  if (a.vec && e0 + PER <= E) {          // rows of whole, aligned vectors
    constexpr int BYTES = PER * (int)sizeof(T);
    if constexpr (BYTES % 16 == 0) {
#pragma unroll
      for (int q = 0; q < BYTES / 16; ++q) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(logits + e0) + q);
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
  if (a.softmax) {
    m = l[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += e0 + i < E ? soft_term<float>(l[i], m) : 0.f;
    sum = warp_sum(sum);
  }
  uint32_t key[PER];
  bool close = false;
  if (a.bias != nullptr || a.groups > 1) {
    const float r = a.softmax && sum > 0.f ? 1.f / sum : 0.f;
    float c[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      // __expf and the product with 1/sum stay inside slack()'s 128 units
      float s = a.softmax ? soft_term<float>(l[i], m) * r : __fdividef(1.f, 1.f + __expf(-l[i]));
      if (!a.softmax && l[i] < -80.f) s = score_of<float>(false, l[i], 0.f, 0.f);   // __fdividef's own range ends there
      if (a.bias != nullptr && e0 + i < E) {
        const float b = __ldg(a.bias + e0 + i);
        s = b < INFINITY ? s + b : -INFINITY;      // NaN and +inf too: such an expert comes last
      }
      c[i] = s;
      key[i] = e0 + i < E ? key_of(a.bias != nullptr ? s : l[i]) : 0u;
    }
    if (a.groups > 1) {
      float* chf = reinterpret_cast<float*>(ch);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (e0 + i < E) chf[e0 + i] = c[i];
      __syncwarp();
      const uint32_t kept = keep_groups(a, chf, lane, &close);
      __syncwarp();
      const int S = E / a.groups;
      int g = e0 / S, left = S - e0 % S;     // this lane's experts run through the groups in order
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (!((kept >> (g & 31)) & 1u)) key[i] = 0u;
        if (--left == 0) { ++g; left = S; }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = e0 + i < E ? key_of(l[i]) : 0u;
  }
  int id = 0;
  if (!close) id = rank_keys<T, PER>(a, logits, key, m, sum, lane, &close);
  if (close) id = route_exactly<T>(a, logits, ch, m, lane);
  // weights of the chosen, from their logits again
  const bool mine = lane < a.top_k;
  float w = mine ? score_of<float>(a.softmax, clean(route_f32(logits[id])), m, sum) : 0.f;
  if (a.renormalise) {
    const float all = warp_sum(w);
    w = all > 0.f ? w / all : 0.f;
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
  if (warp < kPlaceWarps)
    for (long long s = b; s < e; s += 32) {
      const int id = s + lane < e ? a.ids[s + lane] : -1;
      const uint32_t same = __match_any_sync(kFull, id);
      if (id >= 0 && (same & ((1u << lane) - 1u)) == 0) at[warp * E + id] += __popc(same);
      __syncwarp();
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
    for (long long s = b; s < e; s += 32) {
      const int id = s + lane < e ? a.ids[s + lane] : -1;
      const uint32_t same = __match_any_sync(kFull, id);
      const uint32_t before = same & ((1u << lane) - 1u);
      int first = 0;
      if (id >= 0) first = at[warp * E + id];
      __syncwarp();
      if (id >= 0) {
        a.order[first + __popc(before)] = (int)(s + lane);
        if (before == 0) at[warp * E + id] = first + __popc(same);
      }
      __syncwarp();
    }
}

template <int PER>
constexpr int route_threads() { return PER <= 8 ? 1024 : 256; }

// Block b routes tokens [b*chunk, (b+1)*chunk).  One block alone also places them.
template <typename T, int PER>
__global__ void __launch_bounds__(route_threads<PER>()) route_kernel(const RouteArgs a, int chunk) {
  extern __shared__ double route_smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32, E = a.experts;
  const int wide = a.choices ? E : 0;
  double* ch = route_smem + (size_t)warp * wide;
  int* hist = reinterpret_cast<int*>(route_smem + (size_t)warps * wide);
  const bool plan = a.offsets != nullptr;
  if (plan)
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  griddep_wait();
  __syncthreads();
  const long long t0 = (long long)blockIdx.x * chunk;
  const long long t1 = t0 + chunk < a.tokens ? t0 + chunk : a.tokens;
  for (long long t = t0 + warp; t < t1; t += warps) route_token<T, PER>(a, t, ch, plan ? hist : nullptr, lane);
  if (!plan) return;
  __syncthreads();
  if (gridDim.x > 1) {
    griddep_launch_dependents();
    for (int e = threadIdx.x; e < E; e += blockDim.x) a.counts[(size_t)blockIdx.x * E + e] = hist[e];
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

// The same blocks' slots, placed: counts of all blocks and of those before.
__global__ void __launch_bounds__(kPlaceThreads) route_place_kernel(const RouteArgs a, int chunk) {
  extern __shared__ int place_smem[];
  const int E = a.experts, lane = threadIdx.x % 32;
  int *total = place_smem, *before = total + E, *at = before + E;
  for (int x = threadIdx.x; x < (2 + kPlaceWarps) * E; x += blockDim.x) place_smem[x] = 0;
  griddep_wait();
  __syncthreads();
  // columns of 32 experts by warps: each warp takes a column's rows in turn with the others
  const int warp = threadIdx.x / 32, blocks = gridDim.x, columns = (E + 31) / 32;
  const int share = columns >= kPlaceWarps ? 1 : kPlaceWarps / columns;     // warps of a column
  for (int c = warp / share; c < columns; c += kPlaceWarps / share) {
    const int e = c * 32 + lane;
    int all = 0, mine = 0;
    if (e < E)
#pragma unroll 16
      for (int b = warp % share; b < blocks; b += share) {
        const int n = __ldcg(a.counts + (size_t)b * E + e);
        all += n;
        mine += b < (int)blockIdx.x ? n : 0;
      }
    if (e < E) {
      atomicAdd(total + e, all);            // whole numbers: any order gives the same sum
      atomicAdd(before + e, mine);
    }
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int all = warp_scan(total, total, E, lane);
    if (blockIdx.x == 0) {
      for (int e = lane; e < E; e += 32) a.offsets[e] = total[e];
      if (lane == 0) a.offsets[E] = all;
    }
    for (int e = lane; e < E; e += 32) before[e] += total[e];
  }
  __syncthreads();
  const long long t0 = (long long)blockIdx.x * chunk;
  const long long t1 = t0 + chunk < a.tokens ? t0 + chunk : a.tokens;
  place_slots(a, t0 * a.top_k, t1 * a.top_k, before, at);
}

// Blocks and tokens a block.  One block where its warps have at most four tokens each
// (a second launch costs 2 to 3 us, four tokens a warp about as much); else up to a block
// of 32 warps, or four of 8, on each of a GB300's 152 SMs.
struct RoutePlan {
  int blocks, chunk;
};
RoutePlan plan_route(int tokens, int experts) {
  const int warps = experts <= 256 ? 32 : 8;
  const int most = experts <= 256 ? 152 : 608;
  RoutePlan p;
  if (tokens <= 4 * warps) {
    p.blocks = 1;
    p.chunk = tokens;
    return p;
  }
  const long long want = ((long long)tokens + warps - 1) / warps;
  const int blocks = want < most ? (int)want : most;
  p.chunk = (tokens + blocks - 1) / blocks;
  p.blocks = (tokens + p.chunk - 1) / p.chunk;
  return p;
}

template <typename T, int PER>
int launch_impl(const RouteArgs& a, cudaStream_t s) {
  const RoutePlan p = plan_route(a.tokens, a.experts);
  const int threads = route_threads<PER>();
  const size_t smem = (size_t)(threads / 32) * (a.choices ? a.experts : 0) * sizeof(double) +
                      (size_t)a.experts * (1 + kPlaceWarps) * sizeof(int);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_smem_once(done, route_kernel<T, PER>,
                                (int)((threads / 32) * 32 * PER * sizeof(double) + 32 * PER * (1 + kPlaceWarps) * sizeof(int)));
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
  cfg.blockDim = dim3(kPlaceThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)a.experts * (2 + kPlaceWarps) * sizeof(int);
  return cudaLaunchKernelEx(&cfg, route_place_kernel, a, p.chunk);
}

template <typename T>
int launch_type(const RouteArgs& a, cudaStream_t s) {
  if (a.experts <= 32) return launch_impl<T, 1>(a, s);
  if (a.experts <= 64) return launch_impl<T, 2>(a, s);
  if (a.experts <= 128) return launch_impl<T, 4>(a, s);
  if (a.experts <= 256) return launch_impl<T, 8>(a, s);
  if (a.experts <= 512) return launch_impl<T, 16>(a, s);
  return launch_impl<T, 32>(a, s);
}

}  // namespace

size_t route_ws_bytes(int tokens, int experts) {
  const RoutePlan p = plan_route(tokens, experts);
  return p.blocks > 1 ? (size_t)p.blocks * experts * sizeof(int) : 0;
}

int launch_route(const RouteArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_type<__nv_bfloat16>(a, s) : launch_type<float>(a, s);
}

}  // namespace g3

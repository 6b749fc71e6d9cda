// Sampling one token of each row of logits (gemm_sample_*; the header states the
// rules).
//
// Weights become whole numbers, mass = floor(2^40 w), so every sum below is exact
// and does not depend on the order in which threads add: histograms may use
// atomics, and the token is the same on every run, for every split of the row and in
// every kernel here.  Both cuts (top-k by count, top-p by mass) are prefixes of the
// ranking, so each is a place in it: a key (the logit's bits in order) and an index.
// No row is sorted as a whole.
//
// A draw reads its row once (HBM: 2 or 4 bytes a token) and computes little, so what
// it takes is the latency of its steps.  Three kernels:
//   * sample_cluster_kernel: a cluster of up to eight blocks holds a row in shared
//     memory.  Up to 64 ranks: candidates that a bound from the groups' largest lets
//     through, ranked in one warp.  Longer top-k, and top-p alone: a list of up to 2048
//     candidates in the first block, cut and drawn by histograms.  What does not fit:
//     a search by histograms over the cluster.
//   * sample_stream_kernel: many rows with up to 64 ranks, a block or a few a row.
//   * sample_kernel: rows beyond the cluster's shared memory (360448), radix searches
//     over global memory by one block a row: 8 rows of 2^20 bf16 0.76 ms greedy, 16 ms
//     with top-k and top-p (a pass of the row for each of eight digits and more).
// Measured on one GB300, GPU time: one row of 32000 with top-k 50, top-p and min-p
// 9 us; 64 rows of 32000 bf16: the same settings 11 us, top-k 1000 with top-p 25 us,
// top-p alone 21 to 35 us (flat rows need the search), no cut 13 us; 384 rows of
// 131071 fp32 (201 MB): 61 us, 3.3 TB/s, against 141 us by the cluster kernel.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cstddef>

#include "internal.h"
#include "ptx.cuh"

namespace g3 {
namespace {

using ull = unsigned long long;
constexpr int THREADS = 1024, WARPS = THREADS / 32;
constexpr uint32_t kKeyNegInf = 0x007fffffu;   // order_key(-inf), the lowest key
constexpr int kNotDone = -2;                   // token of a row that sample_stream_kernel gives up

// A logit as an unsigned number in the same order; NaN counts as -inf and -0 as 0
__device__ __forceinline__ uint32_t order_key(float l) {
  if (l != l) l = -INFINITY;
  const uint32_t u = __float_as_uint(l + 0.f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float((key >> 31) ? key & 0x7fffffffu : ~key);
}

// z and w of a logit
struct Row {
  float top, inv_t;
};
__device__ __forceinline__ float logit_z(const Row& r, float l) {
  return r.top == INFINITY ? (l == INFINITY ? 0.f : -INFINITY) : __fmul_rn(__fsub_rn(l, r.top), r.inv_t);
}
__device__ __forceinline__ float logit_weight(const Row& r, float l) {
  const float w = expf(logit_z(r, l));
  return l > -INFINITY && w == w ? w : 0.f;   // -inf never, whatever the temperature
}
// floor(2^40 w) for 0 <= w <= 1, from w's own bits: 24 of them, shifted by its exponent
// (the conversion instruction to 64 bits is slow)
__device__ __forceinline__ ull mass_of(float w) {
  const uint32_t u = __float_as_uint(w);
  const int e = (int)(u >> 23) - (127 + 23 - 40);            // the last bit's place
  const uint32_t f = (u & 0x7fffffu) | 0x800000u;
  return e >= 0 ? (ull)f << e : e > -24 ? (ull)(f >> -e) : 0;   // subnormals are far below 2^-40
}

// What is kept: keys above `key`, and the first `ties` (by index) equal to it
struct Cut {
  uint32_t key;
  int ties;
};

// The smallest whole number x with double(x) >= bound, so that m < x just when
// double(m) < bound: one conversion in place of one a token (fp64 is slow here).
__device__ __forceinline__ ull whole_bound(double bound) {
  if (!(bound > 0.0)) return 0;
  if (bound >= 0x1p63) return ~0ull;
  ull x = __double2ull_ru(bound);
  // from 2^53 on, numbers a little below may round up to the bound
  while (x > 0 && __ull2double_rn(x - 1) >= bound) --x;
  return x;
}
// floor(u * total) within 0 .. total - 1; u NaN or negative: 0
__device__ __forceinline__ ull draw_target(float u, ull total) {
  const double at = __dmul_rn((double)u, __ull2double_rn(total));
  const ull target = at > 0.0 ? __double2ull_rz(at) : 0;
  return target < total ? target : total - 1;
}

struct Shared {
  ull mass[256];
  unsigned count[256];
  ull warp_mass[WARPS];
  unsigned warp_count[WARPS];
  ull above;
  unsigned above_n;
  unsigned digit;
  Cut cut;
  int token;
};

template <typename T>
struct Logits {
  const T* p;
  __device__ __forceinline__ float operator()(int i) const {
    if constexpr (sizeof(T) == 2) return __bfloat162float(p[i]);
    else return p[i];
  }
};

// The lowest key present among keys >= floor_key for which `before` (the count or
// the mass of all larger keys) still satisfies keep(); returns it with the count
// and mass above it and its own count.  keep(count, mass) must hold for (0, 0).
template <class L, class Keep>
__device__ uint32_t search(const L& logit, int vocab, const Row& row, uint32_t floor_key, Keep keep, Shared& sh,
                           unsigned& n_above, ull& m_above, unsigned& n_equal) {
  uint32_t prefix = 0, mask = 0;
  n_above = 0;
  m_above = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    __syncthreads();
    if (threadIdx.x < 256) {
      sh.mass[threadIdx.x] = 0;
      sh.count[threadIdx.x] = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < vocab; i += THREADS) {
      const float l = logit(i);
      const uint32_t key = order_key(l);
      if (key >= floor_key && (key & mask) == prefix) {
        const unsigned d = (key >> shift) & 255u;
        atomicAdd(&sh.count[d], 1u);
        const ull m = mass_of(logit_weight(row, l));
        if (m) atomicAdd(&sh.mass[d], m);
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned c = n_above;
      ull m = m_above;
      int best = -1;
      unsigned bc = 0;
      ull bm = 0;
      for (int d = 255; d >= 0; --d) {
        if (sh.count[d] == 0) continue;
        if (!keep(c, m)) break;
        best = d;
        bc = c;
        bm = m;
        c += sh.count[d];
        m += sh.mass[d];
      }
      sh.digit = (unsigned)best;
      sh.above_n = bc;
      sh.above = bm;
    }
    __syncthreads();
    prefix |= sh.digit << shift;
    mask |= 255u << shift;
    n_above = sh.above_n;
    m_above = sh.above;
    n_equal = sh.count[sh.digit];
  }
  __syncthreads();
  return prefix;
}

template <typename T>
__global__ void __launch_bounds__(THREADS) sample_kernel(const SampleArgs a) {
  __shared__ Shared sh;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int r = blockIdx.x, vocab = a.vocab, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const Logits<T> logit{static_cast<const T*>(a.logits) + (long long)r * a.ld};
  const float t = a.temperature ? a.temperature[r] : 1.f;
  const int k = a.top_k ? a.top_k[r] : 0;
  const float p = a.top_p ? a.top_p[r] : 1.f;
  const float least = a.min_p ? a.min_p[r] : 0.f;
  const float u = a.u[r];
  // only the first rank: also where no weight, 1 at most, can reach min_p
  const bool greedy = !(t >= FLT_MIN) || k == 1 || !(least <= 1.f);

  // the largest key and the first index that has it
  uint32_t top = 0;
  for (int i = threadIdx.x; i < vocab; i += THREADS) top = max(top, order_key(logit(i)));
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) sh.warp_count[warp] = top;
  __syncthreads();
  for (int w = 0; w < WARPS; ++w) top = max(top, sh.warp_count[w]);
  __syncthreads();
  if (top <= kKeyNegInf) {   // nothing can be taken
    if (threadIdx.x == 0) {
      a.token[r] = -1;
      if (a.logprob) a.logprob[r] = -INFINITY;
    }
    return;
  }
  const Row row{key_logit(top), __fdiv_rn(1.f, t >= FLT_MIN ? t : 1.f)};

  // cuts; key 0 keeps everything
  Cut cut{0u, vocab};
  unsigned n_above = 0, n_equal = 0;
  ull m_above = 0;
  if (greedy) {
    cut = Cut{top, 1};
  } else {
    if (k > 0 && k < vocab) {
      const uint32_t key = search(logit, vocab, row, 0u, [&](unsigned c, ull) { return c < (unsigned)k; }, sh, n_above,
                                  m_above, n_equal);
      cut = Cut{key, (int)((unsigned)k - n_above)};
    }
    if (!(p >= 1.f)) {
      // the mass that top-k kept
      ull m = 0;
      for (int i = threadIdx.x; i < vocab; i += THREADS) {
        const float l = logit(i);
        if (order_key(l) > cut.key) m += mass_of(logit_weight(row, l));
      }
      for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
      if (lane == 0) sh.warp_mass[warp] = m;
      __syncthreads();
      m = 0;
      for (int w = 0; w < WARPS; ++w) m += sh.warp_mass[w];
      if (cut.key > kKeyNegInf) m += (ull)cut.ties * mass_of(logit_weight(row, key_logit(cut.key)));
      const ull bound = whole_bound(__dmul_rn((double)p, __ull2double_rn(m)));
      const uint32_t key = search(logit, vocab, row, cut.key, [&](unsigned c, ull before) {
        return c == 0 || before < bound;
      }, sh, n_above, m_above, n_equal);
      // how many of the equal ones have less than the bound before them
      const ull one = key > kKeyNegInf ? mass_of(logit_weight(row, key_logit(key))) : 0;
      int lo = 1, hi = (int)n_equal;
      if (key == cut.key) hi = min(hi, cut.ties);
      while (lo < hi) {   // the first always; the j-th (from 0) if before + j * one is below
        const int mid = (lo + hi + 1) / 2;
        if (m_above + (ull)(mid - 1) * one < bound) lo = mid;
        else hi = mid - 1;
      }
      cut = Cut{key, lo};
    }
  }

  // each warp holds a contiguous part of the row, so that parts are in index order
  const int part = (vocab + WARPS - 1) / WARPS, from = min(vocab, warp * part), to = min(vocab, from + part);
  unsigned ties = 0;
  for (int i0 = from; i0 < to; i0 += 32) {
    const int i = i0 + lane;
    ties += __popc(__ballot_sync(0xffffffffu, i < to && order_key(logit(i)) == cut.key));
  }
  if (lane == 0) sh.warp_count[warp] = ties;
  __syncthreads();
  unsigned ties_before = 0;
  for (int w = 0; w < warp; ++w) ties_before += sh.warp_count[w];
  // mass kept of each element of this warp's part, in index order
  auto kept = [&](int i0, unsigned& seen) -> ull {
    const int i = i0 + lane;
    const float l = i < to ? logit(i) : -INFINITY;
    const uint32_t key = i < to ? order_key(l) : 0u;
    const unsigned eq = __ballot_sync(0xffffffffu, i < to && key == cut.key);
    const bool in = key > cut.key || (i < to && key == cut.key &&
                                      seen + __popc(eq & ((1u << lane) - 1u)) < (unsigned)cut.ties);
    seen += __popc(eq);
    if (!in) return 0;
    const float w = logit_weight(row, l);
    return w >= least || greedy ? mass_of(w) : 0;
  };
  ull m = 0;
  unsigned seen = ties_before;
  for (int i0 = from; i0 < to; i0 += 32) m += kept(i0, seen);
  for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
  if (lane == 0) sh.warp_mass[warp] = m;
  __syncthreads();
  ull total = 0, before = 0;
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += sh.warp_mass[w];
    total += sh.warp_mass[w];
  }
  const ull target = draw_target(u, total);
  if (before <= target && target < before + m) {     // one warp holds the token
    seen = ties_before;
    for (int i0 = from; i0 < to; i0 += 32) {
      const ull x = kept(i0, seen);
      ull run = x;
      for (int o = 1; o < 32; o <<= 1) {
        const ull y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + run > target);
      if (past) {
        if (lane == __ffs(past) - 1) {
          const int i = i0 + lane;
          a.token[r] = i;
          // greedy: T is one token's mass, and z is 0
          if (a.logprob) a.logprob[r] = logit_z(row, logit(i)) - logf(__ull2float_rn(total) * 0x1p-40f);
        }
        break;
      }
      before += __shfl_sync(0xffffffffu, run, 31);
    }
  }
}


// ------------------------------------------------------------------ a row in a cluster
// A cluster of C blocks holds a row as keys in shared memory, a warp's 128 * Q next to
// one another (so that warps, then blocks, are in index order).  The logits are read
// once; everything after that works on the keys, with one histogram or list and a
// few exchanges over the cluster.  Quad q of a lane holds the keys of indices
// base + (4 q + k) * 32 + lane, k = 0 .. 3.
constexpr int FT = 512, FW = FT / 32;         // threads and warps of a block
constexpr int MAX_C = 8;
constexpr int MAX_Q = 22;                     // quads of a thread: 8 * FT * 88 logits, 180 KB of keys
constexpr int LIST = 2048;                    // candidates that the first block can sort
constexpr int LOCAL = 2048;                   // room for a list's copies
constexpr int SMALL_K = 64;                   // largest top_k whose ranks fit two to a lane of one warp
constexpr int SEG = LIST / MAX_C;             // a block's part of the list then
constexpr int TOP_K_LIST = 1024;              // ranks that the first block can draw from: two a thread
constexpr int SAMPLE_Q = 4;                   // quads of a thread before a row takes more blocks
constexpr int STREAM_LONG = 160;              // length from which a list's own bound is taken, see its use
constexpr int STREAM_PART = 15000;            // logits of a row that are worth a block, see its use
constexpr float ZERO_Z = 28.f;                // expf(-28) < 2^-40: no mass

// Bins a unit of the logit, for FT bins even in it.  No range, or an infinite one: all in
// one bin.  Below 1.5e-36 the quotient would be infinite, and a bin's lower edge the
// range's upper end; held to the largest number, fewer bins cover the range.
__device__ __forceinline__ float bins_over(float range) {
  static_assert(FT == 512, "bins");
  return range > 0.f && range < INFINITY ? fminf(511.9f / range, FLT_MAX) : 0.f;
}

// A cut by rank: kept are larger keys, and equal ones up to index idx
struct Place {
  uint32_t key;
  int idx;
  __device__ __forceinline__ bool keeps(uint32_t k, int i) const { return k > key || (k == key && i <= idx); }
};

struct alignas(16) Cluster {
  union {
    // the search's histograms by turns: one is read by the cluster while the other fills
    struct {
      unsigned count[2][FT], mass[2][3][FT];
    };
    ull local[LOCAL];       // copies of a list
  };
  unsigned bins[FT];        // the threshold's histogram
  ull list[LIST];           // first block: candidates, key << 32 | ~index
  ull all[MAX_C * FW];      // every warp's kept mass
  ull warp_mass[FW], warp_above[FW];   // read by the cluster
  unsigned warp_count[FW];  // read by the cluster
  unsigned red[2][FW];
  unsigned top, low, bound_key;   // read by the cluster
  float group_mass[FW], block_mass;   // the latter too
  unsigned lo[2], hi[2];    // read by the cluster, by turns
  unsigned seg_n[MAX_C];    // first block: of each block, in parts of the list
  ull few[SMALL_K];         // the first ranks
  ulonglong2 few_mass[SMALL_K];   // index, mass
  unsigned local_n, local_at;
  unsigned best, n_above;
  ull m_above, bound;
  ull scan_m[FW];
  unsigned scan_c[FW];
  Place cut;                // first block's, or the tie's owner's: read by the cluster
};

__device__ __forceinline__ void sync_cluster(int C) {
  if (C == 1) __syncthreads();
  else cluster_sync();
}
// `p` of this block's shared memory, in block r of the cluster
template <typename T>
__device__ __forceinline__ T* in_block(T* p, int r) {
  uint64_t out;
  asm("mapa.u64 %0, %1, %2;" : "=l"(out) : "l"(reinterpret_cast<uint64_t>(p)), "r"(r));
  return reinterpret_cast<T*>(out);
}

// Sums of all lower threads' values over the block; `c` and `m` become exclusive
// prefixes.  Ends with shared memory free for the next call after a barrier.
__device__ __forceinline__ void block_prefix(Cluster& sh, unsigned& c, ull& m) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const unsigned c0 = c;
  const ull m0 = m;
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned x = __shfl_up_sync(0xffffffffu, c, o);
    const ull y = __shfl_up_sync(0xffffffffu, m, o);
    if (lane >= o) {
      c += x;
      m += y;
    }
  }
  if (lane == 31) {
    sh.scan_c[warp] = c;
    sh.scan_m[warp] = m;
  }
  __syncthreads();
  c -= c0;
  m -= m0;
  for (int w = 0; w < warp; ++w) {
    c += sh.scan_c[w];
    m += sh.scan_m[w];
  }
}

// Sorts list[0 .. n2), largest first: E values a thread in registers, neighbours; steps
// within a thread, within a warp by shuffles, others through shared memory.  The
// warps that hold values.
template <int E>
__device__ __forceinline__ void sort_values(Cluster& sh, int n2) {
  const int tid = threadIdx.x, threads = n2 / E;
  ull x[E];
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = sh.list[tid * E + e];
  // of a pair in a descending run the lower place keeps the larger value
  auto keep = [](ull& v, ull other, bool larger) { v = (v < other) == larger ? other : v; };
  for (int size = 2; size <= n2; size <<= 1)
    for (int step = size >> 1; step > 0; step >>= 1) {
      if (step < E) {
        ull y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const ull z1 = x[e ^ 1], z2 = E > 2 ? x[(e ^ 2) % E] : z1;
          y[e] = step == 1 ? z1 : z2;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) keep(x[e], y[e], ((e & step) == 0) == (((tid * E + e) & size) == 0));
      } else if (step < 32 * E) {
        const bool larger = ((tid * E & step) == 0) == ((tid * E & size) == 0);
#pragma unroll
        for (int e = 0; e < E; ++e) keep(x[e], __shfl_xor_sync(0xffffffffu, x[e], step / E), larger);
      } else {
        const bool larger = ((tid * E & step) == 0) == ((tid * E & size) == 0);
        asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");   // the last step's values have been read
#pragma unroll
        for (int e = 0; e < E; ++e) sh.local[e * threads + tid] = x[e];
        asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
#pragma unroll
        for (int e = 0; e < E; ++e) keep(x[e], sh.local[e * threads + (tid ^ (step / E))], larger);
      }
    }
#pragma unroll
  for (int e = 0; e < E; ++e) sh.list[tid * E + e] = x[e];
}
// n2 a power of two, 64 .. LIST; whole block
__device__ __forceinline__ void sort_list(Cluster& sh, int n2) {
  static_assert(LIST == 4 * FT && LOCAL >= LIST, "four values a thread");
  const int tid = threadIdx.x;
  if (n2 <= FT) {
    if (tid < n2) sort_values<1>(sh, n2);
  } else if (n2 <= 2 * FT) {
    sort_values<2>(sh, n2);
  } else {
    sort_values<4>(sh, n2);
  }
  __syncthreads();
}

// Zeros behind the list's first m entries, up to a power of two, which is returned
__device__ __forceinline__ int pad_list(Cluster& sh, int m) {
  int n2 = 64;
  while (n2 < m) n2 <<= 1;
  for (int i = m + threadIdx.x; i < n2; i += FT) sh.list[i] = 0;
  __syncthreads();
  return n2;
}

// The draw where the first block's list holds every token that can be kept, the list
// sorted by rank for both cuts, then by index for the draw.  `mass`: what top-p takes
// its share of, 0 for the mass of the k first.  Entries of 0 are no tokens.
__device__ __forceinline__ void draw_by_sorting(const SampleArgs& a, Cluster& sh, int r, int n, int k, float p,
                                                float least, float u, float t, ull mass) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  constexpr int PER = LIST / FT;                     // places of a thread
  sort_list(sh, pad_list(sh, n));
  const unsigned top = (unsigned)(sh.list[0] >> 32);
  const Row row{key_logit(top), __fdiv_rn(1.f, t)};
  int kept = min(n, k);
  auto totals = [&]() {
    ull total = 0;
    for (int w = 0; w < FW; ++w) total += sh.scan_m[w];
    return total;
  };
  if (!(p >= 1.f)) {
    ull m[PER], before = 0;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int i = tid * PER + q;
      m[q] = i < kept ? mass_of(logit_weight(row, key_logit((unsigned)(sh.list[i] >> 32)))) : 0;
      before += m[q];
    }
    unsigned none = 0;
    block_prefix(sh, none, before);
    if (warp == 0) {
      const ull x = whole_bound(__dmul_rn((double)p, __ull2double_rn(mass ? mass : totals())));
      if (lane == 0) sh.m_above = x;
    }
    __syncthreads();
    const ull bound = sh.m_above;
    int ranks = 0;                                   // of this thread that top-p keeps
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int i = tid * PER + q;
      if (i < kept && (i == 0 || before < bound)) ranks = i + 1;
      before += m[q];
    }
    ranks = __reduce_max_sync(0xffffffffu, ranks);
    if (lane == 0) sh.red[0][warp] = ranks;
    __syncthreads();
    for (int w = 0; w < FW; ++w) ranks = max(ranks, (int)sh.red[0][w]);
    kept = ranks;
  }
  // by index: ~index << 32 | key, largest first
  __syncthreads();                                   // list[0] has been read
  for (int i = tid; i < kept; i += FT) {
    const ull x = sh.list[i];
    sh.list[i] = (x << 32) | (x >> 32);
  }
  sort_list(sh, pad_list(sh, kept));
  ull m[PER], before = 0;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int i = tid * PER + q;
    m[q] = 0;
    if (i < kept) {
      const unsigned key = (unsigned)sh.list[i];
      const float w = logit_weight(row, key_logit(key));
      if (w >= least) m[q] = mass_of(w);
    }
    before += m[q];
  }
  unsigned none = 0;
  block_prefix(sh, none, before);
  const ull total = totals();
  if (warp == 0) {
    const ull x = draw_target(u, total);
    if (lane == 0) sh.m_above = x;
  }
  __syncthreads();
  const ull target = sh.m_above;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    if (before <= target && target < before + m[q]) {
      const ull x = sh.list[tid * PER + q];
      a.token[r] = (int)~(unsigned)(x >> 32);
      if (a.logprob)
        a.logprob[r] = logit_z(row, key_logit((unsigned)x)) - logf(__ull2float_rn(total) * 0x1p-40f);
    }
    before += m[q];
  }
}

// The bin of sh.bins in which the k-th count is, FT if there are fewer; one warp
__device__ __forceinline__ unsigned kth_bin(const Cluster& sh, int k) {
  constexpr int PER = FT / 32;
  const int lane = threadIdx.x % 32;
  unsigned c[PER], own = 0;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    c[q] = sh.bins[lane * PER + q];
    own += c[q];
  }
  unsigned before = own;
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  before -= own;
  unsigned best = FT;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    if (before < (unsigned)k && before + c[q] >= (unsigned)k) best = lane * PER + q;
    before += c[q];
  }
  return __reduce_min_sync(0xffffffffu, best);
}

// The same without sorting, where no bin of the three histograms is crowded: the k-th
// rank and top-p's cut by bins even in the logit, the draw by bins even in the index;
// the tokens of the bin in question are compared with one another.  Where a bin is
// crowded, the cuts before it stand: what they drop is 0 in the list.
constexpr int EDGE = 512;                            // tokens of a bin that are compared
enum class Bins { drawn, crowded, cut_and_crowded }; // the last: top-p is in the list already

__device__ __forceinline__ Bins draw_by_bins(const SampleArgs& a, Cluster& sh, int r, int n, int k, float p, float least,
                                             float u, float t, ull mass) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  // the tokens of the bin in question and their masses lie in the unused parts of the
  // histograms' memory
  unsigned (*hist)[FT] = sh.mass[0];                 // three words, as in the search
  ull* edge = reinterpret_cast<ull*>(&sh.mass[1][0][0]);
  ull* edge_mass = reinterpret_cast<ull*>(&sh.count[0][0]);
  static_assert(sizeof(sh.count) >= EDGE * 8 && sizeof(sh.mass[1]) >= EDGE * 8 && offsetof(Cluster, mass) % 8 == 0 &&
                    sizeof(sh.mass[0]) % 8 == 0, "edge");
  unsigned hi = 0, lo = 0xffffffffu;
  for (int i = tid; i < n; i += FT) {
    const unsigned key = (unsigned)(sh.list[i] >> 32);
    hi = max(hi, key);
    lo = min(lo, key);
  }
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (lane == 0) {
    sh.red[0][warp] = hi;
    sh.red[1][warp] = lo;
  }
  sh.bins[tid] = 0;
  for (int w = 0; w < 3; ++w) hist[w][tid] = 0;
  __syncthreads();
  const unsigned top = __reduce_max_sync(0xffffffffu, sh.red[0][lane % FW]);
  lo = __reduce_min_sync(0xffffffffu, sh.red[1][lane % FW]);
  const Row row{key_logit(top), __fdiv_rn(1.f, t)};
  const float scale = bins_over(row.top - key_logit(lo));
  auto bin = [&](ull x) { return min(FT - 1, (int)((row.top - key_logit((unsigned)(x >> 32))) * scale)); };
  auto mass_at = [&](ull x) { return mass_of(logit_weight(row, key_logit((unsigned)(x >> 32)))); };
  auto add = [&](int b, ull m) {
    atomicAdd(&hist[0][b], (unsigned)m & 0x3fffu);
    atomicAdd(&hist[1][b], (unsigned)(m >> 14) & 0x1fffu);
    if (m >> 27) atomicAdd(&hist[2][b], (unsigned)(m >> 27));
  };
  auto sum = [&](int b) { return (ull)hist[0][b] + ((ull)hist[1][b] << 14) + ((ull)hist[2][b] << 27); };
  // f(entry, place) for this thread's entries
  auto each = [&](auto f) {
    for (int i = tid; i < n; i += FT)
      if (sh.list[i]) f(sh.list[i], i);
  };

  // ---- the k-th rank
  if (n > k) {
    each([&](ull x, int) { atomicAdd(&sh.bins[bin(x)], 1u); });
    __syncthreads();
    unsigned c = sh.bins[tid];
    const unsigned own = c;
    ull none = 0;
    block_prefix(sh, c, none);
    if (c < (unsigned)k && c + own >= (unsigned)k) {
      sh.best = tid;
      sh.n_above = c;
    }
    if (tid == 0) sh.local_n = 0;
    __syncthreads();
    const int best = (int)sh.best, above = (int)sh.n_above;
    if (sh.bins[best] > EDGE) return Bins::crowded;
    each([&](ull x, int i) {
      const int b = bin(x);
      if (b == best) edge[atomicAdd(&sh.local_n, 1u)] = x;
      if (b > best) sh.list[i] = 0;
    });
    __syncthreads();
    const int m = (int)sh.local_n;
    each([&](ull x, int i) {
      if (bin(x) != best) return;
      int rank = above;
      for (int j = 0; j < m; ++j) rank += edge[j] > x;
      if (rank >= k) sh.list[i] = 0;
    });
    __syncthreads();
    sh.bins[tid] = 0;
    __syncthreads();
  }

  // ---- top-p
  if (!(p >= 1.f)) {
    each([&](ull x, int) {
      const ull m = mass_at(x);
      const int b = bin(x);
      if (m) add(b, m);
      atomicAdd(&sh.bins[b], 1u);
    });
    __syncthreads();
    const ull own = sum(tid);
    ull before = own;
    unsigned none = 0;
    block_prefix(sh, none, before);
    if (warp == 0) {
      ull total = mass;
      if (total == 0)
        for (int w = 0; w < FW; ++w) total += sh.scan_m[w];
      const ull x = whole_bound(__dmul_rn((double)p, __ull2double_rn(total)));
      if (lane == 0) sh.bound = x;
    }
    if (tid == 0) {
      sh.best = 0;
      sh.local_n = 0;
    }
    __syncthreads();
    const ull bound = sh.bound;
    if (own && (before == 0 || before < bound)) atomicMax(&sh.best, (unsigned)tid);
    __syncthreads();
    const int best = (int)sh.best;
    if (tid == best) sh.m_above = before;
    __syncthreads();
    if (sh.bins[best] > EDGE) return Bins::crowded;
    each([&](ull x, int i) {
      const int b = bin(x);
      if (b == best) {
        const unsigned at = atomicAdd(&sh.local_n, 1u);
        edge[at] = x;
        edge_mass[at] = mass_at(x);
      }
      if (b > best) sh.list[i] = 0;
    });
    __syncthreads();
    const int m = (int)sh.local_n;
    const ull above = sh.m_above;
    each([&](ull x, int i) {
      if (bin(x) != best) return;
      ull y = above;
      for (int j = 0; j < m; ++j) y += edge[j] > x ? edge_mass[j] : 0;
      if (y != 0 && y >= bound) sh.list[i] = 0;
    });
    __syncthreads();
    sh.bins[tid] = 0;
    for (int w = 0; w < 3; ++w) hist[w][tid] = 0;
    __syncthreads();
  }

  // ---- min-p, and the draw in index order
  const int width = (a.vocab + FT - 1) / FT;
  auto place = [&](ull x) { return (int)((unsigned)~(unsigned)x / (unsigned)width); };
  auto kept = [&](ull x) -> ull {
    const float w = logit_weight(row, key_logit((unsigned)(x >> 32)));
    return w >= least ? mass_of(w) : 0;
  };
  each([&](ull x, int) {
    const ull m = kept(x);
    if (m == 0) return;
    add(place(x), m);
    atomicAdd(&sh.bins[place(x)], 1u);
  });
  __syncthreads();
  const ull own = sum(tid);
  ull before = own;
  unsigned none = 0;
  block_prefix(sh, none, before);
  ull total = 0;
  for (int w = 0; w < FW; ++w) total += sh.scan_m[w];
  if (warp == 0) {
    const ull x = draw_target(u, total);
    if (lane == 0) sh.bound = x;
  }
  if (tid == 0) sh.local_n = 0;
  __syncthreads();
  const ull target = sh.bound;
  if (before <= target && target < before + own) {
    sh.best = tid;
    sh.m_above = before;
  }
  __syncthreads();
  const int best = (int)sh.best;
  if (sh.bins[best] > EDGE) return Bins::cut_and_crowded;
  each([&](ull x, int) {
    if (place(x) != best) return;
    const ull m = kept(x);
    if (m == 0) return;
    const unsigned at = atomicAdd(&sh.local_n, 1u);
    edge[at] = x;
    edge_mass[at] = m;
  });
  __syncthreads();
  const int m = (int)sh.local_n;
  for (int i = tid; i < m; i += FT) {
    const ull x = edge[i];
    const unsigned index = ~(unsigned)x;
    ull y = sh.m_above;
    for (int j = 0; j < m; ++j) y += ~(unsigned)edge[j] < index ? edge_mass[j] : 0;
    if (y <= target && target < y + edge_mass[i]) {
      a.token[r] = (int)index;
      if (a.logprob)
        a.logprob[r] = logit_z(row, key_logit((unsigned)(x >> 32))) - logf(__ull2float_rn(total) * 0x1p-40f);
    }
  }
  return Bins::drawn;
}

__device__ __forceinline__ void draw_from_list(const SampleArgs& a, Cluster& sh, int r, int n, int k, float p, float least,
                                               float u, float t, ull mass) {
  const Bins done = draw_by_bins(a, sh, r, n, k, p, least, u, t, mass);
  if (done == Bins::drawn) return;
  __syncthreads();
  // top-p's share is of the tokens before it cut: it must not cut again
  draw_by_sorting(a, sh, r, n, k, done == Bins::cut_and_crowded ? 1.f : p, least, u, t, mass);
}

// The same for k up to SMALL_K, with the candidates in the list's C parts: ranks by
// counting, then one warp with two ranks a lane.
__device__ __forceinline__ void draw_from_few(const SampleArgs& a, Cluster& sh, int r, int C, int k, float p, float least,
                              float u, float t) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  int n = 0;
  for (int c = 0; c < C; ++c) {
    const int m = (int)sh.seg_n[c];
    for (int i = tid; i < m; i += FT) sh.local[n + i] = sh.list[c * SEG + i];
    n += m;
  }
  __syncthreads();
  const ull* list = sh.local;
  if (n > FT / 4) {
    // far more than k of them: a histogram of all leaves the k first and their bin's
    unsigned hi = 0, lo = 0xffffffffu;
    for (int i = tid; i < n; i += FT) {
      const unsigned key = (unsigned)(list[i] >> 32);
      hi = max(hi, key);
      lo = min(lo, key);
    }
    hi = __reduce_max_sync(0xffffffffu, hi);
    lo = __reduce_min_sync(0xffffffffu, lo);
    if (lane == 0) {
      sh.red[0][warp] = hi;
      sh.red[1][warp] = lo;
    }
    if (tid == 0) sh.local_n = 0;
    __syncthreads();
    hi = __reduce_max_sync(0xffffffffu, sh.red[0][lane % FW]);
    lo = __reduce_min_sync(0xffffffffu, sh.red[1][lane % FW]);
    const float ltop = key_logit(hi), scale = bins_over(ltop - key_logit(lo));
    auto bin = [&](ull x) { return min(FT - 1, (int)((ltop - key_logit((unsigned)(x >> 32))) * scale)); };
    for (int i = tid; i < n; i += FT) atomicAdd(&sh.bins[bin(list[i])], 1u);
    __syncthreads();
    if (warp == 0) {
      const unsigned best = kth_bin(sh, k);
      if (lane == 0) sh.best = best;
    }
    __syncthreads();
    const int best = (int)sh.best;
    for (int i = tid; i < n; i += FT) {
      const ull x = list[i];
      if (bin(x) <= best) sh.list[atomicAdd(&sh.local_n, 1u)] = x;
    }
    __syncthreads();
    list = sh.list;
    n = (int)sh.local_n;
  }
  // P lanes count how many candidates are larger than one of them
  const int P = n <= FT / 16 ? 16 : n <= FT / 8 ? 8 : n <= FT / 4 ? 4 : n <= FT / 2 ? 2 : 1, part = tid % P;
  for (int i0 = 0; i0 < n; i0 += FT / P) {
    const int i = i0 + tid / P;
    const ull x = i < n ? list[i] : ~0ull;
    int larger = 0;
#pragma unroll 4
    for (int j = part; j < n; j += P) larger += list[j] > x;
    for (int o = 1; o < P; o <<= 1) larger += __shfl_xor_sync(0xffffffffu, larger, o);
    if (part == 0 && larger < k && i < n) sh.few[larger] = x;
  }
  __syncthreads();
  if (warp != 0) return;
  const int kept = min(n, k);
  const ull x[2] = {lane < kept ? sh.few[lane] : 0, lane + 32 < kept ? sh.few[lane + 32] : 0};
  const Row row{key_logit((unsigned)(sh.few[0] >> 32)), __fdiv_rn(1.f, t)};
  ull m[2];
  float z[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float l = key_logit((unsigned)(x[q] >> 32)), w = logit_weight(row, l);
    z[q] = logit_z(row, l);
    m[q] = x[q] == 0 ? 0 : mass_of(w);
  }
  auto prefix = [&](ull v) {                         // sum of the lower lanes' and this one's
    for (int o = 1; o < 32; o <<= 1) {
      const ull y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    return v;
  };
  int ranks = kept;
  if (!(p >= 1.f)) {
    const ull p0 = prefix(m[0]), all0 = __shfl_sync(0xffffffffu, p0, 31);
    const ull p1 = all0 + prefix(m[1]), total = __shfl_sync(0xffffffffu, p1, 31);
    const ull bound = whole_bound(__dmul_rn((double)p, __ull2double_rn(total)));
    ranks = __popc(__ballot_sync(0xffffffffu, lane < kept && (lane == 0 || p0 - m[0] < bound))) +
            __popc(__ballot_sync(0xffffffffu, lane + 32 < kept && p1 - m[1] < bound));
  }
  // min-p, and the running mass in index order
  ull sum = 0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = lane + 32 * q;
    if (i >= ranks || !(logit_weight(row, key_logit((unsigned)(x[q] >> 32))) >= least)) m[q] = 0;
    sh.few_mass[i] = make_ulonglong2((unsigned)~(unsigned)x[q], m[q]);
    sum += m[q];
  }
  __syncwarp();
  const ull total = __shfl_sync(0xffffffffu, prefix(sum), 31);
  const ull target = draw_target(u, total);
  ull before[2] = {0, 0};
#pragma unroll 4
  for (int j = 0; j < ranks; ++j) {
    const ulonglong2 y = sh.few_mass[j];
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if ((unsigned)y.x < (unsigned)~(unsigned)x[q]) before[q] += y.y;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q)
    if (before[q] <= target && target < before[q] + m[q]) {
      a.token[r] = (int)~(unsigned)x[q];
      if (a.logprob) a.logprob[r] = z[q] - logf(__ull2float_rn(total) * 0x1p-40f);
    }
}

template <typename T>
__device__ __forceinline__ void cluster_row(const SampleArgs& a, const int C, const int Q, const int r, const bool more) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Cluster& sh = *reinterpret_cast<Cluster*>(smem_raw);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  uint4* const keys = reinterpret_cast<uint4*>(smem_raw + sizeof(Cluster)) + warp * Q * 32 + lane;   // quad q at [q * 32]
  const int rank = C == 1 ? 0 : (int)cluster_ctarank();
  const int base = (rank * FW + warp) * 128 * Q + lane;   // index of key k of quad q: base + (4 q + k) * 32

  const float t_in = a.temperature ? a.temperature[r] : 1.f;
  const int k = a.top_k ? a.top_k[r] : 0;
  const float p = a.top_p ? a.top_p[r] : 1.f;
  const float least = a.min_p ? a.min_p[r] : 0.f;
  const float u = a.u[r];
  // only the first rank: also where no weight, 1 at most, can reach min_p
  const bool greedy = !(t_in >= FLT_MIN) || k == 1 || !(least <= 1.f);
  const float t = t_in >= FLT_MIN ? t_in : 1.f;
  // ---- read the row.  Groups are the keys at one place k of a thread's quads.
  unsigned group[4] = {0, 0, 0, 0};
  {
    const T* row = static_cast<const T*>(a.logits) + (long long)r * a.ld;
#pragma unroll 4
    for (int q = 0; q < Q; ++q) {
      unsigned key[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = base + (4 * q + k) * 32;
        float l = -INFINITY;
        if (i < a.vocab) {
          if constexpr (sizeof(T) == 2) l = __bfloat162float(row[i]);
          else l = row[i];
        }
        key[k] = order_key(l);
        group[k] = max(group[k], key[k]);
      }
      keys[q * 32] = make_uint4(key[0], key[1], key[2], key[3]);
    }
  }
  // f(key, index) for this thread's keys, in index order
  auto each = [&](auto f) {
#pragma unroll 2
    for (int q = 0; q < Q; ++q) {
      const uint4 x = keys[q * 32];
      const int i = base + q * 128;
      f(x.x, i);
      f(x.y, i + 32);
      f(x.z, i + 64);
      f(x.w, i + 96);
    }
  };
  sh.bins[tid] = 0;
  if (tid == 0) {
    sh.local_n = 0;
  }
  if (C > 1) cluster_arrive();                       // this block is there

  // ---- the block's largest key, and its groups' smallest above -inf
  unsigned top = max(max(group[0], group[1]), max(group[2], group[3])), gmin = 0xffffffffu;
#pragma unroll
  for (int q = 0; q < 4; ++q) gmin = min(gmin, group[q] > kKeyNegInf ? group[q] : 0xffffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  gmin = __reduce_min_sync(0xffffffffu, gmin);
  if (lane == 0) {
    sh.red[0][warp] = top;
    sh.red[1][warp] = gmin;
  }
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, sh.red[0][lane % FW]);
  gmin = __reduce_min_sync(0xffffffffu, sh.red[1][lane % FW]);
  if (tid == 0) sh.top = top;

  const bool cuts = !greedy && ((k > 0 && k < a.vocab) || !(p >= 1.f));
  auto block_low = [&]() {                           // the block's smallest key above -inf, for the search
    unsigned low = 0xffffffffu;
    each([&](unsigned key, int) { low = min(low, key > kKeyNegInf ? key : 0xffffffffu); });
    low = __reduce_min_sync(0xffffffffu, low);
    if (lane == 0) sh.warp_count[warp] = low;
    __syncthreads();
    low = __reduce_min_sync(0xffffffffu, sh.warp_count[lane % FW]);
    if (tid == 0) sh.low = low;
  };
  const bool by_list = cuts && k > 0 && k <= SMALL_K, by_mass = cuts && !(k > 0 && k < a.vocab);
  unsigned bound = 0;
  if (by_list || by_mass) {
    // ---- candidates for the first k ranks (top-p alone: for as many as the list may
    // take).  Every group's largest logit is an
    // element, so the k-th largest of them bounds the block's k-th rank from below;
    // a histogram of them finds a bound just under it.  What has no mass is no
    // candidate.
    const float ltop = key_logit(top);
    const unsigned floor_key =
        top <= kKeyNegInf ? 0xffffffffu : ltop == INFINITY ? top : max(kKeyNegInf + 1, order_key(ltop - ZERO_Z * t));
    bound = floor_key;
    if (top > kKeyNegInf) {
      const float scale = bins_over(ltop - key_logit(gmin));
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (group[q] >= floor_key)
          atomicAdd(&sh.bins[min(FT - 1, (int)((ltop - key_logit(group[q])) * scale))], 1u);
      __syncthreads();
      if (warp == 0) {
        const unsigned best = kth_bin(sh, by_list ? k : LIST * 3 / 4 / C);
        if (lane == 0) sh.best = best;
      }
      __syncthreads();
      // the lower edge of that bin, less what the bins' rounding may be off
      if (sh.best < FT)
        bound = max(floor_key, scale > 0.f ? order_key(ltop - (sh.best + 1.01f) / scale) : gmin);
      sh.bins[tid] = 0;
      if (by_mass) {
        // about how much mass the groups' largest have, in the block's largest
        float x = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) x += logit_weight(Row{ltop, __fdiv_rn(1.f, t)}, key_logit(group[q]));
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) sh.group_mass[warp] = x;
      }
    }
  }
  if (C > 1) cluster_wait();
  if (by_list) {
    ull* list = in_block(&sh.list[0], 0);
    // straight into the first block's list, each block's in a part of its own
    each([&](unsigned key, int i) {
      if (key >= bound) {
        const unsigned at = atomicAdd(&sh.local_n, 1u);
        if (at < SEG) list[rank * SEG + at] = ((ull)key << 32) | (unsigned)~i;
      }
    });
    __syncthreads();
    if (tid == 0) *in_block(&sh.seg_n[rank], 0) = sh.local_n;
  } else if (by_mass) {
    __syncthreads();
    float x = top > kKeyNegInf ? sh.group_mass[lane % FW] : 0.f;
    for (int o = FW / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (tid == 0) {
      // A block without candidates (behind the row's end, or all -inf) bounds nothing.
      // 64 rows of 50257 bf16, whose eighth block is empty: p 0.5 at temperature 0.3
      // 74 us where it did, now 44.
      sh.bound_key = top > kKeyNegInf ? bound : 0u;
      sh.block_mass = x;
    }
  } else if (cuts) {
    block_low();
  }
  sync_cluster(C);
  if (by_list) {
    unsigned n = 0;
    bool fits = true;
    for (int c = 0; c < C; ++c) {
      const unsigned x = *in_block(&sh.seg_n[c], 0);
      n += x;
      fits &= x <= SEG;
    }
    if (fits) {
      // the first block has all there is to choose from
      if (rank != 0) {
        cluster_arrive();                            // its counts have been read; nobody reads this block
        if (more) cluster_wait();
        return;
      }
      if (n == 0) {
        if (tid == 0) {
          a.token[r] = -1;
          if (a.logprob) a.logprob[r] = -INFINITY;
        }
      } else {
        draw_from_few(a, sh, r, C, k, p, least, u, t);
      }
      if (C > 1) cluster_sync();
      return;
    }
  }
  for (int c = 0; c < C; ++c) top = max(top, *in_block(&sh.top, c));
  if (top <= kKeyNegInf) {                           // nothing can be taken
    if (rank == 0 && tid == 0) {
      a.token[r] = -1;
      if (a.logprob) a.logprob[r] = -INFINITY;
    }
    sync_cluster(C);                                 // nobody leaves while its memory is read
    return;
  }
  const Row row{key_logit(top), __fdiv_rn(1.f, t)};
  auto mass_at = [&](unsigned key) { return mass_of(logit_weight(row, key_logit(key))); };

  bool few = false;
  if (by_mass) {
    // top-p alone: will the keys that every block's bound lets through reach the cut?
    // Those below it have at most its weight each, a quarter of that on average say.
    // Both ways give the same token; this one costs a pass more where it fails.
    // Measured on 64 rows of 32000 bf16, with the list and by the search: p 0.5 at
    // temperature 0.3 20 and 24 us; p 0.95 at 0.8, which the list seldom reaches, 35
    // and 31 us.
    // Of what the blocks have published alone, so that all of them decide alike.
    float sum = 0.f;
    bound = 0;
    for (int c = 0; c < C; ++c) {
      bound = max(bound, *in_block(&sh.bound_key, c));
      sum += *in_block(&sh.block_mass, c) * logit_weight(row, key_logit(*in_block(&sh.top, c)));
    }
    few = 0.25f * (float)a.vocab * logit_weight(row, key_logit(bound)) <= (1.f - p) * sum;
  }
  if (few) {
    // ---- the mass of all, and of those keys.  Where that reaches the cut, they are
    // all there is to choose from.
    ull all = 0, above = 0;
    unsigned n = 0;
    each([&](unsigned key, int) {
      if (key <= kKeyNegInf) return;
      const ull m = mass_at(key);
      all += m;
      if (key >= bound) {
        above += m;
        ++n;
      }
    });
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, o);
      above += __shfl_xor_sync(0xffffffffu, above, o);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) {
      sh.warp_mass[warp] = all;
      sh.warp_above[warp] = above;
      sh.warp_count[warp] = n;
    }
    sync_cluster(C);
    // a thread a warp of the cluster: totals, and the list places of the blocks before
    all = above = 0;
    n = 0;
    if (tid < C * FW) {
      all = in_block(&sh.warp_mass[0], tid / FW)[tid % FW];
      above = in_block(&sh.warp_above[0], tid / FW)[tid % FW];
      n = in_block(&sh.warp_count[0], tid / FW)[tid % FW];
    }
    unsigned at = tid < rank * FW ? n : 0u;
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, o);
      above += __shfl_xor_sync(0xffffffffu, above, o);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    at = __reduce_add_sync(0xffffffffu, at);
    if (lane == 0 && warp < MAX_C * FW / 32) {
      sh.scan_m[warp] = all;
      sh.all[warp] = above;
      sh.scan_c[warp] = n;
      sh.red[0][warp] = at;
    }
    if (tid == 0) sh.local_n = 0;
    __syncthreads();
    all = above = 0;
    n = at = 0;
    for (int w = 0; w < MAX_C * FW / 32; ++w) {
      all += sh.scan_m[w];
      above += sh.all[w];
      n += sh.scan_c[w];
      at += sh.red[0][w];
    }
    if (warp == 0) {
      const ull x = whole_bound(__dmul_rn((double)p, __ull2double_rn(all)));
      if (lane == 0) sh.bound = x;
    }
    __syncthreads();
    if (n <= LIST && above >= sh.bound) {
      ull* list = in_block(&sh.list[0], 0) + at;
      each([&](unsigned key, int i) {
        if (key >= bound) list[atomicAdd(&sh.local_n, 1u)] = ((ull)key << 32) | (unsigned)~i;
      });
      sync_cluster(C);
      if (rank == 0) draw_from_list(a, sh, r, (int)n, (int)n, p, least, u, t, all);
      if (C > 1) cluster_sync();                     // nobody leaves while its memory is read
      return;
    }
    sync_cluster(C);                                 // the sums have been read
  }

  // ---- cuts, as the last place kept
  Place cut{0u, 0x7fffffff};
  if (greedy) {
    // the first place of the largest key: a search for one rank without its histogram
    unsigned first = 0x7fffffffu;
    each([&](unsigned key, int i) {
      if (key == top) first = min(first, (unsigned)i);
    });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) sh.warp_count[warp] = first;
    sync_cluster(C);
    first = tid < C * FW ? *in_block(&sh.warp_count[tid % FW], tid / FW) : 0x7fffffffu;
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) sh.red[0][warp] = first;
    __syncthreads();
    for (int w = 0; w < FW; ++w) first = min(first, sh.red[0][w]);
    cut = Place{top, (int)first};
    sync_cluster(C);                                 // warp_count has been read
  }
  if (cuts) {
    // ---- the general search: bins even in the logit over the range that has mass; the
    // tokens of the bin with the cut are sorted in the first block's list, or, if
    // they are too many (equal logits), binned again by their keys until one is left
    if (by_list || by_mass) {
      block_low();
      sync_cluster(C);
    }
    unsigned low = sh.low;
    for (int c = 0; c < C; ++c) low = min(low, *in_block(&sh.low, c));
    // The last place kept by count (the first k) or by mass (less than p of all before)
    auto search = [&](bool by_count) -> bool {
      const float scale = bins_over(fminf(ZERO_Z * t, row.top - key_logit(low)));
      auto first_bin = [&](unsigned key) { return min(FT - 1, (int)((row.top - key_logit(key)) * scale)); };
      unsigned n_above = 0, lo = 0, hi = 0;
      ull m_above = 0, bound = 0;
      int bin0 = -1, shift = 0, turn = 0;            // turn: the histogram in use, zero when its turn comes
      __syncthreads();                               // its memory may have held a list
      sh.count[0][tid] = 0;
      for (int w = 0; w < 3; ++w) sh.mass[0][w][tid] = 0;
      __syncthreads();
      // The present level's bin of a token, -1 if it is not one of those in question.
      // Below the floor no token has mass: by rank they come after all that have, and
      // where a cut falls among them does not matter.
      const unsigned floor_key = row.top == INFINITY ? top : max(kKeyNegInf + 1, order_key(row.top - ZERO_Z * t));
      auto bin = [&](unsigned key, int i) {
        if (key < floor_key || !cut.keeps(key, i)) return -1;
        if (bin0 < 0) return first_bin(key);
        return key < lo || key > hi || first_bin(key) != bin0 ? -1 : (int)((hi - key) >> shift);
      };
      auto keep = [&](unsigned c, ull m) { return by_count ? c < (unsigned)k : c == 0 || m < bound; };
      while (true) {
        // Histogram.  A mass has 41 bits and shared memory adds 32 at a time: three
        // words of 14, 13 and 14 bits, whose sums over a block's 45056 tokens at most
        // stay below 2^32.
        each([&](unsigned key, int i) {
          const int x = bin(key, i);
          if (x < 0) return;
          if (by_count) {
            atomicAdd(&sh.count[turn][x], 1u);
            return;
          }
          const ull m = mass_at(key);
          if (m == 0) return;
          atomicAdd(&sh.count[turn][x], 1u);
          atomicAdd(&sh.mass[turn][0][x], (unsigned)m & 0x3fffu);
          if (m >> 14) atomicAdd(&sh.mass[turn][1][x], (unsigned)(m >> 14) & 0x1fffu);
          if (m >> 27) atomicAdd(&sh.mass[turn][2][x], (unsigned)(m >> 27));
        });
        sync_cluster(C);
        // the last turn's: every block has read it by now
        sh.count[turn ^ 1][tid] = 0;
        for (int w = 0; w < 3; ++w) sh.mass[turn ^ 1][w][tid] = 0;
        unsigned c = 0, earlier = 0;                 // earlier: of the blocks before this one
        ull m = 0;
#pragma unroll 4
        for (int q = 0; q < C; ++q) {
          if (q == rank) earlier = c;
          c += in_block(&sh.count[turn][0], q)[tid];
          const unsigned* w = in_block(&sh.mass[turn][0][0], q) + tid;
          m += (ull)w[0] + ((ull)w[FT] << 14) + ((ull)w[2 * FT] << 27);
        }
        const unsigned own = c;
        block_prefix(sh, c, m);
        if (tid == 0) sh.best = 0;
        if (bin0 < 0 && !by_count) {
          if (warp == 0) {
            ull total = 0;
            for (int w = 0; w < FW; ++w) total += sh.scan_m[w];
            const ull x = whole_bound(__dmul_rn((double)p, __ull2double_rn(total)));
            if (lane == 0) sh.bound = x;
          }
          __syncthreads();
          bound = sh.bound;
        } else {
          __syncthreads();
        }
        c += n_above;
        m += m_above;
        if (own && keep(c, m)) atomicMax(&sh.best, (unsigned)tid);
        __syncthreads();
        if (tid == (int)sh.best) {
          sh.n_above = c;
          sh.m_above = m;
          sh.red[0][0] = own;
          sh.local_at = earlier;
          sh.local_n = 0;
        }
        __syncthreads();
        const int best = (int)sh.best;
        const unsigned n_equal = sh.red[0][0];
        n_above = sh.n_above;
        m_above = sh.m_above;
        if (by_count && bin0 < 0 && k <= TOP_K_LIST && n_above + n_equal <= LIST) {
          // the first k ranks and the rest of the last one's bin fit the first block's
          // list, one block's after another's: what is left is its to do
          const unsigned mine = __reduce_add_sync(0xffffffffu, tid <= best ? earlier : 0u);
          if (lane == 0) sh.scan_c[warp] = mine;
          if (tid == 0) sh.local_n = 0;
          __syncthreads();
          ull* list = in_block(&sh.list[0], 0) + __reduce_add_sync(0xffffffffu, lane < FW ? sh.scan_c[lane] : 0u);
          each([&](unsigned key, int i) {
            const int x = bin(key, i);
            if (x >= 0 && x <= best) list[atomicAdd(&sh.local_n, 1u)] = ((ull)key << 32) | (unsigned)~i;
          });
          sync_cluster(C);
          if (rank == 0) draw_from_list(a, sh, r, (int)(n_above + n_equal), k, p, least, u, t, 0);
          return true;
        }
        if (n_equal <= TOP_K_LIST) {
          // few enough to sort: the blocks' tokens of that bin, one block's after another's
          ull* list = in_block(&sh.list[0], 0) + sh.local_at;
          each([&](unsigned key, int i) {
            if (bin(key, i) == best && (by_count || mass_at(key))) list[atomicAdd(&sh.local_n, 1u)] = ((ull)key << 32) | (unsigned)~i;
          });
          sync_cluster(C);
          if (rank == 0) {
            sort_list(sh, pad_list(sh, (int)n_equal));
            constexpr int PER = TOP_K_LIST / FT;
            ull own_m[PER], before = 0;
#pragma unroll
            for (int q = 0; q < PER; ++q) {
              const int i = tid * PER + q;
              own_m[q] = i < (int)n_equal ? mass_at((unsigned)(sh.list[i] >> 32)) : 0;
              before += own_m[q];
            }
            unsigned none = 0;
            block_prefix(sh, none, before);
            before += m_above;
            int last = 0;
#pragma unroll
            for (int q = 0; q < PER; ++q) {
              const int i = tid * PER + q;
              if (i < (int)n_equal && keep(n_above + i, before)) last = i;
              before += own_m[q];
            }
            last = __reduce_max_sync(0xffffffffu, last);
            if (lane == 0) sh.red[0][warp] = last;
            __syncthreads();
            last = __reduce_max_sync(0xffffffffu, (int)sh.red[0][lane % FW]);
            const ull x = sh.list[last];
            if (tid < C) *in_block(&sh.cut, tid) = Place{(unsigned)(x >> 32), (int)~(unsigned)x};
          }
          sync_cluster(C);
          cut = sh.cut;
          return false;
        }
        if (bin0 < 0) {
          // the keys in that bin
          lo = 0xffffffffu;
          hi = 0;
          each([&](unsigned key, int i) {
            if (bin(key, i) == best && (by_count || mass_at(key))) {
              lo = min(lo, key);
              hi = max(hi, key);
            }
          });
          lo = __reduce_min_sync(0xffffffffu, lo);
          hi = __reduce_max_sync(0xffffffffu, hi);
          __syncthreads();
          if (lane == 0) {
            sh.red[0][warp] = lo;
            sh.red[1][warp] = hi;
          }
          __syncthreads();
          if (tid == 0) {
            for (int w = 1; w < FW; ++w) {
              lo = min(lo, sh.red[0][w]);
              hi = max(hi, sh.red[1][w]);
            }
            sh.lo[0] = lo;
            sh.hi[0] = hi;
          }
          sync_cluster(C);
          for (int q = 0; q < C; ++q) {
            lo = min(lo, *in_block(&sh.lo[0], q));
            hi = max(hi, *in_block(&sh.hi[0], q));
          }
          bin0 = best;
        } else {
          const unsigned from = (unsigned)best << shift;   // bins are counted from hi down
          const unsigned span = (1u << shift) - 1u;
          hi -= from;
          lo = max(lo, hi >= span ? hi - span : 0u);
        }
        turn ^= 1;
        if (lo == hi) {
          // one key: how many of its n_equal tokens, lowest index first
          const ull one = mass_at(hi);
          unsigned least_n = 1, most = n_equal;
          while (least_n < most) {
            const unsigned mid = (least_n + most + 1) / 2;
            if (keep(n_above + mid - 1, m_above + (ull)(mid - 1) * one)) least_n = mid;
            else most = mid - 1;
          }
          if (least_n == n_equal) {
            if (hi > cut.key) cut = Place{hi, 0x7fffffff};
            // the next search sets this block's histograms to zero: not before every
            // block has read them
            sync_cluster(C);
            return false;
          }
          // the index of that token
          unsigned seen = 0;
          each([&](unsigned key, int i) {
            seen += __popc(__ballot_sync(0xffffffffu, key == hi && cut.keeps(key, i)));
          });
          sync_cluster(C);                           // warp_count is free
          if (lane == 0) sh.warp_count[warp] = seen;
          sync_cluster(C);
          unsigned before = 0;
          for (int q = lane; q < rank * FW + warp; q += 32) before += *in_block(&sh.warp_count[q % FW], q / FW);
          before = __reduce_add_sync(0xffffffffu, before);
          if (before < least_n && least_n <= before + seen) {
            unsigned at = before;
            each([&](unsigned key, int i) {
              const bool mine = key == hi && cut.keeps(key, i);
              const unsigned eq = __ballot_sync(0xffffffffu, mine);
              if (mine && at + __popc(eq & ((2u << lane) - 1u)) == least_n)
                for (int q = 0; q < C; ++q) *in_block(&sh.cut, q) = Place{hi, i};
              at += __popc(eq);
            });
          }
          sync_cluster(C);
          cut = sh.cut;
          return false;
        }
        shift = max(0, 32 - __clz(hi - lo) - 9);
      }
    };
    if (k > 0 && k < a.vocab && search(true)) {
      if (C > 1) cluster_sync();                     // nobody leaves while its memory is read
      return;
    }
    if (!(p >= 1.f)) search(false);
  }

  // ---- the draw: every warp's kept mass, then the warp in which the target falls
  auto kept = [&](unsigned key, int i) -> ull {
    if (!cut.keeps(key, i) || key <= kKeyNegInf) return 0;
    const float w = logit_weight(row, key_logit(key));
    return w >= least || greedy ? mass_of(w) : 0;
  };
  ull m = 0;
  each([&](unsigned key, int i) { m += kept(key, i); });
  for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
  if (lane == 0) sh.warp_mass[warp] = m;
  sync_cluster(C);
  {
    ull before = tid < C * FW ? in_block(&sh.warp_mass[0], tid / FW)[tid % FW] : 0;
    unsigned none = 0;
    block_prefix(sh, none, before);
    if (tid < C * FW) sh.all[tid] = before;
  }
  __syncthreads();
  ull total = 0;
  for (int w = 0; w < FW; ++w) total += sh.scan_m[w];
  if (warp == 0) {
    const ull x = draw_target(u, total);
    if (lane == 0) sh.m_above = x;
  }
  __syncthreads();
  const ull target = sh.m_above;
  ull before = sh.all[rank * FW + warp];
  if (before <= target && target < before + m) {
    bool found = false;
    each([&](unsigned key, int i) {
      const ull x = found ? 0 : kept(key, i);
      if (!__any_sync(0xffffffffu, x != 0)) return;
      ull run = x;
      for (int o = 1; o < 32; o <<= 1) {
        const ull y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + run > target);
      if (past && lane == __ffs(past) - 1) {
        a.token[r] = i;
        if (a.logprob)
          a.logprob[r] = logit_z(row, key_logit(key)) - logf(__ull2float_rn(total) * 0x1p-40f);
      }
      found = past != 0;
      before += __shfl_sync(0xffffffffu, run, 31);
    });
  }
  if (C > 1) cluster_sync();                         // nobody leaves while its memory is read
}

// Whether sample_stream_kernel takes row r; all settings are read at once
__device__ __forceinline__ bool streams(const SampleArgs& a, long long r) {
  const float t = a.temperature ? a.temperature[r] : 1.f, least = a.min_p ? a.min_p[r] : 0.f;
  const int k = a.top_k ? a.top_k[r] : 0;
  return !(t >= FLT_MIN) | !(least <= 1.f) | (k > 0) & (k <= SMALL_K);
}

// A cluster takes every n-th row of its n clusters, after sample_stream_kernel (`rest`)
// those that it left.
template <typename T>
__global__ void __launch_bounds__(FT, 2) sample_cluster_kernel(const SampleArgs a, const int C, const int Q, const int rest) {
  const int n = (int)gridDim.x / C;
  long long r0 = blockIdx.x / C;
  auto mine = [&]() { return r0 + (long long)(threadIdx.x % 32) * n; };
  // the settings are older than sample_stream_kernel, which has waited for all before it
  bool streamed = rest && mine() < a.rows && streams(a, mine());
  griddep_wait();
  // after sample_stream_kernel not early: the next call's blocks would gather on the SMs
  // that these leave first (608 x 131071 86 us, now 78)
  if (!rest && threadIdx.x == 0) griddep_launch_dependents();
  while (r0 < a.rows) {
    const bool left = mine() < a.rows && (!streamed || a.token[mine()] == kNotDone);
    for (unsigned m = __ballot_sync(0xffffffffu, left); m; m &= m - 1) {
      cluster_row<T>(a, C, Q, (int)(r0 + (long long)(__ffs(m) - 1) * n), rest);
      __syncthreads();                               // shared memory is free
    }
    r0 += 32ll * n;
    streamed = rest && mine() < a.rows && streams(a, mine());
  }
}

// ------------------------------------------------------------------ a row a block
// Many rows at once, for those whose draw is among the first SMALL_K ranks (or the
// first alone): a block, or C of them for every C-th tile, streams through a row and
// lists what may be among them.  The k-th largest of its first logits' groups bounds the
// k-th rank of the row from below, so a thread's later logits are mostly a maximum and
// one comparison a tile; every fourth tile a long list's own k-th rank is a better
// bound.  A row of which four tiles hold more than the list (ascending logits, say) is
// left to the other kernel.
//
// What bounds it: latency and issue; two blocks an SM (64 registers a thread) each wait
// for their loads, the bound and the draw in turn.  384 x 131071, top-k 50: fp32 61 us
// (201 MB), bf16 46 us (101 MB), of which the second launch takes 3 to 6 us; the 80 rows
// that 304 blocks leave take half as long as the 304.  The next tiles' loads stay as
// they came until their turn: widened on arrival, bf16 rows wait for them (62 us).
constexpr int TILE_BYTES = 64;                // of a thread, in 16-byte vectors

// The list's bound for the k-th rank: a histogram of its keys; drops what is below it.
// Whole block, after a barrier.
__device__ __forceinline__ unsigned tighten(Cluster& sh, int k) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, n = (int)sh.local_n;
  unsigned hi = 0, lo = 0xffffffffu;
  for (int i = tid; i < n; i += FT) {
    const unsigned key = (unsigned)(sh.list[i] >> 32);
    hi = max(hi, key);
    lo = min(lo, key);
    sh.local[i] = sh.list[i];
  }
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (lane == 0) {
    sh.red[0][warp] = hi;
    sh.red[1][warp] = lo;
  }
  sh.bins[tid] = 0;
  __syncthreads();
  hi = __reduce_max_sync(0xffffffffu, sh.red[0][lane % FW]);
  lo = __reduce_min_sync(0xffffffffu, sh.red[1][lane % FW]);
  const float ltop = key_logit(hi), scale = bins_over(ltop - key_logit(lo));
  auto bin = [&](ull x) { return min(FT - 1, (int)((ltop - key_logit((unsigned)(x >> 32))) * scale)); };
  for (int i = tid; i < n; i += FT) atomicAdd(&sh.bins[bin(sh.local[i])], 1u);
  if (tid == 0) sh.local_n = 0;
  __syncthreads();
  if (warp == 0) {
    const unsigned best = kth_bin(sh, k);
    if (lane == 0) sh.best = best;
  }
  __syncthreads();
  const int best = (int)sh.best;
  unsigned bound = 0xffffffffu;                      // the lowest key kept
  for (int i = tid; i < n; i += FT) {
    const ull x = sh.local[i];
    if (bin(x) <= best) {
      sh.list[atomicAdd(&sh.local_n, 1u)] = x;
      bound = min(bound, (unsigned)(x >> 32));
    }
  }
  bound = __reduce_min_sync(0xffffffffu, bound);
  if (lane == 0) sh.red[0][warp] = bound;
  __syncthreads();
  bound = __reduce_min_sync(0xffffffffu, sh.red[0][lane % FW]);
  __syncthreads();
  return bound;
}

template <typename T>
__global__ void __launch_bounds__(FT, 2) sample_stream_kernel(const SampleArgs a, const int C) {
  __shared__ Cluster sh;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int rank = C == 1 ? 0 : (int)cluster_ctarank(), r = blockIdx.x / C;
  const float t_in = a.temperature ? a.temperature[r] : 1.f;
  const int k_in = a.top_k ? a.top_k[r] : 0;
  const float p_in = a.top_p ? a.top_p[r] : 1.f;
  const float least_in = a.min_p ? a.min_p[r] : 0.f;
  const float u = a.u[r];
  const bool greedy = !(t_in >= FLT_MIN) || k_in == 1 || !(least_in <= 1.f);
  if (!greedy && !(k_in > 0 && k_in <= SMALL_K)) return;
  const int k = greedy ? 1 : k_in;
  const float p = greedy ? 1.f : p_in, least = greedy ? 0.f : least_in, t = t_in >= FLT_MIN ? t_in : 1.f;
  const T* row = static_cast<const T*>(a.logits) + (long long)r * a.ld;
  // 16-byte vectors from the boundary below the row on: logit e of vector v of the
  // block's tile x has index ((x * C + rank) * VECS + v) * FT + tid) * VEC + e - head.
  constexpr int VEC = 16 / (int)sizeof(T), VECS = TILE_BYTES / 16, TILE = VEC * VECS;
  const int head = (int)(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
  struct Tile {
    uint32_t w[TILE_BYTES / 4];
    __device__ __forceinline__ float operator[](int v) const {
      if constexpr (sizeof(T) == 4) return __uint_as_float(w[v]);
      else return __uint_as_float(v % 2 ? w[v / 2] & 0xffff0000u : w[v / 2] << 16);
    }
    __device__ __forceinline__ float most() const {  // NaN is passed over
      if constexpr (sizeof(T) == 4) {
        float m = fmaxf((*this)[0], (*this)[1]);
#pragma unroll
        for (int v = 2; v < TILE; ++v) m = fmaxf(m, (*this)[v]);
        return m;
      } else {
        auto two = [&](int i) { return *reinterpret_cast<const __nv_bfloat162*>(&w[i]); };
        __nv_bfloat162 m = __hmax2(two(0), two(1));
#pragma unroll
        for (int i = 2; i < TILE / 2; ++i) m = __hmax2(m, two(i));
        return fmaxf(__low2float(m), __high2float(m));
      }
    }
  };
  auto index = [&](int x, int v) { return (((x * C + rank) * VECS + v) * FT + tid) * VEC - head; };
  auto load = [&](int x, Tile& l) {
    // all of the tile is within the row
    const bool inside = (x * C + rank > 0 || head == 0) && (x * C + rank + 1) * (FT * TILE) - head <= a.vocab;
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      const int i = index(x, v);
      if (inside || (i >= 0 && i + VEC <= a.vocab)) {
        const uint4 y = *reinterpret_cast<const uint4*>(row + i);
        l.w[v * 4] = y.x;
        l.w[v * 4 + 1] = y.y;
        l.w[v * 4 + 2] = y.z;
        l.w[v * 4 + 3] = y.w;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (sizeof(T) == 4) {
            l.w[v * 4 + q] = __float_as_uint(i + q >= 0 && i + q < a.vocab ? (float)row[i + q] : -INFINITY);
          } else {
            const int j = i + 2 * q;
            const float lo = j >= 0 && j < a.vocab ? (float)row[j] : -INFINITY;
            const float hi = j + 1 >= 0 && j + 1 < a.vocab ? (float)row[j + 1] : -INFINITY;
            l.w[v * 4 + q] = __float_as_uint(lo) >> 16 | __float_as_uint(hi);
          }
        }
      }
    }
  };
  const int tiles = ((a.vocab + head + FT * TILE - 1) / (FT * TILE) - rank + C - 1) / C;   // this block's
  Tile l, next;
  load(0, l);
  if (tiles > 1) load(1, next);
  sh.bins[tid] = 0;
  if (tid == 0) sh.local_n = 0;

  // ---- the first logits' bound
  unsigned group[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < TILE; ++i) group[i % 4] = max(group[i % 4], order_key(l[i]));
  if (TILE == 16 && tiles > 1) {                     // 32 logits a thread for either type
#pragma unroll
    for (int i = 0; i < TILE; ++i) group[i % 4] = max(group[i % 4], order_key(next[i]));
  }
  unsigned top = max(max(group[0], group[1]), max(group[2], group[3])), gmin = 0xffffffffu;
#pragma unroll
  for (int q = 0; q < 4; ++q) gmin = min(gmin, group[q] > kKeyNegInf ? group[q] : 0xffffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  gmin = __reduce_min_sync(0xffffffffu, gmin);
  if (lane == 0) {
    sh.red[0][warp] = top;
    sh.red[1][warp] = gmin;
  }
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, sh.red[0][lane % FW]);
  gmin = __reduce_min_sync(0xffffffffu, sh.red[1][lane % FW]);
  unsigned bound = kKeyNegInf + 1;                   // -inf is never taken
  if (top > kKeyNegInf) {
    const float ltop = key_logit(top);
    bound = ltop == INFINITY ? top : max(bound, order_key(ltop - ZERO_Z * t));   // below: no mass
    const float scale = bins_over(ltop - key_logit(gmin));
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (group[q] >= bound) atomicAdd(&sh.bins[min(FT - 1, (int)((ltop - key_logit(group[q])) * scale))], 1u);
    __syncthreads();
    if (warp == 0) {
      const unsigned best = kth_bin(sh, k);
      if (lane == 0) sh.best = best;
    }
    __syncthreads();
    // the lower edge of that bin, less what the bins' rounding may be off
    if (sh.best < FT) bound = max(bound, scale > 0.f ? order_key(ltop - (sh.best + 1.01f) / scale) : gmin);
  }
  // ---- the tiles
  auto look = [&](int x, const Tile& l) {
    const float lbound = key_logit(bound);
    if (!(l.most() >= lbound)) return;
    // a warp is here almost always before the bound is tight, seldom after; one loop
    // over what was found, not a branch a logit: 384 x 131071 bf16 62 us, now 46 us
    unsigned found = 0;
#pragma unroll
    for (int v = 0; v < TILE; ++v) found |= l[v] >= lbound ? 1u << v : 0u;
#pragma unroll 1
    for (; found; found &= found - 1) {
      const int v = __ffs(found) - 1, i = index(x, v / VEC) + v % VEC;
      const unsigned at = atomicAdd(&sh.local_n, 1u);
      if (at < LIST) sh.list[at] = ((ull)order_key((float)row[i]) << 32) | (unsigned)~i;
    }
  };
  bool fits = true;
  for (int x = 0; x < tiles; x += 2) {
    look(x, l);
    if (x + 2 < tiles) load(x + 2, l);
    if (x + 1 < tiles) look(x + 1, next);
    if (x + 3 < tiles) load(x + 3, next);
    // every fourth tile, and after the last: is the list long?
    if (x % 4 == 2 || x + 2 >= tiles) {
      __syncthreads();
      const unsigned n = sh.local_n;
      __syncthreads();                               // n has been read
      fits = n <= LIST;
      if (!fits) break;
      // from 1024, 512, 256, 160 on: 200 x 260000 bf16 58, 55, 52, 51 us
      if (n > STREAM_LONG) bound = max(bound, tighten(sh, k));
    }
  }
  unsigned n = fits ? sh.local_n : 0;
  if (C > 1) {
    // the row's first block gets the others' lists, in parts of its own
    if (n > SEG) {
      __syncthreads();                               // n has been read
      tighten(sh, k);
      n = sh.local_n;
      fits = n <= SEG;
    }
    cluster_sync();                                  // it needs no more of the list than its part
    if (fits && rank > 0)
      for (int i = tid; i < (int)n; i += FT) in_block(&sh.list[0], 0)[rank * SEG + i] = sh.list[i];
    if (tid == 0) *in_block(&sh.seg_n[rank], 0) = fits ? n : LIST + 1;
    cluster_sync();
    if (rank > 0) return;
    n = 0;
    for (int c = 0; c < C; ++c) n += sh.seg_n[c];
    fits = n <= LIST;
  } else if (tid == 0) {
    sh.seg_n[0] = n;
  }
  if (!fits || n == 0) {
    if (tid == 0) {
      a.token[r] = fits ? -1 : kNotDone;
      if (fits && a.logprob) a.logprob[r] = -INFINITY;
    }
    return;
  }
  sh.bins[tid] = 0;
  __syncthreads();
  draw_from_few(a, sh, r, C, k, p, least, u, t);
}

// A launch of `grid` blocks, `cluster` at a time, that may begin before its stream's
// last kernel has ended
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  Launch(long long grid, int threads, int cluster, size_t smem, cudaStream_t s) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
  }
  template <class... Params, class... Args>
  int operator()(void (*kernel)(Params...), Args... args) {
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
};

template <typename T>
int launch_any(const SampleArgs& a, int num_sms, cudaStream_t s) {
  const long long most = (long long)MAX_C * FT * 4 * MAX_Q;
  if (a.vocab > most || a.rows > 0x7fffffff / MAX_C)
    return Launch(a.rows, THREADS, 1, 0, s)(sample_kernel<T>, a);
  // Blocks of a row: more shorten its passes, and lengthen the exchanges.  Quads a
  // thread 2, 4, 8, 16: one row of 32000 8.4, 8.4, 8.7, 9.9 us, 64 rows with settings
  // of their own 41, 37, 49, 53 us.
  int C = 1;
  while (C < MAX_C && C * FT * SAMPLE_Q * 4 < a.vocab) C <<= 1;
  const int Q = (a.vocab + C * FT * 4 - 1) / (C * FT * 4);
  constexpr int most_smem = (int)sizeof(Cluster) + MAX_Q * FT * 16;
  static_assert(most_smem <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = set_smem_once(smem_set, sample_cluster_kernel<T>, most_smem);
  if (e != cudaSuccess) return e;
  const size_t smem = sizeof(Cluster) + (size_t)Q * FT * 16;
  // More rows than the GPU holds clusters at once: what can stream does, a row a block
  // or a few.  Measured (bf16, top-k 50), by the cluster kernel alone and with it:
  // 140 x 16384 10.8 and 10.9 us, 170 x 16384 17.6 and 11.9, 72 x 32000 11.5 and 12.0,
  // 80 x 32000 19.4 and 12.8, 36 x 131071 15.0 and 16.0, 40 x 131071 25.2 and 17.0.  A
  // row of one block is quicker there: 512 x 8192 16.7 and 20.5 us.  Where every row is
  // the cluster kernel's the other costs 3 us (152 x 32000, no cut, 28.9 and 31.5).
  int stream = 0;
  if (C > 1) {
    static std::atomic<int> held[MAX_C + 1][MAX_Q + 1];   // the devices of a process are alike
    int n = held[C][Q].load(std::memory_order_relaxed);
    if (n == 0) {
      Launch one(C, FT, C, smem, s);
      e = cudaOccupancyMaxActiveClusters(&n, sample_cluster_kernel<T>, &one.cfg);
      if (e != cudaSuccess) return e;
      held[C][Q].store(n, std::memory_order_relaxed);
    }
    stream = a.rows > n;
  }
  int clusters = a.rows;
  if (stream) {
    // Blocks of a row: while two an SM hold them all.  1, 2 and 4: 152 x 16384 11.3,
    // 12.2, 22 us, 152 x 131071 31.8, 24.6, 34 us, 48 x 131071 23.7, 21.1, 18.4 us.
    int S = 1;
    while (S < 4 && a.rows * S <= num_sms && a.vocab >= 2 * S * STREAM_PART) S <<= 1;
    e = (cudaError_t)Launch((long long)a.rows * S, FT, S, 0, s)(sample_stream_kernel<T>, a, S);
    if (e != cudaSuccess) return e;
    // Clusters for the rows that are left: few are soon done where there are none, many
    // share them evenly.  4, 12 and 24 blocks an SM: 384 x 131071 (f32, top-k 50) 63,
    // 68 and 74 us, all of them flat top-p rows 755, 632 and 630 us.
    clusters = std::min(a.rows, 12 * num_sms / C);
  }
  return Launch((long long)clusters * C, FT, C, smem, s)(sample_cluster_kernel<T>, a, C, Q, stream);
}

}  // namespace

int launch_sample(const SampleArgs& a, int num_sms, cudaStream_t s) {
  return a.bf16 ? launch_any<__nv_bfloat16>(a, num_sms, s) : launch_any<float>(a, num_sms, s);
}

}  // namespace g3

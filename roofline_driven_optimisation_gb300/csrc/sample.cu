// Sampling one token of each row of logits (gemm_sample_*; the header states the
// rules).
//
// Weights become whole numbers, mass = floor(2^40 w), so every sum below is exact
// and does not depend on the order in which threads add: histograms may use
// atomics, and the token is the same on every run and for every split of the row.
// A row's ranking is never sorted.  Both cuts (top-k by count, top-p by mass) are
// prefixes of the ranking, so each is a key (the logit's bits in order) and how
// many of the tokens with just that key are kept, lowest index first; a radix
// search over the key's four bytes finds it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "internal.h"
#include "ptx.cuh"

namespace g3 {
namespace {

using ull = unsigned long long;
constexpr int THREADS = 1024, WARPS = THREADS / 32;
constexpr uint32_t kKeyNegInf = 0x007fffffu;   // order_key(-inf), the lowest key

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
__device__ __forceinline__ ull mass_of(float w) { return __float2ull_rz(__fmul_rn(w, 1099511627776.f)); }

// What is kept: keys above `key`, and the first `ties` (by index) equal to it
struct Cut {
  uint32_t key;
  int ties;
};

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
  const bool greedy = !(t >= FLT_MIN);
  const int k = a.top_k ? a.top_k[r] : 0;
  const float p = a.top_p ? a.top_p[r] : 1.f;
  const float least = a.min_p ? a.min_p[r] : 0.f;
  const float u = a.u[r];

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
  const Row row{key_logit(top), greedy ? 1.f : __fdiv_rn(1.f, t)};

  // cuts; key 0 keeps everything
  Cut cut{0u, vocab};
  unsigned n_above = 0, n_equal = 0;
  ull m_above = 0;
  if (greedy || k == 1) {
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
      const double bound = __dmul_rn((double)p, __ull2double_rn(m));
      const uint32_t key = search(logit, vocab, row, cut.key, [&](unsigned c, ull before) {
        return c == 0 || __ull2double_rn(before) < bound;
      }, sh, n_above, m_above, n_equal);
      // how many of the equal ones have less than the bound before them
      const ull one = key > kKeyNegInf ? mass_of(logit_weight(row, key_logit(key))) : 0;
      int lo = 1, hi = (int)n_equal;
      if (key == cut.key) hi = min(hi, cut.ties);
      while (lo < hi) {   // the first always; the j-th (from 0) if before + j * one is below
        const int mid = (lo + hi + 1) / 2;
        if (__ull2double_rn(m_above + (ull)(mid - 1) * one) < bound) lo = mid;
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
    return w >= least || key == top ? mass_of(w) : 0;
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
  const double at = __dmul_rn((double)u, __ull2double_rn(total));
  ull target = at > 0.0 ? __double2ull_rz(at) : 0;   // NaN: 0
  if (target >= total) target = total - 1;
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
          if (a.logprob) a.logprob[r] = logit_z(row, logit(i)) - logf((float)(__ull2double_rn(total) * 0x1p-40));
        }
        break;
      }
      before += __shfl_sync(0xffffffffu, run, 31);
    }
  }
}

template <class Kernel>
int launch(Kernel kernel, dim3 grid, const SampleArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(THREADS);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int launch_sample(const SampleArgs& a, int num_sms, cudaStream_t s) {
  (void)num_sms;
  if (a.bf16) return launch(sample_kernel<__nv_bfloat16>, dim3((unsigned)a.rows), a, s);
  return launch(sample_kernel<float>, dim3((unsigned)a.rows), a, s);
}

}  // namespace g3

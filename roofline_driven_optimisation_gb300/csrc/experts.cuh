// Which rows an expert has, where a row's values come from and where its product goes;
// shared by the block-scaled products.  Everything read from the caller's tables is
// checked here before it becomes an address.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace g3 {

// Rows [begin, begin + count) of the product are expert e's; a range that does not fit
// the call is reported and taken as empty.
__device__ __forceinline__ void expert_rows(const BlocksArgs& a, int e, int& begin, int& count) {
  if (a.offsets == nullptr) {
    begin = 0;
    count = a.rows;
    return;
  }
  begin = a.offsets[e];
  const int end = a.offsets[e + 1];
  count = end - begin;
  if (begin < 0 || end < begin || end > a.rows) {
    report_status(a.status, 1, kSiteExperts);
    begin = count = 0;
  }
}

// Rows that no range covers: nothing multiplies them, so one block says so.
__device__ __forceinline__ bool uncovered_rows(const BlocksArgs& a) {
  return a.offsets != nullptr && (a.offsets[0] != 0 || a.offsets[a.experts] != a.rows);
}

// Row p: `from` A's row (-1: none, taken as zeros), `to` C's row (-1: not stored).
__device__ __forceinline__ void expert_row(const BlocksArgs& a, int p, int& from, int& to) {
  from = to = p;
  if (a.gather == 0 && a.scatter == 0) return;
  const int slot = a.order[p];
  const bool fits = slot >= 0 && slot < a.rows;
  if (!fits) report_status(a.status, 1, kSiteExperts);
  if (a.gather != 0) from = fits ? slot / a.gather : -1;
  if (a.scatter != 0) to = fits ? slot : -1;
}

// ---------------------------------------------------------------- items of the tcgen05 kernels
// One item: `rows` rows p0 .. of expert e, column tile nb.
struct Item {
  int e, p0, rows, nb;
};
// Walks the items of one CTA; every role has its own.  pre[e]: row tiles of the experts
// before e; beg, num: their rows.
struct Walk {
  const int *pre, *beg, *num;
  int nt, tiles_n, e;
  __device__ __forceinline__ Item at(int it) {
    while (it >= pre[e + 1] * tiles_n) ++e;
    const int x = it - pre[e] * tiles_n, tiles = pre[e + 1] - pre[e];
    const int t = x % tiles;
    Item i;
    i.e = e;
    i.nb = x / tiles;
    i.p0 = beg[e] + t * nt;
    i.rows = min(nt, num[e] - t * nt);
    return i;
  }
};

// The lists of a Walk, in shared memory, by one warp: row tiles of NT.  Ranges that overlap
// may come to more tiles than the host has counted on; there is no item then.
constexpr int kListBytes = (3 * kBlocksMaxExperts + 4) * 4;
template <int NT>
__device__ __forceinline__ void list_row_tiles(const BlocksArgs& a, int* pre, int* beg, int* num, int lane) {
  long long run = 0;
  const bool uncovered = blockIdx.x == 0 && lane == 0 && uncovered_rows(a);
  for (int e0 = 0; e0 < a.experts; e0 += 32) {
    const int e = e0 + lane;
    int b = 0, n = 0;
    if (e < a.experts) expert_rows(a, e, b, n);
    const unsigned tiles = ((unsigned)n + NT - 1) / NT;   // 2^26 at most: 32 lanes' fit
    unsigned s = tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned o = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += o;
    }
    if (e < a.experts) {
      pre[e] = (int)(run + s - tiles);
      beg[e] = b;
      num[e] = n;
    }
    run += __shfl_sync(0xffffffffu, s, 31);
  }
  if (lane == 0) {
    const bool fits = run <= blocks_row_tiles(a.rows, a.experts, NT);
    if (!fits || uncovered) report_status(a.status, 1, kSiteExperts);
    pre[a.experts] = fits ? (int)run : 0;
  }
}

// The one item number `it` of a line as a Walk's, into out[0..3] (expert, first row, rows,
// column tile; 0 rows where there are fewer items), by one warp.
template <int NT>
__device__ __forceinline__ void find_item(const BlocksArgs& a, int tiles_n, long long it, int* out, int lane) {
  long long run = 0;                                   // items of the experts before
  const bool uncovered = blockIdx.x == 0 && lane == 0 && uncovered_rows(a);
  if (lane == 0) out[2] = 0;
  __syncwarp();
  for (int e0 = 0; e0 < a.experts; e0 += 32) {
    const int e = e0 + lane;
    int b = 0, n = 0;
    if (e < a.experts) expert_rows(a, e, b, n);
    const int tiles = (int)(((unsigned)n + NT - 1) / NT);
    long long s = (long long)tiles * tiles_n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += o;
    }
    const long long first = run + s - (long long)tiles * tiles_n;
    if (it >= first && it < run + s) {                 // one lane at most
      const int x = (int)(it - first), t = x % tiles;
      out[0] = e;
      out[1] = b + t * NT;
      out[2] = min(NT, n - t * NT);
      out[3] = x / tiles;
    }
    run += __shfl_sync(0xffffffffu, s, 31);
    if (it < run) break;
  }
  if (uncovered) report_status(a.status, 1, kSiteExperts);
}

// ---------------------------------------------------------------- two sums in one instruction
__device__ __forceinline__ void fma2(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ float part2(uint64_t v, int i) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return __uint_as_float(i ? hi : lo);
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t both(float v) { return pack2(__float_as_uint(v), __float_as_uint(v)); }

// silu(gate) * up, twice.  exp(-g) as 2^-p * (1 + r ln 2), p the rounded g * log2(e) and r what
// that rounding left out, so that only the approximate operations and five roundings are left:
// silu is off by at most 5.6 * 2^-24 of itself (of every fp32 gate; expf and a division: 4.2),
// eight instructions in two values' place, and ex2 and rcp for each, where those take forty a
// value (an epilogue of 128 x 256 products: 7.1 us with those, 4.5 one value at a time).  From
// -87.34 down 1/(1 + e^-g) is below 2^-126 and silu 0 (it is less than 2^-119 there; of -inf it
// is NaN), and g is held to 88 in the exponent alone.
__device__ __forceinline__ uint64_t swiglu_near2(uint64_t g, uint64_t u) {
  constexpr float kLog2e = 1.4426950408889634f, kLog2eRest = 1.925963033500e-08f, kLn2 = 0.6931471805599453f;
  uint64_t c = pack2(__float_as_uint(fminf(fmaxf(part2(g, 0), -88.f), 88.f)),
                     __float_as_uint(fminf(fmaxf(part2(g, 1), -88.f), 88.f)));
  const uint64_t p = mul2(c, both(kLog2e));
  uint64_t r = p;
  fma2(r, c, both(-kLog2e));
  fma2(r, c, both(-kLog2eRest));
  float e[2], q[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[i]) : "f"(-part2(p, i)));
  const uint64_t e2 = pack2(__float_as_uint(e[0]), __float_as_uint(e[1]));
  uint64_t d = e2;
  fma2(d, e2, mul2(r, both(kLn2)));
  d = add2(d, both(1.f));
#pragma unroll
  for (int i = 0; i < 2; ++i) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q[i]) : "f"(part2(d, i)));
  return mul2(mul2(g, pack2(__float_as_uint(q[0]), __float_as_uint(q[1]))), u);
}

// alpha * v + beta * C, rounded once to C's type
__device__ __forceinline__ void blocks_store(const BlocksArgs& a, long long m, int n, float v) {
  v *= a.alpha;
  if (a.out_bf16) {
    __nv_bfloat16* c = static_cast<__nv_bfloat16*>(a.C) + m * a.ldc + n;
    if (a.beta != 0.f) v = fmaf(a.beta, __bfloat162float(*c), v);
    *c = __float2bfloat16_rn(v);
  } else {
    float* c = static_cast<float*>(a.C) + m * a.ldc + n;
    if (a.beta != 0.f) v = fmaf(a.beta, *c, v);
    *c = v;
  }
}

}  // namespace g3

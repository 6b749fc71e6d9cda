// Appending to a paged 8-bit key/value cache, with the position rotation of Q and
// K on the way (gemm_kv_append; the header states the arithmetic).
//
// A scale belongs to one page and head, so the work is cut the same way: one
// item is the part of a page that the call writes, times one head.  What an item
// stores depends on nothing outside it, and the rotation, the largest magnitude
// and the codes are computed with the same roundings in every kernel here, so
// all give the same bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"
#include "row_walk.cuh"

namespace g3 {
namespace {

// (a, b) turned by the angle of cosine c and sine s; no fused multiply-add, so
// that every product and sum is rounded by itself
__device__ __forceinline__ float2 turn(float a, float b, float c, float s) {
  return make_float2(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)), __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)));
}

// Two fp32 values in one register pair; each half of a packed product is rounded by
// itself.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 halves_of(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Sums of packed products, in scalar form: a packed sum was seen contracted with the
// packed products before it into a fused multiply-add, which skips a rounding.
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  const float2 x = halves_of(a), y = halves_of(b);
  return pair(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  const float2 x = halves_of(a), y = halves_of(b);
  return pair(__fsub_rn(x.x, y.x), __fsub_rn(x.y, y.y));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// One item: the rows of sequence b's call that fall into one page.
struct Item {
  int b, row0, n;     // sequence; first of its rows in this page, and how many
  int pos0, col;      // position of that row; the page's column in the table
};

// Finds item number i: items count the pages that each sequence writes, in sequence
// order.  Called by the whole block; the first warp looks, four sequences a lane.
// False when there is no such item.
__device__ bool find_item(const KvAppendArgs& a, int i, Item& out) {
  __shared__ Item found;
  __shared__ int found_flag;
  constexpr int PER = 4;
  if (threadIdx.x < 32) {
    const int P = a.c.P, lane = threadIdx.x;
    int before = 0;
    bool hit = false;
    for (int b0 = 0; b0 < a.c.seqs && !hit && before <= i; b0 += 32 * PER) {
      int first[PER], n[PER], base[PER], count[PER], own = 0;
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        const int b = b0 + lane * PER + q;
        first[q] = n[q] = base[q] = count[q] = 0;
        if (b < a.c.seqs) {
          base[q] = a.base[b];
          kv_rows(a.start, b, a.tokens, a.max_new, a.status, kSiteKvAppend, first[q], n[q]);
        }
      }
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        if (n[q] > 0) {
          // positions base .. base+n-1 must exist in the tables of angles
          if (base[q] < 0 || base[q] > a.positions - n[q]) report_status(a.status, 1, kSiteKvAppend);
          else count[q] = (base[q] + n[q] - 1) / P - base[q] / P + 1;
        }
        own += count[q];
      }
      int excl = own;
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, excl, o);
        if (lane >= o) excl += t;
      }
      const int all = __shfl_sync(0xffffffffu, excl, 31);
      excl += before - own;
      bool mine = false;
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        if (count[q] > 0 && i >= excl && i < excl + count[q]) {
          found.b = b0 + lane * PER + q;
          found.col = base[q] / P + (i - excl);
          // the page's end may lie behind 2^31 - 1, the last row does not
          const int lo = max(base[q], found.col * P);
          const int hi = (int)min((long long)base[q] + n[q], ((long long)found.col + 1) * P);
          found.row0 = first[q] + (lo - base[q]);
          found.n = hi - lo;
          found.pos0 = lo;
          mine = true;
        }
        excl += count[q];
      }
      hit = __any_sync(0xffffffffu, mine);
      before += all;
    }
    if (lane == 0) found_flag = hit;
  }
  __syncthreads();
  out = found;
  return found_flag != 0;
}

__device__ __forceinline__ float block_max(float x, float* red) {
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
  __syncthreads();
  x = red[0];
  for (int w = 1; w < (int)blockDim.x / 32; ++w) x = fmaxf(x, red[w]);
  __syncthreads();
  return x;
}

// Codes of an item's page that were there before the call, from scale s0 to the
// larger scale with reciprocal r.
template <int FMT>
__device__ __forceinline__ uint32_t recode(uint32_t code, float s0, float r) {
  const float2 v = kv_value2<FMT>(code);
  return kv_code2<FMT>(__fmul_rn(__fmul_rn(v.x, s0), r), 0.f) & 0xffu;
}

// ------------------------------------------------------------------ generic
// Any head width, page size, rotation width and alignment: a block for each
// item and head, one value (or one pair of the rotation) at a time.  Bound by the latency
// of its loads, of which K and V take two passes.  4096 tokens, 32 query and 8 key heads:
// 80 wide in pages of 16 41 us, 128 wide with half of it turned 76 (whole, on the fast
// kernel, 23), in pages of 256 tokens 158; 16384 of 32 and 32 heads with 32 of 128 turned
// 646.
template <int FMT>
__global__ void __launch_bounds__(128) kv_append_generic_kernel(const KvAppendArgs a) {
  __shared__ float red[4];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  Item it;
  if (!find_item(a, blockIdx.x, it)) return;
  const int D = a.c.D, R = a.rot, half = R / 2;
  const int hh = blockIdx.y;   // query heads, then key heads, then value heads
  const int kind = hh < a.Hq ? 0 : hh < a.Hq + a.c.H ? 1 : 2;
  const int h = kind == 0 ? hh : (hh - a.Hq) % a.c.H;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(kind == 0 ? a.Q : kind == 1 ? a.K : a.V);
  const long long ld = kind == 0 ? a.ldq : kind == 1 ? a.ldk : a.ldv;
  const int rot = kind == 2 ? 0 : half;   // pairs that turn
  // unit u of a row: pair u for u < rot, then single values
  const int units = rot + (D - 2 * rot);
  auto unit = [&](int u, int& d0, int& d1) {
    if (u < rot) {
      d0 = a.interleaved ? 2 * u : u;
      d1 = a.interleaved ? 2 * u + 1 : u + half;
    } else {
      d0 = u + rot;
      d1 = -1;
    }
  };
  auto value = [&](int t, int u, int& d0, int& d1) -> float2 {
    unit(u, d0, d1);
    const __nv_bfloat16* x = src + (long long)(it.row0 + t) * ld + (long long)h * D;
    const float x0 = __bfloat162float(x[d0]);
    if (d1 < 0) return make_float2(x0, 0.f);
    const long long at = (long long)(it.pos0 + t) * half + u;
    return turn(x0, __bfloat162float(x[d1]), a.cos[at], a.sin[at]);
  };
  int d0, d1;
  if (kind == 0) {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.Qo);
    for (RowWalk e(threadIdx.x, blockDim.x, units); e.within(it.n); e.next()) {
      const int t = (int)e.row;
      const float2 y = value(t, e.at, d0, d1);
      __nv_bfloat16* o = out + (long long)(it.row0 + t) * a.ldqo + (long long)h * D;
      o[d0] = __float2bfloat16_rn(y.x);
      if (d1 >= 0) o[d1] = __float2bfloat16_rn(y.y);
    }
    return;
  }
  const int g = kv_page(a.c, it.b, it.col, a.status, kSiteKvAppend);
  if (g < 0) return;
  float* scale = (kind == 1 ? a.c.ks : a.c.vs) + (long long)g * a.c.H + h;
  uint8_t* codes = (kind == 1 ? a.c.k : a.c.v) + (long long)g * a.c.ps + (long long)h * a.c.hs;
  float m = 0.f;
  for (RowWalk e(threadIdx.x, blockDim.x, units); e.within(it.n); e.next()) {
    const float2 y = value((int)e.row, e.at, d0, d1);
    m = fmaxf(m, fmaxf(fabsf(y.x), fabsf(y.y)));
  }
  const int held = it.pos0 % a.c.P;              // earlier tokens of this page
  const float s0 = held > 0 ? *scale : 0.f;
  m = block_max(m, red);                         // every thread has read *scale
  const float s = fmaxf(s0, kv_scale_for<FMT>(m)), r = kv_recip(s);
  for (RowWalk e(threadIdx.x, blockDim.x, units); e.within(it.n); e.next()) {
    const int t = (int)e.row;
    const float2 y = value(t, e.at, d0, d1);
    uint8_t* o = codes + (long long)(held + t) * a.c.ts;
    const uint32_t c2 = kv_code2<FMT>(__fmul_rn(y.x, r), __fmul_rn(y.y, r));
    o[d0] = (uint8_t)c2;
    if (d1 >= 0) o[d1] = (uint8_t)(c2 >> 8);
  }
  if (s > s0 && held > 0) {
    for (RowWalk e(threadIdx.x, blockDim.x, D); e.within(held); e.next()) {
      uint8_t* o = codes + (long long)e.row * a.c.ts + e.at;
      *o = (uint8_t)recode<FMT>(*o, s0, r);
    }
  }
  if (threadIdx.x == 0) *scale = s;
}

// ------------------------------------------------------------------ fast
// D 64 or 128, whole heads turned, pages of 16 to 128 tokens, rows on 16 bytes.
// The bound is HBM (2 bytes in and 1 or 2 out a value); what a kernel has to do is
// read each value once, with enough loads in flight, and keep it until its page's
// scale is known.  Measured on one GB300 (6.79 TB/s copied): 16384 tokens of 32 query
// and 32 key heads of 128, E4M3, 679.5 MB in 129 us, 5.3 TB/s, 0.78 of the copy rate
// (DRAM 66 % busy, the issue slots 44 %; the rest is the wait for a head's copies and
// the barrier a head).  7 prompts of about 611 tokens (25 MB) 9.6 us, 64 x 1 token
// 3.6 us, one token 2.4 us: launch and one chain of dependent loads.

// eight bf16 as four pairs of floats: neighbours
__device__ __forceinline__ void unpack8(const uint4& v, uint64_t (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
// eight bf16 of each vector as pairs (x[i], x[i + 1]) of the firsts and the seconds of
// each neighbours
__device__ __forceinline__ void split8(const uint4& v, uint64_t (&even)[2], uint64_t (&odd)[2]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    even[i] = pair(__uint_as_float(w[2 * i] << 16), __uint_as_float(w[2 * i + 1] << 16));
    odd[i] = pair(__uint_as_float(w[2 * i] & 0xffff0000u), __uint_as_float(w[2 * i + 1] & 0xffff0000u));
  }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <int FMT>
__device__ __forceinline__ uint32_t codes4(uint64_t lo, uint64_t hi, uint64_t r2) {
  const float2 a = halves_of(mul2(lo, r2)), b = halves_of(mul2(hi, r2));
  return kv_code2<FMT>(a.x, a.y) | (kv_code2<FMT>(b.x, b.y) << 16);
}
template <int FMT>
__device__ __forceinline__ uint32_t recode4(uint32_t c, float s0, float r) {
  const float2 a = kv_value2<FMT>(c & 0xffffu), b = kv_value2<FMT>(c >> 16);
  return kv_code2<FMT>(__fmul_rn(__fmul_rn(a.x, s0), r), __fmul_rn(__fmul_rn(a.y, s0), r)) |
         (kv_code2<FMT>(__fmul_rn(__fmul_rn(b.x, s0), r), __fmul_rn(__fmul_rn(b.y, s0), r)) << 16);
}

// A few tokens a sequence, MAXT at most (a decode step, drafted tokens): a warp for
// each sequence, page and head with the tokens in registers, so that the latency of a
// call is one chain of loads (row range and position; row, page and angles; scale), and
// no block waits.
constexpr int DEC_WARPS = 4;

template <int FMT, int D, int MAXT>
__global__ void __launch_bounds__(DEC_WARPS * 32) kv_append_tokens_kernel(const KvAppendArgs a, const int pages) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  constexpr int PP = D / 64;                       // pairs of a lane
  const int lane = threadIdx.x % 32, hh = blockIdx.x * DEC_WARPS + threadIdx.x / 32;
  const int b = pages == 1 ? blockIdx.y : blockIdx.y / pages, nth = blockIdx.y - b * pages;   // its nth page
  if (hh >= a.Hq + 2 * a.c.H) return;
  const int kind = hh < a.Hq ? 0 : hh < a.Hq + a.c.H ? 1 : 2;
  const int h = kind == 0 ? hh : (hh - a.Hq) - (kind - 1) * a.c.H;
  const int base = a.base[b];
  int first, all;
  kv_rows(a.start, b, a.tokens, a.max_new, a.status, kSiteKvAppend, first, all);
  if (all == 0) return;
  if (base < 0 || base > a.positions - all) {
    report_status(a.status, 1, kSiteKvAppend);
    return;
  }
  const int col = base / a.c.P + nth, end = base + all;
  const long long page = (long long)col * a.c.P;   // the page's first position, and its end: up to 2^31 and more
  if (page >= end) return;
  const int pos = max(base, (int)page), n = (int)min((long long)end, page + a.c.P) - pos, held = pos - (int)page;
  const int row = first + (pos - base);
  const long long ld = kind == 0 ? a.ldq : kind == 1 ? a.ldk : a.ldv;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(kind == 0 ? a.Q : kind == 1 ? a.K : a.V) +
                             (long long)row * ld + (long long)h * D;
  // values d0 .., d1 ..: PP each; a pair of the rotation, or neighbours
  const bool halves = kind != 2 && !a.interleaved;
  const int d0 = halves ? lane * PP : lane * 2 * PP, d1 = halves ? d0 + D / 2 : d0 + PP;
  float x[MAXT][2 * PP];
#pragma unroll
  for (int t = 0; t < MAXT; ++t) {
#pragma unroll
    for (int i = 0; i < 2 * PP; ++i) x[t][i] = 0.f;
    if (t >= n) continue;
    const __nv_bfloat16* p = src + t * ld;
    if constexpr (PP == 2) {
      const uint32_t u = *reinterpret_cast<const uint32_t*>(p + d0), v = *reinterpret_cast<const uint32_t*>(p + d1);
      x[t][0] = __uint_as_float(u << 16);
      x[t][1] = __uint_as_float(u & 0xffff0000u);
      x[t][2] = __uint_as_float(v << 16);
      x[t][3] = __uint_as_float(v & 0xffff0000u);
    } else {
      x[t][0] = __bfloat162float(p[d0]);
      x[t][1] = __bfloat162float(p[d1]);
    }
  }
  // the page and its scale while the rows arrive
  const int g = kind == 0 ? 0 : kv_page(a.c, b, col, a.status, kSiteKvAppend);
  if (g < 0) return;
  float* scale = (kind == 1 ? a.c.ks : a.c.vs) + (long long)g * a.c.H + h;
  const float s0 = kind != 0 && held > 0 ? *scale : 0.f;
  if (kind != 2) {
    // halves: pairs (x[i], x[PP + i]); interleaved: (x[2i], x[2i + 1])
#pragma unroll
    for (int t = 0; t < MAXT; ++t) {
      if (t >= n) continue;
      const long long at = (long long)(pos + t) * (D / 2) + lane * PP;
#pragma unroll
      for (int i = 0; i < PP; ++i) {
        const float c = a.cos[at + i], s = a.sin[at + i];
        float& p = halves ? x[t][i] : x[t][2 * i];
        float& q = halves ? x[t][PP + i] : x[t][2 * i + 1];
        const float2 y = turn(p, q, c, s);
        p = y.x;
        q = y.y;
      }
    }
  }
  if (kind == 0) {
#pragma unroll
    for (int t = 0; t < MAXT; ++t) {
      if (t >= n) continue;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.Qo) + (long long)(row + t) * a.ldqo + (long long)h * D;
      if constexpr (PP == 2) {
        *reinterpret_cast<uint32_t*>(o + d0) = pack2(x[t][0], x[t][1]);
        *reinterpret_cast<uint32_t*>(o + d1) = pack2(x[t][2], x[t][3]);
      } else {
        o[d0] = __float2bfloat16_rn(x[t][0]);
        o[d1] = __float2bfloat16_rn(x[t][1]);
      }
    }
    return;
  }
  uint8_t* codes = (kind == 1 ? a.c.k : a.c.v) + (long long)g * a.c.ps + (long long)h * a.c.hs;
  float m = 0.f;
#pragma unroll
  for (int t = 0; t < MAXT; ++t)
#pragma unroll
    for (int i = 0; i < 2 * PP; ++i) m = fmaxf(m, fabsf(x[t][i]));
  m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
  const float s = fmaxf(s0, kv_scale_for<FMT>(m)), r = kv_recip(s);
#pragma unroll
  for (int t = 0; t < MAXT; ++t) {
    if (t >= n) continue;
    uint8_t* o = codes + (long long)(held + t) * a.c.ts;
    if constexpr (PP == 2) {
      *reinterpret_cast<uint16_t*>(o + d0) = (uint16_t)kv_code2<FMT>(__fmul_rn(x[t][0], r), __fmul_rn(x[t][1], r));
      *reinterpret_cast<uint16_t*>(o + d1) = (uint16_t)kv_code2<FMT>(__fmul_rn(x[t][2], r), __fmul_rn(x[t][3], r));
    } else {
      const uint32_t c = kv_code2<FMT>(__fmul_rn(x[t][0], r), __fmul_rn(x[t][1], r));
      o[d0] = (uint8_t)c;
      o[d1] = (uint8_t)(c >> 8);
    }
  }
  if (s > s0 && held > 0) {
    constexpr int LANES = D / 4;                   // lanes of a row of codes
    const int sub = lane / LANES, at = lane % LANES * 4;
#pragma unroll 4
    for (int t = sub; t < held; t += 32 / LANES) {
      uint32_t* w = reinterpret_cast<uint32_t*>(codes + (long long)t * a.c.ts + at);
      *w = recode4<FMT>(*w, s0, r);
    }
  }
  if (lane == 0) *scale = s;
}

// Prompts: a block takes one item and walks through `per` heads of it, 16 values of a
// row a thread (a pair of octets that turn together, or neighbours), TPT rows a
// thread.  The angles are read once for all heads.  Every thread copies its own bytes
// of the next STAGES heads ahead into shared memory, so nothing waits for them but the
// thread itself; the one barrier a head is for the largest magnitude.  Steps on 16384
// tokens: a page of four heads in registers with two blocks an SM 149 us, two heads
// and packed products 142, these copies 138, one loop for each of Q, K and V with
// running addresses 129 (99 to 71 million instructions).  Six stages ahead, or two or
// eight rounds of blocks in place of four, change it by 2 % at most.
constexpr int STAGES = 4;
constexpr int PAGE_THREADS = 512;

template <int FMT, int D, int TPT>
__global__ void __launch_bounds__(PAGE_THREADS, TPT == 1 ? 2 : 1) kv_append_pages_kernel(const KvAppendArgs a, const int per) {
  extern __shared__ __align__(16) uint8_t ahead[];   // [stage][row of the thread][octet][thread] 16 bytes
  __shared__ unsigned big[3];
  constexpr int CH = D / 16;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  if (threadIdx.x < 3) big[threadIdx.x] = 0;
  Item it;
  if (!find_item(a, blockIdx.x, it)) return;
  const int t0 = threadIdx.x / CH, c = threadIdx.x % CH, step = blockDim.x / CH;
  const int held = it.pos0 % a.c.P, n = it.n;
  const int from = blockIdx.y * per, to = min(a.Hq + 2 * a.c.H, from + per);   // query, key, value heads
  const int k_from = a.Hq, v_from = a.Hq + a.c.H;
  // octets of this thread: of a rotation by halves, or neighbours
  const int dn0 = c * 16, dn1 = dn0 + 8, dr0 = a.interleaved ? dn0 : c * 8, dr1 = a.interleaved ? dn1 : dr0 + D / 2;

  // ---- the copies ahead: a running place in Q, then K, then V
  const uint32_t mine = smem_u32(ahead) + threadIdx.x * 16, octet = blockDim.x * 16;   // [stage][row][octet][thread]
  const uint32_t stage_bytes = octet * 2 * TPT;
  const __nv_bfloat16* fetch_row[TPT];
  int fetch_head = from;
  uint32_t fetch_to = mine;
  auto fetch_start = [&]() {                         // the row in the tensor that fetch_head is in
    const int kind = fetch_head < k_from ? 0 : fetch_head < v_from ? 1 : 2;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(kind == 0 ? a.Q : kind == 1 ? a.K : a.V) +
                               (long long)(fetch_head - (kind == 0 ? 0 : kind == 1 ? k_from : v_from)) * D;
    const long long ld = kind == 0 ? a.ldq : kind == 1 ? a.ldk : a.ldv;
#pragma unroll
    for (int q = 0; q < TPT; ++q) {
      const int t = t0 + q * step;
      fetch_row[q] = src + (long long)(it.row0 + (t < n ? t : 0)) * ld;
    }
  };
  auto fetch = [&]() {
    if (fetch_head < to) {
      const bool value = fetch_head >= v_from;
      const int d0 = value ? dn0 : dr0, d1 = value ? dn1 : dr1;
#pragma unroll
      for (int q = 0; q < TPT; ++q) {
        const bool read = t0 + q * step < n;
        cp_async_16(fetch_to + q * 2 * octet, fetch_row[q] + d0, read);
        cp_async_16(fetch_to + q * 2 * octet + octet, fetch_row[q] + d1, read);
        fetch_row[q] += D;
      }
      ++fetch_head;
      if (fetch_head == k_from || fetch_head == v_from) fetch_start();
      fetch_to = fetch_to + stage_bytes == mine + STAGES * stage_bytes ? mine : fetch_to + stage_bytes;
    }
    cp_async_commit();                               // one group a head, also an empty one
  };
  fetch_start();
#pragma unroll
  for (int i = 0; i < STAGES; ++i) fetch();
  uint64_t co[TPT][4], si[TPT][4];                   // angles of eight pairs, two in each
  if (from < v_from) {
#pragma unroll
    for (int q = 0; q < TPT; ++q) {
      const int t = min(t0 + q * step, n - 1);
      const long long at = (long long)(it.pos0 + t) * (D / 2) + c * 8;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(a.cos + at + 4 * i);
        const float4 y = *reinterpret_cast<const float4*>(a.sin + at + 4 * i);
        co[q][2 * i] = pair(x.x, x.y);
        co[q][2 * i + 1] = pair(x.z, x.w);
        si[q][2 * i] = pair(y.x, y.y);
        si[q][2 * i + 1] = pair(y.z, y.w);
      }
    }
  }
  int stage = 0, turn = 0;
  // the next head's 16 values, turned: neighbours in pairs, d0's octet then d1's
  auto values = [&](auto turned, auto by_halves, uint64_t (&x)[TPT][8]) {
    cp_async_wait<STAGES - 1>();
    const uint4* in = reinterpret_cast<const uint4*>(ahead + stage * stage_bytes) + threadIdx.x;
#pragma unroll
    for (int q = 0; q < TPT; ++q) {
      const uint4 u = in[q * 2 * blockDim.x], v = in[(q * 2 + 1) * blockDim.x];
      if constexpr (!decltype(turned)::value || decltype(by_halves)::value) {
        uint64_t p[4], w[4];
        unpack8(u, p);
        unpack8(v, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (decltype(turned)::value) {
            x[q][i] = sub2(mul2(p[i], co[q][i]), mul2(w[i], si[q][i]));
            x[q][4 + i] = add2(mul2(w[i], co[q][i]), mul2(p[i], si[q][i]));
          } else {
            x[q][i] = p[i];
            x[q][4 + i] = w[i];
          }
        }
      } else {
        uint64_t even[4], odd[4];
        split8(u, reinterpret_cast<uint64_t(&)[2]>(even[0]), reinterpret_cast<uint64_t(&)[2]>(odd[0]));
        split8(v, reinterpret_cast<uint64_t(&)[2]>(even[2]), reinterpret_cast<uint64_t(&)[2]>(odd[2]));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 y = halves_of(sub2(mul2(even[i], co[q][i]), mul2(odd[i], si[q][i])));
          const float2 z = halves_of(add2(mul2(odd[i], co[q][i]), mul2(even[i], si[q][i])));
          x[q][2 * i] = pair(y.x, z.x);
          x[q][2 * i + 1] = pair(y.y, z.y);
        }
      }
    }
    stage = (stage + 1) % STAGES;
    fetch();                                         // into the slots just read
  };
  auto queries = [&](auto by_halves, int h0, int h1) {
    constexpr bool H = decltype(by_halves)::value;
    const int d0 = H ? c * 8 : dn0, d1 = H ? d0 + D / 2 : dn1;
    __nv_bfloat16* out[TPT];
#pragma unroll
    for (int q = 0; q < TPT; ++q)
      out[q] = static_cast<__nv_bfloat16*>(a.Qo) + (long long)(it.row0 + t0 + q * step) * a.ldqo + (long long)h0 * D;
    for (int h = h0; h < h1; ++h) {
      uint64_t x[TPT][8];
      values(std::true_type{}, by_halves, x);
#pragma unroll
      for (int q = 0; q < TPT; ++q) {
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = halves_of(x[q][i]);
          y[i] = pack2(f.x, f.y);
        }
        if (t0 + q * step < n) {
          *reinterpret_cast<uint4*>(out[q] + d0) = make_uint4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<uint4*>(out[q] + d1) = make_uint4(y[4], y[5], y[6], y[7]);
        }
        out[q] += D;
      }
    }
  };
  // Key or value heads h0 .. h1-1 of page g.  Three words take the magnitudes by
  // turns: one fills, one is read, one is set back.
  auto stored = [&](auto turned, auto by_halves, uint8_t* all, float* scales, int g, int h0, int h1) {
    constexpr bool H = decltype(turned)::value && decltype(by_halves)::value;
    const int d0 = H ? c * 8 : dn0, d1 = d0 + D / 2;
    uint8_t* codes = all + (long long)g * a.c.ps + (long long)h0 * a.c.hs;
    float* scale = scales + (long long)g * a.c.H + h0;
    const long long at = (long long)(held + t0) * a.c.ts + d0, row_step = (long long)step * a.c.ts;
    for (int h = h0; h < h1; ++h, codes += a.c.hs, ++scale) {
      const float s0 = held > 0 ? *scale : 0.f;
      uint64_t x[TPT][8];
      values(turned, by_halves, x);
      float m = 0.f;
#pragma unroll
      for (int q = 0; q < TPT; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = halves_of(x[q][i]);
          m = max3(m, fabsf(f.x), fabsf(f.y));
        }
      // magnitudes order as their bits; the atomic is a maximum, so its order is free
      const unsigned w = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
      if (threadIdx.x % 32 == 0) atomicMax(&big[turn], w);
      __syncthreads();                               // and every thread has the old scale
      const float s = fmaxf(s0, kv_scale_for<FMT>(__uint_as_float(big[turn]))), r = kv_recip(s);
      const int back = turn == 0 ? 2 : turn - 1;
      turn = turn == 2 ? 0 : turn + 1;
      if (threadIdx.x == 0) {
        big[back] = 0;
        *scale = s;
      }
      const uint64_t r2 = pair(r, r);
#pragma unroll
      for (int q = 0; q < TPT; ++q) {
        const uint2 lo = make_uint2(codes4<FMT>(x[q][0], x[q][1], r2), codes4<FMT>(x[q][2], x[q][3], r2));
        const uint2 hi = make_uint2(codes4<FMT>(x[q][4], x[q][5], r2), codes4<FMT>(x[q][6], x[q][7], r2));
        if (t0 + q * step < n) {
          uint8_t* o = codes + at + q * row_step;
          if constexpr (H) {
            *reinterpret_cast<uint2*>(o) = lo;
            *reinterpret_cast<uint2*>(o + (d1 - d0)) = hi;
          } else {
            *reinterpret_cast<uint4*>(o) = make_uint4(lo.x, lo.y, hi.x, hi.y);
          }
        }
      }
      if (held > 0 && s > s0) {
        for (int e = threadIdx.x; e < held * (D / 4); e += blockDim.x) {
          uint32_t* w4 = reinterpret_cast<uint32_t*>(codes + (long long)(e / (D / 4)) * a.c.ts) + e % (D / 4);
          *w4 = recode4<FMT>(*w4, s0, r);
        }
      }
    }
  };
  using std::false_type;
  using std::true_type;
  if (from < k_from) {
    if (a.interleaved) queries(false_type{}, from, min(to, k_from));
    else queries(true_type{}, from, min(to, k_from));
  }
  const int g = to > k_from ? kv_page(a.c, it.b, it.col, a.status, kSiteKvAppend) : -1;
  if (g >= 0) {                                      // the same for the whole block
    const int k0 = max(from, k_from), k1 = min(to, v_from), v0 = max(from, v_from);
    if (k0 < k1) {
      if (a.interleaved) stored(true_type{}, false_type{}, a.c.k, a.c.ks, g, k0 - k_from, k1 - k_from);
      else stored(true_type{}, true_type{}, a.c.k, a.c.ks, g, k0 - k_from, k1 - k_from);
    }
    if (v0 < to) stored(false_type{}, false_type{}, a.c.v, a.c.vs, g, v0 - v_from, to - v_from);
  }
  cp_async_wait<0>();                                // nothing lands after the block has left
}

template <class Kernel, class... More>
int launch(Kernel kernel, dim3 grid, dim3 block, size_t smem, const KvAppendArgs& a, cudaStream_t s, More... more) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, more...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int FMT, int D, int TPT>
int launch_pages(const KvAppendArgs& a, long long items, int threads, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = set_smem_once(smem_set, kv_append_pages_kernel<FMT, D, TPT>, STAGES * TPT * 32 * PAGE_THREADS);
  if (e != cudaSuccess) return e;
  // heads of a block: as many as leave the GPU four rounds of blocks
  const int heads = a.Hq + 2 * a.c.H;
  const long long resident = (long long)num_sms * (2 * PAGE_THREADS / threads);
  long long groups = (4 * resident + items - 1) / items;
  groups = groups < 1 ? 1 : groups > (heads + 1) / 2 ? (heads + 1) / 2 : groups;
  const int per = (int)((heads + groups - 1) / groups);
  return launch(kv_append_pages_kernel<FMT, D, TPT>, dim3((unsigned)items, (unsigned)((heads + per - 1) / per)),
                dim3((unsigned)threads), (size_t)STAGES * TPT * 32 * threads, a, s, per);
}

template <int FMT, int D>
int launch_fast(const KvAppendArgs& a, long long items, int num_sms, cudaStream_t s) {
  const int heads = a.Hq + 2 * a.c.H;
  // Up to 16 tokens a sequence, a warp keeps them, as long as the grid's second extent
  // holds the sequences' pages.  Measured (32 query and 8 key heads of 128, pages of
  // 64), this kernel against the one below: 64 sequences of up to 3 tokens 5.2 against
  // 17.3 us, of up to 14 9.9 against 17.6; 256 of up to 14 24.2 against 44.7.  One
  // sequence of 8 tokens 4.2 against 4.2, of 15 6.3 against 4.2: a few sequences of
  // many tokens keep more threads busy below.
  const long long pages = (a.max_new + a.c.P - 2) / a.c.P + 1;
  if ((a.max_new <= 8 || (a.max_new <= 16 && a.c.seqs >= 32)) && a.c.seqs * pages <= 65535) {
    const dim3 grid((unsigned)((heads + DEC_WARPS - 1) / DEC_WARPS), (unsigned)(a.c.seqs * pages)), block(DEC_WARPS * 32);
    if (a.max_new == 1) return launch(kv_append_tokens_kernel<FMT, D, 1>, grid, block, 0, a, s, (int)pages);
    if (a.max_new == 2) return launch(kv_append_tokens_kernel<FMT, D, 2>, grid, block, 0, a, s, (int)pages);
    if (a.max_new <= 8) return launch(kv_append_tokens_kernel<FMT, D, 8>, grid, block, 0, a, s, (int)pages);
    return launch(kv_append_tokens_kernel<FMT, D, 16>, grid, block, 0, a, s, (int)pages);
  }
  // a page's threads, 16 values of a row each, two rows where that is above 512
  const int threads = a.c.P * (D / 16), tpt = threads <= PAGE_THREADS ? 1 : threads / PAGE_THREADS;
  if constexpr (D == 128)
    if (tpt == 2) return launch_pages<FMT, D, 2>(a, items, threads / 2, num_sms, s);
  return launch_pages<FMT, D, 1>(a, items, threads, num_sms, s);
}

}  // namespace

int launch_kv_append(const KvAppendArgs& a, bool fast, int num_sms, cudaStream_t s) {
  // a sequence of n rows writes at most (n - 1) / P + 2 pages
  const long long items = (long long)a.tokens / a.c.P + 2ll * (a.c.seqs < a.tokens ? a.c.seqs : a.tokens);
  if (items > 0x7fffffffll) return cudaErrorInvalidValue;
  if (fast) {
    if (a.c.fmt == kKvE4M3)
      return a.c.D == 128 ? launch_fast<kKvE4M3, 128>(a, items, num_sms, s) : launch_fast<kKvE4M3, 64>(a, items, num_sms, s);
    return a.c.D == 128 ? launch_fast<kKvInt8, 128>(a, items, num_sms, s) : launch_fast<kKvInt8, 64>(a, items, num_sms, s);
  }
  const dim3 grid((unsigned)items, (unsigned)(a.Hq + 2 * a.c.H));
  if (a.c.fmt == kKvE4M3) return launch(kv_append_generic_kernel<kKvE4M3>, grid, dim3(128), 0, a, s);
  return launch(kv_append_generic_kernel<kKvInt8>, grid, dim3(128), 0, a, s);
}

}  // namespace g3

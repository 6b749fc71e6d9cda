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

#include "internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace g3 {
namespace {

// (a, b) turned by the angle of cosine c and sine s; no fused multiply-add, so
// that every product and sum is rounded by itself
__device__ __forceinline__ float2 turn(float a, float b, float c, float s) {
  return make_float2(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)), __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)));
}

// One item: the rows of sequence b's call that fall into one page.
struct Item {
  int b, row0, n;     // sequence; first of its rows in this page, and how many
  int pos0, col;      // position of that row; the page's column in the table
};

// Finds item number i: items count the pages that each sequence writes, in
// sequence order.  Called by the whole block (blockDim.x a multiple of 32, at
// most 1024).  False when there is no such item.
__device__ bool find_item(const KvAppendArgs& a, int i, Item& out) {
  __shared__ int warp_sum[32];
  __shared__ Item found;
  __shared__ int found_flag;
  const int P = a.c.P;
  if (threadIdx.x == 0) found_flag = 0;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  int before = 0;
  for (int b0 = 0; b0 < a.c.seqs; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int first = 0, n = 0, base = 0, count = 0;
    if (b < a.c.seqs) {
      kv_rows(a.start, b, a.tokens, a.max_new, a.status, kSiteKvAppend, first, n);
      if (n > 0) {
        base = a.base[b];
        // positions base .. base+n-1 must exist in the tables of angles
        if (base < 0 || base > a.positions - n) {
          report_status(a.status, 1, kSiteKvAppend);
          n = 0;
        } else {
          count = (base + n - 1) / P - base / P + 1;
        }
      }
    }
    int incl = count;
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    __syncthreads();   // the previous round's readers are done with warp_sum
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int excl = before + incl - count, all = before;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) excl += warp_sum[w];
      all += warp_sum[w];
    }
    if (count > 0 && i >= excl && i < excl + count) {
      found.b = b;
      found.col = base / P + (i - excl);
      const int lo = max(base, found.col * P), hi = min(base + n, (found.col + 1) * P);
      found.row0 = first + (lo - base);
      found.n = hi - lo;
      found.pos0 = lo;
      found_flag = 1;
    }
    before = all;
    if (before > i) break;
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
// item and head, one value (or one pair of the rotation) at a time.
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
    for (int e = threadIdx.x; e < it.n * units; e += blockDim.x) {
      const int t = e / units;
      const float2 y = value(t, e % units, d0, d1);
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
  for (int e = threadIdx.x; e < it.n * units; e += blockDim.x) {
    const float2 y = value(e / units, e % units, d0, d1);
    m = fmaxf(m, fmaxf(fabsf(y.x), fabsf(y.y)));
  }
  const int held = it.pos0 % a.c.P;              // earlier tokens of this page
  const float s0 = held > 0 ? *scale : 0.f;
  m = block_max(m, red);                         // every thread has read *scale
  const float s = fmaxf(s0, kv_scale_for<FMT>(m)), r = kv_recip(s);
  for (int e = threadIdx.x; e < it.n * units; e += blockDim.x) {
    const int t = e / units;
    const float2 y = value(t, e % units, d0, d1);
    uint8_t* o = codes + (long long)(held + t) * a.c.ts;
    const uint32_t c2 = kv_code2<FMT>(__fmul_rn(y.x, r), __fmul_rn(y.y, r));
    o[d0] = (uint8_t)c2;
    if (d1 >= 0) o[d1] = (uint8_t)(c2 >> 8);
  }
  if (s > s0 && held > 0) {
    for (int e = threadIdx.x; e < held * D; e += blockDim.x) {
      uint8_t* o = codes + (long long)(e / D) * a.c.ts + e % D;
      *o = (uint8_t)recode<FMT>(*o, s0, r);
    }
  }
  if (threadIdx.x == 0) *scale = s;
}

template <class Kernel>
int launch(Kernel kernel, dim3 grid, dim3 block, const KvAppendArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int launch_kv_append(const KvAppendArgs& a, bool fast, int num_sms, cudaStream_t s) {
  // a sequence of n rows writes at most (n - 1) / P + 2 pages
  const long long items = a.max_new == 1 ? a.tokens : (long long)a.tokens / a.c.P + 2ll * min(a.c.seqs, a.tokens);
  if (items > 0x7fffffffll) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)items, (unsigned)(a.Hq + 2 * a.c.H));
  if (a.c.fmt == kKvE4M3) return launch(kv_append_generic_kernel<kKvE4M3>, grid, dim3(128), a, s);
  return launch(kv_append_generic_kernel<kKvInt8>, grid, dim3(128), a, s);
}

}  // namespace g3

// Rows held in E4M3 with a scale for each block of 1 x 128 values (activations) or
// 128 x 128 (weights): gemm_fp8_quantise_*.
//
// With a the largest magnitude of a block (NaN ignored, at most FLT_MAX):
//
//     s = a / 448, or 0 below 2^-126;  code = x * (1/s) to nearest even on E4M3's grid
//
// every operation rounded to fp32 by itself, as the paged cache's codes are.  One pass:
// a block's values stay in registers between the maximum and the codes, so each input
// byte is read once and each output byte written once; HBM bounds it (3 bytes a bf16
// value).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace g3 {
namespace {

constexpr int QB = 128;            // values of a block along a row
constexpr int HALF = 16;           // lanes that share 128 values of a row: 8 each
constexpr int THREADS = 256;
constexpr int HALVES = THREADS / HALF;

template <typename T>
__device__ __forceinline__ float q_f32(T v);
template <>
__device__ __forceinline__ float q_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float q_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// 8 values from x[0..7], of which `n` exist (0 in the place of the others)
template <typename T>
__device__ __forceinline__ void load8(const T* x, int n, bool vec, float (&v)[8]) {
  if (vec && n >= 8) {
#pragma unroll
    for (int q = 0; q < (int)sizeof(T) / 2; ++q) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(x) + q);
      alignas(16) T part[16 / sizeof(T)];
      *reinterpret_cast<uint4*>(part) = w;
#pragma unroll
      for (int i = 0; i < (int)(16 / sizeof(T)); ++i) v[q * (int)(16 / sizeof(T)) + i] = q_f32(part[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? q_f32(x[i]) : 0.f;
  }
}

__device__ __forceinline__ float big8(const float (&v)[8]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[i]));     // fmaxf leaves NaN out
  return a;
}

__device__ __forceinline__ void store8(uint8_t* q, int n, bool vec, float r, const float (&v)[8]) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = kv_code2<kKvE4M3>(__fmul_rn(v[2 * i], r), __fmul_rn(v[2 * i + 1], r));
  if (vec && n >= 8) {
    *reinterpret_cast<uint2*>(q) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = (uint8_t)(c[i / 2] >> (8 * (i & 1)));
  }
}

// 1 x 128: a warp 8 blocks of a row, sixteen lanes a block, every load in flight before
// the first maximum.  With `place`, row r is written `copies` times, to rows place[r *
// copies + j] of the codes and scales (each slot of a token's, in the order of experts).
template <typename T, bool PLACED>
__global__ void __launch_bounds__(THREADS) quantise_rows_kernel(const __grid_constant__ QuantiseArgs a, int groups) {
  constexpr int U = 4;
  griddep_wait();
  const int lane = threadIdx.x % 32;
  const long long unit = (long long)blockIdx.x * (THREADS / 32) + threadIdx.x / 32;
  const long long row = unit / groups;
  if (row >= a.rows) return;
  const int col0 = (int)(unit - row * groups) * (2 * U * QB) + lane * 8;       // lanes 16 .. 31 the next block
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  float v[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int col = col0 + u * 2 * QB;
    load8(x + col, min(max(a.cols - col, 0), 8), a.vec_x, v[u]);
  }
  float s[U], r[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float big = big8(v[u]);
#pragma unroll
    for (int d = HALF / 2; d; d >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
    s[u] = kv_scale_for<kKvE4M3>(big);
    r[u] = kv_recip(s[u]);
  }
  const int copies = PLACED ? a.copies : 1;
  for (int j = 0; j < copies; ++j) {
    long long to = row;
    if (PLACED) {
      to = a.place[row * copies + j];
      // a slot that `order` does not have was given no row: what is there is by chance
      if (to < 0 || to >= (long long)a.rows * copies || a.order[to] != (int)(row * copies + j)) continue;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int col = col0 + u * 2 * QB, n = min(max(a.cols - col, 0), 8);
      store8(a.codes + to * a.ldq + col, n, a.vec_q, r[u], v[u]);
      if (lane % HALF == 0 && n > 0) a.scales[to * a.lds + col / QB] = s[u];
    }
  }
}

// place[order[p]] = p, for the numbers that fit
__global__ void __launch_bounds__(THREADS) invert_kernel(const int* order, int n, int* place, int* status) {
  griddep_wait();
  const int p = (int)(blockIdx.x * (long long)THREADS + threadIdx.x);
  if (p >= n) return;
  const int slot = order[p];
  if (slot >= 0 && slot < n) place[slot] = p;
  else report_status(status, 1, kSiteExperts);
}

// 128 x 128: a thread block a block of values, 8 rows a half warp, all in registers.
template <typename T>
__global__ void __launch_bounds__(THREADS) quantise_tiles_kernel(const QuantiseArgs a) {
  __shared__ float part[THREADS / 32];
  griddep_wait();
  const int lane = threadIdx.x % HALF, half = threadIdx.x / HALF;
  const T* X = static_cast<const T*>(a.x);
  const int col = (int)blockIdx.x * QB + lane * 8;
  for (long long tile = blockIdx.y; tile * QB < a.rows; tile += gridDim.y) {
    float v[QB / HALVES][8];
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < QB / HALVES; ++i) {
      const long long row = tile * QB + i * HALVES + half;
      const int n = row < a.rows ? min(max(a.cols - col, 0), 8) : 0;
      load8(X + row * a.ldx + col, n, a.vec_x, v[i]);
      big = fmaxf(big, big8(v[i]));
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = big;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) big = fmaxf(big, part[w]);
    const float s = kv_scale_for<kKvE4M3>(big), r = kv_recip(s);
#pragma unroll
    for (int i = 0; i < QB / HALVES; ++i) {
      const long long row = tile * QB + i * HALVES + half;
      const int n = row < a.rows ? min(max(a.cols - col, 0), 8) : 0;
      store8(a.codes + row * a.ldq + col, n, a.vec_q, r, v[i]);
    }
    if (threadIdx.x == 0) a.scales[tile * a.lds + blockIdx.x] = s;
    __syncthreads();                      // part[] is read by all before the next tile's
  }
}

template <typename T>
int launch_type(const QuantiseArgs& a, cudaStream_t s) {
  const int per_row = (a.cols + QB - 1) / QB;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.block_rows == 1) {
    const int groups = (per_row + 7) / 8;
    const long long blocks = ((long long)a.rows * groups + THREADS / 32 - 1) / (THREADS / 32);
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3((unsigned)blocks, 1, 1);
    return a.place != nullptr ? cudaLaunchKernelEx(&cfg, quantise_rows_kernel<T, true>, a, groups)
                              : cudaLaunchKernelEx(&cfg, quantise_rows_kernel<T, false>, a, groups);
  }
  const int tiles = (a.rows + QB - 1) / QB;
  cfg.gridDim = dim3((unsigned)per_row, (unsigned)(tiles < 65535 ? tiles : 65535), 1);
  return cudaLaunchKernelEx(&cfg, quantise_tiles_kernel<T>, a);
}

}  // namespace

int launch_fp8_quantise(const QuantiseArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_type<__nv_bfloat16>(a, s) : launch_type<float>(a, s);
}

int launch_invert(const int* order, int n, int* place, int* status, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)n + THREADS - 1) / THREADS), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, invert_kernel, order, n, place, status);
}

}  // namespace g3

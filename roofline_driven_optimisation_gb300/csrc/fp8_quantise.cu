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
// n / 128 rounded up, for n up to 2^31 - 1
__host__ __device__ constexpr int count_blocks(int n) { return n / QB + (n % QB != 0); }

// 8 values from x[0..7], of which `n` exist (0 in the place of the others), as they came:
// bf16 values take half the registers that way.  (Plain loads here and below: the compiler
// may move read-only ones before griddep_wait.)
template <typename T>
struct Eight {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* x, int n, bool vec) {
    if (vec && n >= 8) {
#pragma unroll
      for (int q = 0; q < (int)sizeof(T) / 2; ++q) w[q] = reinterpret_cast<const uint4*>(x)[q];
    } else {
      alignas(16) T part[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) part[i] = i < n ? x[i] : T(0.f);
#pragma unroll
      for (int q = 0; q < (int)sizeof(T) / 2; ++q) w[q] = *reinterpret_cast<const uint4*>(part + q * 16 / sizeof(T));
    }
  }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t u[4] = {w[i * sizeof(T) / 16].x, w[i * sizeof(T) / 16].y, w[i * sizeof(T) / 16].z, w[i * sizeof(T) / 16].w};
    if constexpr (sizeof(T) == 4) return __uint_as_float(u[i % 4]);
    else return __uint_as_float(i % 2 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
  }
  __device__ __forceinline__ float big() const {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(at(i)));     // fmaxf leaves NaN out
    return a;
  }
  __device__ __forceinline__ void store(uint8_t* q, int n, bool vec, float r) const {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = kv_code2<kKvE4M3>(__fmul_rn(at(2 * i), r), __fmul_rn(at(2 * i + 1), r));
    if (vec && n >= 8) {
      *reinterpret_cast<uint2*>(q) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) q[i] = (uint8_t)(c[i / 2] >> (8 * (i & 1)));
    }
  }
};

// 1 x 128: a warp 2 U blocks of a row, sixteen lanes a block, every load in flight before
// the first maximum, and as many warps as an SM takes (16384 x 4096 bf16: 83 us with four
// blocks a half warp of 1024 threads an SM in turn, 61 one unit a warp, 37 with bf16 values
// kept as they came and a row's scales stored side by side: 0.82 of the copy rate, issue 72
// %).  With `place`, row
// r is written `copies` times, to rows place[r * copies + j] of the codes and scales (each
// slot of a token's, in the order of experts).
template <typename T>
constexpr int units_u() { return sizeof(T) == 2 ? 4 : 2; }

template <typename T, bool PLACED>
__global__ void __launch_bounds__(THREADS, 5) quantise_rows_kernel(const __grid_constant__ QuantiseArgs a, int groups) {
  constexpr int U = units_u<T>();
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32;
  const long long unit = (long long)blockIdx.x * (THREADS / 32) + threadIdx.x / 32;
  const long long row = a.units32 ? (unsigned)unit / (unsigned)groups : unit / groups;
  if (row >= a.rows) return;
  const int first = (int)(unit - row * groups) * 2 * U;             // its first block
  const int col0 = first * QB + lane * 8;                           // lanes 16 .. 31 the next block
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  Eight<T> v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int col = col0 + u * 2 * QB;
    v[u].load(x + col, min(max(a.cols - col, 0), 8), a.vec_x);
  }
  float s[U], mine = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float big = v[u].big();
#pragma unroll
    for (int d = HALF / 2; d; d >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
    s[u] = kv_scale_for<kKvE4M3>(big);
    // lane i < 2 U: the i-th block's scale, so that the row's are stored side by side
    const float other = __shfl_sync(0xffffffffu, s[u], (lane & 1) * HALF);
    if (lane / 2 == u) mine = other;
  }
  const int blocks = count_blocks(a.cols);
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
      const int col = col0 + u * 2 * QB;
      v[u].store(a.codes + to * a.ldq + col, min(max(a.cols - col, 0), 8), a.vec_q, kv_recip(s[u]));
    }
    if (lane < 2 * U && first + lane < blocks) a.scales[to * a.lds + first + lane] = mine;
  }
}

// place[order[p]] = p, for the numbers that fit
__global__ void __launch_bounds__(THREADS) invert_kernel(const int* order, int n, int* place, int* status) {
  griddep_wait();
  griddep_launch_dependents();
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
    Eight<T> v[QB / HALVES];
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < QB / HALVES; ++i) {
      const long long row = tile * QB + i * HALVES + half;
      v[i].load(X + row * a.ldx + col, row < a.rows ? min(max(a.cols - col, 0), 8) : 0, a.vec_x);
    }
#pragma unroll
    for (int i = 0; i < QB / HALVES; ++i) big = fmaxf(big, v[i].big());
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
      v[i].store(a.codes + row * a.ldq + col, row < a.rows ? min(max(a.cols - col, 0), 8) : 0, a.vec_q, r);
    }
    if (threadIdx.x == 0) a.scales[tile * a.lds + blockIdx.x] = s;
    __syncthreads();                      // part[] is read by all before the next tile's
  }
}

template <typename T>
int launch_type(const QuantiseArgs& a, cudaStream_t s) {
  const int per_row = count_blocks(a.cols);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.block_rows == 1) {
    constexpr int each = 2 * units_u<T>();
    const int groups = (per_row + each - 1) / each;
    const long long blocks = ((long long)a.rows * groups + THREADS / 32 - 1) / (THREADS / 32);
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3((unsigned)blocks, 1, 1);
    QuantiseArgs q = a;
    q.units32 = blocks * (THREADS / 32) < 0x7fffffffll;
    return a.place != nullptr ? cudaLaunchKernelEx(&cfg, quantise_rows_kernel<T, true>, q, groups)
                              : cudaLaunchKernelEx(&cfg, quantise_rows_kernel<T, false>, q, groups);
  }
  const int tiles = count_blocks(a.rows);
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

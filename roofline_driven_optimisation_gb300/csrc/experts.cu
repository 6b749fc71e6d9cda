// What the experts' products need beside the tensor-core kernel: the generic product of
// block-scaled E4M3 matrices (any size and alignment) and the weighted sum of each
// token's experts.
//
// Product, for the rows of one matrix or of each expert:
//
//     C[m][n] = alpha * sum over blocks b of sa[m][b] * sb[b][n/128] * S_b + beta * C[m][n]
//     S_b = sum over the 128 k of block b of A[m][k] * B[k][n]
//
// with A's and B's codes as they are in S_b, and every sum in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "epilogue.cuh"
#include "experts.cuh"
#include "internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace g3 {
namespace {

// ---------------------------------------------------------------- generic product
// A block of 256 threads computes 16 rows x 128 columns: thread t column t % 128 of 8
// rows.  A's slice goes through shared memory, B's codes come straight from memory (a
// warp reads 32 neighbours).  Right for every call; the fast kernel takes the rest.
constexpr int GM = 16, GN = 128, GK = 16;

__device__ __forceinline__ float code_f32(uint8_t c) { return kv_value2<kKvE4M3>(c).x; }

template <bool SW>
__global__ void __launch_bounds__(256) blocks_generic_kernel(const BlocksArgs a) {
  __shared__ float As[GK][GM];
  __shared__ int Rows[GM], Outs[GM];
  __shared__ float Part[SW ? GM : 1][4];
  const int tx = threadIdx.x % GN, ty = threadIdx.x / GN;
  const int n = (int)blockIdx.x * GN + tx;
  const int kblocks = (a.K + kBlocksK - 1) / kBlocksK;
  // row tiles of all experts in a line; this block takes every gridDim.y-th
  long long tile = blockIdx.y, first = 0;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && uncovered_rows(a)) report_status(a.status, 1, kSiteExperts);
  for (int e = 0; e < a.experts; ++e) {
    int begin, count;
    expert_rows(a, e, begin, count);
    const long long tiles = ((long long)count + GM - 1) / GM;
    for (; tile < first + tiles; tile += gridDim.y) {
      const int p0 = begin + (int)(tile - first) * GM;
      const int rows = min(GM, begin + count - p0);
      __syncthreads();                      // the tile before has read Rows and Outs
      if (threadIdx.x < GM) {
        int r = -1, o = -1;
        if ((int)threadIdx.x < rows) expert_row(a, p0 + threadIdx.x, r, o);
        Rows[threadIdx.x] = r;
        Outs[threadIdx.x] = o;
      }
      float acc[GM / 2], acc2[SW ? GM / 2 : 1];
#pragma unroll
      for (int i = 0; i < GM / 2; ++i) {
        acc[i] = 0.f;
        if (SW) acc2[SW ? i : 0] = 0.f;
      }
      const uint8_t* B = a.B + e * a.b_stride;
      const uint8_t* B2 = SW ? a.B2 + e * a.b_stride : nullptr;
      for (int kb = 0; kb < kblocks; ++kb) {
        float part[GM / 2], part2[SW ? GM / 2 : 1];
#pragma unroll
        for (int i = 0; i < GM / 2; ++i) {
          part[i] = 0.f;
          if (SW) part2[SW ? i : 0] = 0.f;
        }
        const int k1 = min(a.K, (kb + 1) * kBlocksK);
        for (int k0 = kb * kBlocksK; k0 < k1; k0 += GK) {
          __syncthreads();
          {
            const int kk = threadIdx.x % GK, m = threadIdx.x / GK;
            const int r = Rows[m];
            As[kk][m] = r >= 0 && k0 + kk < k1 ? code_f32(a.A[r * a.lda + k0 + kk]) : 0.f;
          }
          __syncthreads();
#pragma unroll
          for (int kk = 0; kk < GK; ++kk) {
            const bool in = n < a.N && k0 + kk < k1;
            const float b = in ? code_f32(B[(long long)(k0 + kk) * a.ldb + n]) : 0.f;
#pragma unroll
            for (int i = 0; i < GM / 2; ++i) part[i] = fmaf(As[kk][2 * i + ty], b, part[i]);
            if (SW) {
              const float b2 = in ? code_f32(B2[(long long)(k0 + kk) * a.ldb + n]) : 0.f;
#pragma unroll
              for (int i = 0; i < GM / 2; ++i) part2[SW ? i : 0] = fmaf(As[kk][2 * i + ty], b2, part2[SW ? i : 0]);
            }
          }
        }
        const long long at = e * a.sb_stride + kb * a.ldsb + blockIdx.x;
        const float sb = a.sb[at], sb2 = SW ? a.sb2[at] : 0.f;
#pragma unroll
        for (int i = 0; i < GM / 2; ++i) {
          const int r = Rows[2 * i + ty];
          const float sa = r >= 0 ? a.sa[r * a.ldsa + kb] : 0.f;
          acc[i] = fmaf(part[i], sa * sb, acc[i]);
          if (SW) acc2[SW ? i : 0] = fmaf(part2[SW ? i : 0], sa * sb2, acc2[SW ? i : 0]);
        }
      }
      __syncthreads();
      if constexpr (SW) {
        float h[GM / 2];
#pragma unroll
        for (int i = 0; i < GM / 2; ++i) {
          h[i] = n < a.N ? swiglu_combine(acc[i], acc2[i]) : 0.f;
          float big = fmaxf(fabsf(h[i]), 0.f);          // NaN is left out
#pragma unroll
          for (int d = 16; d; d >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
          if (threadIdx.x % 32 == 0) Part[2 * i + ty][tx / 32] = big;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < GM / 2; ++i) {
          const int m = 2 * i + ty;
          if (m >= rows) continue;
          const float s = kv_scale_for<kKvE4M3>(fmaxf(fmaxf(Part[m][0], Part[m][1]), fmaxf(Part[m][2], Part[m][3])));
          const long long p = p0 + m;
          if (n < a.N) a.hq[p * a.ldh + n] = (uint8_t)kv_code2<kKvE4M3>(__fmul_rn(h[i], kv_recip(s)), 0.f);
          if (tx == 0) a.hs[p * a.ldhs + blockIdx.x] = s;
        }
      } else {
#pragma unroll
        for (int i = 0; i < GM / 2; ++i) {
          const long long o = Outs[2 * i + ty];
          if (o >= 0 && n < a.N) blocks_store(a, o, n, acc[i]);
        }
      }
    }
    first += tiles;
  }
}

// ---------------------------------------------------------------- weighted sums
// A block 1024 columns of a token, a thread 8 of them: its top_k rows' parts, 128 bytes in
// flight, added in order.  y in fp32, or in fp16 times a scale for each 128 columns.  Reads top_k *
// cols values of y a token once: HBM (or L2) bounds it (16384 tokens of 8 slots of 4096 in 16
// bits: 189 us for 1.2 GB, the copy rate's 183).
constexpr int COMBINE_THREADS = 128;
template <bool SCALED>
__global__ void __launch_bounds__(COMBINE_THREADS, 6) combine_kernel(const __grid_constant__ CombineArgs a) {
  constexpr int WORDS = SCALED ? 1 : 2, FLIGHT = 8 / WORDS;      // 16-byte vectors of 8 values; rows in flight
  using T = std::conditional_t<SCALED, __half, float>;
  griddep_wait();
  const long long t = blockIdx.x;
  const int c = (int)(blockIdx.y * COMBINE_THREADS + threadIdx.x) * 8;
  if (c >= a.cols) return;
  const float* w = a.weights + t * a.top_k;
  const T* y = static_cast<const T*>(a.y) + t * a.top_k * a.ldy + c;
  const float* ys = SCALED ? a.ys + t * a.top_k * a.ldys + c / 128 : nullptr;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + t * a.ldo + c;
  float sum[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) sum[q] = 0.f;
  for (int j0 = 0; j0 < a.top_k; j0 += FLIGHT) {                 // rows of y are whole vectors
    uint4 v[FLIGHT][WORDS];
    float f[FLIGHT], s[FLIGHT];
#pragma unroll
    for (int j = 0; j < FLIGHT; ++j) {
      const bool in = j0 + j < a.top_k;
#pragma unroll
      for (int q = 0; q < WORDS; ++q)
        v[j][q] = in ? reinterpret_cast<const uint4*>(y + (j0 + j) * a.ldy)[q] : make_uint4(0u, 0u, 0u, 0u);
      f[j] = in ? w[j0 + j] : 0.f;
      s[j] = SCALED && in ? ys[(j0 + j) * a.ldys] : 1.f;
    }
#pragma unroll
    for (int j = 0; j < FLIGHT; ++j) {
      if (j0 + j >= a.top_k) break;
#pragma unroll
      for (int q = 0; q < WORDS; ++q) {
        const uint32_t u[4] = {v[j][q].x, v[j][q].y, v[j][q].z, v[j][q].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (SCALED) {                                // the product with a power of two is exact
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            sum[2 * i] = fmaf(f[j], x.x * s[j], sum[2 * i]);
            sum[2 * i + 1] = fmaf(f[j], x.y * s[j], sum[2 * i + 1]);
          } else {
            sum[4 * q + i] = fmaf(f[j], __uint_as_float(u[i]), sum[4 * q + i]);
          }
        }
      }
    }
  }
  if (a.vec && c + 8 <= a.cols) {
    uint32_t r[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(sum[2 * q], sum[2 * q + 1]);
      r[q] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(o) = make_uint4(r[0], r[1], r[2], r[3]);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (c + q < a.cols) o[q] = __float2bfloat16_rn(sum[q]);
  }
}

}  // namespace

int launch_blocks_generic(const BlocksArgs& a, cudaStream_t s) {
  const long long tiles = ((long long)a.rows + GM - 1) / GM + (a.offsets != nullptr ? a.experts : 0);
  const dim3 grid((unsigned)((a.N + GN - 1) / GN), (unsigned)(tiles < 65535 ? tiles : 65535), 1);
  if (a.B2 != nullptr)
    blocks_generic_kernel<true><<<grid, 256, 0, s>>>(a);
  else
    blocks_generic_kernel<false><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

int launch_experts_combine(const CombineArgs& a, cudaStream_t s) {
  const int across = (a.cols + 8 * COMBINE_THREADS - 1) / (8 * COMBINE_THREADS);
  if (across > 65535) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.tokens, (unsigned)across, 1);
  cfg.blockDim = dim3(COMBINE_THREADS, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.ys != nullptr ? cudaLaunchKernelEx(&cfg, combine_kernel<true>, a) : cudaLaunchKernelEx(&cfg, combine_kernel<false>, a);
}

}  // namespace g3

// Attention of a sequence's newest tokens over its paged 8-bit cache
// (gemm_kv_attention; the header states the mathematics).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace g3 {
namespace {

// The sequence that row `row` belongs to, and its place among the sequence's n
// new rows; false if no sequence holds it.
__device__ __forceinline__ bool find_row(const KvAttnArgs& a, int row, int& b, int& i, int& n) {
  int first;
  if (a.start == nullptr) {
    b = row;
    i = 0;
    n = 1;
    return row < a.c.seqs;
  }
  int lo = 0, hi = a.c.seqs;   // the last b with start[b] <= row
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.start[mid] <= row) lo = mid;
    else hi = mid;
  }
  b = lo;
  kv_rows(a.start, b, a.tokens, a.max_new, a.status, kSiteKvAttn, first, n);
  i = row - first;
  return i >= 0 && i < n;
}

// Tokens of sequence b in the cache, held to what its table row can address.
__device__ __forceinline__ int kv_length(const KvAttnArgs& a, int b) {
  const int len = a.lengths[b];
  const long long most = (long long)a.c.cols * a.c.P;
  if (len < 0 || len > most) {
    report_status(a.status, 1, kSiteKvAttn);
    return len < 0 ? 0 : (int)most;
  }
  return len;
}

// ------------------------------------------------------------------ generic
// Any head width (to 512), page size and stride: one block for each query row
// and head, keys in chunks of one a thread, the softmax online in fp32.
constexpr int GT = 128;   // threads, and keys in a chunk
constexpr int GD = 512;   // widest head

template <int FMT>
__global__ void __launch_bounds__(GT) kv_attention_generic_kernel(const KvAttnArgs a) {
  __shared__ float q[GD], p[GT], red[GT / 32];
  __shared__ long long at[GT];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int D = a.c.D, row = blockIdx.x, hq = blockIdx.y, h = hq / (a.Hq / a.c.H);
  int b, i, n;
  if (!find_row(a, row, b, i, n)) return;
  const int keys = kv_length(a, b) - n + i + 1;   // keys this row sees
  const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.Q) + (long long)row * a.ldq + (long long)hq * D;
  for (int d = threadIdx.x; d < D; d += GT) q[d] = __bfloat162float(qr[d]);
  float acc[GD / GT] = {};
  float m = -INFINITY, l = 0.f;
  for (int j0 = 0; j0 < keys; j0 += GT) {
    const int j = j0 + threadIdx.x;
    float s = -INFINITY, vs = 0.f;
    long long off = -1;
    __syncthreads();   // q is written; the previous chunk's readers are done
    if (j < keys) {
      const int g = kv_page(a.c, b, j / a.c.P, a.status, kSiteKvAttn);
      if (g >= 0) {
        off = (long long)g * a.c.ps + (long long)h * a.c.hs + (long long)(j % a.c.P) * a.c.ts;
        const uint8_t* kc = a.c.k + off;
        float dot = 0.f;
        for (int d = 0; d < D; ++d) dot = fmaf(q[d], kv_value2<FMT>(kc[d]).x, dot);
        s = dot * a.c.ks[(long long)g * a.c.H + h] * a.scale;
        vs = a.c.vs[(long long)g * a.c.H + h];
      }
    }
    at[threadIdx.x] = off;
    float mx = s;
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = mx;
    __syncthreads();
    mx = m;
    for (int w = 0; w < GT / 32; ++w) mx = fmaxf(mx, red[w]);
    const float mu = mx == -INFINITY ? 0.f : mx;
    const float e = off >= 0 ? expf(s - mu) : 0.f, alpha = expf(m - mu);
    m = mx;
    p[threadIdx.x] = e * vs;
    float sum = e;
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();   // red has been read
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = sum;
    __syncthreads();
    l *= alpha;
    for (int w = 0; w < GT / 32; ++w) l += red[w];
#pragma unroll
    for (int c = 0; c < GD / GT; ++c) {
      const int d = c * GT + threadIdx.x;
      if (d >= D) break;
      float x = acc[c] * alpha;
      for (int t = 0; t < min(GT, keys - j0); ++t)
        if (at[t] >= 0) x = fmaf(p[t], kv_value2<FMT>(a.c.v[at[t] + d]).x, x);
      acc[c] = x;
    }
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.O) + (long long)row * a.ldo + (long long)hq * D;
#pragma unroll
  for (int c = 0; c < GD / GT; ++c) {
    const int d = c * GT + threadIdx.x;
    // l == 0: no key was seen; a NaN sum must come out as NaN
    if (d < D) out[d] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[c] / l);
  }
}

template <class Kernel>
int launch(Kernel kernel, dim3 grid, dim3 block, const KvAttnArgs& a, cudaStream_t s) {
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

int launch_kv_attention_generic(const KvAttnArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.tokens, (unsigned)a.Hq);
  if (a.c.fmt == kKvE4M3) return launch(kv_attention_generic_kernel<kKvE4M3>, grid, dim3(GT), a, s);
  return launch(kv_attention_generic_kernel<kKvInt8>, grid, dim3(GT), a, s);
}

}  // namespace g3

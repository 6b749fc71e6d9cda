// Runs swiglu_near2 of csrc/experts.cuh, and swiglu_combine of csrc/epilogue.cuh, on gates
// from `first` on, count of them by their bits, against 64 bits: the largest relative errors
// in half steps of fp32 (2^-24) from -87.3 on, and the largest magnitude below.
#include <cuda_runtime.h>

#include <cstdint>

#include "epilogue.cuh"
#include "experts.cuh"

namespace {

// out: [0] the largest error, [1] the largest magnitude below -87.3, [2], [3] the same of the
// generic form; as bits of positive floats.  wrong: gates whose NaN or infinity is not what it
// should be.
__global__ void check(uint32_t first, uint64_t count, float u, unsigned* out, unsigned* wrong) {
  for (uint64_t i = blockIdx.x * (uint64_t)blockDim.x + threadIdx.x; i < count; i += (uint64_t)gridDim.x * blockDim.x) {
    const float g = __uint_as_float(first + (uint32_t)i);
    const uint64_t two = g3::swiglu_near2(g3::both(g), g3::both(u));
    const float got[2] = {g3::part2(two, (int)(i & 1)), g3::swiglu_combine(g, u)};
    for (int k = 0; k < 2; ++k) {
      if (!isfinite(g)) {
        if (g == INFINITY ? got[k] != u * INFINITY : !isnan(got[k])) atomicAdd(wrong, 1u);
        continue;
      }
      const double want = (double)g / (1.0 + exp(-(double)g)) * (double)u;
      if (g < -87.3f) {
        atomicMax(out + 2 * k + 1, __float_as_uint(fabsf(got[k])));
      } else if (!isfinite(got[k])) {
        if (fabs(want) <= 3.4e38) atomicAdd(wrong, 1u);
      } else {
        // of denormal numbers half a step is 2^-150, of silu before the product with u as well
        const double of = fmax(fabs(want), 0x1p-126 * fmax(1.0, fabs((double)u)));
        atomicMax(out + 2 * k, __float_as_uint((float)(fabs((double)got[k] - want) / of * 0x1p24)));
      }
    }
  }
}

}  // namespace

extern "C" int silu_check(uint32_t first, uint64_t count, float u, float* errors, unsigned* wrong) {
  unsigned* d = nullptr;
  cudaError_t e = cudaMalloc(&d, 5 * sizeof(unsigned));
  if (e == cudaSuccess) e = cudaMemset(d, 0, 5 * sizeof(unsigned));
  if (e == cudaSuccess) {
    check<<<152 * 8, 256>>>(first, count, u, d, d + 4);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = cudaMemcpy(errors, d, 4 * sizeof(unsigned), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemcpy(wrong, d + 4, sizeof(unsigned), cudaMemcpyDeviceToHost);
  cudaFree(d);
  return (int)e;
}

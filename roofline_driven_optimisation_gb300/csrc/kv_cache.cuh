// The paged 8-bit key/value cache as the kernels see it: where a token's codes
// are, what a code stands for, and which rows of a call belong to which
// sequence.  Everything a kernel reads from the caller's tables is checked here
// before it becomes an address.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace g3 {

constexpr int kKvE4M3 = 0, kKvInt8 = 1;

template <int FMT>
__host__ __device__ constexpr float kv_qmax() {
  return FMT == kKvE4M3 ? 448.f : 127.f;
}

// ---------------------------------------------------------------- codes
// x (already times 1/scale) on the format's grid, nearest even, saturating at
// qmax.  NaN: E4M3's NaN, INT8's 0.
template <int FMT>
__device__ __forceinline__ uint32_t kv_code2(float lo, float hi) {   // two codes, lo in bits 0-7
  if constexpr (FMT == kKvE4M3) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  } else {
    // rounded first, then held to 127: the conversion takes NaN to 0 and saturates
    const int a = min(max(__float2int_rn(lo), -127), 127);
    const int b = min(max(__float2int_rn(hi), -127), 127);
    return (uint32_t)(a & 0xff) | ((uint32_t)(b & 0xff) << 8);
  }
}

// two codes (bits 0-15) as fp16, exact: E4M3 and the whole numbers to 127 fit
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)c));
  return r;
}

template <int FMT>
__device__ __forceinline__ float2 kv_value2(uint32_t c) {
  if constexpr (FMT == kKvE4M3) {
    const uint32_t h = e4m3x2_to_f16x2(c);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
  } else {
    return make_float2((float)(int8_t)(c & 0xff), (float)(int8_t)((c >> 8) & 0xff));
  }
}

// ---------------------------------------------------------------- scales
// The scale that a largest magnitude asks for: a / qmax, 0 below the smallest
// normal number (whose reciprocal could overflow).  `a` ignores NaN (fmaxf) and
// is FLT_MAX at most, so the scale is always finite.
template <int FMT>
__device__ __forceinline__ float kv_scale_for(float a) {
  const float s = __fdiv_rn(fminf(a, FLT_MAX), kv_qmax<FMT>());
  return s >= FLT_MIN ? s : 0.f;
}
__device__ __forceinline__ float kv_recip(float s) { return s >= FLT_MIN ? __frcp_rn(s) : 0.f; }

// ---------------------------------------------------------------- rows of a sequence
// Rows first .. first+n-1 of the call's `tokens` rows; a range that does not fit
// is reported and taken as empty.
__device__ __forceinline__ void kv_rows(const int* start, int b, int tokens, int max_new, int* status, int site,
                                        int& first, int& n) {
  if (start == nullptr) {
    first = b;
    n = 1;
    return;
  }
  first = start[b];
  const int end = start[b + 1];
  n = end - first;
  if (first < 0 || end < first || end > tokens || n > max_new) {
    report_status(status, 1, site);
    first = n = 0;
  }
}

// Page number of column `col` of sequence b's table row, or -1 (reported) if
// the column or the number is outside the cache.
__device__ __forceinline__ int kv_page(const KvCache& c, int b, int col, int* status, int site) {
  int g = -1;
  if (col >= 0 && col < c.cols) g = c.table[(long long)b * c.tstride + col];
  if (g < 0 || g >= c.pages) {
    report_status(status, 1, site);
    return -1;
  }
  return g;
}

}  // namespace g3

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

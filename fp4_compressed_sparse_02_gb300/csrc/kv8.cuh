// What the kernels of the paged 8-bit cache share: a step's rows, sequences and pages.
#pragma once

#include "common.cuh"

namespace csa2 {

// The sequence of row t: s with start[s] <= t < start[s+1], or -1 for a row of padding.  Whatever
// start holds, a result >= 0 is below S and satisfies both inequalities.
__device__ __forceinline__ int find_seq(const int* __restrict__ start, int S, int t) {
  if (t < start[0] || t >= start[S]) return -1;
  int lo = 0, hi = S;                    // start[lo] <= t < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Position of row t of sequence s, or -1 (with an error bit) outside its row of the page table.
__device__ __forceinline__ int row_pos(const csa2_kv8_cache& c, const int* start, const int* length, int s, int t,
                                       unsigned int* err) {
  const long long p = (long long)length[s] - ((long long)start[s + 1] - t);
  if (p < 0 || p >= (long long)c.max_pages * kPage) {
    raise_error(err, CSA2_DEVERR_PAGE_SLOT);
    return -1;
  }
  return (int)p;
}

// Page id of page j (< max_pages) of sequence s, or -1 (with an error bit).
__device__ __forceinline__ int page_id(const csa2_kv8_cache& c, int s, int j, unsigned int* err) {
  const int page = __ldg(c.page_table + (long long)s * c.max_pages + j);
  if (page < 0 || page >= c.num_pages) {
    raise_error(err, CSA2_DEVERR_PAGE_ID);
    return -1;
  }
  return page;
}

// Four E4M3 bytes as float32.  Exact; NaN stays NaN.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float* f) {
  const uint32_t lo = e4m3x2_lo_f16x2(w), hi = e4m3x2_hi_f16x2(w);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
}

// Two float32 -> two E4M3 bytes (a in the low one), round to nearest even, saturating.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

}  // namespace csa2

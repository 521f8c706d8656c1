// What the kernels of the paged 8-bit cache share: a step's rows, sequences and pages.
#pragma once

#include "common.cuh"

namespace csa2 {

// Every load of tables, rows, scales and bytes is an ordinary one behind pdl_wait(): the kernel before on the stream may be the
// one that writes them, and it still runs when this one's CTAs start.  (Page ids by ld_s32: where the compiler may move
// them, the tiles' conversion of the values comes out slower, 342 us against 274 for 32 x 6 tokens.)

// The sequence of row t: s with start[s] <= t < start[s+1], or -1 for a row of padding.  Whatever
// start holds, a result >= 0 is below S and satisfies both inequalities.  By a whole warp, for one t: 32 starts at a
// time, so that up to 32 sequences take one round of loads and 1024 two.
__device__ __forceinline__ int find_seq(const int* start, int S, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = S;                    // start[lo] <= t < start[hi], once both have been looked at
  const int last = start[S];
  while (true) {
    const int step = (hi - lo + 31) >> 5, i = lo + step * lane;
    const uint32_t in = __ballot_sync(0xffffffffu, i < hi && start[i] <= t);
    if (lo == 0 && hi == S && ((in & 1) == 0 || t >= last)) return -1;
    const int at = 31 - __clz(in);
    lo += step * at;
    hi = min(hi, lo + step);
    if (hi - lo <= 1) return lo;
  }
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
  const int page = ld_s32(c.page_table + (long long)s * c.max_pages + j);
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

// Two float32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 w, x, y;\n"
      " mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 w, x, y;\n"
      " mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// The NaNs among four E4M3 bytes: 1 in the byte of each.
__device__ __forceinline__ uint32_t e4m3x4_nans(uint32_t w) {
  return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
}

}  // namespace csa2

// What the two attention kernels of the paged 8-bit cache share: rows and what they see, spans of the work and the
// parts that they leave.
#pragma once

#include <limits.h>
#include <math.h>

#include "internal.h"
#include "kv8.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace csa2 {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr uint32_t kWaitPolls = 1u << 22;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const void* map, int x, int y, int z, uint64_t* mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      :: "r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(map), "r"((uint32_t)__cvta_generic_to_shared(mbar)),
         "r"(x), "r"(y), "r"(z)
      : "memory");
}

// The power of two that brings a row whose largest magnitude is `top` into [2^14, 2^15), and the one that undoes it;
// 1 for a row of zeros or with an infinity or NaN.
__device__ __forceinline__ void row_factor(float top, float& f, float& undo) {
  const int e = (int)(__float_as_uint(top) >> 23);         // biased exponent; 0: zero or below 2^-126
  f = undo = 1.f;
  if (top == 0.f || e >= 255) return;
  const int k = 14 - (e - 127);                            // -113 .. 141
  const int k1 = k > 127 ? 127 : k;
  f = __uint_as_float((uint32_t)(k1 + 127) << 23);
  undo = k1 == 127 ? 5.877471754111438e-39f : __uint_as_float((uint32_t)(127 - k1) << 23);   // 2^-127 is subnormal
}

// ---- rows of a sequence ----------------------------------------------------------------------

struct Rows {
  int t0, n;                             // first row of the step, rows x group
  int end, length;                       // start[s+1], length[s]
};

__device__ __forceinline__ Rows rows_of(const csa2_kv8_attn_args& a, int s, int G) {
  Rows r;
  r.t0 = a.start[s];
  r.end = a.start[s + 1];
  r.length = a.length[s];
  const int e = min(r.end, a.T);
  r.n = r.t0 >= 0 && e > r.t0 ? (e - r.t0) * G : 0;
  return r;
}

// What row t sees: positions [lo, hi).
__device__ __forceinline__ void seen_by(const csa2_kv8_attn_args& a, const Rows& r, int t, int& lo, int& hi,
                                        unsigned int* err) {
  const long long p = (long long)r.length - ((long long)r.end - t);
  if (p < 0 || p >= (long long)a.cache.max_pages * kPage) {
    raise_error(err, CSA2_DEVERR_PAGE_SLOT);
    lo = hi = 0;
    return;
  }
  hi = (int)p + 1;
  lo = a.window > 0 && hi > a.window ? hi - a.window : 0;
}

// ---- spans and parts -------------------------------------------------------------------------

struct Part {                            // a stream that begins in a span and does not end there
  int rows, t0, r0, h;                   // rows = 0: none
  int last;                              // the span in which it ends
};

struct Kv8Params {
  csa2_kv8_attn_args a;
  int G, aligned;                        // aligned: bit 0 q's rows, bit 1 out's rows on 16 bytes, bit 2 on 32
  int spans, most;                       // most: rows of a part's place
  Part* part;                            // [spans]
  float2* ml;                            // [spans][2][most] maximum, sum; [1]: of the stream that goes on from here
  float* o;                              // [spans][2][most][D] sums of weighted values
  float2* second_ml;                     // tiles of up to 128 rows: [spans][most] maximum, sum, and
  float* second;                         // [spans][most][D] sums of weighted values, of the second group's earlier runs
};

// One plane as [num_pages * Hkv][64][D] bytes, boxes of `tokens` tokens, swizzled over the rows' width.
inline bool plane_map(CUtensorMap* map, const void* base, const csa2_kv8_cache& c, int tokens) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dim[3] = {(cuuint64_t)c.D, kPage, (cuuint64_t)c.num_pages * c.Hkv};
  const cuuint64_t stride[2] = {(cuuint64_t)c.D, (cuuint64_t)c.D * kPage};
  const cuuint32_t box[3] = {(cuuint32_t)c.D, (cuuint32_t)tokens, 1}, one[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dim, stride, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, c.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// kv8_tile.cu
constexpr int kTileSpans = 152;
// Rows of its tiles: a sequence's rows of a key head, if they fit.
inline int tile_rows(const csa2_kv8_attn_args& a) {
  const long long rows = (long long)a.max_new * (a.Hq / a.cache.Hkv);
  return rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
}
cudaError_t launch_kv8_tile(const Kv8Params& p, cudaStream_t st);
uint32_t read_clear_error_kv8_tile();

}  // namespace csa2

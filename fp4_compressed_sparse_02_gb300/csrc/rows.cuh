// Device helpers of the row operators (norm.cu, fp4.cu): 16 consecutive channels at a time,
// and the FP4 / E4M3 quantisers of such a group.
#pragma once

#include "common.cuh"

namespace csa2 {

// 16 channels of a row as float32; vec: the address is 16-byte aligned and all 16 exist.
// Channels from n on are 0.
__device__ __forceinline__ void load16(float* v, const void* base, long long off, bool f32, bool vec, int n) {
  if (f32) {
    const float* p = static_cast<const float*>(base) + off;
    if (vec) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(p + 4 * i);
        v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = i < n ? p[i] : 0.f;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + off;
    if (vec) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 q = *reinterpret_cast<const uint4*>(p + 8 * i);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
          v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = i < n ? bf16_bits_to_f32(p[i]) : 0.f;
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ void store16(const float* v, void* base, long long off, bool f32, bool vec, int n) {
  if (f32) {
    float* p = static_cast<float*>(base) + off;
    if (vec) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(p + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) p[i] = v[i];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(base) + off;
    if (vec) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<uint4*>(p + 8 * i) =
            make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                       pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) p[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
    }
  }
}

// Bits of max |v|: magnitudes order like their bit patterns, and a NaN is above all of them.
__device__ __forceinline__ uint32_t amax_bits16(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// FP4 codes and scale of 16 channels u (csa2_fp4_quant): w0 the first eight codes, w1 the
// others.  The code is E2M1 of the correctly rounded quotient u / s.  Only the side of the seven
// borders m s (m = 1/4, 3/4, 5/4, 7/4, 5/2, 7/2, 5) matters, and m s is exact: a u off a border
// is off by 2^-24 of it or more.  One Newton step (Markstein 1990: q = u y with y = RN(1/s),
// q - (s q - u) y with both steps fused) leaves 2^-47, so it decides as the division does, and
// u = m s gives m itself, whose tie the conversion resolves.  Written with s q - u, a zero keeps
// its sign.  Magnitudes that could overflow take the division.
__device__ __forceinline__ void fp4_encode16(const float* u, uint32_t& w0, uint32_t& w1, uint32_t& sbyte) {
  const float a = __uint_as_float(amax_bits16(u));
  sbyte = cvt_e4m3(__fdiv_rn(a, 6.0f));
  const float s = e4m3_to_f32(sbyte);
  w0 = w1 = 0;
  if (!(s > 0.f)) return;
  float q[16];
  if (a < 1e30f) {
    const float y = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float q0 = __fmul_rn(u[i], y);
      q[i] = __fmaf_rn(-__fmaf_rn(s, q0, -u[i]), y, q0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = __fdiv_rn(u[i], s);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w0 |= cvt_e2m1x2(q[2 * i], q[2 * i + 1]) << (8 * i);
    w1 |= cvt_e2m1x2(q[8 + 2 * i], q[9 + 2 * i]) << (8 * i);
  }
}

// Byte offset of scale c (16 columns each) of row r in the scale tiles of FP4 rows with nkt
// column tiles; c % 4 == 0 addresses the four bytes of one row and tile.
__device__ __forceinline__ long long fp4_scale_offset(int r, int c, int nkt) {
  return ((long long)(r >> 7) * nkt + (c >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (c & 3);
}

}  // namespace csa2

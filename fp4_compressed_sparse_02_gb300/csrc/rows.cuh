// Device helpers of the row operators (norm.cu, fp4.cu): 16 consecutive channels at a time as
// eight float32 pairs, whose adds, products and fused products take one instruction a pair, and
// the FP4 / E4M3 quantisers of such a group.
#pragma once

#include "common.cuh"

namespace csa2 {

// Two float32 in one register pair; every operation rounds each half to nearest.
using f32x2 = uint64_t;
__device__ __forceinline__ f32x2 pk(float a, float b) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 unpk(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 sub2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// Two bf16 in a word as a float32 pair, and back (rounded to nearest).
__device__ __forceinline__ f32x2 bf16_pair(uint32_t w) {
  return pk(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint32_t pack_bf16(f32x2 v) {
  const float2 f = unpk(v);
  return pack_bf16(f.x, f.y);
}

// Loads that stay behind pdl_wait() and in order with this thread's own stores (an output may be
// the input itself), which ld.global.nc and __ldg do not promise: what the previous kernel on the
// stream wrote is read after it.
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {   // 16 bytes that nobody reads again
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
__device__ __forceinline__ uint4 ld_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
__device__ __forceinline__ float ld_f32(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ int ld_s32(const int* p) {
  int v;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 16 channels of a row as they lie in memory: 8 words of bf16 pairs or 16 of float32.  wide: the
// address is 32-byte aligned, not only 16; one access then takes the sectors that two half-sector
// accesses each would touch.
template <bool F32>
struct Raw16 {
  uint4 q[F32 ? 4 : 2];
  __device__ __forceinline__ void load(const void* base, long long off, bool wide) {   // read once
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + off * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); i += 2) {
      if (wide) {
        asm volatile("ld.global.L1::no_allocate.L2::256B.v8.u32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(q[i].x), "=r"(q[i].y), "=r"(q[i].z), "=r"(q[i].w), "=r"(q[i + 1].x), "=r"(q[i + 1].y),
                       "=r"(q[i + 1].z), "=r"(q[i + 1].w) : "l"(p + i));
      } else {
        q[i] = ld_once_v4(p + i);
        q[i + 1] = ld_once_v4(p + i + 1);
      }
    }
  }
  __device__ __forceinline__ void load_again(const void* base, long long off) {        // what others read too
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + off * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); ++i) q[i] = ld_v4(p + i);
  }
  __device__ __forceinline__ void negate() {
    const uint32_t m = F32 ? 0x80000000u : 0x80008000u;
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); ++i) q[i].x ^= m, q[i].y ^= m, q[i].z ^= m, q[i].w ^= m;
  }
  __device__ __forceinline__ f32x2 pair(int i) const {    // channels 2 i, 2 i + 1
    if (F32) {
      const uint4& v = q[i / 2];
      return i % 2 ? pk(__uint_as_float(v.z), __uint_as_float(v.w)) : pk(__uint_as_float(v.x), __uint_as_float(v.y));
    }
    const uint4& v = q[i / 4];
    return bf16_pair(i % 4 == 0 ? v.x : i % 4 == 1 ? v.y : i % 4 == 2 ? v.z : v.w);
  }
  __device__ __forceinline__ void store(void* base, long long off, bool wide) const {
    uint4* p = reinterpret_cast<uint4*>(static_cast<char*>(base) + off * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); i += 2) {
      if (wide) {
        asm volatile("st.global.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};"
                     :: "r"(q[i].x), "r"(q[i].y), "r"(q[i].z), "r"(q[i].w), "r"(q[i + 1].x), "r"(q[i + 1].y),
                        "r"(q[i + 1].z), "r"(q[i + 1].w), "l"(p + i) : "memory");
      } else {
        p[i] = q[i];
        p[i + 1] = q[i + 1];
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); ++i) q[i] = make_uint4(0, 0, 0, 0);
  }
};

// 16 channels one at a time, for rows that are not aligned.
__device__ __forceinline__ void load16_any(f32x2* v, const void* base, long long off, bool f32) {
  float e[16];
#pragma unroll
  for (int i = 0; i < 16; ++i)
    e[i] = f32 ? static_cast<const float*>(base)[off + i] : bf16_bits_to_f32(static_cast<const uint16_t*>(base)[off + i]);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = pk(e[2 * i], e[2 * i + 1]);
}

template <bool F32>
__device__ __forceinline__ void store16(const f32x2* v, void* base, long long off, bool wide) {
  Raw16<F32> r;
#pragma unroll
  for (int i = 0; i < (F32 ? 4 : 2); ++i) {
    if (F32) {
      const float2 a = unpk(v[2 * i]), b = unpk(v[2 * i + 1]);
      r.q[i] = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
    } else {
      r.q[i] = make_uint4(pack_bf16(v[4 * i]), pack_bf16(v[4 * i + 1]), pack_bf16(v[4 * i + 2]), pack_bf16(v[4 * i + 3]));
    }
  }
  r.store(base, off, wide);
}

// max(|a|, |b|, |c|), NaN if one is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <int NP>
__device__ __forceinline__ float amax_pairs(const f32x2* v) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const float2 f = unpk(v[i]);
    m = max3_abs(f.x, f.y, m);
  }
  return m;
}
__device__ __forceinline__ float amax16(const f32x2* v) { return amax_pairs<8>(v); }

// The same over a warp's lanes.
__device__ __forceinline__ float warp_max_abs(float v) {
  float d;
  asm volatile("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
  return d;
}

// Quotients by an invariant divisor (Markstein, "Computation of elementary functions on the IBM
// RISC System/6000", 1990): with y = RN(1 / s), q = RN(u y) is within two steps of u / s, the
// remainder u - s q is exact in a fused product, and adding remainder * y leaves an error of 2^-47
// before the rounding; a second such step gives the correctly rounded quotient.  The
// arguments are negated, n = -u and ny = -y, so that a remainder of +0 keeps the sign of a zero.
__device__ __forceinline__ f32x2 quotient_step(f32x2 q, f32x2 n, f32x2 s, f32x2 ny) { return fma2(fma2(s, q, n), ny, q); }

// v = RN(-v / s), both steps.  s in [2^-60, 2^60] (quotient_ok), and no quotient near the ends of float32's
// range: one that overflows becomes an infinity or a NaN.  Values so small that a remainder
// underflows give zero codes either way.
__device__ __forceinline__ bool quotient_ok(float s) { return s >= 0x1p-60f && s <= 0x1p60f; }
__device__ __forceinline__ void quotients16(f32x2* v, float s) {
  const float y = -__frcp_rn(s);
  const f32x2 ny = pk(y, y), ss = pk(s, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = quotient_step(quotient_step(mul2(v[i], ny), v[i], ss, ny), v[i], ss, ny);
}

// Eight float32 -> eight E2M1 codes in a word, the first in the low nibble.
__device__ __forceinline__ uint32_t e2m1x8(const f32x2* q) {
  const float2 a = unpk(q[0]), b = unpk(q[1]), c = unpk(q[2]), d = unpk(q[3]);
  uint32_t r;
  asm("{\n .reg .b8 t0, t1, t2, t3;\n cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 t1, %4, %3;\n cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 t3, %8, %7;\n mov.b32 %0, {t0, t1, t2, t3};\n}"
      : "=r"(r) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return r;
}

// FP4 codes and scale of the 16 channels u = -n (csa2_fp4_quant) with a = max |u| <= 2^60: w[0] the first
// eight codes, w[1] the others, w[2] the scale byte.  The code is E2M1 of the correctly rounded
// quotient u / s.  Only the side of the seven borders m s (m = 1/4, 3/4, 5/4, 7/4, 5/2, 7/2, 5)
// matters, and m s is exact: a u off a border is off by 2^-24 of it or more, so one quotient step,
// with a reciprocal good to a step, decides as the division does, and u = m s gives m itself, whose
// tie the conversion resolves.  The same holds for the scale: the borders between E4M3 values,
// times 6, are exact.
__device__ __forceinline__ void fp4_encode16(const f32x2* n, float a, uint32_t* w) {
  const float a0 = __fmul_rn(a, 1.0f / 6.0f);
  w[2] = cvt_e4m3(__fmaf_rn(__fmaf_rn(-6.0f, a0, a), 1.0f / 6.0f, a0));
  const float s = e4m3_to_f32(w[2]);
  w[0] = w[1] = 0;
  if (!(s > 0.f)) return;
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(-s));
  const f32x2 ny = pk(y, y), ss = pk(s, s);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    f32x2 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = quotient_step(mul2(n[4 * h + i], ny), n[4 * h + i], ss, ny);
    w[h] = e2m1x8(q);
  }
}

// The same by the definition, for any x and g: u = x / g.
static __device__ __noinline__ void fp4_encode16_any(const f32x2* x, float g, uint32_t* w) {
  f32x2 u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = unpk(x[i]);
    u[i] = pk(__fdiv_rn(f.x, g), __fdiv_rn(f.y, g));
  }
  w[2] = cvt_e4m3(__fdiv_rn(amax16(u), 6.0f));
  const float s = e4m3_to_f32(w[2]);
  w[0] = w[1] = 0;
  if (!(s > 0.f)) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = unpk(u[i]);
    u[i] = pk(__fdiv_rn(f.x, s), __fdiv_rn(f.y, s));
  }
  w[0] = e2m1x8(u);
  w[1] = e2m1x8(u + 4);
}

__device__ __forceinline__ void e4m3x16(const f32x2* q, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpk(q[2 * i]), b = unpk(q[2 * i + 1]);
    asm("{\n .reg .b16 t0, t1;\n cvt.rn.satfinite.e4m3x2.f32 t0, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 t1, %4, %3;\n"
        " mov.b32 %0, {t0, t1};\n}" : "=r"(w[i]) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  }
}
static __device__ __noinline__ void fp8_encode16_any(const f32x2* n, float s, uint32_t* w) {
  f32x2 q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = unpk(n[i]);
    q[i] = pk(__fdiv_rn(-f.x, s), __fdiv_rn(-f.y, s));
  }
  e4m3x16(q, w);
}

// E4M3 bytes of RN(-n / s) with s = RN(max |n| / 448), four words; zero where s is not positive.  n is used up.
__device__ __forceinline__ void fp8_encode16(f32x2* n, float s, uint32_t* w) {
  if (quotient_ok(s)) {
    quotients16(n, s);
    e4m3x16(n, w);
  } else if (s > 0.f) {
    f32x2 t[8];
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = n[i];
    fp8_encode16_any(t, s, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = b[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = 0;
  }
}

// Byte offset of scale c (16 columns each) of row r in the scale tiles of FP4 rows with nkt
// column tiles; c % 4 == 0 addresses the four bytes of one row and tile.
__device__ __forceinline__ long long fp4_scale_offset(int r, int c, int nkt) {
  return ((long long)(r >> 7) * nkt + (c >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (c & 3);
}

}  // namespace csa2

// Residual addition and root-mean-square norm (csa2_rms_norm), with the output in bf16,
// float32, E4M3 with scales, or FP4 rows.
#include "internal.h"
#include "rows.cuh"

namespace csa2 {

namespace {

constexpr int kMaxThreads = 1024;

struct NormParams {
  const void* x;
  const void* res;
  void* res_out;
  const void* w;
  void* out;
  float* out_scale;
  uint8_t* tiles;
  const float* gscale;
  long long sx, sr, so_res, so;
  int T, D, nkt;
  float eps;
  int group;
  bool x32, r32, w32, vx, vr, vro, vw, vo;   // element types; 16-byte accesses allowed
};

// (hi, lo) += (b, blo): the rounding error of the float32 sum goes into lo (Knuth's TwoSum).
__device__ __forceinline__ void add2(float& hi, float& lo, float b, float blo) {
  const float s = __fadd_rn(hi, b);
  const float t = __fsub_rn(s, hi);
  lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(b, t)) + blo;
  hi = s;
}

__device__ __forceinline__ void warp_add2(float& hi, float& lo) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float b = __shfl_xor_sync(0xffffffffu, hi, o), bl = __shfl_xor_sync(0xffffffffu, lo, o);
    add2(hi, lo, b, bl);
  }
}

}  // namespace

// One CTA per row; thread t holds the 16-channel chunks t, t + blockDim, ... (NCH of them) from
// the addition to the last store, so the row is read once and written once.
//
// The sum of squares is kept in two float32 words: a square of a float32 is h^2 = p + fma(h, h,
// -p) exactly, and every addition passes its rounding error on.  The mean then differs from the
// exact one by 2^-46, and the float32 it rounds to, and with it every 4- or 8-bit code, does not
// depend on the split of the row over threads.
template <int OUT, int NCH>
__global__ void __launch_bounds__(kMaxThreads) k_rms_norm(NormParams p) {
  pdl_wait();
  pdl_trigger();
  __shared__ float2 part[32];
  __shared__ uint32_t apart[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarp = blockDim.x >> 5;
  const int nchunk = (p.D + 15) / 16;
  if (OUT == CSA2_FP4E2M1X2 && blockIdx.x >= p.T) {       // scales of the rows past the last
    const int r0 = p.T, r1 = (p.T + 127) & ~127;
    for (int i = tid; i < (r1 - r0) * p.nkt; i += blockDim.x)
      *reinterpret_cast<uint32_t*>(p.tiles + fp4_scale_offset(r0 + i / p.nkt, 4 * (i % p.nkt), p.nkt)) = 0;
    return;
  }
  const long long row = blockIdx.x;
  float h[NCH][16];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int ch = tid + c * blockDim.x, n = min(16, p.D - 16 * ch);
    if (ch >= nchunk) {
#pragma unroll
      for (int i = 0; i < 16; ++i) h[c][i] = 0.f;
      continue;
    }
    load16(h[c], p.x, row * p.sx + 16 * ch, p.x32, p.vx && n == 16, n);
    if (p.res) {
      float r[16];
      load16(r, p.res, row * p.sr + 16 * ch, p.r32, p.vr && n == 16, n);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        h[c][i] += r[i];
        if (!p.r32) h[c][i] = __bfloat162float(__float2bfloat16_rn(h[c][i]));
      }
      store16(h[c], p.res_out, row * p.so_res + 16 * ch, p.r32, p.vro && n == 16, n);
    }
  }
  // the second pass, of a row whose squares leave float32's range, scales by 2^-64
  float ms = 0.f;
#pragma unroll 1
  for (float sc = 1.f;; sc = 0x1p-64f) {
    float hi = 0.f, lo = 0.f;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float v = h[c][i] * sc;
        const float q = __fmul_rn(v, v);
        add2(hi, lo, q, __fmaf_rn(v, v, -q));
      }
    warp_add2(hi, lo);
    if (sc != 1.f) __syncthreads();                       // every warp has read the first partials
    if (lane == 0) part[warp] = make_float2(hi, lo);
    __syncthreads();
    const float2 z = lane < nwarp ? part[lane] : make_float2(0.f, 0.f);
    hi = z.x, lo = z.y;
    warp_add2(hi, lo);
    // (hi + lo) / D rounded once: the remainder of the rounded quotient is exact
    const float fd = (float)p.D;
    const float q = __fdiv_rn(hi, fd);
    ms = q + __fdiv_rn(__fmaf_rn(-q, fd, hi) + lo, fd);
    if (isfinite(hi)) {
      if (sc != 1.f) ms = ms * 0x1p64f * 0x1p64f;
      break;
    }
    ms = hi;
    if (sc != 1.f) break;
  }
  const float r = __fdiv_rn(1.0f, __fsqrt_rn(ms + p.eps));
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int ch = tid + c * blockDim.x, n = min(16, p.D - 16 * ch);
    float w[16];
    if (p.w && ch < nchunk) {
      load16(w, p.w, 16 * ch, p.w32, p.vw && n == 16, n);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = 1.f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) h[c][i] = __fmul_rn(__fmul_rn(h[c][i], r), w[i]);
    if (OUT == CSA2_BF16 || OUT == CSA2_F32) {
      if (ch < nchunk) store16(h[c], p.out, row * p.so + 16 * ch, OUT == CSA2_F32, p.vo && n == 16, n);
    } else if (OUT == CSA2_FP4E2M1X2) {
      if (p.gscale) {
        const float g = __ldg(p.gscale);
#pragma unroll
        for (int i = 0; i < 16; ++i) h[c][i] = __fdiv_rn(h[c][i], g);
      }
      uint32_t w0, w1, sb = 0;
      if (ch < nchunk) {
        fp4_encode16(h[c], w0, w1, sb);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + row * (p.D / 2) + 8 * ch) = make_uint2(w0, w1);
      }
      // the four scale bytes of a row and column tile, from four neighbouring lanes
      sb |= __shfl_down_sync(0xffffffffu, sb, 1) << 8;
      sb |= __shfl_down_sync(0xffffffffu, sb, 2) << 16;
      if ((ch & 3) == 0 && ch < nchunk)
        *reinterpret_cast<uint32_t*>(p.tiles + fp4_scale_offset((int)row, ch, p.nkt)) = sb;
    }
  }
  if (OUT == CSA2_FP8E4M3) {
    float rs = 0.f;
    if (p.group == 0) {                                   // one scale for the row
      uint32_t m = 0;
#pragma unroll
      for (int c = 0; c < NCH; ++c) m = max(m, amax_bits16(h[c]));
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0) apart[warp] = m;
      __syncthreads();
      m = __reduce_max_sync(0xffffffffu, lane < nwarp ? apart[lane] : 0u);
      rs = __fdiv_rn(__uint_as_float(m), 448.0f);
      if (tid == 0) p.out_scale[row] = rs;
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int ch = tid + c * blockDim.x, n = min(16, p.D - 16 * ch);
      float s = rs;
      if (p.group) {                                      // 128 channels: eight lanes
        uint32_t m = amax_bits16(h[c]);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 4));
        s = __fdiv_rn(__uint_as_float(m), 448.0f);
        if ((ch & 7) == 0 && ch < nchunk) p.out_scale[row * ((p.D + 127) / 128) + ch / 8] = s;
      }
      if (ch >= nchunk) continue;
      uint32_t b[4] = {0, 0, 0, 0};
      if (s > 0.f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) b[i / 4] |= cvt_e4m3(__fdiv_rn(h[c][i], s)) << (8 * (i % 4));
      }
      uint8_t* o = static_cast<uint8_t*>(p.out) + row * p.so + 16 * ch;
      if (p.vo && n == 16) {
        *reinterpret_cast<uint4*>(o) = make_uint4(b[0], b[1], b[2], b[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < n) o[i] = (uint8_t)(b[i / 4] >> (8 * (i % 4)));
      }
    }
  }
}

static bool vec_ok(const void* p, long long stride, int esize) {
  return ((uintptr_t)p & 15) == 0 && (stride * esize) % 16 == 0;
}

cudaError_t launch_rms_norm(const csa2_rms_norm_args& a, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const bool fp4 = a.out_form == CSA2_FP4E2M1X2;
  NormParams p{};
  p.x = a.x, p.sx = a.x_stride, p.x32 = a.x_dtype == CSA2_F32;
  p.res = a.residual, p.sr = a.residual_stride, p.r32 = a.res_dtype == CSA2_F32;
  p.res_out = a.residual_out, p.so_res = a.residual_out_stride;
  p.w = a.weight, p.w32 = a.weight_dtype == CSA2_F32;
  p.out = fp4 ? a.out4.codes : a.out;
  p.so = a.out_stride;
  p.out_scale = a.out_scale;
  p.tiles = a.out4.scales, p.gscale = fp4 ? a.out4.gscale : nullptr;
  p.T = a.T, p.D = a.D, p.nkt = (a.D + 63) / 64;
  p.eps = a.eps, p.group = a.scale_group;
  p.vx = vec_ok(a.x, a.T > 1 ? a.x_stride : 0, p.x32 ? 4 : 2);
  p.vr = vec_ok(a.residual, a.T > 1 ? a.residual_stride : 0, p.r32 ? 4 : 2);
  p.vro = vec_ok(a.residual_out, a.T > 1 ? a.residual_out_stride : 0, p.r32 ? 4 : 2);
  p.vw = vec_ok(a.weight, 0, 1);
  p.vo = vec_ok(a.out, a.T > 1 ? a.out_stride : 0, a.out_form == CSA2_F32 ? 4 : a.out_form == CSA2_BF16 ? 2 : 1);
  const int nchunk = (a.D + 15) / 16;
  const int nch = nchunk > kMaxThreads ? 2 : 1;
  const int threads = ((nchunk + nch - 1) / nch + 31) & ~31;
  const unsigned grid = (unsigned)a.T + (fp4 && a.T % 128 ? 1u : 0u);
#define CSA2_NORM(O) \
  return nch == 1 ? launch_k(k_rms_norm<O, 1>, grid, threads, 0, st, p) : launch_k(k_rms_norm<O, 2>, grid, threads, 0, st, p)
  switch (a.out_form) {
    case CSA2_BF16: CSA2_NORM(CSA2_BF16);
    case CSA2_F32: CSA2_NORM(CSA2_F32);
    case CSA2_FP8E4M3: CSA2_NORM(CSA2_FP8E4M3);
    default: CSA2_NORM(CSA2_FP4E2M1X2);
  }
#undef CSA2_NORM
}

}  // namespace csa2

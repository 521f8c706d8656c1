// Residual addition and root-mean-square norm (csa2_rms_norm), with the output in bf16,
// float32, E4M3 with scales, or FP4 rows.
#include "internal.h"
#include "rows.cuh"

namespace csa2 {

namespace {

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
  int T, D, nkt, lanes;
  float eps;
  int group;
  bool x32, r32, w32;
};

// (hi, lo) += (b, blo) in two float32 words: the rounding error of the sum goes into lo (Knuth's
// TwoSum), once for a pair of sums.
__device__ __forceinline__ void sum_pair(f32x2& hi, f32x2& lo, f32x2 b) {
  const f32x2 s = add2(hi, b), t = sub2(s, hi);
  lo = add2(lo, add2(sub2(hi, sub2(s, t)), sub2(b, t)));
  hi = s;
}
__device__ __forceinline__ void sum2(float& hi, float& lo, float b, float blo) {
  const float s = __fadd_rn(hi, b), t = __fsub_rn(s, hi);
  lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(b, t)) + blo;
  hi = s;
}
__device__ __forceinline__ void lanes_sum2(float& hi, float& lo, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) {
    const float b = __shfl_xor_sync(0xffffffffu, hi, o), bl = __shfl_xor_sync(0xffffffffu, lo, o);
    sum2(hi, lo, b, bl);
  }
}

// The sum of squares of 16 channels (times sc^2) in two words.  A square is h^2 = p + fma(h, h, -p)
// exactly; that of a bf16 value has no second word.
template <bool EXACT>
__device__ __forceinline__ void squares16(const f32x2* h, float sc, float& hi, float& lo) {
  f32x2 a = 0, b = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const f32x2 v = sc == 1.f ? h[i] : mul2(h[i], pk(sc, sc));
    const f32x2 q = mul2(v, v);
    sum_pair(a, b, q);
    if (!EXACT) b = add2(b, fma2(v, v, mul2(q, pk(-1.f, -1.f))));
  }
  const float2 ah = unpk(a), bl = unpk(b);
  hi = ah.x, lo = bl.x;
  sum2(hi, lo, ah.y, bl.y);
}

// RN((hi + lo) / D): the remainder of the rounded quotient is exact.
__device__ __forceinline__ float mean2(float hi, float lo, int D) {
  const float d = (float)D, q = __fdiv_rn(hi, d);
  return q + __fdiv_rn(__fmaf_rn(-q, d, hi) + lo, d);
}

// The scale byte of a chunk and those of the next three of its row, which neighbouring lanes hold.
__device__ __forceinline__ uint32_t merge_scales(uint32_t sb, int ch, int nchunk) {
  const uint32_t b = __shfl_down_sync(0xffffffffu, sb, 1);
  if (ch + 1 < nchunk) sb |= b << 8;
  const uint32_t c = __shfl_down_sync(0xffffffffu, sb, 2);
  if (ch + 2 < nchunk) sb |= c << 16;
  return sb;
}

// Zero scales for the rows past the last, up to a whole tile of 128.
__device__ __forceinline__ void zero_tail(const NormParams& p) {
  const int n = ((p.T + 127) & ~127) - p.T;
  for (int i = threadIdx.x; i < n * p.nkt; i += blockDim.x)
    *reinterpret_cast<uint32_t*>(p.tiles + fp4_scale_offset(p.T + i / p.nkt, 4 * (i % p.nkt), p.nkt)) = 0;
}

}  // namespace

// Aligned rows of D = 16 c channels, D <= 8192.  A thread holds one 16-channel chunk of a row from the
// addition to the last store, so the row is read once and written once, and its weights for
// every row it works on.  SMALL (D <= 512): p.lanes lanes of a warp share a row; otherwise a CTA
// does, with one barrier for the sum (and one for a row's E4M3 scale).  The next row's loads are
// issued before this row's arithmetic.
//
// The sum of squares is kept in two float32 words.  The mean then differs from the exact one by
// 2^-46, and the float32 it rounds to, and with it every 4- or 8-bit code, does not depend on the
// split of the row over threads.
template <int OUT, bool X32, int RES, bool SMALL>
__global__ void __launch_bounds__(SMALL ? 256 : 512) k_rms_norm(NormParams p) {
  pdl_wait();
  pdl_trigger();
  __shared__ float2 part[2][16];
  __shared__ float apart[2][16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarp = blockDim.x >> 5;
  const int nchunk = p.D / 16;
  int grid = gridDim.x;
  if (OUT == CSA2_FP4E2M1X2 && (p.T & 127)) {
    if (blockIdx.x == --grid) return zero_tail(p);
  }
  const int rpb = SMALL ? (int)blockDim.x / p.lanes : 1;  // rows of a CTA at a time
  const int ch = SMALL ? lane & (p.lanes - 1) : tid;
  const bool has = ch < nchunk;
  f32x2 w[8];
  if (p.w && has) {
    if (p.w32) {
      Raw16<true> r;
      r.load(p.w, 16 * ch, true);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = r.pair(i);
    } else {
      Raw16<false> r;
      r.load(p.w, 16 * ch, true);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = r.pair(i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pk(1.f, 1.f);
  }
  const float g = OUT == CSA2_FP4E2M1X2 && p.gscale ? ld_f32(p.gscale) : 1.f;
  Raw16<X32> xr;
  Raw16<RES == 2> rr;
  const long long step = (long long)grid * rpb;
  long long row = (long long)blockIdx.x * rpb + (SMALL ? tid / p.lanes : 0);
  const auto fetch = [&](long long r) {
    if (has && r < p.T) {
      xr.load(p.x, r * p.sx + 16 * ch);
      if (RES) rr.load(p.res, r * p.sr + 16 * ch);
    } else {
      xr.zero();
      if (RES) rr.zero();
    }
  };
  fetch(row);
  // a warp's rows are neighbours: it runs while its first exists (a CTA's row is the same in all)
  for (int par = 0; row - (SMALL ? lane / p.lanes : 0) < p.T; row += step, par ^= 1) {
    const bool mine = has && row < p.T;
    f32x2 h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = RES ? add2(xr.pair(i), rr.pair(i)) : xr.pair(i);
    if (RES == 1) {
      uint32_t b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        b[i] = pack_bf16(h[i]);
        h[i] = bf16_pair(b[i]);
      }
      if (mine) {
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.res_out) + row * p.so_res + 16 * ch);
        o[0] = make_uint4(b[0], b[1], b[2], b[3]);
        o[1] = make_uint4(b[4], b[5], b[6], b[7]);
      }
    } else if (RES == 2) {
      if (mine) store16<true>(h, p.res_out, row * p.so_res + 16 * ch);
    }
    fetch(row + step);
    float ms;
    {
      constexpr bool EXACT = RES == 1 || (RES == 0 && !X32);
      float hi, lo;
      squares16<EXACT>(h, 1.f, hi, lo);
      lanes_sum2(hi, lo, SMALL ? p.lanes : 32);
      if (!SMALL) {
        if (lane == 0) part[par][warp] = make_float2(hi, lo);
        __syncthreads();
        const float2 z = (lane & 15) < nwarp ? part[par][lane & 15] : make_float2(0.f, 0.f);
        hi = z.x, lo = z.y;
        lanes_sum2(hi, lo, 16);
      }
      ms = mean2(hi, lo, p.D);
      // squares beyond float32's range: once more, scaled by 2^-64
      const bool big = !isfinite(hi);
      if (SMALL ? __any_sync(0xffffffffu, big) : big) {
        float hi2, lo2;
        squares16<EXACT>(h, 0x1p-64f, hi2, lo2);
        lanes_sum2(hi2, lo2, SMALL ? p.lanes : 32);
        if (!SMALL) {
          __syncthreads();                                // every warp has read the first sums
          if (lane == 0) part[par][warp] = make_float2(hi2, lo2);
          __syncthreads();
          const float2 z = (lane & 15) < nwarp ? part[par][lane & 15] : make_float2(0.f, 0.f);
          hi2 = z.x, lo2 = z.y;
          lanes_sum2(hi2, lo2, 16);
        }
        if (big) ms = isfinite(hi2) ? mean2(hi2, lo2, p.D) * 0x1p64f * 0x1p64f : hi2;
      }
    }
    // quantised forms take the negated value (rows.cuh)
    constexpr bool NEG = OUT == CSA2_FP8E4M3 || OUT == CSA2_FP4E2M1X2;
    const float r0 = __fdiv_rn(1.0f, __fsqrt_rn(ms + p.eps)), r = NEG ? -r0 : r0;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = mul2(mul2(h[i], pk(r, r)), w[i]);
    if (OUT == CSA2_BF16 || OUT == CSA2_F32) {
      if (mine) store16<OUT == CSA2_F32>(h, p.out, row * p.so + 16 * ch);
    } else if (OUT == CSA2_FP4E2M1X2) {
      if (p.gscale) {                                     // u = RN(y / g), negated again
        f32x2 u[8];
        quotients16(u, h, g, amax16(h));
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = mul2(u[i], pk(-1.f, -1.f));
      }
      uint32_t w0 = 0, w1 = 0, sb = 0;
      if (mine) {
        fp4_encode16(h, w0, w1, sb);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + row * (p.D / 2) + 8 * ch) = make_uint2(w0, w1);
      }
      sb = merge_scales(sb, ch, nchunk);
      if (mine && (ch & 3) == 0) *reinterpret_cast<uint32_t*>(p.tiles + fp4_scale_offset((int)row, ch, p.nkt)) = sb;
    } else {
      float m = has ? amax16(h) : 0.f;
      if (p.group || SMALL) {                             // 128 channels are eight lanes, or a row's lanes
        const int over = p.group && (!SMALL || p.lanes > 8) ? 8 : p.lanes;
        for (int o = over >> 1; o > 0; o >>= 1) m = max3_abs(m, __shfl_xor_sync(0xffffffffu, m, o), 0.f);
      } else {
        for (int o = 16; o > 0; o >>= 1) m = max3_abs(m, __shfl_xor_sync(0xffffffffu, m, o), 0.f);
        if (lane == 0) apart[par][warp] = m;
        __syncthreads();
        m = (lane & 15) < nwarp ? apart[par][lane & 15] : 0.f;
        for (int o = 8; o > 0; o >>= 1) m = max3_abs(m, __shfl_xor_sync(0xffffffffu, m, o), 0.f);
      }
      const float s = __fdiv_rn(m, 448.0f);
      uint32_t b[4];
      if (mine) {
        fp8_encode16(h, s, m, b);
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + row * p.so + 16 * ch) = make_uint4(b[0], b[1], b[2], b[3]);
        if (p.group ? (ch & 7) == 0 : ch == 0)
          p.out_scale[p.group ? row * ((p.D + 127) / 128) + ch / 8 : row] = s;
      }
    }
  }
}

// Any row: odd widths, unaligned rows, D up to 32768.  A CTA a row; chunks are read and written
// channel by channel, two to a thread above 16384 channels.
template <int OUT, int NCH>
__global__ void __launch_bounds__(1024) k_rms_norm_any(NormParams p) {
  pdl_wait();
  pdl_trigger();
  __shared__ float2 part[32];
  __shared__ float apart[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarp = blockDim.x >> 5;
  const int nchunk = (p.D + 15) / 16;
  if (OUT == CSA2_FP4E2M1X2 && blockIdx.x >= p.T) return zero_tail(p);
  const long long row = blockIdx.x;
  f32x2 h[NCH][8];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int ch = tid + c * blockDim.x, n = min(16, p.D - 16 * ch);
    load16_any(h[c], p.x, row * p.sx + 16 * ch, p.x32, n);
    if (p.res && n > 0) {
      f32x2 r[8];
      load16_any(r, p.res, row * p.sr + 16 * ch, p.r32, n);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[c][i] = add2(h[c][i], r[i]);
        if (!p.r32) h[c][i] = bf16_pair(pack_bf16(h[c][i]));
      }
      store16_any(h[c], p.res_out, row * p.so_res + 16 * ch, p.r32, n);
    }
  }
  // the second pass, of a row whose squares leave float32's range, scales by 2^-64
  float ms = 0.f;
#pragma unroll 1
  for (float sc = 1.f;; sc = 0x1p-64f) {
    float hi = 0.f, lo = 0.f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      float a, b;
      squares16<false>(h[c], sc, a, b);
      sum2(hi, lo, a, b);
    }
    lanes_sum2(hi, lo, 32);
    if (sc != 1.f) __syncthreads();                       // every warp has read the first partials
    if (lane == 0) part[warp] = make_float2(hi, lo);
    __syncthreads();
    const float2 z = lane < nwarp ? part[lane] : make_float2(0.f, 0.f);
    hi = z.x, lo = z.y;
    lanes_sum2(hi, lo, 32);
    ms = mean2(hi, lo, p.D);
    if (isfinite(hi)) {
      if (sc != 1.f) ms = ms * 0x1p64f * 0x1p64f;
      break;
    }
    ms = hi;
    if (sc != 1.f) break;
  }
  constexpr bool NEG = OUT == CSA2_FP8E4M3 || OUT == CSA2_FP4E2M1X2;
  const float r0 = __fdiv_rn(1.0f, __fsqrt_rn(ms + p.eps)), r = NEG ? -r0 : r0;
  float rm = 0.f;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int ch = tid + c * blockDim.x, n = min(16, p.D - 16 * ch);
    f32x2 w[8];
    if (p.w && n > 0) {
      load16_any(w, p.w, 16 * ch, p.w32, n);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pk(1.f, 1.f);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) h[c][i] = mul2(mul2(h[c][i], pk(r, r)), w[i]);
    if (OUT == CSA2_BF16 || OUT == CSA2_F32) {
      if (n > 0) store16_any(h[c], p.out, row * p.so + 16 * ch, OUT == CSA2_F32, n);
    } else if (OUT == CSA2_FP4E2M1X2) {
      if (p.gscale) {
        f32x2 u[8];
        quotients16(u, h[c], ld_f32(p.gscale), amax16(h[c]));
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] = mul2(u[i], pk(-1.f, -1.f));
      }
      uint32_t w0 = 0, w1 = 0, sb = 0;
      if (ch < nchunk) {
        fp4_encode16(h[c], w0, w1, sb);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + row * (p.D / 2) + 8 * ch) = make_uint2(w0, w1);
      }
      sb = merge_scales(sb, ch, nchunk);
      if ((ch & 3) == 0 && ch < nchunk)
        *reinterpret_cast<uint32_t*>(p.tiles + fp4_scale_offset((int)row, ch, p.nkt)) = sb;
    } else if (ch < nchunk) {
      rm = max3_abs(rm, amax16(h[c]), 0.f);
    }
  }
  if (OUT == CSA2_FP8E4M3) {
    if (p.group == 0) {                                   // one scale for the row
      for (int o = 16; o > 0; o >>= 1) rm = max3_abs(rm, __shfl_xor_sync(0xffffffffu, rm, o), 0.f);
      if (lane == 0) apart[warp] = rm;
      __syncthreads();
      rm = lane < nwarp ? apart[lane] : 0.f;
      for (int o = 16; o > 0; o >>= 1) rm = max3_abs(rm, __shfl_xor_sync(0xffffffffu, rm, o), 0.f);
      if (tid == 0) p.out_scale[row] = __fdiv_rn(rm, 448.0f);
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int ch = tid + c * blockDim.x, n = min(16, p.D - 16 * ch);
      float m = rm;
      if (p.group) {                                      // 128 channels: eight lanes
        m = ch < nchunk ? amax16(h[c]) : 0.f;
        for (int o = 4; o > 0; o >>= 1) m = max3_abs(m, __shfl_xor_sync(0xffffffffu, m, o), 0.f);
        if ((ch & 7) == 0 && ch < nchunk) p.out_scale[row * ((p.D + 127) / 128) + ch / 8] = __fdiv_rn(m, 448.0f);
      }
      if (ch >= nchunk) continue;
      uint32_t b[4];
      fp8_encode16(h[c], __fdiv_rn(m, 448.0f), m, b);
      uint8_t* o = static_cast<uint8_t*>(p.out) + row * p.so + 16 * ch;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) o[i] = (uint8_t)(b[i / 4] >> (8 * (i % 4)));
    }
  }
}

namespace {

template <int OUT, bool X32, int RES, bool SMALL>
cudaError_t launch_aligned(const NormParams& p, int threads, cudaStream_t st) {
  static int resident[17] = {0};                          // CTAs the GPU holds, by warps of a CTA
  int& r = resident[threads / 32];
  if (!r) {
    int dev = 0, sms = 0, per = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, k_rms_norm<OUT, X32, RES, SMALL>, threads, 0);
    if (e != cudaSuccess) return e;
    r = sms * (per > 0 ? per : 1);
  }
  const int rpb = SMALL ? threads / p.lanes : 1;
  const int blocks = (p.T + rpb - 1) / rpb;
  const unsigned tail = OUT == CSA2_FP4E2M1X2 && p.T % 128 ? 1u : 0u;
  return launch_k(k_rms_norm<OUT, X32, RES, SMALL>, (unsigned)(blocks < r ? blocks : r) + tail, threads, 0, st, p);
}

template <int OUT>
cudaError_t launch_form(const NormParams& p, bool aligned, cudaStream_t st) {
  if (aligned && p.D <= 8192) {
    const int res = !p.res ? 0 : p.r32 ? 2 : 1;
    const bool small = p.D <= 512;
    const int threads = small ? 256 : (p.D / 16 + 31) & ~31;
#define CSA2_NORM(X, R) \
  if (p.x32 == X && res == R) \
    return small ? launch_aligned<OUT, X, R, true>(p, threads, st) : launch_aligned<OUT, X, R, false>(p, threads, st)
    CSA2_NORM(false, 0);
    CSA2_NORM(false, 1);
    CSA2_NORM(false, 2);
    CSA2_NORM(true, 0);
    CSA2_NORM(true, 1);
    CSA2_NORM(true, 2);
#undef CSA2_NORM
  }
  const int nchunk = (p.D + 15) / 16, nch = nchunk > 1024 ? 2 : 1;
  const int threads = ((nchunk + nch - 1) / nch + 31) & ~31;
  const unsigned grid = (unsigned)p.T + (OUT == CSA2_FP4E2M1X2 && p.T % 128 ? 1u : 0u);
  return nch == 1 ? launch_k(k_rms_norm_any<OUT, 1>, grid, threads, 0, st, p)
                  : launch_k(k_rms_norm_any<OUT, 2>, grid, threads, 0, st, p);
}

bool rows_aligned(const void* p, long long stride, int esize) {
  return ((uintptr_t)p & 15) == 0 && (stride * esize) % 16 == 0;
}

}  // namespace

cudaError_t launch_rms_norm(const csa2_rms_norm_args& a, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const bool fp4 = a.out_form == CSA2_FP4E2M1X2, many = a.T > 1;
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
  p.lanes = 1;
  while (p.lanes < 32 && p.lanes * 16 < a.D) p.lanes *= 2;
  const int rb = p.r32 ? 4 : 2;
  const bool aligned =
      a.D % 16 == 0 && rows_aligned(a.x, many ? a.x_stride : 0, p.x32 ? 4 : 2) &&
      rows_aligned(a.residual, many ? a.residual_stride : 0, rb) &&
      rows_aligned(a.residual_out, many ? a.residual_out_stride : 0, rb) && rows_aligned(a.weight, 0, 1) &&
      (fp4 || rows_aligned(a.out, many ? a.out_stride : 0, a.out_form == CSA2_F32 ? 4 : a.out_form == CSA2_BF16 ? 2 : 1));
  switch (a.out_form) {
    case CSA2_BF16: return launch_form<CSA2_BF16>(p, aligned, st);
    case CSA2_F32: return launch_form<CSA2_F32>(p, aligned, st);
    case CSA2_FP8E4M3: return launch_form<CSA2_FP8E4M3>(p, aligned, st);
    default: return launch_form<CSA2_FP4E2M1X2>(p, aligned, st);
  }
}

}  // namespace csa2

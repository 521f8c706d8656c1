// Residual addition and root-mean-square norm (csa2_rms_norm), with the output in bf16,
// float32, E4M3 with scales, or FP4 rows.
#include <cfloat>

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
  bool x32, r32, w32, wide;                // wide: rows of x, the residual and the output are 32-byte aligned
};

// (hi, lo) += (b, blo) in two float32 words: the rounding error of the sum goes into lo (Knuth's
// TwoSum).  The low words are added first, so that the sum is the same with its operands exchanged: two lanes that
// add each other's words get the same pair.
__device__ __forceinline__ void sum2(float& hi, float& lo, float b, float blo) {
  const float s = __fadd_rn(hi, b), t = __fsub_rn(s, hi);
  lo = __fadd_rn(__fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(b, t)), __fadd_rn(lo, blo));
  hi = s;
}
__device__ __forceinline__ void lanes_sum2(float& hi, float& lo, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) {
    const float b = __shfl_xor_sync(0xffffffffu, hi, o), bl = __shfl_xor_sync(0xffffffffu, lo, o);
    sum2(hi, lo, b, bl);
  }
}

// The sum of squares of NP <= 16 pairs of channels (scaled: times 2^-128) in two words.  The running sums
// start at a power of two c of at least 16 times the largest square, so every step's rounding error
// is h^2 - (s - s_before), a difference that is exact and a fused product that keeps 2^-48 of c; c
// leaves the sums exactly.  Two steps a pair fewer than TwoSum.
template <int NP>
__device__ __forceinline__ void squares(const f32x2* h, bool scaled, float& hi, float& lo) {
  const float m = amax_pairs<NP>(h) * (scaled ? 0x1p-64f : 1.f), q = __fmul_rn(m, m);
  const float c = __uint_as_float((__float_as_uint(fminf(q, 0x1p100f)) & 0x7f800000u) + (5u << 23));
  f32x2 a = pk(c, c), b = 0;
  if (!scaled) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const f32x2 s = fma2(h[i], h[i], a);
      b = add2(b, fma2(h[i], h[i], sub2(a, s)));
      a = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const f32x2 v = mul2(h[i], pk(0x1p-64f, 0x1p-64f)), s = fma2(v, v, a);
      b = add2(b, fma2(v, v, sub2(a, s)));
      a = s;
    }
  }
  const float2 ah = unpk(sub2(a, pk(c, c))), bl = unpk(b);
  hi = ah.x, lo = bl.x;
  sum2(hi, lo, ah.y, bl.y);
  if (!(q < 0x1p100f)) hi = m <= FLT_MAX ? INFINITY : q;  // beyond the range: infinite or NaN, or treated as such
}

// RN((hi + lo) / D): a rounded quotient (rows.cuh) whose remainder, exact, takes the rest along.
__device__ __forceinline__ float mean2(float hi, float lo, int D) {
  const float d = (float)D, y = __frcp_rn(d), q0 = __fmul_rn(hi, y);
  const float q = __fmaf_rn(__fmaf_rn(-q0, d, hi), y, q0);
  return __fmaf_rn(__fmaf_rn(-q, d, hi) + lo, y, q);
}

// 1 / sqrt(ms + eps) of the two-word sum of a row's squares; scaled: the sum is that of the squares
// times 2^-128.
__device__ __forceinline__ float inverse_rms(float hi, float lo, int D, float eps, bool scaled) {
  float ms = hi;                                          // an infinity or a NaN stays one
  if (isfinite(hi)) {
    ms = mean2(hi, lo, D);
    if (scaled) ms = ms * 0x1p64f * 0x1p64f;
  }
  return __fdiv_rn(1.0f, __fsqrt_rn(ms + eps));
}

// The weights of a chunk, 1 where there are none.
__device__ __forceinline__ void load_weights(f32x2* w, const NormParams& p, int ch, bool has) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pk(1.f, 1.f);
  if (!p.w || !has) return;
  if (p.w32) {
    Raw16<true> r;
    r.load_again(p.w, 16 * ch);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = r.pair(i);
  } else {
    Raw16<false> r;
    r.load_again(p.w, 16 * ch);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = r.pair(i);
  }
}

// h = x + residual, rounded to the residual's type; a bf16 sum is left in rr too.  The sum of two bf16
// is exact in float32, or one is so small that it moves neither rounding: rounding once gives
// what rounding to float32 first gives.
template <bool X32, int RES>
__device__ __forceinline__ void add_residual(f32x2* h, const Raw16<X32>& xr, Raw16<RES == 2>& rr) {
  if constexpr (RES == 1) {
    uint32_t b[8];
    if constexpr (X32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = pack_bf16(add2(xr.pair(i), rr.pair(i)));
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        b[4 * j] = add_bf16x2(xr.q[j].x, rr.q[j].x), b[4 * j + 1] = add_bf16x2(xr.q[j].y, rr.q[j].y);
        b[4 * j + 2] = add_bf16x2(xr.q[j].z, rr.q[j].z), b[4 * j + 3] = add_bf16x2(xr.q[j].w, rr.q[j].w);
      }
    }
    rr.q[0] = make_uint4(b[0], b[1], b[2], b[3]);
    rr.q[1] = make_uint4(b[4], b[5], b[6], b[7]);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = rr.pair(i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = RES ? add2(xr.pair(i), rr.pair(i)) : xr.pair(i);
  }
}

// The scale byte of a chunk and those of the next three of its row, which neighbouring lanes hold.
__device__ __forceinline__ uint32_t merge_scales(uint32_t sb, int ch, int nchunk) {
  const uint32_t b = __shfl_down_sync(0xffffffffu, sb, 1);
  if (ch + 1 < nchunk) sb |= b << 8;
  const uint32_t c = __shfl_down_sync(0xffffffffu, sb, 2);
  if (ch + 2 < nchunk) sb |= c << 16;
  return sb;
}

// FP4 of 16 channels v: y over the matrix's scale g where there is one (dividing negates, rows.cuh), else -y.
__device__ __forceinline__ void fp4_chunk(f32x2* v, bool over, float g, uint32_t* w) {
  f32x2 n[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) n[i] = v[i];
  if (over) quotients16(n, g);
  const float a = amax16(n);
  if (quotient_ok(g) && a <= 0x1p60f) {
    fp4_encode16(n, a, w);
  } else {
    f32x2 t[8];
    uint32_t b[3];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = over ? v[i] : mul2(v[i], pk(-1.f, -1.f));
    fp4_encode16_any(t, g, b);
    w[0] = b[0], w[1] = b[1], w[2] = b[2];
  }
}

// Zero scales for the rows past the last, up to a whole tile of 128.
__device__ __forceinline__ void zero_tail(const NormParams& p) {
  const int n = ((p.T + 127) & ~127) - p.T;
  for (int i = threadIdx.x; i < n * p.nkt; i += blockDim.x)
    *reinterpret_cast<uint32_t*>(p.tiles + fp4_scale_offset(p.T + i / p.nkt, 4 * (i % p.nkt), p.nkt)) = 0;
}

}  // namespace

// The kernels below keep the sum of squares in two float32 words, the same pair in every lane of a row.  The mean
// differs from the exact one by some 2^-44 of it for rows of like values, 2^-38 where one channel outweighs the others
// (emulated on a CPU; 2^-33 if every rounding of squares() fell the same way; 2^-149 if that is more).  The float32 it
// rounds to, and with it every 4- or 8-bit code, is that of the exact mean, and the same for each split of the row over
// threads, unless the mean lies that near the middle between two float32: one row in 2^19, or 2^13.

// Aligned rows of D = 16 c channels, D <= 512: p.lanes lanes of a warp share a row, each holds one
// 16-channel chunk from the addition to the last store, and its weights for every row it works on.
// The next rows' loads are issued before this row's arithmetic.
template <int OUT, bool X32, int RES>
__global__ void __launch_bounds__(256) k_rms_norm_small(NormParams p) {
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  const int nchunk = p.D / 16;
  int grid = gridDim.x;
  if (OUT == CSA2_FP4E2M1X2 && (p.T & 127)) {
    if (blockIdx.x == --grid) return zero_tail(p);
  }
  const int rpb = (int)blockDim.x / p.lanes;              // rows of a CTA at a time
  const int ch = lane & (p.lanes - 1);
  const bool has = ch < nchunk;
  f32x2 w[8];
  load_weights(w, p, ch, has);
  const float g = OUT == CSA2_FP4E2M1X2 && p.gscale ? ld_f32(p.gscale) : 1.f;
  Raw16<X32> xr;
  Raw16<RES == 2> rr;
  const long long step = (long long)grid * rpb;
  long long row = (long long)blockIdx.x * rpb + tid / p.lanes;
  const auto fetch = [&](long long r) {
    if (has && r < p.T) {
      xr.load(p.x, r * p.sx + 16 * ch, p.wide);
      if (RES) rr.load(p.res, r * p.sr + 16 * ch, p.wide);
    } else {
      xr.zero();
      rr.zero();
    }
  };
  fetch(row);
  // a warp's rows are neighbours: it runs while its first exists
  for (; row - lane / p.lanes < p.T; row += step) {
    const bool mine = has && row < p.T;
    f32x2 h[8];
    add_residual<X32, RES>(h, xr, rr);
    if (RES == 2 && mine) store16<true>(h, p.res_out, row * p.so_res + 16 * ch, p.wide);
    if (RES == 1 && mine) rr.store(p.res_out, row * p.so_res + 16 * ch, p.wide);   // the sum, in bf16
    fetch(row + step);
    float r = 0.f;
    bool done = false;
    for (bool scaled = false;; scaled = true) {           // again where squares leave float32's range
      float hi, lo;
      squares<8>(h, scaled, hi, lo);
      lanes_sum2(hi, lo, p.lanes);
      const float v = inverse_rms(hi, lo, p.D, p.eps, scaled);
      if (!done) r = v;                                   // rows of the warp that were fine keep what they had
      done = isfinite(hi);
      if (scaled || !__any_sync(0xffffffffu, !done)) break;
    }
    // quantised forms take the negated value (rows.cuh); dividing by the matrix's scale negates
    if (OUT == CSA2_FP8E4M3 || (OUT == CSA2_FP4E2M1X2 && !p.gscale)) r = -r;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = mul2(mul2(h[i], pk(r, r)), w[i]);
    if (OUT == CSA2_BF16 || OUT == CSA2_F32) {
      if (mine) store16<OUT == CSA2_F32>(h, p.out, row * p.so + 16 * ch, p.wide);
    } else if (OUT == CSA2_FP4E2M1X2) {
      uint32_t e[3] = {0, 0, 0};
      if (mine) {
        fp4_chunk(h, p.gscale, g, e);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + row * (p.D / 2) + 8 * ch) = make_uint2(e[0], e[1]);
      }
      const uint32_t sb = merge_scales(e[2], ch, nchunk);
      if (mine && (ch & 3) == 0) *reinterpret_cast<uint32_t*>(p.tiles + fp4_scale_offset((int)row, ch, p.nkt)) = sb;
    } else {
      float m = has ? amax16(h) : 0.f;
      const int over = p.group && p.lanes > 8 ? 8 : p.lanes;   // 128 channels are eight lanes
      for (int o = over >> 1; o > 0; o >>= 1) m = max3_abs(m, __shfl_xor_sync(0xffffffffu, m, o), 0.f);
      const float s = __fdiv_rn(m, 448.0f);
      uint32_t b[4];
      if (mine) {
        fp8_encode16(h, s, b);
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + row * p.so + 16 * ch) = make_uint4(b[0], b[1], b[2], b[3]);
        if (p.group ? (ch & 7) == 0 : ch == 0)
          p.out_scale[p.group ? row * ((p.D + 127) / 128) + ch / 8 : row] = s;
      }
    }
  }
}

// Aligned rows of D = 16 c channels, D <= 8192: a CTA a row at a time, one chunk a thread from the
// addition to the last store; one barrier for the sum (and one for a row's E4M3 scale).  The next
// row's loads are issued before this row's arithmetic.
//   What bounds it: 8192 x 5120 with a residual to FP4 (275 MB, 40.6 us at the copy rate) takes 50.0 us, 5.5 TB/s;
// 55 us when two 16-byte accesses touch every sector where one of 32 bytes does.  One CTA an SM 73 us, two
// (76 registers a thread) 55, three (64 registers, spills) 53 us.  Copying the next row to shared memory
// instead of registers took 69 us; two chunks a thread 70 us.
template <int OUT, bool X32, int RES>
__global__ void __launch_bounds__(512) k_rms_norm(NormParams p) {
  pdl_wait();
  pdl_trigger();
  __shared__ float2 part[2][16];
  __shared__ float apart[2][16];
  const int tid = threadIdx.x, ch = tid, lane = tid & 31, warp = tid >> 5, nwarp = blockDim.x >> 5;
  const int nchunk = p.D / 16;
  const bool has = ch < nchunk;
  int grid = gridDim.x;
  if (OUT == CSA2_FP4E2M1X2 && (p.T & 127)) {
    if (blockIdx.x == --grid) return zero_tail(p);
  }
  f32x2 w[8];
  load_weights(w, p, ch, has);
  const float g = OUT == CSA2_FP4E2M1X2 && p.gscale ? ld_f32(p.gscale) : 1.f;
  Raw16<X32> xr;
  Raw16<RES == 2> rr;
  xr.zero();
  rr.zero();
  long long row = blockIdx.x;
  if (has && row < p.T) {
    xr.load(p.x, row * p.sx + 16 * ch, p.wide);
    if (RES) rr.load(p.res, row * p.sr + 16 * ch, p.wide);
  }
  for (int par = 0; row < p.T; row += grid, par ^= 1) {
    f32x2 h[8];
    add_residual<X32, RES>(h, xr, rr);
    if (has) {
      if (RES == 2) store16<true>(h, p.res_out, row * p.so_res + 16 * ch, p.wide);
      if (RES == 1) rr.store(p.res_out, row * p.so_res + 16 * ch, p.wide);   // the sum, in bf16
      if (row + grid < p.T) {
        xr.load(p.x, (row + grid) * p.sx + 16 * ch, p.wide);
        if (RES) rr.load(p.res, (row + grid) * p.sr + 16 * ch, p.wide);
      }
    }
    float r;
    for (bool scaled = false;; scaled = true) {           // again where squares leave float32's range
      float hi, lo;
      squares<8>(h, scaled, hi, lo);
      lanes_sum2(hi, lo, 32);
      if (scaled) __syncthreads();                        // every warp has read the first sums
      if (lane == 0) part[par][warp] = make_float2(hi, lo);
      __syncthreads();
      const float2 z = (lane & 15) < nwarp ? part[par][lane & 15] : make_float2(0.f, 0.f);
      hi = z.x, lo = z.y;
      lanes_sum2(hi, lo, 16);
      r = inverse_rms(hi, lo, p.D, p.eps, scaled);
      if (scaled || isfinite(hi)) break;
    }
    // quantised forms take the negated value (rows.cuh); dividing by the matrix's scale negates
    if (OUT == CSA2_FP8E4M3 || (OUT == CSA2_FP4E2M1X2 && !p.gscale)) r = -r;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = mul2(mul2(h[i], pk(r, r)), w[i]);
    if (OUT == CSA2_BF16 || OUT == CSA2_F32) {
      if (has) store16<OUT == CSA2_F32>(h, p.out, row * p.so + 16 * ch, p.wide);
    } else if (OUT == CSA2_FP4E2M1X2) {
      uint32_t e[3] = {0, 0, 0};
      if (has) {
        fp4_chunk(h, p.gscale, g, e);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + row * (p.D / 2) + 8 * ch) = make_uint2(e[0], e[1]);
      }
      const uint32_t sb = merge_scales(e[2], ch, nchunk);
      if (has && (ch & 3) == 0) *reinterpret_cast<uint32_t*>(p.tiles + fp4_scale_offset((int)row, ch, p.nkt)) = sb;
    } else {
      float m = has ? amax16(h) : 0.f;
      if (p.group) {                                      // 128 channels: eight lanes
        for (int o = 4; o > 0; o >>= 1) m = max3_abs(m, __shfl_xor_sync(0xffffffffu, m, o), 0.f);
      } else {
        m = warp_max_abs(m);
        if (lane == 0) apart[par][warp] = m;
        __syncthreads();
        m = warp_max_abs(lane < nwarp ? apart[par][lane] : 0.f);
      }
      const float s = __fdiv_rn(m, 448.0f);
      if (has) {
        uint32_t b[4];
        fp8_encode16(h, s, b);
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + row * p.so + 16 * ch) = make_uint4(b[0], b[1], b[2], b[3]);
        if (p.group ? (ch & 7) == 0 : ch == 0) p.out_scale[p.group ? row * ((p.D + 127) / 128) + ch / 8 : row] = s;
      }
    }
  }
}

// Any row: odd widths, unaligned rows, D up to 32768.  A CTA a row, or up to 512 channels a warp a row and
// kAnyRows rows a CTA (THREADS = 32 * kAnyRows).  N channels a thread: a warp takes 32 N neighbouring
// channels and reads and writes them 32 at a time, so that every offset is a constant and a row costs few
// instructions beside its bytes; the quantised forms pass the row through shared memory to 16-channel chunks
// (17 words apart, so that the lanes' banks differ).
//   4099 x 1001 from float32 to bf16 (24.6 MB, 3.6 us at the copy rate), float32 weights: 5.2 us with N = 16, 6.3 with 8,
// 9.7 with 4 (every warp adds the whole row's sums); bf16 weights 5.8 us; 8.5 us with channels a CTA's width apart, whose addresses are computed
// one by one; 10.8 us with that form's next row loaded ahead (more registers, fewer rows at a time).
//   20000 x 333 (40 MB, 5.9 us): 9.7 us, against 20.6 us with a CTA of one warp a row.  Up to 1024 channels a warp (N = 32)
// gains as little as it loses: 4099 x 1001 5.1 us, with a residual 8.6 against 7.9 us.
//   Aligned rows above 8192 channels come here too, and pay for the narrow accesses: 2048 x 12288 in bf16 with a residual 63 us
// (201 MB, 29.7 us at the copy rate), 2048 x 16384 77 us (39.5), to FP4 92 us (32.4); 1024 x 32768, two CTAs' registers in
// one with spills, 87 us (39.5).  k_rms_norm takes 23 us for 2048 x 8192 (19.8).
constexpr int kAnyRows = 4;

template <int OUT, int N, int THREADS>
__global__ void __launch_bounds__(THREADS) k_rms_norm_any(NormParams p) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float rows[];
  __shared__ float2 part[32];
  __shared__ float apart[32];
  constexpr bool WARP = THREADS == 32 * kAnyRows;
  constexpr int ROWS = WARP ? kAnyRows : 1;
  const int lane = threadIdx.x & 31, warp = WARP ? 0 : threadIdx.x >> 5, tid = 32 * warp + lane;
  const int nwarp = WARP ? 1 : blockDim.x >> 5, nt = 32 * nwarp;
  if (OUT == CSA2_FP4E2M1X2 && (long long)blockIdx.x * ROWS >= p.T) return zero_tail(p);
  const long long row = WARP ? (long long)blockIdx.x * ROWS + threadIdx.x / 32 : blockIdx.x;
  if (WARP && row >= p.T) return;
  float* buf = rows + (WARP ? threadIdx.x / 32 * ((p.D + 15) / 16 * 17) : 0);
  const auto sync = [] {
    if (WARP)
      __syncwarp();
    else
      __syncthreads();
  };
  // a warp's 32 N channels are neighbours, so that every offset below is a constant
  const int first = warp * 32 * N + lane, left = p.D - first;
  const auto load = [&](float (&v)[N], const void* base, long long at, bool f32) {
    if (f32) {
      const float* b = static_cast<const float*>(base) + at + first;
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = 32 * k < left ? b[32 * k] : 0.f;
    } else {
      const uint16_t* b = static_cast<const uint16_t*>(base) + at + first;
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = bf16_bits_to_f32(32 * k < left ? b[32 * k] : (uint16_t)0);
    }
  };
  const auto store = [&](const float (&v)[N], void* base, long long at, bool f32) {
    if (f32) {
      float* b = static_cast<float*>(base) + at + first;
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (32 * k < left) b[32 * k] = v[k];
    } else {
      uint16_t* b = static_cast<uint16_t*>(base) + at + first;
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (32 * k < left) b[32 * k] = __bfloat16_as_ushort(__float2bfloat16_rn(v[k]));
    }
  };
  float h[N];
  load(h, p.x, row * p.sx, p.x32);
  if (p.res) {
    float q[N];
    load(q, p.res, row * p.sr, p.r32);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      h[k] += q[k];
      if (!p.r32) h[k] = __bfloat162float(__float2bfloat16_rn(h[k]));
    }
    store(h, p.res_out, row * p.so_res, p.r32);
  }
  float r;
  for (bool scaled = false;; scaled = true) {             // again where squares leave float32's range
    float hi, lo;
    f32x2 v[N / 2];
#pragma unroll
    for (int k = 0; k < N / 2; ++k) v[k] = pk(h[2 * k], h[2 * k + 1]);
    squares<N / 2>(v, scaled, hi, lo);
    lanes_sum2(hi, lo, 32);
    if (!WARP) {
      if (scaled) __syncthreads();                        // every warp has read the first sums
      if (lane == 0) part[warp] = make_float2(hi, lo);
      __syncthreads();
      const float2 z = lane < nwarp ? part[lane] : make_float2(0.f, 0.f);
      hi = z.x, lo = z.y;
      lanes_sum2(hi, lo, 32);
    }
    r = inverse_rms(hi, lo, p.D, p.eps, scaled);
    if (scaled || isfinite(hi)) break;
  }
  if (OUT == CSA2_FP8E4M3 || (OUT == CSA2_FP4E2M1X2 && !p.gscale)) r = -r;   // as in k_rms_norm
  float w[N];
  if (p.w) load(w, p.w, 0, p.w32);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    h[k] = __fmul_rn(h[k], r);
    if (p.w) h[k] = __fmul_rn(h[k], w[k]);
  }
  if (OUT == CSA2_BF16 || OUT == CSA2_F32) return store(h, p.out, row * p.so, OUT == CSA2_F32);
  float* at = buf + (first >> 4) * 17 + (lane & 15);
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (32 * k < left) at[34 * k] = h[k];
  const int nchunk = (p.D + 15) / 16;
  for (int i = p.D + tid; i < 16 * nchunk; i += nt) buf[(i >> 4) * 17 + (i & 15)] = 0.f;
  sync();
  const auto chunk = [&](f32x2* v, int ch) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = ch < nchunk ? pk(buf[ch * 17 + 2 * i], buf[ch * 17 + 2 * i + 1]) : 0;
  };
  const int rounds = (nchunk + nt - 1) / nt;
  float rm = 0.f;
  if (OUT == CSA2_FP8E4M3 && p.group == 0) {
    for (int k = 0; k < rounds; ++k) {
      f32x2 v[8];
      chunk(v, k * nt + tid);
      rm = max3_abs(rm, amax16(v), 0.f);
    }
    rm = warp_max_abs(rm);
    if (!WARP) {
      if (lane == 0) apart[warp] = rm;
      __syncthreads();
      rm = warp_max_abs(lane < nwarp ? apart[lane] : 0.f);
    }
    if (tid == 0) p.out_scale[row] = __fdiv_rn(rm, 448.0f);
  }
  for (int k = 0; k < rounds; ++k) {
    const int ch = k * nt + tid;
    f32x2 v[8];
    chunk(v, ch);
    if (OUT == CSA2_FP4E2M1X2) {
      uint32_t e[3] = {0, 0, 0};
      if (ch < nchunk) {
        fp4_chunk(v, p.gscale, p.gscale ? ld_f32(p.gscale) : 1.f, e);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + row * (p.D / 2) + 8 * ch) = make_uint2(e[0], e[1]);
      }
      const uint32_t sb = merge_scales(e[2], ch, nchunk);
      if ((ch & 3) == 0 && ch < nchunk)
        *reinterpret_cast<uint32_t*>(p.tiles + fp4_scale_offset((int)row, ch, p.nkt)) = sb;
    } else {
      float m = rm;
      if (p.group) {                                      // 128 channels: eight lanes
        m = amax16(v);
        for (int o = 4; o > 0; o >>= 1) m = max3_abs(m, __shfl_xor_sync(0xffffffffu, m, o), 0.f);
        if ((ch & 7) == 0 && ch < nchunk) p.out_scale[row * ((p.D + 127) / 128) + ch / 8] = __fdiv_rn(m, 448.0f);
      }
      uint32_t b[4];
      fp8_encode16(v, __fdiv_rn(m, 448.0f), b);
      if (ch < nchunk)
#pragma unroll
        for (int i = 0; i < 16; ++i) buf[ch * 17 + i] = __uint_as_float((b[i / 4] >> (8 * (i % 4))) & 0xffu);
    }
  }
  if (OUT == CSA2_FP8E4M3) {
    sync();
    for (int i = tid; i < p.D; i += nt)
      static_cast<uint8_t*>(p.out)[row * p.so + i] = (uint8_t)__float_as_uint(buf[(i >> 4) * 17 + (i & 15)]);
  }
}

namespace {

// A persistent grid: as many CTAs as the GPU holds at once (looked up once for a kernel, shape and device).
template <typename K>
cudaError_t launch_rows(K* kernel, PerDevice<int>& resident, const NormParams& p, int rows, int threads, bool tail,
                        cudaStream_t st) {
  const int* most = nullptr;
  const cudaError_t e = resident.get(&most, [&](int& n) {
    int sms = 0, per = 0;
    cudaError_t e = sm_count(&sms);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, 0);
    n = sms * (per > 0 ? per : 1);
    return e;
  });
  if (e != cudaSuccess) return e;
  const long long blocks = ((long long)p.T + rows - 1) / rows;
  return launch_k(kernel, (unsigned)(blocks < *most ? blocks : *most) + (tail ? 1u : 0u), threads, 0, st, p);
}

template <int OUT, bool X32, int RES>
cudaError_t launch_aligned(const NormParams& p, cudaStream_t st) {
  const bool tail = OUT == CSA2_FP4E2M1X2 && p.T % 128;
  if (p.D <= 512) {
    static PerDevice<int> resident;
    return launch_rows(k_rms_norm_small<OUT, X32, RES>, resident, p, 256 / p.lanes, 256, tail, st);
  }
  static PerDevice<int> resident[17];                     // by warps of a CTA
  const int threads = (p.D / 16 + 31) & ~31;
  return launch_rows(k_rms_norm<OUT, X32, RES>, resident[threads / 32], p, 1, threads, tail, st);
}

template <int OUT, int N, int THREADS>
cudaError_t launch_any(const NormParams& p, cudaStream_t st) {
  constexpr bool quantised = OUT == CSA2_FP8E4M3 || OUT == CSA2_FP4E2M1X2, warp = THREADS == 32 * kAnyRows;
  const int threads = warp ? THREADS : ((p.D + N - 1) / N + 31) & ~31;
  const size_t smem = quantised ? (size_t)((p.D + 15) / 16) * 17 * 4 * (warp ? kAnyRows : 1) : 0;
  if (quantised && !warp) {
    static SmemLimit limit;
    const cudaError_t e = limit.raise(k_rms_norm_any<OUT, N, THREADS>, 2048 * 17 * 4);
    if (e != cudaSuccess) return e;
  }
  const unsigned blocks = warp ? (unsigned)(((long long)p.T + kAnyRows - 1) / kAnyRows) : (unsigned)p.T;
  const bool tail = OUT == CSA2_FP4E2M1X2 && p.T % 128;
  return launch_k(k_rms_norm_any<OUT, N, THREADS>, blocks + (tail ? 1u : 0u), threads, smem, st, p);
}

template <int OUT>
cudaError_t launch_form(const NormParams& p, bool aligned, cudaStream_t st) {
  if (aligned && p.D <= 8192) {
    const int res = !p.res ? 0 : p.r32 ? 2 : 1;
#define CSA2_NORM(X, R) \
  if (p.x32 == X && res == R) return launch_aligned<OUT, X, R>(p, st)
    CSA2_NORM(false, 0);
    CSA2_NORM(false, 1);
    CSA2_NORM(false, 2);
    CSA2_NORM(true, 0);
    CSA2_NORM(true, 1);
    CSA2_NORM(true, 2);
#undef CSA2_NORM
  }
  if (p.D <= 512) return launch_any<OUT, 16, 32 * kAnyRows>(p, st);
  return p.D <= 16384 ? launch_any<OUT, 16, 1024>(p, st) : launch_any<OUT, 32, 1024>(p, st);
}

bool rows_aligned(const void* p, long long stride, int esize, int to = 16) {
  return ((uintptr_t)p & (to - 1)) == 0 && (stride * esize) % to == 0;
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
  const int xb = p.x32 ? 4 : 2, ob = a.out_form == CSA2_F32 ? 4 : a.out_form == CSA2_BF16 ? 2 : 1;
  const auto rows_to = [&](int to) {
    return rows_aligned(a.x, many ? a.x_stride : 0, xb, to) && rows_aligned(a.residual, many ? a.residual_stride : 0, rb, to) &&
           rows_aligned(a.residual_out, many ? a.residual_out_stride : 0, rb, to) &&
           (a.out_form > CSA2_F32 || rows_aligned(a.out, many ? a.out_stride : 0, ob, to));
  };
  const bool aligned = a.D % 16 == 0 && rows_to(16) && rows_aligned(a.weight, 0, 1) &&
                       (a.out_form != CSA2_FP8E4M3 || rows_aligned(a.out, many ? a.out_stride : 0, 1));
  p.wide = aligned && rows_to(32);
  switch (a.out_form) {
    case CSA2_BF16: return launch_form<CSA2_BF16>(p, aligned, st);
    case CSA2_F32: return launch_form<CSA2_F32>(p, aligned, st);
    case CSA2_FP8E4M3: return launch_form<CSA2_FP8E4M3>(p, aligned, st);
    default: return launch_form<CSA2_FP4E2M1X2>(p, aligned, st);
  }
}

}  // namespace csa2

// Rotary positions (csa2_rope) and their tables (csa2_rope_table).
#include <cmath>

#include "internal.h"
#include "rows.cuh"

namespace csa2 {

CSA2_DEFINE_ERROR_WORD(g_err_rope);

namespace {

struct RopeParams {
  const void* x;
  void* out;
  const int* pos;
  const float* cos;
  const float* sin;
  long long xt, xh, ot, oh;
  int H, D, d_rope, first, max_pos, units, turn_units;
  bool inverse;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_bits_to_f32(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f32(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// V channels of type T moved as one access (16 bytes, or one element when V == 1).
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

}  // namespace

// A unit is V neighbouring channels that are copied, or that turn: V channels of V/2
// interleaved pairs (V = 1: one pair), or V channels of each half.  A thread keeps its unit and
// runs over heads, so a token's angles are read once for all of them.  A token with a bad
// position is copied as it is.
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(256) k_rope(RopeParams p) {
  pdl_wait();
  pdl_trigger();
  using Vt = Vec<T, V>;
  constexpr int NP = INTERLEAVED ? (V > 1 ? V / 2 : 1) : V;   // pairs of a unit
  const long long t = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + t * p.xt;
  T* o = static_cast<T*>(p.out) + t * p.ot;
  const int h0 = blockIdx.y * blockDim.y + threadIdx.y, hs = gridDim.y * blockDim.y;
  const int half = p.d_rope / 2;
  const int ps = ld_s32(p.pos + t);
  const bool turns = ps >= 0 && ps < p.max_pos;
  if (!turns && threadIdx.x == 0 && threadIdx.y == 0) raise_error(&g_err_rope, CSA2_DEVERR_POS);
  for (int u = threadIdx.x; u < p.units; u += blockDim.x) {
    if (u >= p.turn_units) {                              // channels that are copied
      int c = (u - p.turn_units) * V;
      if (c >= p.first) c += p.d_rope;
      for (int h = h0; h < p.H; h += hs)
        *reinterpret_cast<Vt*>(o + h * p.oh + c) = *reinterpret_cast<const Vt*>(x + h * p.xh + c);
      continue;
    }
    float cs[NP], sn[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const long long at = (long long)ps * half + u * NP + i;
      cs[i] = turns ? ld_f32(p.cos + at) : 1.f;
      sn[i] = turns ? ld_f32(p.sin + at) : 0.f;
      if (p.inverse) sn[i] = -sn[i];
    }
    if (INTERLEAVED && V > 1) {
      const int c = p.first + u * V;
      for (int h = h0; h < p.H; h += hs) {
        Vt v = *reinterpret_cast<const Vt*>(x + h * p.xh + c);
        if (turns) {
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            float a = to_f32(v.e[2 * i]), b = to_f32(v.e[2 * i + (V > 1)]);
            rope_pair(a, b, cs[i], sn[i]);
            v.e[2 * i] = from_f32<T>(a);
            v.e[2 * i + (V > 1)] = from_f32<T>(b);
          }
        }
        *reinterpret_cast<Vt*>(o + h * p.oh + c) = v;
      }
    } else {
      const int c = p.first + (INTERLEAVED ? 2 * u : u * V), c2 = INTERLEAVED ? c + 1 : c + half;
      for (int h = h0; h < p.H; h += hs) {
        Vt v = *reinterpret_cast<const Vt*>(x + h * p.xh + c), w = *reinterpret_cast<const Vt*>(x + h * p.xh + c2);
        if (turns) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float a = to_f32(v.e[i]), b = to_f32(w.e[i]);
            rope_pair(a, b, cs[i], sn[i]);
            v.e[i] = from_f32<T>(a);
            w.e[i] = from_f32<T>(b);
          }
        }
        *reinterpret_cast<Vt*>(o + h * p.oh + c) = v;
        *reinterpret_cast<Vt*>(o + h * p.oh + c2) = w;
      }
    }
  }
}

namespace {

template <typename T, int V>
cudaError_t launch_rope_v(const csa2_rope_args& a, RopeParams p, cudaStream_t st) {
  const bool in_place = a.out == a.x;
  p.turn_units = a.interleaved ? (V > 1 ? a.d_rope / V : a.d_rope / 2) : a.d_rope / 2 / V;
  p.units = p.turn_units + (in_place ? 0 : (a.D - a.d_rope) / V);
  const int tx = p.units < 256 ? p.units : 256;
  const int ty = 256 / tx < a.H ? 256 / tx : a.H;
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int per = (a.H + ty - 1) / ty;                    // CTAs that give each thread one head
  long long gy = (8LL * sms + a.T - 1) / a.T;             // fill the GPU, then several heads a thread
  if (gy > per) gy = per;
  const dim3 grid((unsigned)a.T, (unsigned)gy), block((unsigned)tx, (unsigned)ty);
  return a.interleaved ? launch_k(k_rope<T, V, true>, grid, block, 0, st, p)
                       : launch_k(k_rope<T, V, false>, grid, block, 0, st, p);
}

}  // namespace

cudaError_t launch_rope(const csa2_rope_args& a, cudaStream_t st) {
  if (a.T == 0 || a.H == 0) return cudaSuccess;
  RopeParams p{};
  p.x = a.x, p.out = a.out, p.pos = a.pos, p.cos = a.rope_cos, p.sin = a.rope_sin;
  p.xt = a.x_stride_t, p.xh = a.x_stride_h, p.ot = a.out_stride_t, p.oh = a.out_stride_h;
  p.H = a.H, p.D = a.D, p.d_rope = a.d_rope, p.first = a.rot_first, p.max_pos = a.rope_max_pos;
  p.inverse = a.inverse != 0;
  const int v = a.dtype == CSA2_F32 ? 4 : 8;
  const bool vec = ((uintptr_t)a.x & 15) == 0 && ((uintptr_t)a.out & 15) == 0 && a.x_stride_t % v == 0 &&
                   a.x_stride_h % v == 0 && a.out_stride_t % v == 0 && a.out_stride_h % v == 0 && a.D % v == 0 &&
                   a.rot_first % v == 0 && (a.interleaved ? a.d_rope : a.d_rope / 2) % v == 0;
  if (a.dtype == CSA2_F32) return vec ? launch_rope_v<float, 4>(a, p, st) : launch_rope_v<float, 1>(a, p, st);
  return vec ? launch_rope_v<uint16_t, 8>(a, p, st) : launch_rope_v<uint16_t, 1>(a, p, st);
}

// ---------------------------------------------------------------------------------
// Tables
// ---------------------------------------------------------------------------------
namespace {

struct TableParams {
  float* cos;
  float* sin;
  int positions, half;
  float magnitude;
  unsigned long long turn[128];   // turns per position of channel i, times 2^64
};

}  // namespace

// The angle p f_i in turns, modulo 1, is a 64-bit product; its nearest multiple of a quarter
// turn picks which of +-sin, +-cos of the remainder (at most an eighth of a turn) is which.
__global__ void __launch_bounds__(256) k_rope_table(TableParams t) {
  pdl_wait();
  pdl_trigger();
  const long long n = (long long)t.positions * t.half;
  for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (long long)gridDim.x * blockDim.x) {
    const unsigned long long a = (unsigned long long)(e / t.half) * t.turn[e % t.half];
    const unsigned long long q = (a + (1ull << 61)) >> 62;          // quarter turns, 0..4
    const long long r = (long long)(a - (q << 62));                 // remainder, +-2^61
    float s, c;
    sincospif((float)r * 0x1p-63f, &s, &c);                         // half turns
    const float cv = (q & 1) ? s : c, sv = (q & 1) ? c : s;
    t.cos[e] = t.magnitude * (((q + 1) & 2) ? -cv : cv);
    t.sin[e] = t.magnitude * ((q & 2) ? -sv : sv);
  }
}

cudaError_t launch_rope_table(const csa2_rope_table_args& a, cudaStream_t st) {
  if (a.positions == 0) return cudaSuccess;
  TableParams t{};
  t.cos = a.rope_cos, t.sin = a.rope_sin, t.positions = a.positions, t.half = a.d_rope / 2;
  t.magnitude = (float)a.magnitude;
  const double two_pi = 6.283185307179586476925;
  double lo = 0, hi = 0;
  if (a.scaling == CSA2_ROPE_YARN) {
    // the channel that turns n times within the original context
    const auto channel = [&](double n) {
      return a.d_rope * std::log(a.orig_positions / (n * two_pi)) / (2 * std::log(a.theta));
    };
    lo = std::fmax(std::floor(channel(a.beta_fast)), 0.0);
    hi = std::fmin(std::ceil(channel(a.beta_slow)), (double)(a.d_rope - 1));
  }
  for (int i = 0; i < t.half; ++i) {
    double f = std::pow(a.theta, -2.0 * i / a.d_rope);
    if (a.scaling == CSA2_ROPE_LINEAR) f /= a.factor;
    if (a.scaling == CSA2_ROPE_YARN) {
      const double slow = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
      f = f / a.factor * slow + f * (1 - slow);
    }
    const double turn = f / two_pi;                       // below 1/6: theta > 1
    t.turn[i] = (unsigned long long)std::ldexp(turn, 64);
  }
  const long long n = (long long)t.positions * t.half;
  const long long blocks = (n + 255) / 256;
  return launch_k(k_rope_table, (unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)), 256, 0, st, t);
}

uint32_t read_clear_error_rope() {
  unsigned int v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_err_rope, sizeof(v));
  if (v) cudaMemcpyToSymbol(g_err_rope, &z, sizeof(z));
  return v;
}

}  // namespace csa2

// Rotary positions (csa2_rope) and their tables (csa2_rope_table).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "internal.h"
#include "rows.cuh"

namespace csa2 {

CSA2_DEFINE_ERROR_WORD(g_err_rope);

namespace {

constexpr int kThreads = 128;

struct RopeParams {
  const void* x;
  void* out;
  const int* pos;
  const float* cos;
  const float* sin;
  long long xt, xh, ot, oh;
  int T, H, D, d_rope, first, max_pos, units, turn_units;
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

// N floats from a 4 N- (16- at most) byte aligned address.
template <int N>
__device__ __forceinline__ void load_angles(float* v, const float* p) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 q = ld_v4(p + i);
      v[i] = __uint_as_float(q.x), v[i + 1] = __uint_as_float(q.y);
      v[i + 2] = __uint_as_float(q.z), v[i + 3] = __uint_as_float(q.w);
    }
  } else if constexpr (N == 2) {
    asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "l"(p));
  } else {
    v[0] = ld_f32(p);
  }
}

// A unit is V neighbouring channels that are copied, or that turn: V channels of V/2
// interleaved pairs (V = 1: one pair), or V channels of each half.  A thread keeps its unit and
// runs over heads, so a token's angles are read once for all of them, and over tokens, whose
// positions it reads one ahead: a CTA for each token spends its life waiting for the position
// and then for the angles.  A token with a bad position is copied as it is.
//   What bounds it: memory.  8192 tokens x 64 heads x 128 channels in bf16 (273 MB, 40.2 us at the copy
// rate): 46.0 us; a CTA for each token 52.4 us, two heads' loads at once 51 us (fewer CTAs fit),
// 256 threads 46.4 us.  The same on rows that start off every boundary (V = 1): 64 us with eight heads' loads at once,
// 71 with four, 177 with one.
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, V > 1 ? 10 : 8) k_rope(RopeParams p) {
  pdl_wait();
  pdl_trigger();
  using Vt = Vec<T, V>;
  constexpr int NP = INTERLEAVED ? (V > 1 ? V / 2 : 1) : V;   // pairs of a unit
  constexpr int PARTS = INTERLEAVED && V > 1 ? 1 : 2;         // vectors of a unit that turns
  constexpr int HEADS = V > 1 ? 1 : 8;                        // of a thread at once: single channels need more in flight
  const int h0 = blockIdx.y * blockDim.y + threadIdx.y, hs = gridDim.y * blockDim.y;
  const int half = p.d_rope / 2;
  int next = blockIdx.x < p.T ? ld_s32(p.pos + blockIdx.x) : 0;   // a token's position, one token ahead
  for (long long t = blockIdx.x; t < p.T; t += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + t * p.xt;
    T* o = static_cast<T*>(p.out) + t * p.ot;
    const int ps = next;
    const bool good = ps >= 0 && ps < p.max_pos;
    if (t + gridDim.x < p.T) next = ld_s32(p.pos + t + gridDim.x);
    if (!good && threadIdx.x == 0 && threadIdx.y == 0) raise_error(&g_err_rope, CSA2_DEVERR_POS);
    for (int u = threadIdx.x; u < p.units; u += blockDim.x) {
      const bool turn = u < p.turn_units, turns = turn && good;
      int c = (u - p.turn_units) * V, c2 = 0;             // the unit's channels
      if (!turn) {
        if (c >= p.first) c += p.d_rope;
      } else {
        c = p.first + (PARTS == 2 && INTERLEAVED ? 2 * u : u * V);
        c2 = INTERLEAVED ? c + 1 : c + half;
      }
      float cs[NP], sn[NP];
      if (turns) {
        load_angles<NP>(cs, p.cos + (long long)ps * half + u * NP);
        load_angles<NP>(sn, p.sin + (long long)ps * half + u * NP);
      }
      for (int h = h0; h < p.H; h += HEADS * hs) {
        Vt v[HEADS], w[HEADS];
#pragma unroll
        for (int j = 0; j < HEADS; ++j) {
          if (HEADS > 1 && h + j * hs >= p.H) break;
          const T* from = x + (h + j * hs) * p.xh;
          v[j] = *reinterpret_cast<const Vt*>(from + c);
          if (PARTS == 2 && turn) w[j] = *reinterpret_cast<const Vt*>(from + c2);
        }
#pragma unroll
        for (int j = 0; j < HEADS; ++j) {
          if (HEADS > 1 && h + j * hs >= p.H) break;
          if (turns) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              T& e0 = PARTS == 1 ? v[j].e[2 * i] : v[j].e[i];
              T& e1 = PARTS == 1 ? v[j].e[2 * i + (V > 1)] : w[j].e[i];
              float a = to_f32(e0), b = to_f32(e1);
              rope_pair(a, b, cs[i], p.inverse ? -sn[i] : sn[i]);
              e0 = from_f32<T>(a);
              e1 = from_f32<T>(b);
            }
          }
          T* to = o + (h + j * hs) * p.oh;
          *reinterpret_cast<Vt*>(to + c) = v[j];
          if (PARTS == 2 && turn) *reinterpret_cast<Vt*>(to + c2) = w[j];
        }
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
  const auto k = a.interleaved ? k_rope<T, V, true> : k_rope<T, V, false>;
  static PerDevice<int> resident[2];                      // CTAs the GPU holds at once
  const int* most = nullptr;
  const cudaError_t e = resident[a.interleaved != 0].get(&most, [&](int& n) {
    int sms = 0, per = 0;
    cudaError_t e = sm_count(&sms);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, k, kThreads, 0);
    n = sms * (per > 0 ? per : 1);
    return e;
  });
  if (e != cudaSuccess) return e;
  const int r = *most;
  const int tx = p.units < kThreads ? p.units : kThreads;
  const int ty = kThreads / tx < a.H ? kThreads / tx : a.H;
  const int per = (a.H + ty - 1) / ty;                    // CTAs that give each thread one head
  long long gy = (r + a.T - 1LL) / a.T;                     // fill the GPU, then several heads a thread
  if (gy > per) gy = per;
  const long long gx = a.T < r / gy ? a.T : r / gy;
  const dim3 grid((unsigned)(gx > 0 ? gx : 1), (unsigned)gy), block((unsigned)tx, (unsigned)ty);
  return launch_k(k, grid, block, 0, st, p);
}

}  // namespace

cudaError_t launch_rope(const csa2_rope_args& a, cudaStream_t st) {
  if (a.T == 0 || a.H == 0) return cudaSuccess;
  RopeParams p{};
  p.x = a.x, p.out = a.out, p.pos = a.pos, p.cos = a.rope_cos, p.sin = a.rope_sin;
  p.xt = a.x_stride_t, p.xh = a.x_stride_h, p.ot = a.out_stride_t, p.oh = a.out_stride_h;
  p.T = a.T, p.H = a.H, p.D = a.D, p.d_rope = a.d_rope, p.first = a.rot_first, p.max_pos = a.rope_max_pos;
  p.inverse = a.inverse != 0;
  const int v = a.dtype == CSA2_F32 ? 4 : 8;
  const bool vec = ((uintptr_t)a.x & 15) == 0 && ((uintptr_t)a.out & 15) == 0 && a.x_stride_t % v == 0 &&
                   a.x_stride_h % v == 0 && a.out_stride_t % v == 0 && a.out_stride_h % v == 0 && a.D % v == 0 &&
                   a.rot_first % v == 0 && (a.interleaved ? a.d_rope : a.d_rope / 2) % v == 0 &&
                   ((uintptr_t)a.rope_cos & 15) == 0 && ((uintptr_t)a.rope_sin & 15) == 0;
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
  f32x2 m, minus_m, low;          // the magnitude as a float32, minus it, and what that leaves out, over it: each twice
  unsigned long long turn[128];   // turns per position of channel i, times 2^64
};

// The magnitude m (1 + low) times sin and cos of pi/2 x / 2^32 for a pair of |x| <= 2^31 (an eighth of a turn at most):
// Taylor's series to the powers 9 and 10, whose next terms are below 2e-9, at the rounded angle a, and the first
// derivative for what the rounding (of x's last 8 bits, of pi and of the product) left out.  What cosine and sine
// differ from 1 and a by, low among it, is small; 1 and a times m join it in the last rounding, whose half step is most of the
// error: 2 to 7 % more in root mean square than rounding alone (emulated on a CPU), where rounding the functions and
// then their products made it 28 to 107 % more.
__device__ __forceinline__ void sincos_pair(int x0, int x1, const TableParams& p, f32x2& s, f32x2& c) {
  const float q = 1.57079632679489662f * 0x1p-32f;
  const float ql = (float)((1.57079632679489662 - (double)1.57079632679489662f) * 0x1p-32);
  const auto k = [](float v) { return pk(v, v); };
  const f32x2 xh = pk((float)(x0 & ~255), (float)(x1 & ~255));
  const f32x2 xl = pk((float)(x0 & 255), (float)(x1 & 255));
  const f32x2 na = mul2(xh, k(-q)), z = mul2(na, na);     // -a, a^2
  const f32x2 left = fma2(xh, k(ql), fma2(xl, k(q), fma2(xh, k(q), na)));   // what a leaves out
  f32x2 t = fma2(z, k(-1.0f / 3628800), k(1.0f / 40320));
  t = fma2(z, t, k(-1.0f / 720));
  t = fma2(z, t, k(1.0f / 24));
  t = fma2(z, t, k(-0.5f));
  c = fma2(fma2(z, t, fma2(left, na, p.low)), p.m, p.m);
  t = fma2(z, k(1.0f / 362880), k(-1.0f / 5040));
  t = fma2(z, t, k(1.0f / 120));
  t = fma2(z, t, k(-1.0f / 6));
  t = fma2(z, t, p.low);
  s = fma2(na, p.minus_m, fma2(mul2(na, t), p.minus_m, mul2(left, c)));
}

}  // namespace

// The angle p f_i in turns, modulo 1, is a 64-bit product that a thread carries from one of its
// positions to the next by an addition.  Its nearest multiple of a quarter turn picks which of
// +-sin, +-cos of the remainder is which.  V channels a thread (4, or 1 where half % 4 != 0).
//   1,048,576 positions x 32 pairs (268 MB written, 39.5 us at the copy rate): 38.1 us; with the library's
// sincospif and a 64-bit division for the place it took 271 us, with the magnitude packed in registers instead of the
// parameters 39.9 us.
template <int V>
__global__ void __launch_bounds__(256) k_rope_table(const __grid_constant__ TableParams t) {
  pdl_wait();
  pdl_trigger();
  const int groups = t.half / V, slots = blockDim.x / groups, slot = threadIdx.x / groups;
  if (slot >= slots) return;
  const int i0 = (threadIdx.x - slot * groups) * V;
  const int step = gridDim.x * slots;
  int p = blockIdx.x * slots + slot;
  unsigned long long a[V], d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    a[i] = (unsigned long long)p * t.turn[i0 + i];
    d[i] = (unsigned long long)step * t.turn[i0 + i];
  }
  for (; p < t.positions; p += step) {
    float c[V + V % 2], s[V + V % 2];
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const int j = V > 1 ? i + 1 : i;
      // the fraction of a quarter turn, as a signed number the distance to the nearest one
      const int x0 = (int)__funnelshift_l((uint32_t)a[i], (uint32_t)(a[i] >> 32), 2);
      const int x1 = (int)__funnelshift_l((uint32_t)a[j], (uint32_t)(a[j] >> 32), 2);
      f32x2 sp, cp;
      sincos_pair(x0, x1, t, sp, cp);
      const float2 sv = unpk(sp), cv = unpk(cp);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // bits 31, 30: the nearest multiple of a quarter turn
        const uint32_t q = (uint32_t)(a[k ? j : i] >> 32) + 0x20000000u;
        const float sk = k ? sv.y : sv.x, ck = k ? cv.y : cv.x;
        const bool odd = q & 0x40000000u;
        c[i + k] = __uint_as_float(__float_as_uint(odd ? sk : ck) ^ ((q + 0x40000000u) & 0x80000000u));
        s[i + k] = __uint_as_float(__float_as_uint(odd ? ck : sk) ^ (q & 0x80000000u));
      }
    }
    const long long at = (long long)p * t.half + i0;
    if constexpr (V == 4) {
      *reinterpret_cast<float4*>(t.cos + at) = make_float4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<float4*>(t.sin + at) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
      t.cos[at] = c[0];
      t.sin[at] = s[0];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] += d[i];
  }
}

cudaError_t launch_rope_table(const csa2_rope_table_args& a, cudaStream_t st) {
  if (a.positions == 0) return cudaSuccess;
  TableParams t{};
  t.cos = a.rope_cos, t.sin = a.rope_sin, t.positions = a.positions, t.half = a.d_rope / 2;
  const auto twice = [](float v) {
    uint32_t u;
    memcpy(&u, &v, sizeof(u));
    return (f32x2)u << 32 | u;
  };
  const float m = (float)a.magnitude;
  t.m = twice(m), t.minus_m = twice(-m), t.low = twice(m > 0.f ? (float)((a.magnitude - m) / m) : 0.f);
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
  const bool vec = t.half % 4 == 0 && ((uintptr_t)t.cos & 15) == 0 && ((uintptr_t)t.sin & 15) == 0;
  const int slots = 256 / (vec ? t.half / 4 : t.half);    // half <= 128
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // About twelve positions a thread, but from five CTAs an SM (as many as run at once) to 24.  us by CTAs an SM:
  //     65,536 x 32   5: 4.0,  8: 4.5, 12: 5.4, 24: 5.7      1,048,576 x 32   5: 40.1,  8: 40.3, 12: 38.1, 24: 38.6
  //     65,536 x 64   5: 6.4,  8: 7.4, 12: 9.0, 24: 14.8     1,048,576 x 64   5: 79.5,  8: 80.8, 12: 77.9, 24: 74.5
  //    262,144 x 32   5: 11.2, 8: 11.3, 12: 11.5, 24: 12.9    524,288 x 32   5: 20.7,  9: 20.3, 12: 20.4, 24: 21.2
  // Not whole numbers of them cost more: 524,288 x 32 21.3 us with 6.7.
  const int all = (t.positions + slots - 1) / slots;
  const int per_sm = std::min(std::max(all / 12 / sms + 1, 5), 24), blocks = std::min(all, per_sm * sms);
  return vec ? launch_k(k_rope_table<4>, (unsigned)blocks, 256, 0, st, t) : launch_k(k_rope_table<1>, (unsigned)blocks, 256, 0, st, t);
}

uint32_t read_clear_error_rope() {
  unsigned int v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_err_rope, sizeof(v));
  if (v) cudaMemcpyToSymbol(g_err_rope, &z, sizeof(z));
  return v;
}

}  // namespace csa2

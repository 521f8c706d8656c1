// Attention over the paged 8-bit cache (csa2_kv8_attn).
#include "internal.h"
#include "kv8.cuh"

namespace csa2 {

CSA2_DEFINE_ERROR_WORD(g_err_kv8);

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void store_out(const csa2_kv8_attn_args& a, long long i, float v) {
  if (a.out_dtype == CSA2_F32) reinterpret_cast<float*>(a.out)[i] = v;
  else reinterpret_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16_rn(v);
}

// A CTA a (row, query head), four warps that take every fourth page: a key a lane for the scores, D / 32 channels a
// lane for the values.
template <int D>
__global__ void __launch_bounds__(128) k_kv8_attn(const csa2_kv8_attn_args a) {
  constexpr int kPer = D / 32;
  __shared__ float q[D], s_o[4][D], s_m[4], s_l[4];
  const csa2_kv8_cache& c = a.cache;
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, hq = blockIdx.y, h = hq / (a.Hq / c.Hkv), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = find_seq(a.start, a.S, t);
  if (s < 0) return;
  const int pos = row_pos(c, a.start, a.length, s, t, &g_err_kv8);
  if (threadIdx.x < D)
    q[threadIdx.x] = bf16_bits_to_f32(a.q[t * a.q_stride_t + hq * a.q_stride_h + threadIdx.x]) * (a.softmax_scale * kLog2e);
  __syncthreads();
  const int from = a.window > 0 && pos + 1 > a.window ? pos + 1 - a.window : 0;
  const int* list = a.pages ? a.pages + ((long long)t * c.Hkv + h) * a.list_len : nullptr;
  const int first = list ? 0 : from >> kPageShift;
  const int last = pos < 0 ? 0 : list ? a.list_len : (pos >> kPageShift) + 1;
  float m = -INFINITY, l = 0.f, o[kPer] = {};
  for (int i = first + warp; i < last; i += 4) {
    const int j = list ? list[i] : i;
    if (j < 0) continue;
    if (j >= c.max_pages) {
      if (lane == 0) raise_error(&g_err_kv8, CSA2_DEVERR_PAGE_SLOT);
      continue;
    }
    if (j > pos >> kPageShift) continue;
    const int page = page_id(c, s, j, &g_err_kv8);
    if (page < 0) continue;
    const long long ph = (long long)page * c.Hkv + h;
    const float ks = c.k_scale[ph], vs = c.v_scale[ph];
    for (int b = 0; b < kPage; b += 32) {
      const int token = j * kPage + b + lane;
      const bool seen = token <= pos && token >= from;
      const uint32_t see = __ballot_sync(0xffffffffu, seen);
      if (!see) continue;
      float x = -INFINITY;
      if (seen) {
        const uint32_t* k = reinterpret_cast<const uint32_t*>(c.k + (ph * kPage + b + lane) * D);
        float dot = 0.f;
        for (int e = 0; e < D / 4; ++e) {
          float f[4];
          e4m3x4_to_f32(k[e], f);
          dot += f[0] * q[4 * e] + f[1] * q[4 * e + 1] + f[2] * q[4 * e + 2] + f[3] * q[4 * e + 3];
        }
        x = dot * ks;
      }
      float top = x;
#pragma unroll
      for (int e = 16; e > 0; e >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, e));
      const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2f(m - base), p = seen ? exp2f(x - base) : 0.f;
      m = mn;
      l = l * alpha + p;
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[e] *= alpha;
      for (uint32_t left = see; left; left &= left - 1) {
        const int r = __ffs(left) - 1;
        const float w = __shfl_sync(0xffffffffu, p, r) * vs;
        const uint8_t* v = c.v + (ph * kPage + b + r) * D + lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] += w * e4m3_to_f32(v[e]);
      }
    }
  }
#pragma unroll
  for (int e = 16; e > 0; e >>= 1) l += __shfl_xor_sync(0xffffffffu, l, e);
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) s_o[warp][lane * kPer + e] = o[e];
  __syncthreads();
  const float top = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3])), base = top == -INFINITY ? 0.f : top;
  float sum = 0.f, v = 0.f;
  for (int w = 0; w < 4; ++w) {
    const float f = exp2f(s_m[w] - base);
    sum += s_l[w] * f;
    if (threadIdx.x < D) v += s_o[w][threadIdx.x] * f;
  }
  const long long row = (long long)t * a.Hq + hq;
  if (threadIdx.x < D) store_out(a, row * D + threadIdx.x, sum == 0.f ? 0.f : v / sum);
  if (threadIdx.x == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

}  // namespace

size_t kv8_attn_workspace_bytes(const csa2_kv8_attn_args&) { return 0; }

cudaError_t launch_kv8_attn(const csa2_kv8_attn_args& a, void*, cudaStream_t st) {
  if (a.T == 0 || a.S == 0) return cudaSuccess;
  const dim3 grid(a.T, a.Hq);
  return a.cache.D == 64 ? launch_k(k_kv8_attn<64>, grid, dim3(128), 0, st, a)
                         : launch_k(k_kv8_attn<128>, grid, dim3(128), 0, st, a);
}

uint32_t read_clear_error_kv8() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_err_kv8, sizeof(v));
  if (v) cudaMemcpyToSymbol(g_err_kv8, &z, sizeof(z));
  return v;
}

}  // namespace csa2

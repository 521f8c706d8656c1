// The paged 8-bit cache's tables, append and page selection (csa2_page_plan, csa2_kv8_append,
// csa2_kv8_select).
#include <limits.h>

#include "internal.h"
#include "kv8.cuh"

namespace csa2 {

CSA2_DEFINE_ERROR_WORD(g_err_paged);

namespace {

// ---- block scans ----------------------------------------------------------------------------

// Inclusive sum over the block (a multiple of 32 threads, at most 1024); *total its last value.  warp_sums: 33 values.
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();                       // the sums of a scan before this one have been read
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < warps ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[warps - 1];
  return v + (warp ? warp_sums[warp - 1] : 0);
}

// ---- csa2_page_plan -------------------------------------------------------------------------

constexpr int kPlanThreads = 1024;

// One CTA: the two prefix sums (rows, pages) over the sequences, 1024 at a time, and the new entries of the page table.
__global__ void __launch_bounds__(kPlanThreads) k_plan_scan(const csa2_page_plan_args a) {
  __shared__ long long sums[33];
  __shared__ int first_page[kPlanThreads], pages_before[kPlanThreads + 1];
  pdl_wait();
  pdl_trigger();
  long long rows = 0, pages = 0;         // of the sequences before this chunk
  const int head = a.free_head[0];
  unsigned int err = 0;
  if (threadIdx.x == 0) a.start[0] = 0;
  for (int s0 = 0; s0 < a.S; s0 += kPlanThreads) {
    const int s = s0 + threadIdx.x;
    long long held = 0, add = 0;
    if (s < a.S) {
      held = a.length[s];
      add = a.add[s];
      if (held < 0 || add < 0) err |= CSA2_DEVERR_N_VIS;
      held = held < 0 ? 0 : held;
      add = add < 0 ? 0 : add;
      const long long room = (long long)a.max_pages * kPage - held;
      if (add > room) {
        err |= CSA2_DEVERR_TOKENS;
        add = room < 0 ? 0 : room;
      }
    }
    long long total;
    const long long end = rows + block_scan(add, sums, &total);
    if (end > a.tokens && add > 0) err |= CSA2_DEVERR_TOKENS;
    const long long e = end < a.tokens ? end : a.tokens;
    const long long b = end - add < a.tokens ? end - add : a.tokens;
    rows += total;
    const long long now = held + (e - b);
    const int p0 = (int)((held + kPage - 1) / kPage), p1 = (int)((now + kPage - 1) / kPage);
    const int need = s < a.S ? p1 - p0 : 0;
    const long long pe = block_scan(need, sums, &total);
    if (s < a.S) {
      a.start[s + 1] = (int)e;
      a.new_length[s] = (int)now;
    }
    first_page[threadIdx.x] = p0;
    pages_before[threadIdx.x + 1] = (int)pe;
    if (threadIdx.x == 0) pages_before[0] = 0;
    __syncthreads();
    for (long long i = threadIdx.x; i < total; i += kPlanThreads) {
      int lo = 0, hi = kPlanThreads;     // pages_before[lo] <= i < pages_before[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pages_before[mid] <= i) lo = mid; else hi = mid;
      }
      const long long at = head + pages + i;
      int page = -1;
      if (at >= 0 && at < a.num_free) page = a.free_pages[at];
      else err |= CSA2_DEVERR_NO_PAGE;
      a.page_table[(long long)(s0 + lo) * a.max_pages + first_page[lo] + (i - pages_before[lo])] = page;
    }
    pages += total;
  }
  if (threadIdx.x == 0) {
    const long long h = head + pages;
    a.new_head[0] = (int)(h < a.num_free ? h : (a.num_free > head ? a.num_free : head));
  }
  if (err) raise_error(&g_err_paged, err);
}

// A thread a row.
__global__ void __launch_bounds__(256) k_plan_rows(const csa2_page_plan_args a) {
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= a.tokens) return;
  const int s = find_seq(a.start, a.S, t);
  int pos = -1, slot = -1;
  if (s >= 0) {
    pos = a.new_length[s] - (a.start[s + 1] - t);
    const int page = a.page_table[(long long)s * a.max_pages + pos / kPage];
    if (page >= 0) slot = page * kPage + pos % kPage;
  }
  a.seq[t] = s;
  a.pos[t] = pos;
  a.slot[t] = slot;
}

// ---- csa2_kv8_append ------------------------------------------------------------------------

// The least 2^e, e >= -126, with a <= 448 * 2^e (a >= 0, finite): 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_for(float a) {
  const uint32_t u = __float_as_uint(a);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < -126 ? -126 : e;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

constexpr int kAppendThreads = 256;      // half of them for the keys, half for the values

struct AppendParams {
  csa2_kv8_append_args a;
  int range;                             // rows whose pages one CTA sees to
};

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
  if constexpr (sizeof(T) == 2) return bf16_bits_to_f32(x);
  else return x;
}

template <typename T, int D, bool VEC>
__device__ __forceinline__ void load8(const T* p, float* f) {
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_f32(p[i]);
  } else if constexpr (sizeof(T) == 2) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(v[i] << 16);
      f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  } else {
    const float4 w = reinterpret_cast<const float4*>(p)[0], z = reinterpret_cast<const float4*>(p)[1];
    f[0] = w.x; f[1] = w.y; f[2] = w.z; f[3] = w.w;
    f[4] = z.x; f[5] = z.y; f[6] = z.z; f[7] = z.w;
  }
}

// A CTA a (range of rows, head): the pages whose first new token lies in the range, one after the other.
template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(kAppendThreads) k_kv8_append(const AppendParams p) {
  constexpr int kHalf = kAppendThreads / 2, kPer = D / 8, kRows = kHalf / kPer;   // threads a row, rows a turn
  __shared__ float s_max[kAppendThreads / 32], s_sum[kHalf / kPer][D], s_top[4];
  const csa2_kv8_append_args& a = p.a;
  const csa2_kv8_cache& c = a.cache;
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.y, half = threadIdx.x >= kHalf, tid = threadIdx.x - half * kHalf;
  const int row0 = tid / kPer, ch = tid % kPer * 8;
  const long long st = half ? a.v_stride_t : a.k_stride_t, sh = half ? a.v_stride_h : a.k_stride_h;
  const T* x = reinterpret_cast<const T*>(half ? a.v : a.k) + h * sh + ch;
  int t = blockIdx.x * p.range;
  const int t_end = min(a.T, t + p.range);
  while (t < t_end) {
    const int s = find_seq(a.start, a.S, t);
    if (s < 0) {                         // padding: before the first row, or to the end
      if (t >= a.start[a.S]) return;
      t = a.start[0];
      continue;
    }
    const int begin = a.start[s], end = min(a.start[s + 1], a.T);
    const int pos = row_pos(c, a.start, a.length, s, t, &g_err_paged);
    if (pos < 0) {
      ++t;
      continue;
    }
    const int held = pos & (kPage - 1), n = min(kPage - held, end - t);
    if (t != begin && held) {            // the page of an earlier row
      t += n;
      continue;
    }
    const int page = page_id(c, s, pos >> kPageShift, &g_err_paged);
    if (page < 0) {
      t += n;
      continue;
    }
    const long long ph = (long long)page * c.Hkv + h;
    float* scale_at = (half ? c.v_scale : c.k_scale) + ph;
    uint8_t* bytes = (half ? c.v : c.k) + ph * (kPage * D);
    const float was = held ? *scale_at : 0.f;
    float top = 0.f;
    for (int r = row0; r < n; r += kRows) {
      float f[8];
      load8<T, D, VEC>(x + (t + r) * st, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float m = fabsf(f[i]);
        if (m <= 3.402823466e38f) top = fmaxf(top, m);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHalf / 32; ++i) top = fmaxf(top, s_max[half * (kHalf / 32) + i]);
    const float scale = fmaxf(scale_for(top), was);
    if (held && scale > was) {
      const float ratio = __fdiv_rn(was, scale);
      for (int i = tid; i < held * D / 4; i += kHalf) {
        uint32_t* w = reinterpret_cast<uint32_t*>(bytes) + i;
        float f[4];
        e4m3x4_to_f32(*w, f);
        *w = cvt_e4m3x2(f[0] * ratio, f[1] * ratio) | cvt_e4m3x2(f[2] * ratio, f[3] * ratio) << 16;
      }
    }
    const float inv = __fdiv_rn(1.f, scale);                 // a power of two: exact
    for (int r = row0; r < n; r += kRows) {
      float f[8];
      load8<T, D, VEC>(x + (t + r) * st, f);
      uint2 w;
      w.x = cvt_e4m3x2(f[0] * inv, f[1] * inv) | cvt_e4m3x2(f[2] * inv, f[3] * inv) << 16;
      w.y = cvt_e4m3x2(f[4] * inv, f[5] * inv) | cvt_e4m3x2(f[6] * inv, f[7] * inv) << 16;
      *reinterpret_cast<uint2*>(bytes + (held + r) * D + ch) = w;
    }
    __syncthreads();                                         // the page's bytes are written, s_max is read
    if (tid == 0) *scale_at = scale;
    if (c.mean && held + n == kPage) {
      if (!half) {
        float m[8] = {};
        for (int r = row0; r < kPage; r += kRows) {
          const uint2 w = *reinterpret_cast<const uint2*>(bytes + r * D + ch);
          float f[8];
          e4m3x4_to_f32(w.x, f);
          e4m3x4_to_f32(w.y, f + 4);
#pragma unroll
          for (int i = 0; i < 8; ++i) m[i] += f[i] == f[i] ? f[i] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s_sum[row0][ch + i] = m[i];
      }
      __syncthreads();
      float m = 0.f;
      if (threadIdx.x < D) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) m += s_sum[r][threadIdx.x];
        float u = fabsf(m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, o));
        if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = u;
      }
      __syncthreads();
      if (threadIdx.x < D) {
        float u = s_top[0];
#pragma unroll
        for (int i = 1; i < D / 32; ++i) u = fmaxf(u, s_top[i]);
        u = __fdiv_rn(u, 127.f);
        c.mean[ph * D + threadIdx.x] = (int8_t)(u > 0.f ? __float2int_rn(__fdiv_rn(m, u)) : 0);
        if (threadIdx.x == 0) c.mean_scale[ph] = u * 0.015625f * scale;
      }
      __syncthreads();                                       // the sums are read before the next page's
    }
    t += n;
  }
}

// ---- csa2_kv8_select ------------------------------------------------------------------------

constexpr int kSelectThreads = 256;

// A CTA a (row, key head): scores as ordered keys in shared memory, the k-th by four 8-bit digits, the kept pages in
// ascending order.
template <int D>
__global__ void __launch_bounds__(kSelectThreads) k_kv8_select(const csa2_kv8_select_args a) {
  extern __shared__ uint32_t keys[];
  __shared__ int8_t r8[D];
  __shared__ float s_top[kSelectThreads / 32];
  __shared__ uint32_t hist[256];
  __shared__ long long sums[33];
  __shared__ uint32_t s_pick[2];
  const csa2_kv8_cache& c = a.cache;
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const int s = find_seq(a.start, a.S, t);
  if (s < 0) return;
  const long long row = (long long)t * c.Hkv + h;
  int* out = a.pages + row * a.k;
  int pos = row_pos(c, a.start, a.length, s, t, &g_err_paged);
  if (pos >= a.max_length) {
    if (tid == 0) raise_error(&g_err_paged, CSA2_DEVERR_N_VIS);
    pos = -1;
  }
  const int P = pos < 0 ? 0 : (pos >> kPageShift) + 1;
  if (P <= a.k) {
    for (int i = tid; i < a.k; i += kSelectThreads) out[i] = i < P ? i : -1;
    if (tid == 0) a.count[row] = P;
    return;
  }
  const int G = a.Hq / c.Hkv;
  float q = 0.f;
  if (tid < D) {
    double sum = 0.0;
    for (int g = 0; g < G; ++g)
      sum += (double)bf16_bits_to_f32(a.q[t * a.q_stride_t + (long long)(h * G + g) * a.q_stride_h + tid]);
    q = (float)sum;
  }
  float top = fabsf(q) <= 3.402823466e38f ? fabsf(q) : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) s_top[tid >> 5] = top;
  __syncthreads();
  if (tid < D) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) top = fmaxf(top, s_top[i]);
    const float u = __fdiv_rn(top, 127.f);
    float r = u > 0.f ? rintf(__fdiv_rn(q, u)) : 0.f;
    r = r != r ? 0.f : fminf(fmaxf(r, -127.f), 127.f);
    r8[tid] = (int8_t)r;
  }
  __syncthreads();
  const int lo = a.first, hi = P - a.recent, want = a.k - a.first - a.recent;
  for (int j = lo + tid; j < hi; j += kSelectThreads) {
    const int page = page_id(c, s, j, &g_err_paged);
    uint32_t key = 0;                                        // a page outside the cache comes last
    if (page >= 0) {
      const int* m = reinterpret_cast<const int*>(c.mean + ((long long)page * c.Hkv + h) * D);
      int dot = 0;
      for (int i = 0; i < D / 4; ++i) dot = __dp4a(m[i], reinterpret_cast<const int*>(r8)[i], dot);
      key = float_key(__fmul_rn((float)dot, c.mean_scale[(long long)page * c.Hkv + h]));
    }
    keys[j - lo] = key;
  }
  const int M = hi - lo;
  uint32_t prefix = 0;
  int left = want;                                           // still to take among the keys with this prefix
  for (int shift = 24; shift >= 0 && left > 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
    for (int i = tid; i < M; i += kSelectThreads)
      if ((keys[i] & mask) == prefix) atomicAdd(&hist[keys[i] >> shift & 255], 1u);
    __syncthreads();
    if (tid == 0) {
      int n = 0, d = 255;
      while (d > 0 && n + (int)hist[d] < left) n += hist[d--];
      s_pick[0] = prefix | (uint32_t)d << shift;
      s_pick[1] = left - n;
    }
    __syncthreads();
    prefix = s_pick[0];
    left = s_pick[1];
  }
  // above the threshold all, of those equal to it the first `left`
  for (int i = tid; i < a.first; i += kSelectThreads) out[i] = i;
  for (int i = tid; i < a.recent; i += kSelectThreads) out[a.k - a.recent + i] = hi + i;
  if (tid == 0) a.count[row] = a.k;
  if (want == 0) return;
  long long above = 0, equal = 0;
  for (int i0 = 0; i0 < M; i0 += kSelectThreads) {
    const int i = i0 + tid;
    const bool g = i < M && keys[i] > prefix, e = i < M && keys[i] == prefix;
    long long total;
    const long long in = block_scan((long long)g << 32 | (long long)e, sums, &total);
    const long long ga = above + (in >> 32) - g, ea = equal + (in & 0xffffffff) - e;   // before this page
    if (g || (e && ea < left)) out[a.first + ga + (ea < left ? ea : left)] = lo + i;
    above += total >> 32;
    equal += total & 0xffffffff;
  }
}

}  // namespace

cudaError_t launch_page_plan(const csa2_page_plan_args& a, cudaStream_t st) {
  cudaError_t e = launch_k(k_plan_scan, dim3(1), dim3(kPlanThreads), 0, st, a);
  if (e != cudaSuccess || a.tokens == 0) return e;
  return launch_k(k_plan_rows, dim3((a.tokens + 255) / 256), dim3(256), 0, st, a);
}

cudaError_t launch_kv8_append(const csa2_kv8_append_args& a, cudaStream_t st) {
  if (a.T == 0 || a.S == 0) return cudaSuccess;
  AppendParams p;
  p.a = a;
  const long long tasks = (long long)a.T * a.cache.Hkv;
  p.range = (int)(tasks / 2432 < 1 ? 1 : tasks / 2432 > 64 ? 64 : tasks / 2432);
  const dim3 grid((a.T + p.range - 1) / p.range, a.cache.Hkv);
  const size_t unit = a.x_dtype == CSA2_BF16 ? 2 : 4;
  auto rows = [&](const void* x, int64_t t, int64_t h) {
    return (((uintptr_t)x | (uintptr_t)(t * unit) | (uintptr_t)(h * unit)) & 15) == 0;
  };
  const bool vec = rows(a.k, a.k_stride_t, a.k_stride_h) && rows(a.v, a.v_stride_t, a.v_stride_h);
  auto go = [&](auto* kernel) { return launch_k(kernel, grid, dim3(kAppendThreads), 0, st, p); };
  if (a.x_dtype == CSA2_BF16) {
    if (a.cache.D == 64) return vec ? go(k_kv8_append<uint16_t, 64, true>) : go(k_kv8_append<uint16_t, 64, false>);
    return vec ? go(k_kv8_append<uint16_t, 128, true>) : go(k_kv8_append<uint16_t, 128, false>);
  }
  if (a.cache.D == 64) return vec ? go(k_kv8_append<float, 64, true>) : go(k_kv8_append<float, 64, false>);
  return vec ? go(k_kv8_append<float, 128, true>) : go(k_kv8_append<float, 128, false>);
}

size_t kv8_select_workspace_bytes(const csa2_kv8_select_args&) { return 0; }

cudaError_t launch_kv8_select(const csa2_kv8_select_args& a, void*, cudaStream_t st) {
  if (a.T == 0 || a.S == 0) return cudaSuccess;
  const size_t smem = 4 * (size_t)((a.max_length + kPage - 1) / kPage);
  static SmemLimit limit64, limit128;
  cudaError_t e;
  if (a.cache.D == 64) {
    if ((e = limit64.raise(k_kv8_select<64>, smem)) != cudaSuccess) return e;
    return launch_k(k_kv8_select<64>, dim3(a.T, a.cache.Hkv), dim3(kSelectThreads), smem, st, a);
  }
  if ((e = limit128.raise(k_kv8_select<128>, smem)) != cudaSuccess) return e;
  return launch_k(k_kv8_select<128>, dim3(a.T, a.cache.Hkv), dim3(kSelectThreads), smem, st, a);
}

uint32_t read_clear_error_paged() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_err_paged, sizeof(v));
  if (v) cudaMemcpyToSymbol(g_err_paged, &z, sizeof(z));
  return v;
}

}  // namespace csa2

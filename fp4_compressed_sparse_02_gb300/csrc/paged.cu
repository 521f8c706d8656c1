// The paged 8-bit cache's tables, append and page selection (csa2_page_plan, csa2_kv8_append,
// csa2_kv8_select).
#include <limits.h>
#include <math.h>

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

// What a sequence holds and gets before rows run out: (held, add), with error bits.
__device__ __forceinline__ void plan_counts(const csa2_page_plan_args& a, int s, long long& held, long long& add, unsigned int& err) {
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

// Up to 1024 sequences, a thread a sequence: every CTA has both prefix sums (rows, pages) in shared memory and sees to its
// share of the rows and of the new pages.  CTA 0 writes the sequences' values; where those are the inputs themselves,
// it is the only one.  Bound by the launch and by two rounds of dependent loads: 4.1 us for 64 rows, 8.5 us for 262,144
// (3.1 MB).  As two kernels, one CTA's sums and then the rows, those took 8 and 14 us of a graph.
__global__ void __launch_bounds__(kPlanThreads) k_plan(const csa2_page_plan_args a, int rows) {
  __shared__ long long sums[33];
  __shared__ int start[kPlanThreads + 1], now[kPlanThreads], old_pages[kPlanThreads], pages_before[kPlanThreads + 1];
  pdl_wait();
  pdl_trigger();
  const int s = threadIdx.x;
  const int head = a.free_head[0];
  unsigned int err = 0;
  long long held = 0, add = 0, total;
  if (s < a.S) plan_counts(a, s, held, add, err);
  const long long end = block_scan(add, sums, &total);
  if (end > a.tokens && add > 0) err |= CSA2_DEVERR_TOKENS;
  const int e = (int)(end < a.tokens ? end : a.tokens), b = (int)(end - add < a.tokens ? end - add : a.tokens);
  const long long len = held + (e - b);
  const int p0 = (int)((held + kPage - 1) / kPage), p1 = (int)((len + kPage - 1) / kPage);
  const long long pe = block_scan(p1 - p0, sums, &total);
  start[s + 1] = e;
  now[s] = (int)len;
  old_pages[s] = p0;
  pages_before[s + 1] = (int)pe;
  if (s == 0) start[0] = pages_before[0] = 0;
  __syncthreads();                       // and every input of this CTA has been read
  if (blockIdx.x == 0) {
    if (s < a.S) {
      a.start[s + 1] = e;
      a.new_length[s] = (int)len;
    }
    if (s == 0) {
      const long long h = head + total;
      a.start[0] = 0;
      a.new_head[0] = (int)(h < a.num_free ? h : (a.num_free > head ? a.num_free : head));
    }
  }
  auto taken = [&](long long i) {        // the i-th page of this call, -1 if there is none
    const long long at = head + i;
    return at >= 0 && at < a.num_free ? a.free_pages[at] : -1;
  };
  auto find = [&](const int* before, int x) {                // before[lo] <= x < before[hi]
    int lo = 0, hi = a.S;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
  };
  for (long long i = (long long)blockIdx.x * kPlanThreads + s; i < total; i += (long long)gridDim.x * kPlanThreads) {
    const int q = find(pages_before, (int)i), page = taken(i);
    if (head + i < 0 || head + i >= a.num_free) err |= CSA2_DEVERR_NO_PAGE;
    a.page_table[(long long)q * a.max_pages + old_pages[q] + (i - pages_before[q])] = page;
  }
  const int t0 = blockIdx.x * rows, t1 = min(a.tokens, t0 + rows), last = start[a.S];
  for (int t = t0 + s; t < t1; t += kPlanThreads) {
    int q = -1, pos = -1, slot = -1;
    if (t < last) {
      q = find(start, t);
      pos = now[q] - (start[q + 1] - t);
      const int j = pos / kPage;
      const int page = j >= old_pages[q] ? taken(pages_before[q] + (j - old_pages[q])) : a.page_table[(long long)q * a.max_pages + j];
      if (page >= 0) slot = page * kPage + pos % kPage;
    }
    a.seq[t] = q;
    a.pos[t] = pos;
    a.slot[t] = slot;
  }
  if (err) raise_error(&g_err_paged, err);
}

// More sequences than that, or many rows in place.  One CTA: the two prefix sums (rows, pages) over the sequences, 1024 at a time, and the new entries of the page table.
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
      plan_counts(a, s, held, add, err);
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

// The rows after it, a thread a row.
__global__ void __launch_bounds__(256) k_plan_rows(const csa2_page_plan_args a) {
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= a.tokens) return;
  int s = -1, pos = -1, slot = -1;
  if (t < a.start[a.S]) {
    s = 0;
    for (int hi = a.S; hi - s > 1;) {
      const int mid = (s + hi) >> 1;
      if (a.start[mid] <= t) s = mid; else hi = mid;
    }
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

constexpr int kAppendThreads = 128;

struct AppendParams {
  csa2_kv8_append_args a;
  int range;                             // rows whose pages one CTA sees to
};

// Eight channels of a row as they come.
template <typename T>
struct Eight {
  uint4 w[sizeof(T) / 2];

  template <bool VEC>
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    } else if constexpr (sizeof(T) == 2) {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (uint32_t)p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
      w[0] = make_uint4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = make_uint4(__float_as_uint(p[4 * i]), __float_as_uint(p[4 * i + 1]), __float_as_uint(p[4 * i + 2]),
                          __float_as_uint(p[4 * i + 3]));
    }
  }
  // The larger of `top` and the largest magnitude; NaNs count as nothing.  bf16 two at a time.
  __device__ __forceinline__ float largest(float top) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
      __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v[0]));
#pragma unroll
      for (int i = 1; i < 4; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v[i])));
      return fmaxf(top, fmaxf(__bfloat162float(m.x), __bfloat162float(m.y)));
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        top = fmaxf(fmaxf(fmaxf(top, fabsf(__uint_as_float(w[i].x))), fabsf(__uint_as_float(w[i].y))),
                    fmaxf(fabsf(__uint_as_float(w[i].z)), fabsf(__uint_as_float(w[i].w))));
      return top;
    }
  }
  __device__ __forceinline__ void values(float* f) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(w[i].x);
        f[4 * i + 1] = __uint_as_float(w[i].y);
        f[4 * i + 2] = __uint_as_float(w[i].z);
        f[4 * i + 3] = __uint_as_float(w[i].w);
      }
    }
  }
};

__device__ __forceinline__ void add_bytes(float2* m, uint2 w) {            // a NaN counts as 0
  const uint32_t nx = e4m3x4_nans(w.x), ny = e4m3x4_nans(w.y);
  if (nx | ny) {
    w.x &= ~(nx * 0xffu);
    w.y &= ~(ny * 0xffu);
  }
  const uint32_t h[4] = {e4m3x2_lo_f16x2(w.x), e4m3x2_hi_f16x2(w.x), e4m3x2_lo_f16x2(w.y), e4m3x2_hi_f16x2(w.y)};
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = add2(m[i], __half22float2(*reinterpret_cast<const __half2*>(&h[i])));
}

// A CTA a (range of rows, head, plane): the pages whose first new token lies in the range, one after the other.  A page's new
// rows are loaded at once and stay in registers from the largest magnitude to the summary.  38K rows of 8 x 128 in bf16
// (234 MB): 46 us, 0.75 of the copy rate, of which loading alone fills a part: a CTA's barriers stand between its
// loads and its stores, and eight CTAs an SM overlap them.  Keys and values in one CTA of 256 threads: 56 us.  The same
// rows in float32 (390 MB), four CTAs an SM: 75 us from a cold L2, 0.77, where bf16 takes 52.
template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(kAppendThreads, sizeof(T) == 2 ? 8 : 4) k_kv8_append(const AppendParams p) {
  constexpr int kPer = D / 8, kRows = kAppendThreads / kPer, kTurns = kPage / kRows;   // threads a row, rows a turn
  __shared__ float s_max[kAppendThreads / 32], s_sum[kRows][D], s_top[4];
  const csa2_kv8_append_args& a = p.a;
  const csa2_kv8_cache& c = a.cache;
  pdl_wait();
  pdl_trigger();
  const int plane = blockIdx.x & 1, h = blockIdx.x / 2 % c.Hkv, tid = threadIdx.x;   // 0: keys, 1: values
  const int row0 = tid / kPer, ch = tid % kPer * 8;
  const long long st = plane ? a.v_stride_t : a.k_stride_t, sh = plane ? a.v_stride_h : a.k_stride_h;
  const T* x = reinterpret_cast<const T*>(plane ? a.v : a.k) + h * sh + ch;
  int t = blockIdx.x / 2 / c.Hkv * p.range;
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
    Eight<T> rows[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i)
      if (row0 + i * kRows < n) rows[i].template load<VEC>(x + (t + row0 + i * kRows) * st);
    const int page = page_id(c, s, pos >> kPageShift, &g_err_paged);
    if (page < 0) {
      t += n;
      continue;
    }
    const long long ph = (long long)page * c.Hkv + h;
    float* scale_at = (plane ? c.v_scale : c.k_scale) + ph;
    uint8_t* bytes = (plane ? c.v : c.k) + ph * (kPage * D);
    const float was = held ? *scale_at : 0.f;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < kTurns; ++i)
      if (row0 + i * kRows < n) top = rows[i].largest(top);
    if (top == INFINITY) {               // infinities do not take part
      top = 0.f;
#pragma unroll
      for (int i = 0; i < kTurns; ++i)
        if (row0 + i * kRows < n) {
          float f[8];
          rows[i].values(f);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (fabsf(f[e]) < INFINITY) top = fmaxf(top, fabsf(f[e]));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 31) == 0) s_max[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAppendThreads / 32; ++i) top = fmaxf(top, s_max[i]);
    const float scale = fmaxf(scale_for(top), was);
    if (held && scale > was) {
      const float ratio = __fdiv_rn(was, scale);
      for (int i = tid; i < held * D / 4; i += kAppendThreads) {
        uint32_t* w = reinterpret_cast<uint32_t*>(bytes) + i;
        float f[4];
        e4m3x4_to_f32(*w, f);
        *w = cvt_e4m3x2(f[0] * ratio, f[1] * ratio) | cvt_e4m3x2(f[2] * ratio, f[3] * ratio) << 16;
      }
    }
    const bool full = c.mean && !plane && held + n == kPage;
    const float inv = __fdiv_rn(1.f, scale);                 // a power of two: exact
    float2 m[4] = {};
#pragma unroll
    for (int i = 0; i < kTurns; ++i)
      if (row0 + i * kRows < n) {
        float f[8];
        rows[i].values(f);
        uint32_t e[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const float2 y = mul2(make_float2(f[2 * d], f[2 * d + 1]), make_float2(inv, inv));
          e[d] = cvt_e4m3x2(y.x, y.y);
        }
        const uint2 w = make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
        *reinterpret_cast<uint2*>(bytes + (held + row0 + i * kRows) * D + ch) = w;
        if (full) add_bytes(m, w);
      }
    __syncthreads();                                         // old bytes are as they stay, s_max is read
    if (tid == 0) *scale_at = scale;
    if (full) {
      for (int r = row0; r < held; r += kRows) add_bytes(m, *reinterpret_cast<const uint2*>(bytes + r * D + ch));
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(&s_sum[row0][ch + 2 * i]) = m[i];
      __syncthreads();
      float sum = 0.f;
      if (threadIdx.x < D) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) sum += s_sum[r][threadIdx.x];
        float u = fabsf(sum);
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
        c.mean[ph * D + threadIdx.x] = (int8_t)(u > 0.f ? __float2int_rn(__fdiv_rn(sum, u)) : 0);
        if (threadIdx.x == 0) c.mean_scale[ph] = u * 0.015625f * scale;
      }
      __syncthreads();                                       // the sums are read before the next page's
    }
    t += n;
  }
}

// ---- csa2_kv8_select ------------------------------------------------------------------------
//
// Scores, then picks.  The scores of up to 8 rows of one sequence and key head are one product of their 8-bit queries
// with the pages' 8-bit summaries: whole numbers up to 127 are exact in fp16 and their sums of 128 products
// stay below 2^24, so mma.sync gives the exact dot products whatever its order.  Bound by memory latency: 512 summaries a
// CTA, 128 a warp in four rounds (32 rows at up to 128K: 16 us for 45 MB); eight rows share what they read (2048 rows: 38 us).
constexpr int kTile = 8, kScoreThreads = 128, kScorePages = 512;

struct SelectParams {
  csa2_kv8_select_args a;
  int G, aligned;                        // aligned: q's rows on 8 bytes
  int t0, t1;                            // rows of this launch
  int stride;                            // keys of a (row, head)
  uint32_t* keys;                        // [t1 - t0][Hkv][stride], by page: larger = better
};

// Four signed bytes as two fp16 pairs: (byte ^ 0x80) under 0x64 is 1024 + 128 + byte.
__device__ __forceinline__ void s8x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t x = w ^ 0x80808080u;
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));                 // 1152
  uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
  const __half2 u = __hsub2(*reinterpret_cast<__half2*>(&a), bias), v = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&u);
  hi = *reinterpret_cast<const uint32_t*>(&v);
}

// The 8-bit query of row t and head h, spread over a warp (D / 32 channels a lane), as packed bytes.  The heads' sum is
// carried with its rounding errors, so that it is rounded once.
template <int D>
__device__ __forceinline__ uint32_t query8(const SelectParams& p, int t, int h, int lane) {
  constexpr int kPer = D / 32;
  const csa2_kv8_select_args& a = p.a;
  const uint16_t* q = a.q + t * a.q_stride_t + (long long)h * p.G * a.q_stride_h + lane * kPer;
  float s[kPer] = {}, err[kPer] = {};
#pragma unroll 8
  for (int g = 0; g < p.G; ++g) {
    const uint16_t* row = q + g * a.q_stride_h;
    float x[kPer];
    if (p.aligned) {
      uint32_t w[kPer / 2];
      if constexpr (kPer == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(row);
        w[0] = v.x;
        w[1] = v.y;
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(row);
      }
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) x[i] = bf16_bits_to_f32(row[i]);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float n = __fadd_rn(s[i], x[i]), b = __fsub_rn(n, s[i]);
      err[i] = __fadd_rn(err[i], __fadd_rn(__fsub_rn(s[i], __fsub_rn(n, b)), __fsub_rn(x[i], b)));
      s[i] = n;
    }
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const bool finite = fabsf(s[i]) <= 3.402823466e38f;
    if (finite) s[i] = __fadd_rn(s[i], err[i]);
    if (fabsf(s[i]) <= 3.402823466e38f) top = fmaxf(top, fabsf(s[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float u = __fdiv_rn(top, 127.f);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    float r = u > 0.f ? rintf(__fdiv_rn(s[i], u)) : 0.f;
    r = r != r ? 0.f : fminf(fmaxf(r, -127.f), 127.f);
    w |= ((uint32_t)(int)r & 0xffu) << 8 * i;
  }
  return w;
}

// A CTA (tile of 8 rows of one sequence, 512 pages, head); a warp 128 pages, 32 at a time.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) k_kv8_score(const SelectParams p) {
  constexpr int kKs = D / 16, kW = D / 64;                   // products a tile, 16-byte words of a lane's quarter row
  __shared__ uint32_t r8[kTile][D / 4];
  const csa2_kv8_select_args& a = p.a;
  const csa2_kv8_cache& c = a.cache;
  pdl_wait();
  pdl_trigger();
  // Slot floor(start / 8) + s and the ones after it hold the tiles of sequence s (starts within this launch's rows).
  auto begin = [&](int s) {
    const int x = a.start[s];
    return x < p.t0 ? p.t0 : x > p.t1 ? p.t1 : x;
  };
  int s = 0, hi = a.S;
  const int slot = blockIdx.x, h = blockIdx.z, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  while (hi - s > 1) {
    const int mid = (s + hi) >> 1;
    if ((begin(mid) - p.t0) / kTile + mid <= slot) s = mid; else hi = mid;
  }
  const int b = begin(s), t = b + (slot - (b - p.t0) / kTile - s) * kTile, n = min(kTile, begin(s + 1) - t);
  if (t < b || n <= 0) return;
  const long long last = (long long)a.length[s] - ((long long)a.start[s + 1] - (t + n - 1));
  if (last < 0) return;
  const long long most = last / kPage + 1;
  const int P = (int)(most < p.stride ? most : p.stride), end = (P < c.max_pages ? P : c.max_pages) - a.recent;
  const int first = a.first + blockIdx.y * kScorePages;
  if (most <= a.k || first >= end) return;
  for (int i = warp; i < n; i += kScoreThreads / 32) {
    const uint32_t w = query8<D>(p, t + i, h, lane);
    if constexpr (D == 128) r8[i][lane] = w;
    else reinterpret_cast<uint16_t*>(r8[i])[lane] = (uint16_t)w;
  }
  __syncthreads();
  const int g = lane >> 2, q4 = lane & 3;
  uint32_t qb[kKs][2];
#pragma unroll
  for (int j = 0; j < kKs; ++j) s8x4_to_f16(g < n ? r8[g][q4 * kKs + j] : 0u, qb[j][0], qb[j][1]);
  const int stop = min(end, first + kScorePages);
  for (int j0 = first + warp * 32; j0 < stop; j0 += kScoreThreads) {
    const int j = j0 + lane, page = j < stop ? page_id(c, s, j, &g_err_paged) : -1;
    const float scale = page >= 0 ? c.mean_scale[(long long)page * c.Hkv + h] : 0.f;
    uint4 w[4][kW];                      // summaries of pages j0 + 8 i + g, channels D/4 * q4 ...
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = __shfl_sync(0xffffffffu, page, 8 * i + g);
      const uint4* m = reinterpret_cast<const uint4*>(c.mean + ((long long)(id < 0 ? 0 : id) * c.Hkv + h) * D + q4 * (D / 4));
#pragma unroll
      for (int e = 0; e < kW; ++e) w[i][e] = m[e];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < kW; ++e) {
        const uint32_t x[4] = {w[2 * i][e].x, w[2 * i][e].y, w[2 * i][e].z, w[2 * i][e].w};
        const uint32_t y[4] = {w[2 * i + 1][e].x, w[2 * i + 1][e].y, w[2 * i + 1][e].z, w[2 * i + 1][e].w};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint32_t a0, a1, a2, a3;
          s8x4_to_f16(x[v], a0, a2);
          s8x4_to_f16(y[v], a1, a3);
          mma_f16_16816(d, a0, a1, a2, a3, qb[4 * e + v][0], qb[4 * e + v][1]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at = 16 * i + 8 * (e >> 1) + g, row = 2 * q4 + (e & 1);
        const float f = __shfl_sync(0xffffffffu, scale, at);
        const int id = __shfl_sync(0xffffffffu, page, at);
        // a page outside the cache comes last
        if (row < n && j0 + at < stop)
          p.keys[((long long)(t + row - p.t0) * c.Hkv + h) * p.stride + j0 + at] = id < 0 ? 0u : float_key(__fmul_rn(d[e], f));
      }
    }
  }
}

// Rows with at most 32 K pages, a warp a (row, head): lane l holds keys l, l + 32, ...; the k-th best bit by bit, by
// ballots.  16,384 pairs of 512 pages: 33 us, where a CTA a pair took 113; 66 keys a lane, for 2048 pages, 17 us against 10.
template <int K>
__global__ void __launch_bounds__(256) k_kv8_pick_warp(const SelectParams p) {
  const csa2_kv8_select_args& a = p.a;
  const csa2_kv8_cache& c = a.cache;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, i = blockIdx.x * 8 + (threadIdx.x >> 5), t = p.t0 + i / c.Hkv, h = i % c.Hkv;
  if (t >= p.t1) return;
  const int s = find_seq(a.start, a.S, t);
  if (s < 0) return;
  const long long row = (long long)t * c.Hkv + h;
  int* out = a.pages + row * a.k;
  int pos = row_pos(c, a.start, a.length, s, t, &g_err_paged);
  if (pos >= a.max_length) {
    if (lane == 0) raise_error(&g_err_paged, CSA2_DEVERR_N_VIS);
    pos = -1;
  }
  const int P = pos < 0 ? 0 : (pos >> kPageShift) + 1;
  if (P <= a.k) {
    for (int j = lane; j < a.k; j += 32) out[j] = j < P ? j : -1;
    if (lane == 0) a.count[row] = P;
    return;
  }
  const int lo = a.first, hi = P - a.recent, M = hi - lo, want = a.k - a.first - a.recent;
  for (int j = lane; j < a.first; j += 32) out[j] = j;
  for (int j = lane; j < a.recent; j += 32) out[a.k - a.recent + j] = hi + j;
  if (lane == 0) a.count[row] = a.k;
  if (want == 0) return;
  const uint32_t* src = p.keys + ((long long)(t - p.t0) * c.Hkv + h) * p.stride + lo;
  uint32_t key[K];
#pragma unroll
  for (int j = 0; j < K; ++j) key[j] = j * 32 + lane < M ? src[j * 32 + lane] : 0u;
  // the largest threshold that at least `want` keys reach; keys of bad pages are 0, and M > want keys reach that
  uint32_t least = 0;
  for (uint32_t bit = 1u << 31; bit; bit >>= 1) {
    const uint32_t at = least | bit;
    int n = 0;
#pragma unroll
    for (int j = 0; j < K; ++j) n += key[j] >= at;
    n = __reduce_add_sync(0xffffffffu, n);
    if (n >= want) least = at;
    if (n == want) break;                                    // exactly those
  }
  int above = 0;
#pragma unroll
  for (int j = 0; j < K; ++j) above += key[j] > least;
  int left = want - __reduce_add_sync(0xffffffffu, above);   // to take of those equal to it, from the first on
  const uint32_t under = (1u << lane) - 1;
  int at = a.first;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const bool in = j * 32 + lane < M;
    const uint32_t equal = __ballot_sync(0xffffffffu, in && key[j] == least);
    const bool take = in && (key[j] > least || (key[j] == least && __popc(equal & under) < left));
    const uint32_t taken = __ballot_sync(0xffffffffu, take);
    if (take) out[at + __popc(taken & under)] = lo + j * 32 + lane;
    at += __popc(taken);
    left = max(0, left - __popc(equal));
  }
}

// A CTA a (row, head): the k-th best key by digits of 11, 11 and 10 bits, then the kept pages in ascending order.  10 us for 256
// pairs of up to 2048 pages, 13 for 8 of 16,384.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) k_kv8_pick(const SelectParams p) {
  constexpr int kBins = 2048, kPerThread = kBins / THREADS, kPickWarps = THREADS / 32;
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[kBins];
  __shared__ int s_warp[2][kPickWarps + 1], s_pick[2];
  const csa2_kv8_select_args& a = p.a;
  const csa2_kv8_cache& c = a.cache;
  pdl_wait();
  pdl_trigger();
  const int t = p.t0 + blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
    for (int i = tid; i < a.k; i += THREADS) out[i] = i < P ? i : -1;
    if (tid == 0) a.count[row] = P;
    return;
  }
  const int lo = a.first, hi = P - a.recent, M = hi - lo, want = a.k - a.first - a.recent;
  for (int i = tid; i < a.first; i += THREADS) out[i] = i;
  for (int i = tid; i < a.recent; i += THREADS) out[a.k - a.recent + i] = hi + i;
  if (tid == 0) a.count[row] = a.k;
  if (want == 0) return;
  const uint32_t* src = p.keys + ((long long)(t - p.t0) * c.Hkv + h) * p.stride + lo;
  for (int i = tid; i < M; i += THREADS) keys[i] = src[i];
  for (int i = tid; i < kBins; i += THREADS) hist[i] = 0;
  __syncthreads();
  uint32_t prefix = 0, mask = 0;
  int left = want;                                           // still to take among the keys with this prefix
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit = pass == 2 ? 1023u : 2047u;
    for (int i = tid; i < M; i += THREADS)
      if ((keys[i] & mask) == prefix) atomicAdd(&hist[keys[i] >> shift & digit], 1u);
    __syncthreads();
    // bins from the top: thread i has kPerThread of them, below those of threads before it
    int own[kPerThread], sum = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      own[i] = (int)hist[kBins - 1 - (tid * kPerThread + i)];
      sum += own[i];
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) s_warp[0][warp] = inc;
    __syncthreads();
    int before = inc - sum;
    for (int i = 0; i < warp; ++i) before += s_warp[0][i];
    if (before < left && before + sum >= left) {
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) {
        if (before < left && before + own[i] >= left) {
          s_pick[0] = kBins - 1 - (tid * kPerThread + i);
          s_pick[1] = left - before;
          break;
        }
        before += own[i];
      }
    }
    for (int i = tid; i < kBins; i += THREADS) hist[i] = 0;
    __syncthreads();
    prefix |= (uint32_t)s_pick[0] << shift;
    mask |= digit << shift;
    left = s_pick[1];
  }
  // above the threshold all, of those equal to it the first `left`; a warp has a run of the pages
  const int run = ((M + kPickWarps - 1) / kPickWarps + 31) & ~31, i0 = warp * run, i1 = min(M, i0 + run);
  int above = 0, equal = 0;
  for (int i = i0 + lane; i - lane < i1; i += 32) {
    above += __popc(__ballot_sync(0xffffffffu, i < i1 && keys[i] > prefix));
    equal += __popc(__ballot_sync(0xffffffffu, i < i1 && keys[i] == prefix));
  }
  if (lane == 0) {
    s_warp[0][warp] = above;
    s_warp[1][warp] = equal;
  }
  __syncthreads();
  above = equal = 0;
  for (int i = 0; i < warp; ++i) {
    above += s_warp[0][i];
    equal += s_warp[1][i];
  }
  for (int i = i0 + lane; i - lane < i1; i += 32) {
    const bool g = i < i1 && keys[i] > prefix, e = i < i1 && keys[i] == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, g), be = __ballot_sync(0xffffffffu, e), under = (1u << lane) - 1;
    const int ga = above + __popc(bg & under), ea = equal + __popc(be & under);
    if (g || (e && ea < left)) out[a.first + ga + min(ea, left)] = lo + i;
    above += __popc(bg);
    equal += __popc(be);
  }
}

// Rows of one launch: as many as keep their keys within 256 MB.
int select_stride(const csa2_kv8_select_args& a) { return (a.max_length + kPage - 1) / kPage; }
int select_rows(const csa2_kv8_select_args& a) {
  const long long row = (long long)a.cache.Hkv * (select_stride(a) > 0 ? select_stride(a) : 1);
  const long long n = (1LL << 26) / row;
  return (int)(n < 1 ? 1 : n < a.T ? n : a.T);
}

template <int D>
cudaError_t launch_select(SelectParams& p, cudaStream_t st) {
  static SmemLimit limit_many;
  const csa2_kv8_select_args& a = p.a;
  const int rows = select_rows(a);
  for (p.t0 = 0; p.t0 < a.T; p.t0 = p.t1) {
    p.t1 = a.T - p.t0 < rows ? a.T : p.t0 + rows;
    cudaError_t e = cudaSuccess;
    if (p.stride > a.k) {
      const dim3 grid((p.t1 - p.t0) / kTile + a.S, (p.stride + kScorePages - 1) / kScorePages, a.cache.Hkv);
      e = launch_k(k_kv8_score<D>, grid, dim3(kScoreThreads), 0, st, p);
      if (e != cudaSuccess) return e;
    }
    const size_t smem = 4 * (size_t)p.stride;
    const dim3 grid(p.t1 - p.t0, a.cache.Hkv);
    const dim3 warps((unsigned)(((long long)(p.t1 - p.t0) * a.cache.Hkv + 7) / 8));
    if (p.stride <= 256) {
      e = launch_k(k_kv8_pick_warp<8>, warps, dim3(256), 0, st, p);
    } else if (p.stride <= 640) {
      e = launch_k(k_kv8_pick_warp<20>, warps, dim3(256), 0, st, p);
    } else if (p.stride <= 1024) {
      e = launch_k(k_kv8_pick_warp<32>, warps, dim3(256), 0, st, p);
    } else if (p.stride <= 4096) {
      e = launch_k(k_kv8_pick<256>, grid, dim3(256), smem, st, p);
    } else {
      e = limit_many.raise(k_kv8_pick<1024>, smem);
      if (e == cudaSuccess) e = launch_k(k_kv8_pick<1024>, grid, dim3(1024), smem, st, p);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_page_plan(const csa2_page_plan_args& a, cudaStream_t st) {
  // In place one CTA writes all rows: 7 us for 8192, 149 us for 262,144 of 16 sequences.
  const bool in_place = a.new_length == a.length || a.new_head == a.free_head;
  if (a.S <= kPlanThreads && a.S > 0 && (!in_place || a.tokens <= 4096)) {
    const int most = in_place ? 1 : 152, rows = kPlanThreads * (int)(1 + (long long)(a.tokens - 1) / ((long long)most * kPlanThreads));
    return launch_k(k_plan, dim3(a.tokens > rows ? (a.tokens + rows - 1) / rows : 1), dim3(kPlanThreads), 0, st, a, rows);
  }
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
  const long long ctas = (long long)((a.T + p.range - 1) / p.range) * a.cache.Hkv * 2;   // a token's heads and planes side by side
  if (ctas > INT_MAX) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)ctas);
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

size_t kv8_select_workspace_bytes(const csa2_kv8_select_args& a) {
  return 4 * (size_t)select_rows(a) * a.cache.Hkv * select_stride(a);
}

cudaError_t launch_kv8_select(const csa2_kv8_select_args& a, void* ws, cudaStream_t st) {
  if (a.T == 0 || a.S == 0) return cudaSuccess;
  SelectParams p;
  p.a = a;
  p.G = a.Hq / a.cache.Hkv;
  p.aligned = (((uintptr_t)a.q | (uintptr_t)(2 * a.q_stride_t) | (uintptr_t)(2 * a.q_stride_h)) & 7) == 0;
  p.stride = select_stride(a);
  p.keys = static_cast<uint32_t*>(ws);
  return a.cache.D == 64 ? launch_select<64>(p, st) : launch_select<128>(p, st);
}

uint32_t read_clear_error_paged() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_err_paged, sizeof(v));
  if (v) cudaMemcpyToSymbol(g_err_paged, &z, sizeof(z));
  return v;
}

}  // namespace csa2

// Attention over the paged 8-bit cache (csa2_kv8_attn).
//
// Rows are (new token, query head of the group) pairs of one sequence and key head; a tile of rows
// against the tiles of its sequence's pages is one stream.  k_kv8_stream runs streams of at most 16 rows.
#include "kv8_attn.cuh"

namespace csa2 {

CSA2_DEFINE_ERROR_WORD(g_err_kv8);

namespace {

// ---- streams of at most 16 rows --------------------------------------------------------------
//
// Every warp is on its own: the half pages (32 tokens) of all streams, one stream after the other,
// are cut into equal spans, one for each warp, whatever the sequences' lengths are.  A stream cut by
// the border of a span leaves its parts (running maximum, sum, unnormalised output) in the
// workspace and k_kv8_join puts them together, in the order of the warps.
//
// A warp's half pages come by TMA into its own ring of 8 KB stages (keys, then values), swizzled so that
// the reads below meet no bank twice.  E4M3 bytes become fp16 pairs in registers (exact), products are
// mma.sync m16n8k16.  Tiles of 16 rows stand on M, with 8 tokens (scores) or 8 channels (values) on N; tiles of 8 rows
// stand on N, with 16 tokens or channels on M, which halves the products and asks for one 8 x 8 transpose of the weights
// for 8 tokens.  A lane's K fragment is 32 consecutive channels of one token (a permutation of the channels that Q's
// fragments share), its V fragment the bytes of two neighbouring tokens interleaved; at 16 rows the scores'
// accumulators are the weights' A fragments.  The scales stay out of fp16: a page's key scale multiplies its logits, its value scale
// its partial output, in float32.
//
// Bound by memory where a batch has the bytes (64 sequences of up to 64K tokens, 8 x 128 channels: 4.2 GB in 625-650 us,
// 0.95-0.98 of the copy rate); by a warp's own chain of products and conversions, three warps a scheduler, where pages come
// from L2 (2048 rows of 32 listed pages each: 0.88 ms for 8.6 GB, which the copies alone take 0.43 ms for); by two launches
// and four dependent loads where there is little (one row over 4097 tokens: 10 + 6 us).  Left out: E4M3 products by
// mma.sync (100 instructions more a half page than fp16 ones with their conversions: 1.17 ms); kLeast of 1 to 8 is all the
// same at one row.
constexpr int kWarps = 4, kLeast = 4, kHalf = kPage / 2;
// Weights are 2^15 times exp2(logit - maximum), so that fp16 reaches down to 2^-40 of the largest: a million tokens that are
// smaller than that count for nothing.  Without the factor it reaches 2^-25, and behind a token that leads by 17 nats all
// others were lost.
constexpr float kWeight = 15.f, kWeightUndo = 1.f / 32768.f;

// CTAs an SM.  Three, at 168 registers a thread and two stages a warp, where 8 rows have lists and pages come from L2
// (2048 rows over 32 pages each, with their selection: 0.97 ms, 1.10 at two); two, with three stages, where the bytes come from memory (64 sequences
// up to 64K: 649 us against 654) and at 16 rows, whose accumulators do not fit 168 registers.
template <int D, int RT, bool LIST>
struct Shape {
  static constexpr int kCtas = RT == 8 && LIST ? 3 : 2, kSpans = kCtas * 152 * kWarps;
  static constexpr int kStage = 2 * kHalf * D, kStages = (kCtas == 3 ? 16384 : 24576) / kStage;
  static constexpr int kBytes = kWarps * kStages * kStage;
};

// N channels of the output from element `at` on.
template <int N>
__device__ __forceinline__ void store_piece(const csa2_kv8_attn_args& a, long long at, const float* v, bool aligned) {
  if (a.out_dtype == CSA2_F32) {
    float* out = reinterpret_cast<float*>(a.out) + at;
    if (aligned) {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) reinterpret_cast<float4*>(out)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) out[i] = v[i];
    }
    return;
  }
  uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + at;
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = bf16x2(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
    if (aligned) {
      reinterpret_cast<uint4*>(out)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) out[8 * i + j] = (uint16_t)(w[j / 2] >> 16 * (j & 1));
    }
  }
}

// An 8 x 8 matrix of 16-bit values, two of row lane / 4 a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// RT: rows of a tile, 8 or 16.  LIST: streams are (row, head) pairs over their listed pages.
template <int D, int RT, bool LIST>
__global__ void __launch_bounds__(32 * kWarps, (Shape<D, RT, LIST>::kCtas))
k_kv8_stream(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const Kv8Params p) {
  using L = Shape<D, RT, LIST>;
  constexpr int kSt = L::kStages, kStage = L::kStage, kKs = D / 16, kR = RT / 8, kSpans = L::kSpans;
  constexpr bool kT = RT == 8;           // rows on N
  constexpr int kNt = kT ? D / 16 : D / 8;                   // accumulators of four
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint64_t bars[kWarps][kSt];
  const csa2_kv8_attn_args& a = p.a;
  const csa2_kv8_cache& c = a.cache;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q4 = lane & 3;
  // the rows whose sums this lane keeps: g and g + 8, or the two of its accumulators' columns
  auto own = [&](int i) { return kT ? 2 * q4 + i : g + 8 * i; };
  constexpr int kLane0 = kT ? 4 : 1, kLane1 = kT ? 32 : 4;   // lanes at these distances hold the same rows
  const int G = p.G, Hkv = c.Hkv, span = blockIdx.x * kWarps + warp;
  uint8_t* ring = smem + warp * kSt * kStage;
  const uint32_t ring_s = smem_u32(ring);
  if ((smem_u32(smem) & 1023) != 0) {                      // uniform: the ring's swizzle counts on it
    if (threadIdx.x == 0) raise_error(&g_err_kv8, CSA2_DEVERR_SMEM_ALIGN);
    return;
  }
  if (lane < kSt) tc::mbar_init(&bars[warp][lane], 1);
  __syncwarp();
  pdl_wait();
  pdl_trigger();

  // The work: half pages of sequence s, all its streams together.
  auto work = [&](int s, int& count, int& first) -> long long {
    const Rows r = rows_of(a, s, G);
    const long long limit = (long long)c.max_pages * kPage;
    const long long len = r.length < 0 ? 0 : r.length < limit ? r.length : limit;
    long long lo = 0;
    if (a.window > 0) {
      lo = (long long)r.length - ((long long)r.end - r.t0) + 1 - a.window;
      lo = lo < 0 ? 0 : lo < len ? lo : len;
    }
    first = (int)(lo / kHalf);
    count = (int)((len + kHalf - 1) / kHalf) - first;
    if (count < 1) count = 1;            // rows that see nothing are written all the same
    return (long long)((r.n + RT - 1) / RT) * Hkv * count;
  };
  const int list_tiles = (G + RT - 1) / RT;
  long long total, base = 0, mine = 0;   // of sequence (LIST: of everything) `s`: its begin and its work
  int s = 0, count = 0, first = 0;
  long long pos, stop, per;
  auto cut = [&] {
    per = (total + kSpans - 1) / kSpans;
    if (per < kLeast) per = kLeast;
    pos = span * per;
    stop = pos + per < total ? pos + per : total;
  };
  if constexpr (LIST) {
    count = 2 * a.list_len;
    total = mine = (long long)a.T * list_tiles * Hkv * count;
    cut();
  } else {
    // Sums over 32 sequences at a time, then within the 32 that hold this warp's begin.
    long long* sums = reinterpret_cast<long long*>(smem + L::kBytes);
    const int chunks = (a.S + 31) / 32;
    long long before = 0;
    int chunk = 0;
    if (chunks > 1) {
      for (int i = warp; i < chunks; i += kWarps) {
        int x, y;
        long long w = i * 32 + lane < a.S ? work(i * 32 + lane, x, y) : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
        if (lane == 0) sums[i] = w;
      }
      __syncthreads();
      total = 0;
      for (int i = 0; i < chunks; i += 32) {
        long long w = i + lane < chunks ? sums[i + lane] : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
        total += w;
      }
      cut();
      if (pos < stop)
        while (before + sums[chunk] <= pos) before += sums[chunk++];
    }
    long long w = 0;
    int x = 0, y = 0;
    if (chunk * 32 + lane < a.S) w = work(chunk * 32 + lane, x, y);
    long long inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (chunks <= 1) {
      total = __shfl_sync(0xffffffffu, inc, 31);
      cut();
    }
    if (pos < stop) {
      const int at = __ffs(__ballot_sync(0xffffffffu, before + inc > pos)) - 1;
      s = chunk * 32 + at;
      mine = __shfl_sync(0xffffffffu, w, at);
      base = before + __shfl_sync(0xffffffffu, inc, at) - mine;
      count = __shfl_sync(0xffffffffu, x, at);
      first = __shfl_sync(0xffffffffu, y, at);
    }
  }

  Part part = {0, 0, 0, 0, 0};
  uint32_t phase = 0;                    // of each stage's barrier
  bool dead = false;
  while (pos < stop) {
    if constexpr (!LIST) {
      while (pos >= base + mine) {
        base += mine;
        mine = work(++s, count, first);
      }
    }
    // ---- the stream, and the span's part of it
    const long long rel = pos - base;
    const long long u = rel / count;
    const int x = (int)(rel - u * count), take = (int)(count - x < stop - pos ? count - x : stop - pos);
    const int h = (int)(u % Hkv);
    const bool begins = x == 0, ends = x + take == count;
    int r0;                              // first row of the tile
    Rows rows;
    const int* list = nullptr;
    if constexpr (LIST) {
      const int tt = (int)(u / Hkv), t = tt / list_tiles;
      r0 = tt % list_tiles * RT;
      s = find_seq(a.start, a.S, t);
      if (s < 0) {                       // padding: nothing to write, not even parts
        pos += take;
        continue;
      }
      rows = rows_of(a, s, G);
      rows.t0 = t;
      rows.n = G;
      list = a.pages + ((long long)t * Hkv + h) * a.list_len;
    } else {
      r0 = (int)(u / Hkv) * RT;
      rows = rows_of(a, s, G);
    }
    const int nrows = min(RT, rows.n - r0);
    // ---- what this lane's rows see
    int lo[2], hi[2], lo_min = INT_MAX, lo_max = 0, hi_min = INT_MAX, hi_max = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lo[i] = 0;
      hi[i] = INT_MAX;
      if (own(i) < nrows) {
        seen_by(a, rows, rows.t0 + (r0 + own(i)) / G, lo[i], hi[i], &g_err_kv8);
        lo_min = min(lo_min, lo[i]);
        lo_max = max(lo_max, lo[i]);
        hi_min = min(hi_min, hi[i]);
        hi_max = max(hi_max, hi[i]);
      }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      if (o >= kLane0 && o < kLane1) continue;
      lo_min = min(lo_min, __shfl_xor_sync(0xffffffffu, lo_min, o));
      lo_max = max(lo_max, __shfl_xor_sync(0xffffffffu, lo_max, o));
      hi_min = min(hi_min, __shfl_xor_sync(0xffffffffu, hi_min, o));
      hi_max = max(hi_max, __shfl_xor_sync(0xffffffffu, hi_max, o));
    }
    // ---- half pages y0 .. y1 of the stream (LIST: of the list, else from `first` on), those in sight
    int y0 = x, y1 = x + take;
    if constexpr (!LIST) {
      y0 = max(y0, lo_min / kHalf - first);
      y1 = min(y1, (hi_max + kHalf - 1) / kHalf - first);
    }
    // Lane i: first token (-1: to be skipped), page and scales of half page 32 b + i for the batch b that is being
    // issued, [1], and the one before it, [0], which may still be worked on.
    int bt[2] = {-1, -1}, bp = 0;
    float bk[2] = {}, bv[2] = {};
    auto load_batch = [&](int b) {
      bt[0] = bt[1];
      bk[0] = bk[1];
      bv[0] = bv[1];
      bt[1] = -1;
      const int y = b + lane;
      if (y < y1) {
        int j, half;
        if constexpr (LIST) {
          j = list[y >> 1];
          half = y & 1;
          if (j >= c.max_pages) {
            raise_error(&g_err_kv8, CSA2_DEVERR_PAGE_SLOT);
            j = -1;
          }
        } else {
          j = (first + y) >> 1;
          half = (first + y) & 1;
        }
        const int token = j * kPage + half * kHalf;
        if (j >= 0 && token < hi_max && token + kHalf > lo_min) {
          const int page = page_id(c, s, j, &g_err_kv8);
          if (page >= 0) {
            bt[1] = token;
            bp = page;
            const long long ph = (long long)page * Hkv + h;
            bk[1] = c.k_scale[ph];
            bv[1] = c.v_scale[ph] * kWeightUndo;
          }
        }
      }
    };
    int issued = y0;
    auto issue = [&] {                   // the next half page into its stage
      const int b = (issued - y0) & 31;
      if (b == 0) load_batch(issued);
      const int st = (issued - y0) % kSt;
      const int token = __shfl_sync(0xffffffffu, bt[1], b), page = __shfl_sync(0xffffffffu, bp, b);
      if (lane == 0 && token >= 0) {
        tc::mbar_arrive_expect_tx(&bars[warp][st], kStage);
        tma_load_3d(ring + st * kStage, &mk, 0, token & kHalf, page * Hkv + h, &bars[warp][st]);
        tma_load_3d(ring + st * kStage + kHalf * D, &mv, 0, token & kHalf, page * Hkv + h, &bars[warp][st]);
      }
      ++issued;
    };
    for (int i = 0; i < kSt - 1; ++i)
      if (issued < y1) issue();
    // ---- their query in fragments, while the first copies are under way
    float mul[2], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, held[2] = {0.f, 0.f};
    uint32_t qa[kKs][2 * kR];
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int r = g + 8 * i;
      float v[D / 4];
#pragma unroll
      for (int e = 0; e < D / 4; ++e) v[e] = 0.f;
      if (r < nrows) {
        const int t = rows.t0 + (r0 + r) / G;
        const uint16_t* q = a.q + t * a.q_stride_t + (long long)(h * G + (r0 + r) % G) * a.q_stride_h + q4 * (D / 4);
        if (p.aligned & 1) {
#pragma unroll
          for (int e = 0; e < D / 32; ++e) {
            const uint4 w = reinterpret_cast<const uint4*>(q)[e];
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[8 * e + 2 * j] = __uint_as_float(ws[j] << 16);
              v[8 * e + 2 * j + 1] = __uint_as_float(ws[j] & 0xffff0000u);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < D / 4; ++e) v[e] = bf16_bits_to_f32(q[e]);
        }
      }
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < D / 4; ++e) top = fabsf(v[e]) >= top ? fabsf(v[e]) : (v[e] != v[e] ? INFINITY : top);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      float f, undo;
      row_factor(top, f, undo);
      if constexpr (kT) {
        mul[0] = __shfl_sync(0xffffffffu, undo, 8 * q4) * (a.softmax_scale * kLog2e);
        mul[1] = __shfl_sync(0xffffffffu, undo, 8 * q4 + 4) * (a.softmax_scale * kLog2e);
      } else {
        mul[i] = undo * (a.softmax_scale * kLog2e);
      }
#pragma unroll
      for (int j = 0; j < kKs; ++j) {
        qa[j][i] = f16x2(v[4 * j] * f, v[4 * j + 1] * f);
        qa[j][kR + i] = f16x2(v[4 * j + 2] * f, v[4 * j + 3] * f);
      }
    }
    float o[kNt][4];
#pragma unroll
    for (int n = 0; n < kNt; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;

    for (int y = y0; y < y1; ++y) {
      __syncwarp();                      // every lane has read the stage that is filled next
      if (issued < y1 && !dead) issue();
      const int st = (y - y0) % kSt;
      if (y >= issued) break;            // after a wait that gave up
      const bool old = (y - y0) >> 5 != (issued - 1 - y0) >> 5;
      const int token0 = __shfl_sync(0xffffffffu, old ? bt[0] : bt[1], (y - y0) & 31);
      if (token0 < 0) continue;
      if (!tc::mbar_wait(&bars[warp][st], phase >> st & 1, kWaitPolls)) {
        if (!dead) raise_error(&g_err_kv8, CSA2_DEVERR_TIMEOUT);
        dead = true;
      }
      dead = __any_sync(0xffffffffu, dead);
      phase ^= 1u << st;
      if (dead) continue;                // the copies in flight are still waited for
      const float2 sc = make_float2(__shfl_sync(0xffffffffu, old ? bk[0] : bk[1], (y - y0) & 31),
                                    __shfl_sync(0xffffffffu, old ? bv[0] : bv[1], (y - y0) & 31));
      const uint32_t kb = ring_s + st * kStage, vb = kb + kHalf * D;
      const bool border = token0 < lo_max || token0 + kHalf > hi_min;
      auto key = [&](int r, uint32_t* w) {                   // this lane's quarter of token r's key
        if constexpr (D == 128) {
          const uint4 w0 = lds128(kb + r * 128 + (((2 * q4) ^ (r & 7)) << 4));
          const uint4 w1 = lds128(kb + r * 128 + (((2 * q4 + 1) ^ (r & 7)) << 4));
          w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
          w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
        } else {
          const uint4 w0 = lds128(kb + r * 64 + ((q4 ^ (r >> 1 & 3)) << 4));
          w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
        }
      };
      // scores sx[i][..] of row own(i): tokens at(n)
      constexpr int kN = kT ? 4 : 8;
      float sx[2][kN];
      auto at = [&](int n) { return kT ? 8 * n + g : 8 * (n >> 1) + 2 * q4 + (n & 1); };
#pragma unroll
      for (int n = 0; n < (kT ? 2 : 4); ++n) {
        uint32_t w[D / 16];
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        if constexpr (kT) {
          uint32_t w8[D / 16];
          key(16 * n + g, w);
          key(16 * n + 8 + g, w8);
#pragma unroll
          for (int j = 0; j < kKs; ++j)
            mma_f16_16816(d, e4m3x2_lo_f16x2(w[j]), e4m3x2_lo_f16x2(w8[j]), e4m3x2_hi_f16x2(w[j]), e4m3x2_hi_f16x2(w8[j]),
                          qa[j][0], qa[j][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) sx[e & 1][2 * n + (e >> 1)] = d[e];
        } else {
          key(8 * n + g, w);
#pragma unroll
          for (int j = 0; j < kKs; ++j)
            mma_f16_16816(d, qa[j][0], qa[j][1], qa[j][2 * kR - 2], qa[j][2 * kR - 1], e4m3x2_lo_f16x2(w[j]), e4m3x2_hi_f16x2(w[j]));
#pragma unroll
          for (int e = 0; e < 4; ++e) sx[e >> 1][2 * n + (e & 1)] = d[e];
        }
      }
      float alpha[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float f = mul[i] * sc.x;
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          float v = sx[i][n] * f;
          if (border) v = token0 + at(n) >= lo[i] && token0 + at(n) < hi[i] ? v : -INFINITY;
          sx[i][n] = v;
          top = fmaxf(top, v);
        }
#pragma unroll
        for (int e = kLane0; e < kLane1; e <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, e));
        const float mn = fmaxf(m[i], top), z0 = mn == -INFINITY ? 0.f : mn, z = __fsub_ru(z0, kWeight);   // (a weight above 2^15 would leave fp16)
        alpha[i] = ex2(m[i] - z0);
        m[i] = mn;
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          sx[i][n] = ex2(sx[i][n] - z);
          sum += sx[i][n];
        }
        l[i] = l[i] * alpha[i] + sum;
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int n = 0; n < kNt; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][e] *= alpha[kT ? e & 1 : e >> 1];
        held[0] *= alpha[0];
        held[1] *= alpha[1];
      }
      // Sums of sums: added one by one to a sum near 1, small weights of a long stream would be rounded away (a token that
      // leads a million others by 17 nats: lse off by 1.4e-3).
      if (((y - y0) & 31) == 31) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          held[i] += l[i];
          l[i] = 0.f;
        }
      }
      // values: this lane's rows 16 kt + {2 q4, 2 q4 + 1, 8 + 2 q4, 9 + 2 q4}, channels D/8 * g ...
      constexpr int kVw = D / 32;        // words of a row a lane
      uint32_t vw[2][4][kVw];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * kt + 2 * q4 + (e & 1) + 8 * (e >> 1);
          if constexpr (D == 128) {
            const uint4 w = lds128(vb + r * 128 + ((g ^ (r & 7)) << 4));
            vw[kt][e][0] = w.x; vw[kt][e][1] = w.y; vw[kt][e][2] = w.z; vw[kt][e][3] = w.w;
          } else {
            const uint2 w = lds64(vb + r * 64 + (((g >> 1) ^ (r >> 1 & 3)) << 4) + (g & 1) * 8);
            vw[kt][e][0] = w.x; vw[kt][e][1] = w.y;
          }
        }
      // the weights of 16 tokens as a fragment: A of 16 rows, or, transposed, B of 8
      uint32_t pa[2][kT ? 2 : 4];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if constexpr (kT) {
            pa[kt][e] = transpose8(f16x2(sx[0][2 * kt + e], sx[1][2 * kt + e]));
          } else {
            pa[kt][e] = f16x2(sx[e][4 * kt], sx[e][4 * kt + 1]);
            pa[kt][2 + e] = f16x2(sx[e][4 * kt + 2], sx[e][4 * kt + 3]);
          }
        }
      constexpr int kDt = kT ? 2 : 4;    // accumulators of a word's four channels
      auto product = [&](const uint32_t (&pw)[2][kT ? 2 : 4], int w, float (&d)[kDt][4]) {
#pragma unroll
        for (int n = 0; n < kDt; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) d[n][e] = 0.f;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          uint32_t b[2][2];              // [token pair][bytes 0, 1 or 2, 3]: bytes of both tokens side by side
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            b[e][0] = __byte_perm(vw[kt][2 * e][w], vw[kt][2 * e + 1][w], 0x5140);
            b[e][1] = __byte_perm(vw[kt][2 * e][w], vw[kt][2 * e + 1][w], 0x7362);
          }
          if constexpr (kT) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
              mma_f16_16816(d[n], e4m3x2_lo_f16x2(b[0][n]), e4m3x2_hi_f16x2(b[0][n]), e4m3x2_lo_f16x2(b[1][n]),
                            e4m3x2_hi_f16x2(b[1][n]), pw[kt][0], pw[kt][1]);
          } else {
#pragma unroll
            for (int n = 0; n < 4; ++n)
              mma_f16_16816(d[n % kDt], pw[kt][0], pw[kt][1], pw[kt][kT ? 0 : 2], pw[kt][kT ? 0 : 3],
                            n & 1 ? e4m3x2_hi_f16x2(b[0][n >> 1]) : e4m3x2_lo_f16x2(b[0][n >> 1]),
                            n & 1 ? e4m3x2_hi_f16x2(b[1][n >> 1]) : e4m3x2_lo_f16x2(b[1][n >> 1]));
          }
        }
      };
      if (border) {
        // Rows of V that no row of the tile sees may hold anything: they count as zero.  A NaN that only some rows
        // see is taken out of the product and given to those rows alone.
        bool nan = false;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int token = token0 + 16 * kt + 2 * q4 + (e & 1) + 8 * (e >> 1);
            const bool see = token >= lo_min && token < hi_max;
#pragma unroll
            for (int w = 0; w < kVw; ++w) {
              vw[kt][e][w] = see ? vw[kt][e][w] : 0u;
              nan |= e4m3x4_nans(vw[kt][e][w]) != 0;
            }
          }
        if (__any_sync(0xffffffffu, nan)) {
          uint32_t keep[2][4][kVw], see[2][kT ? 2 : 4];
#pragma unroll
          for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int w = 0; w < kVw; ++w) {
                const uint32_t v = vw[kt][e][w], at = e4m3x4_nans(v);   // 1 in each NaN's byte
                keep[kt][e][w] = v & ~(at * 0xffu);
                vw[kt][e][w] = at * 0x38u;                   // E4M3 of 1
              }
            auto one = [&](int i, int n) { return token0 + at(n) >= lo[i] && token0 + at(n) < hi[i] ? 0x3c00u : 0u; };
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if constexpr (kT) {
                see[kt][e] = transpose8(one(0, 2 * kt + e) | one(1, 2 * kt + e) << 16);
              } else {
                see[kt][e] = one(e, 4 * kt) | one(e, 4 * kt + 1) << 16;
                see[kt][2 + e] = one(e, 4 * kt + 2) | one(e, 4 * kt + 3) << 16;
              }
            }
          }
#pragma unroll
          for (int w = 0; w < kVw; ++w) {
            float d[kDt][4];
            product(see, w, d);
#pragma unroll
            for (int n = 0; n < kDt; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (d[n][e] != 0.f) o[kDt * w + n][e] = NAN;
          }
#pragma unroll
          for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int w = 0; w < kVw; ++w) vw[kt][e][w] = keep[kt][e][w];
        }
      }
#pragma unroll
      for (int w = 0; w < kVw; ++w) {
        float d[kDt][4];
        product(pa, w, d);
#pragma unroll
        for (int n = 0; n < kDt; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[kDt * w + n][e] += d[n][e] * sc.y;
      }
    }
    __syncwarp();                        // the stages are free for the next stream
    if (dead) break;
    // ---- its result, or its part
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += held[i];
#pragma unroll
      for (int e = kLane0; e < kLane1; e <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], e);
      l[i] *= kWeightUndo;
      const int r = own(i);
      if (r < nrows) {
        // a piece of the row's channels: an eighth, of lane g, or a quarter, of columns 2 q4 and 2 q4 + 1 of every tile
        constexpr int kPiece = kT ? D / 8 : D / 4;
        const int piece = kT ? g : q4;
        float v[kPiece];
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
          v[kT ? 2 * n : n] = o[n][kT ? i : 2 * i];
          v[kT ? 2 * n + 1 : kNt + n] = o[n][kT ? 2 + i : 2 * i + 1];
        }
        if (begins && ends) {
          const long long row = (long long)(rows.t0 + (r0 + r) / G) * a.Hq + h * G + (r0 + r) % G;
          const float inv = l[i] == 0.f ? 0.f : __fdiv_rn(1.f, l[i]);
#pragma unroll
          for (int e = 0; e < kPiece; ++e) v[e] *= inv;
          store_piece<kPiece>(a, row * D + piece * kPiece, v, p.aligned & 2);
          if (piece == 0 && a.lse) a.lse[row] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
        } else {
          const long long to = ((long long)span * 2 + (begins ? 1 : 0)) * p.most + r;
          if (piece == 0) p.ml[to] = make_float2(m[i], l[i]);
          float4* dst = reinterpret_cast<float4*>(p.o + to * D + piece * kPiece);
#pragma unroll
          for (int e = 0; e < kPiece / 4; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
      }
    }
    if (begins && !ends) part = Part{nrows, rows.t0, r0, h, span + (int)((count - take + per - 1) / per)};
    pos += take;
  }
  if (lane == 0) p.part[span] = part;
}

// A CTA (span, eight rows): the stream that begins there and goes on in the next ones, a warp a row, a lane
// D / 32 channels.  Rows lie apart in the workspace, so eight loads a lane are under way at once; 6 us at 33 parts of 8 rows.
template <int D>
__global__ void __launch_bounds__(256, 2) k_kv8_join(const Kv8Params p) {
  constexpr int kPer = D / 32, kAhead = 8;
  const csa2_kv8_attn_args& a = p.a;
  pdl_wait();
  pdl_trigger();
  const int w0 = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Part part = p.part[w0];
  const int last = min(part.last, p.spans - 1), r = blockIdx.y * 8 + warp;
  if (r < part.rows) {
    auto at = [&](int w) { return ((long long)w * 2 + (w == w0 ? 1 : 0)) * p.most + r; };
    float top = -INFINITY, sum = 0.f, v[kPer] = {};
    for (int b = w0; b <= last; b += 32) {
      const int w = b + lane, n = min(32, last - b + 1);
      const float2 ml = w <= last ? p.ml[at(w)] : make_float2(-INFINITY, 0.f);
      float mn = fmaxf(top, ml.x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      const float z = mn == -INFINITY ? 0.f : mn, alpha = ex2(top - z), f = ex2(ml.x - z);
      top = mn;
      sum = sum * alpha + ml.y * f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[e] *= alpha;
      for (int i = 0; i < n; i += kAhead) {
        float o[kAhead][kPer];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const float* src = p.o + at(b + min(i + j, n - 1)) * D + lane * kPer;
          if constexpr (kPer == 4) {
            const float4 x = *reinterpret_cast<const float4*>(src);
            o[j][0] = x.x; o[j][1] = x.y; o[j][2] = x.z; o[j][3] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(src);
            o[j][0] = x.x; o[j][1] = x.y;
          }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const float fi = __shfl_sync(0xffffffffu, f, (i + j) & 31);
#pragma unroll
          for (int e = 0; e < kPer; ++e) v[e] += i + j < n ? o[j][e] * fi : 0.f;
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const long long row = (long long)(part.t0 + (part.r0 + r) / p.G) * a.Hq + part.h * p.G + (part.r0 + r) % p.G;
    const float inv = sum == 0.f ? 0.f : __fdiv_rn(1.f, sum);
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const long long i = row * D + lane * kPer + e;
      if (a.out_dtype == CSA2_F32) reinterpret_cast<float*>(a.out)[i] = v[e] * inv;
      else reinterpret_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16_rn(v[e] * inv);
    }
    if (lane == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

struct Layout {
  size_t part = 0, ml, o, second_ml, second, bytes;
  Layout(int spans, int rows, int D, bool split) {
    ml = up256(sizeof(Part) * spans);
    o = ml + up256(sizeof(float2) * spans * 2 * rows);
    second_ml = o + up256(sizeof(float) * spans * 2 * rows * D);
    second = second_ml + (split ? up256(sizeof(float2) * spans * rows) : 0);
    bytes = second + (split ? sizeof(float) * spans * rows * D : 0);
  }
};

template <int D, int RT, bool LIST>
cudaError_t launch_stream(const CUtensorMap& mk, const CUtensorMap& mv, const Kv8Params& p, cudaStream_t st) {
  static SmemLimit limit;
  const size_t smem = Shape<D, RT, LIST>::kBytes + (LIST ? 0 : 8 * (size_t)((p.a.S + 31) / 32));
  cudaError_t e = limit.raise(k_kv8_stream<D, RT, LIST>, smem);
  if (e != cudaSuccess) return e;
  return launch_k(k_kv8_stream<D, RT, LIST>, dim3(152 * Shape<D, RT, LIST>::kCtas), dim3(32 * kWarps), smem, st, mk, mv, p);
}

// Whether a sequence's rows of a key head fit a tile of 8.
bool takes_eight(const csa2_kv8_attn_args& a) {
  return (a.pages ? 1 : (long long)a.max_new) * (a.Hq / a.cache.Hkv) <= 8;
}

template <int D>
cudaError_t launch_rows(const Kv8Params& p, cudaStream_t st) {
  CUtensorMap mk, mv;
  if (!plane_map(&mk, p.a.cache.k, p.a.cache, kHalf) || !plane_map(&mv, p.a.cache.v, p.a.cache, kHalf))
    return cudaErrorInvalidValue;
  if (takes_eight(p.a)) return p.a.pages ? launch_stream<D, 8, true>(mk, mv, p, st) : launch_stream<D, 8, false>(mk, mv, p, st);
  return p.a.pages ? launch_stream<D, 16, true>(mk, mv, p, st) : launch_stream<D, 16, false>(mk, mv, p, st);
}

// Rows of a sequence and key head from which tiles take over from the streams of 16: those would read the pages once for
// every 16 rows.  32 sequences of 24K tokens, 8 key heads: 16 rows 269 us as a stream and 332 as tiles of 64, 24 rows 510
// and 334; 64 rows 998 and 340.
bool takes_tiles(const csa2_kv8_attn_args& a) {
  return !a.pages && (long long)a.max_new * (a.Hq / a.cache.Hkv) > 16;
}

int spans_of(const csa2_kv8_attn_args& a) {
  return takes_tiles(a) ? kTileSpans : a.pages && takes_eight(a) ? Shape<64, 8, true>::kSpans : Shape<64, 8, false>::kSpans;
}
int most_of(const csa2_kv8_attn_args& a) { return takes_tiles(a) ? tile_rows(a) : takes_eight(a) ? 8 : 16; }
Layout layout_of(const csa2_kv8_attn_args& a) {
  return Layout(spans_of(a), most_of(a), a.cache.D, takes_tiles(a) && tile_rows(a) < 256);
}

}  // namespace

size_t kv8_attn_workspace_bytes(const csa2_kv8_attn_args& a) {
  return layout_of(a).bytes;
}

cudaError_t launch_kv8_attn(const csa2_kv8_attn_args& a, void* ws, cudaStream_t st) {
  if (a.T == 0 || a.S == 0) return cudaSuccess;
  const bool tiles = takes_tiles(a);
  Kv8Params p;
  p.a = a;
  p.G = a.Hq / a.cache.Hkv;
  const bool q16 = (((uintptr_t)a.q | (uintptr_t)(2 * a.q_stride_t) | (uintptr_t)(2 * a.q_stride_h)) & 15) == 0;
  p.aligned = (q16 ? 1 : 0) | (((uintptr_t)a.out & 15) == 0 ? 2 : 0) | (((uintptr_t)a.out & 31) == 0 ? 4 : 0);
  p.spans = spans_of(a);
  p.most = most_of(a);
  const Layout at = layout_of(a);
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.part = reinterpret_cast<Part*>(w + at.part);
  p.ml = reinterpret_cast<float2*>(w + at.ml);
  p.o = reinterpret_cast<float*>(w + at.o);
  p.second_ml = reinterpret_cast<float2*>(w + at.second_ml);
  p.second = reinterpret_cast<float*>(w + at.second);
  cudaError_t e = tiles ? launch_kv8_tile(p, st) : a.cache.D == 64 ? launch_rows<64>(p, st) : launch_rows<128>(p, st);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.spans, p.most / 8);
  return a.cache.D == 64 ? launch_k(k_kv8_join<64>, grid, dim3(256), 0, st, p)
                         : launch_k(k_kv8_join<128>, grid, dim3(256), 0, st, p);
}

uint32_t read_clear_error_kv8() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_err_kv8, sizeof(v));
  if (v) cudaMemcpyToSymbol(g_err_kv8, &z, sizeof(z));
  return v | read_clear_error_kv8_tile();
}

}  // namespace csa2

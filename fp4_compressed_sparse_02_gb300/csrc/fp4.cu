// FP4 rows: the quantiser (csa2_fp4_quant) and the product with FP4 weights (csa2_fp4_linear).
#include <cfloat>

#include "internal.h"
#include "rows.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace csa2 {

CSA2_DEFINE_ERROR_WORD(g_err_fp4);

// ---------------------------------------------------------------------------------
// Quantiser
// ---------------------------------------------------------------------------------
namespace {

struct QuantRowsParams {
  const void* x;
  uint8_t* codes;
  uint8_t* tiles;
  const float* gscale;
  long long sx;
  int T, K, nkt;
};

constexpr int kQuantTiles = 4;   // column tiles (of 64 columns) of a CTA

}  // namespace

// CTA = 128 rows x 4 column tiles, 256 threads: half a warp takes 16 groups (256 columns) of a
// row, so codes leave in 128-byte runs; the scale bytes meet in shared memory and leave as
// whole 512-byte tiles, zero where there is no row or column.
template <bool X32, bool VEC>
__global__ void __launch_bounds__(256, 5) k_fp4_quant(QuantRowsParams p) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint4 tile[kQuantTiles * 32];
  const int tid = threadIdx.x;
  const int nct = (p.nkt + kQuantTiles - 1) / kQuantTiles;
  const int rt = blockIdx.x / nct, kt0 = (blockIdx.x % nct) * kQuantTiles;
  const long long r0 = rt * 128LL;
  const int rows = (int)min(128LL, p.T - r0);
  const int c = kt0 * 4 + (tid & 15), r1 = tid >> 4;      // the thread's 16-column group and first row of 16
  if (tid < kQuantTiles * 32) tile[tid] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  if (16 * c < p.K) {
    const float g = p.gscale ? ld_f32(p.gscale) : 1.f;
    const bool over = p.gscale != nullptr, fast = quotient_ok(g);
    long long x = (r0 + r1) * p.sx + 16 * c;
    uint8_t* codes = p.codes + (r0 + r1) * (p.K / 2) + 8 * c;
    uint8_t* sf = reinterpret_cast<uint8_t*>(tile) + fp4_scale_offset(r1, c & 15, kQuantTiles);
#pragma unroll 2
    for (int r = r1; r < rows; r += 16) {
      f32x2 n[8];                                         // u, negated (rows.cuh)
      if (VEC) {
        Raw16<X32> raw;
        raw.load(p.x, x, false);
        if (!over) raw.negate();                          // dividing by g negates
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = raw.pair(i);
      } else {
        load16_any(n, p.x, x, X32);
        if (!over)
#pragma unroll
          for (int i = 0; i < 8; ++i) n[i] = mul2(n[i], pk(-1.f, -1.f));
      }
      if (over) quotients16(n, g);
      const float a = amax16(n);
      uint32_t w[3];
      if (fast && a <= 0x1p60f) {
        fp4_encode16(n, a, w);
      } else {
        f32x2 t[8];
        uint32_t b[3];
        load16_any(t, p.x, x, X32);
        fp4_encode16_any(t, g, b);
        w[0] = b[0], w[1] = b[1], w[2] = b[2];
      }
      *reinterpret_cast<uint2*>(codes) = make_uint2(w[0], w[1]);
      sf[(r & 16) * 16 + (r >> 5) * 4] = (uint8_t)w[2];
      x += 16 * p.sx;
      codes += 8 * (long long)p.K;
    }
  }
  __syncthreads();
  if (tid < kQuantTiles * 32 && kt0 + (tid >> 5) < p.nkt)
    reinterpret_cast<uint4*>(p.tiles)[((long long)rt * p.nkt + kt0) * 32 + tid] = tile[tid];
}

cudaError_t launch_fp4_quant(const csa2_fp4_quant_args& a, cudaStream_t st) {
  if (a.out.rows == 0) return cudaSuccess;
  QuantRowsParams p{};
  p.x = a.x, p.codes = a.out.codes, p.tiles = a.out.scales, p.gscale = a.out.gscale;
  p.sx = a.x_stride, p.T = a.out.rows, p.K = a.out.cols, p.nkt = (a.out.cols + 63) / 64;
  const bool x32 = a.x_dtype == CSA2_F32;
  const bool vec = ((uintptr_t)a.x & 15) == 0 && (p.T == 1 || (a.x_stride * (x32 ? 4 : 2)) % 16 == 0);
  const long long grid = (long long)((p.nkt + kQuantTiles - 1) / kQuantTiles) * ((p.T + 127) / 128);
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  const auto k = x32 ? (vec ? k_fp4_quant<true, true> : k_fp4_quant<true, false>)
                     : (vec ? k_fp4_quant<false, true> : k_fp4_quant<false, false>);
  return launch_k(k, (unsigned)grid, 256, 0, st, p);
}

// ---------------------------------------------------------------------------------
// Product
// ---------------------------------------------------------------------------------
namespace lin {

constexpr int BM = 128;                    // weight rows (output features) of a tile: TMEM lanes
constexpr int BKB = 128;                   // bytes of codes per row and stage: 256 columns
constexpr int THREADS = 192;               // warps 0..3 epilogue, 4 loads, 5 products
constexpr uint32_t MAX_POLL = 1u << 24;

template <int BN>                          // tokens, up to 128: TMEM columns
struct Cfg {
  static constexpr int A = BM * BKB, B = BN * BKB, SF = 4 * 512;   // SF: scale tiles of w, and of x
  static constexpr int STAGE = A + B + 2 * SF;
  static constexpr int STAGES = (212 * 1024) / STAGE < 9 ? (212 * 1024) / STAGE : 9;
  // stages of a CTA that leaves room for a second one on its SM (TMEM: 256 columns each)
  static constexpr int STAGES2 = (113 * 1024) / STAGE < 4 ? (113 * 1024) / STAGE : 4;
  static constexpr int SMEM = STAGES * STAGE + 256;
  static constexpr int DCOLS = BN < 32 ? 32 : BN;
  static constexpr int SFCOLS = 32;        // scale columns of a stage: 4 per 64-column step, for w and for x
  static_assert(B % 1024 == 0 && STAGE % 1024 == 0, "operand tiles start on 1024-byte boundaries");
  static_assert(STAGES2 * STAGE >= BN * 512, "a partial result fits where the stages were");
  static_assert(DCOLS + STAGES * SFCOLS <= 512 && DCOLS + STAGES2 * SFCOLS <= 256, "TMEM columns");
};

struct Params {
  const uint8_t* wt;                       // scale tiles of the weights
  const uint8_t* xt;                       // scale tiles of x
  const float* gx;
  const float* gw;
  void* out;
  int T, N, nkt, stages, tmem_cols;
  bool out32, vec4;                        // vec4: rows of out are whole, aligned groups of four
};

// Instruction descriptor of kind::mxf4nvf4: E2M1 operands (1), both K-major, E4M3 scales (0),
// M x N x 64.
__host__ __device__ constexpr uint32_t idesc(int M, int N) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The descriptors' upper words are constants and their lower words the address / 16 (csrc/tc.cuh),
// so that the issuing thread adds one 32-bit offset an instruction: at 100 to 200 cycles of
// tensor work per product, its own instructions are what a product waits for.
constexpr uint32_t kOperandHi = (1024 >> 4) | (1u << 14) | (2u << 29);   // SBO 1024, version, 128-byte swizzle
constexpr uint32_t kScaleHi = (128 >> 4) | (1u << 14);                   // SBO 128, version, no swizzle

// The tensor map (a kernel parameter) into the cache its copies read it from.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" :: "l"(map) : "memory");
}

// One lane of the converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}

// One 512-byte scale tile into four TMEM columns (column j, lane l: the four scales of row
// 32 j + l), repeated for the four lane quarters.
__device__ __forceinline__ void sf_copy(uint32_t tmem, uint32_t lo) {
  asm volatile("{\n .reg .b64 t;\n mov.b64 t, {%1, %2};\n tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], t;\n}"
               :: "r"(tmem), "r"(lo), "r"(kScaleHi) : "memory");
}

__device__ __forceinline__ void mma_fp4(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 ta, tb;\n setp.ne.b32 p, %6, 0;\n"
      " mov.b64 ta, {%1, %7};\n mov.b64 tb, {%2, %7};\n"
      " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], ta, tb, %3, [%4], [%5], p;\n}"
      :: "r"(d), "r"(a), "r"(b), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(kOperandHi) : "memory");
}

__device__ __forceinline__ float4 ld_dsmem_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

template <typename P>
__device__ __forceinline__ void put(const P& p, long long at, float v) {
  if (p.out32)
    static_cast<float*>(p.out)[at] = v;
  else
    static_cast<uint16_t*>(p.out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Four neighbouring results, of which the first n exist.
template <typename P>
__device__ __forceinline__ void put4(const P& p, long long at, int n, float a, float b, float c, float d) {
  if (p.vec4) {
    if (p.out32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(a, b, c, d);
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = make_uint2(pack_bf16(a, b), pack_bf16(c, d));
    return;
  }
  put(p, at, a);
  if (n > 1) put(p, at + 1, b);
  if (n > 2) put(p, at + 2, c);
  if (n > 3) put(p, at + 3, d);
}

}  // namespace lin

// Up to 128 tokens, and more where the tiles are few (launch_fp4_linear): what bounds it is reading the weights
// once.  Tile = 128 features x BN tokens of out^T = w x^T, so that few tokens fill the N side of the product and
// the weights stream through the M side.  A cluster of S CTAs splits the sum over K; each leaves its float32
// partial in shared memory and the CTAs add them in rank order.
//   Occupancy: at 1 x 5120 -> 32768 (256 tiles) one CTA an SM with nine stages takes 20.4 us, two
// with four stages 16.5 us (its loads alone take as long; the floor of 94 MB is 13.9 us): a second
// CTA's loads run during the first's start and end.  Prefetching further tiles into L2 made it 18 to
// 20 us.
//   Split, 1 x 32768 -> 5120 (40 tiles), two CTAs an SM: S = 1 51 us, 3 21 us, 4 17.7 us, 6 16.8 us, 7 26 us
// (clusters of seven pack badly: some wait for a second round).  launch_linear takes the S of least cost in stages.
template <int BN>
__global__ void __launch_bounds__(lin::THREADS)
    k_fp4_linear(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx, lin::Params p) {
  using namespace lin;
  using C = Cfg<BN>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.stages * C::STAGE);
  uint64_t* empty = full + C::STAGES;
  uint64_t* accf = empty + C::STAGES;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(accf + 1);
  volatile int* failed = reinterpret_cast<volatile int*>(accf + 2);
  const int S = (int)gridDim.x / ((p.N + BM - 1) / BM);   // CTAs of a cluster
  const int rank = blockIdx.x % S;
  const int f0 = (blockIdx.x / S) * BM, t0 = blockIdx.y * BN, nt = min(BN, p.T - t0);   // several token tiles: BN = 128
  const int nkb = (p.nkt + 3) / 4;
  const int kb0 = (int)((long long)nkb * rank / S), kb1 = (int)((long long)nkb * (rank + 1) / S);
  // the same in every CTA; the barriers of a cluster are reached either way
  const bool aligned = (smem_u32(smem) & 1023) == 0;
  if (warp == 5) tc::tmem_alloc(tslot, p.tmem_cols);
  if (tid == 0) {
    prefetch_map(&mw);
    prefetch_map(&mx);
    for (int s = 0; s < C::STAGES; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(accf, 1);
    *failed = 0;
    if (!aligned) {
      raise_error(&g_err_fp4, CSA2_DEVERR_SMEM_ALIGN);
      *failed = 1;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  pdl_wait();                                             // all of the above runs beside the previous kernel's end
  pdl_trigger();
  const uint32_t tb = *tslot;
  int issued = kb0;                                       // loads of [kb0, issued) are on their way
  if (warp == 4) {
    if (lane == 0 && aligned) {
      for (int kb = kb0; kb < kb1; ++kb) {
        const int it = kb - kb0, s = it % p.stages;
        if (it >= p.stages && !tc::mbar_wait(&empty[s], (uint32_t)((it / p.stages - 1) & 1), MAX_POLL)) {
          raise_error(&g_err_fp4, CSA2_DEVERR_TIMEOUT);
          *failed = 1;
          break;
        }
        uint8_t* st = smem + s * C::STAGE;
        const int steps = min(4, p.nkt - 4 * kb);         // 64-column steps of this stage
        tc::mbar_arrive_expect_tx(&full[s], (uint32_t)(C::A + C::B + steps * 1024));
        tc::tma_load_2d(st, &mw, kb * BKB, f0, &full[s]);
        tc::tma_load_2d(st + C::A, &mx, kb * BKB, t0, &full[s]);
        uint8_t* sf = st + C::A + C::B;
        tc::bulk_load(sf, p.wt + ((long long)(f0 >> 7) * p.nkt + 4 * kb) * 512, steps * 512, &full[s]);
        tc::bulk_load(sf + C::SF, p.xt + ((long long)(t0 >> 7) * p.nkt + 4 * kb) * 512, steps * 512, &full[s]);
        issued = kb + 1;
      }
    }
  } else if (warp == 5) {
    if (aligned) {
      constexpr uint32_t id = idesc(BM, BN);
      const uint32_t sf0 = tb + C::DCOLS, base = smem_u32(smem) >> 4;
      int s = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!__all_sync(0xffffffffu, tc::mbar_wait(&full[s], phase, MAX_POLL))) {
          if (lane == 0) {
            raise_error(&g_err_fp4, CSA2_DEVERR_TIMEOUT);
            *failed = 1;
          }
          break;
        }
        tc::fence_after_sync();
        const uint32_t a = base + (uint32_t)s * (C::STAGE >> 4), sft = sf0 + (uint32_t)s * C::SFCOLS;
        const int steps = min(4, p.nkt - 4 * kb);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < steps) {
              sf_copy(sft + 4 * k, a + ((C::A + C::B + 512 * k) >> 4));
              sf_copy(sft + 16 + 4 * k, a + ((C::A + C::B + C::SF + 512 * k) >> 4));
            }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < steps)
              mma_fp4(tb, a + 2 * k, a + ((C::A + 32 * k) >> 4), id, sft + 4 * k, sft + 16 + 4 * k, kb > kb0 || k > 0);
          tc::mma_commit(&empty[s]);
        }
        __syncwarp();
        if (++s == p.stages) s = 0, phase ^= 1;
      }
      if (elect_one()) tc::mma_commit(accf);
      __syncwarp();
    }
  } else if (aligned) {
    if (!tc::mbar_wait_warp(accf, 0, MAX_POLL)) {
      if (lane == 0) {
        raise_error(&g_err_fp4, CSA2_DEVERR_TIMEOUT);
        *failed = 1;
      }
    }
    tc::fence_after_sync();
  }
  __syncthreads();
  const bool bad = *failed != 0;
  if (warp == 4 && lane == 0 && bad) {                    // copies in flight land before the CTA leaves
    for (int kb = issued - min(issued - kb0, p.stages); kb < issued; ++kb)
      tc::mbar_wait(&full[(kb - kb0) % p.stages], (uint32_t)(((kb - kb0) / p.stages) & 1), MAX_POLL);
  }
  const float alpha = (p.gx ? ld_f32(p.gx) : 1.f) * (p.gw ? ld_f32(p.gw) : 1.f);
  // the tile through shared memory, token by token, so that neighbouring lanes store neighbouring features
  if (warp < 4 && !bad) {
    const uint32_t tq = tb + ((uint32_t)(32 * warp) << 16);
    float* part = reinterpret_cast<float*>(smem) + 32 * warp + lane;
#pragma unroll 1
    for (int c = 0; c < nt; c += 32) {
      uint32_t v[32];
      tc::tmem_ld32(tq + (uint32_t)c, v);
      tc::tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c + i < nt) part[(c + i) * BM] = __uint_as_float(v[i]);
    }
  }
  __syncwarp();
  if (S > 1)
    tc::cluster_sync();
  else
    __syncthreads();
  if (!bad && S == 1 && !p.vec4) {                        // a warp a token, neighbouring lanes neighbouring features
    const int n = p.N - f0 - lane;
#pragma unroll 4
    for (int t = warp; t < nt; t += THREADS / 32) {
      const float* s = reinterpret_cast<const float*>(smem) + t * BM + lane;
      const long long at = (long long)(t0 + t) * p.N + f0 + lane;
#pragma unroll
      for (int i = 0; i < BM; i += 32)
        if (i < n) put(p, at + i, s[i] * alpha);
    }
  }
  if (!bad && f0 + 4 * lane < p.N) {                      // a warp a token: four features a lane
    const int f = f0 + 4 * lane;
    constexpr int WARPS = THREADS / 32;
    if (S == 1) {
      if (p.vec4) {
#pragma unroll 4
        for (int t = warp; t < nt; t += WARPS) {
          const float4 s = reinterpret_cast<const float4*>(smem)[t * (BM / 4) + lane];
          put4(p, (long long)(t0 + t) * p.N + f, p.N - f, s.x * alpha, s.y * alpha, s.z * alpha, s.w * alpha);
        }
      }
    } else {
      // the parts of two tokens on their way at once, of one where there are more parts than four: 777 x 4128 -> 1000
      // (S = 2) 8.6 us, one by one 9.7; 384 x 4096 -> 1024 (S = 5) 6.3 us, two tokens 6.7
      const int step = S * WARPS, many = S <= 4 ? 2 : 1;
      for (int t = rank * WARPS + warp; t < nt; t += many * step) {
        float4 v[2][8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t at = smem_u32(smem) + ((t + u * step) * BM + 4 * lane) * 4;
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (q < S && u < many && t + u * step < nt) v[u][q] = ld_dsmem_f4(tc::mapa(at, q));
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int tu = t + u * step;
          if (u >= many || tu >= nt) continue;
          float4 s = v[u][0];
#pragma unroll
          for (int q = 1; q < 8; ++q)
            if (q < S) s.x += v[u][q].x, s.y += v[u][q].y, s.z += v[u][q].z, s.w += v[u][q].w;
          put4(p, (long long)(t0 + tu) * p.N + f, p.N - f, s.x * alpha, s.y * alpha, s.z * alpha, s.w * alpha);
        }
      }
    }
  }
  __syncwarp();
  if (S > 1) tc::cluster_sync();                          // peers have read this CTA's partial
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 5) tc::tmem_dealloc(tb, p.tmem_cols);
}

// ---------------------------------------------------------------------------------
// Product of many tokens: CTA pairs
// ---------------------------------------------------------------------------------
namespace pairs {

using lin::BKB;
using lin::BM;
using lin::MAX_POLL;
constexpr int BN = 256;                    // features of a tile; each CTA holds half of their rows
constexpr int EPI = 8;                     // epilogue warps; then a warp of loads, one of products
constexpr int THREADS = 32 * (EPI + 2);
constexpr int A = BM * BKB, B = BN / 2 * BKB, SFA = 4 * 512, SFB = 2 * 4 * 512;
constexpr int STAGE = A + B + SFA + SFB;   // 38 KB
constexpr int STAGES = 5;
constexpr int SLICE = 2048;                // 32 rows x 32 bf16 columns on their way out
constexpr int OUT = STAGES * STAGE;        // two slices for each epilogue warp
constexpr int BARS = OUT + EPI * 2 * SLICE;
constexpr int SMEM = BARS + 256;
constexpr int SFCOLS = 16 + 32;            // scale columns of a stage, beside the accumulator: a stage's scales
                                           // stay until its products are done
static_assert(STAGE % 1024 == 0 && OUT % 1024 == 0 && BN + STAGES * SFCOLS <= 512, "alignment, TMEM columns");

template <int TOKENS>
struct Few {                               // k_fp4_linear_few: few tokens on the N side
  static constexpr int SF = TOKENS > 128 ? SFB : SFA;     // scale tiles of the tokens
  static constexpr int B = TOKENS / 2 * BKB, STAGE = A + B + SFA + SF;
  static constexpr int STAGES = (212 * 1024) / STAGE < 8 ? (212 * 1024) / STAGE : 8;
  static constexpr int SMEM = STAGES * STAGE + 256;
  static_assert(STAGE % 1024 == 0 && TOKENS + STAGES * SFCOLS <= 512, "alignment, TMEM columns");
  static_assert(TOKENS % 64 == 0 && STAGES * STAGE >= TOKENS * BM * 4, "a partial result fits where the stages were");
};

struct Params {
  const float* gx;
  const float* gw;
  void* out;
  int T, N, nkt, nft, ntt, band, split;
  int first, last;                         // tiles of this launch
  bool out32, vec4;
};

__device__ __forceinline__ void tmem_alloc2(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
               :: "r"((uint32_t)__cvta_generic_to_shared(slot)), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(taddr), "r"(ncols) : "memory");
}

// The scale tile at the same place in both CTAs' shared memory into both CTAs' TMEM.
__device__ __forceinline__ void sf_copy2(uint32_t tmem, uint32_t lo) {
  asm volatile("{\n .reg .b64 t;\n mov.b64 t, {%1, %2};\n tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], t;\n}"
               :: "r"(tmem), "r"(lo), "r"(lin::kScaleHi) : "memory");
}

__device__ __forceinline__ void mma_fp4_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t sfa, uint32_t sfb,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 ta, tb;\n setp.ne.b32 p, %6, 0;\n"
      " mov.b64 ta, {%1, %7};\n mov.b64 tb, {%2, %7};\n"
      " tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], ta, tb, %3, [%4], [%5], p;\n}"
      :: "r"(d), "r"(a), "r"(b), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(lin::kOperandHi) : "memory");
}

// Arrive on the mbarrier at this place in every CTA of `mask` once the products issued so far
// are done.
__device__ __forceinline__ void commit_pair(uint64_t* mbar, uint16_t mask) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               :: "r"((uint32_t)__cvta_generic_to_shared(mbar)), "h"(mask) : "memory");
}

// TMA load into this CTA's shared memory that completes on an mbarrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(void* dst, const void* map, int x, int y, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
      :: "r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(map), "r"(mbar), "r"(x), "r"(y)
      : "memory");
}

__device__ __forceinline__ void arrive_cluster(uint32_t mbar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(mbar) : "memory");
}

// TMA store of the box at (x, y) from shared memory, in a bulk group of this thread.
__device__ __forceinline__ void tma_store(const void* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n"
               "cp.async.bulk.commit_group;"
               :: "l"(map), "r"(src), "r"(x), "r"(y) : "memory");
}
template <int PENDING>
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" :: "n"(PENDING) : "memory");
}

// 32 columns of 32 rows (a lane's) into shared memory as a TMA store wants them: float32 rows of 128
// bytes, 16-byte chunk j at j ^ (row % 8), or bf16 rows of 64 bytes, chunk j at j ^ (row / 2 % 4).
__device__ __forceinline__ void stage32(const uint32_t (&v)[32], uint32_t at, int lane, float alpha, bool out32) {
  if (out32) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" :: "r"(at + lane * 128 + ((j ^ (lane & 7)) << 4)),
                   "f"(__uint_as_float(v[4 * j]) * alpha), "f"(__uint_as_float(v[4 * j + 1]) * alpha),
                   "f"(__uint_as_float(v[4 * j + 2]) * alpha), "f"(__uint_as_float(v[4 * j + 3]) * alpha) : "memory");
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = pack_bf16(__uint_as_float(v[8 * j + 2 * i]) * alpha, __uint_as_float(v[8 * j + 2 * i + 1]) * alpha);
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" :: "r"(at + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)),
                   "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
    }
  }
}

// stage32's rows out of shared memory to rows that TMA cannot address: a lane a column, `rows` values from `at` on
// (2048 x 5120 -> 8191: 40 us, against 48 us with the accumulator held until the last store; half a warp a row
// and two values a store took 47 us).
template <typename P>
__device__ __forceinline__ void store_rows(const P& p, uint32_t slice, int lane, long long at, int rows) {
  constexpr int BATCH = 8;
  at += lane;
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += BATCH) {                // a batch of rows' values, then their stores
    uint32_t e[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int r = r0 + i;
      if (p.out32)
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(e[i])
                     : "r"(slice + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + 4 * (lane & 3)));
      else
        asm volatile("{\n .reg .u16 t;\n ld.shared.u16 t, [%1];\n cvt.u32.u16 %0, t;\n}" : "=r"(e[i])
                     : "r"(slice + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + 2 * (lane & 7)));
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (r0 + i >= rows) continue;
      if (p.out32)
        static_cast<uint32_t*>(p.out)[at + (long long)(r0 + i) * p.N] = e[i];
      else
        static_cast<uint16_t*>(p.out)[at + (long long)(r0 + i) * p.N] = (uint16_t)e[i];
    }
  }
}

// Tile t: bands of `band` token tiles; within a band the token tile runs fastest (8192 x 5120 -> 32768: bands of
// 8 444 us, 16 440 us, 64 437 us).
__device__ __forceinline__ void place(const Params& p, int t, int& ft, int& tt) {
  const int per = p.band * p.nft, bnd = t / per, first = bnd * p.band;
  const int w = min(p.band, p.ntt - first), r = t - bnd * per;
  ft = r / w;
  tt = first + r % w;
}

}  // namespace pairs

// Persistent CTA pairs: a tile is 256 tokens x 256 features, each CTA holds 128 tokens and half of
// the features' rows, and the products of the pair read both halves.  The accumulator takes
// half of TMEM and the scales part of the rest, so the next tile starts when this one has been
// read: eight warps take it into registers in one go and release it before anything is stored.
//   What bounds it, 8192 x 5120 -> 32768: products alone take 316 us, the loads alone 279 us, the
// scale copies alone 282 us; all of it 422 us, 6.5 PFLOP/s, in bursts of a few ms (433 us on the slowest of three boards);
// back to back, under the power cap, 465 us, 5.9 PFLOP/s.  Each
// step's scales are copied right before its product: all of a stage's first, then its products, took 434 us
// (414 without the results), the next stage's before this one's products a fourth more.
//   Tile: 256 x 192 with two accumulators (results stored while the next tile runs) took 526 us:
// per product it loads a sixth more.  Reading the accumulator 32 columns at a time between stores
// took 496 us.  Two thirds of an earlier 1270 us was the issuing thread's own descriptor arithmetic.
//   Split over K in a cluster (the last round of few tiles), 256 x 32768 -> 5120 (20 tiles): 1 46 us, 2 31 us, 3 26 us,
// 4 40 us (20 clusters of eight do not all run at once).
// TMA_OUT: rows of the result that TMA can address; otherwise warps store them 32 columns at a time.
template <bool TMA_OUT>
__global__ void __launch_bounds__(pairs::THREADS, 1)
    k_fp4_linear_pair(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                      const __grid_constant__ CUtensorMap msx, const __grid_constant__ CUtensorMap msw,
                      const __grid_constant__ CUtensorMap mo, pairs::Params p) {
  using namespace pairs;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + BARS);   // the leader's are used
  uint64_t* empty = full + STAGES;
  uint64_t* accf = empty + STAGES;                        // accumulator complete
  uint64_t* acce = accf + 1;                              // read by both CTAs (the leader's)
  uint32_t* tslot = reinterpret_cast<uint32_t*>(acce + 1);
  volatile uint32_t* failed = tslot + 1;
  // cluster: `split` pairs that share a tile's sum over K; split > 1 only with one tile a cluster
  const int S = p.split, crank = (int)tc::cluster_ctarank(), part = crank >> 1;
  const uint32_t rank = crank & 1, leader = crank & ~1;   // rank 0 leads its pair
  const uint16_t both = (uint16_t)(3u << leader);
  const bool aligned = (smem_u32(smem) & 1023) == 0;      // the same in every CTA
  if (warp == EPI + 1) tmem_alloc2(tslot, 512);
  if (tid == 0) {
    lin::prefetch_map(&mw);
    lin::prefetch_map(&mx);
    lin::prefetch_map(&msw);
    lin::prefetch_map(&msx);
    for (int s = 0; s < STAGES; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(accf, 1);
    tc::mbar_init(acce, 2 * EPI);
    *failed = 0;
    if (!aligned) raise_error(&g_err_fp4, CSA2_DEVERR_SMEM_ALIGN);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();                                     // barriers and TMEM of both CTAs are there
  tc::fence_after_sync();
  pdl_wait();                                             // all of the above runs beside the previous kernel's end
  pdl_trigger();
  const uint32_t tb = *tslot;
  const int npair = gridDim.x / (2 * S), pr = p.first + blockIdx.x / (2 * S);
  const int ntile = p.last, nkb = (p.nkt + 3) / 4;
  const int kb0 = (int)((long long)nkb * part / S), kb1 = (int)((long long)nkb * (part + 1) / S);
  const bool run = aligned && tb == 0;                    // all 512 columns: they start at 0
  if (warp == EPI) {
    if (lane == 0 && run) {
      int s = 0, fill = 0;                                // fill: how often the stages have been filled
      bool ok = true;
      for (int t = pr; t < ntile && ok; t += npair) {
        int ft, tt;
        place(p, t, ft, tt);
        const int t0 = (2 * tt + (int)rank) * BM, f0 = ft * BN;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (fill > 0 && !tc::mbar_wait(&empty[s], (uint32_t)((fill - 1) & 1), MAX_POLL)) {
            raise_error(&g_err_fp4, CSA2_DEVERR_TIMEOUT);
            *failed = 1;
            ok = false;
            break;
          }
          uint8_t* st = smem + s * STAGE;
          if (rank == 0) tc::mbar_arrive_expect_tx(&full[s], 2u * STAGE);
          const uint32_t mb = tc::mapa(smem_u32(&full[s]), leader);
          tma_load_pair(st, &mx, kb * BKB, t0, mb);
          tma_load_pair(st + A, &mw, kb * BKB, f0 + (int)rank * (BN / 2), mb);
          tma_load_pair(st + A + B, &msx, kb * 256, t0 >> 7, mb);
          tma_load_pair(st + A + B + SFA, &msw, kb * 256, f0 >> 7, mb);
          if (++s == STAGES) s = 0, ++fill;
        }
      }
    }
  } else if (warp == EPI + 1) {
    if (rank == 0 && run) {
      constexpr uint32_t id = lin::idesc(2 * BM, BN);
      const uint32_t base = smem_u32(smem) >> 4;
      int s = 0;
      uint32_t phase = 0, drained = 1;                    // the first tile finds the accumulator free
      bool ok = true;
      for (int t = pr; t < ntile && ok; t += npair) {
        if (!tc::mbar_wait_warp(acce, drained, MAX_POLL)) {
          if (lane == 0) {
            raise_error(&g_err_fp4, CSA2_DEVERR_TIMEOUT);
            *failed = 1;
          }
          break;
        }
        drained ^= 1;
        tc::fence_after_sync();
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!__all_sync(0xffffffffu, tc::mbar_wait(&full[s], phase, MAX_POLL))) {
            if (lane == 0) {
              raise_error(&g_err_fp4, CSA2_DEVERR_TIMEOUT);
              *failed = 1;
            }
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint32_t a = base + (uint32_t)s * (STAGE >> 4), sft = BN + (uint32_t)s * SFCOLS;
          const int nt = min(4, p.nkt - 4 * kb);
          if (lin::elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < nt) {
                sf_copy2(sft + 4 * k, a + ((A + B + 512 * k) >> 4));
                sf_copy2(sft + 16 + 8 * k, a + ((A + B + SFA + 512 * k) >> 4));
                sf_copy2(sft + 20 + 8 * k, a + ((A + B + SFA + 2048 + 512 * k) >> 4));
                mma_fp4_pair(0, a + 2 * k, a + ((A + 32 * k) >> 4), id, sft + 4 * k, sft + 16 + 8 * k,
                             kb > kb0 || k > 0);
              }
            commit_pair(&empty[s], both);
          }
          __syncwarp();
          if (++s == STAGES) s = 0, phase ^= 1;
        }
        if (lin::elect_one()) commit_pair(accf, both);
        __syncwarp();
      }
    }
  } else if (run) {
    // warp w: rows (tokens) 32 (w % 4) .. of the CTA's 128, columns (features) 128 (w / 4) ..
    const float alpha = (p.gx ? ld_f32(p.gx) : 1.f) * (p.gw ? ld_f32(p.gw) : 1.f);
    const uint32_t slice = smem_u32(smem + OUT + warp * 2 * SLICE);
    const uint32_t tq = ((uint32_t)(32 * (warp & 3)) << 16) + 128u * (warp >> 2);
    uint32_t phase = 0;
    for (int t = pr; t < ntile; t += npair) {
      int ft, tt;
      place(p, t, ft, tt);
      if (!tc::mbar_wait_warp(accf, phase, MAX_POLL)) {
        if (lane == 0) {
          raise_error(&g_err_fp4, CSA2_DEVERR_TIMEOUT);
          *failed = 1;
        }
        break;
      }
      phase ^= 1;
      tc::fence_after_sync();
      if (S > 1) {                                        // this pair's part of the sum, 16-byte chunk j at j ^ (row % 8)
        const uint32_t row = 32 * (warp & 3) + lane, at = smem_u32(smem) + row * 1024;
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          uint32_t v[32];
          tc::tmem_ld32(tq + (uint32_t)c, v);
          tc::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};"
                         :: "r"(at + ((((warp >> 2) * 32 + c / 4 + j) ^ (row & 7)) << 4)), "r"(v[4 * j]),
                         "r"(v[4 * j + 1]), "r"(v[4 * j + 2]), "r"(v[4 * j + 3]) : "memory");
        }
        break;                                            // the cluster's only tile
      }
      const int t0 = (2 * tt + (int)rank) * BM + 32 * (warp & 3), f0 = ft * BN + 128 * (warp >> 2);
      uint32_t acc[4][32];                                // all of this warp's part, so that it is free at once
#pragma unroll
      for (int i = 0; i < 4; ++i) tc::tmem_ld32(tq + 32u * i, acc[i]);
      tc::tmem_ld_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_cluster(tc::mapa(smem_u32(acce), leader));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (t0 >= p.T || f0 + 32 * i >= p.N) continue;
        if (TMA_OUT) {
          // the slice's last store has read it (float32 slices take both halves)
          if (lane == 0) p.out32 ? store_wait_read<0>() : store_wait_read<1>();
          __syncwarp();
          const uint32_t at = slice + (p.out32 ? 0u : (uint32_t)(i & 1) * SLICE);
          stage32(acc[i], at, lane, alpha, p.out32);
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tma_store(&mo, f0 + 32 * i, t0, at);
        } else {
          stage32(acc[i], slice, lane, alpha, p.out32);
          __syncwarp();
          store_rows(p, slice, lane, (long long)t0 * p.N + f0 + 32 * i, f0 + 32 * i + lane < p.N ? min(32, p.T - t0) : 0);
          __syncwarp();
        }
      }
    }
    if (lane == 0) store_wait_read<0>();
  }
  if (S > 1) {
    // the parts of a row, in the order of K, from the CTAs that hold it; each adds its share of rows
    __syncwarp();
    tc::cluster_sync();
    if (warp < EPI && run) {
      const float alpha = (p.gx ? ld_f32(p.gx) : 1.f) * (p.gw ? ld_f32(p.gw) : 1.f);
      int ft, tt;
      place(p, pr, ft, tt);
      const int t0 = (2 * tt + (int)rank) * BM, rows = min(BM, p.T - t0);
      for (int u = part * 32 * EPI + tid; u < rows * (BN / 4); u += S * 32 * EPI) {
        const int row = u / (BN / 4), j = u % (BN / 4), f = ft * BN + 4 * j;
        if (f >= p.N) continue;
        const uint32_t at = smem_u32(smem) + row * 1024 + ((j ^ (row & 7)) << 4);
        float4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q < S) v[q] = lin::ld_dsmem_f4(tc::mapa(at, 2 * q + rank));
        float4 e = v[0];
#pragma unroll
        for (int q = 1; q < 4; ++q)
          if (q < S) e.x += v[q].x, e.y += v[q].y, e.z += v[q].z, e.w += v[q].w;
        lin::put4(p, (long long)(t0 + row) * p.N + f, p.N - f, e.x * alpha, e.y * alpha, e.z * alpha, e.w * alpha);
      }
    }
  }
  tc::fence_before_sync();
  __syncwarp();
  __syncthreads();
  if (tid == 0 && *failed)                                // given up: the copies in flight land in a few us
    for (int i = 0; i < 2000; ++i) __nanosleep(1000);
  __syncwarp();
  tc::cluster_sync();                                     // the peer's loads, products and arrivals are done
  if (warp == EPI + 1) tmem_dealloc2(tb, 512);
}

// Up to BN tokens on CTA pairs: a tile is 256 features x BN tokens of out^T = w x^T, each CTA holds 128
// features' weights and half of the tokens' rows, so the pair reads the tokens once and its products
// are no wider than the tokens.  A cluster of S pairs splits the sum over K; the CTAs of a rank add the parts as
// k_fp4_linear does, with loads from the peers' shared memory (bulk copies of each owner's tokens to it took 1.2
// to 2 us more).
//   What bounds it, 192 x 32768 -> 5120 (20 tiles split in three, 23.2 us; 14.7 us at the copy rate): 60 of 76 pairs
// have work, each CTA takes in 34 KB every 0.4 us, which is 45 bytes a cycle; start, end and adding take
// 6 us.  Pairs of 256 x 256 (the tokens on the M side, a quarter of each product empty) took 26.0 us, CTAs of
// 128 x 192 28 us.
template <int BN>
__global__ void __launch_bounds__(pairs::THREADS, 1)
    k_fp4_linear_few(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                     const __grid_constant__ CUtensorMap msw, const __grid_constant__ CUtensorMap msx, pairs::Params p) {
  using namespace pairs;
  using C = Few<BN>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE);   // the leader's are used
  uint64_t* empty = full + C::STAGES;
  uint64_t* accf = empty + C::STAGES;                     // accumulator complete
  uint32_t* tslot = reinterpret_cast<uint32_t*>(accf + 1);
  volatile uint32_t* failed = tslot + 1;
  const int S = p.split, crank = (int)tc::cluster_ctarank(), part = crank >> 1;
  const uint32_t rank = crank & 1, leader = crank & ~1;   // rank 0 leads its pair
  const uint16_t both = (uint16_t)(3u << leader);
  const bool aligned = (smem_u32(smem) & 1023) == 0;      // the same in every CTA
  if (warp == EPI + 1) tmem_alloc2(tslot, 512);
  if (tid == 0) {
    lin::prefetch_map(&mw);
    lin::prefetch_map(&mx);
    lin::prefetch_map(&msw);
    lin::prefetch_map(&msx);
    for (int s = 0; s < C::STAGES; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(accf, 1);
    *failed = 0;
    if (!aligned) raise_error(&g_err_fp4, CSA2_DEVERR_SMEM_ALIGN);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();                                     // barriers and TMEM of both CTAs are there
  tc::fence_after_sync();
  pdl_wait();                                             // all of the above runs beside the previous kernel's end
  pdl_trigger();
  const uint32_t tb = *tslot;
  const int nkb = (p.nkt + 3) / 4;
  const int kb0 = (int)((long long)nkb * part / S), kb1 = (int)((long long)nkb * (part + 1) / S);
  const int f0 = ((int)blockIdx.x / (2 * S) * 2 + (int)rank) * BM;
  const bool run = aligned && tb == 0;                    // all 512 columns: they start at 0
  if (warp == EPI) {
    if (lane == 0 && run) {
      int s = 0, fill = 0;                                // fill: how often the stages have been filled
      for (int kb = kb0; kb < kb1; ++kb) {
        if (fill > 0 && !tc::mbar_wait(&empty[s], (uint32_t)((fill - 1) & 1), MAX_POLL)) {
          raise_error(&g_err_fp4, CSA2_DEVERR_TIMEOUT);
          *failed = 1;
          break;
        }
        uint8_t* st = smem + s * C::STAGE;
        if (rank == 0) tc::mbar_arrive_expect_tx(&full[s], 2u * C::STAGE);
        const uint32_t mb = tc::mapa(smem_u32(&full[s]), leader);
        tma_load_pair(st, &mw, kb * BKB, f0, mb);
        tma_load_pair(st + A, &mx, kb * BKB, (int)rank * (BN / 2), mb);
        tma_load_pair(st + A + C::B, &msw, kb * 256, f0 >> 7, mb);
        tma_load_pair(st + A + C::B + SFA, &msx, kb * 256, 0, mb);
        if (++s == C::STAGES) s = 0, ++fill;
      }
    }
  } else if (warp == EPI + 1) {
    if (rank == 0 && run) {
      constexpr uint32_t id = lin::idesc(2 * BM, BN);
      const uint32_t base = smem_u32(smem) >> 4;
      int s = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!__all_sync(0xffffffffu, tc::mbar_wait(&full[s], phase, MAX_POLL))) {
          if (lane == 0) {
            raise_error(&g_err_fp4, CSA2_DEVERR_TIMEOUT);
            *failed = 1;
          }
          break;
        }
        tc::fence_after_sync();
        const uint32_t a = base + (uint32_t)s * (C::STAGE >> 4), sft = BN + (uint32_t)s * SFCOLS;
        const int steps = min(4, p.nkt - 4 * kb);
        if (lin::elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < steps) {
              sf_copy2(sft + 4 * k, a + ((A + C::B + 512 * k) >> 4));
              sf_copy2(sft + 16 + 8 * k, a + ((A + C::B + SFA + 512 * k) >> 4));
              if (BN > 128) sf_copy2(sft + 20 + 8 * k, a + ((A + C::B + SFA + 2048 + 512 * k) >> 4));
              mma_fp4_pair(0, a + 2 * k, a + ((A + 32 * k) >> 4), id, sft + 4 * k, sft + 16 + 8 * k, kb > kb0 || k > 0);
            }
          commit_pair(&empty[s], both);
        }
        __syncwarp();
        if (++s == C::STAGES) s = 0, phase ^= 1;
      }
      if (lin::elect_one()) commit_pair(accf, both);
      __syncwarp();
    }
  } else if (run) {
    if (!tc::mbar_wait_warp(accf, 0, MAX_POLL)) {
      if (lane == 0) {
        raise_error(&g_err_fp4, CSA2_DEVERR_TIMEOUT);
        *failed = 1;
      }
    } else {
      // warp w: features 32 (w % 4) .. of the CTA's 128, half of the tokens; token by token into the stages' place
      tc::fence_after_sync();
      const uint32_t tq = (uint32_t)(32 * (warp & 3)) << 16;
      float* at = reinterpret_cast<float*>(smem) + 32 * (warp & 3) + lane;
      const int c1 = min(p.T, BN / 2 * (warp / 4 + 1));
#pragma unroll 1
      for (int c = BN / 2 * (warp / 4); c < c1; c += 32) {
        uint32_t v[32];
        tc::tmem_ld32(tq + (uint32_t)c, v);
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) at[(c + i) * BM] = __uint_as_float(v[i]);
      }
    }
  }
  __syncwarp();
  tc::cluster_sync();                                     // every part of the sum is there
  if (warp < EPI && run && f0 + 4 * lane < p.N) {         // a warp a token: four features a lane
    const float alpha = (p.gx ? ld_f32(p.gx) : 1.f) * (p.gw ? ld_f32(p.gw) : 1.f);
    const int f = f0 + 4 * lane;
    // two tokens' loads on their way at once: one by one costs 0.75 us more at S = 2, four 0.7 us at S = 3
    const int step = S * EPI;
    for (int t = part * EPI + warp; t < p.T; t += 2 * step) {
      float4 v[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t at = smem_u32(smem) + ((t + u * step) * BM + 4 * lane) * 4;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q < S && t + u * step < p.T) v[u][q] = lin::ld_dsmem_f4(tc::mapa(at, 2 * q + rank));
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int tu = t + u * step;
        if (tu >= p.T) continue;
        float4 e = v[u][0];
#pragma unroll
        for (int q = 1; q < 4; ++q)
          if (q < S) e.x += v[u][q].x, e.y += v[u][q].y, e.z += v[u][q].z, e.w += v[u][q].w;
        lin::put4(p, (long long)tu * p.N + f, p.N - f, e.x * alpha, e.y * alpha, e.z * alpha, e.w * alpha);
      }
    }
  }
  tc::fence_before_sync();
  __syncwarp();
  __syncthreads();
  if (tid == 0 && *failed)                                // given up: the copies in flight land in a few us
    for (int i = 0; i < 2000; ++i) __nanosleep(1000);
  __syncwarp();
  tc::cluster_sync();                                     // the peer's loads, products and reads are done
  if (warp == EPI + 1) tmem_dealloc2(tb, 512);
}

namespace {

bool groups_of_four(const csa2_fp4_linear_args& a) {
  return a.w.rows % 4 == 0 && ((uintptr_t)a.out & (a.out_dtype == CSA2_F32 ? 15 : 7)) == 0;
}

// How many clusters of s units, s = 1 .. 8 at most, the GPU holds at once.
struct Clusters {
  int of[9];
};

// How many clusters of `cta` CTAs of a kernel the GPU holds at once.
template <typename K>
int resident_clusters(K* kernel, int cta, int threads, size_t smem) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cta;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = (unsigned)cta;
  cfg.blockDim = (unsigned)threads;
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

// uint8 matrix [rows][bytes], boxes of box_rows x 128 bytes, 128-byte swizzle: packed FP4 codes
// as the K-major operand of the product.
bool codes_map(CUtensorMap* map, const void* base, long long rows, long long bytes, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t gdim[2] = {(cuuint64_t)bytes, (cuuint64_t)rows};
  const cuuint64_t gstride[1] = {(cuuint64_t)bytes};
  const cuuint32_t box[2] = {(cuuint32_t)lin::BKB, (cuuint32_t)box_rows};
  const cuuint32_t estride[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), gdim, gstride, box, estride,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The scale tiles of FP4 rows as a matrix [row tiles][512 column tiles' bytes] of 8-byte words, boxes
// of box_tiles x 4 tiles; tiles past the last read as zero.
bool scales_map(CUtensorMap* map, const csa2_fp4_rows& m, int box_tiles) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t nkt = (cuuint64_t)((m.cols + 63) / 64);
  const cuuint64_t gdim[2] = {nkt * 64, (cuuint64_t)((m.rows + 127) / 128)};
  const cuuint64_t gstride[1] = {nkt * 512};
  const cuuint32_t box[2] = {256, (cuuint32_t)box_tiles};
  const cuuint32_t estride[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, 2, m.scales, gdim, gstride, box, estride,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The output [rows][cols] as boxes of 32 rows x 32 columns, rows of 64 (bf16) or 128 (float32)
// swizzled bytes in shared memory.
bool out_map(CUtensorMap* map, void* base, long long rows, long long cols, bool f32) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t gdim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t gstride[1] = {(cuuint64_t)cols * (f32 ? 4 : 2)};
  const cuuint32_t box[2] = {32, 32};
  const cuuint32_t estride[2] = {1, 1};
  return enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, gdim, gstride, box,
             estride, CU_TENSOR_MAP_INTERLEAVE_NONE, f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool TMA_OUT>
cudaError_t launch_linear_pair(const csa2_fp4_linear_args& a, cudaStream_t st) {
  using namespace pairs;
  CUtensorMap mx, mw, msx, msw, mo{};
  pairs::Params p{};
  p.out32 = a.out_dtype == CSA2_F32;
  if (!codes_map(&mx, a.x.codes, a.x.rows, a.x.cols / 2, BM) || !codes_map(&mw, a.w.codes, a.w.rows, a.w.cols / 2, BN / 2) ||
      !scales_map(&msx, a.x, 1) || !scales_map(&msw, a.w, 2) ||
      (TMA_OUT && !out_map(&mo, a.out, a.x.rows, a.w.rows, p.out32)))
    return cudaErrorInvalidValue;
  p.gx = a.x.gscale, p.gw = a.w.gscale, p.out = a.out;
  p.T = a.x.rows, p.N = a.w.rows, p.nkt = (a.x.cols + 63) / 64;
  p.nft = (p.N + BN - 1) / BN, p.ntt = (p.T + 2 * BM - 1) / (2 * BM);
  p.band = 64;
  const long long ntile = (long long)p.nft * p.ntt;
  if (ntile > INT32_MAX / 2) return cudaErrorInvalidConfiguration;
  p.vec4 = groups_of_four(a);
  static PerDevice<Clusters> resident;
  const Clusters* clusters_of = nullptr;
  cudaError_t e = resident.get(&clusters_of, [](Clusters& c) {
    cudaError_t e = cudaFuncSetAttribute(k_fp4_linear_pair<TMA_OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    for (int s = 4; s >= 1; --s) c.of[s] = resident_clusters(k_fp4_linear_pair<TMA_OUT>, 2 * s, THREADS, SMEM);
    return c.of[1] ? cudaSuccess : cudaErrorInvalidConfiguration;
  });
  if (e != cudaSuccess) return e;
  const int* pairs_at = clusters_of->of;                  // clusters of s pairs
  // few tiles: split the sum as far as every cluster still runs at once, two stages a CTA or more
  const int nkb = (p.nkt + 3) / 4;
  const auto split_of = [&](long long tiles) {
    int split = 1;
    for (int s = 2; s <= 4; ++s)
      if (tiles <= pairs_at[s] && 2 * s <= nkb) split = s;
    return split;
  };
  const auto launch = [&](long long first, long long tiles, int split) {
    p.first = (int)first, p.last = (int)(first + tiles), p.split = split;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2u * (unsigned)split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const long long clusters = split > 1 || tiles < pairs_at[1] ? tiles : pairs_at[1];
    cfg.gridDim = dim3(2u * (unsigned)(split * clusters));
    cfg.blockDim = pairs::THREADS;
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_fp4_linear_pair<TMA_OUT>, mx, mw, msx, msw, mo, p);
  };
  // A last round of a few tiles costs what a full one does.  Where splitting it saves more than a second
  // launch and the partial sums cost, it is launched apart: 1024 x 32768 -> 5120 (80 tiles on 76 pairs,
  // 96 stages saved) 84.9 -> 64.7 us, but 1024 x 5120 -> 5120 (15 saved) 19.7 -> 22.2 us.
  const long long rest = ntile % pairs_at[1];
  const int split = split_of(rest);
  if (ntile > pairs_at[1] && rest > 0 && split > 1 && nkb - nkb / split >= 32) {
    e = launch(0, ntile - rest, 1);
    return e != cudaSuccess ? e : launch(ntile - rest, rest, split);
  }
  return launch(0, ntile, split_of(ntile));
}

template <int BN>
cudaError_t launch_linear_few(const csa2_fp4_linear_args& a, cudaStream_t st) {
  using namespace pairs;
  CUtensorMap mx, mw, msx, msw;
  if (!codes_map(&mw, a.w.codes, a.w.rows, a.w.cols / 2, BM) || !codes_map(&mx, a.x.codes, a.x.rows, a.x.cols / 2, BN / 2) ||
      !scales_map(&msw, a.w, 1) || !scales_map(&msx, a.x, BN > 128 ? 2 : 1))
    return cudaErrorInvalidValue;
  pairs::Params p{};
  p.gx = a.x.gscale, p.gw = a.w.gscale, p.out = a.out, p.out32 = a.out_dtype == CSA2_F32, p.vec4 = groups_of_four(a);
  p.T = a.x.rows, p.N = a.w.rows, p.nkt = (a.x.cols + 63) / 64;
  const int tiles = (p.N + 2 * BM - 1) / (2 * BM), nkb = (p.nkt + 3) / 4;
  static PerDevice<Clusters> resident;
  const Clusters* clusters_of = nullptr;
  cudaError_t e = resident.get(&clusters_of, [](Clusters& c) {
    cudaError_t e = cudaFuncSetAttribute(k_fp4_linear_few<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<BN>::SMEM);
    if (e != cudaSuccess) return e;
    for (int s = 4; s >= 1; --s) c.of[s] = resident_clusters(k_fp4_linear_few<BN>, 2 * s, THREADS, Few<BN>::SMEM);
    return c.of[1] ? cudaSuccess : cudaErrorInvalidConfiguration;
  });
  if (e != cudaSuccess) return e;
  const int* pairs_at = clusters_of->of;                  // clusters of s pairs
  p.split = 1;
  for (int s = 2; s <= 4; ++s)
    if (tiles <= pairs_at[s] && 2 * s <= nkb) p.split = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2u * (unsigned)p.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)(p.split * tiles));
  cfg.blockDim = pairs::THREADS;
  cfg.dynamicSmemBytes = Few<BN>::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_fp4_linear_few<BN>, mw, mx, msw, msx, p);
}

template <int BN>
cudaError_t launch_linear(const csa2_fp4_linear_args& a, cudaStream_t st) {
  using C = lin::Cfg<BN>;
  CUtensorMap mw, mx;
  if (!codes_map(&mw, a.w.codes, a.w.rows, a.w.cols / 2, lin::BM) ||
      !codes_map(&mx, a.x.codes, a.x.rows, a.x.cols / 2, BN))
    return cudaErrorInvalidValue;
  lin::Params p{};
  p.wt = a.w.scales, p.xt = a.x.scales, p.gx = a.x.gscale, p.gw = a.w.gscale, p.out = a.out;
  p.T = a.x.rows, p.N = a.w.rows, p.nkt = (a.x.cols + 63) / 64, p.out32 = a.out_dtype == CSA2_F32;
  p.vec4 = groups_of_four(a);
  const int ft = (p.N + lin::BM - 1) / lin::BM, tt = (p.T + BN - 1) / BN, nkb = (p.nkt + 3) / 4;
  const long long tiles = (long long)ft * tt;
  static PerDevice<Clusters> resident;
  const Clusters* clusters_of = nullptr;
  cudaError_t e = resident.get(&clusters_of, [](Clusters& c) {
    cudaError_t e = cudaFuncSetAttribute(k_fp4_linear<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const size_t smem2 = (size_t)C::STAGES2 * C::STAGE + 256;
    for (int s = 8; s >= 1; --s) c.of[s] = resident_clusters(k_fp4_linear<BN>, s, lin::THREADS, smem2);
    return c.of[1] ? cudaSuccess : cudaErrorInvalidConfiguration;
  });
  if (e != cudaSuccess) return e;
  // Clusters of s CTAs that the GPU holds at once, a CTA an SM: the occupancy call counts one of these kernels an SM
  // (152 76 46 36 28 23 15 15 of them on 152 SMs) though two have room and run (see the times by S above).
  const int* one = clusters_of->of;
  // Few tiles (under three quarters of the SMs): split the sum where the stages saved are worth adding the
  // parts.  Costs in stages, fitted to 148 sizes: clusters that do not all fit on SMs of their own share some, whose
  // stages take 1.65 times as long together; adding costs what a tile of 128 tokens writes and reads, less for fewer.
  //   us by S, parts loaded one token at a time:
  //             1 x 1024 -> 512    1: 3.2, 4: 3.4       128 x 1024 -> 512    1: 4.1, 2: 6.7
  //             1 x 4096 -> 5120   3: 4.8, 6: 4.8       777 x 4128 -> 1000   2: 9.7, 5: 10.5
  //           500 x 8192 -> 1000   4: 8.3, 7: 10.1      384 x 8192 -> 2560   2: 12.3, 4: 10.8
  //            32 x 8192 -> 2560   5: 5.6, 8: 6.1
  // More tiles than SMs: two CTAs an SM.
  int S = 1;
  if (4 * tiles <= 3 * one[1]) {
    float best = FLT_MAX;
    for (int s = 1; s <= 8 && (s == 1 || 2 * s <= nkb); ++s) {
      if (tiles > 2 * one[s]) continue;
      const bool shared = tiles > one[s];
      const float stages = (shared ? 1.65f : 1.f) * nkb / s + (shared ? 2.1f * BN / 128 : 0.f);
      const float cost = stages + (s > 1 ? 3.f + BN / 32.f + s * BN * (0.3f / 128) : 0.f);
      if (cost < best) best = cost, S = s;
    }
  }
  p.stages = S == 1 && tiles <= one[1] ? C::STAGES : C::STAGES2;
  p.tmem_cols = 128;
  while (p.tmem_cols < C::DCOLS + p.stages * C::SFCOLS) p.tmem_cols *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ft * S), (unsigned)tt);
  cfg.blockDim = lin::THREADS;
  cfg.dynamicSmemBytes = (size_t)p.stages * C::STAGE + 256;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_fp4_linear<BN>, mw, mx, p);
}

}  // namespace

cudaError_t launch_fp4_linear(const csa2_fp4_linear_args& a, cudaStream_t st) {
  if (a.x.rows == 0 || a.w.rows == 0) return cudaSuccess;
  const int T = a.x.rows, nkb = (a.x.cols + 255) / 256, ft = (a.w.rows + 127) / 128;
  if (T <= 16) return launch_linear<16>(a, st);
  if (T <= 32) return launch_linear<32>(a, st);
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // 33 to 256 tokens, sums that split over two pairs or more (36 clusters of four CTAs run at once on 152 SMs, hence nine
  // nineteenths of the SMs in feature tiles): what a CTA can take in is the bound, and a pair's CTAs take in half of the tokens each.  Single CTAs split eight
  // ways below 16 feature tiles, and start and end sooner, which decides short sums.  us, single CTAs or
  // wide pairs against pairs on few tokens:
  //    64 x  4096 -> 2560   6.7   5.4      64 x  8192 -> 5120   7.9  7.8      64 x 32768 -> 5120  19.9 20.3
  //   128 x  2560 -> 5120   6.3   6.7     128 x  3584 -> 5120   8.9  7.0     128 x 32768 -> 5120  22.7 21.6
  //   192 x  2048 -> 5120   5.6   7.4     192 x  5120 -> 5120   9.6  8.6     192 x 32768 -> 5120  26.0 23.3
  //   256 x  4096 -> 5120   8.8   9.4     256 x  8192 -> 5120  11.9 11.3     192 x 32768 -> 512   10.9 15.5
  if (T <= 256 && ft >= 16 && ft <= sms * 9 / 19 && nkb >= (T <= 128 ? 14 : 18) && (T > 64 || nkb <= 32)) {
    if (T <= 64) return launch_linear_few<64>(a, st);
    if (T <= 128) return launch_linear_few<128>(a, st);
    return T <= 192 ? launch_linear_few<192>(a, st) : launch_linear_few<256>(a, st);
  }
  if (T <= 64) return launch_linear<64>(a, st);
  // Single CTAs while their 128 x 128 tiles run at once, two on an SM, and a CTA's share of the sum is
  // short: they start and end in 3 us, pairs in 5 to 6 us (and 3 us more where they split the sum), but
  // a pair does 256 x 256 in little more time than a CTA its 128 x 128.  us, single against pairs:
  //   384 x 1024 -> 5120 (120 tiles, 4 stages)   4.4  6.5      384 x 8192 -> 5120 (32 stages)  15.3  15.7
  //   384 x 16384 -> 5120 (64 stages)            27.3 25.6     768 x 4096 -> 5120 (240, 16)    10.6  11.0
  //   192 x 16384 -> 5120 (80, 64)               17.7 17.7     192 x 32768 -> 5120 (80, 128)   28.3  26.1
  const long long tiles = (T + 127LL) / 128 * ft;
  if (T <= 128 || (tiles <= 2 * sms && tiles * nkb <= 32LL * sms)) return launch_linear<128>(a, st);
  const bool tma = ((uintptr_t)a.out & 15) == 0 && (long long)a.w.rows * (a.out_dtype == CSA2_F32 ? 4 : 2) % 16 == 0;
  return tma ? launch_linear_pair<true>(a, st) : launch_linear_pair<false>(a, st);
}

uint32_t read_clear_error_fp4() {
  unsigned int v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_err_fp4, sizeof(v));
  if (v) cudaMemcpyToSymbol(g_err_fp4, &z, sizeof(z));
  return v;
}

}  // namespace csa2

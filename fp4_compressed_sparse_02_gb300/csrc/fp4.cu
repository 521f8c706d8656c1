// FP4 rows: the quantiser (csa2_fp4_quant) and the product with FP4 weights (csa2_fp4_linear).
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
  bool x32, vx;
};

constexpr int kQuantTiles = 4;   // column tiles (of 64 columns) of a CTA

}  // namespace

// CTA = 128 rows x 4 column tiles, 256 threads: half a warp takes 16 groups (256 columns) of a
// row, so codes leave in 128-byte runs; the scale bytes meet in shared memory and leave as
// whole 512-byte tiles, zero where there is no row or column.
__global__ void __launch_bounds__(256) k_fp4_quant(QuantRowsParams p) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint4 tile[kQuantTiles * 32];
  const int tid = threadIdx.x;
  if (tid < kQuantTiles * 32) tile[tid] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  const int nct = (p.nkt + kQuantTiles - 1) / kQuantTiles;
  const int rt = blockIdx.x / nct, r0 = rt * 128, kt0 = (blockIdx.x % nct) * kQuantTiles;
  const int rows = min(128, p.T - r0);
  const int g = tid & 15, c = kt0 * 4 + g;                // the thread's 16-column group
  if (16 * c < p.K) {
    const float gs = p.gscale ? __ldg(p.gscale) : 1.f;
#pragma unroll 2
    for (int r = tid >> 4; r < rows; r += 16) {
      const long long row = r0 + r;
      float u[16];
      load16(u, p.x, row * p.sx + 16 * c, p.x32, p.vx, 16);
      if (p.gscale) {
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i] = __fdiv_rn(u[i], gs);
      }
      uint32_t w0, w1, sb;
      fp4_encode16(u, w0, w1, sb);
      *reinterpret_cast<uint2*>(p.codes + row * (p.K / 2) + 8 * c) = make_uint2(w0, w1);
      reinterpret_cast<uint8_t*>(tile)[fp4_scale_offset(r, g, kQuantTiles)] = (uint8_t)sb;
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
  p.x32 = a.x_dtype == CSA2_F32;
  p.vx = ((uintptr_t)a.x & 15) == 0 && (p.T == 1 || (a.x_stride * (p.x32 ? 4 : 2)) % 16 == 0);
  const long long grid = (long long)((p.nkt + kQuantTiles - 1) / kQuantTiles) * ((p.T + 127) / 128);
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_k(k_fp4_quant, (unsigned)grid, 256, 0, st, p);
}

// ---------------------------------------------------------------------------------
// Product
// ---------------------------------------------------------------------------------
namespace lin {

constexpr int BM = 128;                    // weight rows (output features) of a tile: TMEM lanes
constexpr int BKB = 128;                   // bytes of codes per row and stage: 256 columns
constexpr int THREADS = 192;               // warps 0..3 epilogue, 4 loads, 5 products
constexpr uint32_t MAX_POLL = 1u << 24;

template <int BN>                          // tokens of a tile: TMEM columns
struct Cfg {
  static constexpr int XATOMS = (BN + 127) / 128;                  // 128-row scale tiles of x
  static constexpr int A = BM * BKB, B = BN * BKB, SFA = 4 * 512, SFB = XATOMS * 4 * 512;
  static constexpr int STAGE = A + B + SFA + SFB;
  static constexpr int STAGES = (212 * 1024) / STAGE < 9 ? (212 * 1024) / STAGE : 9;
  static constexpr int SMEM = STAGES * STAGE + 256;
  static constexpr int DCOLS = BN < 32 ? 32 : BN;
  // two sets of scale columns: 4 per 64-column step for w, 4 per step and atom for x
  static constexpr int SFCOLS = 16 + 16 * XATOMS;
  static constexpr int COLS = DCOLS + 2 * SFCOLS <= 128 ? 128 : DCOLS + 2 * SFCOLS <= 256 ? 256 : 512;
  static_assert(B % 1024 == 0 && STAGE % 1024 == 0, "operand tiles start on 1024-byte boundaries");
};

struct Params {
  const uint8_t* wt;                       // scale tiles of the weights
  const uint8_t* xt;                       // scale tiles of x
  const float* gx;
  const float* gw;
  void* out;
  int T, N, nkt;
  bool out32;
};

// Instruction descriptor of kind::mxf4nvf4: E2M1 operands (1), both K-major, E4M3 scales (0),
// M x N x 64.
__host__ __device__ constexpr uint32_t idesc(int M, int N) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Shared-memory descriptor of one scale tile: 8-row groups of 16-byte rows, 128 bytes apart,
// no swizzle.
__device__ __forceinline__ uint64_t sf_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

// One 512-byte scale tile into four TMEM columns (column j, lane l: the four scales of row
// 32 j + l), repeated for the four lane quarters.
__device__ __forceinline__ void sf_copy(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(tmem), "l"(desc) : "memory");
}

__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}"
      :: "r"(d), "l"(a), "l"(b), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
}

__device__ __forceinline__ float4 ld_dsmem_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

__device__ __forceinline__ void put(const Params& p, long long at, float v) {
  if (p.out32)
    static_cast<float*>(p.out)[at] = v;
  else
    static_cast<uint16_t*>(p.out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

}  // namespace lin

// Tile = 128 features x BN tokens of out^T = w x^T, so that few tokens fill the N side of the
// product and the weights stream through the M side.  A cluster of S CTAs splits the sum over
// K; each leaves its float32 partial in shared memory and the CTAs add them in rank order.
template <int BN>
__global__ void __launch_bounds__(lin::THREADS, 1)
    k_fp4_linear(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx, lin::Params p) {
  using namespace lin;
  using C = Cfg<BN>;
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE);
  uint64_t* empty = full + C::STAGES;
  uint64_t* accf = empty + C::STAGES;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(accf + 1);
  volatile int* failed = reinterpret_cast<volatile int*>(accf + 2);
  const int S = (int)gridDim.x / ((p.N + BM - 1) / BM);   // CTAs of a cluster
  const int rank = blockIdx.x % S;
  const int f0 = (blockIdx.x / S) * BM, t0 = blockIdx.y * BN;
  const int nkb = (p.nkt + 3) / 4;
  const int kb0 = (int)((long long)nkb * rank / S), kb1 = (int)((long long)nkb * (rank + 1) / S);
  // the same in every CTA; the barriers of a cluster are reached either way
  const bool aligned = (smem_u32(smem) & 1023) == 0;
  if (warp == 5) tc::tmem_alloc(tslot, C::COLS);
  if (tid == 0) {
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
  const uint32_t tb = *tslot;
  const int xa0 = t0 >> 7;                                // first scale tile row of the tokens
  const int xatoms = min(C::XATOMS, ((p.T + 127) >> 7) - xa0);
  int issued = kb0;                                       // loads of [kb0, issued) are on their way
  if (warp == 4) {
    if (lane == 0 && aligned) {
      for (int kb = kb0; kb < kb1; ++kb) {
        const int it = kb - kb0, s = it % C::STAGES;
        if (it >= C::STAGES && !tc::mbar_wait(&empty[s], (uint32_t)((it / C::STAGES - 1) & 1), MAX_POLL)) {
          raise_error(&g_err_fp4, CSA2_DEVERR_TIMEOUT);
          *failed = 1;
          break;
        }
        uint8_t* st = smem + s * C::STAGE;
        const int nt = min(4, p.nkt - 4 * kb);            // 64-column steps of this stage
        tc::mbar_arrive_expect_tx(&full[s], (uint32_t)(C::A + C::B + nt * 512 * (1 + xatoms)));
        tc::tma_load_2d(st, &mw, kb * BKB, f0, &full[s]);
        tc::tma_load_2d(st + C::A, &mx, kb * BKB, t0, &full[s]);
        uint8_t* sf = st + C::A + C::B;
        tc::bulk_load(sf, p.wt + ((long long)(f0 >> 7) * p.nkt + 4 * kb) * 512, nt * 512, &full[s]);
        for (int j = 0; j < xatoms; ++j)
          tc::bulk_load(sf + C::SFA + j * 2048, p.xt + ((long long)(xa0 + j) * p.nkt + 4 * kb) * 512, nt * 512, &full[s]);
        issued = kb + 1;
      }
    }
  } else if (warp == 5) {
    if (lane == 0 && aligned) {
      constexpr uint32_t id = idesc(BM, BN);
      const uint32_t sf0 = tb + C::DCOLS;
      // tokens that start inside a 128-row scale tile start at a later column of it
      const uint32_t xcol = (uint32_t)((t0 & 127) >> 5);
      for (int kb = kb0; kb < kb1; ++kb) {
        const int it = kb - kb0, s = it % C::STAGES;
        if (!tc::mbar_wait(&full[s], (uint32_t)((it / C::STAGES) & 1), MAX_POLL)) {
          raise_error(&g_err_fp4, CSA2_DEVERR_TIMEOUT);
          *failed = 1;
          break;
        }
        tc::fence_after_sync();
        const uint32_t a = smem_u32(smem + s * C::STAGE), b = a + C::A, sf = b + C::B;
        const uint32_t sft = sf0 + (it & 1) * C::SFCOLS;
        const int nt = min(4, p.nkt - 4 * kb);
        for (int k = 0; k < nt; ++k) {
          sf_copy(sft + 4 * k, sf_desc(sf + 512 * k));
#pragma unroll
          for (int j = 0; j < C::XATOMS; ++j)
            sf_copy(sft + 16 + 4 * (C::XATOMS * k + j), sf_desc(sf + C::SFA + 2048 * j + 512 * k));
        }
        for (int k = 0; k < nt; ++k)
          mma_fp4(tb, tc::smem_desc_sw128(a + 32 * k, 16, 1024), tc::smem_desc_sw128(b + 32 * k, 16, 1024), id,
                  sft + 4 * k, sft + 16 + 4 * C::XATOMS * k + xcol, (it | k) != 0 ? 1u : 0u);
        tc::mma_commit(&empty[s]);
      }
      tc::mma_commit(accf);
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
    for (int kb = issued - min(issued - kb0, C::STAGES); kb < issued; ++kb)
      tc::mbar_wait(&full[(kb - kb0) % C::STAGES], (uint32_t)(((kb - kb0) / C::STAGES) & 1), MAX_POLL);
  }
  const int nt = min(BN, p.T - t0);                       // tokens that exist
  const float alpha = (p.gx ? __ldg(p.gx) : 1.f) * (p.gw ? __ldg(p.gw) : 1.f);
  if (warp < 4 && !bad) {
    const uint32_t tq = tb + ((uint32_t)(32 * warp) << 16);
    const int f = 32 * warp + lane;
    float* part = reinterpret_cast<float*>(smem);
#pragma unroll 1
    for (int c = 0; c < nt; c += 32) {
      uint32_t v[32];
      tc::tmem_ld32(tq + (uint32_t)c, v);
      tc::tmem_ld_wait();
      if (S > 1) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c + i < nt) part[(c + i) * BM + f] = __uint_as_float(v[i]);
      } else if (f0 + f < p.N) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c + i < nt) put(p, (long long)(t0 + c + i) * p.N + f0 + f, __uint_as_float(v[i]) * alpha);
      }
    }
  }
  __syncwarp();
  if (S > 1) {
    tc::cluster_sync();
    if (warp < 4 && !bad) {
      const uint32_t mine = smem_u32(smem);
      for (int u = rank * 128 + tid; u < nt * (BM / 4); u += S * 128) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q = 0; q < S; ++q) {
          const float4 v = ld_dsmem_f4(tc::mapa(mine, q) + 16 * u);
          s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        const int t = u / (BM / 4), f = f0 + 4 * (u % (BM / 4));
        const float e[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (f + i < p.N) put(p, (long long)(t0 + t) * p.N + f + i, e[i] * alpha);
      }
    }
    __syncwarp();
    tc::cluster_sync();                                   // peers have read this CTA's partial
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 5) tc::tmem_dealloc(tb, C::COLS);
}

namespace {

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
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int ft = (p.N + lin::BM - 1) / lin::BM, tt = (p.T + BN - 1) / BN, nkb = (p.nkt + 3) / 4;
  // few tiles: split the sum until the tiles fill the GPU, each CTA keeping two stages or more
  int S = 1;
  while (S < 8 && 2LL * S * ft * tt <= sms && 4 * S <= nkb) S *= 2;
  static bool attr_set = false;
  if (!attr_set) {
    cudaError_t e = cudaFuncSetAttribute(k_fp4_linear<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    attr_set = true;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ft * S), (unsigned)tt);
  cfg.blockDim = lin::THREADS;
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_fp4_linear<BN>, mw, mx, p);
}

}  // namespace

cudaError_t launch_fp4_linear(const csa2_fp4_linear_args& a, cudaStream_t st) {
  if (a.x.rows == 0 || a.w.rows == 0) return cudaSuccess;
  const int T = a.x.rows;
  if (T <= 16) return launch_linear<16>(a, st);
  if (T <= 32) return launch_linear<32>(a, st);
  if (T <= 64) return launch_linear<64>(a, st);
  if (T <= 128) return launch_linear<128>(a, st);
  return launch_linear<256>(a, st);
}

uint32_t read_clear_error_fp4() {
  unsigned int v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_err_fp4, sizeof(v));
  if (v) cudaMemcpyToSymbol(g_err_fp4, &z, sizeof(z));
  return v;
}

}  // namespace csa2

// Attention over the paged 8-bit cache for many rows (csa2_kv8_attn): tiles of rows on the tcgen05 tensor cores.
//
// S = Q K^T and O += P V with float32 accumulators in TMEM, 128 tokens a step.  The keys' bytes are the operand as
// they come from memory: Q, scaled by a power of two, is the sum of two E4M3 values, exactly for every bf16 within 2^-9
// of its row's largest and to 2^-17 of the largest below that.  P is fp16, and the values' bytes become
// fp16 (exact) once a step, by warps of their own.  Two groups of rows take turns: one's softmax runs
// under the other's products.
//
// 256 rows and 128 tokens are 67 MFLOP, 2080 cycles of the tensor core; a step takes some 3300: a group's chain of scores
// (products, wake-up, TMEM loads, maximum, exponentials, weights) lasts longer than the other group's products.  4096 new
// tokens at 32K and a fresh prompt, 64 heads of 128: 3.2 to 3.4 ms (the longer one after the other, into the power cap), 1.27 to
// 1.33 PFLOP/s, 0.65 to 0.68 of the measured peak; 32 x 6 tokens at 8K to 32K, 48 rows: 274 us, 0.73 of the copy rate.
#include "kv8_attn.cuh"
#include "kv8_order.h"

namespace csa2 {

CSA2_DEFINE_ERROR_WORD(g_err_kv8_tile);

namespace {

// Warps 0: TMA; 1 and 2: the products of group 0 and 1; 4-7 and 8-11: the softmax of group 0 and 1 (a row tile, or the
// even and odd steps, see SPLIT), a row a thread; 12-15: values to fp16.  The warps that must not be late come first: a
// scheduler prefers its older warps.  The softmax keeps a row of scores in registers, which the others give up.
constexpr int kStep = 128, kThreads = 512, kLoad = 0, kMma = 1, kSoftmax = 4, kConvert = 12;
constexpr int kSoftmaxRegs = 184, kOtherRegs = 72;           // 256 threads each: 65,536, what 512 threads of 128 are launched with
constexpr int kInfo = 8;                 // steps whose scales are kept: more than can be under way
constexpr int kRing = 3;                 // steps of bytes under way
constexpr uint32_t kPollNs = 200, kTilePolls = 1u << 20;    // (a poll without a limit wakes late: 5 % at 4096 new tokens)
// Steps of a group whose sums are taken by themselves.  The tensor core drops what lies below the last bit of a sum, so that O
// would be too small by 1e-7 for each of a step's eight products (by 0.7 % after a million tokens), and a sum of weights
// near 1 leaves no room for small ones.  A run's O is off by 2^-12 at most.  4096 new tokens at 32K: 3.35 ms, as without
// runs; 3.43 with runs of 128 steps, 3.69 of 64 (before both ends of a run shared their code).
constexpr int kRun = 256;
// Weights are 2^kWeight times exp2(logit - top), and the maximum is up to 2^kFollow above top: together within fp16, which
// reaches down to 2^-36 of a weight at top.  top is rounded, the product in x f - top is not: for logits below 2^28 (base 2),
// whose units are 16 at most, the sums below are rounded so that a weight stays within 2^15.5 and the largest above
// 2^-8.  Beyond, a row is NaN; rounding the products first cost 3 to 10 % of 4096 new tokens at 32K.
constexpr float kWeight = 11.f, kFollow = 4.f, kWeightUndo = 1.f / 2048.f, kMostLogit = 268435456.f;
constexpr int kOver = 12;                // what beginning a stream costs, in steps
constexpr int kCopy = 2047;              // sequences whose starts and lengths the plan copies

template <int D>
struct Smem {
  static constexpr int kRaw = kStep * D, kQ = 2 * 128 * D, kF = kStep * D * 2;
  static constexpr int kK = 2 * kQ, kV = kK + kRing * kRaw, kVf = kV + kRing * kRaw, kBytes = kVf + 2 * kF;
};

// A stream of a slot: one tile of rows of a sequence, against the steps [step, step + count).
struct Slot {
  Rows rows;
  int s, r0, n;                          // sequence, first row of the tile, rows; n = 0: an empty slot
  int lo, hi;                            // what any row sees
  int lo_max, hi_min;                    // what all rows see
  int step, count;
};

struct Shared {
  uint64_t k_full[kRing], k_empty[kRing], v_full[kRing], v_empty[kRing], vf_full[2], vf_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2], turn[2], q_full, done;
  float2 ks[kInfo], vs[kInfo];           // scales of a step's two pages; -1: not there
  float2 ml[128];                        // SPLIT: the second group's maximum and sum
  float unit[4];                         // of the last segments: the largest value scale
  int nan[4];                            // a NaN value that only some rows see was taken out
  float top[4];
  long long scan[kThreads / 32];
  long long total, begin;                // of the plan: all streams' cost, that before `slot`
  int slot, dead;
  Slot first;                            // slot `slot`
  uint32_t tmem;
};

// Shared-memory descriptor of a K-major operand in 8 bits, rows of D bytes swizzled over their width.
template <int D>
__device__ __forceinline__ uint64_t desc8(uint32_t saddr) {
  uint64_t d = tc::smem_desc_sw128(saddr, 16, 8 * D);
  if constexpr (D == 64) d += (uint64_t)2 << 61;             // SWIZZLE_64B
  return d;
}

// E4M3 operands, float32 accumulators.
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}"
      :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// One thread of a warp whose threads are together.  The compiler knows that it is one, keeps the products' operands in
// uniform registers and issues a product in a few instructions; behind `lane == 0` it takes several times as many, and
// the warp, which shares its scheduler with two busy softmax warps, falls behind the tensor core (4096 new tokens at 32K:
// 6.1 ms).
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred P;\n elect.sync _|P, 0xffffffff;\n selp.u32 %0, 1, 0, P;\n}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void sts64(uint32_t a, uint2 v) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" :: "r"(a), "r"(v.x), "r"(v.y) : "memory");
}

// A whole 32-byte sector of one thread's own row, and back.
__device__ __forceinline__ void stg256(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
}

__device__ __forceinline__ void ldg256(const void* p, float* v) {
  asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]) : "l"(p) : "memory");
}

__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

// A bounded wait of one thread.  After one has given up, all others of the CTA do
// at once: every role still goes through its loops, so the kernel ends.
__device__ __forceinline__ bool await(uint64_t* bar, uint32_t parity, Shared& m) {
  const uint32_t at = smem_u32(bar);
  uint32_t done, polls = 0;
  while (true) {
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done) : "r"(at), "r"(parity), "r"(kPollNs) : "memory");
    if (done) return true;
    if (*(volatile int*)&m.dead) return false;
    if (++polls == kTilePolls) {
      *(volatile int*)&m.dead = 1;
      raise_error(&g_err_kv8_tile, CSA2_DEVERR_TIMEOUT);
      return false;
    }
  }
}

// The same by every thread of a warp, which are together again after it.
__device__ __forceinline__ void await_warp(uint64_t* bar, uint32_t parity, Shared& m) {
  await(bar, parity, m);
  __syncwarp();
}

// The wait for loads from TMEM, as a step that their values pass through.
__device__ __forceinline__ void tmem_arrived(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :: "memory");
}

// ---- the work --------------------------------------------------------------------------------

// Slot floor(start * G / RT) + s and the ones after it hold the row tiles of sequence s.
template <int RT>
__device__ __forceinline__ long long first_slot(const Kv8Params& p, const int* start, int s) {
  const int x = start[s];
  return (long long)(x < 0 ? 0 : x > p.a.T ? p.a.T : x) * p.G / RT + s;
}

template <int RT>
__device__ __forceinline__ int slots_of(const Kv8Params& p) { return (int)((long long)p.a.T * p.G / RT) + p.a.S; }

// Slot `slot`, of a sequence from s on; start and length: the step's, or a copy.
template <int RT>
__device__ __forceinline__ Slot slot_of(const Kv8Params& p, const int* start, const int* length, int s, int slot) {
  const csa2_kv8_attn_args& a = p.a;
  Slot t = {};
  while (s + 1 < a.S && first_slot<RT>(p, start, s + 1) <= slot) ++s;
  t.s = s;
  t.rows.t0 = start[s];
  t.rows.end = start[s + 1];
  t.rows.length = length[s];
  const int e = min(t.rows.end, a.T);
  t.rows.n = t.rows.t0 >= 0 && e > t.rows.t0 ? (e - t.rows.t0) * p.G : 0;
  const long long r0 = (slot - first_slot<RT>(p, start, s)) * RT;
  if (r0 < 0 || r0 >= t.rows.n) return t;
  t.r0 = (int)r0;
  t.n = min(RT, t.rows.n - t.r0);
  const int limit = a.cache.max_pages * kPage;
  auto seen = [&](int r) {               // positions up to which row r sees, as if the table had no end
    return (long long)t.rows.length - ((long long)t.rows.end - (t.rows.t0 + r / p.G)) + 1;
  };
  auto clamp = [&](long long x) { return (int)(x < 0 ? 0 : x > limit ? limit : x); };
  const long long from = seen(t.r0), to = seen(t.r0 + t.n - 1);
  t.hi_min = clamp(from);
  t.hi = clamp(to);
  t.lo = a.window > 0 ? clamp(from - a.window) : 0;
  t.lo_max = a.window > 0 ? clamp(to - a.window) : 0;
  if (from < 1 || to > limit) t.hi_min = 0;                // rows outside the table see nothing
  t.step = t.lo / kStep;
  t.count = (t.hi + kStep - 1) / kStep - t.step;
  if (t.count < 1) t.count = 1;          // rows that see nothing are written all the same
  return t;
}

// What a slot's stream costs, in steps.
__device__ __forceinline__ int cost_of(const Slot& t) { return t.count > 0 ? t.count + kOver : 0; }

// A CTA's span of all streams' cost (slot by slot, head by head), walked by every role alike.  A cut within a stream's
// first kOver units is a cut before its first step.
template <int RT>
struct Walk {
  Slot t;
  int slot, h, x, take;                  // the segment: steps x .. x + take of the stream
  int spent;                             // its cost
  long long left;                        // cost of the span that is still to come, with the segment's
  int n;                                 // segments before this one

  __device__ __forceinline__ void cut(int at) {              // at: cost of the stream that earlier spans have
    const int rest = cost_of(t) - at;
    spent = (int)(rest < left ? rest : left);
    x = max(0, at - kOver);
    take = max(0, at + spent - kOver) - x;
  }
  __device__ __forceinline__ Walk(const Kv8Params& p, const Shared& m, long long per) {
    const long long begin = blockIdx.x * per;
    left = m.total - begin < per ? m.total - begin : per;
    n = 0;
    if (left <= 0) return;
    slot = m.slot;
    t = m.first;
    const long long rel = begin - m.begin;
    h = (int)(rel / cost_of(t));
    cut((int)(rel % cost_of(t)));
    if (take == 0) {
      n = -1;
      next(p);
    }
  }
  __device__ __forceinline__ bool on() const { return left > 0; }
  __device__ __forceinline__ void next(const Kv8Params& p) {
    ++n;
    do {
      left -= spent;
      if (left <= 0) return;
      if (++h == p.a.cache.Hkv) {
        h = 0;
        do {
          if (++slot >= slots_of<RT>(p)) {                   // only if `start` does not ascend
            left = 0;
            return;
          }
          t = slot_of<RT>(p, p.a.start, p.a.length, t.s, slot);
        } while (t.count == 0);
      }
      cut(0);
    } while (take == 0);
  }
  __device__ __forceinline__ bool begins() const { return x == 0; }
  __device__ __forceinline__ bool ends() const { return x + take == t.count; }
};

// RT: rows of a stream.  256: the groups are two tiles of 128 rows that share every step.  128 and 64 (SPLIT): the groups
// have the same rows, one the even steps and one the odd ones, and are added up at the end of a segment.  At 64 rows two
// threads of a softmax warp share a row (M = 64 puts 16 rows into each quarter of the TMEM lanes), half the columns each.
template <int D, int RT>
__global__ void __launch_bounds__(kThreads, 1)
k_kv8_tile(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const Kv8Params p) {
  constexpr bool SPLIT = RT < 256;
  constexpr int kM = RT == 64 ? 64 : 128, kCols = kStep * kM / 128, kDims = D * kM / 128;   // scores and channels of a thread
  using L = Smem<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Shared m;
  const csa2_kv8_attn_args& a = p.a;
  const csa2_kv8_cache& c = a.cache;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = p.G;
  const uint32_t base = smem_u32(smem);
  if ((base & 1023) != 0) {              // uniform: the swizzles count on it
    if (tid == 0) raise_error(&g_err_kv8_tile, CSA2_DEVERR_SMEM_ALIGN);
    return;
  }
  if (warp == kMma) tc::tmem_alloc(&m.tmem, 512);
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      tc::mbar_init(&m.k_full[i], 1);
      tc::mbar_init(&m.k_empty[i], SPLIT ? 1 : 2);
      tc::mbar_init(&m.v_full[i], 1);
      tc::mbar_init(&m.v_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&m.vf_full[i], 4);
      tc::mbar_init(&m.vf_empty[i], SPLIT ? 1 : 2);
      tc::mbar_init(&m.s_full[i], 1);
      tc::mbar_init(&m.p_full[i], 4);
      tc::mbar_init(&m.o_full[i], 1);
      tc::mbar_init(&m.turn[i], 1);
    }
    tc::mbar_init(&m.q_full, SPLIT ? 4 : 8);
    tc::mbar_init(&m.done, 2);
    m.dead = 0;
  }
  pdl_wait();
  pdl_trigger();

  // ---- the plan: steps of all slots, and the slot in which this CTA's span begins
  const int slots = slots_of<RT>(p);
  const int chunk = (slots + kThreads - 1) / kThreads;
  const int c0 = min(slots, tid * chunk), c1 = min(slots, c0 + chunk);
  const int *start = a.start, *length = a.length;
  if (a.S <= kCopy) {                    // into the ring, which is empty yet
    int* copy = reinterpret_cast<int*>(smem + L::kK);
    for (int i = tid; i <= a.S; i += kThreads) {
      copy[i] = a.start[i];
      if (i < a.S) copy[kCopy + 1 + i] = a.length[i];
    }
    start = copy;
    length = copy + kCopy + 1;
  }
  __syncthreads();
  int s0 = 0;                            // the sequence of slot c0
  for (int end = a.S; end - s0 > 1;) {
    const int mid = (s0 + end) >> 1;
    if (first_slot<RT>(p, start, mid) <= c0) s0 = mid; else end = mid;
  }
  long long mine = 0;
  for (int i = c0, s = s0; i < c1; ++i) {
    const Slot t = slot_of<RT>(p, start, length, s, i);
    s = t.s;
    mine += cost_of(t);
  }
  mine *= c.Hkv;
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) m.scan[warp] = inc;
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  long long total = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) inc += m.scan[i];
    total += m.scan[i];
  }
  const long long even = (total + kTileSpans - 1) / kTileSpans, per = even > kOver + 2 ? even : kOver + 2;
  const long long begin = blockIdx.x * per;
  if (tid == 0) m.total = total;
  if (begin < total && inc > begin && inc - mine <= begin) {
    long long at = inc - mine;
    Slot t = slot_of<RT>(p, start, length, s0, c0);
    int i = c0;
    while (i < c1 - 1 && at + (long long)cost_of(t) * c.Hkv <= begin) {
      at += (long long)cost_of(t) * c.Hkv;
      t = slot_of<RT>(p, start, length, t.s, ++i);
    }
    m.slot = i;
    m.begin = at;
    m.first = t;
  }
  tc::fence_proxy_async_smem();          // the initialised barriers and the copy's end, for the copies to come
  __syncthreads();
  const uint32_t tb = m.tmem;

  if (warp < kSoftmax || warp >= kConvert) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kOtherRegs));
    Walk<RT> w(p, m, per);
    if (warp == kLoad) {
      // ---- TMA: the pages of each step, keys and values
      int step = 0;                      // steps so far
      for (; w.on(); w.next(p)) {
        const int pages = (w.t.hi + kPage - 1) / kPage, page0 = 2 * (w.t.step + w.x);
        int id = -1;                     // lane i: page page0 + 32 b + i
        float ks = -1.f, vs = -1.f;
        for (int j = 0; j < w.take; ++j, ++step) {
          if ((j & 15) == 0) {
            const int y = page0 + 2 * j + lane;
            id = y >= w.t.lo / kPage && y < pages && 2 * j + lane < 2 * w.take ? page_id(c, w.t.s, y, &g_err_kv8_tile) : -1;
            ks = vs = -1.f;
            if (id >= 0) {
              ks = c.k_scale[(long long)id * c.Hkv + w.h];
              vs = c.v_scale[(long long)id * c.Hkv + w.h];
            }
          }
          const int at = (j & 15) * 2, b = step % kRing;
          const uint32_t turn = (step / kRing & 1) ^ 1;
          const int id0 = __shfl_sync(0xffffffffu, id, at), id1 = __shfl_sync(0xffffffffu, id, at + 1);
          const float k0 = __shfl_sync(0xffffffffu, ks, at), k1 = __shfl_sync(0xffffffffu, ks, at + 1);
          const float v0 = __shfl_sync(0xffffffffu, vs, at), v1 = __shfl_sync(0xffffffffu, vs, at + 1);
          if (lane == 0) {
            const uint32_t bytes = ((id0 >= 0) + (id1 >= 0)) * (L::kRaw / 2);
            if (await(&m.k_empty[b], turn, m)) {
              m.ks[step % kInfo] = make_float2(k0, k1);
              m.vs[step % kInfo] = make_float2(v0, v1);
              uint8_t* dst = smem + L::kK + b * L::kRaw;
              tc::mbar_arrive_expect_tx(&m.k_full[b], bytes);
              if (id0 >= 0) tma_load_3d(dst, &mk, 0, 0, id0 * c.Hkv + w.h, &m.k_full[b]);
              if (id1 >= 0) tma_load_3d(dst + L::kRaw / 2, &mk, 0, 0, id1 * c.Hkv + w.h, &m.k_full[b]);
            }
            if (await(&m.v_empty[b], turn, m)) {
              uint8_t* dst = smem + L::kV + b * L::kRaw;
              tc::mbar_arrive_expect_tx(&m.v_full[b], bytes);
              if (id0 >= 0) tma_load_3d(dst, &mv, 0, 0, id0 * c.Hkv + w.h, &m.v_full[b]);
              if (id1 >= 0) tma_load_3d(dst + L::kRaw / 2, &mv, 0, 0, id1 * c.Hkv + w.h, &m.v_full[b]);
            }
          }
          __syncwarp();
        }
      }
      if (*(volatile int*)&m.dead && lane == 0)              // no copy outlives the CTA
        for (int i = 0; i < kRing; ++i)
          for (int back = 1; back <= kRing; ++back) {
            const int st = step - back;
            if (st < 0 || st % kRing != i) continue;
            tc::mbar_wait(&m.k_full[i], st / kRing & 1, kTilePolls / 64);
            tc::mbar_wait(&m.v_full[i], st / kRing & 1, kTilePolls / 64);
          }
    } else if (warp == kMma || warp == kMma + 1) {
      // ---- products, a warp a group: the weights' product with the values and, right after it, the scores of the group's
      // next step.  A product's issue lasts about as long as the product, so what a warp waits for is hidden behind
      // the other's.  The groups take turns: left alone they fall into step, both softmaxes and then both products
      // (4096 new tokens at 32K: 4.5 ms).
      constexpr uint32_t id_s = tc::idesc_f16(kM, kStep, 0, 0, 0), id_o = tc::idesc_f16(kM, D, 0, 0, 1);   // E4M3 is type 0, as fp16
      constexpr int kBy = SPLIT ? 2 : 1;
      const int grp = warp - kMma;
      const uint64_t q_desc = desc8<D>(base + (SPLIT ? 0 : grp * L::kQ)), k_desc = desc8<D>(base + L::kK);
      const uint64_t v_desc = tc::smem_desc_sw128(base + L::kVf, 16384, 1024);
      const uint32_t s_at = tb + grp * 128, o_at = tb + 256 + grp * 128;
      int step = 0;                      // of the segment's first
      uint32_t ps = 0, turns = 0;        // parity of the weights, turns had
      auto scores = [&](int st) {
        const uint64_t kb = k_desc + (uint32_t)(st % kRing * (L::kRaw >> 4));
#pragma unroll
        for (int i = 0; i < D / 16; ++i)                     // Q's first part, then its second
          mma_f8_ss(s_at, q_desc + (i / (D / 32) * (128 * D) + i % (D / 32) * 32) / 16, kb + i % (D / 32) * 2, id_s, i > 0);
        tc::mma_commit(&m.s_full[grp]);
        tc::mma_commit(&m.k_empty[st % kRing]);
      };
      for (; w.on(); w.next(p)) {
        product_order<kBy, kRun>(
            grp, step, w.take, [&] { await_warp(&m.q_full, w.n & 1, m); },
            [&](int st) { await_warp(&m.k_full[st % kRing], st / kRing & 1, m); },
            [&](int st) {
              tc::fence_after_sync();
              if (elect()) scores(st);
              __syncwarp();
            },
            [&](int st) { await_warp(&m.vf_full[st & 1], st >> 1 & 1, m); },
            [&] { await_warp(&m.turn[grp], (turns++ & 1) ^ (grp ? 0 : 1), m); },
            [&] {
              await_warp(&m.p_full[grp], ps, m);
              ps ^= 1;
            },
            [&](int st, bool add, bool out, bool on) {
              tc::fence_after_sync();
              if (elect()) {
                const uint64_t vb = v_desc + (uint32_t)((st & 1) * (L::kF >> 4));
#pragma unroll
                for (int i = 0; i < kStep / 16; ++i)
                  tc::mma_f16_ts(o_at, s_at + i * 8, vb + i * (2048 / 16), id_o, add || i > 0);
                tc::mma_commit(&m.vf_empty[st & 1]);
                if (out) tc::mma_commit(&m.o_full[grp]);
                if (on) scores(st + kBy);
                tc::mbar_arrive(&m.turn[grp ^ 1]);
              }
              __syncwarp();
            },
            [&] {
              if (elect()) tc::mbar_arrive(&m.turn[grp ^ 1]);
              __syncwarp();
            });
        step += w.take;
      }
      if (*(volatile int*)&m.dead) {                         // nor a product
        if (elect()) tc::mma_commit(&m.done);
        tc::mbar_wait(&m.done, 0, kTilePolls);
      }
    } else if (warp >= kConvert) {
      // ---- values: E4M3 to fp16, a token a thread, into the product's layout (atoms of 64 channels x 128 tokens)
      const int r = tid - kConvert * 32;
      int step = 0;
      for (; w.on(); w.next(p)) {
        const Slot& t = w.t;
        // in units of the largest scale of the segment, times 2^-7: exact for scales down to 2^-22 of it
        float top = 0.f;
        const int y1 = min((t.hi + kPage - 1) / kPage, 2 * (t.step + w.x + w.take));
        for (int y = max(t.lo / kPage, 2 * (t.step + w.x)) + r; y < y1; y += 128) {
          const int id = ld_s32(c.page_table + (long long)t.s * c.max_pages + y);
          if (id >= 0 && id < c.num_pages) top = fmaxf(top, c.v_scale[(long long)id * c.Hkv + w.h]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) m.top[warp - kConvert] = top;
        named_sync(2, 128);
        top = fmaxf(fmaxf(m.top[0], m.top[1]), fmaxf(m.top[2], m.top[3]));
        if (!(top > 0.f && top < INFINITY)) top = 1.f;
        if (r == 0) {
          m.unit[w.n & 3] = top;
          m.nan[w.n & 3] = 0;
        }
        named_sync(2, 128);
        for (int j = 0; j < w.take; ++j, ++step) {
          const int token = (t.step + w.x + j) * kStep + r, b = step % kRing;
          const bool border = token < t.lo_max || token >= t.hi_min;         // not every row sees it
          const uint32_t raw = base + L::kV + b * L::kRaw + r * D, dst = base + L::kVf + (step & 1) * L::kF + r * 128;
          await_warp(&m.v_full[b], step / kRing & 1, m);
          uint4 x[D / 16];
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            if constexpr (D == 128) x[i] = lds128(raw + ((i ^ (r & 7)) << 4));
            else x[i] = lds128(raw + ((i ^ (r >> 1 & 3)) << 4));
          }
          const float2 vs = m.vs[step % kInfo];
          float f = r < kPage ? vs.x : vs.y;
          const bool there = f != -1.f && token < t.hi && token >= t.lo;
          f = there ? f * 128.f / top : 0.f;
          if (!there || border) {
            bool nan = false;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              uint32_t* v = reinterpret_cast<uint32_t*>(&x[i]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t at = e4m3x4_nans(v[e]);   // 1 in each NaN's byte
                v[e] = there ? v[e] & ~(at * 0xffu) : 0u;                     // `border`: rows get their NaNs at the end
                nan |= there && at != 0;
              }
            }
            if (nan) *(volatile int*)&m.nan[w.n & 3] = 1;
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&m.v_empty[b]);
          await_warp(&m.vf_empty[step & 1], (step >> 1 & 1) ^ 1, m);
          const __half2 f2 = __half2half2(__float2half_rn(f));
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[2 * e] = e4m3x2_lo_f16x2(v[e]);
              o[2 * e + 1] = e4m3x2_hi_f16x2(v[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&o[e]), f2);
              o[e] = *reinterpret_cast<const uint32_t*>(&y);
            }
            const uint32_t atom = dst + (i >> 2) * 16384;
            sts128(atom + ((((2 * i) & 7) ^ (r & 7)) << 4), make_uint4(o[0], o[1], o[2], o[3]));
            sts128(atom + ((((2 * i + 1) & 7) ^ (r & 7)) << 4), make_uint4(o[4], o[5], o[6], o[7]));
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&m.vf_full[step & 1]);
        }
      }
    }
  } else {
    // ---- softmax: a row a thread (kM = 64: two threads)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kSoftmaxRegs));
    Walk<RT> w(p, m, per);
    const int grp = (warp - kSoftmax) >> 2, half = kM == 64 ? lane >> 4 : 0;
    const int r = (warp & 3) * (kM / 4) + lane % (kM / 4);
    const uint32_t lanes = tb + ((uint32_t)(warp & 3) << 21), s_at = lanes + grp * 128, o_at = lanes + 256 + grp * 128;
    auto load_o = [&](uint32_t at, float* v) {               // 32 channels of this thread
      if constexpr (kM == 64) tc::tmem_ld16x2_32<kDims>(at, reinterpret_cast<uint32_t*>(v));
      else tc::tmem_ld32(at, reinterpret_cast<uint32_t*>(v));
    };
    auto store_o = [&](uint32_t at, const float* v) {
      if constexpr (kM == 64) {
        tc::tmem_st16x2_16<kDims>(at, reinterpret_cast<const uint32_t*>(v));
        tc::tmem_st16x2_16<kDims>(at + 16, reinterpret_cast<const uint32_t*>(v + 16));
      } else {
        tc::tmem_st32(at, reinterpret_cast<const uint32_t*>(v));
      }
    };
    constexpr int kBy = SPLIT ? 2 : 1;
    int step = 0, seen = 0, outs = 0;   // steps of earlier segments; scores, sums waited for
    Part part = {0, 0, 0, 0, 0};
    // Earlier runs' maximum, sum and O of a row: in its part's place, the second group's of a SPLIT in their own
    const bool aside = SPLIT && grp == 1;
    for (; w.on(); w.next(p)) {
      const Slot& t = w.t;
      const int row = (SPLIT ? 0 : grp * 128) + r;
      const bool real = row < t.n;
      int lo = 0, hi = INT_MAX;
      const int tok = real ? t.rows.t0 + (t.r0 + row) / G : 0, hq = real ? w.h * G + (t.r0 + row) % G : 0;
      if (real) seen_by(a, t.rows, tok, lo, hi, &g_err_kv8_tile);
      // The warp's rows of Q, kRows at a time: scaled by a power of two to below 2^8, as the sums of two E4M3 rows.
      // The next head's rows are asked for meanwhile.
      float mul = 0.f;
      {
        constexpr int kLanes = D / 8, kRows = 32 / kLanes, kAhead = kM / 4 / kRows < 8 ? kM / 4 / kRows : 8;   // lanes a row, rows at a time, loads ahead
        const int sub = lane % kLanes, ch = sub >> 1;
        const long long mine = real ? tok * a.q_stride_t + (long long)hq * a.q_stride_h : -1;
#pragma unroll 1
        for (int i0 = 0; i0 < kM / 4 / kRows; i0 += kAhead) {
          uint4 v[kAhead];
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const long long at = __shfl_sync(0xffffffffu, mine, (i0 + i) * kRows + lane / kLanes);
            v[i] = make_uint4(0, 0, 0, 0);
            if (at >= 0) {
              const uint16_t* q = a.q + at + sub * 8;
              if (p.aligned & 1) {
                v[i] = *reinterpret_cast<const uint4*>(q);
              } else {
                v[i].x = q[0] | (uint32_t)q[1] << 16;
                v[i].y = q[2] | (uint32_t)q[3] << 16;
                v[i].z = q[4] | (uint32_t)q[5] << 16;
                v[i].w = q[6] | (uint32_t)q[7] << 16;
              }
            }
          }
          // the largest magnitudes, as bits: infinities and NaNs are above all others; all rows' together, a step at a time
          uint32_t big[kAhead];
          float f[kAhead];
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            big[i] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) big[i] = max(big[i], max(u[e] << 16 & 0x7fffffffu, u[e] & 0x7fff0000u));
          }
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1)
#pragma unroll
            for (int i = 0; i < kAhead; ++i) big[i] = max(big[i], __shfl_xor_sync(0xffffffffu, big[i], o));
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            float undo;
            row_factor(__uint_as_float(big[i]), f[i], undo);
            f[i] *= 0.0078125f;
            const float back = __shfl_sync(0xffffffffu, undo * 128.f * (a.softmax_scale * kLog2e), lane % kRows * kLanes);
            if (lane % (kM / 4) / kRows == i0 + i) mul = back;
          }
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            if (SPLIT && grp == 1) continue;
            uint32_t h4[4], l4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 y = mul2(make_float2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xffff0000u)), make_float2(f[i], f[i]));
              h4[e] = cvt_e4m3x2(y.x, y.y);
              const uint32_t first = e4m3x2_to_f16x2((uint16_t)h4[e]);
              const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&first));
              l4[e] = cvt_e4m3x2(y.x - z.x, y.y - z.y);
            }
            uint2 hi8 = make_uint2(h4[0] | h4[1] << 16, h4[2] | h4[3] << 16), lo8 = make_uint2(l4[0] | l4[1] << 16, l4[2] | l4[3] << 16);
            if (big[i] >= 0x7f800000u) hi8 = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);   // an infinity makes its row NaN, as a NaN does
            const int qr = (warp & 3) * (kM / 4) + (i0 + i) * kRows + lane / kLanes;
            const uint32_t at = base + (SPLIT ? 0 : grp * L::kQ) + qr * D +
                                ((D == 128 ? ch ^ (qr & 7) : ch ^ (qr >> 1 & 3)) << 4) + (sub & 1) * 8;
            sts64(at, hi8);
            sts64(at + 128 * D, lo8);
          }
        }
        if (!SPLIT || grp == 0) {
          tc::fence_proxy_async_smem();
          tc::fence_before_sync();       // the last segment's TMEM reads
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&m.q_full);
        }
        if (mine >= 0 && w.h + 1 < c.Hkv) {
          const uint16_t* q = a.q + mine + G * a.q_stride_h;
#pragma unroll
          for (int i = 0; i < D; i += 64) asm volatile("prefetch.global.L2 [%0];" :: "l"(q + i));
        }
      }
      float top = -INFINITY, l = 0.f;
      bool any = false;                  // a step of this run has been added to O
      const int grp0 = SPLIT ? grp : 0;
      for (int j = grp0; j < w.take;) {
        const int end = min(w.take, j + kRun * kBy);
        for (; j < end; j += kBy) {
          await_warp(&m.s_full[grp], seen++ & 1, m);
          tc::fence_after_sync();
          const float2 ks = m.ks[(step + j) % kInfo];
          const int token0 = (t.step + w.x + j) * kStep;
          // positive, so that a masked score's -infinity stays one; a page that is not there is masked as a whole
          const float f0 = fmaxf(mul * (ks.x == -1.f ? 1.f : ks.x), 1.17549435e-38f);
          const float f1 = fmaxf(mul * (ks.y == -1.f ? 1.f : ks.y), 1.17549435e-38f);
          const bool border = __any_sync(0xffffffffu, token0 < lo || token0 + kStep > hi || ks.x == -1.f || ks.y == -1.f);
          const int from0 = ks.x == -1.f ? INT_MAX : lo - token0, from1 = ks.y == -1.f ? INT_MAX : lo - token0;
          const int to = hi == INT_MAX ? INT_MAX : hi - token0;
          float x[kCols];                  // of tokens 64 * half + ...
          if constexpr (kM == 64) {
            tc::tmem_ld16x2_32<64>(s_at, reinterpret_cast<uint32_t*>(x));
            tc::tmem_ld16x2_32<64>(s_at + 32, reinterpret_cast<uint32_t*>(x + 32));
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) tc::tmem_ld32(s_at + 32 * i, reinterpret_cast<uint32_t*>(x + 32 * i));
          }
#pragma unroll
          for (int i = 0; i < kCols / 32; ++i) tmem_arrived(x + 32 * i);
          if (border) {
#pragma unroll
            for (int e = 0; e < kCols; ++e) {
              const int from = kM == 64 ? (half ? from1 : from0) : e < kPage ? from0 : from1, at = kM == 64 ? 64 * half + e : e;
              x[e] = at >= from && at < to ? x[e] : -INFINITY;
            }
          }
          float mx[kCols / 32];
#pragma unroll
          for (int i = 0; i < kCols / 32; ++i) {
            mx[i] = fmaxf(x[32 * i], x[32 * i + 1]);
#pragma unroll
            for (int e = 2; e < 32; e += 2) mx[i] = max3(mx[i], x[32 * i + e], x[32 * i + e + 1]);
          }
          float now;
          if constexpr (kM == 64) {
            now = fmaxf(mx[0], mx[1]) * (half ? f1 : f0);
            now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 16));
          } else {
            now = fmaxf(fmaxf(mx[0], mx[1]) * f0, fmaxf(mx[2], mx[3]) * f1);
          }
          // The maximum follows only when it grows by more than 2^kFollow (a published method of attention kernels): weights
          // above it are as exact in fp16, and O and the sum are rescaled a few times a row.
          const bool follow = now > __fadd_rd(top, kFollow) || (top == -INFINITY && now > top);
          if (__any_sync(0xffffffffu, follow)) {
            const float alpha = follow ? ex2(top - now) : 1.f;
            if (follow) top = now;
            l *= alpha;
            if (any) {
#pragma unroll 1
              for (int i = 0; i < kDims; i += 32) {
                float v[32];
                load_o(o_at + i, v);
                tmem_arrived(v);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] *= alpha;
                store_o(o_at + i, v);
              }
            }
          }
          any = true;
          const float z = top == -INFINITY ? 0.f : top;
          float2 sum[4] = {};
          const float2 zz = make_float2(__fadd_rd(kWeight, -z), __fadd_rd(kWeight, -z));
#pragma unroll
          for (int i = 0; i < kCols / 32; ++i) {
            const float f = kM == 64 ? (half ? f1 : f0) : i < 2 ? f0 : f1;
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float2 y = fma2(make_float2(x[32 * i + 2 * e], x[32 * i + 2 * e + 1]), make_float2(f, f), zz);
              y.x = ex2(y.x);
              y.y = ex2(y.y);
              w[e] = f16x2(y.x, y.y);
              sum[e & 3] = add2(sum[e & 3], y);
            }
            if constexpr (kM == 64) {      // over the scores
              tc::tmem_st16x2_16<32>(s_at + 16 * i, w);
            } else {
              tc::tmem_st8(s_at + 16 * i, w);
              tc::tmem_st8(s_at + 16 * i + 8, w + 8);
            }
          }
          sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
          l += sum[0].x + sum[0].y;
          tc::tmem_st_wait();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&m.p_full[grp]);
        }
        if (kM == 64) l += __shfl_xor_sync(0xffffffffu, l, 16);
        await_warp(&m.o_full[grp], outs++ & 1, m);
        tc::fence_after_sync();
        if ((w.take - grp0 + kBy - 1) / kBy > kRun) {
          // ---- a run's sums: with those of earlier ones, to the workspace or, at last, back into TMEM
          const bool more = j / kBy > kRun, last = j >= w.take;
          const long long at = ((long long)blockIdx.x * (aside ? 1 : 2) + (!aside && w.begins() ? 1 : 0)) * p.most + row;
          float2* ml = (aside ? p.second_ml : p.ml) + at;
          float* run = (aside ? p.second : p.o) + at * D + half * kDims;
          float2 old = make_float2(-INFINITY, 0.f);
          if (real && more) old = *ml;
          const float back = old.x == top ? 1.f : ex2(old.x - top);
          l += old.y * back;
          __syncwarp();
          if (real && half == 0) *ml = make_float2(top, l);
#pragma unroll 1
          for (int i = 0; i < kDims; i += 32) {
            float v[32];
            load_o(o_at + i, v);
            tmem_arrived(v);
            if (real && more) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                float u[8];
                ldg256(run + i + e, u);
#pragma unroll
                for (int d = 0; d < 8; ++d) v[e + d] += u[d] * back;
              }
            }
            __syncwarp();
            if (last) {
              store_o(o_at + i, v);
            } else if (real) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) stg256(run + i + e, reinterpret_cast<const uint32_t*>(v + e));
            }
          }
          if (last) {
            tc::tmem_st_wait();
          } else {
            l = 0.f;
            any = false;
          }
        }
      }
      // ---- the segment's result, or its part
      const bool two = SPLIT && w.take > 1;                  // both groups have steps
      l *= kWeightUndo;
      if (fabsf(top) >= kMostLogit && top != -INFINITY) l = NAN;
      if (SPLIT && grp == 1 && half == 0) m.ml[r] = make_float2(top, l);
      if (SPLIT) {
        tc::fence_before_sync();
        named_sync(1, 256);
        tc::fence_after_sync();
      }
      if (!SPLIT || grp == 0) {
        const long long at = ((long long)blockIdx.x * 2 + (w.begins() ? 1 : 0)) * p.most + row;
        float a0 = 1.f, a1 = 0.f;
        if (two) {
          const float2 o = m.ml[r];
          const float n = fmaxf(top, o.x), z = n == -INFINITY ? 0.f : n;
          a0 = ex2(top - z);
          a1 = ex2(o.x - z);
          l = l * a0 + o.y * a1;
          top = n;
        }
        const bool whole = w.begins() && w.ends();
        const float unit = m.unit[w.n & 3] * (0.0078125f * kWeightUndo);
        const float inv = whole ? (l == 0.f ? 0.f : __fdiv_rn(1.f, l)) : 1.f;
        const bool nan = m.nan[w.n & 3] != 0;
        const long long out_row = (long long)tok * a.Hq + hq;
#pragma unroll 1
        for (int i0 = 0; i0 < kDims; i0 += 32) {
          const int i = half * kDims + i0;                   // the channels' first
          float v[32];
          load_o(o_at + i0, v);
          tmem_arrived(v);
          if (two) {
            float u[32];
            load_o(o_at + 128 + i0, u);
            tmem_arrived(u);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = v[e] * a0 + u[e] * a1;
          }
          if (!real) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = v[e] * unit * inv;
          if (nan) {                     // the NaNs that this row sees, among the tokens that not all rows see
            const int u0 = (t.step + w.x) * kStep, u1 = u0 + w.take * kStep;
            uint32_t bits = 0;
#pragma unroll 1
            for (int side = 0; side < 2; ++side) {
              const int b = max(max(u0, lo), side ? max(t.hi_min, t.lo_max) : t.lo), e = min(min(u1, hi), side ? t.hi : t.lo_max);
#pragma unroll 1
              for (int y = b; y < e; ++y) {
                const int id = ld_s32(c.page_table + (long long)t.s * c.max_pages + y / kPage);
                if (id < 0 || id >= c.num_pages) continue;
                const uint8_t* src = c.v + (((long long)id * c.Hkv + w.h) * kPage + y % kPage) * D + i;
#pragma unroll 1
                for (int d = 0; d < 32; ++d) bits |= (uint32_t)((src[d] & 0x7f) == 0x7f) << d;
              }
            }
#pragma unroll
            for (int d = 0; d < 32; ++d)
              if (bits >> d & 1) v[d] = NAN;
          }
          if (!whole) {
            float* dst = p.o + at * D + i;
#pragma unroll
            for (int e = 0; e < 32; e += 8) stg256(dst + e, reinterpret_cast<const uint32_t*>(v + e));
          } else if (a.out_dtype == CSA2_F32) {
            float* dst = reinterpret_cast<float*>(a.out) + out_row * D + i;
            if (p.aligned & 4) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) stg256(dst + e, reinterpret_cast<const uint32_t*>(v + e));
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) dst[e] = v[e];
            }
          } else {
            uint16_t* dst = reinterpret_cast<uint16_t*>(a.out) + out_row * D + i;
            uint32_t o[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = bf16x2(v[2 * e], v[2 * e + 1]);
            if (p.aligned & 4) {
              stg256(dst, o);
              stg256(dst + 16, o + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) dst[e] = (uint16_t)(o[e / 2] >> 16 * (e & 1));
            }
          }
        }
        if (real && half == 0) {
          if (!whole) p.ml[at] = make_float2(top, l);
          else if (a.lse) a.lse[out_row] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
        }
      }
      if (SPLIT) {
        tc::fence_before_sync();
        named_sync(1, 256);              // the second group's output and sums have been read
        tc::fence_after_sync();
      }
      if (w.begins() && !w.ends())
        part = Part{t.n, t.rows.t0, t.r0, w.h, (int)blockIdx.x + (int)((t.count - w.take + per - 1) / per)};
      step += w.take;
    }
    if (tid == kSoftmax * 32) p.part[blockIdx.x] = part;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMma) tc::tmem_dealloc(tb, 512);
}

template <int D, int RT>
cudaError_t launch(const CUtensorMap& mk, const CUtensorMap& mv, const Kv8Params& p, cudaStream_t st) {
  static SmemLimit limit;
  const cudaError_t e = limit.raise(k_kv8_tile<D, RT>, Smem<D>::kBytes);
  if (e != cudaSuccess) return e;
  return launch_k(k_kv8_tile<D, RT>, dim3(kTileSpans), dim3(kThreads), Smem<D>::kBytes, st, mk, mv, p);
}

template <int D>
cudaError_t launch_of(const Kv8Params& p, cudaStream_t st) {
  CUtensorMap mk, mv;
  if (!plane_map(&mk, p.a.cache.k, p.a.cache, kPage) || !plane_map(&mv, p.a.cache.v, p.a.cache, kPage))
    return cudaErrorInvalidValue;
  const int rows = tile_rows(p.a);
  if (rows == 64) return launch<D, 64>(mk, mv, p, st);
  return rows == 128 ? launch<D, 128>(mk, mv, p, st) : launch<D, 256>(mk, mv, p, st);
}

}  // namespace

cudaError_t launch_kv8_tile(const Kv8Params& p, cudaStream_t st) {
  return p.a.cache.D == 64 ? launch_of<64>(p, st) : launch_of<128>(p, st);
}

uint32_t read_clear_error_kv8_tile() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_err_kv8_tile, sizeof(v));
  if (v) cudaMemcpyToSymbol(g_err_kv8_tile, &z, sizeof(z));
  return v;
}

}  // namespace csa2

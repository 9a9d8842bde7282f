// attn_masked_tc.cu -- attention whose rows read only some of the keys, on the tensor
// cores: prompts with a sliding window and sinks (packed K and V), and many query rows
// a kv head (drafted trees, chunks of a prompt) over a paged bf16 or E4M3 cache.
//
// For the row at position p, over the keys that it reads (p - j < W or j < S; of a
// tree's nodes, its line of parents):
//     m = max_j s_j,  l = sum_j exp(s_j - m),  o = sum_j exp(s_j - m) v_j / l,
// the cascade of [E] §2.2 in its incremental form ([E] §2.3).  The plan (which rows
// and keys an item has, how items are shared out) is in attn_masked_tc.cuh.
//
// A CTA takes items of two 128-row query tiles (a, b).  An event is a key tile for one
// of them; events go in the order (key tile, a before b).  Per event of tile x:
//   1. S = Q_x K_j^T (tcgen05 kind::f16, M = N = 128, fp32 in tensor memory), into the
//      one S that both tiles use in turn;
//   2. softmax warpgroup x, a thread a row: reads its 128 scores into registers, which
//      frees S for the next event; keys the row does not read at -inf (only where some
//      row reads a part); running maximum moved lazily (by more than 2^8 only);
//      P_x = 2^(S c - m) as bf16;
//   3. O_x += P_x V_j (P the tensor-memory A operand).
// Half key tiles that a query tile does not read are left out of its event.
// Tensor memory: S, P_a, P_b, O_a, O_b, at d = 128 all of its 512 columns.  One warp
// issues the S products, another P.V: S may be as far ahead as its tiles are there, a
// warpgroup that ends an event finds its next scores, the two run half an event out of
// phase, and the tensor core has the one's products during the other's softmax.
// What it took for 128 keys of both tiles (clock stamps; the products alone take 2048
// clocks): 4900 clocks with S_a, S_b and P over S (the next S waits for P.V); 3835 in
// units of 64 keys with two S buffers a tile (48 clocks a step for half the keys); 5000
// with one S and one warp for all products, whose waits and commits (70 to 200 clocks
// each) then follow one another; 2800 to 3000 as it is.
//
// Measured (heads 32 / 8 of 128; calls among others):
//   prompt of 16384, window 4096              740 us   1.30 PFLOP/s (69 % of cuBLAS)
//   6 prompts of 100-4000, window 1024        217 us   0.71 PFLOP/s: ten key tiles an
//     item at 1.47 us, and 6.5 us beside them (1 start, 3.5 more in three masked tiles,
//     0.35 the last product, 1.7 the output)
//   8 trees of 64 nodes, 2-16k tokens, bf16   92 us    3.3 TB/s
//   16 trees of 16 nodes, 0.5-8k, E4M3        122 us   1.2 TB/s: one tile an item (64 of
//     its rows are there), so S, softmax and P.V follow one another, and the widening
//     shares issue slots and the conversion unit with the softmax (whose registers spill
//     there: 172 bytes of stores, 388 of loads); bf16 77 us, 3.8 TB/s (means of six batches)
// Counters (8192 tokens, window 4096): tensor pipe 49 % of the time, DRAM 4 %, stalls an
// issue: wait 1.6, long scoreboard 1.5, no instruction 0.6.
//
// Rounding: P is rounded to bf16 (half a step, 2^-8 of a weight; l sums the unrounded
// ones), since both operands of an MMA have one type and V is bf16.
//
// Masked places.  Scores are selected, not added to.  A value that is not finite
// would reach rows that do not read it as 0 * inf, so a guard warp looks the values of
// every partly read tile over; rows of such a tile that are not finite are zeroed in
// shared memory, and the softmax threads of the rows that do read them add weight
// times value themselves.
#include <math.h>

#include <vector>

#include "attn_masked_tc.cuh"

namespace rf {
namespace masked {

constexpr int kHalf = 128 * 128;                      // 128 rows of 64 values: 16 KB
constexpr float kLazy = 8.f;
constexpr float kTop = 7.f;                           // E4M3: log2 of P's first largest

template <int D, bool kPaged, bool kF8>
struct Cfg {
  // TMA, S, P.V, guard; softmax a; softmax b; E4M3: four warps that widen the codes
  static constexpr int kThreads = kF8 ? 512 : 384;
  // Registers: 384 threads start with 168 each (64512): the softmax warpgroups take 216
  // (55296) of them, the others keep 72 (9216).  512 start with 128 each (65536): 200
  // (51200) and 56 (14336).
  static constexpr int kSoftmaxRegs = kF8 ? 200 : 216, kOtherRegs = kF8 ? 56 : 72;
  static constexpr int kTile = D / 64 * kHalf;        // 128 rows of D 16-bit values
  static constexpr int kQSlots = D == 64 ? 4 : (kF8 ? 2 : 3);
  // E4M3: a tile's softmax waits for that tile's queries, and converts them in place.
  using Queries = QTurns<kQSlots, kF8>;
  // Places of K and of V tiles (E4M3: widened; two of V, since the next waits for P.V; one
  // and a third of codes is as fast)
  static constexpr int kKs = kF8 ? (D == 64 ? 2 : 1) : (D == 64 ? 4 : 2);
  static constexpr int kVs = kF8 ? 2 : kKs;
  static constexpr int kRing = kQSlots * kTile;
  static constexpr int kRawOff = kRing + (kKs + kVs) * kTile;
  static constexpr int kRaw = kF8 ? BK * D : 0;       // a tile's codes, K and V in turn
  static constexpr int kRawPairs = kF8 ? (D == 64 ? 5 : 2) : 1;
  static constexpr int kBarOff = kRawOff + 2 * kRawPairs * kRaw;
  static constexpr int kSmem = kBarOff + 2048 + 1024; // barriers; alignment
  // Prompts: the output goes through the item's own Q tile to whole 128-byte lines.
  static constexpr bool kStaged = !kPaged;
  static constexpr uint32_t kIdescS = make_idesc(BQ, BK, kF8 ? 0 : 1, 0, 0);
  static constexpr uint32_t kIdescHalf = make_idesc(BQ, kUnit, kF8 ? 0 : 1, 0, 0);
  static constexpr uint32_t kIdescO = make_idesc(BQ, D, kF8 ? 0 : 1, 0, 1);
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(1 + kVs + (kF8 ? kRawPairs : 0) <= 8 && 1 + kKs + (kF8 ? kRawPairs : 0) <= 8,
                "records");
};
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;                         // 128 columns
__device__ __forceinline__ uint32_t col_p(int x) { return 128 + x * 64; }
__device__ __forceinline__ uint32_t col_o(int x) { return 256 + x * 128; }

struct Params {
  Geo geo;
  __nv_bfloat16* O;
  const void* V;                                      // bf16, or codes
  int64_t ldo, ldv, n_v;                              // elements between tokens; of V
  const float* k_scale;
  const float* v_scale;
  const int* parents;
  const int* block_table;
  int Hq, num_pages, page_size, page_shift, max_pages;
  float c_log2;
  float4* ws_o;                                       // [slots][2][D / 4][128]
  float4* ws_st;                                      // [slots][2][128]: M, m, l
  int4* ws_cut;                                       // [grid]: see the kernel
  unsigned* err;
};

constexpr int kPieces = 3;

struct Bars {
  uint64_t q_full[4], q_empty[4];
  uint64_t full[8], empty[8];                         // of K's places, from 4 on V's
  // A V tile is looked over.  By the key tile's number, not by V's place: a query tile's
  // softmax waits for tiles that it takes only, and a parity tells tile m's phase where the
  // one before is complete; with the scores of tile m there, that of tile m - 8 is (see rec).
  uint64_t v_ok[8];
  uint64_t s_full[2], p_full[2], pv_done[2];          // of a query tile's events
  uint64_t s_read;                                    // of all events: S is in registers
  uint64_t drain[2];
  // Per key tile, like scale and its parts below: tile m's takes the place of tile m - 8's.
  // It is written once V of tile m - 1 has a place to be copied to: the one of tile
  // m - 1 - kVs, whose P.V is done, or (E4M3) the codes' of tile m - 1 - kRawPairs, which are
  // widened, so that V's place of tile m - 1 - kRawPairs - kVs had been left by its P.V.  And
  // K of tile m - 1 has one, by the same count with kKs: S of tile m - 1 - kRawPairs - kKs is
  // done.  Cfg asserts that both are tile m - 8 or later.  The softmax warps of a query tile
  // look at those of key tiles that it takes only, which P.V does not pass without them.
  unsigned rec[8];
  unsigned bad[4][4];                                 // per V stage: values that are not finite
  // E4M3: codes have come, are widened; queries are; per key tile, the pages' scales as
  // they come, and per 16 keys the key scale and log2 of the value scale
  uint64_t raw_full[2][5], raw_empty[2][5], q_ok[4];
  float sc_k[8][8], sc_v[8][8];
  float2 scale[8][8];
  // The TMA warp's pieces, for the softmax: walked once, ahead of time.
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  union {
    struct {                                          // of the plan, before there are pieces
      int64_t warp_sum[16];
      int warp_items[16], warp_most[16];
    };
    struct {
      Piece piece[kPieces];                           // j0 < 0: there are no more
      QPlace q[kPieces][2];                           // where its query tiles are
    };
  };
  int64_t x[2];                                       // the CTA's range
  int g, h, j;                                        // where it begins
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Bars) <= 2048, "barriers");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// The same value in every lane, which the compiler then knows (uniform registers, which
// the tensor core's instructions take their operands from).
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// mbar_wait of a whole warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}
// One column of this thread's lane (waits for it).
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r)
      : "r"(taddr)
      : "memory");
  return r;
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on `bar` when this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// Two E4M3 codes (the low or high half of a word) -> two f16, exact.
__device__ __forceinline__ uint32_t widen(uint32_t w, bool high) {
  uint32_t r;
  if (high)
    asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;}" : "=r"(r) : "r"(w));
  else
    asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float f16_to_f32(uint32_t w, bool high) {
  float r;
  asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;}" : "=f"(r) : "r"(high ? w >> 16 : w));
  return r;
}
// Bits 0 .. n - 1 of a word.
__device__ __forceinline__ unsigned below(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u);
}

// What the TMA warp tells the MMA threads and the guard about a key tile.
enum : unsigned {
  kTakes = 1u,              // << (2 x + h): tile x takes half h
  kFirst = 16u,             // of its piece
  kLast = 32u,
  kHasB = 64u,              // the piece has a tile b
  kPartly = 128u,           // << h: some row may not read all keys of half h
  kEnd = 512u,              // of the CTA's range
  kYield = 1024u,           // P.V lets S go first (see there)
  kPages = 16,              // over a cache, from this bit on: bit per 16 keys that are there
};

template <int D, bool kPaged, bool kF8>
__global__ void __launch_bounds__((Cfg<D, kPaged, kF8>::kThreads), 1)
    attn_masked_kernel(const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  using C = Cfg<D, kPaged, kF8>;
  constexpr int kThreads = C::kThreads;
  static_assert(kPaged || !kF8, "codes are a cache's");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kBarOff);
  volatile int* abort_flag = &bars->abort;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int cta = (int)blockIdx.x;
  const Geo& geo = p.geo;
  uint8_t* ring = smem + C::kRing;

  // The merge may take its place as soon as CTAs leave; it waits for the end of this grid.
  if (kPaged) asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&bars->q_full[i]), 1);
      mbar_init(smem_u32(&bars->q_empty[i]), C::kStaged ? 1 + 4 : 1);
      mbar_init(smem_u32(&bars->q_ok[i]), BQ);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_u32(&bars->full[i]), kF8 ? 2 : 1);       // a copy, or the widening warps
      mbar_init(smem_u32(&bars->v_ok[i]), kF8 ? 2 : 1);
      mbar_init(smem_u32(&bars->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->s_full[i]), kPaged ? 2 : 1);  // the product; over a cache, rec
      mbar_init(smem_u32(&bars->p_full[i]), BQ);
      mbar_init(smem_u32(&bars->pv_done[i]), 1);
    }
    mbar_init(smem_u32(&bars->s_read), 4);            // a warpgroup's warps
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(smem_u32(&bars->piece_full[i]), 1);
      mbar_init(smem_u32(&bars->piece_empty[i]), 8);  // both warpgroups' warps
    }
    mbar_init(smem_u32(&bars->drain[0]), 1);
    mbar_init(smem_u32(&bars->drain[1]), 1);
    if (kF8) {
      for (int i = 0; i < C::kRawPairs; ++i) {
        mbar_init(smem_u32(&bars->raw_full[0][i]), 1 + 32);     // the copies' bytes; scales
        mbar_init(smem_u32(&bars->raw_full[1][i]), 1);
        mbar_init(smem_u32(&bars->raw_empty[0][i]), 2);
        mbar_init(smem_u32(&bars->raw_empty[1][i]), 2);
      }
    }
    bars->abort = 0;
    bars->x[0] = bars->x[1] = 0;
    bars->g = bars->h = bars->j = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars->tmem), kTmemCols);
    tmem_relinquish();
  }

  // ---- plan: add up all tiles, find where this CTA's range begins
  const int ng = geo.B * geo.npairs;
  const int per = (ng + kThreads - 1) / kThreads;
  const int g_lo = min((int)threadIdx.x * per, ng), g_hi = min(g_lo + per, ng);
  int64_t mine = 0;
  int items = 0, most = 0;                            // (items: at most B Tq Hq, below 2^31)
  for (int g = g_lo; g < g_hi; ++g) {
    const int n = places(geo, group_of(geo, g, cta == 0, p.err));
    mine += (int64_t)n * geo.Hkv;
    items += kPaged && n > 0 ? geo.Hkv : 0;
    most = max(most, n);
  }
  int64_t incl = mine;
  int incl_items = items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
    if (kPaged) {
      const int u = __shfl_up_sync(0xffffffffu, incl_items, o);
      if (lane >= o) incl_items += u;
    }
  }
  if (kPaged) most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) {
    bars->warp_sum[warp] = incl;
    bars->warp_items[warp] = incl_items;
    bars->warp_most[warp] = most;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int64_t pre = incl - mine, total = 0;
  int pre_items = incl_items - items, all_items = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) {
      pre += bars->warp_sum[w];
      pre_items += bars->warp_items[w];
    }
    total += bars->warp_sum[w];
    all_items += bars->warp_items[w];
    most = max(most, bars->warp_most[w]);
  }
  const int grid = total < (int64_t)gridDim.x ? (int)total : (int)gridDim.x;
  if (kPaged && cta < grid && keeps_items(all_items, most, total, grid)) {
    for (int i = 0; i < 2; ++i) {                     // item cta + i begins a range
      const int x = cta + i;
      if (x >= all_items) {
        if (threadIdx.x == 0) bars->x[i] = total;
      } else if (x >= pre_items && x - pre_items < items) {
        int64_t at = pre;
        int left = x - pre_items;
        for (int g = g_lo; g < g_hi; ++g) {
          const int n = places(geo, group_of(geo, g, false, p.err));
          if (n > 0 && left < geo.Hkv) {
            bars->x[i] = at + (int64_t)left * n;
            if (i == 0) {
              bars->g = g;
              bars->h = left;
            }
            break;
          }
          at += (int64_t)n * geo.Hkv;
          left -= n > 0 ? geo.Hkv : 0;
        }
      }
    }
  } else if (cta < grid) {
    const Split64 split(total, grid);
    for (int i = 0; i < 2; ++i) {
      const int64_t x = split.start(cta + i);
      if (x >= total) {
        if (threadIdx.x == 0) bars->x[i] = total;
      } else if (x >= pre && x - pre < mine) {        // in this thread's groups: walk to it
        int64_t at = pre;
        for (int g = g_lo; g < g_hi; ++g) {
          const Group w = group_of(geo, g, false, p.err);
          const int n = places(geo, w);
          const int64_t all = (int64_t)n * geo.Hkv;
          if (x - at < all) {
            const int h = (int)((x - at) / n), off = (int)((x - at) % n);
            const bool up = !kPaged && snaps_up(off, n);
            bars->x[i] = kPaged ? x : x - off + (up ? n : 0);
            if (i == 0) {
              bars->g = g;
              bars->h = h;
              bars->j = kPaged ? off : (up ? w.n : 0);
            }
            break;
          }
          at += all;
        }
      }
    }
  }
  __syncthreads();
  const uint32_t tmem = (uint32_t)uniform((int)bars->tmem);
  const int64_t x0 = bars->x[0], x1 = bars->x[1];
  if (kPaged && threadIdx.x == 0 && RF_IN(p.err, cta, gridDim.x)) {
    // For the merge: the item in which this CTA's range begins, if that is its first cut:
    // its pieces (0: it is not), group and head.
    int pieces = 0;
    if (x1 > x0 && bars->j > 0) {
      const Split64 split(total, grid);
      const int64_t first = x0 - bars->j;
      if (split.start(cta - 1) <= first)
        pieces = split.owner(first + group_of(geo, bars->g, false, p.err).n - 1) - (cta - 1) + 1;
    }
    p.ws_cut[cta] = make_int4(pieces, bars->g, bars->h, 0);
  }
  Walk walk(bars->g, bars->h, bars->j, x1 - x0);
  Piece c;
  bool ok = true;

  if (warp < 4) {
    regs_dec<C::kOtherRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------- TMA
      const uint64_t pol_kv = policy_evict_last(), pol_q = policy_evict_first();
      typename C::Queries queries(geo);               // issued
      int nt = 0;                                     // key tiles issued
      unsigned in_flight = 0;                         // stages filled so far (2 a key tile)
      for (int np = 0; ok; ++np) {
        const int pc = np % kPieces;
        const bool last = !walk.next(geo, c, p.err);
        if (last) c.j0 = -1;
        ok = np < kPieces ||
             warp_wait(smem_u32(&bars->piece_empty[pc]), (uint32_t)((np / kPieces - 1) & 1));
        if (!ok) break;
        QPlace qa = {0, 0}, qb = {0, 0};
        if (!last) {
          qa = queries.next(0);
          if (tile_of(geo, c.w, 1).has()) qb = queries.next(1);
        }
        if (lane == 0) {
          bars->piece[pc] = c;
          bars->q[pc][0] = qa;
          bars->q[pc][1] = qb;
          mbar_arrive(smem_u32(&bars->piece_full[pc]));
        }
        if (last) break;
        const Tile ta = tile_of(geo, c.w, 0), tb = tile_of(geo, c.w, 1);
        auto load_q = [&](const QPlace& at, const Tile& t) {
          ok = at.turn == 0 ||
               warp_wait(smem_u32(&bars->q_empty[at.slot]), (uint32_t)((at.turn - 1) & 1));
          if (!ok) return;
          if (lane == 0) {
            const uint32_t bar = smem_u32(&bars->q_full[at.slot]);
            const uint32_t dst = smem_u32(smem + at.slot * C::kTile);
            mbar_arrive_expect_tx(bar, (uint32_t)(D / 64 * geo.tpt * geo.G * 128));
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
              tma_load_3d_hint(dst + i * kHalf, &tmQ, bar, 64 * i, c.h * geo.G, c.w.q0 + t.t0, pol_q);
          }
        };
        load_q(qa, ta);
        // Q_b behind the first keys: its place may still have an output in it
        if (!C::kStaged && ok && tb.has()) load_q(qb, tb);
        const Whole whole = whole_of(geo, c.w);
        for (int j = c.j0; ok && j < c.j1; ++j, ++nt) {
          const int key0 = key0_of(c.w, j);
          unsigned rec = (ta.takes(2 * j) ? 1u : 0u) | (ta.takes(2 * j + 1) ? 2u : 0u) |
                         (tb.takes(2 * j) ? 4u : 0u) | (tb.takes(2 * j + 1) ? 8u : 0u) |
                         (j == c.j0 ? kFirst : 0u) | (j == c.j1 - 1 ? kLast : 0u) |
                         (j == c.j1 - 1 && walk.left <= 0 ? kEnd : 0u) |
                         (tb.has() ? kHasB : 0u) | (whole.partly(geo, key0, kUnit) ? kPartly : 0u) |
                         (whole.partly(geo, key0 + kUnit, kUnit) ? kPartly << 1 : 0u);
          auto both = [&](int i) {                    // query tiles take key tile i
            return i < c.j1 && (ta.takes(2 * i) || ta.takes(2 * i + 1)) &&
                   (tb.takes(2 * i) || tb.takes(2 * i + 1));
          };
          if (both(j) && both(j + 1)) rec |= kYield;
          // over a cache: lane i has the tile's page i
          int row = 0;
          int64_t scale_at = 0;
          bool there = false;
          if (kPaged) {
            const int first = key0 + lane * p.page_size;
            const bool read = lane < BK >> p.page_shift && first < c.w.lk;
            if (read) {
              const int page = ld_int(p.block_table,
                                      (int64_t)c.w.b * p.max_pages + (first >> p.page_shift),
                                      (int64_t)geo.B * p.max_pages, p.err);
              // a page in which no row reads anything may be anything
              const int ctx = c.w.lk - c.w.lq;
              const int lo = geo.window > 0 ? (geo.tree ? ctx : ctx + c.w.t0) - geo.window + 1 : 0;
              const bool wanted = first + p.page_size > lo || first < geo.sinks;
              there = wanted && (unsigned)page < (unsigned)p.num_pages;
              if (wanted && !there) raise_error(p.err, kDevErrInput);
              row = (page * geo.Hkv + c.h) * p.page_size;
              scale_at = (int64_t)page * geo.Hkv + c.h;
            }
          }
          const unsigned pages = __ballot_sync(0xffffffffu, there);
          if (kPaged) {
            const int per16 = p.page_size >> 4;       // bits of a page
            unsigned bits = 0;
            for (unsigned m = pages; m != 0; m &= m - 1)
              bits |= ((1u << per16) - 1u) << ((__ffs((int)m) - 1) * per16);
            rec |= bits << kPages;
          }
#pragma unroll
          for (int v = 0; v < 2; ++v) {               // K, then V
            const int rp = nt % C::kRawPairs;
            const int ks = v ? C::kVs : C::kKs, st = nt % ks, sb = v ? 4 + st : st;
            const uint32_t bar = smem_u32(kF8 ? &bars->raw_full[v][rp] : &bars->full[sb]);
            if (kF8)
              ok = nt < C::kRawPairs || warp_wait(smem_u32(&bars->raw_empty[v][rp]),
                                                  (uint32_t)((nt / C::kRawPairs - 1) & 1));
            else
              ok = nt < ks || warp_wait(smem_u32(&bars->empty[sb]), (uint32_t)((nt / ks - 1) & 1));
            if (!ok) break;
            const uint32_t dst = smem_u32(kF8 ? smem + C::kRawOff + (2 * rp + v) * C::kRaw
                                              : ring + ((v ? C::kKs : 0) + st) * C::kTile);
            const CUtensorMap* tm = v ? &tmV : &tmK;
            if (kPaged) {
              if (lane == 0) {
                if (v == 0) bars->rec[nt % 8] = rec;
                mbar_arrive_expect_tx(bar, (uint32_t)(__popc(pages) * p.page_size * D * (kF8 ? 1 : 2)));
              }
              __syncwarp();
              if (kF8) {                              // 128-byte rows: a key, or two of 64 dims
                if (there) {
                  tma_load_2d_hint(dst + lane * p.page_size * D, tm, bar, 0, D == 128 ? row : row >> 1, pol_kv);
                  if (v == 0 && RF_IN(p.err, scale_at, (int64_t)p.num_pages * geo.Hkv)) {
                    cp_async4(smem_u32(&bars->sc_k[nt % 8][lane]), p.k_scale + scale_at);
                    cp_async4(smem_u32(&bars->sc_v[nt % 8][lane]), p.v_scale + scale_at);
                  }
                }
                if (v == 0) cp_async_arrive(bar);
              } else if (there) {
#pragma unroll
                for (int i = 0; i < D / 64; ++i)
                  tma_load_2d_hint(dst + i * kHalf + lane * p.page_size * 128, tm, bar, 64 * i, row,
                                   pol_kv);
              }
            } else if (lane == 0) {
              if (v == 0) bars->rec[nt % 8] = rec;
              mbar_arrive_expect_tx(bar, C::kTile);
#pragma unroll
              for (int i = 0; i < D / 64; ++i)
                tma_load_3d_hint(dst + i * kHalf, tm, bar, 64 * i, c.h, c.w.k0 + key0, pol_kv);
            }
            ++in_flight;
          }
          if (C::kStaged && ok && j == c.j0 && tb.has()) load_q(qb, tb);
        }
        if (*abort_flag) ok = false;
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) {
        raise_error(p.err, kDevErrTimeout);
        *abort_flag = 1;
        // copies in flight land before shared memory is released
        for (int x = 0; x < 2; ++x) {
          const int n = x ? queries.nb : queries.na;
          // (the piece's own may not have been issued: two more)
          for (int i = max(0, n - queries.places() - 2); i < n; ++i) {
            const QPlace at = queries.at(x, i);
            (void)mbar_wait(smem_u32(&bars->q_full[at.slot]), (uint32_t)(at.turn & 1), 1000000ull);
          }
        }
        constexpr unsigned kPlaces = 2 * (kF8 ? C::kRawPairs : C::kKs);
        for (unsigned i = in_flight > kPlaces ? in_flight - kPlaces : 0; i < in_flight; ++i)
          (void)mbar_wait(smem_u32(kF8 ? &bars->raw_full[i % 2][i / 2 % C::kRawPairs]
                                       : &bars->full[i % 2 * 4 + i / 2 % C::kKs]),
                          (i / kPlaces) & 1, 1000000ull);
      }
    } else if (warp < 3) {
      // ---------------------------------------------------------- MMA: S (warp 1), P.V (warp 2)
      // The whole warp runs the schedule, one lane issues: with the schedule in one lane an
      // MMA took 100 clocks to issue (its operands went through vector registers).
      bool more = x1 > x0;
      const bool leader = elect_one();
      if (warp == 1) {
        const uint64_t qd = sw128_desc(smem_u32(smem), 1024, 16);
        const uint64_t kd = sw128_desc(smem_u32(ring), 1024, 16);
        typename C::Queries queries(geo);
        QPlace qa = {0, 0}, qb = {0, 0};              // the piece's
        int events = 0;
        for (int nt = 0; ok && more; ++nt) {
          const int pr = nt % C::kKs;
          ok = warp_wait(smem_u32(&bars->full[pr]), (uint32_t)((nt / C::kKs) & 1));
          if (!ok) break;
          const unsigned rec = (unsigned)uniform((int)bars->rec[nt % 8]);
          more = !(rec & kEnd);
          const int tiles = (rec & kHasB) ? 2 : 1;
          if (rec & kFirst) {
            qa = queries.next(0);
            if (tiles == 2) qb = queries.next(1);
          }
#pragma unroll 1
          for (int x = 0; ok && x < tiles; ++x) {
            const int slot = x ? qb.slot : qa.slot;
            if (rec & kFirst)
              ok = warp_wait(smem_u32(kF8 ? &bars->q_ok[slot] : &bars->q_full[slot]),
                             (uint32_t)((x ? qb.turn : qa.turn) & 1));
            const unsigned halves = (rec >> (2 * x)) & 3u;
            if (ok && halves) {
              if (events > 0) ok = warp_wait(smem_u32(&bars->s_read), (uint32_t)((events - 1) & 1));
              if (!ok) break;
              ++events;
              tc_fence_after();
              const int h = halves == 2u ? 1 : 0;     // the first half it takes
              const uint64_t a = qd + (uint64_t)((slot * C::kTile) >> 4);
              const uint64_t b = kd + (uint64_t)((pr * C::kTile + h * kUnit * 128) >> 4);
              const uint32_t idesc = halves == 3u ? C::kIdescS : C::kIdescHalf;
              if (leader) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                  const uint64_t off = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
                  mma_bf16_ss(tmem + kColS + h * kUnit, a + off, b + off, idesc, k != 0);
                }
                mma_commit(smem_u32(&bars->s_full[x]));
                // the softmax may read rec (and scale), which came with the keys
                if (kPaged) mbar_arrive(smem_u32(&bars->s_full[x]));
              }
            }
            if (ok && (rec & kLast) && leader) mma_commit(smem_u32(&bars->q_empty[slot]));
          }
          if (ok && leader) mma_commit(smem_u32(&bars->empty[pr]));
          if (*abort_flag) ok = false;
          ok = __all_sync(0xffffffffu, ok);
        }
      } else {
        const uint64_t vd = sw128_desc(smem_u32(ring + C::kKs * C::kTile), 1024, kHalf);
        unsigned phase = 0, fresh = 3;                // bit x: of p_full[x]; O_x is to be overwritten
        constexpr int kPolls = 24;
        for (int nt = 0; ok && more; ++nt) {
          const int pr = nt % C::kVs;
          ok = warp_wait(smem_u32(&bars->v_ok[nt % 8]), (uint32_t)((nt / 8) & 1));
          if (!ok) break;
          const unsigned rec = (unsigned)uniform((int)bars->rec[nt % 8]);
          more = !(rec & kEnd);
          if (rec & kFirst) fresh = 3u;
          // values that are not finite are in O before the first product
          unsigned bad = 0;
          if (kPaged || (rec & (3u * kPartly))) {
            const unsigned* b = bars->bad[pr];
            bad = (unsigned)uniform(((b[0] | b[1]) ? 1 : 0) | ((b[2] | b[3]) ? 2 : 0));
          }
          const uint64_t b = vd + (uint64_t)((pr * C::kTile) >> 4);
#pragma unroll 1
          for (int x = 0; ok && x < 2; ++x) {
            const unsigned halves = (rec >> (2 * x)) & 3u;
            if (!halves) continue;
            ok = warp_wait(smem_u32(&bars->p_full[x]), (phase >> x) & 1u);
            if (!ok) break;
            // The S product that the same warpgroup will read next runs about now, and is
            // waited for; P is not, before that warpgroup's next one.  So this product lets
            // it end first (3670 -> 3000 clocks for a key tile of both): an order that
            // nothing relies on, looked for kPolls times (some 800 clocks) and no longer.
            if (rec & kYield) {
              const uint32_t next = smem_u32(&bars->s_full[x]);
              for (int i = 0; i < kPolls; ++i)
                if (__any_sync(0xffffffffu, mbar_test_wait(next, ((phase >> x) & 1u) ^ 1u))) break;
            }
            tc_fence_after();
            bool onto = !((fresh >> x) & 1u) || (halves & bad) != 0u;
            if (leader) {
#pragma unroll
              for (int k = 0; k < BK / 16; ++k) {
                if (!((halves >> (k / 4)) & 1u)) continue;
                mma_bf16_ts(tmem + col_o(x), tmem + col_p(x) + k * 8,
                            b + (uint64_t)((k * 16 * 128) >> 4), C::kIdescO, onto);
                onto = true;
              }
              mma_commit(smem_u32(&bars->pv_done[x]));
            }
            fresh &= ~(1u << x);
            phase ^= 1u << x;
          }
          if (ok && leader) mma_commit(smem_u32(&bars->empty[4 + pr]));
          if (*abort_flag) ok = false;
          ok = __all_sync(0xffffffffu, ok);
        }
      }
      if (!ok) {
        raise_error(p.err, kDevErrTimeout);
        *abort_flag = 1;
      }
      // nothing may still run on the tensor core when memory is released
      if (leader) mma_commit(smem_u32(&bars->drain[warp - 1]));
      (void)mbar_wait(smem_u32(&bars->drain[warp - 1]), 0, 1000000000ull);
    } else if (!kF8) {
      // ---------------------------------------------------------- guard
      bool more = x1 > x0;
      // an exponent of ones carries into the sign's place
      auto ones = [](const uint4& w) {
        return ((w.x & 0x7F807F80u) + 0x00800080u) | ((w.y & 0x7F807F80u) + 0x00800080u) |
               ((w.z & 0x7F807F80u) + 0x00800080u) | ((w.w & 0x7F807F80u) + 0x00800080u);
      };
      for (int nt = 0; ok && more; ++nt) {
        const int pr = nt % C::kVs;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->full[4 + pr]),
                                               (uint32_t)((nt / C::kVs) & 1)));
        if (!ok) break;
        const unsigned rec = bars->rec[nt % 8];
        more = !(rec & kEnd);
        const unsigned pages = kPaged ? (rec >> kPages) & 0xFFu : 0xFFu;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          unsigned bad[2] = {0u, 0u};
          if (((rec >> h) & kPartly) || pages != 0xFFu) {
            uint4* v = reinterpret_cast<uint4*>(ring + (C::kKs + pr) * C::kTile) + h * (kUnit * 8);
            unsigned seen = 0;
#pragma unroll
            for (int i = 0; i < D / 64; ++i)          // 64 rows of 128 bytes
#pragma unroll 8
              for (int k = lane; k < kUnit * 8; k += 32) seen |= ones(v[i * (kHalf / 16) + k]);
            if (__any_sync(0xffffffffu, (seen & 0x80008000u) != 0u)) {
#pragma unroll 1
              for (int r = 0; r < kUnit; ++r) {       // which rows; they become zeros
                uint4* at = v + (lane >> 3) * (kHalf / 16) + r * 8 + (lane & 7);
                const bool hit = lane < D / 8 && (ones(*at) & 0x80008000u) != 0u;
                if (!__any_sync(0xffffffffu, hit)) continue;
                bad[0] |= r < 32 ? 1u << r : 0u;
                bad[1] |= r >= 32 ? 1u << (r & 31) : 0u;
                if (lane < D / 8) *at = make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
            }
          }
          if (lane == 0) {
            bars->bad[pr][2 * h] = bad[0];
            bars->bad[pr][2 * h + 1] = bad[1];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->v_ok[nt % 8]));
        if (*abort_flag) ok = false;
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) {
        raise_error(p.err, kDevErrTimeout);
        *abort_flag = 1;
      }
    }
  } else if (kF8 && warp >= 12) {
    // ------------------------------------------------------------ E4M3: codes to f16
    // Two warps for K and two for V, a lane a key.  A code of NaN is dealt with as the guard
    // does with bf16.
    regs_dec<C::kOtherRegs>();
    const int v = (warp - 12) >> 1, h = warp & 1;     // K or V; the half of the key tile
    bool more = x1 > x0;
    for (int nt = 0; ok && more; ++nt) {
      const int ks = v ? C::kVs : C::kKs, pr = nt % ks, rp = nt % C::kRawPairs;
      ok = warp_wait(smem_u32(&bars->raw_full[v][rp]), (uint32_t)((nt / C::kRawPairs) & 1));
      if (!ok) break;
      const unsigned rec = bars->rec[nt % 8];
      more = !(rec & kEnd);
      if (v == 0 && h == 0) {                         // the scales of 16 keys each
        if (lane < 8) {
          const bool in = (rec >> (kPages + lane)) & 1u;
          const int page = lane >> (p.page_shift - 4);
          bars->scale[nt % 8][lane] = make_float2(in ? bars->sc_k[nt % 8][page] : 1.f,
                                                  in ? __log2f(bars->sc_v[nt % 8][page]) : 0.f);
        }
      }
      ok = nt < ks || warp_wait(smem_u32(&bars->empty[4 * v + pr]), (uint32_t)((nt / ks - 1) & 1));
      if (!ok) break;
      const bool alone = v == 1 && (((rec >> h) & kPartly) || ((rec >> kPages) & 0xFFu) != 0xFFu);
#pragma unroll 1
      for (int i32 = 0; i32 < 2; ++i32) {
        const int key = h * kUnit + i32 * 32 + lane;
        const int row = D == 128 ? key : key >> 1, base = D == 128 ? 0 : (key & 1) * 4;
        const uint8_t* raw = smem + C::kRawOff + (2 * rp + v) * C::kRaw + row * 128;
        uint8_t* out = ring + ((v ? C::kKs : 0) + pr) * C::kTile + key * 128;
        bool zero = false;
        if (alone) {
          unsigned nan = 0;
#pragma unroll 1
          for (int i = 0; i < D / 16; ++i) {
            const uint4 w = *reinterpret_cast<const uint4*>(raw + (((base + i) ^ (row & 7)) << 4));
            nan |= ((w.x & 0x7F7F7F7Fu) + 0x01010101u) | ((w.y & 0x7F7F7F7Fu) + 0x01010101u) |
                   ((w.z & 0x7F7F7F7Fu) + 0x01010101u) | ((w.w & 0x7F7F7F7Fu) + 0x01010101u);
          }
          zero = (nan & 0x80808080u) != 0u;
        }
        const unsigned bad = __ballot_sync(0xffffffffu, zero);
        if (v == 1 && lane == 0) bars->bad[pr][2 * h + i32] = bad;
#pragma unroll 2
        for (int i = 0; i < D / 16; ++i) {
          uint4 w = *reinterpret_cast<const uint4*>(raw + (((base + i) ^ (row & 7)) << 4));
          if (zero) w = make_uint4(0u, 0u, 0u, 0u);
          uint8_t* at = out + (i >> 2) * kHalf;
          const int ch = (2 * i) & 7;
          *reinterpret_cast<uint4*>(at + ((ch ^ (key & 7)) << 4)) =
              make_uint4(widen(w.x, false), widen(w.x, true), widen(w.y, false), widen(w.y, true));
          *reinterpret_cast<uint4*>(at + (((ch + 1) ^ (key & 7)) << 4)) =
              make_uint4(widen(w.z, false), widen(w.z, true), widen(w.w, false), widen(w.w, true));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&bars->raw_empty[v][rp]));
        mbar_arrive(smem_u32(v ? &bars->v_ok[nt % 8] : &bars->full[pr]));
      }
      if (*abort_flag) ok = false;
      ok = __all_sync(0xffffffffu, ok);
    }
    if (!ok) {
      raise_error(p.err, kDevErrTimeout);
      *abort_flag = 1;
    }
  } else {
    // ------------------------------------------------------------ softmax of tile x
    regs_inc<C::kSoftmaxRegs>();
    const int x = warp >= 8 ? 1 : 0;
    const int r = (warp & 3) * 32 + lane;             // row of the tile
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + kColS, p_addr = tmem + lane_off + col_p(x);
    const uint32_t o_addr = tmem + lane_off + col_o(x);
    const uint64_t c2 = f2(p.c_log2, p.c_log2);
    const int my_t = r / geo.G, my_g = r - my_t * geo.G;
    int nt = 0, cnt = 0;                              // key tiles; events of this warpgroup
    int64_t s0 = x0 - (x1 > x0 ? bars->j : 0);        // first tile of the piece's item
    for (int np = 0; ok; ++np) {
      const int pc = np % kPieces;
      ok = warp_wait(smem_u32(&bars->piece_full[pc]), (uint32_t)((np / kPieces) & 1));
      if (!ok) break;
      c = bars->piece[pc];
      const QPlace place = bars->q[pc][x];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->piece_empty[pc]));
      if (c.j0 < 0) break;
      const Tile t = tile_of(geo, c.w, x);
      const int64_t item0 = s0;
      s0 += c.w.n;
      const int j_base = nt - c.j0;                   // key tile j is the CTA's j_base + j th
      nt += c.j1 - c.j0;
      if (!t.has()) continue;
      const int slot = place.slot;
      const int tok = t.t0 + my_t;
      const bool real = my_t < geo.tpt && tok < t.t1;
      const int ctx = c.w.lk - c.w.lq;
      int pos = ctx + tok;                            // the row's position; < 0: it reads nothing
      if (geo.tree) {
        bool line = real && ctx >= 0;
        int u = tok, depth = 0;
        while (line) {
          const int up = ld_int(p.parents, (int64_t)c.w.b * geo.max_q + u,
                                (int64_t)geo.B * geo.max_q, p.err);
          if (up == -1) break;
          line = up >= 0 && up < u;
          u = up;
          ++depth;
        }
        if (real && !line && c.w.lk > 0) raise_error(p.err, kDevErrInput);
        pos = line ? ctx + depth : -1;
      }
      if (!real) pos = -1;
      float m_ref = -INFINITY, l_run = 0.f;
      float M_ref = -INFINITY, f_row = 0.f;           // E4M3: P's reference; the row's factor
      if (kF8) {
        // The row's queries as f16, scaled by a power of two to a largest element in
        // [2^14, 2^15): exact down to 2^-28 of it.
        if (!warp_wait(smem_u32(&bars->q_full[slot]), (uint32_t)(place.turn & 1))) {
          ok = false;
          break;
        }
        uint8_t* q = smem + slot * C::kTile + r * 128;
        // (Two short loops: unrolled whole they took 3.3 us, instructions to fetch and spills.)
        unsigned mx = 0;                              // largest finite magnitude, as bits
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          const uint4 u = *reinterpret_cast<const uint4*>(q + (i >> 3) * kHalf + (((i & 7) ^ (r & 7)) << 4));
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const unsigned lo = w[k] & 0x7FFFu, hi = (w[k] >> 16) & 0x7FFFu;
            if (lo < 0x7F80u) mx = max(mx, lo);
            if (hi < 0x7F80u) mx = max(mx, hi);
          }
        }
        const int e = max((int)(mx >> 7), 15);        // biased exponent
        const float up = __uint_as_float((unsigned)(268 - e) << 23);
        f_row = p.c_log2 * __uint_as_float((unsigned)(e - 14) << 23);
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          uint4* at = reinterpret_cast<uint4*>(q + (i >> 3) * kHalf + (((i & 7) ^ (r & 7)) << 4));
          const uint4 u = *at;
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
          uint32_t h[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            asm("cvt.rn.f16x2.f32 %0, %1, %2;"
                : "=r"(h[k])
                : "f"(bf16hi(w[k]) * up), "f"(bf16lo(w[k]) * up));
          *at = make_uint4(h[0], h[1], h[2], h[3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(smem_u32(&bars->q_ok[slot]));
      }
      const int cnt0 = cnt;
      // one event: halves (bits) of the CTA's key tile `tile`, at key0; part: of which
      // halves some row may not read all keys
      auto event = [&](int key0, int tile, unsigned halves, unsigned part) -> bool {
        unsigned w[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};   // keys it reads
        if (part) {
          const int hi = geo.tree ? min(ctx, pos + 1) : pos + 1;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int k = key0 + 32 * q;
            w[q] = below(hi - k);
            if (geo.window > 0) w[q] &= ~below(pos - geo.window + 1 - k) | below(geo.sinks - k);
            if (pos < 0) w[q] = 0u;
          }
          if (geo.tree && key0 + BK > ctx && pos >= 0) {
            int u = tok;
            for (int at = pos; u >= 0 && ctx + u >= key0; --at) {      // node u at position `at`
              const int bit = ctx + u - key0;
              if (bit >= 0 && bit < BK &&
                  (geo.window == 0 || at > pos - geo.window || at < geo.sinks)) {
#pragma unroll
                for (int q = 0; q < 4; ++q) w[q] |= (bit >> 5) == q ? 1u << (bit & 31) : 0u;
              }
              const int up = ld_int(p.parents, (int64_t)c.w.b * geo.max_q + u,
                                    (int64_t)geo.B * geo.max_q, p.err);
              u = up < u ? up : -1;
            }
          }
        }
        if (!warp_wait(smem_u32(&bars->s_full[x]), (uint32_t)(cnt & 1))) return false;
        tc_fence_after();
        const unsigned pages = kPaged ? (bars->rec[tile % 8] >> kPages) & 0xFFu : 0xFFu;
        uint32_t v[4][32];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if ((halves >> h) & 1u) {
            tmem_ld32(s_addr + 64 * h, v[2 * h]);
            tmem_ld32(s_addr + 64 * h + 32, v[2 * h + 1]);
          }
        tmem_ld_wait();
        tc_fence_before();                            // S may be overwritten
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->s_read));
        if (pages != 0xFFu) {                         // keys whose pages are not there
          part = 3u;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            w[q] &= ((pages >> (2 * q)) & 1u ? 0xFFFFu : 0u) |
                    ((pages >> (2 * q + 1)) & 1u ? 0xFFFF0000u : 0u);
        }
        if (part)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (((halves >> h) & 1u) &&
                __any_sync(0xffffffffu, (w[2 * h] & w[2 * h + 1]) != 0xFFFFFFFFu)) {
#pragma unroll
              for (int q = 2 * h; q < 2 * h + 2; ++q)
#pragma unroll
                for (int i = 0; i < 32; ++i) v[q][i] = (w[q] >> i) & 1u ? v[q][i] : 0xff800000u;
            }
        // row maximum (chains of their own)
        const bool fresh = cnt == cnt0;
        float alpha = 1.f;                            // of O_x
        const float2* scale = bars->scale[tile % 8];
        if (!kF8) {
          float mh[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if ((halves >> h) & 1u) {
              float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int q = 2 * h; q < 2 * h + 2; ++q)
#pragma unroll
                for (int i = 0; i < 32; i += 2)
                  mx4[(i >> 1) & 3] = fmax3(mx4[(i >> 1) & 3], __uint_as_float(v[q][i]),
                                            __uint_as_float(v[q][i + 1]));
              mh[h] = fmaxf(fmax3(mx4[0], mx4[1], mx4[2]), mx4[3]);
            }
          const float mt = fmaxf(mh[0], mh[1]) * p.c_log2;
          if (fresh) {
            m_ref = mt;                               // P.V of the first event overwrites O
          } else if (mt > m_ref + kLazy) {
            alpha = ex2(m_ref - mt);
            l_run *= alpha;
            m_ref = mt;
          }
        } else {
          // e = s f_row ks (log2 of a weight); m for the sum, M for P = 2^(e + log2 vs - M)
          float mt = -INFINITY, Mt = -INFINITY;
#pragma unroll
          for (int g = 0; g < 8; ++g)
            if ((halves >> (g >> 2)) & 1u) {
              float a = -INFINITY, b = -INFINITY;
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const uint32_t* u = &v[g >> 1][(g & 1) * 16 + i];
                a = fmax3(a, __uint_as_float(u[0]), __uint_as_float(u[1]));
                b = fmax3(b, __uint_as_float(u[2]), __uint_as_float(u[3]));
              }
              const float2 sc = scale[g];
              const float e = fmaxf(a, b) * fmaxf(f_row * sc.x, 1.17549435e-38f);
              mt = fmaxf(mt, e);
              Mt = fmaxf(Mt, e + sc.y);
            }
          Mt -= kTop;
          if (fresh) {
            m_ref = mt;
            M_ref = Mt;
          } else {
            if (mt > m_ref + kLazy) {
              l_run *= ex2(m_ref - mt);
              m_ref = mt;
            }
            if (Mt > M_ref + kLazy) {
              alpha = ex2(M_ref - Mt);
              M_ref = Mt;
            }
          }
        }
        const bool move = !fresh && __any_sync(0xffffffffu, alpha != 1.f);
        // P_x may be overwritten and O_x is complete once the last event's P.V is done
        auto settle = [&]() -> bool {
          if (cnt > 0 && !warp_wait(smem_u32(&bars->pv_done[x]), (uint32_t)((cnt - 1) & 1))) return false;
          tc_fence_after();
          if (move) {
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[32];
              tmem_ld32(o_addr + q * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(o_addr + q * 32, o);
            }
          }
          return true;
        };
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
        if (!settle()) return false;
        // P = 2^(S c - m) as bf16 pairs (E4M3: f16, with the value scale), and the row sum
        // (four chains)
        const float M_use = M_ref == -INFINITY ? 0.f : M_ref;
        const uint64_t negm2 = f2(-m_use, -m_use);
        uint64_t sum4[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if ((halves >> h) & 1u) {
            uint32_t pk[32];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint64_t fac = c2, top = 0ull;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                if (kF8 && i % 8 == 0) {              // the next 16 keys
                  const float2 sc = scale[4 * h + 2 * q + i / 8];
                  const float fk = fmaxf(f_row * sc.x, 1.17549435e-38f);
                  const float up = fminf(ex2(sc.y + (m_use - M_use)), 8.5e37f);
                  fac = f2(fk, fk);
                  top = f2(up, up);
                }
                float t0, t1;
                f2_split(ffma2(f2(__uint_as_float(v[2 * h + q][2 * i]),
                                  __uint_as_float(v[2 * h + q][2 * i + 1])),
                               fac, negm2),
                         t0, t1);
                const float p0 = ex2(t0), p1 = ex2(t1);
                sum4[i & 3] = fadd2(sum4[i & 3], f2(p0, p1));
                if (kF8) {
                  float w0, w1;
                  f2_split(fmul2(f2(p0, p1), top), w0, w1);
                  pk[q * 16 + i] = pack_f16x2(w0, w1);
                } else {
                  pk[q * 16 + i] = pack_bf16x2(p0, p1);
                }
              }
            }
            tmem_st32(p_addr + 32 * h, pk);
          }
        float s_lo, s_hi;
        f2_split(fadd2(fadd2(sum4[0], sum4[1]), fadd2(sum4[2], sum4[3])), s_lo, s_hi);
        l_run += s_lo + s_hi;
        tmem_st_wait();
        if (part) {
          const int pr = tile % C::kVs;
          if (!warp_wait(smem_u32(&bars->v_ok[tile % 8]), (uint32_t)((tile / 8) & 1))) return false;
          const unsigned* bad = bars->bad[pr];
          if (((halves & 1u) && (bad[0] | bad[1])) || ((halves & 2u) && (bad[2] | bad[3]))) {
            // values that are not finite, for the rows that read them: P times value
            if (fresh) {
#pragma unroll 1
              for (int i = 0; i < D; ++i) tmem_st1(o_addr + i, 0u);
              tmem_st_wait();
            }
#pragma unroll 1
            for (int k = 0; k < BK; ++k) {
              if (!((halves >> (k >> 6)) & 1u) || !((bad[k >> 5] >> (k & 31)) & 1u)) continue;
              const unsigned rw = k < 32 ? w[0] : (k < 64 ? w[1] : (k < 96 ? w[2] : w[3]));
              const bool reads = (rw >> (k & 31)) & 1u;
              const uint32_t two = tmem_ld1(p_addr + k / 2);
              const float pk = kF8 ? f16_to_f32(two, k & 1) : ((k & 1) ? bf16hi(two) : bf16lo(two));
              int64_t at;                             // the value's first element
              bool inside;
              if (kPaged) {
                const int page = key0 + k < c.w.lk
                                     ? ld_int(p.block_table,
                                              (int64_t)c.w.b * p.max_pages + ((key0 + k) >> p.page_shift),
                                              (int64_t)geo.B * p.max_pages, p.err)
                                     : -1;
                at = (((int64_t)page * geo.Hkv + c.h) * p.page_size + ((key0 + k) & (p.page_size - 1))) * D;
                inside = (unsigned)page < (unsigned)p.num_pages;
              } else {
                at = (int64_t)(c.w.k0 + key0 + k) * p.ldv + (int64_t)c.h * D;
                inside = key0 + k < c.w.lk;
              }
#pragma unroll 1
              for (int i = 0; i < D; ++i) {
                float o = __uint_as_float(tmem_ld1(o_addr + i));
                if (reads && inside && RF_IN(p.err, at + i, p.n_v)) {
                  const float val =
                      kF8 ? f16_to_f32(widen(static_cast<const uint8_t*>(p.V)[at + i], false), false)
                          : __bfloat162float(static_cast<const __nv_bfloat16*>(p.V)[at + i]);
                  o = fmaf(pk, val, o);
                }
                __syncwarp();
                tmem_st1(o_addr + i, __float_as_uint(o));
                tmem_st_wait();
              }
            }
          }
        }
        tc_fence_before();
        mbar_arrive(smem_u32(&bars->p_full[x]));
        ++cnt;
        return true;
      };
      const Whole whole = whole_of(geo, c.w);
      // tiles whose keys every row reads: window tiles from `begin` to `end`
      const int over = c.w.start - c.w.lead * BK;     // key0 of window tile j is over + j * BK
      const int full0 = max(c.w.lead, (max(whole.begin, c.w.start) - over + BK - 1) / BK);
      const int full1 = (max(whole.end, over) - over) / BK;
#pragma unroll 1
      for (int j = c.j0; j < c.j1; ++j) {
        int key0 = 0;
        unsigned halves = 3u, part = 0u;
        if (j < full0 || j >= full1 || kPaged) key0 = key0_of(c.w, j);
        if (j < full0 || j >= full1) {
          halves = (t.takes(2 * j) ? 1u : 0u) | (t.takes(2 * j + 1) ? 2u : 0u);
          if (!halves) continue;
          part = (whole.partly(geo, key0, kUnit) ? 1u : 0u) |
                 (whole.partly(geo, key0 + kUnit, kUnit) ? 2u : 0u);
        }
        ok = event(key0, j_base + j, halves, part);
        if (!ok) break;
      }
      if (*abort_flag) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // the piece's last product (over a cache, a tile may have no unit in it)
      if (cnt > cnt0 &&
          !__all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->pv_done[x]), (uint32_t)((cnt - 1) & 1)) && !*abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (pos < 0) l_run = 0.f;                       // it reads nothing: zeros
      const bool all = !kPaged || c.whole();
      const int64_t state = slot_of(cta, item0, x0) * 2 + x;
      const int64_t row = ((int64_t)c.w.q0 + tok) * p.ldo + (int64_t)(c.h * geo.G + my_g) * D;
      const bool out = real && RF_IN(p.err, row + D - 1,
                                     ((int64_t)(kPaged ? geo.B * geo.max_q : geo.total_q) - 1) * p.ldo +
                                         (int64_t)p.Hq * D);
      // E4M3: 2^(M - m) / l in two factors, since 2^(M - m) itself may underflow
      const float half = kF8 ? ex2(0.5f * (M_ref - m_ref)) : 1.f;
      const float inv = l_run == 0.f ? 0.f : half / l_run;
      uint8_t* stage = smem + slot * C::kTile;        // (its queries came before their scores)
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        tmem_ld32(o_addr + q * 32, o);
        tmem_ld_wait();
        if (all) {
          if (out || C::kStaged) {
            // a row that read no key: zeros, whatever O holds
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t u[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                u[k] = l_run == 0.f ? 0u
                                    : pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * inv * half,
                                                  __uint_as_float(o[8 * i + 2 * k + 1]) * inv * half);
              const uint4 o8 = make_uint4(u[0], u[1], u[2], u[3]);
              if (C::kStaged) {
                const int ch = q * 4 + i;
                *reinterpret_cast<uint4*>(stage + (ch >> 3) * kHalf + r * 128 +
                                          (((ch & 7) ^ (r & 7)) << 4)) = o8;
              } else {
                reinterpret_cast<uint4*>(p.O + row)[q * 4 + i] = o8;
              }
            }
          }
        } else if (real) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int64_t at = (state * (D / 4) + q * 8 + i) * BQ + r;
            if (RF_IN(p.err, at, (int64_t)4 * gridDim.x * (D / 4) * BQ))
              p.ws_o[at] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                       __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
          }
        }
      }
      if (C::kStaged) {
        // A row of its own for each lane cost 32 lines a store and 1.6 us a tile; 8 lanes
        // write a line of a row now.
        __syncwarp();
        const unsigned outs = __ballot_sync(0xffffffffu, out);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int from = i * 4 + (lane >> 3);       // the row's lane
          const int64_t at = __shfl_sync(0xffffffffu, row, from);
          const uint8_t* line = stage + (r - lane + from) * 128 + (((lane & 7) ^ (from & 7)) << 4);
          if ((outs >> from) & 1u)
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              reinterpret_cast<uint4*>(p.O + at)[h * 8 + (lane & 7)] =
                  *reinterpret_cast<const uint4*>(line + h * kHalf);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->q_empty[slot]));
      }
      if (!all && real && RF_IN(p.err, state * BQ + r, (int64_t)4 * gridDim.x * BQ))
        p.ws_st[state * BQ + r] = make_float4(kF8 ? M_ref : m_ref, m_ref, l_run, 0.f);
      tc_fence_before();                              // O is read before the next product writes it
    }
    if (!ok) {
      raise_error(p.err, kDevErrTimeout);
      *abort_flag = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the states of the items that are cut between CTAs.  Block (c - 1, x, part) has
// the item in which CTA c's range begins, if that is the item's first cut: tile x, kDims
// of its dims, a thread a row; pieces in key order.  The first is CTA c - 1's last, the
// others are the first of the CTAs from c on.
constexpr int kDims = 8;
template <int D>
__global__ void __launch_bounds__(BQ) merge_kernel(const __grid_constant__ Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Geo& geo = p.geo;
  const int c = (int)blockIdx.x + 1, x = blockIdx.y, part = blockIdx.z, r = threadIdx.x;
  const int ctas = (int)gridDim.x + 1;                // of the attention kernel
  if (!RF_IN(p.err, c, ctas)) return;
  const int4 cut = __ldcg(&p.ws_cut[c]);
  const int pieces = cut.x;
  if (pieces == 0) return;
  const Group w = group_of(geo, cut.y, false, p.err);
  const Tile t = tile_of(geo, w, x);
  const int my_t = r / geo.G, tok = t.t0 + my_t;
  if (my_t >= geo.tpt || tok >= t.t1) return;
  // All pieces' references first, then their sums, each loop with many loads in flight
  // and no branch (one running loop took 0.5 us a piece).  A piece that read no key has
  // l = 0, and its O may be anything.
  constexpr int kQuads = kDims / 4;
  const int64_t slots = (int64_t)4 * ctas;
  auto slot = [&](int i) -> int64_t {
    return (i == 0 ? 2 * (int64_t)(c - 1) + 1 : 2 * (int64_t)(c - 1 + i)) * 2 + x;
  };
  auto state = [&](int64_t s) -> float4 {
    return RF_IN(p.err, s, slots) ? __ldcg(&p.ws_st[s * BQ + r]) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float M = -INFINITY, m = -INFINITY, l = 0.f, v[kDims];        // bf16: M = m
#pragma unroll 8
  for (int i = 0; i < pieces; ++i) {
    const float4 st = state(slot(i));
    M = fmaxf(M, st.z == 0.f ? -INFINITY : st.x);
    m = fmaxf(m, st.z == 0.f ? -INFINITY : st.y);
  }
  const float Mu = M == -INFINITY ? 0.f : M, mu = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int k = 0; k < kDims; ++k) v[k] = 0.f;
#pragma unroll 4
  for (int i = 0; i < pieces; ++i) {
    const int64_t s = slot(i), at = (s * (D / 4) + part * kQuads) * BQ + r;
    const float4 st = state(s);
    const bool some = st.z != 0.f;
    const float f = some ? ex2(st.x - Mu) : 0.f;
    l = fmaf(st.z, some ? ex2(st.y - mu) : 0.f, l);
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
      const float4 u = RF_IN(p.err, at + k * BQ, slots * (D / 4) * BQ) ? __ldcg(&p.ws_o[at + k * BQ])
                                                                      : make_float4(0.f, 0.f, 0.f, 0.f);
      v[4 * k] = fmaf(some ? u.x : 0.f, f, v[4 * k]);
      v[4 * k + 1] = fmaf(some ? u.y : 0.f, f, v[4 * k + 1]);
      v[4 * k + 2] = fmaf(some ? u.z : 0.f, f, v[4 * k + 2]);
      v[4 * k + 3] = fmaf(some ? u.w : 0.f, f, v[4 * k + 3]);
    }
  }
  const int64_t row = ((int64_t)w.q0 + tok) * p.ldo +
                      (int64_t)(cut.z * geo.G + (r - my_t * geo.G)) * D + part * kDims;
  if (!RF_IN(p.err, row + kDims - 1, ((int64_t)geo.B * geo.max_q - 1) * p.ldo + (int64_t)p.Hq * D))
    return;
  const float half = M == m ? 1.f : ex2(0.5f * (M - m));
  const float inv = l == 0.f ? 0.f : half / l;
#pragma unroll
  for (int i = 0; i < kDims / 8; ++i) {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      u[k] = l == 0.f ? 0u : pack_bf16x2(v[8 * i + 2 * k] * inv * half, v[8 * i + 2 * k + 1] * inv * half);
    reinterpret_cast<uint4*>(p.O + row)[i] = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

template <int D, bool kPaged, bool kF8>
cudaError_t launch(const CUtensorMap (&tm)[3], Params& p, int grid, cudaStream_t s) {
  using C = Cfg<D, kPaged, kF8>;
  auto kern = attn_masked_kernel<D, kPaged, kF8>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<grid, C::kThreads, C::kSmem, s>>>(tm[0], tm[1], tm[2], p);
  e = cudaGetLastError();
  if (e != cudaSuccess || !kPaged || grid < 2) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid - 1, p.geo.max_q > p.geo.tpt ? 2 : 1, D / kDims);
  cfg.blockDim = dim3(BQ, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_kernel<D>, p);
}

size_t pad256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace masked

using masked::Geo;

namespace {

Geo packed_geo(const int* cu_q, const int* cu_k, int B, int Hkv, int G, int max_q, int total_q,
               int total_k, int window, int sinks) {
  Geo g = {};
  g.cu_q = cu_q;
  g.cu_k = cu_k;
  g.B = B;
  g.Hkv = Hkv;
  g.G = G;
  g.tpt = masked::BQ / G;
  g.npairs = (int)(((int64_t)max_q + 2 * g.tpt - 1) / (2 * g.tpt));
  g.max_q = max_q;
  g.total_q = total_q;
  g.total_k = total_k;
  g.window = window;
  g.sinks = sinks;
  return g;
}

Geo paged_geo(const int* seq_lens, int B, int Hkv, int G, int Tq, int max_len, int window, int sinks,
              bool tree) {
  Geo g = packed_geo(nullptr, nullptr, B, Hkv, G, Tq, 0, 0, window, sinks);
  g.seq_lens = seq_lens;
  g.max_len = max_len;
  g.tree = tree;
  return g;
}

}  // namespace

cudaError_t launch_attn_fwd_window(const void* Q, int64_t ldq, const void* K, int64_t ldk,
                                   const void* V, int64_t ldv, void* O, int64_t ldo,
                                   const int* cu_q, const int* cu_k, int B, int Hq, int Hkv,
                                   int max_q, int total_q, int total_k, int d, float scale,
                                   int window, int sinks, unsigned* err, cudaStream_t s) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidValue;
  masked::Params p = {};
  p.geo = packed_geo(cu_q, cu_k, B, Hkv, Hq / Hkv, max_q, total_q, total_k, window, sinks);
  p.O = static_cast<__nv_bfloat16*>(O);
  p.V = V;
  p.ldo = ldo;
  p.ldv = ldv;
  p.n_v = (int64_t)(total_k - 1) * ldv + (int64_t)Hkv * d;
  p.Hq = Hq;
  p.c_log2 = scale * 1.4426950408889634f;
  p.err = err;
  CUtensorMap tm[3];
  const CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!encode_tmap_3d(&tm[0], t, Q, d, Hq, total_q, d * 2, ldq * 2, 64, p.geo.G, p.geo.tpt, true) ||
      !encode_tmap_3d(&tm[1], t, K, d, Hkv, total_k, d * 2, ldk * 2, 64, 1, masked::BK, true) ||
      !encode_tmap_3d(&tm[2], t, V, d, Hkv, total_k, d * 2, ldv * 2, 64, 1, masked::BK, true))
    return cudaErrorInvalidValue;
  return d == 64 ? masked::launch<64, false, false>(tm, p, sms, s)
                 : masked::launch<128, false, false>(tm, p, sms, s);
}

// Workspace: partial states [2 SMs][2][d / 4][128] float4, (M, m, l) [2 SMs][2][128],
// the cuts [SMs].
size_t masked_rows_workspace_bytes(int d) {
  const int sms = sm_count();
  if (sms <= 0) return 0;
  const size_t rows = (size_t)sms * 4 * masked::BQ;
  return rows * d * sizeof(float) + rows * sizeof(float4) + masked::pad256(sms * sizeof(int4));
}

cudaError_t launch_masked_rows(const PagedKV& c, const Mask& mask, const void* Q, void* O, int Hq,
                               int Tq, float scale, void* workspace, unsigned* err,
                               cudaStream_t s) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidValue;
  masked::Params p = {};
  p.geo = paged_geo(c.seq_lens, c.B, c.Hkv, Hq / c.Hkv, Tq, c.max_pages * c.page_size, mask.window,
                    mask.sinks, mask.parents != nullptr);
  p.O = static_cast<__nv_bfloat16*>(O);
  p.V = c.v;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.ldo = (int64_t)Hq * c.d;
  const uint64_t keys = (uint64_t)c.num_pages * c.Hkv * c.page_size;
  p.n_v = (int64_t)keys * c.d;
  p.parents = mask.parents;
  p.block_table = c.block_table;
  p.Hq = Hq;
  p.num_pages = c.num_pages;
  p.page_size = c.page_size;
  p.page_shift = c.page_size == 16 ? 4 : (c.page_size == 32 ? 5 : (c.page_size == 64 ? 6 : 7));
  p.max_pages = c.max_pages;
  p.c_log2 = scale * 1.4426950408889634f;
  p.err = err;
  const size_t rows = (size_t)sms * 4 * masked::BQ;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.ws_o = reinterpret_cast<float4*>(ws);
  ws += rows * c.d * sizeof(float);
  p.ws_st = reinterpret_cast<float4*>(ws);
  ws += rows * sizeof(float4);
  p.ws_cut = reinterpret_cast<int4*>(ws);
  CUtensorMap tm[3];
  const CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int d = c.d;
  if (!encode_tmap_3d(&tm[0], t, Q, d, Hq, (uint64_t)c.B * Tq, d * 2, (uint64_t)Hq * d * 2, 64,
                      p.geo.G, p.geo.tpt, true))
    return cudaErrorInvalidValue;
  const bool f8 = c.dtype == RF_E4M3;
  for (int i = 0; i < 2; ++i) {
    const void* base = i ? c.v : c.k;
    if (!(f8 ? encode_tmap_2d(&tm[1 + i], CU_TENSOR_MAP_DATA_TYPE_UINT8, base, 128, keys * d / 128,
                              128, 128, c.page_size * d / 128, true)
             : encode_tmap_2d(&tm[1 + i], t, base, d, keys, d * 2, 64, c.page_size, true)))
      return cudaErrorInvalidValue;
  }
  if (f8)
    return d == 64 ? masked::launch<64, true, true>(tm, p, sms, s)
                   : masked::launch<128, true, true>(tm, p, sms, s);
  return d == 64 ? masked::launch<64, true, false>(tm, p, sms, s)
                 : masked::launch<128, true, false>(tm, p, sms, s);
}

// Host-side walk of the plan (the functions of the header, shared by host and device)
// for `sms` CTAs.  Returns 0 when every invariant holds, else the number of the first
// that fails:
//   1 no index leaves its array;
//   2 the CTAs' pieces, end to end, are all items' tiles, in order, once;
//   3 a prompt's items are whole; over a cache a CTA cuts at most its first and its
//     last item, into slots of their own;
//   4 the merge counts a cut item's pieces and finds their slots, in key order;
//   5 every row with tokens lies in one tile of one item;
//   6 every key that a row reads lies in exactly one half of a key tile that its tile
//     takes;
//   7 over a cache whose queries are converted in place, a query tile's place is never
//     the other's, and its loads are counted one by one; a prompt's query tiles all take
//     something of their item.
int masked_plan_selfcheck(const int* seq_lens, const int* cu_q, const int* cu_k, int B, int Hkv,
                          int G, int max_q, int total_q, int total_k, int window, int sinks,
                          int tree, int sms) {
  using namespace masked;
  const Geo p = seq_lens ? paged_geo(seq_lens, B, Hkv, G, max_q, total_k, window, sinks, tree != 0)
                         : packed_geo(cu_q, cu_k, B, Hkv, G, max_q, total_q, total_k, window, sinks);
  unsigned err = 0;
  const int ng = p.B * p.npairs;
  std::vector<int64_t> pre((size_t)ng + 1, 0);
  int64_t items = 0;
  int most = 0;
  for (int g = 0; g < ng; ++g) {
    const int n = places(p, group_of(p, g, true, &err));
    pre[(size_t)g + 1] = pre[(size_t)g] + (int64_t)n * Hkv;
    most = imax(most, n);
    items += n > 0 ? Hkv : 0;
  }
  const int64_t total = pre[(size_t)ng];
  if (err & kDevErrBounds) return 1;
  const int grid = total < sms ? (int)total : sms;
  std::vector<int> want_rows((size_t)B, 0), rows((size_t)B, 0);
  for (int g = 0; g < ng; ++g) {
    const Group w = group_of(p, g, false, &err);
    want_rows[(size_t)w.b] = w.lq;
    if (w.n > 0) rows[(size_t)w.b] += w.t1 - w.t0;
    for (int x = 0; w.n > 0 && x < 2; ++x) {
      const Tile t = tile_of(p, w, x);
      if (!t.has()) continue;
      if (t.t1 - t.t0 > p.tpt) return 5;
      bool takes = seq_lens != nullptr;
      for (int u = 0; u < 2 * w.n; ++u) takes |= t.takes(u);
      if (!takes) return 7;
      for (int i = t.t0; i < t.t1; ++i) {
        // a tree's node may be at any position from its first on, and reads no other key
        const int at[2] = {p.tree ? w.lk - w.lq : w.lk - w.lq + i, p.tree ? w.lk - 1 : w.lk - w.lq + i};
        for (int key = 0; key < w.lk; ++key) {
          const bool reads = key <= at[1] && (window == 0 || at[0] - key < window || key < sinks);
          int hits = 0;
          for (int u = 0; u < 2 * w.n; ++u) {
            const int k0 = key0_of(w, u >> 1) + (u & 1) * kUnit;
            hits += t.takes(u) && key >= k0 && key < k0 + kUnit;
          }
          if (reads ? hits != 1 : hits > 1) return 6;
        }
      }
    }
  }
  for (int b = 0; b < B; ++b)
    if (rows[(size_t)b] != want_rows[(size_t)b]) return 5;
  if (total == 0) return 0;
  const Split64 split(total, grid);
  const bool keep = seq_lens && keeps_items(items, most, total, grid);
  std::vector<int64_t> begins;                        // of the items, if they are kept
  for (int g = 0; keep && g < ng; ++g)
    for (int h = 0; h < Hkv && pre[(size_t)g + 1] > pre[(size_t)g]; ++h)
      begins.push_back(pre[(size_t)g] + (pre[(size_t)g + 1] - pre[(size_t)g]) / Hkv * h);
  int64_t at = 0;                                     // where the last range ended
  int wg = -1, wh = Hkv - 1, wj = 0, wn = 0;          // the next tile in the order of all
  std::vector<unsigned char> used((size_t)2 * sms, 0);
  std::vector<int64_t> parts;                         // of the item being cut
  for (int c = 0; c < grid; ++c) {
    int64_t r[2];
    int start[3] = {0, 0, 0};
    for (int i = 0; i < 2; ++i) {
      r[i] = !keep ? split.start(c + i)
                   : ((size_t)(c + i) < begins.size() ? begins[(size_t)(c + i)] : total);
      if (r[i] >= total) continue;
      int g = 0;
      while (pre[(size_t)g + 1] <= r[i]) ++g;
      const Group w = group_of(p, g, false, &err);
      const int n = places(p, w);
      const int h = (int)((r[i] - pre[(size_t)g]) / n), off = (int)((r[i] - pre[(size_t)g]) % n);
      const bool up = !seq_lens && snaps_up(off, n);
      if (!seq_lens) r[i] += (up ? n : 0) - off;
      if (i == 0) {
        start[0] = g;
        start[1] = h;
        start[2] = seq_lens ? off : (up ? w.n : 0);
      }
    }
    if (r[0] != at || r[1] < r[0]) return 2;
    at = r[1];
    Walk walk(start[0], start[1], start[2], r[1] - r[0]);
    Piece pc;
    QTurns<2, true> q2(p);
    QTurns<4, true> q4(p);
    int turns[2][2][4] = {};                          // of 2 and 4 places, by tile and place
    auto in_turn = [&](int (&n)[2][4], int x, QPlace q) {
      return n[1 - x][q.slot] == 0 && q.turn == n[x][q.slot]++;
    };
    int cuts = 0;
    int64_t s0 = r[0] - (r[1] > r[0] ? start[2] : 0);
    while (walk.next(p, pc, &err)) {
      if (err & kDevErrBounds) return 1;
      const int64_t item0 = s0;
      s0 += pc.w.n;
      for (int x = 0; seq_lens && x < 2; ++x)
        if (tile_of(p, pc.w, x).has() &&
            !(in_turn(turns[0], x, q2.next(x)) && in_turn(turns[1], x, q4.next(x))))
          return 7;
      for (int j = pc.j0; j < pc.j1; ++j) {
        if (wj == wn) {                               // on to the next item
          wj = 0;
          if (++wh == Hkv) {
            wh = 0;
            do {
              ++wg;
            } while (wg < ng && pre[(size_t)wg + 1] == pre[(size_t)wg]);
          }
          if (wg >= ng) return 2;
          wn = group_of(p, wg, false, &err).n;
        }
        const Group w = group_of(p, wg, false, &err);
        if (pc.w.b != w.b || pc.w.t0 != w.t0 || pc.h != wh || j != wj) return 2;
        ++wj;
      }
      if (pc.whole()) continue;
      if (!seq_lens || keep || ++cuts > 2) return 3;
      const int64_t slot = slot_of(c, item0, r[0]);
      if (slot < 0 || slot >= 2 * (int64_t)sms || used[(size_t)slot]++) return 3;
      if (pc.j0 == 0) parts.clear();
      parts.push_back(slot);
      if (pc.j1 == pc.w.n) {                          // the last piece: as the merge finds them
        const int64_t s1 = item0 + pc.w.n;
        const int c0 = split.owner(item0), pieces = split.owner(s1 - 1) - c0 + 1;
        if ((int)parts.size() != pieces || split.start(c0 + 1) <= item0 || split.start(c0) > item0)
          return 4;
        for (int i = 0; i < pieces; ++i)
          if (parts[(size_t)i] != (i == 0 ? 2 * (int64_t)c0 + 1 : 2 * (int64_t)(c0 + i))) return 4;
      }
    }
  }
  if (at != total || wj != wn || wh != Hkv - 1) return 2;
  for (++wg; wg < ng; ++wg)
    if (pre[(size_t)wg + 1] != pre[(size_t)wg]) return 2;
  return 0;
}

}  // namespace rf

// decode_paged.cu -- decode attention over a paged cache, bf16 or E4M3 with
// one scale per (page, kv head) for keys and one for values.
//
// For kv head h of sequence b, the R = Tq * G query rows (Tq query tokens of
// G = Hq / Hkv heads) all read the same keys, so they form one tile:
//     s_rj = scale * ks_j * (q_r . kc_j),    j <= len - Tq + t(r),
//     o_r  = sum_j softmax(s_r)_j vs_j vc_j
// with kc, vc the stored codes (or bf16 values) and ks, vs the scales of key
// j's page.  Tiles hold 8 or 16 rows; more rows make more tiles (a tile is
// named by b and hr = h * tiles + tile).
//
// What bounds it, up to 16 rows: memory.  Every cached byte is read once for each
// tile of its kv head, and the arithmetic per byte is small (16 flop at G = 8 in
// E4M3).  mma.sync keeps the operands in registers, which is what an 8-bit cache needs: codes are
// widened on their way into the fragments and never go back to shared memory.
// The cache is the A operand (16 keys or 16 dims by 16) and the few query
// rows are the B operand (n = 8), so a fragment is widened once for all rows of
// a tile and no MMA row is padding:
//     S^T = K Q^T    (keys x rows),      O^T += V^T P^T   (dims x rows).
// S^T's accumulators become P^T's fragments by one movmatrix each.
//
// Numerics.  E4M3: codes are exact in f16; a query row is scaled by a power
// of two to a largest element in [2^14, 2^15), so its bf16 elements are exact
// in f16 down to 2^-28 of the row's largest; products are summed in fp32.
// The value scales enter the exponent: with e_j = log2 of the unnormalised
// weight, the kernel keeps a running maximum and a reference,
//     m = max_j e_j   for the sum   l = sum_j 2^(e_j - m),
//     M               for           o = sum_j 2^(e_j + log2 vs_j - M) vc_j,
// and out = o 2^(M - m) / l.  P = 2^(e_j + log2 vs_j - M) is rounded to f16
// (2^-11), finer than the bf16 output, and f16 keeps that for 29 binades, 2^-14
// to 2^15.  So M puts the largest P so far at 2^15; and since a key whose weight
// dwarfs all others' may have a value of zero, M comes down again where a whole
// chunk lies more than 16 binades below it: to the chunk's own largest, at most
// 48 binades, which o in fp32 holds (2^15 448 2^30 2^48 < 2^103).  bf16: P is
// split in two bf16 parts (hi + lo, 2^-17 together) for two MMAs, since
// values may be anything bf16 holds; M = m.
//
// Partition.  The 32-key chunks of all tiles, end to end in the order (b, hr,
// chunk), are cut into one equal range per CTA (at tile borders where all tiles
// are short) and each of these into one per warp.  A warp streams its range through a private ring of TMA stages and
// keeps the running state; where a tile begins and ends in a warp's range the
// warp writes its output itself.  At the end of the kernel one CTA barrier
// follows: the states of tiles cut between warps are merged by the CTA, and
// those cut between CTAs through the workspace by the CTA that draws the
// tile's last ticket, always in key order, so the bits do not depend on the
// order of arrival.  Lengths are read on the device: every CTA adds up all
// B lengths itself, so a captured graph follows lengths that change.  The
// tickets are zeroed by a small kernel before, whose programmatic dependent
// this one is.
//
// Inside a CTA: eight consumer warps (four where a stage is 16 KB), each with a
// ring of two to four stages of 32 keys, and four producer warps, half a warp a
// ring, that look pages up, issue the copies and fetch the scales.  With the
// copies issued by the consumers themselves a chunk took 1.7 us of a warp's
// time, 0.65 of it for the issue; now 1.05, and eight warps outrun memory.
//
// Measured (GB300, CUDA graph, inputs larger than L2; copy rate 6683 GB/s; bytes
// of the lengths that were timed, a mean of three batches):
//   32 x 24-32k keys, 8 kv heads of 4, E4M3   276 us   1.84 GB   6.7 TB/s
//   32 x 2048 keys, the same                  30.5 us  0.13 GB   4.4 TB/s
//   32 x 24-32k keys, 2 kv heads of 16, E4M3  92 us    0.46 GB   5.0 TB/s
//   9 x 3-20k keys, 7 kv heads of 5, bf16     60 us    0.36 GB   5.9 TB/s
//   48 x 1-4k keys, 16 heads of 64, bf16      68 us    0.41 GB   6.0 TB/s
//   16 x 0.5-8k keys, 4 kv heads of 8, four query tokens   0.07 GB in E4M3, 43 us;
//     0.14 GB in bf16, 55 us (32 rows are two tiles; a warp's chunk of 16 rows in
//     E4M3 takes 2.1 us, latency of the softmax and MMA chains, so memory waits;
//     that instance spills 32 bytes, too)
//   1 x 1000 keys, 8 kv heads of 4, E4M3      10.9 us, all latency: the plan 2,
//     page and first chunk 1.5, the chunk 1 (clock stamps); launch and merges.
// Of what a mid-sized call takes above its bytes (10 us for 32 x 2048 keys), 3.6
// pass before the first copy and 1.5 until it is in; the rest is the spread of the
// warps' ends and the merges.  Tried and left out: 32-row tiles with four warps (63
// against 43 us for the four query tokens: one warp a scheduler does not hide
// its own latency); values fetched during the softmax at eight rows (275 -> 280).
//
// Masked places.  Keys behind a sequence's last may hold anything: scores are
// selected, not added to, and values are replaced by zero.  Where the last Tq
// keys hold an infinity or NaN, which rows that may not read them would meet
// as 0 * inf, the chunk's product is taken token by token, and each row takes
// the one of its own token.
#include <math.h>

#include <algorithm>
#include <vector>

#include "rf_device.cuh"
#include "rf_internal.h"

namespace rf {
namespace {

constexpr int kChunk = 32;          // keys of a stage
constexpr int kTileRows = 16;       // query rows of a tile (at most)

// Sizes of one instance.
template <bool kF8, int D, int NT>
struct Cfg {
  static constexpr int kRowBytes = kF8 ? D : 2 * D;
  static constexpr int kTensorBytes = kChunk * kRowBytes;       // K or V of a stage
  static constexpr int kStageBytes = 2 * kTensorBytes;
  static constexpr int kWarps = kStageBytes > 8192 ? 4 : 8;
  static constexpr int kStages = kF8 ? (D == 128 ? 2 : 4) : (NT == 1 ? 3 : 2);
  static constexpr int kRings = kWarps / 4;                     // of a producer warp
  static constexpr int kConsumers = kWarps * 32;
  static constexpr int kThreads = kConsumers + 128;             // + four producer warps
  // Registers: 384 threads start with 168 each (64512); the two consumer
  // warpgroups take 208 (53248) of them and the producers keep 88 (11264).
  // With four consumer warps everyone has the compiler's 255 at most.
  static constexpr int kConsumerRegs = kWarps == 8 ? 208 : 0;
  static constexpr int kProducerRegs = kWarps == 8 ? 88 : 0;
  static constexpr int kRows = 8 * NT;
  static constexpr int kPitch = D + 4;                          // floats of a state's row
  static constexpr int kStateBytes = kRows * kPitch * 4 + kRows * 16;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kSmem = 1024 + kRingBytes + kWarps * kStateBytes;
  static_assert(kStateBytes <= kStages * kStageBytes, "a state fits the warp's ring");
};

// ------------------------------------------------------------- the plan
// The same code on the device and, for the self-check, on the host.

struct Lens {
  const int* seq_lens;
  int B, HR;               // HR: tiles of a sequence
  int max_len;
};

__host__ __device__ __forceinline__ int seq_len(const Lens& p, int b, bool report, unsigned* err) {
  const int len = ld_int(p.seq_lens, b, p.B, err);
  if (len < 0 || len > p.max_len) {
    if (report) note_error(err, kDevErrInput);
    return 0;
  }
  return len;
}
__host__ __device__ __forceinline__ unsigned num_chunks(int len) {
  return ((unsigned)len + kChunk - 1) / kChunk;
}

// T chunks over g CTAs (or warps) in ranges, the first T % g of them one longer.
struct Split {
  unsigned q, rem;
  __host__ __device__ __forceinline__ Split(unsigned T, unsigned g) : q(T / g), rem(T % g) {}
  __host__ __device__ __forceinline__ unsigned start(unsigned c) const {
    return c * q + (c < rem ? c : rem);
  }
  __host__ __device__ __forceinline__ unsigned owner(unsigned x) const {
    const unsigned big = rem * (q + 1);
    return x < big ? x / (q + 1) : rem + (x - big) / q;
  }
};

// As many CTAs as give every warp at least one chunk.
__host__ __device__ __forceinline__ unsigned ctas_for(unsigned total, unsigned sms, unsigned W) {
  const unsigned want = total / W + (total % W ? 1u : 0u);
  return want < 1u ? 1u : (want < sms ? want : sms);
}

// Short tiles are not cut between CTAs: merging through the workspace costs
// about 3.5 us, three or four chunks' time.  Where no tile has more than 2 W
// chunks (two a warp), the CTAs' ranges therefore begin at the tile border that
// is next to the even cut.
__host__ __device__ __forceinline__ bool keeps_tiles(unsigned max_chunks, unsigned W) {
  return max_chunks <= 2 * W;
}
// The border next to chunk x, the off-th of a tile of nck.
__host__ __device__ __forceinline__ unsigned snap(unsigned x, unsigned off, unsigned nck) {
  return 2 * off < nck ? x - off : x - off + nck;
}

// Where the chunks of all tiles stand in one order: chunk ck of tile hr of
// sequence b (of len keys, nck chunks a tile).
struct Cursor {
  int b, hr, len;
  unsigned ck, nck;
  // Chunk `off` of the tiles of sequence b0, of len0 keys; false if there is none.
  __host__ __device__ __forceinline__ bool init(const Lens& p, int b0, int len0, unsigned off) {
    b = b0;
    len = len0;
    nck = num_chunks(len);
    hr = 0;
    ck = 0;
    if (nck == 0 || off / nck >= (unsigned)p.HR) return false;
    hr = (int)(off / nck);
    ck = off % nck;
    return true;
  }
  // On to the next chunk; false if there is none (on the device: the lengths
  // changed under the kernel).
  __host__ __device__ __forceinline__ bool next(const Lens& p, unsigned* err) {
    if (++ck < nck) return true;
    ck = 0;
    if (++hr < p.HR) return true;
    hr = 0;
    while (++b < p.B) {
      len = seq_len(p, b, false, err);
      nck = num_chunks(len);
      if (nck > 0) return true;
    }
    return false;
  }
};

// Workspace slot of CTA c's part of a tile that begins at chunk s0 (in the
// order of all chunks) and is cut between CTAs: only the first and the last
// tile of a CTA's range can be.
__host__ __device__ __forceinline__ int64_t slot_of(const Split& ctas, unsigned s0, unsigned c) {
  return 2 * (int64_t)c + (s0 < ctas.start(c) ? 0 : 1);
}

// ------------------------------------------------------------- device side

struct Params {
  const __nv_bfloat16* Q;
  __nv_bfloat16* O;
  const int* block_table;
  const float* k_scale;
  const float* v_scale;
  float* ws_o;            // [2 * grid][16][D]
  float4* ws_st;          // [2 * grid][16]: M, m, l
  unsigned* tickets;      // [B * HR]
  unsigned* err;
  Lens lens;
  int Hq, Hkv, G, Tq, R, tiles;            // HR = Hkv * tiles
  int num_pages, page_size, page_shift, max_pages;      // page_size = 1 << page_shift
  float scale_log2;
};

struct Meta {             // of a stage, written when its copies are issued
  float ks[2], vs[2];     // scales of the two 16-key halves (cp.async)
  int b, hr, ck, len;     // as in Cursor
  int valid;              // bit i: half i's page is one of the cache's
  int pad[3];
};

struct Seg {              // a state left at the barrier
  int b, hr, len;
  unsigned s0;            // first chunk of the tile in the order of all chunks
};

template <int W, int S>
struct Shared {
  uint64_t full[W][S], empty[W][S];
  Meta meta[W][S];
  Seg seg[W][2];          // [0] the warp's first state, [1] its last
  int has[W][2];
  unsigned warp_sum[W + 4], warp_most[W + 4], border[2];
  int start_b[W], start_len[W];
  unsigned start_off[W];
  int fail;
  int last[2];
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <bool kF8>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (kF8)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Volatile, so that they stay between the wait for a stage and its refill, but
// without a memory clobber: the arithmetic between them may move.
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t* w) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr));
}
__device__ __forceinline__ void lds64(uint32_t addr, uint32_t* w) {
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
}

// Two E4M3 codes (the low or high half of a word) -> two f16, exact.
__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The same for weights, whose largest is 2^15 but for the rounding of its
// exponent: not above f16's largest value.
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// E4M3's M (see the file's head): log2 of the largest P, and by how many binades
// a chunk may lie below M before M comes down, and how far it may.
constexpr float kTopP = 15.f, kLag = 16.f, kDrop = 48.f;
__device__ __forceinline__ float next_ref(float M, float chunk, float top) {
  return chunk < M - kLag ? fmaxf(chunk, top - kDrop) : fmaxf(M, chunk);
}
// out = o x y: 2^(M - m) / l in two factors, since 2^(M - m) itself may underflow.
// (0, 0) for a row without keys.
__device__ __forceinline__ float2 out_factors(float M, float m, float l) {
  const float y = ex2(0.5f * (M - m));
  return l == 0.f ? make_float2(0.f, 0.f) : make_float2(y / l, y);
}

template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
  if (N > 0) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N > 0 ? N : 24));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
  if (N > 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N > 0 ? N : 24));
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on `bar` when this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Waits until the kernel before this one (a programmatic dependent of it) has
// completed and its writes are visible.
__device__ __forceinline__ void griddep_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ unsigned atom_acq_rel_add(unsigned* p, unsigned v) {
  unsigned r;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(r) : "l"(p), "r"(v) : "memory");
  return r;
}

// ------------------------------------------------------------- fragments

// E4M3.  A stage's K (and V) is [32 keys][D bytes], 128-byte swizzled rows;
// at D = 64 a 128-byte row holds two keys.
template <int D>
__device__ __forceinline__ uint32_t f8_off(int key, int byte) {
  const int row = D == 128 ? key : key >> 1;
  const int col = D == 128 ? byte : (key & 1) * 64 + byte;
  return (uint32_t)(row * 128 + (((col >> 4) ^ (row & 7)) << 4) + (col & 15));
}
// bf16: boxes of 64 dims, [32 keys][128 bytes] each.
__device__ __forceinline__ uint32_t bf_off(int key, int c16) {
  return (uint32_t)((c16 >> 3) * (kChunk * 128) + key * 128 + (((c16 & 7) ^ (key & 7)) << 4));
}

// K fragments of 16 keys (half mt) for one k-step of 16 dims.  Which dims a
// k-step holds is free as long as Q's fragments agree.  E4M3: lane (g, c)
// holds dims [c D/4, (c+1) D/4) of keys g and g + 8, four a step, so that
// its loads are 16 bytes.  bf16: natural order, by ldmatrix.
template <bool kF8, int D>
struct KFrag {
  uint32_t w0[D / 16], w1[D / 16];
  __device__ __forceinline__ void load(uint32_t base, int mt, int lane) {
    if (kF8) {
      const int g = lane >> 2, c = lane & 3;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        lds128(base + f8_off<D>(mt * 16 + g, c * (D / 4) + 16 * i), w0 + 4 * i);
        lds128(base + f8_off<D>(mt * 16 + g + 8, c * (D / 4) + 16 * i), w1 + 4 * i);
      }
    }
  }
  __device__ __forceinline__ void get(uint32_t base, int mt, int lane, int ks,
                                      uint32_t (&a)[4]) const {
    if (kF8) {
      a[0] = widen_lo(w0[ks]);
      a[1] = widen_lo(w1[ks]);
      a[2] = widen_hi(w0[ks]);
      a[3] = widen_hi(w1[ks]);
    } else {
      const int mi = lane >> 3, mr = lane & 7;
      ldsm4(base + bf_off(mt * 16 + (mi & 1) * 8 + mr, 2 * ks + (mi >> 1)), a);
    }
  }
};

// O += V^T P^T for the 16 keys of half mt.  Which dims an m-tile holds is
// free too.  E4M3: lane (g, c) reads dims [g D/8, (g+1) D/8) of keys 2c, 2c+1,
// 2c+8, 2c+9; m-tile i's rows g and g + 8 are dims g D/8 + 2i and + 1.
// bf16: natural order.  Modes: kAll; kMask, keys at or beyond lim (counted
// within the chunk) are replaced by zero; kSome, the same, and only the rows
// whose bit is set in `rows` (bit 2 nt + e for this lane's row 2c + e) take
// the result.
enum { kAll, kMasked, kSome };
template <bool kF8, int D, int NT, int kMode>
__device__ __forceinline__ void pv16(float (&o)[D / 16][NT][4], uint32_t base, int mt, int lane,
                                     int lim, unsigned rows,
                                     const uint32_t (&p)[NT][kF8 ? 1 : 2][2]) {
  constexpr bool kMask = kMode != kAll;
  auto accumulate = [&](float(&acc)[4], const uint32_t(&a)[4], int nt) {
    float x[4] = {acc[0], acc[1], acc[2], acc[3]};
    mma16816<kF8>(x, a, p[nt][0][0], p[nt][0][1]);
    if (!kF8) mma16816<kF8>(x, a, p[nt][kF8 ? 0 : 1][0], p[nt][kF8 ? 0 : 1][1]);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc[e] = kMode != kSome || ((rows >> (2 * nt + (e & 1))) & 1u) ? x[e] : acc[e];
  };
  const int c = lane & 3;
  if (kF8) {
    constexpr int NW = D / 32;                   // words a key
    const int g = lane >> 2;
    uint32_t v[4][NW];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = mt * 16 + 2 * c + (i & 1) + (i >> 1) * 8;
      if (D == 128) lds128(base + f8_off<D>(key, g * (D / 8)), v[i]);
      else lds64(base + f8_off<D>(key, g * (D / 8)), v[i]);
      if (kMask && key >= lim)
#pragma unroll
        for (int j = 0; j < NW; ++j) v[i][j] = 0u;
    }
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      // bytes (key0 dim0, key1 dim0, key0 dim1, key1 dim1), then dims 2 and 3
      const uint32_t x0 = __byte_perm(v[0][j], v[1][j], 0x5140);
      const uint32_t x1 = __byte_perm(v[0][j], v[1][j], 0x7362);
      const uint32_t y0 = __byte_perm(v[2][j], v[3][j], 0x5140);
      const uint32_t y1 = __byte_perm(v[2][j], v[3][j], 0x7362);
      const uint32_t a0[4] = {widen_lo(x0), widen_hi(x0), widen_lo(y0), widen_hi(y0)};
      const uint32_t a1[4] = {widen_lo(x1), widen_hi(x1), widen_lo(y1), widen_hi(y1)};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        accumulate(o[2 * j][nt], a0, nt);
        accumulate(o[2 * j + 1][nt], a1, nt);
      }
    }
  } else {
    const int mi = lane >> 3, mr = lane & 7;
    // which of this lane's keys 2c, 2c+1 (low, high halves), 2c+8, 2c+9 stay
    uint32_t keep0 = 0xFFFFFFFFu, keep1 = 0xFFFFFFFFu;
    if (kMask) {
      const int k0 = mt * 16 + 2 * c;
      keep0 = (k0 < lim ? 0xFFFFu : 0u) | (k0 + 1 < lim ? 0xFFFF0000u : 0u);
      keep1 = (k0 + 8 < lim ? 0xFFFFu : 0u) | (k0 + 9 < lim ? 0xFFFF0000u : 0u);
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t a[4];
      ldsm4t(base + bf_off(mt * 16 + (mi >> 1) * 8 + mr, 2 * i + (mi & 1)), a);
      if (kMask) {
        a[0] &= keep0;
        a[1] &= keep0;
        a[2] &= keep1;
        a[3] &= keep1;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) accumulate(o[i][nt], a, nt);
    }
  }
}

// Whether any value of keys [lo, hi) of the chunk is an infinity or NaN.
template <bool kF8, int D>
__device__ __forceinline__ bool any_nonfinite(uint32_t base, int lane, int lo, int hi) {
  bool bad = false;
  for (int key = lo; key < hi; ++key) {
    if (kF8) {
      if (lane < D / 16) {
        uint32_t w[4];
        lds128(base + f8_off<D>(key, lane * 16), w);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 32; e += 8) bad |= ((w[j] >> e) & 0x7Fu) == 0x7Fu;
      }
    } else if (lane < D / 8) {
      uint32_t w[4];
      lds128(base + bf_off(key, lane), w);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        bad |= (w[j] & 0x7F80u) == 0x7F80u || (w[j] & 0x7F800000u) == 0x7F800000u;
    }
  }
  return __any_sync(0xffffffffu, bad);
}

// ------------------------------------------------------------- the kernel

template <bool kF8, int D, int NT>
__global__ void __launch_bounds__(Cfg<kF8, D, NT>::kThreads, 1)
    decode_paged_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ Params p) {
  using C = Cfg<kF8, D, NT>;
  constexpr int W = C::kWarps, S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared<W, S> sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int cta = (int)blockIdx.x;
  const Lens& lens = p.lens;
  uint8_t* ring = smem + (warp < W ? warp : 0) * (S * C::kStageBytes);     // a consumer's
  const int64_t n_qo = (int64_t)lens.B * p.Tq * p.Hq * D;     // elements of Q and O

  // ---- plan: add up all lengths; find where each warp's range begins
  if (warp == W + 3) {                 // while the first warps fetch their lengths
    for (int i = lane; i < W * S; i += 32) {
      // the copies' bytes and, for E4M3, the two lanes that fetch scales
      mbar_init(smem_u32(&sh.full[i / S][i % S]), kF8 ? 3 : 1);
      mbar_init(smem_u32(&sh.empty[i / S][i % S]), 1);
    }
    fence_mbar_init();
    if (lane == 0) {
      sh.fail = 0;
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
    }
  }
  const bool consumer = warp < W;
  if (consumer && lane < 2) sh.has[warp][lane] = 0;
  if (consumer && lane == 0) sh.start_b[warp] = sh.start_len[warp] = 0;
  const int per = (lens.B + C::kThreads - 1) / C::kThreads;
  const int b_lo = min((int)threadIdx.x * per, lens.B), b_hi = min(b_lo + per, lens.B);
  unsigned mine = 0, most = 0;
  int first_len = 0;
  bool empty = false;
  for (int b = b_lo; b < b_hi; ++b) {
    const int len = seq_len(lens, b, cta == 0, p.err);
    if (b == b_lo) first_len = len;
    empty |= len == 0;
    most = max(most, num_chunks(len));
    mine += num_chunks(len) * (unsigned)lens.HR;
  }
  unsigned incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) {
    sh.warp_sum[warp] = incl;
    sh.warp_most[warp] = most;
  }
  const bool empties = __syncthreads_or(empty);
  unsigned pre = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < W + 4; ++w) {
    if (w < warp) pre += sh.warp_sum[w];
    total += sh.warp_sum[w];
    most = max(most, sh.warp_most[w]);
  }
  const unsigned grid = ctas_for(total, gridDim.x, W);
  const Split ctas(total, grid);
  unsigned r0 = ctas.start(cta), r1 = (unsigned)cta < grid ? ctas.start(cta + 1) : r0;
  if (keeps_tiles(most, W)) {
    for (int i = 0; i < 2; ++i) {
      const unsigned x = i ? r1 : r0;
      if (threadIdx.x == 0 && x >= total) sh.border[i] = total;
      if (x >= pre && x - pre < mine) {
        unsigned at = pre;
        for (int b = b_lo, len = first_len; b < b_hi;) {
          const unsigned nck = num_chunks(len), n = nck * (unsigned)lens.HR;
          if (x - at < n) {
            sh.border[i] = snap(x, (x - at) % nck, nck);
            break;
          }
          at += n;
          if (++b < b_hi) len = seq_len(lens, b, false, p.err);
        }
      }
    }
    __syncthreads();
    if ((unsigned)cta < grid) {
      r0 = sh.border[0];
      r1 = sh.border[1];
    }
  }
  const Split warps(r1 - r0, W);
  for (int w = 0; w < W; ++w) {
    const unsigned x = r0 + warps.start(w);
    if (x >= pre && x - pre < mine) {            // in this thread's sequences: walk to it
      unsigned at = pre;
      for (int b = b_lo, len = first_len; b < b_hi;) {
        const unsigned n = num_chunks(len) * (unsigned)lens.HR;
        if (x - at < n) {
          sh.start_b[w] = b;
          sh.start_len[w] = len;
          sh.start_off[w] = x - at;
          break;
        }
        at += n;
        if (++b < b_hi) len = seq_len(lens, b, false, p.err);
      }
    }
  }
  __syncthreads();
  // element of Q and O at which row r of kv head h of sequence b begins
  auto row_at = [&](int b, int h, int r) {
    const int t = p.Tq == 1 ? 0 : r / p.G;
    return (((int64_t)b * p.Tq + t) * p.Hq + (int64_t)h * p.G + (r - t * p.G)) * D;
  };

  if (!consumer) {
    setmaxnreg_dec<C::kProducerRegs>();
    // ---- producers: half a warp (or a whole one) keeps a consumer's ring full
    constexpr int kLanes = 32 / C::kRings;
    const int hl = lane % kLanes;
    const int w = (warp - W) * C::kRings + lane / kLanes;
    const unsigned half = C::kRings == 1 ? 0xFFFFFFFFu : (lane < 16 ? 0xFFFFu : 0xFFFF0000u);
    unsigned count = (unsigned)cta < grid ? warps.start(w + 1) - warps.start(w) : 0u;
    Cursor cur = {0, 0, 0, 0, 0};
    if (count > 0 && !cur.init(lens, sh.start_b[w], sh.start_len[w], sh.start_off[w])) count = 0;
    unsigned issued = 0;
    // evict first, so that queries, tables and states stay in L2 (32 x 2k keys 31.6 us
    // without, 30.2 with).  A cache that one tile a kv head reads passes through once;
    // several tiles read it once each
    const uint64_t policy = policy_evict_first();
    int pt = -1, pt_b = -1, pt_base = 0;  // kLanes entries of a block table row, one a lane
    bool failed = false;
    uint64_t t0 = 0;                      // since when nothing could be issued
    while (__any_sync(0xffffffffu, issued < count)) {
      const int slot = (int)(issued % S);
      bool go = issued < count &&
                (issued < S || mbar_test_wait(smem_u32(&sh.empty[w][slot]), (issued / S - 1) & 1));
      go = __shfl_sync(0xffffffffu, go, 0, kLanes);          // as the ring's first lane saw it
      if (!__any_sync(0xffffffffu, go)) {
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        failed = now - t0 > kDefaultWaitNs || *(volatile int*)&sh.fail;
        failed = __any_sync(0xffffffffu, failed);
        if (failed) break;
        __nanosleep(20);
        continue;
      }
      t0 = 0;
      if (!go) continue;
      Meta& mt = sh.meta[w][slot];
      const int first = (int)(cur.ck * kChunk);
      const int pg = first >> p.page_shift, in_page = first & (p.page_size - 1);
      const int halves = p.page_size < kChunk ? 2 : 1;
      if (cur.b != pt_b || pg < pt_base || pg + halves > pt_base + kLanes) {
        pt_b = cur.b;
        pt_base = pg;
        const int e = pg + hl;
        pt = e < (cur.len + p.page_size - 1) >> p.page_shift
                 ? ld_int(p.block_table, (int64_t)cur.b * p.max_pages + e,
                          (int64_t)lens.B * p.max_pages, p.err)
                 : -1;
      }
      const int h = p.tiles == 1 ? cur.hr : cur.hr / p.tiles;
      int page[2], valid = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int e = i < halves ? pg + i : pg;
        page[i] = __shfl_sync(half, pt, e - pt_base, kLanes);
        const bool ok = (unsigned)page[i] < (unsigned)p.num_pages;
        if (!ok) {
          if (hl == 0 && e * p.page_size < cur.len) raise_error(p.err, kDevErrInput);
          page[i] = 0;                             // read something of the cache; masked
        }
        valid |= ok ? 1 << i : 0;
      }
      const uint32_t bar = smem_u32(&sh.full[w][slot]);
      if (hl == 0) {
        mt.b = cur.b;
        mt.hr = cur.hr;
        mt.ck = (int)cur.ck;
        mt.len = cur.len;
        mt.valid = valid;
        const uint32_t dst = smem_u32(smem + (w * S + slot) * C::kStageBytes);
        mbar_arrive_expect_tx(bar, C::kStageBytes);
        constexpr int kKeysPerRow = kF8 && D == 64 ? 2 : 1;       // of the tensor map
        constexpr int kBoxes = !kF8 && D == 128 ? 2 : 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i >= halves) break;
          const int32_t y =
              ((page[i] * p.Hkv + h) * p.page_size + (halves == 2 ? 0 : in_page)) / kKeysPerRow;
          const uint32_t at = dst + i * (16 / kKeysPerRow) * 128;
#pragma unroll
          for (int x = 0; x < kBoxes; ++x) {
            tma_load_2d_hint(at + x * (kChunk * 128), &tmK, bar, 64 * x, y, policy);
            tma_load_2d_hint(at + x * (kChunk * 128) + C::kTensorBytes, &tmV, bar, 64 * x, y,
                             policy);
          }
        }
      }
      if (kF8 && hl < 2) {
        const int64_t at = (int64_t)(hl ? page[1] : page[0]) * p.Hkv + h;
        if (RF_IN(p.err, at, (int64_t)p.num_pages * p.Hkv)) {
          cp_async4(smem_u32(&mt.ks[hl]), p.k_scale + at);
          cp_async4(smem_u32(&mt.vs[hl]), p.v_scale + at);
        }
        cp_async_arrive(bar);
      }
      if (issued > 0 && cur.ck == 0) {             // the tile's queries: into L1 meanwhile
        for (int i = hl; i < C::kRows * (D / 64); i += kLanes) {       // pieces of 128 bytes
          const int r = (cur.hr - h * p.tiles) * kTileRows + i % C::kRows;
          if (r < p.R)
            asm volatile("prefetch.global.L1 [%0];" ::"l"(p.Q + row_at(cur.b, h, r) +
                                                          64 * (i / C::kRows)));
        }
      }
      ++issued;
      if (issued < count && !cur.next(lens, p.err)) count = issued;
    }
    if (failed && hl == 0) {
      raise_error(p.err, kDevErrTimeout);
      // copies in flight land before shared memory is released
      for (unsigned x = issued > S ? issued - S : 0; x < issued; ++x)
        (void)mbar_wait(smem_u32(&sh.full[w][x % S]), (x / S) & 1, 1000000ull);
    }
    return;
  }
  setmaxnreg_inc<C::kConsumerRegs>();

  // sequences without keys: their rows are zeros
  if (empties)
    for (int b = cta; b < lens.B; b += (int)gridDim.x) {
      if (seq_len(lens, b, false, p.err) > 0) continue;
      const int64_t n = (int64_t)p.Tq * p.Hq * D / 8;
      for (int64_t i = threadIdx.x; i < n; i += C::kConsumers)
        if (RF_IN(p.err, (b * n + i) * 8 + 7, n_qo))
          reinterpret_cast<uint4*>(p.O)[b * n + i] = make_uint4(0u, 0u, 0u, 0u);
    }
  if ((unsigned)cta >= grid || total == 0) {
    griddep_wait();
    return;
  }
  const unsigned x0 = r0 + warps.start(warp);
  const unsigned count = warps.start(warp + 1) - warps.start(warp);   // chunks of this warp

  // ---- the warp's range
  float o[D / 16][NT][4];
  float m[NT][2], M[NT][2], top[NT][2], l[NT][2], f[NT][2];    // top: M's largest
  int lim[NT][2];
  uint32_t q[D / 16][NT][2];
  unsigned done = 0;
  bool failed = false, fresh = true, first_seg = true;
  int cur_b = 0, cur_hr = 0, cur_len = 0;

  auto load_q = [&]() {
    const int h = p.tiles == 1 ? cur_hr : cur_hr / p.tiles;
    const int r0_ = (cur_hr - h * p.tiles) * kTileRows;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0_ + nt * 8 + g;
      const int64_t at = row_at(cur_b, h, r);
      const bool ok = r < p.R && RF_IN(p.err, at + D - 1, n_qo);
      if (kF8) {
        uint32_t w[D / 8];                    // bf16 pairs: dims [c D/4, (c+1) D/4)
        const uint4* src = reinterpret_cast<const uint4*>(p.Q + at + c * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 x = ok ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
          w[4 * i] = x.x;
          w[4 * i + 1] = x.y;
          w[4 * i + 2] = x.z;
          w[4 * i + 3] = x.w;
        }
        unsigned mx = 0;                      // largest finite magnitude, as bits
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const unsigned lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
          if (lo < 0x7F80u) mx = max(mx, lo);
          if (hi < 0x7F80u) mx = max(mx, hi);
        }
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = max((int)(mx >> 7), 15);           // biased exponent
        const float up = __uint_as_float((unsigned)(268 - e) << 23);
        const float fr = p.scale_log2 * __uint_as_float((unsigned)(e - 14) << 23);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          q[i >> 1][nt][i & 1] = pack_f16x2(bf16lo(w[i]) * up, bf16hi(w[i]) * up);
        f[nt][0] = __shfl_sync(0xffffffffu, fr, 8 * c);
        f[nt][1] = __shfl_sync(0xffffffffu, fr, 8 * c + 4);
      } else {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(p.Q + at);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          q[ks][nt][0] = ok ? __ldg(src + 8 * ks + c) : 0u;
          q[ks][nt][1] = ok ? __ldg(src + 8 * ks + c + 4) : 0u;
        }
        f[nt][0] = f[nt][1] = p.scale_log2;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = p.Tq == 1 ? 0 : min((r0_ + nt * 8 + 2 * c + e) / p.G, p.Tq - 1);
        lim[nt][e] = cur_len - p.Tq + t + 1;             // keys this row reads
      }
    }
  };

  // This warp's state -> buffer: rows of D floats, then (M, m, l).
  auto put_state = [&](uint8_t* buf) {
    float* fo = reinterpret_cast<float*>(buf);
    float4* st = reinterpret_cast<float4*>(buf + C::kRows * C::kPitch * 4);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nt * 8 + 2 * c + e;
        float* row = fo + r * C::kPitch;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          if (kF8) {
            *reinterpret_cast<float2*>(row + g * (D / 8) + 2 * i) =
                make_float2(o[i][nt][e], o[i][nt][e + 2]);
          } else {
            row[16 * i + g] = o[i][nt][e];
            row[16 * i + g + 8] = o[i][nt][e + 2];
          }
        }
        if (g == 0) st[r] = make_float4(M[nt][e], m[nt][e], l[nt][e], 0.f);
      }
  };

  // A whole tile's rows, from the registers.
  auto put_rows = [&]() {
    const int h = p.tiles == 1 ? cur_hr : cur_hr / p.tiles;
    const int r0_ = (cur_hr - h * p.tiles) * kTileRows;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float2 w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        w[e] = kF8 ? out_factors(M[nt][e], m[nt][e], l[nt][e])
                   : make_float2(l[nt][e] == 0.f ? 0.f : 1.f / l[nt][e], 1.f);
      if (kF8) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = r0_ + nt * 8 + 2 * c + e;
          const int64_t at = row_at(cur_b, h, r) + g * (D / 8);
          if (r < p.R && RF_IN(p.err, at + D / 8 - 1, n_qo)) {
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
              uint32_t u[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                u[k] = pack_bf16x2(o[4 * i + k][nt][e] * w[e].x * w[e].y,
                                   o[4 * i + k][nt][e + 2] * w[e].x * w[e].y);
              reinterpret_cast<uint4*>(p.O + at)[i] = make_uint4(u[0], u[1], u[2], u[3]);
            }
          }
        }
      } else {
        const int r = r0_ + nt * 8 + g;
        const int64_t at = row_at(cur_b, h, r);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t u =
                movmatrix(pack_bf16x2(o[i][nt][2 * k] * w[0].x, o[i][nt][2 * k + 1] * w[1].x));
            if (r < p.R && RF_IN(p.err, at + 16 * i + 8 * k + 2 * c + 1, n_qo))
              reinterpret_cast<uint32_t*>(p.O + at)[8 * i + 4 * k + c] = u;
          }
      }
    }
  };

  for (unsigned it = 0; it < count; ++it) {
    const int slot = (int)(it % S);
    const Meta& mt = sh.meta[warp][slot];
    if (fresh) {
      // the first tile's queries are fetched while its first chunk is on its way
      if (it == 0) {
        Cursor cur;
        (void)cur.init(lens, sh.start_b[warp], sh.start_len[warp], sh.start_off[warp]);
        cur_b = cur.b;
        cur_hr = cur.hr;
        cur_len = cur.len;
        load_q();
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[nt][e] = M[nt][e] = top[nt][e] = -INFINITY;
          l[nt][e] = 0.f;
        }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
    }
    const bool ok = mbar_wait(smem_u32(&sh.full[warp][slot]), (it / S) & 1);
    if (!__all_sync(0xffffffffu, ok)) {
      failed = true;
      done = it;
      break;
    }
    const int ck = mt.ck;
    if (fresh && it > 0) {
      cur_b = mt.b;
      cur_hr = mt.hr;
      cur_len = mt.len;
      load_q();
    }
    fresh = false;
    const uint32_t kb = smem_u32(ring + slot * C::kStageBytes), vb = kb + C::kTensorBytes;
    const int key0 = ck * kChunk;
    const int valid = mt.valid;
    const bool tail = key0 + kChunk > cur_len - p.Tq + 1 || valid != 3;
    float kscale[2], lv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool in = ((valid >> i) & 1) && key0 + 16 * i < cur_len;
      kscale[i] = kF8 && in ? mt.ks[i] : 1.f;
      lv[i] = kF8 ? (in ? __log2f(mt.vs[i]) : 0.f) : 0.f;
    }

    // ---- S^T = K Q^T.  An accumulator's products follow one another, so the two
    // halves (and at NT = 1 the even and odd k-steps) go in parallel chains.
    float s[2][NT][4];
    {
      constexpr int kChains = NT == 1 ? 2 : 1;
      float s2[2][kChains][NT][4];
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
        for (int x = 0; x < kChains; ++x)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s2[h2][x][nt][e] = 0.f;
      KFrag<kF8, D> kf[2];
      kf[0].load(kb, 0, lane);
      kf[1].load(kb, 1, lane);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          uint32_t a[4];
          kf[h2].get(kb, h2, lane, ks, a);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816<kF8>(s2[h2][ks % kChains][nt], a, q[ks][nt][0], q[ks][nt][1]);
        }
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[h2][nt][e] = kChains == 2 ? s2[h2][0][nt][e] + s2[h2][kChains - 1][nt][e]
                                        : s2[h2][0][nt][e];
    }

    // ---- running maxima and sums (log2 units); element (k, e): key g + 8 k, row 2c + e
    // (step by step for all rows together, so that their chains overlap)
    uint32_t pb[2][NT][kF8 ? 1 : 2][2];
    const bool two = kF8 && lv[0] != lv[1];
    float cm[NT][2], cM[NT][2], mu[NT][2], Mu[NT][2], a_o[NT][2];
    if (tail) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (key0 + 16 * h2 + g + 8 * k >= lim[nt][e] || !((valid >> h2) & 1))
                s[h2][nt][2 * k + e] = -INFINITY;
    }
    // the factors are positive, so the largest product has the largest score; one
    // that underflows (queries and a page of zeros, whose products are 0 either
    // way) must not turn a masked -inf into NaN
    float sc[2][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx[2];
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          sc[h2][nt][e] = fmaxf(f[nt][e] * kscale[h2], 1.17549435e-38f);
          mx[h2] = fmaxf(s[h2][nt][e], s[h2][nt][2 + e]) * sc[h2][nt][e];
        }
        cm[nt][e] = fmaxf(mx[0], mx[1]);
        cM[nt][e] = fmaxf(mx[0] + (lv[0] - kTopP), mx[1] + (lv[1] - kTopP));
      }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          cm[nt][e] = fmaxf(cm[nt][e], __shfl_xor_sync(0xffffffffu, cm[nt][e], x));
    if (two) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            cM[nt][e] = fmaxf(cM[nt][e], __shfl_xor_sync(0xffffffffu, cM[nt][e], x));
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) cM[nt][e] = cm[nt][e] + (lv[0] - kTopP);
    }
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mn = fmaxf(m[nt][e], cm[nt][e]);
        mu[nt][e] = mn == -INFINITY ? 0.f : mn;
        l[nt][e] *= ex2(m[nt][e] - mu[nt][e]);
        m[nt][e] = mn;
        if (kF8) top[nt][e] = fmaxf(top[nt][e], cM[nt][e]);
        const float Mn = kF8 ? next_ref(M[nt][e], cM[nt][e], top[nt][e]) : mn;
        Mu[nt][e] = Mn == -INFINITY ? 0.f : Mn;
        a_o[nt][e] = ex2(M[nt][e] - Mu[nt][e]);
        moved |= Mn != M[nt][e];
        M[nt][e] = Mn;
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float v = s[h2][nt][2 * k + e], x = sc[h2][nt][e];
            const float pr = ex2(fmaf(v, x, -mu[nt][e]));
            l[nt][e] += pr;
            w[e] = kF8 ? ex2(fmaf(v, x, lv[h2] - Mu[nt][e])) : pr;
          }
          // P^T as B fragments
          if (kF8) {
            pb[h2][nt][0][k] = movmatrix(pack_weights(w[0], w[1]));
          } else {
            const uint32_t hi = pack_bf16x2(w[0], w[1]);
            pb[h2][nt][0][k] = movmatrix(hi);
            pb[h2][nt][kF8 ? 0 : 1][k] =
                movmatrix(pack_bf16x2(w[0] - bf16lo(hi), w[1] - bf16hi(hi)));
          }
        }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          o[i][nt][0] *= a_o[nt][0];
          o[i][nt][1] *= a_o[nt][1];
          o[i][nt][2] *= a_o[nt][0];
          o[i][nt][3] *= a_o[nt][1];
        }
    }

    // ---- O^T += V^T P^T
    if (!tail) {
      pv16<kF8, D, NT, kAll>(o, vb, 0, lane, 0, 0u, pb[0]);
      pv16<kF8, D, NT, kAll>(o, vb, 1, lane, 0, 0u, pb[1]);
    } else {
      int end[2];                              // keys of each half that exist
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) end[h2] = ((valid >> h2) & 1) ? cur_len - key0 : 0;
      const int lo = max(cur_len - p.Tq + 1 - key0, 0), hi = min(cur_len - key0, kChunk);
      if (p.Tq > 1 && any_nonfinite<kF8, D>(vb, lane, lo, hi)) {
#pragma unroll 1
        for (int t = 0; t < p.Tq; ++t) {       // the rows of one query token at a time
          unsigned rows = 0;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (((cur_hr % p.tiles) * kTileRows + nt * 8 + 2 * c + e) / p.G == t)
                rows |= 1u << (2 * nt + e);
          if (!__any_sync(0xffffffffu, rows != 0)) continue;
          const int seen = cur_len - p.Tq + t + 1 - key0;
          pv16<kF8, D, NT, kSome>(o, vb, 0, lane, min(end[0], seen), rows, pb[0]);
          pv16<kF8, D, NT, kSome>(o, vb, 1, lane, min(end[1], seen), rows, pb[1]);
        }
      } else {
        pv16<kF8, D, NT, kMasked>(o, vb, 0, lane, end[0], 0u, pb[0]);
        pv16<kF8, D, NT, kMasked>(o, vb, 1, lane, end[1], 0u, pb[1]);
      }
    }

    // ---- the stage is free; end of a tile or of the range
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.empty[warp][slot]));
    const bool tile_end = (unsigned)ck + 1 == num_chunks(cur_len);
    if (tile_end || it + 1 == count) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);
      const unsigned s0 = x0 + it - (unsigned)ck;      // the tile's first chunk
      if (tile_end && s0 >= x0) {
        put_rows();
      } else {
        // the first state has a buffer of its own, since the ring is in use;
        // the last one (nothing is in flight any more) takes the ring
        const int which = first_seg ? 0 : 1;
        put_state(which == 0 ? smem + C::kRingBytes + warp * C::kStateBytes : ring);
        if (lane == 0) {
          sh.has[warp][which] = 1;
          Seg& sg = sh.seg[warp][which];
          sg.b = cur_b;
          sg.hr = cur_hr;
          sg.len = cur_len;
          sg.s0 = s0;
        }
      }
      first_seg = false;
      fresh = true;
    }
  }
  if (failed) {
    raise_error(p.err, kDevErrTimeout);
    sh.fail = 1;                               // ends the producers
    // copies in flight land before shared memory is released (the producer may
    // have ended already)
    for (unsigned x = done; x < count && x < done + S; ++x)
      (void)mbar_wait(smem_u32(&sh.full[warp][x % S]), (x / S) & 1, 1000000ull);
  }
  griddep_wait();                              // the tickets are zero
  named_bar_sync(1, C::kConsumers);
  if (sh.fail) return;

  // ---- merge the states that warps left, in key order
  // entry e = (warp e / 2, state e % 2); groups of neighbouring entries belong to
  // one tile
  constexpr int E = 2 * W;
  const bool here = lane < E && sh.has[(lane >> 1) % W][lane & 1] != 0;
  const unsigned mask = __ballot_sync(0xffffffffu, here);
  if (mask == 0) return;
  const unsigned my_s0 = sh.seg[(lane >> 1) % W][lane & 1].s0;
  const unsigned below = mask & ((1u << lane) - 1u);
  const int prev = below ? 31 - __clz((int)below) : lane;
  const unsigned prev_s0 = __shfl_sync(0xffffffffu, my_s0, prev);
  const unsigned starts = __ballot_sync(0xffffffffu, here && (below == 0 || prev_s0 != my_s0));
  const int n_groups = __popc(starts);
  auto state_of = [&](int e) {
    return (e & 1) ? smem + (e >> 1) * (S * C::kStageBytes)
                   : smem + C::kRingBytes + (e >> 1) * C::kStateBytes;
  };
  const int rows = min(p.R, C::kRows);       // of a tile (its last one may have fewer)
  auto has_row = [&](int hr, int r) { return p.tiles == 1 || hr % p.tiles * kTileRows + r < p.R; };
  const int64_t n_slots = 2 * (int64_t)gridDim.x * kTileRows;
  // first entries of the (at most two) tiles that are cut between CTAs: the
  // first and the last group
  int cut0 = -1, cut1 = -1;
  {
    const int ea = __ffs(starts) - 1, eb = 31 - __clz((int)starts);
    const Seg &sa = sh.seg[ea >> 1][ea & 1], &sb = sh.seg[eb >> 1][eb & 1];
    if (sa.s0 < r0 || sa.s0 + num_chunks(sa.len) > r1) cut0 = ea;
    if (eb != ea && sb.s0 + num_chunks(sb.len) > r1) cut1 = eb;
  }
  // half a warp for every group and row, an entry's (M, m, l) a lane
  constexpr int NV = D / 16;                 // dims a lane holds of a row
  const int hw = threadIdx.x >> 4, l16 = lane & 15;
  const unsigned half = lane < 16 ? 0xFFFFu : 0xFFFF0000u;
  auto max16 = [&](float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(half, v, o));
    return v;
  };
  auto sum16 = [&](float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(half, v, o);
    return v;
  };
  auto put_row = [&](const Seg& sg, int r, float2 w, const float (&v)[NV]) {
    const int h = p.tiles == 1 ? sg.hr : sg.hr / p.tiles;
    const int64_t at = row_at(sg.b, h, (sg.hr - h * p.tiles) * kTileRows + r) + NV * l16;
    if (!RF_IN(p.err, at + NV - 1, n_qo)) return;
    uint32_t u[NV / 2];
#pragma unroll
    for (int i = 0; i < NV / 2; ++i)
      u[i] = pack_bf16x2(v[2 * i] * w.x * w.y, v[2 * i + 1] * w.x * w.y);
    if (NV == 8)
      *reinterpret_cast<uint4*>(p.O + at) = make_uint4(u[0], u[1], u[NV / 2 - 2], u[NV / 2 - 1]);
    else
      *reinterpret_cast<uint2*>(p.O + at) = make_uint2(u[0], u[1]);
  };
#pragma unroll 1
  for (int i = hw; i < n_groups * rows; i += 2 * W) {
    int gi = i / rows;
    const int r = i - gi * rows;
    unsigned left = starts;
    for (; gi > 0; --gi) left &= left - 1;
    const int e0 = __ffs(left) - 1;
    const unsigned rest = left & (left - 1);
    const int e1 = rest ? __ffs(rest) - 1 : E;           // entries e0 .. e1 - 1
    const Seg sg = sh.seg[e0 >> 1][e0 & 1];
    if (!has_row(sg.hr, r)) continue;
    float4 st = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
    if (l16 >= e0 && l16 < e1 && ((mask >> l16) & 1u))
      st = reinterpret_cast<const float4*>(state_of(l16) + C::kRows * C::kPitch * 4)[r];
    const float Mx = max16(st.x), mx = max16(st.y);
    const float Mu = Mx == -INFINITY ? 0.f : Mx, mu = mx == -INFINITY ? 0.f : mx;
    const float wo = ex2(st.x - Mu), L = sum16(st.z * ex2(st.y - mu));
    float v[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] = 0.f;
#pragma unroll 2
    for (int e = e0; e < e1; ++e) {
      const float we = __shfl_sync(half, wo, e, 16);
      if ((mask >> e) & 1u) {
        const float4* row = reinterpret_cast<const float4*>(
            reinterpret_cast<const float*>(state_of(e)) + r * C::kPitch + NV * l16);
#pragma unroll
        for (int k = 0; k < NV / 4; ++k) {
          const float4 x = row[k];
          v[4 * k] = fmaf(x.x, we, v[4 * k]);
          v[4 * k + 1] = fmaf(x.y, we, v[4 * k + 1]);
          v[4 * k + 2] = fmaf(x.z, we, v[4 * k + 2]);
          v[4 * k + 3] = fmaf(x.w, we, v[4 * k + 3]);
        }
      }
    }
    if (e0 != cut0 && e0 != cut1) {
      put_row(sg, r, out_factors(Mu, mu, L), v);
    } else {
      const int64_t at = slot_of(ctas, sg.s0, cta) * kTileRows + r;
      if (RF_IN(p.err, at, n_slots)) {
        float4* dst = reinterpret_cast<float4*>(p.ws_o + at * D + NV * l16);
#pragma unroll
        for (int k = 0; k < NV / 4; ++k)
          dst[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        if (l16 == 0) p.ws_st[at] = make_float4(Mx, mx, L, 0.f);
      }
    }
  }
  if (cut0 < 0 && cut1 < 0) return;
  // ---- tiles cut between CTAs: the last CTA to arrive merges.  The barrier
  // orders the CTA's stores before the ticket's release.
  named_bar_sync(1, C::kConsumers);
  if (threadIdx.x < 2) {
    const int e0 = threadIdx.x ? cut1 : cut0;
    unsigned last = 0;
    if (e0 >= 0) {
      const Seg& sg = sh.seg[e0 >> 1][e0 & 1];
      const unsigned s1 = sg.s0 + num_chunks(sg.len);
      const unsigned pieces = ctas.owner(s1 - 1) - ctas.owner(sg.s0) + 1;
      const int64_t tile = (int64_t)sg.b * lens.HR + sg.hr;
      if (RF_IN(p.err, tile, (int64_t)lens.B * lens.HR))
        last = atom_acq_rel_add(&p.tickets[tile], 1u) == pieces - 1;
    }
    sh.last[threadIdx.x] = (int)last;
  }
  named_bar_sync(1, C::kConsumers);
#pragma unroll 1
  for (int i = hw; i < 2 * rows; i += 2 * W) {
    const int k2 = i / rows, r = i - k2 * rows;
    const int ek = k2 ? cut1 : cut0;
    if (ek < 0 || !sh.last[k2]) continue;
    const Seg sg = sh.seg[ek >> 1][ek & 1];
    if (!has_row(sg.hr, r)) continue;
    const unsigned s1 = sg.s0 + num_chunks(sg.len);
    const int c0 = (int)ctas.owner(sg.s0), pieces = (int)ctas.owner(s1 - 1) - c0 + 1;
    auto at_piece = [&](int j) { return slot_of(ctas, sg.s0, c0 + j) * kTileRows + r; };
    // 16 pieces at a time, a piece's (M, m, l) a lane, with the running maxima
    // carried over; the loads of kBatch pieces' rows go together
    float Mx = -INFINITY, mx = -INFINITY, L = 0.f, v[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] = 0.f;
    for (int j0 = 0; j0 < pieces; j0 += 16) {
      constexpr int kBatch = 4;
      const int n = min(pieces - j0, 16);
      float4 x[kBatch][NV / 4];
      auto load = [&](int j) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
#pragma unroll
          for (int k = 0; k < NV / 4; ++k) {
            x[u][k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j + u < n && RF_IN(p.err, at_piece(j0 + j + u), n_slots))
              x[u][k] = __ldcg(reinterpret_cast<const float4*>(
                                   p.ws_o + at_piece(j0 + j + u) * D + NV * l16) + k);
          }
      };
      load(0);
      float4 st = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
      if (l16 < n && RF_IN(p.err, at_piece(j0 + l16), n_slots))
        st = __ldcg(&p.ws_st[at_piece(j0 + l16)]);
      float Mn = max16(st.x), mn = max16(st.y);
      Mn = fmaxf(Mn, Mx);
      mn = fmaxf(mn, mx);
      const float Mu = Mn == -INFINITY ? 0.f : Mn, mu = mn == -INFINITY ? 0.f : mn;
      const float wo = ex2(st.x - Mu), keep = ex2(Mx - Mu);
      const float l_new = sum16(st.z * ex2(st.y - mu));
      L = fmaf(L, ex2(mx - mu), l_new);
      Mx = Mn;
      mx = mn;
#pragma unroll
      for (int k = 0; k < NV; ++k) v[k] *= keep;
      for (int j = 0; j < n; j += kBatch) {
        if (j > 0) load(j);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const float wj = __shfl_sync(half, wo, (j + u) & 15, 16);
          if (j + u < n)
#pragma unroll
            for (int k = 0; k < NV / 4; ++k) {
              v[4 * k] = fmaf(x[u][k].x, wj, v[4 * k]);
              v[4 * k + 1] = fmaf(x[u][k].y, wj, v[4 * k + 1]);
              v[4 * k + 2] = fmaf(x[u][k].z, wj, v[4 * k + 2]);
              v[4 * k + 3] = fmaf(x[u][k].w, wj, v[4 * k + 3]);
            }
        }
      }
    }
    const float Mu = Mx == -INFINITY ? 0.f : Mx, mu = mx == -INFINITY ? 0.f : mx;
    put_row(sg, r, out_factors(Mu, mu, L), v);
  }
}

// Zeroes the tickets.  The decode kernel is its programmatic dependent: it may
// start as soon as this one has, and waits for it just before its tickets.
// What it reads until then was written before this kernel began, which is
// launched the ordinary way.  (A memset in its place has to end before the
// decode kernel starts.)
__global__ void __launch_bounds__(1024) zero_tickets_kernel(unsigned* tickets, int64_t n,
                                                            unsigned* err) {
  asm volatile("griddepcontrol.launch_dependents;");
  for (int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 1024)
    if (RF_IN(err, i, n)) tickets[i] = 0u;
}

template <bool kF8, int D, int NT>
cudaError_t launch(const PagedKV& c, const Params& p, int sms, cudaStream_t s) {
  using C = Cfg<kF8, D, NT>;
  const uint64_t keys = (uint64_t)c.num_pages * c.Hkv * c.page_size;
  const uint32_t box = (uint32_t)(c.page_size < kChunk ? c.page_size : kChunk);
  CUtensorMap tm[2];
  for (int i = 0; i < 2; ++i) {
    const void* base = i == 0 ? c.k : c.v;
    bool ok;
    if (kF8)                       // 128-byte rows: one key, or two of 64 dims
      ok = encode_tmap_2d(&tm[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, base, 128, keys * D / 128, 128,
                          128, box * D / 128, true);
    else
      ok = encode_tmap_2d(&tm[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, D, keys, D * 2, 64, box,
                          true);
    if (!ok) return cudaErrorInvalidValue;
  }
  auto kern = decode_paged_kernel<kF8, D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t tickets = (int64_t)p.lens.B * p.lens.HR;
  const int64_t ctas = (tickets + 1023) / 1024;
  zero_tickets_kernel<<<(unsigned)(ctas < sms ? ctas : sms), 1024, 0, s>>>(p.tickets, tickets,
                                                                          p.err);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms, 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tm[0], tm[1], p);
}

int tiles_of(int R) { return R / kTileRows + (R % kTileRows != 0); }   // R up to 2^31 - 1
size_t pad256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

// Chunks of the fullest batch the cache can hold, over all tiles.
int64_t decode_paged_max_chunks(int B, int Hkv, int R, int max_pages, int page_size) {
  const int64_t tiles = (int64_t)B * Hkv * tiles_of(R);
  const int64_t chunks = ((int64_t)max_pages * page_size + kChunk - 1) / kChunk;
  return tiles >= (1ll << 31) ? (1ll << 31) : tiles * chunks;
}

// Workspace: tickets [B * HR], partial rows [2 * SMs][16][d], their (M, m, l).
size_t decode_paged_workspace_bytes(int B, int Hkv, int R, int d) {
  const int sms = sm_count();
  if (sms <= 0) return 0;
  const size_t rows = (size_t)2 * sms * kTileRows;
  return pad256((size_t)B * Hkv * tiles_of(R) * sizeof(unsigned)) +
         pad256(rows * d * sizeof(float)) + rows * sizeof(float4);
}

cudaError_t launch_decode_paged(const PagedKV& c, const void* Q, void* O, int Hq, int Tq,
                                float scale, void* workspace, unsigned* err, cudaStream_t s) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidValue;
  Params p;
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.O = static_cast<__nv_bfloat16*>(O);
  p.block_table = c.block_table;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.Hq = Hq;
  p.Hkv = c.Hkv;
  p.G = Hq / c.Hkv;
  p.Tq = Tq;
  p.R = p.G * Tq;
  p.tiles = tiles_of(p.R);
  p.lens = Lens{c.seq_lens, c.B, c.Hkv * p.tiles, c.max_pages * c.page_size};
  p.num_pages = c.num_pages;
  p.page_size = c.page_size;
  p.page_shift = c.page_size == 16 ? 4 : (c.page_size == 32 ? 5 : (c.page_size == 64 ? 6 : 7));
  p.max_pages = c.max_pages;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.err = err;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t rows = (size_t)2 * sms * kTileRows;
  p.tickets = reinterpret_cast<unsigned*>(ws);
  ws += pad256((size_t)c.B * p.lens.HR * sizeof(unsigned));
  p.ws_o = reinterpret_cast<float*>(ws);
  ws += pad256(rows * c.d * sizeof(float));
  p.ws_st = reinterpret_cast<float4*>(ws);
  const bool f8 = c.dtype == RF_E4M3, one = p.R <= 8;
#define RF_GO(F8, DD) \
  return one ? launch<F8, DD, 1>(c, p, sms, s) : launch<F8, DD, 2>(c, p, sms, s)
  if (f8) {
    if (c.d == 64) RF_GO(true, 64);
    RF_GO(true, 128);
  }
  if (c.d == 64) RF_GO(false, 64);
  RF_GO(false, 128);
#undef RF_GO
}

// Host-side walk of the partition (the functions above, shared by host and
// device) for `sms` CTAs of `W` warps; seq_lens is a host array.  Returns 0
// when every invariant holds, else the number of the first that fails:
//   1 no index leaves its array;
//   2 the warps' ranges, end to end, are all chunks, in order, once;
//   3 a warp leaves at most two unfinished tiles: its first and its last;
//   4 a CTA leaves at most two tiles to the workspace, in slots of their own;
//   5 a tile cut between CTAs has the parts that the merge counts, in the
//     slots that it reads, in key order.
int decode_paged_plan_selfcheck(const int* seq_lens, int B, int HR, int max_len, int W, int sms) {
  const Lens lens = {seq_lens, B, HR, max_len};
  unsigned err = 0, total = 0, most = 0;
  std::vector<unsigned> pre((size_t)B + 1, 0);
  for (int b = 0; b < B; ++b) {
    const unsigned nck = num_chunks(seq_len(lens, b, true, &err));
    most = std::max(most, nck);
    total += nck * (unsigned)HR;
    pre[(size_t)b + 1] = total;
  }
  auto seq_of = [&](unsigned x) {
    return (int)(std::upper_bound(pre.begin(), pre.end(), x) - pre.begin()) - 1;
  };
  auto border = [&](unsigned x) {
    if (x == total) return total;
    const int b = seq_of(x);
    const unsigned nck = num_chunks(seq_len(lens, b, false, &err));
    return snap(x, (x - pre[(size_t)b]) % nck, nck);
  };
  if (total == 0) return 0;
  const unsigned grid = ctas_for(total, (unsigned)sms, (unsigned)W);
  const Split ctas(total, grid);
  Cursor want = {-1, HR - 1, 0, 0, 0};
  unsigned x = 0;                                       // next chunk in the order of all
  std::vector<std::vector<int64_t>> parts((size_t)B * HR);
  std::vector<unsigned char> used((size_t)2 * sms, 0);
  for (unsigned c = 0; c < grid; ++c) {
    unsigned r0 = ctas.start(c), r1 = ctas.start(c + 1);
    if (keeps_tiles(most, (unsigned)W)) {
      r0 = border(r0);
      r1 = border(r1);
    }
    const Split warps(r1 - r0, (unsigned)W);
    int cut_tiles = 0;
    int64_t last_cut = -1;
    for (int w = 0; w < W; ++w) {
      const unsigned x0 = r0 + warps.start(w), n = warps.start(w + 1) - warps.start(w);
      if (n == 0) continue;
      if (x0 != x) return 2;
      const int b = seq_of(x0);
      Cursor cur;
      if (!cur.init(lens, b, seq_len(lens, b, false, &err), x0 - pre[(size_t)b])) return 2;
      int left = 0;
      for (unsigned i = 0; i < n; ++i, ++x) {
        if (i > 0 && !cur.next(lens, &err)) return 2;
        if (err & kDevErrBounds) return 1;
        if (!want.next(lens, &err)) return 2;
        if (cur.b != want.b || cur.hr != want.hr || cur.ck != want.ck || cur.len != want.len)
          return 2;
        const bool tile_end = cur.ck + 1 == cur.nck;
        if (!tile_end && i + 1 != n) continue;
        const unsigned s0 = x0 + i - cur.ck, s1 = s0 + cur.nck;
        if (tile_end && s0 >= x0) continue;             // written by the warp itself
        if (left == 1 && i + 1 != n) return 3;          // the second state takes the ring
        if (++left > 2) return 3;
        const int64_t tile = (int64_t)cur.b * HR + cur.hr;
        if ((s0 < r0 || s1 > r1) && tile != last_cut) {
          if (keeps_tiles(most, (unsigned)W)) return 4;
          last_cut = tile;
          if (++cut_tiles > 2) return 4;
          const int64_t slot = slot_of(ctas, s0, c);
          if (slot < 0 || slot >= 2 * (int64_t)sms || used[(size_t)slot]++) return 4;
          const unsigned c0 = ctas.owner(s0);
          parts[(size_t)tile].push_back(slot);
          if (c0 + parts[(size_t)tile].size() - 1 != c) return 5;
          if (s1 <= r1 && parts[(size_t)tile].size() != ctas.owner(s1 - 1) - c0 + 1) return 5;
        }
      }
    }
  }
  return x == total ? 0 : 2;
}

}  // namespace rf

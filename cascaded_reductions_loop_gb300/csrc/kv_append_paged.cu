// kv_append_paged.cu -- appends new keys and values to a paged cache, with
// the keys' norm and rotation on the way, and (optionally) the norm and
// rotation of the same tokens' queries in the same launch.
//
// Layout.  Pages are [num_pages][Hkv][page_size][d]; the token at position p
// of sequence b lives in page block_table[b][p / page_size], slot
// p % page_size.  An E4M3 cache has one fp32 scale per (page, kv head) for
// keys and one for values: a value is code * scale.
//
// The 8-bit append is itself a cascade with a running state: the scale of a
// page's head is the smallest power of two s with absmax <= 448 s, and the
// absmax of a page that is filled a token at a time is a running maximum.
// When a new token raises it, the codes that the page holds already are
// rescaled to the new s.  The scale is a power of two so that this rescaling
// is exact except where a code falls into E4M3's subnormals (the format's
// relative step does not depend on the scale, so the choice costs at most one
// of its 18 binades).
//
// Work.  A bf16 cache needs nothing but the rows: a lane group takes a few
// heads of one token (rows kernel).  For E4M3 a scale must have one owner, so
// that no atomics are needed: a work item is one page of one sequence that
// receives tokens.
//  - step kernel (one new token a sequence, or up to 8, the same for all): one
//    lane group for the key rows and one for the value rows of an (item, head);
//    a page that has to be rescaled is rescaled by the whole warp.
//  - prompt kernel: CTAs that stay, each with an equal share of the (item, head)
//    pairs; a head's new rows are held in registers between the absmax and the
//    quantisation, so each is read once.
// Query rows are further CTAs of the same launch (norm_rope.cuh).
//
// What bounds it, measured (GB300, CUDA graph, inputs larger than L2; copy rate
// 6683 GB/s):
//   bf16 cache, 32768 tokens of 8 heads of 128   47 us, 6.1 TB/s: memory
//   bf16 cache, 8192 tokens of the same   15.7 us, 4.5 TB/s
//   bf16 cache, 11 prompts, 6.6k tokens of 16 heads of 64   19.8 us, 5.5 TB/s
//   E4M3 cache, 32768 tokens of 8 heads of 128   62 us, 3.5 TB/s: instructions
//     (norm, rotation, two maxima and two quantisations for eight keys and eight
//     values a lane; issue slots 57 % full) and the barrier between a head's
//     absmax and its quantisation
//   E4M3 cache, 8192 tokens of the same   22.7 us in pages of 64 tokens, 24.4 in
//     pages of 128; with 32 query heads 42.7: the kv CTAs that stay fill the SMs,
//     and the query CTAs begin where they end
//   E4M3 cache, 7 prompts, 10.7k tokens of 8 heads of 128   26 us
//   steps, 32 sequences, 8 kv and 32 query heads   3.5 us in E4M3, 3.2 in bf16:
//     launch latency
// Steps of the E4M3 prompt kernel, for the 7 prompts: one CTA an (item, head) with
// a serial search 36 us; several heads a CTA of 1024 threads, one an SM, 45-58;
// keys and values in CTAs of their own 33; packed arithmetic on shared
// coefficients 31; equal shares over two CTAs of 512 threads an SM, with the next
// head on its way, 27; maxima by one instruction 26.
#include <algorithm>
#include <vector>

#include "norm_rope.cuh"

namespace rf {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------- quantisation

// Exponent field (biased by 127) of the smallest power of two s >= 2^-126
// with a <= 448 s; a >= 0, finite.  448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < 1 ? 1 : e;
}

// Two values (already divided by the scale) -> two E4M3 codes, round to
// nearest even, saturating; NaN -> 0x7F.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// Two E4M3 codes -> two floats (exact).
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  float lo, hi;
  asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return make_float2(lo, hi);
}
// Four codes of a page whose scale grows by 1 / ratio.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  const float2 a = from_e4m3x2(w & 0xFFFFu), b = from_e4m3x2(w >> 16);
  return e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
}
__device__ __forceinline__ uint4 rescale16(uint4 w, float ratio) {
  return make_uint4(rescale4(w.x, ratio), rescale4(w.y, ratio), rescale4(w.z, ratio),
                    rescale4(w.w, ratio));
}

// Largest finite magnitude of eight values (infinities saturate and NaN keeps
// its code: neither sets the scale).  max passes over NaN; where an infinity is
// the largest, the others are looked at again.
__device__ __forceinline__ float absmax8(const Row8& y) {
  float v[8], a = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) f2_split(y.v[k], v[2 * k], v[2 * k + 1]);
#pragma unroll
  for (int k = 0; k < 4; ++k) a = fmax3(a, fabsf(v[2 * k]), fabsf(v[2 * k + 1]));
  if (a == INFINITY) {
    a = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) a = fabsf(v[e]) < INFINITY ? fmaxf(a, fabsf(v[e])) : a;
  }
  return a;
}
// The same of eight bf16 as loaded: magnitudes compare as whole numbers.
__device__ __forceinline__ float absmax8(const Raw8<__nv_bfloat16>& x) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t w = x.w[k] & 0x7FFF7FFFu;
    asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(w));
  }
  uint32_t a = max(m & 0xFFFFu, m >> 16);
  if (a >= 0x7F80u) {
    a = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = x.w[k] & 0x7FFFu, hi = (x.w[k] >> 16) & 0x7FFFu;
      if (lo < 0x7F80u) a = max(a, lo);
      if (hi < 0x7F80u) a = max(a, hi);
    }
  }
  return __uint_as_float(a << 16);
}
// Largest of the lanes' magnitudes (>= 0, so their bits compare as they do): one
// instruction where a butterfly takes five shuffles.
__device__ __forceinline__ float group_max(unsigned lanes, float a) {
  return __uint_as_float(__reduce_max_sync(lanes, __float_as_uint(a)));
}
__device__ __forceinline__ Row8 as_row(const Raw8<__nv_bfloat16>& x) {
  Row8 y;
#pragma unroll
  for (int k = 0; k < 4; ++k) y.v[k] = x.pair(k);
  return y;
}
// Eight values times 1 / scale as codes.
__device__ __forceinline__ uint2 quantise8(const Row8& y, float inv) {
  const uint64_t i2 = f2(inv, inv);
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float lo, hi;
    f2_split(fmul2(y.v[k], i2), lo, hi);
    c[k] = e4m3x2(lo, hi);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The scale of a page's head after the append: a = absmax of the new values,
// s_old the scale of the `off` tokens it holds (not looked at when off = 0).
__device__ __forceinline__ float new_scale(float a, float s_old, int off) {
  const float s = __uint_as_float((uint32_t)scale_exp(a) << 23);
  return off > 0 ? fmaxf(s, s_old) : s;
}

// ------------------------------------------------------------- the plan
// The same code on the device and, for the self-check, on the host.

struct Seqs {
  const int* block_table;
  const int* seq_lens;
  const int* cu;          // cumulative new tokens [B + 1], or nullptr: n_uniform each
  int B, n_uniform, total, num_pages, page_size, max_pages, Hkv;
  int max_len;            // longest length the rotation's tables and the block table allow
};

// New tokens of sequence b: token rows [first, first + n), positions
// [start, start + n).  n = 0 where there is nothing to do.
struct NewTokens {
  int first, n, start;
};

// report: note inconsistent sizes (one caller per sequence is enough).
__host__ __device__ __forceinline__ NewTokens new_tokens(const Seqs& sq, int b, bool report,
                                                         unsigned* err) {
  NewTokens r = {0, 0, 0};
  int c0, c1;
  if (sq.cu) {
    c0 = ld_int(sq.cu, b, sq.B + 1, err);
    c1 = ld_int(sq.cu, b + 1, sq.B + 1, err);
    if (c0 < 0 || c1 < c0 || c1 > sq.total) {
      if (report) note_error(err, kDevErrInput);
      return r;
    }
  } else {
    c0 = b * sq.n_uniform;
    c1 = c0 + sq.n_uniform;
  }
  const int len = ld_int(sq.seq_lens, b, sq.B, err);
  if (len == 0 || c1 == c0) return r;        // a padded row of the batch, or no new tokens
  if (len < c1 - c0 || len > sq.max_len) {
    if (report) note_error(err, kDevErrInput);
    return r;
  }
  r.first = c0;
  r.n = c1 - c0;
  r.start = len - r.n;
  return r;
}

// The last b with cu[b] <= t (0 <= t < total); cu[0] = 0.
__host__ __device__ __forceinline__ int find_seq(const Seqs& sq, int t, unsigned* err) {
  int lo = 0, hi = sq.B;                     // cu[lo] <= t, and (if in order) cu[hi] > t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ld_int(sq.cu, mid, sq.B + 1, err) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Sequence and position of token t; false if there is nothing to do for it.
__host__ __device__ __forceinline__ bool find_token(const Seqs& sq, int t, int* seq, int* pos,
                                                    unsigned* err) {
  const int b = sq.cu ? find_seq(sq, t, err) : t / sq.n_uniform;
  const NewTokens nt = new_tokens(sq, b, false, err);
  *seq = b;
  *pos = nt.start + (t - nt.first);
  return nt.n > 0 && t >= nt.first && t < nt.first + nt.n;
}

// The page of that number of sequence b, or -1 (noted) if it is none of the
// cache's.
__host__ __device__ __forceinline__ int find_page(const Seqs& sq, int b, int64_t page, bool report,
                                                  unsigned* err) {
  const int phys = ld_int(sq.block_table, (int64_t)b * sq.max_pages + page,
                          (int64_t)sq.B * sq.max_pages, err);
  if (phys >= 0 && phys < sq.num_pages) return phys;
  if (report) note_error(err, kDevErrInput);
  return -1;
}

// Notes sequences whose sizes do not fit (thread i of n; a few loads each).
__host__ __device__ __forceinline__ void check_seqs(const Seqs& sq, int i, int n, unsigned* err) {
  for (int b = i; b < sq.B; b += n) (void)new_tokens(sq, b, true, err);
  if (sq.cu && i == 0 &&
      (ld_int(sq.cu, 0, sq.B + 1, err) != 0 || ld_int(sq.cu, sq.B, sq.B + 1, err) != sq.total))
    note_error(err, kDevErrInput);
}

// Items.  Sequence b gets the item numbers [f(b), f(b + 1)), as many as its
// n tokens can touch pages at any offset.  Uniform n: pages_of(n) each.  With
// cu: f(b) = cu[b] / page_size + 2 b, since n tokens touch at most
// n / page_size + 2 pages and the floor of a sum is at least the sum of floors.
__host__ __device__ __forceinline__ int pages_of(int n, int page_size) {
  return (int)(((int64_t)n + page_size - 2) / page_size) + 1;
}
__host__ __device__ __forceinline__ int64_t num_items(int total, int B, int n_uniform, bool has_cu,
                                                      int page_size) {
  return has_cu ? (int64_t)total / page_size + 2 * (int64_t)B
                : (int64_t)B * pages_of(n_uniform, page_size);
}

// The page that item x stands for: new tokens [t0, t0 + n) at positions pos0
// onwards go to slots [off, off + n) of page phys.  n = 0: nothing to do.
struct Item {
  int t0, n, off, pos0, phys;
};
// Page p (0, 1, ..) of those that the new tokens of sequence b touch.
__host__ __device__ __forceinline__ Item item_of(const Seqs& sq, int b, int p, bool report,
                                                 unsigned* err) {
  Item it = {0, 0, 0, 0, 0};
  const NewTokens nt = new_tokens(sq, b, false, err);
  if (nt.n == 0) return it;
  const int64_t page = (int64_t)nt.start / sq.page_size + p;
  const int64_t lo_pos = page * sq.page_size;
  const int64_t end = (int64_t)nt.start + nt.n;
  const int64_t a = lo_pos > nt.start ? lo_pos : nt.start;
  const int64_t z = lo_pos + sq.page_size < end ? lo_pos + sq.page_size : end;
  if (a >= z) return it;
  const int phys = find_page(sq, b, page, report, err);
  if (phys < 0) return it;
  it.t0 = nt.first + (int)(a - nt.start);
  it.n = (int)(z - a);
  it.off = (int)(a - lo_pos);
  it.pos0 = (int)a;
  it.phys = phys;
  return it;
}

// Sequence b's items [lo, lo + n); none where lo < 0 or n <= 0 (tables out of order).
__host__ __device__ __forceinline__ void items_of(const Seqs& sq, int b, int64_t* lo, int64_t* n,
                                                  unsigned* err) {
  if (sq.cu) {
    const int c0 = ld_int(sq.cu, b, sq.B + 1, err), c1 = ld_int(sq.cu, b + 1, sq.B + 1, err);
    *lo = c0 / sq.page_size + 2 * (int64_t)b;
    *n = (int64_t)(c1 / sq.page_size) - c0 / sq.page_size + 2;
  } else {
    *n = pages_of(sq.n_uniform, sq.page_size);
    *lo = b * *n;
  }
}
// Whether item x is one of sequence b's, and which of its pages.
__host__ __device__ __forceinline__ bool item_is_of(const Seqs& sq, int x, int b, int* p,
                                                    unsigned* err) {
  int64_t lo, n;
  items_of(sq, b, &lo, &n, err);
  const int64_t q = x - lo;
  *p = (int)q;
  return q >= 0 && q < n && q <= x;
}

struct Cache {
  uint8_t* pages[2];      // K, V
  float* scale[2];        // E4M3 only
};

using bf16 = __nv_bfloat16;

// ------------------------------------------------------------- rows

// nh query heads of a token by a lane group of CTA `cta` of the query CTAs.
template <int D, int HB, bool kSplit>
__device__ __forceinline__ void query_rows(const Seqs& sq, const NormRope& nr,
                                           const RowsIn<bf16>& q, const RowsOut<bf16>& qo, int Hq,
                                           int nh, int cta, unsigned* err) {
  constexpr int LG = D / 8;
  const int li = threadIdx.x % LG, nblk = (Hq + nh - 1) / nh;
  const int64_t u = (int64_t)cta * (blockDim.x / LG) + threadIdx.x / LG;
  // a warp's groups: neighbouring tokens of one block of heads
  const int blk = (int)(u / sq.total), t = (int)(u - (int64_t)blk * sq.total), h0 = blk * nh;
  int b = 0, pos = 0;
  const bool active = blk < nblk && find_token(sq, t, &b, &pos, err);
  norm_rope_heads<bf16, D, HB, kSplit>(nr, static_cast<const bf16*>(nr.wq), q, qo, sq.total, Hq, t,
                                       h0, nh, pos, active, li, err);
}

// bf16 cache: nh kv heads of a token by a lane group, HB at a time.
template <int D, int HB, bool kSplit>
__global__ void __launch_bounds__(kThreads)
    append_rows_kernel(const Seqs sq, const NormRope nr, const RowsIn<bf16> k, const RowsIn<bf16> v,
                       const RowsIn<bf16> q, const RowsOut<bf16> qo, int Hq, int nh, int nhq,
                       const Cache cache, int kv_ctas, unsigned* err) {
  if ((int)blockIdx.x >= kv_ctas) {
    query_rows<D, HB, kSplit>(sq, nr, q, qo, Hq, nhq, (int)blockIdx.x - kv_ctas, err);
    return;
  }
  constexpr int LG = D / 8;
  const int li = threadIdx.x % LG, nblk = (sq.Hkv + nh - 1) / nh;
  const int64_t u = (int64_t)blockIdx.x * (kThreads / LG) + threadIdx.x / LG;
  const int blk = (int)(u / sq.total), t = (int)(u - (int64_t)blk * sq.total), h0 = blk * nh;
  int b = 0, pos = 0, phys = -1;
  const bool known = blk < nblk && find_token(sq, t, &b, &pos, err);
  if (known) phys = find_page(sq, b, pos / sq.page_size, li == 0, err);
  const bool active = phys >= 0;
  const int64_t n_k = (int64_t)(sq.total - 1) * k.ld + (int64_t)sq.Hkv * D;
  const int64_t n_v = (int64_t)(sq.total - 1) * v.ld + (int64_t)sq.Hkv * D;
  const int64_t n_pages = (int64_t)sq.num_pages * sq.Hkv * sq.page_size * D;
  const int64_t src_k = (int64_t)t * k.ld + 8 * li, src_v = (int64_t)t * v.ld + 8 * li;
  const int64_t head = (int64_t)sq.page_size * D;              // elements of a page's head
  const int64_t dst = (int64_t)phys * sq.Hkv * head + pos % sq.page_size * D + 8 * li;
  const int h1 = active ? min(h0 + nh, sq.Hkv) : h0;
  Raw8<bf16> kx[HB], vx[HB];
  auto load = [&](int h) {
#pragma unroll
    for (int j = 0; j < HB; ++j) {
      kx[j] = {};
      vx[j] = {};
      if (h + j < h1) {
        kx[j] = load8<bf16>(k.p, src_k + (int64_t)(h + j) * D, n_k, err);
        vx[j] = load8<bf16>(v.p, src_v + (int64_t)(h + j) * D, n_v, err);
      }
    }
  };
  load(h0);
  const bf16* wk = static_cast<const bf16*>(nr.wk);
  const Coef cf = load_coef<bf16, D, kSplit>(nr, wk, pos, li, active, err);
  const int batches = (int)__reduce_max_sync(0xffffffffu, (unsigned)(h1 - h0 + HB - 1) / HB);
  for (int i = 0; i < batches; ++i) {
    const int h = h0 + i * HB;
    Raw8<bf16> kc[HB], vc[HB];
#pragma unroll
    for (int j = 0; j < HB; ++j) {
      kc[j] = kx[j];
      vc[j] = vx[j];
    }
    if (i + 1 < batches) load(h + HB);
#pragma unroll
    for (int j = 0; j < HB; ++j) {
      const Row8 y = norm_rope_row<bf16, D, kSplit>(nr, kc[j], wk != nullptr, cf, li);
      const int64_t at = dst + (h + j) * head;
      if (h + j < h1) {
        store8(reinterpret_cast<bf16*>(cache.pages[0]), at, y, n_pages, err);
        if (RF_IN(err, at + 7, n_pages))
          *reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(cache.pages[1]) + at) =
              make_uint4(vc[j].w[0], vc[j].w[1], vc[j].w[2], vc[j].w[3]);
      }
    }
  }
  if (blockIdx.x == 0) check_seqs(sq, (int)threadIdx.x, kThreads, err);
}

// ------------------------------------------------------------- a few tokens a sequence

constexpr int kStepTokens = 8;

template <int D, int TOK, bool kSplit>
__global__ void __launch_bounds__(kThreads)
    append_step_kernel(const Seqs sq, const NormRope nr, const RowsIn<bf16> k, const RowsIn<bf16> v,
                       const RowsIn<bf16> q, const RowsOut<bf16> qo, int Hq, const Cache cache,
                       int kv_ctas, unsigned* err) {
  if ((int)blockIdx.x >= kv_ctas) {
    query_rows<D, 1, kSplit>(sq, nr, q, qo, Hq, 1, (int)blockIdx.x - kv_ctas, err);
    return;
  }
  constexpr int LG = D / 8;                   // lanes of a row
  constexpr int kPairs = 32 / (2 * LG);       // (item, head) pairs of a warp
  const int lane = threadIdx.x & 31, li = lane % LG, grp = lane / LG;
  const bool is_v = grp & 1;
  const int64_t u =
      ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kPairs + (grp >> 1);
  const int pages_each = pages_of(sq.n_uniform, sq.page_size);
  const int x = (int)(u / sq.Hkv), h = (int)(u % sq.Hkv);
  const int b = TOK == 1 ? x : x / pages_each;
  Item it = {0, 0, 0, 0, 0};
  if (b < sq.B) it = item_of(sq, b, x - b * pages_each, h == 0 && !is_v && li == 0, err);

  const RowsIn<bf16>& in = is_v ? v : k;
  const int64_t n_in = (int64_t)(sq.total - 1) * in.ld + (int64_t)sq.Hkv * D;
  Raw8<bf16> raw[TOK];
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    raw[i] = {};
    if (i < it.n)
      raw[i] = load8<bf16>(in.p, (int64_t)(it.t0 + i) * in.ld + (int64_t)h * D + 8 * li, n_in, err);
  }
  const int64_t head = (int64_t)it.phys * sq.Hkv + h;         // (page, head)
  float* sc = is_v ? cache.scale[1] : cache.scale[0];
  const int64_t n_sc = (int64_t)sq.num_pages * sq.Hkv;
  const float s_old = it.n > 0 && it.off > 0 && RF_IN(err, head, n_sc) ? sc[head] : 0.f;
  const bf16* wk = static_cast<const bf16*>(nr.wk);
  const CoefSource<bf16, D, kSplit> source(nr, wk, li, err);
  Row8 y[TOK];
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    const Coef cf = source.get(nr, it.pos0 + i, li, i < it.n && !is_v, err);
    y[i] = norm_rope_row<bf16, D, kSplit>(nr, raw[i], wk != nullptr, cf, li);
    if (is_v) y[i] = as_row(raw[i]);
    if (i < it.n) a = fmaxf(a, absmax8(y[i]));
  }
  constexpr unsigned kGroup = (1u << LG) - 1u;
  a = group_max(kGroup << (grp * LG), a);
  const float s = new_scale(a, s_old, it.off);
  const bool grow = it.n > 0 && it.off > 0 && s > s_old;
  const unsigned growing = __ballot_sync(0xffffffffu, grow && li == 0);   // after everyone's load

  const int64_t n_pages = (int64_t)sq.num_pages * sq.Hkv * sq.page_size * D;
  uint8_t* pages = is_v ? cache.pages[1] : cache.pages[0];
  const float inv = 1.f / s;                                  // exact: a power of two
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    const int64_t row = (head * sq.page_size + it.off + i) * D + 8 * li;
    if (i < it.n && RF_IN(err, row + 7, n_pages))
      *reinterpret_cast<uint2*>(pages + row) = quantise8(y[i], inv);
  }
  if (it.n > 0 && li == 0 && RF_IN(err, head, n_sc)) sc[head] = s;
  // pages whose scale grew: the warp rescales the off * D codes held already
  for (unsigned m = growing; m; m &= m - 1) {
    const int src = __ffs(m) - 1;
    const int64_t at = __shfl_sync(0xffffffffu, head, src) * sq.page_size * D;
    const int n16 = __shfl_sync(0xffffffffu, it.off, src) * D / 16;
    const float ratio = __shfl_sync(0xffffffffu, s_old / s, src);
    uint8_t* pg = ((src / LG) & 1 ? cache.pages[1] : cache.pages[0]) + at;
    for (int i0 = 0; i0 < n16; i0 += 32 * 8) {
      uint4 c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + 32 * j + lane;
        if (i < n16 && RF_IN(err, at + 16 * i + 15, n_pages))
          c[j] = reinterpret_cast<const uint4*>(pg)[i];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + 32 * j + lane;
        if (i < n16 && RF_IN(err, at + 16 * i + 15, n_pages))
          reinterpret_cast<uint4*>(pg)[i] = rescale16(c[j], ratio);
      }
    }
  }
  if (blockIdx.x == 0) check_seqs(sq, (int)threadIdx.x, kThreads, err);
}

// ------------------------------------------------------------- prompts

// The units (item, head), items outermost, are shared out evenly over the kv
// CTAs, as many as run at once.  A CTA's threads cover the page's rows in SW
// sweeps, keys and values together.  An item is looked up once, and its tokens'
// A and B are made once and kept in shared memory, a place of its own for each
// thread (page_size * D * 8 bytes).  TH, the most threads, is 512 with 64
// registers, so that two CTAs share an SM: one works while the other waits.
// Pages of 128 x 128 take 1024 threads, since four sweeps of 512 spill (45
// against 24 us for 8192 tokens of 8 heads); two sweeps spill 32 or 36 bytes.
// The next head's keys are fetched
// as soon as the present ones are in their final form, its values when the
// present ones are stored.
template <int D, int SW, int TH, bool kSplit>
__global__ void __launch_bounds__(TH, 1024 / TH)
    append_prompt_kernel(const Seqs sq, const NormRope nr, const RowsIn<bf16> k,
                         const RowsIn<bf16> v, const RowsIn<bf16> q, const RowsOut<bf16> qo, int Hq,
                         int nhq, const Cache cache, int units, int kv_ctas, unsigned* err) {
  if ((int)blockIdx.x >= kv_ctas) {
    query_rows<D, 2, kSplit>(sq, nr, q, qo, Hq, nhq, (int)blockIdx.x - kv_ctas, err);
    return;
  }
  constexpr int LG = D / 8;
  extern __shared__ uint4 coefs[];                   // [SW][4][threads]
  const int rows = (int)blockDim.x / LG;             // of a sweep
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int li = threadIdx.x % LG, r = threadIdx.x / LG;
  const int u0 = (int)((int64_t)blockIdx.x * units / kv_ctas);
  const int u1 = (int)((int64_t)(blockIdx.x + 1) * units / kv_ctas);
  const int64_t n_k = (int64_t)(sq.total - 1) * k.ld + (int64_t)sq.Hkv * D;
  const int64_t n_v = (int64_t)(sq.total - 1) * v.ld + (int64_t)sq.Hkv * D;
  const int64_t n_pages = (int64_t)sq.num_pages * sq.Hkv * sq.page_size * D;
  const int64_t n_sc = (int64_t)sq.num_pages * sq.Hkv;
  const bool has_w = nr.wk != nullptr;
  __shared__ Item found[2];                          // of two items in turn
  __shared__ int owner[2];
  __shared__ float red[2][2][TH / 32];               // of two heads in turn: one barrier a head
  if (blockIdx.x == 0) check_seqs(sq, (int)threadIdx.x, (int)blockDim.x, err);

  int x = u0 / sq.Hkv, h = u0 - x * sq.Hkv, turn = 0, now = 0;
  if (threadIdx.x == 0) found[0].n = 0, owner[0] = sq.B;
  __syncthreads();
  for (int u = u0; u < u1; ++x, h = 0, now ^= 1) {   // items
    const int h_end = min(sq.Hkv, h + (u1 - u));
    u += h_end - h;
    // the sequences are looked through in parallel, and one thread finds the item.
    // With cu_seqlens out of order several may: the lowest sequence has it, in
    // every CTA that takes heads of it (words from two would make an item of no
    // sequence's, out of all bounds)
    Item mine = {0, 0, 0, 0, 0};
    int mine_of = sq.B;
    for (int b = threadIdx.x; b < sq.B && mine.n == 0; b += blockDim.x) {
      int pg;
      if (item_is_of(sq, x, b, &pg, err)) {
        mine = item_of(sq, b, pg, h == 0, err);
        mine_of = b;
      }
    }
    if (mine.n > 0) atomicMin(&owner[now], mine_of);
    __syncthreads();
    if (mine.n > 0 && owner[now] == mine_of) found[now] = mine;
    if (threadIdx.x == 0) found[now ^ 1].n = 0, owner[now ^ 1] = sq.B;   // read before the barrier
    __syncthreads();
    const Item it = found[now];
    if (it.n == 0) continue;

    int64_t at_k = (int64_t)(it.t0 + r) * k.ld + (int64_t)h * D + 8 * li;
    int64_t at_v = (int64_t)(it.t0 + r) * v.ld + (int64_t)h * D + 8 * li;
    Raw8<bf16> kx[SW], vx[SW];                       // rows beyond the item's are zeros
    auto load = [&](Raw8<bf16>(&to)[SW], const RowsIn<bf16>& in, int64_t& at, int64_t n) {
#pragma unroll
      for (int i = 0; i < SW; ++i) {
        to[i] = {};
        if (r + i * rows < it.n) to[i] = load8<bf16>(in.p, at + i * rows * in.ld, n, err);
      }
      at += D;
    };
    load(kx, k, at_k, n_k);
    load(vx, v, at_v, n_v);
    {
      const CoefSource<bf16, D, kSplit> source(nr, static_cast<const bf16*>(nr.wk), li, err);
#pragma unroll
      for (int i = 0; i < SW; ++i) {
        const int t = r + i * rows;
        const Coef cf = source.get(nr, it.pos0 + t, li, t < it.n, err);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          ulonglong2* at =
              reinterpret_cast<ulonglong2*>(coefs + (4 * i + j) * blockDim.x + threadIdx.x);
          at[0] = make_ulonglong2(cf.a[2 * j], cf.a[2 * j + 1]);
          at[2 * blockDim.x] = make_ulonglong2(cf.b[2 * j], cf.b[2 * j + 1]);
        }
      }
    }
    int64_t head = (int64_t)it.phys * sq.Hkv + h;
    for (; h < h_end; ++h, ++head, turn ^= 1) {
      float s_old[2] = {0.f, 0.f};
      if (it.off > 0 && RF_IN(err, head, n_sc)) {
        s_old[0] = cache.scale[0][head];
        s_old[1] = cache.scale[1][head];
      }
      Row8 ky[SW];
      float a[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < SW; ++i) {
        Coef cf;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const ulonglong2* at =
              reinterpret_cast<const ulonglong2*>(coefs + (4 * i + j) * blockDim.x + threadIdx.x);
          const ulonglong2 ca = at[0], cb = at[2 * blockDim.x];
          cf.a[2 * j] = ca.x;
          cf.a[2 * j + 1] = ca.y;
          cf.b[2 * j] = cb.x;
          cf.b[2 * j + 1] = cb.y;
        }
        ky[i] = norm_rope_row<bf16, D, kSplit>(nr, kx[i], has_w, cf, li);
        if (r + i * rows < it.n) a[0] = fmaxf(a[0], absmax8(ky[i]));
      }
      if (h + 1 < h_end) load(kx, k, at_k, n_k);
#pragma unroll
      for (int i = 0; i < SW; ++i) a[1] = fmaxf(a[1], absmax8(vx[i]));
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        a[w] = group_max(0xffffffffu, a[w]);
        if (lane == 0) red[turn][w][warp] = a[w];
      }
      __syncthreads();                   // after it, too: everyone has read the old scales
      const int64_t base = head * sq.page_size * D;
      float inv[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const float m =
            group_max(0xffffffffu, lane < (int)blockDim.x / 32 ? red[turn][w][lane] : 0.f);
        const float s = new_scale(m, s_old[w], it.off);
        inv[w] = 1.f / s;
        if (threadIdx.x == 0 && RF_IN(err, head, n_sc)) cache.scale[w][head] = s;
        if (it.off > 0 && s > s_old[w]) {
          const float ratio = s_old[w] / s;
          uint4* pg = reinterpret_cast<uint4*>(cache.pages[w] + base);
          for (int i = threadIdx.x; i < it.off * D / 16; i += blockDim.x)
            if (RF_IN(err, base + 16 * i + 15, n_pages)) pg[i] = rescale16(pg[i], ratio);
        }
      }
      const int64_t at0 = base + (int64_t)(it.off + r) * D + 8 * li;
#pragma unroll
      for (int i = 0; i < SW; ++i) {
        const int64_t at = at0 + i * rows * D;
        if (r + i * rows < it.n && RF_IN(err, at + 7, n_pages)) {
          *reinterpret_cast<uint2*>(cache.pages[0] + at) = quantise8(ky[i], inv[0]);
          *reinterpret_cast<uint2*>(cache.pages[1] + at) = quantise8(as_row(vx[i]), inv[1]);
        }
      }
      if (h + 1 < h_end) load(vx, v, at_v, n_v);
    }
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int D, bool kSplit>
cudaError_t launch(const Seqs& sq, const NormRope& nr, const RowsIn<bf16>& k,
                   const RowsIn<bf16>& v, const RowsIn<bf16>& q, const RowsOut<bf16>& qo, int Hq,
                   const Cache& cache, bool f8, int sms, unsigned* err, cudaStream_t s) {
  constexpr int LG = D / 8, per = kThreads / LG;      // lane groups of a CTA
  if (!f8) {
    // keys and values count twice, since a row of both is worked on together
    const int nh = heads_per_group((int64_t)sq.total * sq.Hkv * 2, sq.Hkv, D, sms);
    const int nhq = nh == 1 ? 1 : std::max(4, heads_per_group((int64_t)sq.total * Hq, Hq, D, sms));
    const int64_t kv = ceil_div((int64_t)sq.total * ceil_div(sq.Hkv, nh), per);
    const int64_t q_ctas = ceil_div((int64_t)sq.total * ceil_div(Hq, nhq), per);
    const unsigned grid = (unsigned)(kv + q_ctas);
    // batches of two heads of 64 (19.5 against 21.5 us with four for 6.6k tokens of
    // 16 heads) and of four of 128 (15.7 against 16.9 with two for 8192 of 8)
    if (nh > 1)
      append_rows_kernel<D, D / 32, kSplit><<<grid, kThreads, 0, s>>>(sq, nr, k, v, q, qo, Hq, nh, nhq,
                                                                 cache, (int)kv, err);
    else
      append_rows_kernel<D, 1, kSplit><<<grid, kThreads, 0, s>>>(sq, nr, k, v, q, qo, Hq, nh, nhq,
                                                                 cache, (int)kv, err);
    return cudaGetLastError();
  }
  if (!sq.cu && sq.n_uniform <= kStepTokens) {
    // 32 sequences of 4 tokens and 8 heads: 8.9 us in the prompt kernel
    const int64_t items = num_items(sq.total, sq.B, sq.n_uniform, false, sq.page_size);
    const int64_t kv = ceil_div(items * sq.Hkv, kThreads / (2 * LG));
    const int64_t q_ctas = ceil_div((int64_t)sq.total * Hq, per);
    const unsigned grid = (unsigned)(kv + q_ctas);
    if (sq.n_uniform == 1)
      append_step_kernel<D, 1, kSplit><<<grid, kThreads, 0, s>>>(sq, nr, k, v, q, qo, Hq, cache,
                                                                 (int)kv, err);
    else
      append_step_kernel<D, kStepTokens, kSplit><<<grid, kThreads, 0, s>>>(sq, nr, k, v, q, qo, Hq,
                                                                           cache, (int)kv, err);
    return cudaGetLastError();
  }
  const int pieces = sq.page_size * D / 8;
  const int threads = pieces <= 512 ? pieces : (pieces <= 1024 ? 512 : 1024);
  const int64_t items = num_items(sq.total, sq.B, sq.n_uniform, sq.cu != nullptr, sq.page_size);
  const int nhq = std::max(4, heads_per_group((int64_t)sq.total * Hq, Hq, D, sms));
  const int64_t units = items * sq.Hkv;
  const int64_t kv = std::min(units, (int64_t)sms * 1024 / threads);
  const int64_t q_ctas = ceil_div((int64_t)sq.total * ceil_div(Hq, nhq), threads / LG);
  const unsigned grid = (unsigned)(kv + q_ctas);
  const int smem = pieces * 64;
#define RF_GO(SW, TH)                                                                              \
  do {                                                                                             \
    auto kern = append_prompt_kernel<D, SW, TH, kSplit>;                                           \
    const cudaError_t e =                                                                          \
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);             \
    if (e != cudaSuccess) return e;                                                                \
    kern<<<grid, threads, smem, s>>>(sq, nr, k, v, q, qo, Hq, nhq, cache, (int)units, (int)kv,     \
                                   err);                                                           \
  } while (0)
  if (pieces <= 512) RF_GO(1, 512);
  else if (pieces <= 1024) RF_GO(2, 512);
  else RF_GO(2, (D == 128 ? 1024 : 512));          // 128 x 128
#undef RF_GO
  return cudaGetLastError();
}

Seqs make_seqs(const PagedKV& c, const int* cu, int total, int max_pos) {
  Seqs sq;
  sq.block_table = c.block_table;
  sq.seq_lens = c.seq_lens;
  sq.cu = cu;
  sq.B = c.B;
  sq.n_uniform = cu ? 0 : total / c.B;
  sq.total = total;
  sq.num_pages = c.num_pages;
  sq.page_size = c.page_size;
  sq.max_pages = c.max_pages;
  sq.Hkv = c.Hkv;
  sq.max_len = c.max_pages * c.page_size;             // at most 2^30
  if (max_pos > 0 && max_pos < sq.max_len) sq.max_len = max_pos;
  return sq;
}

}  // namespace

int64_t append_grid_bound(int total, int B, bool has_cu, int page_size, int Hkv, int Hq) {
  return num_items(total, B, has_cu ? 0 : total / B, has_cu, page_size) * Hkv +
         (int64_t)total * ((int64_t)Hkv + Hq);
}

cudaError_t launch_kv_append_paged(const PagedKV& c, const NormRope& nr, const void* K,
                                   int64_t ldk, const void* V, int64_t ldv, const int* cu,
                                   int total, const void* Q, int64_t ldq, void* Qo, int64_t ldqo,
                                   int Hq, unsigned* err, cudaStream_t s) {
  const Seqs sq = make_seqs(c, cu, total, nr.rot > 0 ? nr.max_pos : 0);
  Cache cache = {{static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v)}, {c.k_scale, c.v_scale}};
  const RowsIn<bf16> k = {static_cast<const bf16*>(K), ldk}, v = {static_cast<const bf16*>(V), ldv},
                     q = {static_cast<const bf16*>(Q), ldq};
  const RowsOut<bf16> qo = {static_cast<bf16*>(Qo), ldqo};
  const bool f8 = c.dtype == RF_E4M3;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidValue;
  const bool split = is_split(nr);
  if (c.d == 64)
    return split ? launch<64, true>(sq, nr, k, v, q, qo, Hq, cache, f8, sms, err, s)
                 : launch<64, false>(sq, nr, k, v, q, qo, Hq, cache, f8, sms, err, s);
  return split ? launch<128, true>(sq, nr, k, v, q, qo, Hq, cache, f8, sms, err, s)
               : launch<128, false>(sq, nr, k, v, q, qo, Hq, cache, f8, sms, err, s);
}

// Host-side walk of the items (the functions above, shared by host and
// device).  All arrays are host arrays.  Returns 0 when every invariant
// holds, else the number of the first that fails:
//   1 no index leaves its array;
//   2 an item is of one sequence, its page and slots in the cache and in one page;
//   3 every token of a sequence that is not skipped is written once, to the
//     slot of its position, and no other token is;
//   4 the rows' lookup finds the same position and page for the same tokens;
//   5 inconsistent sizes, and only those, are noted.
// -1 where tables out of order would make the walk too long.
constexpr int64_t kMostWalked = 1ll << 28;
int append_plan_selfcheck(const PagedKV& c, const int* cu, int total, int max_pos) {
  const Seqs sq = make_seqs(c, cu, total, max_pos);
  unsigned err = 0;
  // tables out of order name tokens twice or not at all: only the bounds
  // hold then
  bool order = true;
  if (cu) {
    order = cu[0] == 0 && cu[c.B] == total;
    for (int b = 0; b < c.B; ++b) order = order && cu[b] <= cu[b + 1];
  }
  std::vector<int> pos_of((size_t)total, -1);
  const int64_t n = num_items(total, c.B, sq.n_uniform, cu != nullptr, c.page_size);
  // each sequence's items (in order, all of them together are n; out of order they
  // may be any number of times that, and are walked as long as that takes seconds)
  std::vector<unsigned char> taken((size_t)n, 0);
  int64_t walked = 0;
  for (int b = 0; b < c.B; ++b) {
    int64_t lo, count;
    items_of(sq, b, &lo, &count, &err);
    if (err & kDevErrBounds) return 1;
    if (lo < 0) continue;
    const int64_t end = std::min(n, lo + count);
    walked += std::max<int64_t>(end - lo, 0);
    if (walked > kMostWalked) return -1;
    for (int64_t x = lo; x < end; ++x) {
      int p;
      if (!item_is_of(sq, (int)x, b, &p, &err)) return 2;
      const Item it = item_of(sq, b, p, true, &err);
      if (err & kDevErrBounds) return 1;
      if (it.n == 0) continue;
      if (order && taken[(size_t)x]++) return 2;
      if (it.n < 0 || it.off < 0 || it.off + it.n > c.page_size || it.phys < 0 ||
          it.phys >= c.num_pages || it.t0 < 0 || it.t0 + it.n > total)
        return 2;
      for (int i = 0; i < it.n; ++i) {
        if (order &&
            (pos_of[(size_t)it.t0 + i] != -1 || (it.pos0 + i) % c.page_size != it.off + i))
          return 3;
        pos_of[(size_t)it.t0 + i] = it.pos0 + i;
      }
    }
  }
  bool bad = false;
  std::vector<int> want((size_t)total, -1), seen((size_t)total, -1);
  for (int b = 0; b < c.B; ++b) {
    const int64_t c0 = cu ? cu[b] : (int64_t)b * sq.n_uniform;
    const int64_t c1 = cu ? cu[b + 1] : c0 + sq.n_uniform;
    if (!order) break;
    const int64_t len = c.seq_lens[b];
    if (len == 0 || c1 == c0) continue;
    if (len < c1 - c0 || len > sq.max_len) {
      bad = true;
      continue;
    }
    for (int64_t t = c0; t < c1; ++t) {
      const int64_t pos = len - (c1 - c0) + (t - c0);
      const int page = c.block_table[(int64_t)b * c.max_pages + pos / c.page_size];
      seen[(size_t)t] = (int)pos;
      if (page < 0 || page >= c.num_pages) bad = true;
      else want[(size_t)t] = (int)pos;
    }
  }
  if (order && pos_of != want) return 3;
  for (int t = 0; t < total; ++t) {
    int b = 0, pos = 0;
    const bool active = find_token(sq, t, &b, &pos, &err);
    const int phys = active ? find_page(sq, b, pos / c.page_size, true, &err) : -1;
    if (err & kDevErrBounds) return 1;
    if (order && ((active ? pos : -1) != seen[(size_t)t] ||
                  (phys >= 0 ? pos : -1) != want[(size_t)t]))
      return 4;
  }
  check_seqs(sq, 0, 1, &err);
  if (err & kDevErrBounds) return 1;
  if (!order && !(err & kDevErrInput)) return 5;
  if (order && bad != ((err & kDevErrInput) != 0)) return 5;
  return 0;
}

}  // namespace rf

// norm_rope.cuh -- the norm and rotation of one head's row, shared by
// qk_norm_rope.cu and kv_append_paged.cu.
//
// A row of D elements is held by a group of D / 8 neighbouring lanes, eight
// consecutive elements a lane (one 16-byte load in bf16).  With x the row,
//     y_i = x_i * rstd * w_i,   rstd = rsqrt(mean(x^2) + eps)   (where there is a weight)
// and, for the first rot elements, a rotation of pairs by the token's angles:
//     (a, b) -> (a cos - b sin, b cos + a sin),
// the pair j being elements (j, j + rot / 2) (half-split) or (2j, 2j + 1)
// (interleaved).  Both forms, and unrotated elements, are one formula,
//     out_i = (x_i rstd) A_i + (x_partner(i) rstd) B_i,
//     A_i = w_i cos,   B_i = -+ w_partner(i) sin   (a: -, b: +),
// with the partner in the lane rot / 16 away or in the same lane.  A and B
// depend on the token and on queries or keys only, so a lane group makes them
// once for all heads it takes; a head then costs two packed multiply-adds for
// two elements.  Everything is fp32; the caller rounds once.  rot % 16 == 0, so
// a lane's eight elements are all rotated or none, and all in the same half.
#pragma once

#include "rf_device.cuh"
#include "rf_internal.h"

namespace rf {

// Eight consecutive elements as loaded.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  static constexpr int kWords = 4;
  uint32_t w[4];
  __device__ __forceinline__ float get(int e) const {
    return (e & 1) ? bf16hi(w[e >> 1]) : bf16lo(w[e >> 1]);
  }
  // elements 2 i and 2 i + 1 as packed fp32
  __device__ __forceinline__ uint64_t pair(int i) const { return f2(bf16lo(w[i]), bf16hi(w[i])); }
  __device__ __forceinline__ uint64_t swapped(int i) const {
    return f2(bf16hi(w[i]), bf16lo(w[i]));
  }
};
template <>
struct Raw8<float> {
  static constexpr int kWords = 8;
  uint32_t w[8];
  __device__ __forceinline__ float get(int e) const { return __uint_as_float(w[e]); }
  __device__ __forceinline__ uint64_t pair(int i) const { return f2(get(2 * i), get(2 * i + 1)); }
  __device__ __forceinline__ uint64_t swapped(int i) const {
    return f2(get(2 * i + 1), get(2 * i));
  }
};

// Loads elements [i, i + 8) of a tensor of n elements (zeros outside it, in
// the bounds-checked build).
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p, int64_t i, int64_t n, unsigned* err) {
  Raw8<T> r;
  if (RF_IN(err, i + 7, n) && RF_IN(err, i, n)) {
    const uint4* q = reinterpret_cast<const uint4*>(p + i);
#pragma unroll
    for (int k = 0; k < Raw8<T>::kWords / 4; ++k) {
      const uint4 v = q[k];
      r.w[4 * k] = v.x;
      r.w[4 * k + 1] = v.y;
      r.w[4 * k + 2] = v.z;
      r.w[4 * k + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < Raw8<T>::kWords; ++k) r.w[k] = 0u;
  }
  return r;
}

// Eight results, in packed fp32 pairs.
struct Row8 {
  uint64_t v[4];
};

__device__ __forceinline__ void store8(__nv_bfloat16* p, int64_t i, const Row8& y, int64_t n,
                                       unsigned* err) {
  if (!RF_IN(err, i + 7, n) || !RF_IN(err, i, n)) return;
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float lo, hi;
    f2_split(y.v[k], lo, hi);
    w[k] = pack_bf16x2(lo, hi);
  }
  *reinterpret_cast<uint4*>(p + i) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, int64_t i, const Row8& y, int64_t n,
                                       unsigned* err) {
  if (!RF_IN(err, i + 7, n) || !RF_IN(err, i, n)) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float4 f;
    f2_split(y.v[2 * k], f.x, f.y);
    f2_split(y.v[2 * k + 1], f.z, f.w);
    reinterpret_cast<float4*>(p + i)[k] = f;
  }
}

// A and B of a lane's eight elements, in packed pairs.
struct Coef {
  uint64_t a[4], b[4];
};

// Lane of the group that holds the half-split partners of lane li's elements.
__device__ __forceinline__ int partner_lane(const NormRope& nr, int li) {
  const int h = nr.rot >> 4;                       // lanes per half
  return li < h ? li + h : li - h;
}

// kSplit: half-split rotation (partners in another lane); else interleaved, or
// no rotation at all.
__host__ __forceinline__ bool is_split(const NormRope& nr) { return nr.rot > 0 && !nr.interleaved; }

// Where a lane's coefficients come from: the weights of queries or of keys (or
// null), held as loaded, and the tables.
template <typename T, int D, bool kSplit>
struct CoefSource {
  Raw8<T> own, other;
  bool has_w;
  __device__ __forceinline__ CoefSource(const NormRope& nr, const T* weight, int li, unsigned* err)
      : own{}, other{}, has_w(weight != nullptr) {
    if (!weight) return;
    own = load8<T>(weight, 8 * li, D, err);
    other = own;
    if (kSplit && 8 * li < nr.rot) other = load8<T>(weight, 8 * partner_lane(nr, li), D, err);
  }
  // active = false: nothing is loaded from the tables.
  __device__ __forceinline__ Coef get(const NormRope& nr, int pos, int li, bool active,
                                      unsigned* err) const {
    const int half = nr.rot >> 1;
    const int64_t n = (int64_t)nr.max_pos * half;
    const bool second = kSplit && 8 * li >= half;
    float4 c[2], s[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {                  // unrotated: cos = 1, sin = 0
      c[k] = make_float4(1.f, 1.f, 1.f, 1.f);
      s[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (8 * li < nr.rot && active) {
      const int64_t at = (int64_t)pos * half + (kSplit ? 8 * li - (second ? half : 0) : 4 * li);
#pragma unroll
      for (int k = 0; k < (kSplit ? 2 : 1); ++k)
        if (RF_IN(err, at + 4 * k + 3, n)) {
          c[k] = __ldg(reinterpret_cast<const float4*>(nr.cos + at) + k);
          s[k] = __ldg(reinterpret_cast<const float4*>(nr.sin + at) + k);
        }
    }
    const float cc[8] = {c[0].x, c[0].y, c[0].z, c[0].w, c[1].x, c[1].y, c[1].z, c[1].w};
    const float ss[8] = {s[0].x, s[0].y, s[0].z, s[0].w, s[1].x, s[1].y, s[1].z, s[1].w};
    const float sign = second ? 1.f : -1.f;
    const uint64_t sign2 = f2(sign, sign);
    Coef r;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      r.a[k] = kSplit ? f2(cc[2 * k], cc[2 * k + 1]) : f2(cc[k], cc[k]);
      r.b[k] = kSplit ? fmul2(f2(ss[2 * k], ss[2 * k + 1]), sign2) : f2(-ss[k], ss[k]);
      if (has_w) {
        r.a[k] = fmul2(r.a[k], own.pair(k));
        r.b[k] = fmul2(r.b[k], kSplit ? other.pair(k) : own.swapped(k));
      }
      // unrotated: the partner's term is +0 * -0 = -0, which changes neither zero's
      // sign (and is not made from weights, one of which may be infinite)
      if (8 * li >= nr.rot) r.b[k] = f2(-0.f, -0.f);
    }
    return r;
  }
};

template <typename T, int D, bool kSplit>
__device__ __forceinline__ Coef load_coef(const NormRope& nr, const T* weight, int pos, int li,
                                          bool active, unsigned* err) {
  return CoefSource<T, D, kSplit>(nr, weight, li, err).get(nr, pos, li, active, err);
}

// Norm (has_w) and rotation of a group's row.  Called by all 32 lanes of a
// warp together; has_w may differ between the warp's groups.
template <typename T, int D, bool kSplit>
__device__ __forceinline__ Row8 norm_rope_row(const NormRope& nr, const Raw8<T>& x, bool has_w,
                                              const Coef& cf, int li) {
  constexpr int LG = D / 8;
  float rstd = 1.f;
  if (nr.wq || nr.wk) {                 // the same for every lane: the shuffles need all of them
    uint64_t sq = fmul2(x.pair(0), x.pair(0));
#pragma unroll
    for (int k = 1; k < 4; ++k) sq = ffma2(x.pair(k), x.pair(k), sq);
    float lo, hi;
    f2_split(sq, lo, hi);
    float ss = lo + hi;
#pragma unroll
    for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (has_w) rstd = rsqrtf(fmaf(ss, 1.f / D, nr.eps));
  }
  // partners; +0 where nothing is rotated, since their B is -0 and x may be an
  // infinity
  const bool rotated = 8 * li < nr.rot;
  const int src = kSplit && rotated ? partner_lane(nr, li) : li;
  Raw8<T> p;
#pragma unroll
  for (int k = 0; k < Raw8<T>::kWords; ++k) {
    const uint32_t v = kSplit ? __shfl_sync(0xffffffffu, x.w[k], src, LG) : x.w[k];
    p.w[k] = rotated ? v : 0u;
  }
  const uint64_t r2 = f2(rstd, rstd);
  Row8 y;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint64_t t = fmul2(fmul2(x.pair(k), r2), cf.a[k]);
    y.v[k] = ffma2(fmul2(kSplit ? p.pair(k) : p.swapped(k), r2), cf.b[k], t);
  }
  return y;
}

// Tensors of rows [T][H][D] whose tokens are ld elements apart.
template <typename T>
struct RowsIn {
  const T* p;
  int64_t ld;
};
template <typename T>
struct RowsOut {
  T* p;
  int64_t ld;
};

// How many heads a lane group takes one after the other: as many of 4, 8, 16
// ... as leave 1024 threads for each SM (more heads share a token's A and B, but a
// device must be full), one where even four would not.  By their registers 768
// threads of the bf16 kernels run on an SM at once, and 512 of the fp32 ones and of
// the bf16 append's for heads of 128, so that a grid has 1.3 to 2.7 waves, or 2 to
// 4, or more; the last is a part of one.  `rows`: tokens x heads.
inline int heads_per_group(int64_t rows, int heads, int d, int sms) {
  const int64_t threads = rows * (d / 8);
  int h = 1;
  for (int k = 4; k < 2 * heads && threads / k >= 1024 * (int64_t)sms; k *= 2) h = k;
  return h;
}

// Heads [h0, min(h0 + nh, H)) of token t at position pos, by one lane group, in
// batches of HB: a batch's loads go together, and the next batch's before the
// present one is worked on.  nh: the same for the whole launch, HB divides it.
template <typename T, int D, int HB, bool kSplit>
__device__ __forceinline__ void norm_rope_heads(const NormRope& nr, const T* weight,
                                                const RowsIn<T>& in, const RowsOut<T>& out, int T_,
                                                int H, int t, int h0, int nh, int pos, bool active,
                                                int li, unsigned* err) {
  const int64_t n_in = (int64_t)(T_ - 1) * in.ld + (int64_t)H * D;
  const int64_t n_out = (int64_t)(T_ - 1) * out.ld + (int64_t)H * D;
  const int64_t src = (int64_t)t * in.ld + 8 * li, dst = (int64_t)t * out.ld + 8 * li;
  const int h1 = active ? min(h0 + nh, H) : h0;
  Raw8<T> x[HB];
  auto load = [&](int h) {
#pragma unroll
    for (int j = 0; j < HB; ++j) {
      x[j] = {};
      if (h + j < h1) x[j] = load8<T>(in.p, src + (int64_t)(h + j) * D, n_in, err);
    }
  };
  load(h0);
  const Coef cf = load_coef<T, D, kSplit>(nr, weight, pos, li, active, err);
  // groups of a warp may have fewer heads than others: the shuffles need all
  const int batches = (int)__reduce_max_sync(0xffffffffu, (unsigned)(h1 - h0 + HB - 1) / HB);
  for (int i = 0; i < batches; ++i) {
    const int h = h0 + i * HB;
    Raw8<T> now[HB];
#pragma unroll
    for (int j = 0; j < HB; ++j) now[j] = x[j];
    if (i + 1 < batches) load(h + HB);
#pragma unroll
    for (int j = 0; j < HB; ++j) {
      const Row8 y = norm_rope_row<T, D, kSplit>(nr, now[j], weight != nullptr, cf, li);
      if (h + j < h1) store8(out.p, dst + (int64_t)(h + j) * D, y, n_out, err);
    }
  }
}

}  // namespace rf

// norm_rope.cuh -- the norm and rotation of one head's row, shared by
// qk_norm_rope.cu and kv_append_paged.cu.
//
// A row of D elements is held by a group of D / 8 neighbouring lanes, eight
// consecutive elements a lane (one 16-byte load in bf16).  With x the row,
//     y_i = x_i * rsqrt(mean(x^2) + eps) * w_i        (where there is a weight)
// and, for the first rot elements, a rotation of pairs by the token's angles:
//     (a, b) -> (a cos - b sin, b cos + a sin),
// the pair j being elements (j, j + rot / 2) (half-split) or (2j, 2j + 1)
// (interleaved).  Both forms are one formula per element,
//     out_i = y_i c_i + y_partner(i) s_i,   s_i = -sin for a, +sin for b,
// with the partner in the lane rot / 16 away or in the same lane.  Everything
// is fp32 (one warp-shuffle reduction for the sum of squares); the caller
// rounds once.  rot % 16 == 0, so a lane's eight elements are all rotated or
// none, and all in the same half.
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
};
template <>
struct Raw8<float> {
  static constexpr int kWords = 8;
  uint32_t w[8];
  __device__ __forceinline__ float get(int e) const { return __uint_as_float(w[e]); }
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

__device__ __forceinline__ void store8(__nv_bfloat16* p, int64_t i, const float (&v)[8], int64_t n,
                                       unsigned* err) {
  if (!RF_IN(err, i + 7, n) || !RF_IN(err, i, n)) return;
  *reinterpret_cast<uint4*>(p + i) =
      make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                 pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, int64_t i, const float (&v)[8], int64_t n,
                                       unsigned* err) {
  if (!RF_IN(err, i + 7, n) || !RF_IN(err, i, n)) return;
  reinterpret_cast<float4*>(p + i)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p + i)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// This lane's part of the tables' row of one position: c and signed s of its
// eight elements.  Only called where the lane's elements are rotated.
struct RopeLane {
  float c[8], s[8];
};

__device__ __forceinline__ RopeLane load_rope(const NormRope& nr, int pos, int li, unsigned* err) {
  RopeLane r;
  const int half = nr.rot >> 1;
  const int64_t n = (int64_t)nr.max_pos * half;
  if (nr.interleaved) {
    const int64_t at = (int64_t)pos * half + 4 * li;
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (RF_IN(err, at + 3, n)) {
      c = __ldg(reinterpret_cast<const float4*>(nr.cos + at));
      s = __ldg(reinterpret_cast<const float4*>(nr.sin + at));
    }
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      r.c[e] = cc[e >> 1];
      r.s[e] = (e & 1) ? ss[e >> 1] : -ss[e >> 1];
    }
    return r;
  }
  const bool second = 8 * li >= half;
  const int64_t at = (int64_t)pos * half + 8 * li - (second ? half : 0);
  if (RF_IN(err, at + 7, n)) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(nr.cos + at) + k);
      const float4 s = __ldg(reinterpret_cast<const float4*>(nr.sin + at) + k);
      r.c[4 * k] = c.x;
      r.c[4 * k + 1] = c.y;
      r.c[4 * k + 2] = c.z;
      r.c[4 * k + 3] = c.w;
      r.s[4 * k] = second ? s.x : -s.x;
      r.s[4 * k + 1] = second ? s.y : -s.y;
      r.s[4 * k + 2] = second ? s.z : -s.z;
      r.s[4 * k + 3] = second ? s.w : -s.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      r.c[e] = 1.f;
      r.s[e] = 0.f;
    }
  }
  return r;
}

// Norm weights of a lane's elements and, for the half-split rotation, of its
// partner lane's.
struct WeightLane {
  float own[8], other[8];
};

// Lane of the group that holds the half-split partners of lane li's elements.
__device__ __forceinline__ int partner_lane(const NormRope& nr, int li) {
  const int h = nr.rot >> 4;                       // lanes per half
  return li < h ? li + h : li - h;
}

template <typename T, int D>
__device__ __forceinline__ WeightLane load_weight(const NormRope& nr, const T* w, int li,
                                                  unsigned* err) {
  WeightLane r;
  const Raw8<T> a = load8<T>(w, 8 * li, D, err);
#pragma unroll
  for (int e = 0; e < 8; ++e) r.own[e] = a.get(e);
  if (!nr.interleaved && 8 * li < nr.rot) {
    const Raw8<T> b = load8<T>(w, 8 * partner_lane(nr, li), D, err);
#pragma unroll
    for (int e = 0; e < 8; ++e) r.other[e] = b.get(e);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) r.other[e] = 0.f;
  }
  return r;
}

// Norm (has_w) and rotation (nr.rot > 0) of a group's row.  Called by all 32
// lanes of a warp together; has_w may differ between the warp's groups.
template <typename T, int D>
__device__ __forceinline__ void norm_rope_row(const NormRope& nr, const Raw8<T>& x, bool has_w,
                                              const WeightLane& w, const RopeLane& rp, int li,
                                              float (&out)[8]) {
  constexpr int LG = D / 8;
  float rstd = 1.f;
  if (nr.wq || nr.wk) {                 // the same for every lane: the shuffles need all of them
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x.get(e), x.get(e), ss);
#pragma unroll
    for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    rstd = rsqrtf(fmaf(ss, 1.f / D, nr.eps));
  }
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = has_w ? x.get(e) * rstd * w.own[e] : x.get(e);
  const bool rotated = 8 * li < nr.rot;
  if (nr.rot == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = y[e];
  } else if (nr.interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = rotated ? fmaf(y[e ^ 1], rp.s[e], y[e] * rp.c[e]) : y[e];
  } else {
    Raw8<T> p;
    const int src = rotated ? partner_lane(nr, li) : li;
#pragma unroll
    for (int k = 0; k < Raw8<T>::kWords; ++k) p.w[k] = __shfl_sync(0xffffffffu, x.w[k], src, LG);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float yp = has_w ? p.get(e) * rstd * w.other[e] : p.get(e);
      out[e] = rotated ? fmaf(yp, rp.s[e], y[e] * rp.c[e]) : y[e];
    }
  }
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

// Heads [h0, h0 + HB) (those below H) of token t at position pos, by one lane
// group: loads of all HB heads first, so that each lane has HB loads in flight.
template <typename T, int D, int HB>
__device__ __forceinline__ void norm_rope_heads(const NormRope& nr, const T* weight,
                                                const RowsIn<T>& in, const RowsOut<T>& out, int T_,
                                                int H, int t, int h0, int pos, bool active,
                                                int li, unsigned* err) {
  const int64_t n_in = (int64_t)(T_ - 1) * in.ld + (int64_t)H * D;
  const int64_t n_out = (int64_t)(T_ - 1) * out.ld + (int64_t)H * D;
  Raw8<T> x[HB];
#pragma unroll
  for (int j = 0; j < HB; ++j) {
    if (active && h0 + j < H) {
      x[j] = load8<T>(in.p, (int64_t)t * in.ld + (int64_t)(h0 + j) * D + 8 * li, n_in, err);
    } else {
#pragma unroll
      for (int k = 0; k < Raw8<T>::kWords; ++k) x[j].w[k] = 0u;
    }
  }
  RopeLane rp = {};
  if (active && 8 * li < nr.rot) rp = load_rope(nr, pos, li, err);
  WeightLane w = {};
  if (weight) w = load_weight<T, D>(nr, weight, li, err);
#pragma unroll
  for (int j = 0; j < HB; ++j) {
    float y[8];
    norm_rope_row<T, D>(nr, x[j], weight != nullptr, w, rp, li, y);
    if (active && h0 + j < H)
      store8(out.p, (int64_t)t * out.ld + (int64_t)(h0 + j) * D + 8 * li, y, n_out, err);
  }
}

}  // namespace rf

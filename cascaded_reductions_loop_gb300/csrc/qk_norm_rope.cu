// qk_norm_rope.cu -- RMS norm of every query and key head and the position
// rotation, in one pass over the rows (the formulas stand in norm_rope.cuh).
//
// What bounds it: memory.  Each element is read once and written once.  One
// lane group of d / 8 lanes takes nh heads of one token, in batches of HB whose
// 16-byte loads are in flight together while the batch before is worked on;
// the token's angles and the weights are loaded once for all of them.
//
// Measured (GB300, CUDA graph, inputs larger than L2; copy rate 6683 GB/s):
//   8191 tokens, 32 + 8 heads of 128, bf16, norm, half-split    31 us, 5.5 TB/s
//   32768 and 131072 tokens, the same               108 and 416 us, 6.4 and 6.6 TB/s
//   4096 tokens, 16 + 16 heads of 64, fp32, half rotated        14 us, 4.9 TB/s
//   16384 and 65536 tokens, the same                 46 and 161 us, 5.9 and 6.7 TB/s
//   32 tokens, 32 + 8 heads of 128                             2.3 us: launch
// One head a lane group, everything made anew for it, took 65 us for the first:
// 186 instructions for 32 lanes' loads of 16 bytes, and the issue slots bound it.
// The bf16 sizes lie 5.7 to 5.9 us above 3.13 ns a token (launch, first and last
// wave).  The fp32 ones make 3.4, 3.4 and 13.5 waves of CTAs, two an SM by their
// registers, and the part of a wave counts.
#include "norm_rope.cuh"

namespace rf {
namespace {

constexpr int kThreads = 256;

template <typename T, int D, int HB, bool kSplit>
__global__ void __launch_bounds__(kThreads)
    qk_norm_rope_kernel(const NormRope nr, const RowsIn<T> q, const RowsIn<T> k,
                        const RowsOut<T> qo, const RowsOut<T> ko, const int* __restrict__ positions,
                        int T_, int Hq, int Hkv, int nh, unsigned* err) {
  constexpr int LG = D / 8;
  const int nqb = (Hq + nh - 1) / nh, nblk = nqb + (Hkv + nh - 1) / nh;
  const int li = threadIdx.x % LG;
  const int64_t u = (int64_t)blockIdx.x * (kThreads / LG) + threadIdx.x / LG;
  // a warp's groups: neighbouring tokens of one block of heads
  const int blk = (int)(u / T_), t = (int)(u - (int64_t)blk * T_);
  bool active = blk < nblk;
  int pos = 0;
  if (active && nr.rot > 0) {
    pos = RF_IN(err, t, T_) ? __ldg(positions + t) : 0;
    if (pos < 0 || pos >= nr.max_pos) {            // the tables have no such row
      raise_error(err, kDevErrInput);
      active = false;
    }
  }
  const bool is_q = blk < nqb;
  norm_rope_heads<T, D, HB, kSplit>(nr, static_cast<const T*>(is_q ? nr.wq : nr.wk), is_q ? q : k,
                                    is_q ? qo : ko, T_, is_q ? Hq : Hkv, t,
                                    (is_q ? blk : blk - nqb) * nh, nh, pos, active, li, err);
}

template <typename T, int D>
cudaError_t launch(const NormRope& nr, const void* Q, int64_t ldq, const void* K, int64_t ldk,
                   void* Qo, int64_t ldqo, void* Ko, int64_t ldko, const int* positions, int T_,
                   int Hq, int Hkv, int sms, unsigned* err, cudaStream_t s) {
  const int nh = heads_per_group((int64_t)T_ * (Hq + Hkv), Hq > Hkv ? Hq : Hkv, D, sms);
  const int64_t nblk = (Hq + nh - 1) / nh + (Hkv + nh - 1) / nh;
  const int64_t per = kThreads / (D / 8);
  const unsigned grid = (unsigned)(((int64_t)T_ * nblk + per - 1) / per);
  const RowsIn<T> q = {static_cast<const T*>(Q), ldq}, k = {static_cast<const T*>(K), ldk};
  const RowsOut<T> qo = {static_cast<T*>(Qo), ldqo}, ko = {static_cast<T*>(Ko), ldko};
#define RF_GO(HB, SPLIT)                                  \
  qk_norm_rope_kernel<T, D, HB, SPLIT><<<grid, kThreads, 0, s>>>(nr, q, k, qo, ko, positions, T_, \
                                                                 Hq, Hkv, nh, err)
  if (is_split(nr)) {
    if (nh > 1) RF_GO(4, true);
    else RF_GO(1, true);
  } else {
    if (nh > 1) RF_GO(4, false);
    else RF_GO(1, false);
  }
#undef RF_GO
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(int dtype, const NormRope& nr, const void* Q, int64_t ldq,
                                const void* K, int64_t ldk, void* Qo, int64_t ldqo, void* Ko,
                                int64_t ldko, const int* positions, int T, int Hq, int Hkv, int d,
                                unsigned* err, cudaStream_t s) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidValue;
#define RF_GO(TY, DD)                                                                              \
  return launch<TY, DD>(nr, Q, ldq, K, ldk, Qo, ldqo, Ko, ldko, positions, T, Hq, Hkv, sms, err, s)
  if (dtype == RF_BF16) {
    if (d == 64) RF_GO(__nv_bfloat16, 64);
    RF_GO(__nv_bfloat16, 128);
  }
  if (d == 64) RF_GO(float, 64);
  RF_GO(float, 128);
#undef RF_GO
}

}  // namespace rf

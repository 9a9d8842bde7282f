// qk_norm_rope.cu -- RMS norm of every query and key head and the position
// rotation, in one pass over the rows (the formulas stand in norm_rope.cuh).
//
// What bounds it: memory.  Each element is read once and written once; the
// tables' row of a token (rot x 4 bytes) is read by its head blocks, from L1
// after the first.  One lane group of d / 8 lanes takes HB heads of one token:
// the weights and the token's angles are loaded once for them and the HB
// 16-byte loads are in flight together.
#include "norm_rope.cuh"

namespace rf {
namespace {

constexpr int kThreads = 256;

template <typename T, int D, int HB>
__global__ void __launch_bounds__(kThreads)
    qk_norm_rope_kernel(const NormRope nr, const RowsIn<T> q, const RowsIn<T> k,
                        const RowsOut<T> qo, const RowsOut<T> ko, const int* __restrict__ positions,
                        int T_, int Hq, int Hkv, unsigned* err) {
  constexpr int LG = D / 8;
  const int nqb = (Hq + HB - 1) / HB, nblk = nqb + (Hkv + HB - 1) / HB;
  const int li = threadIdx.x % LG;
  const int64_t u = (int64_t)blockIdx.x * (kThreads / LG) + threadIdx.x / LG;
  const int t = (int)(u / nblk), blk = (int)(u % nblk);
  bool active = t < T_;
  int pos = 0;
  if (active && nr.rot > 0) {
    pos = RF_IN(err, t, T_) ? __ldg(positions + t) : 0;
    if (pos < 0 || pos >= nr.max_pos) {            // the tables have no such row
      raise_error(err, kDevErrInput);
      active = false;
    }
  }
  const bool is_q = blk < nqb;
  norm_rope_heads<T, D, HB>(nr, static_cast<const T*>(is_q ? nr.wq : nr.wk), is_q ? q : k,
                            is_q ? qo : ko, T_, is_q ? Hq : Hkv, t, (is_q ? blk : blk - nqb) * HB,
                            pos, active, li, err);
}

template <typename T, int D, int HB>
cudaError_t launch(const NormRope& nr, const void* Q, int64_t ldq, const void* K, int64_t ldk,
                   void* Qo, int64_t ldqo, void* Ko, int64_t ldko, const int* positions, int T_,
                   int Hq, int Hkv, unsigned* err, cudaStream_t s) {
  const int64_t nblk = (Hq + HB - 1) / HB + (Hkv + HB - 1) / HB;
  const int64_t per = kThreads / (D / 8);
  const int64_t grid = ((int64_t)T_ * nblk + per - 1) / per;
  qk_norm_rope_kernel<T, D, HB><<<(unsigned)grid, kThreads, 0, s>>>(
      nr, RowsIn<T>{static_cast<const T*>(Q), ldq}, RowsIn<T>{static_cast<const T*>(K), ldk},
      RowsOut<T>{static_cast<T*>(Qo), ldqo}, RowsOut<T>{static_cast<T*>(Ko), ldko}, positions, T_,
      Hq, Hkv, err);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(int dtype, const NormRope& nr, const void* Q, int64_t ldq,
                                const void* K, int64_t ldk, void* Qo, int64_t ldqo, void* Ko,
                                int64_t ldko, const int* positions, int T, int Hq, int Hkv, int d,
                                unsigned* err, cudaStream_t s) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidValue;
  // Four heads a lane group where that still fills the device (64 rows of heads
  // for each group of a CTA an SM); one where it would leave SMs idle.
  const bool many = (int64_t)T * (Hq + Hkv) >= (int64_t)sms * 64 * (kThreads * 8 / d);
#define RF_GO(TY, DD)                                                                             \
  return many                                                                                     \
             ? launch<TY, DD, 4>(nr, Q, ldq, K, ldk, Qo, ldqo, Ko, ldko, positions, T, Hq, Hkv,   \
                                 err, s)                                                          \
             : launch<TY, DD, 1>(nr, Q, ldq, K, ldk, Qo, ldqo, Ko, ldko, positions, T, Hq, Hkv,   \
                                 err, s)
  if (dtype == RF_BF16) {
    if (d == 64) RF_GO(__nv_bfloat16, 64);
    RF_GO(__nv_bfloat16, 128);
  }
  if (d == 64) RF_GO(float, 64);
  RF_GO(float, 128);
#undef RF_GO
}

}  // namespace rf

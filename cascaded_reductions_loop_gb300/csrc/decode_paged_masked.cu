// decode_paged_masked.cu -- the instances of the paged decode attention
// (decode_paged.cuh) whose rows read only some of the keys: a window with sinks,
// a tree of drafted tokens.
#include "decode_paged.cuh"

namespace rf {

cudaError_t launch_decode_paged_masked(const PagedKV& c, const Mask& mask, const void* Q, void* O,
                                       int Hq, int Tq, float scale, void* workspace, unsigned* err,
                                       cudaStream_t s) {
  return launch_any<true>(c, mask, Q, O, Hq, Tq, scale, workspace, err, s);
}

}  // namespace rf

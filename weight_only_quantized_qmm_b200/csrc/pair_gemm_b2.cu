// Instantiations of the many-token products of packed weights for 2-bit codes.
#include "pair_gemm.cuh"

namespace qmm {
namespace pg {

cudaError_t dispatch_b2(int op, bool pair, Args& p, Maps& tm, int clusters, cudaStream_t st) {
  return dispatch<2>(op, pair, p, tm, clusters, st);
}

}  // namespace pg
}  // namespace qmm

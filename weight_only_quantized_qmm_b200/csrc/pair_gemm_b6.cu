// Instantiations of the many-token products of packed weights for 6-bit codes.
#include "pair_gemm.cuh"

namespace qmm {
namespace pg {

cudaError_t dispatch_b6(int op, bool pair, Args& p, Maps& tm, int clusters, cudaStream_t st) {
  return dispatch<6>(op, pair, p, tm, clusters, st);
}

}  // namespace pg
}  // namespace qmm

// Instantiations of the many-token products of packed weights for 4-bit codes.
#include "pair_gemm.cuh"

namespace qmm {
namespace pg {

cudaError_t dispatch_b4(int op, bool pair, Args& p, Maps& tm, int clusters, cudaStream_t st) {
  return dispatch<4>(op, pair, p, tm, clusters, st);
}

}  // namespace pg
}  // namespace qmm

// Instantiations of the many-token products of packed weights for 6-bit codes.
#include "pair_gemm.cuh"

namespace qmm {
namespace pg {

cudaError_t dispatch_b6(int op, bool pair, Args& p, Maps& tm, int clusters, cudaStream_t st) {
  return dispatch<6>(op, pair, p, tm, clusters, st);
}

cudaError_t dispatch_both_b6(Args& dx, Maps& dx_maps, const Args& dp, const Maps& dp_maps, int dx_clusters,
                             int dp_pairs, cudaStream_t st) {
  return dispatch_both<6>(dx, dx_maps, dp, dp_maps, dx_clusters, dp_pairs, st);
}

}  // namespace pg
}  // namespace qmm

// The product kernels of linear layers: gradients in one piece (linear_gemm.cuh).
#include "linear_gemm.cuh"

namespace fbob {
namespace lin {

cudaError_t gemm_out(Layout layout, int tile_n, const GemmArgs& g, cudaStream_t s) {
  return layout == kNN ? launch<kNN, kOut>(tile_n, g, "linear_dx", s) : launch<kTN, kOut>(tile_n, g, "linear_dw", s);
}

}  // namespace lin
}  // namespace fbob

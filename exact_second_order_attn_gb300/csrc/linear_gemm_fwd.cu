// The product kernels of linear layers: forward (linear_gemm.cuh).
#include "linear_gemm.cuh"

namespace fbob {
namespace lin {

cudaError_t gemm_forward(int tile_n, const GemmArgs& g, cudaStream_t s) {
  return launch<kNT, kForward>(tile_n, g, "linear_fwd", s);
}

}  // namespace lin
}  // namespace fbob

// The product kernels of linear layers: gradients (linear_gemm.cuh).
#include "linear_gemm.cuh"

namespace fbob {
namespace lin {

cudaError_t gemm_gradients(const GemmArgs& g, cudaStream_t s) {
  return launch<kGradients, kGradient>(256, g, "linear_gradients", s);
}

}  // namespace lin
}  // namespace fbob

// The product kernels of linear layers: second order (linear_gemm.cuh).
#include "linear_gemm.cuh"

namespace fbob {
namespace lin {

cudaError_t gemm_second(int tile_n, const GemmArgs& g, cudaStream_t s) {
  return launch<kNT, kSecond>(tile_n, g, "linear_second", s);
}

}  // namespace lin
}  // namespace fbob

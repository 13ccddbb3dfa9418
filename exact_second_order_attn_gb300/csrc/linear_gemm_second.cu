// The product kernels of linear layers: second order (linear_gemm.cuh).
#include "linear_gemm.cuh"

namespace fbob {
namespace lin {

cudaError_t gemm_second(int tile_n, const GemmArgs& g, cudaStream_t s) {
  return g.fp32 || g.ep.q_planes > 1 || g.ep.dz_planes > 1 ? launch<kNT, kSecondTerms>(128, g, "linear_second", s)
                                                          : launch<kNT, kSecond>(tile_n, g, "linear_second", s);
}

}  // namespace lin
}  // namespace fbob

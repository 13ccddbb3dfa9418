// The product kernels of linear layers: the forward in slabs (linear_gemm.cuh).
#include "linear_gemm.cuh"

namespace fbob {
namespace lin {

cudaError_t gemm_slabs(const GemmArgs& g, cudaStream_t s) { return launch<kNT, kSlab>(256, g, "linear_fwd_slabs", s); }

}  // namespace lin
}  // namespace fbob

// The product kernels of linear layers: contractions in slabs (linear_gemm.cuh).
#include "linear_gemm.cuh"

namespace fbob {
namespace lin {

cudaError_t gemm_slab(Layout layout, const GemmArgs& g, cudaStream_t s) {
  switch (layout) {
    case kNT: return launch<kNT, kSlab>(256, g, "linear_fwd_slabs", s);
    case kNN: return launch<kNN, kSlab>(256, g, "linear_dx_slabs", s);
    case kTN: return launch<kTN, kSlab>(256, g, "linear_dw_slabs", s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace lin
}  // namespace fbob

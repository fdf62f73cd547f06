// The CUDA-core kernels of attention over a paged cache for bf16 inputs (one translation unit per
// type, so that they compile in parallel).
#include "lla_paged_cc.cuh"

namespace lla {
namespace paged {

cudaError_t attend_cc_bf16(const Params& p, int d, int dv, cudaStream_t s) {
  return pick_d<__nv_bfloat16>(p, d, dv, s);
}
cudaError_t mass_cc_bf16(const Params& p, int d, cudaStream_t s) {
  return pick_mass<__nv_bfloat16>(p, d, s);
}
cudaError_t join_bf16(const Params& p, int dv, cudaStream_t s) {
  return pick_join<__nv_bfloat16>(p, dv, s);
}

}  // namespace paged
}  // namespace lla

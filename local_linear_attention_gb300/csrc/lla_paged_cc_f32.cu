// The CUDA-core kernels behind the fp32 attention over a paged cache (one translation unit per type, so
// that they compile in parallel).
#include "lla_paged_cc.cuh"

namespace lla {
namespace paged {

cudaError_t mass_cc_f32(const Params& p, int d, cudaStream_t s) {
  return pick_mass<float>(p, d, s);
}
cudaError_t join_f32(const Params& p, int dv, cudaStream_t s) {
  return pick_join<float>(p, dv, s);
}

}  // namespace paged
}  // namespace lla

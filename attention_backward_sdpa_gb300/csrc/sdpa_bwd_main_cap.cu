// sdpa_bwd_main_cap.cu -- the main kernels (sdpa_bwd_main.cuh) with capped scores
// (score.cuh) and no slopes, for both io types, in their own translation unit so that they compile
// in parallel with the others.
#include "sdpa_bwd_main.cuh"

namespace sdpa {

cudaError_t main_cap_kernel_setup() {
  cudaError_t e = main_variant_setup<false, false, MOD_CAP>();
  if (e == cudaSuccess) e = main_variant_setup<false, true, MOD_CAP>();
  return e;
}

cudaError_t launch_main_cap(const MainMaps& maps, const ChainParams& p, cudaStream_t s) {
  return p.f16 ? launch_main_variant<false, true, MOD_CAP>(maps, p, s)
               : launch_main_variant<false, false, MOD_CAP>(maps, p, s);
}

}  // namespace sdpa

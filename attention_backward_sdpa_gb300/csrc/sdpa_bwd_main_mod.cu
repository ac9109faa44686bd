// sdpa_bwd_main_mod.cu -- the main kernels (sdpa_bwd_main.cuh) with modified
// scores (score.cuh): capped and distance-biased scores and row ranges, for both
// io types, in their own translation unit so that they compile in parallel.
#include "sdpa_bwd_main.cuh"

namespace sdpa {

cudaError_t main_mod_kernel_setup() {
  cudaError_t e = main_variant_setup<false, false, true>();
  if (e == cudaSuccess) e = main_variant_setup<false, true, true>();
  return e;
}

cudaError_t launch_main_mod(const MainMaps& maps, const ChainParams& p, cudaStream_t s) {
  return p.f16 ? launch_main_variant<false, true, true>(maps, p, s)
               : launch_main_variant<false, false, true>(maps, p, s);
}

}  // namespace sdpa

// sdpa_bwd_main_mod.cu -- the main kernels (sdpa_bwd_main.cuh) with modified
// scores (score.cuh) but neither cap nor slopes: row ranges, for both io types, in their own
// translation unit so that they compile in parallel.
#include "sdpa_bwd_main.cuh"

namespace sdpa {

cudaError_t main_mod_kernel_setup() {
  cudaError_t e = main_variant_setup<false, false, MOD_ROWS>();
  if (e == cudaSuccess) e = main_variant_setup<false, true, MOD_ROWS>();
  if (e == cudaSuccess) e = main_cap_kernel_setup();
  if (e == cudaSuccess) e = main_slopes_kernel_setup();
  return e;
}

cudaError_t launch_main_mod(const MainMaps& maps, const ChainParams& p, cudaStream_t s) {
  if (p.mods.slopes != nullptr) return launch_main_slopes(maps, p, s);
  if (p.mods.on == MOD_CAP) return launch_main_cap(maps, p, s);
  return p.f16 ? launch_main_variant<false, true, MOD_ROWS>(maps, p, s)
               : launch_main_variant<false, false, MOD_ROWS>(maps, p, s);
}

}  // namespace sdpa

// sdpa_bwd_main_slopes.cu -- the main kernels (sdpa_bwd_main.cuh) with distance slopes
// (score.cuh), without and with a cap, for both io types. Kernels of their own, because
// the slopes' steps cost the others time (a cap alone 276 -> 270 us, documents alone
// 81 -> 77, both 108 -> 103; B 1, Hq 32, Hkv 8, S 4096, D 128, deterministic).
#include "sdpa_bwd_main.cuh"

namespace sdpa {

cudaError_t main_slopes_kernel_setup() {
  cudaError_t e = main_variant_setup<false, false, MOD_ROWS, true>();
  if (e == cudaSuccess) e = main_variant_setup<false, true, MOD_ROWS, true>();
  if (e == cudaSuccess) e = main_variant_setup<false, false, MOD_CAP, true>();
  if (e == cudaSuccess) e = main_variant_setup<false, true, MOD_CAP, true>();
  return e;
}

cudaError_t launch_main_slopes(const MainMaps& maps, const ChainParams& p, cudaStream_t s) {
  if (p.mods.on == MOD_CAP)
    return p.f16 ? launch_main_variant<false, true, MOD_CAP, true>(maps, p, s)
                 : launch_main_variant<false, false, MOD_CAP, true>(maps, p, s);
  return p.f16 ? launch_main_variant<false, true, MOD_ROWS, true>(maps, p, s)
               : launch_main_variant<false, false, MOD_ROWS, true>(maps, p, s);
}

}  // namespace sdpa

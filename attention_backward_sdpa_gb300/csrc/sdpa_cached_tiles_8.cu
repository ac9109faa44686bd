// sdpa_cached_tiles_8.cu -- the many-rows attention (sdpa_cached_tiles.cuh) over caches of e4m3.
#include "sdpa_cached_tiles.cuh"

namespace sdpa {

cudaError_t launch_cached_tiles_8(const CachedParams& p, cudaStream_t s) {
  return cached_tiles::launch_type<true>(p, s);
}

cudaError_t cached_tiles_8_setup() {
  const cudaError_t e = cached_tiles::setup_type<true, true>();
  return e != cudaSuccess ? e : cached_tiles::setup_type<true, false>();
}

}  // namespace sdpa

// sdpa_cached_tiles_16.cu -- the many-rows attention (sdpa_cached_tiles.cuh) over caches of bf16 and fp16.
#include "sdpa_cached_tiles.cuh"

namespace sdpa {

cudaError_t launch_cached_tiles_16(const CachedParams& p, cudaStream_t s) {
  return cached_tiles::launch_type<false>(p, s);
}

cudaError_t cached_tiles_16_setup() {
  const cudaError_t e = cached_tiles::setup_type<false, true>();
  return e != cudaSuccess ? e : cached_tiles::setup_type<false, false>();
}

}  // namespace sdpa

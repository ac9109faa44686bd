// sdpa_cached_rows_8.cu -- the few-rows attention (sdpa_cached_rows.cuh) over caches of e4m3.
#include "sdpa_cached_rows.cuh"

namespace sdpa {

cudaError_t launch_cached_rows_8(const CachedParams& p, int nr, cudaStream_t s) {
  return p.f16 ? cached_rows::launch_type<cached_rows::E4M3, true>(p, nr, s)
               : cached_rows::launch_type<cached_rows::E4M3, false>(p, nr, s);
}

cudaError_t cached_rows_8_setup() {
  const cudaError_t e = cached_rows::setup_type<cached_rows::E4M3, true>();
  return e != cudaSuccess ? e : cached_rows::setup_type<cached_rows::E4M3, false>();
}

}  // namespace sdpa

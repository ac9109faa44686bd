// rope.cuh -- what the rotary kernels (sdpa_rope.cu, sdpa_kv_cache.cu) share: a frequency as
// a 64-bit fraction of a turn, the sine and cosine of a position's angle, and 16-bit io values.
#pragma once

#include "common.cuh"

namespace sdpa {

constexpr int ROPE_MAX_PAIRS = 256;  // rot_dim <= 512

// 2^64 * f / (2 pi) modulo 2^64, for any finite f.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  double t = f * 0.15915494309189533577;
  t -= floor(t);
  // [0, 1] in two 32-bit pieces (a product by 2^64 may round to 2^64).
  const double hi = floor(t * 4294967296.0);
  const double lo = (t * 4294967296.0 - hi) * 4294967296.0;
  return ((uint64_t)hi << 32) + (uint64_t)lo;
}

__device__ __forceinline__ void angle_sin_cos(uint64_t turn, int pos, float& sn, float& cs) {
  const uint64_t a = turn * (uint64_t)(int64_t)pos;
  sincospif((float)(int32_t)(a >> 32) * 4.6566128730773926e-10f, &sn, &cs);  // 2^-31: half turns
}

// The same from the nearest quarter turn, so that the fp32 angle is at most an eighth of a turn: its
// rounding is a quarter as large. (What is rounded to e4m3 next falls on the other side of a tie less often.)
__device__ __forceinline__ void angle_sin_cos_near(uint64_t turn, int pos, float& sn, float& cs) {
  const uint64_t a = turn * (uint64_t)(int64_t)pos, quarter = (a + (1ull << 61)) >> 62;
  float s, c;
  sincospif((float)(int32_t)((int64_t)(a - (quarter << 62)) >> 32) * 4.6566128730773926e-10f, &s, &c);
  sn = (quarter & 1) ? c : s;
  cs = (quarter & 1) ? s : c;
  if (quarter & 2) sn = -sn;
  if ((quarter + 1) & 2) cs = -cs;
}

template <bool F16>
__device__ __forceinline__ float io_f32(uint16_t v) {
  return F16 ? __half2float(__ushort_as_half(v)) : __uint_as_float((uint32_t)v << 16);
}

}  // namespace sdpa

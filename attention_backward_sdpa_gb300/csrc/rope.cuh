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

// The same from the nearest quarter turn, so that the fp32 angle y is at most an eighth of a turn: its
// rounding is a quarter as large. (What is rounded to e4m3 next falls on the other side of a tie less often.)
// There the Taylor series is enough: |y| <= pi / 4, and what is left out is y^11 / 11! < 1.8e-9 of the sine and
// y^12 / 12! < 1.2e-10 of the cosine. 30 instructions, where the library's call from any angle takes over twice as many
// (and eight of them in line do not fit the instruction cache).
__device__ __forceinline__ void angle_sin_cos_near(uint64_t turn, int pos, float& sn, float& cs) {
  const uint64_t a = turn * (uint64_t)(int64_t)pos;
  const uint32_t top = (uint32_t)(a >> 32), quarter = (top + (1u << 29)) >> 30;  // (3 rounded up: 4, as 0)
  const float y = (float)(int32_t)(top - (quarter << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float z = y * y;
  const float s = fmaf(y * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), y);
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
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

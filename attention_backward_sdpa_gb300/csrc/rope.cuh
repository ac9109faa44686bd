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

// The same from the nearest quarter turn, where |y| <= pi / 4 and the Taylor series is short: what is left out is
// y^11 / 11! < 1.8e-9 of the sine and y^12 / 12! < 1.2e-10 of the cosine. 30 instructions, where the library's call from
// any angle takes over twice as many (and eight of them in line do not fit the instruction cache).
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

// Sine and cosine to 2^-33, as sums of two floats: for rotated values that are rounded to e4m3, where an error of
// fp32's size puts one in a million on the other side of a tie, a whole step of 2^-3 off. The angle is the nearest of 33
// nodes, a 128th of a turn apart, and d, |d| <= pi / 128 (at most 2^24 units of 2^-32 turns, a whole fp32 number, and a
// fraction): sin(n + d) = sin n + (sin n (cos d - 1) + cos n sin d), where only cos n * d is large enough to be
// needed to more than 24 bits.
struct SinCos2 {
  float sh, sl, ch, cl;
};
struct SinCosNodes {
  SinCos2 at[33];
};
constexpr SinCosNodes sin_cos_nodes() {
  SinCosNodes t{};
  for (int k = -16; k <= 16; ++k) {
    const double x = k * (3.14159265358979323846 / 64), z = x * x;
    double sn = 0.0, cs = 0.0;
    for (int i = 11; i >= 0; --i) {  // Taylor, to x^23 and x^22
      sn = 1.0 - sn * z / ((2 * i + 2) * (2 * i + 3));
      cs = 1.0 - cs * z / ((2 * i + 1) * (2 * i + 2));
    }
    sn *= x;
    SinCos2& n = t.at[k + 16];
    n.sh = (float)sn, n.sl = (float)(sn - (float)sn);
    n.ch = (float)cs, n.cl = (float)(cs - (float)cs);
  }
  return t;
}
__device__ __forceinline__ SinCos2 angle_sin_cos_2(uint64_t turn, int pos, const SinCos2* nodes, float mult) {
  const uint64_t a = turn * (uint64_t)(int64_t)pos;
  const uint64_t quarter = (a + (1ull << 61)) >> 62;
  const int64_t x = (int64_t)(a - (quarter << 62));                // at most an eighth of a turn
  const int k = (int)((x + (1ll << 56)) >> 57);                    // the nearest node
  const int64_t r = x - ((int64_t)k << 57);
  const SinCos2 n = nodes[k + 16];
  constexpr float TURN = 1.46291807926715968e-9f;                  // 2 pi / 2^32, and what fp32 leaves of it
  constexpr float REST = (float)(6.283185307179586477 / 4294967296.0 - (double)TURN);
  const float u = (float)(int)(r >> 32), frac = (float)(uint32_t)r * 2.3283064365386963e-10f;
  const float d = u * TURN, dl = fmaf(u, TURN, -d) + fmaf(u, REST, frac * TURN);
  const float z = d * d;
  const float s3 = d * z * fmaf(z, 1.f / 120.f, -1.f / 6.f);       // sin d - d
  const float c2 = z * fmaf(z, 1.f / 24.f, -0.5f) - d * dl;        // cos d - 1
  auto turned = [&](float ah, float al, float bh, float bl, float& hi, float& lo) {  // a cos d + b sin d
    const float p = __fmul_rn(bh, d), e = fmaf(bh, d, -p) + fmaf(bl, d, al) + fmaf(ah, c2, bh * (s3 + dl));
    const float sum = ah + p, back = sum - ah;                     // (exact: sum, and what it leaves)
    const float rest = (ah - (sum - back)) + (p - back) + e;
    hi = sum + rest;
    lo = rest - (hi - sum);
  };
  SinCos2 o;
  turned(n.sh, n.sl, n.ch, n.cl, o.sh, o.sl);
  turned(n.ch, n.cl, -n.sh, -n.sl, o.ch, o.cl);
  if (quarter & 1) {
    const SinCos2 t = o;
    o = SinCos2{t.ch, t.cl, -t.sh, -t.sl};
  }
  if (quarter & 2) o = SinCos2{-o.sh, -o.sl, -o.ch, -o.cl};
  const float sh = __fmul_rn(o.sh, mult), ch = __fmul_rn(o.ch, mult);
  return SinCos2{sh, fmaf(o.sh, mult, -sh) + o.sl * mult, ch, fmaf(o.ch, mult, -ch) + o.cl * mult};
}
// a c + b s from such c and s, rounded to odd: to the neighbour with an odd last bit where it is no fp32 number. A further
// rounding to fewer bits then gives what one rounding of the sum itself would.
__device__ __forceinline__ float dot_odd(float a, float ch, float cl, float b, float sh, float sl) {
  const float p = __fmul_rn(a, ch), q = __fmul_rn(b, sh);
  if (!(fabsf(p + q) < INFINITY)) return p + q;
  const float e = fmaf(a, ch, -p) + fmaf(b, sh, -q) + fmaf(a, cl, b * sl);
  const float sum = p + q, back = sum - p;
  const float rest = (p - (sum - back)) + (q - back) + e;
  const float r = sum + rest, left = rest - (r - sum);
  uint32_t bits = __float_as_uint(r);
  if ((bits & 1u) == 0u && left != 0.f) bits += (left < 0.f) == (r < 0.f) ? 1u : 0xFFFFFFFFu;
  return r == 0.f ? r : __uint_as_float(bits);
}

template <bool F16>
__device__ __forceinline__ float io_f32(uint16_t v) {
  return F16 ? __half2float(__ushort_as_half(v)) : __uint_as_float((uint32_t)v << 16);
}

}  // namespace sdpa

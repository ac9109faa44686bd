// score.cuh -- scores that are modified between the score GEMM and the softmax,
// for the forward and backward kernels instantiated with MOD: a tanh cap, a
// bias that falls with distance, and a range of visible keys per query row.
//
//   y = scale * (q . k)                          the scaled score
//   x = cap * tanh(y / cap)                      with a cap, else x = y
//   x = x - slope[h] * |q + diag - k|            with slopes
//   row q sees the keys of [lo(q), hi(q)) only   with a mask plan
// and the derivative the backward needs is dx/dy = 1 - tanh(y / cap)^2.
//
// The mask plan (sdpa_mask_plan.cu writes it once per batch) holds every row's
// key range, a summary per 64-row query tile, which bounds the key tiles that
// the tile sees and tells which of them need no mask, and a summary per 128-key
// tile, which bounds the query tiles that see it. Document masks and prefix
// masks are such ranges: in the forward a thread owns a row, so its range
// joins the causal and window bounds at no cost per score.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace sdpa {

struct ScoreMods {
  int on;              // run the MOD instantiations
  float cap_in;        // scale / cap: tanh argument per unit of q . k (0: no cap)
  float cap_log2;      // cap * log2(e)
  float cap_small;     // |q . k| up to which the polynomial below serves (may be 0)
  float cap_c[6];      // its coefficients in powers of q . k: TANH_C[i] * cap_in^(2 i + 1)
  const float* slopes; // (Hq,) distance slopes, or null
  // Mask plan regions, or null. lo/hi are keys, clamped to [0, S_kv].
  const int2* ranges;  // [B][n_qt * 64] {lo, hi}; rows past S_q hold {0, 0}
  const int4* q_sum;   // [B][n_qt] {min lo, max hi, max lo, min hi} of the tile's rows (below)
  const int2* k_sum;   // [B][n_kt] {first, last} 64-row query tile that sees the 128-key tile
  const int2* k_rows;  // [B][n_kt * 128] {first, last} query row that sees the key, where `k_exact`
  const int* k_exact;  // [B] whether every key of the batch row is seen by exactly the rows of k_rows
};

// Regions of a mask plan of n_qt 64-row and n_kt 128-key tiles, as byte offsets.
// q_sum: min lo and max hi over the rows with a key (INT_MAX and 0 when no row
// has one); max lo and min hi over all rows below S_q, where a row with no key
// counts as lo = INT_MAX, so that a tile is only taken as unmasked when every
// row sees all of it.
// k_rows, k_exact: where lo and hi of a batch row never decrease from row to row (every
// document and prefix mask), the rows that see a key are neighbours: those up to the
// last with lo <= key, from the first with hi > key. The backward, whose threads own a
// key, then masks by two bounds in registers; for other ranges it reads the 64 row
// ranges of every tile that needs a mask.
struct MaskPlanLayout {
  size_t ranges, q_sum, k_sum, k_rows, k_exact, bytes;
};
__host__ __device__ inline MaskPlanLayout mask_plan_layout(int B, int n_qt, int n_kt) {
  MaskPlanLayout l;
  l.ranges = 0;
  l.q_sum = (l.ranges + (size_t)B * n_qt * 64 * sizeof(int2) + 255) & ~(size_t)255;
  l.k_sum = (l.q_sum + (size_t)B * n_qt * sizeof(int4) + 255) & ~(size_t)255;
  l.k_rows = (l.k_sum + (size_t)B * n_kt * sizeof(int2) + 255) & ~(size_t)255;
  l.k_exact = l.k_rows + (size_t)B * n_kt * 128 * sizeof(int2);
  l.bytes = (l.k_exact + (size_t)B * sizeof(int) + 255) & ~(size_t)255;
  return l;
}

// tanh(y), y = s * cap_in. Two forms, both accurate relative to the value (a large cap
// multiplies whatever absolute error small values have):
//   |y| <= 0.8   an odd polynomial of degree 11 (least-maximum fit of tanh(y) / y in
//                y^2, 5.8e-8 before its roundings), with the powers of cap_in taken
//                into its coefficients: 7 multiply-adds, no division;
//   any y        y N(y^2) / D(y^2), N and D of degree 4, fitted on [0, 8] (6.4e-9,
//                3.1e-7 with the fp32 roundings), y clamped to [-8, 8] (1 - tanh(8) =
//                2.3e-7): 12 multiply-adds and a reciprocal.
// A warp takes the first when all its scores of a tile allow it, which they do unless
// scores come near the cap. (The quotient 1 - 2 / (1 + e^2y) would take two
// special-function results a score where the softmax's exponential already fills that
// unit, and rounds small values to multiples of 2^-24.)
constexpr float TANH_SMALL = 0.8f;
constexpr float TANH_C[6] = {9.999999421e-01f,  -3.333267492e-01f, 1.332104826e-01f,
                             -5.311431475e-02f, 1.909329914e-02f,  -4.355298764e-03f};
constexpr float TANH_CLAMP = 8.0f;

// The polynomial's coefficients as pairs, times `mult` (1: tanh; cap * log2(e): the
// capped score in log2 units).
struct CapCoef {
  uint64_t c[6];
};
__device__ __forceinline__ CapCoef cap_coef(const float (&c)[6], float mult) {
  CapCoef k;
#pragma unroll
  for (int i = 0; i < 6; ++i) k.c[i] = f2_pack(c[i] * mult, c[i] * mult);
  return k;
}
// A pair of scores s: mult * tanh(s * cap_in), |s| <= cap_small.
__device__ __forceinline__ uint64_t tanh2_small(uint64_t s, const CapCoef& k) {
  const uint64_t u = f2_mul(s, s);
  uint64_t r = f2_fma(u, k.c[5], k.c[4]);
  r = f2_fma(u, r, k.c[3]);
  r = f2_fma(u, r, k.c[2]);
  r = f2_fma(u, r, k.c[1]);
  r = f2_fma(u, r, k.c[0]);
  return f2_mul(s, r);
}
// x within [-lim, lim], a NaN kept (a visible score that is not a number has to show).
__device__ __forceinline__ float clamp_nan(float x, float lim) {
  float r;
  asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, %2;\n\tmin.NaN.f32 %0, t, %3;\n\t}" : "=f"(r) : "f"(x), "f"(-lim), "f"(lim));
  return r;
}
// A pair of any scores: tanh(s * cap_in).
__device__ __forceinline__ uint64_t tanh2_any(float s0, float s1, float cap_in) {
  constexpr float N[5] = {9.999999936e-01f, 1.344449871e-01f, 3.571599056e-03f, 2.189467996e-05f, 1.523044372e-08f};
  constexpr float D[5] = {1.0f, 4.677782538e-01f, 2.616444638e-02f, 3.411293732e-04f, 8.522456963e-07f};
  const float y0 = clamp_nan(s0 * cap_in, TANH_CLAMP), y1 = clamp_nan(s1 * cap_in, TANH_CLAMP);
  const uint64_t y = f2_pack(y0, y1), u = f2_mul(y, y);
  uint64_t n = f2_fma(u, f2_pack(N[4], N[4]), f2_pack(N[3], N[3]));
  uint64_t d = f2_fma(u, f2_pack(D[4], D[4]), f2_pack(D[3], D[3]));
#pragma unroll
  for (int i = 2; i >= 0; --i) {
    n = f2_fma(u, n, f2_pack(N[i], N[i]));
    d = f2_fma(u, d, f2_pack(D[i], D[i]));
  }
  float d0, d1, r0, r1;
  f2_unpack(d, d0, d1);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(d0));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(d1));
  return f2_mul(f2_mul(y, n), f2_pack(r0, r1));
}

// The backward's replay of one tile for one thread (its key k against 64 query
// rows): what the modified scores and the masks need besides S^T.
struct ModTile {
  float cap_in, cap_log2, cap_small, scale_log2;
  const float (*cap_c)[6];
  float slope2;        // the head's slope * log2(e) (0 without slopes)
  float dist;          // q0 + diag - k: the distance of row i is |dist + i|
  int q_lo, q_hi;      // rows (relative to the tile) inside the causal / window / length bounds
  int k;
  const int2* ranges;  // the tile's row ranges, or null when every row sees the whole key tile
  bool masked;         // the tile needs a mask (uniform across the warp)
};

// Half H (rows 32 H .. 32 H + 31) of a tile's replay. r: S^T on entry. P gets the
// masked probabilities times the cap's derivative, which is all that the dS step
// reads; w gets the probabilities themselves as io pairs for the dV product.
// (The two are formed together so that no thread holds 64 derivatives.)
template <bool F16, int H>
__device__ __forceinline__ void mod_replay_half(const ModTile& m, const float* lse, uint32_t (&r)[32], float (&P)[64],
                                                uint32_t (&w)[16]) {
  const float4* lse4 = reinterpret_cast<const float4*>(lse) + H * 8;
  if (m.cap_in != 0.f) {
    // r becomes the tanh.
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < 32; i += 2) big = max3(big, fabsf(__uint_as_float(r[i])), fabsf(__uint_as_float(r[i + 1])));
    if (__all_sync(0xffffffffu, big <= m.cap_small)) {
      const CapCoef k = cap_coef(*m.cap_c, 1.f);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        float t0, t1;
        f2_unpack(tanh2_small(f2_pack(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), k), t0, t1);
        r[i] = __float_as_uint(t0);
        r[i + 1] = __float_as_uint(t1);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        float t0, t1;
        f2_unpack(tanh2_any(__uint_as_float(r[i]), __uint_as_float(r[i + 1]), m.cap_in), t0, t1);
        r[i] = __float_as_uint(t0);
        r[i + 1] = __float_as_uint(t1);
      }
    }
  }
  const float c1 = m.cap_in != 0.f ? m.cap_log2 : m.scale_log2;
  const uint64_t c2 = f2_pack(c1, c1);
  float x[32];
#pragma unroll
  for (int i4 = 0; i4 < 8; ++i4) {
    const float4 l = lse4[i4];
    const int i = i4 * 4;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), c2, f2_pack(-l.x, -l.y)), x[i], x[i + 1]);
    f2_unpack(f2_fma(f2_pack(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])), c2, f2_pack(-l.z, -l.w)), x[i + 2],
              x[i + 3]);
  }
  if (m.slope2 != 0.f) {
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = fmaf(-m.slope2, fabsf(m.dist + (float)(H * 32 + i)), x[i]);
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) P[H * 32 + i] = ex2_approx(x[i]);
  if (m.masked) {
    // (r as well: a masked score may be an overflow or NaN, and 0 times that is NaN.)
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (H * 32 + i < m.q_lo || H * 32 + i > m.q_hi) {
        P[H * 32 + i] = 0.f;
        r[i] = 0u;
      }
    if (m.ranges != nullptr) {
      // Two rows per 16-byte load, the same address for the whole warp.
      const int4* rg = reinterpret_cast<const int4*>(m.ranges) + H * 16;
#pragma unroll
      for (int i2 = 0; i2 < 16; ++i2) {
        const int4 v = __ldg(rg + i2);
        if (m.k < v.x || m.k >= v.y) {
          P[H * 32 + 2 * i2] = 0.f;
          r[2 * i2] = 0u;
        }
        if (m.k < v.z || m.k >= v.w) {
          P[H * 32 + 2 * i2 + 1] = 0.f;
          r[2 * i2 + 1] = 0u;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack_io2<F16>(P[H * 32 + 2 * i], P[H * 32 + 2 * i + 1]);
  if (m.cap_in != 0.f) {
    // P times the derivative 1 - t^2.
    const uint64_t one = f2_pack(1.f, 1.f);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float t0 = __uint_as_float(r[i]), t1 = __uint_as_float(r[i + 1]);
      const uint64_t f = f2_fma(f2_pack(-t0, -t1), f2_pack(t0, t1), one);
      f2_unpack(f2_mul(f, f2_pack(P[H * 32 + i], P[H * 32 + i + 1])), P[H * 32 + i], P[H * 32 + i + 1]);
    }
  }
}

}  // namespace sdpa

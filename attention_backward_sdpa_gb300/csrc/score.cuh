// score.cuh -- scores that are modified between the score GEMM and the softmax,
// for the forward and backward kernels instantiated with MOD (MOD_ROWS without a cap,
// MOD_CAP with one): a tanh cap, a bias that falls with distance, and a range of
// visible keys per query row.
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

enum : int { MOD_NONE = 0, MOD_ROWS = 1, MOD_CAP = 2 };

struct ScoreMods {
  int on;              // MOD_NONE, MOD_ROWS or MOD_CAP: which instantiation runs
  float cap_in;        // scale / cap: tanh argument per unit of q . k (0: no cap)
  float cap_log2;      // cap * log2(e)
  float cap_small;     // |q . k| up to which the polynomial below serves (-1: it never does)
  float cap_c[5];      // its coefficients in powers of q . k: TANH_C[i] * cap_in^(2 i + 1), or 0 where that
                       // is no normal fp32 number (cap_small is then lower)
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
//   |y| <= 0.65  an odd polynomial of degree 9 (least-maximum fit of tanh(y) / y in
//                y^2, 1.5e-7 before its roundings), with the powers of cap_in taken
//                into its coefficients: 6 multiply-adds, no division (a lower bound for caps whose
//                powers leave fp32's range);
//   any y        y N(y^2) / D(y^2), N and D of degree 4, fitted on [0, 8] (1.6e-8 with the
//                constants below, 3.1e-7 with the fp32 roundings), y clamped to [-8, 8] (1 - tanh(8) =
//                2.3e-7): 12 multiply-adds and a reciprocal.
// A warp takes the first when all its scores of a tile allow it, which they do unless
// scores come near the cap. (The quotient 1 - 2 / (1 + e^2y) would take two
// special-function results a score where the softmax's exponential already fills that
// unit, and rounds small values to multiples of 2^-24.)
constexpr float TANH_SMALL = 0.65f;
constexpr float TANH_C[5] = {9.999998465e-01f, -3.333150019e-01f, 1.329787373e-01f, -5.151791598e-02f,
                             1.462508501e-02f};
constexpr float TANH_CLAMP = 8.0f;

// The polynomial's coefficients as pairs, times `mult` (1: tanh; cap * log2(e): the
// capped score in log2 units).
struct CapCoef {
  uint64_t c[5];
};
__device__ __forceinline__ CapCoef cap_coef(const float (&c)[5], float mult) {
  CapCoef k;
#pragma unroll
  for (int i = 0; i < 5; ++i) k.c[i] = f2_pack(c[i] * mult, c[i] * mult);
  return k;
}
// N pairs of scores s, |s| <= cap_small, step by step side by side (left to itself the
// compiler may take one pair's dependent steps after another's): r[i] = the polynomial's
// value, so that mult * tanh(s * cap_in) = s * r.
template <int N>
__device__ __forceinline__ void tanh2_poly(const uint64_t (&s)[N], const CapCoef& k, uint64_t (&r)[N]) {
  uint64_t u[N];
#pragma unroll
  for (int i = 0; i < N; ++i) u[i] = f2_mul(s[i], s[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = f2_fma(u[i], k.c[4], k.c[3]);
#pragma unroll
  for (int c = 2; c >= 0; --c)
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = f2_fma(u[i], r[i], k.c[c]);
}
// x within [-lim, lim], a NaN kept (a visible score that is not a number has to show).
__device__ __forceinline__ float clamp_nan(float x, float lim) {
  float r;
  asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, %2;\n\tmin.NaN.f32 %0, t, %3;\n\t}" : "=f"(r) : "f"(x), "f"(-lim), "f"(lim));
  return r;
}
// N pairs of any scores, in place: tanh(s * cap_in). CLAMP: |s * cap_in| may pass TANH_CLAMP.
template <int N, bool CLAMP = true>
__device__ __forceinline__ void tanh2_any(uint64_t (&s)[N], float cap_in) {
  constexpr float NU[5] = {9.999999936e-01f, 1.344449871e-01f, 3.571599056e-03f, 2.189467996e-05f, 1.523044372e-08f};
  constexpr float DE[5] = {1.0f, 4.677782538e-01f, 2.616444638e-02f, 3.411293732e-04f, 8.522456963e-07f};
  uint64_t u[N], n[N], d[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (!CLAMP) {
      s[i] = f2_mul(s[i], f2_pack(cap_in, cap_in));
      continue;
    }
    float y0, y1;
    f2_unpack(s[i], y0, y1);
    s[i] = f2_pack(clamp_nan(y0 * cap_in, TANH_CLAMP), clamp_nan(y1 * cap_in, TANH_CLAMP));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) u[i] = f2_mul(s[i], s[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) n[i] = f2_fma(u[i], f2_pack(NU[4], NU[4]), f2_pack(NU[3], NU[3]));
#pragma unroll
  for (int i = 0; i < N; ++i) d[i] = f2_fma(u[i], f2_pack(DE[4], DE[4]), f2_pack(DE[3], DE[3]));
#pragma unroll
  for (int c = 2; c >= 0; --c) {
#pragma unroll
    for (int i = 0; i < N; ++i) n[i] = f2_fma(u[i], n[i], f2_pack(NU[c], NU[c]));
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = f2_fma(u[i], d[i], f2_pack(DE[c], DE[c]));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float d0, d1, r0, r1;
    f2_unpack(d[i], d0, d1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(d0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(d1));
    s[i] = f2_mul(f2_mul(s[i], n[i]), f2_pack(r0, r1));
  }
}
// Pairs a step takes side by side: 16 where the registers allow it (a thread's 64 scores
// 484 cycles against 598 with 8), 8 in the backward.
constexpr int SIDE = 8, FWD_SIDE = 16;

// The backward's replay of one tile for one thread (its key k against 64 query
// rows): what the modified scores and the masks need besides S^T.
//
// In these kernels everything runs on pairs of neighbouring query rows, and the row
// statistics (preprocess) come negated, so that no step needs a sign of its own: n_lse =
// -(LSE * log2(e) + slope2 * i), i the row within its tile, and n_delta = -delta. With a
// cap, P is then multiplied by t^2 - 1 instead of 1 - t^2, so dS comes out negated, and
// the host hands these kernels -scale for dQ and dK.
struct ModTile {
  float slope2;        // the head's slope * log2(e) (0 without slopes)
  float dist;          // q0 + diag - k: the distance of row i is |dist + i|
  uint32_t see[2];     // by halves of 32 rows: bit i set when row i sees the key
  bool full[2];        // uniform across the warp: all the half's rows see all its keys
  bool ahead[2];       // all the half's rows are at or past the warp's keys: no |.| needed
};

// The call's scaling: c2 = log2(e) times the cap, or times the scale, in pairs (the exponent
// per tanh or per score), and the cap's other constants.
struct ModCap {
  uint64_t c2;
  float cap_in, cap_small;
};
__device__ __forceinline__ ModCap mod_cap(const ScoreMods& m, float scale_log2) {
  const float c = m.cap_in != 0.f ? m.cap_log2 : scale_log2;
  return ModCap{f2_pack(c, c), m.cap_in, m.cap_small};
}

// What half h (0, 1) of a tile looks like.
struct ModHalf {
  uint32_t see;
  bool full, ahead;
};
__device__ __forceinline__ ModHalf mod_half(const ModTile& m, int h) {
  return h ? ModHalf{m.see[1], m.full[1], m.ahead[1]} : ModHalf{m.see[0], m.full[0], m.ahead[0]};
}

// With a cap: whether all of the warp's scores r (32 rows of its keys) are within the polynomial.
template <int N>
__device__ __forceinline__ float mod_largest(const uint32_t (&r)[N]) {
  float big[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; i += 2)
    big[(i >> 1) & 3] = max3(big[(i >> 1) & 3], fabsf(__uint_as_float(r[i])), fabsf(__uint_as_float(r[i + 1])));
  return fmaxf(max3(big[0], big[1], big[2]), big[3]);
}
__device__ __forceinline__ bool mod_small(const ModCap& cap, float largest) {
  return __all_sync(0xffffffffu, largest <= cap.cap_small);
}

// Half h (rows 32 h .. 32 h + 31) of a tile's replay. r: S^T on entry. P gets the masked
// probabilities (with a cap times t^2 - 1), which is all that the dS step reads; w the
// probabilities themselves as io pairs for the dV product. (The two are formed together so
// that no thread holds the derivatives too.)
//
// The straight pass, for a half without a mask or |.| and with mod_small(), in which the
// exponentials (a quarter of the FMA rate) run under the neighbouring pairs' polynomials.
template <int MOD, bool F16, bool SLOPES>
__device__ __forceinline__ void mod_replay_straight(const ModTile& tile, int h, const CapCoef& coef, const ModCap& cap,
                                                    const float* n_lse, const uint32_t (&r)[32], uint64_t (&P)[16],
                                                    uint32_t (&w)[16]) {
  const ulonglong2* l2 = reinterpret_cast<const ulonglong2*>(n_lse) + h * 8;  // two pairs a load
  const uint64_t minus_one = f2_pack(-1.f, -1.f);
  const float bias = -tile.slope2 * tile.dist;  // -slope2 (dist + i): the i part is in the row statistics
  const uint64_t bias2 = f2_pack(bias, bias);
#pragma unroll
  for (int blk = 0; blk < 16 / SIDE; ++blk) {
    uint64_t t[SIDE], x[SIDE];
#pragma unroll
    for (int i = 0; i < SIDE; ++i) t[i] = f2_pack(r[2 * (blk * SIDE + i)], r[2 * (blk * SIDE + i) + 1]);
    if constexpr (MOD == MOD_CAP) {
      tanh2_poly(t, coef, x);
#pragma unroll
      for (int i = 0; i < SIDE; ++i) t[i] = f2_mul(t[i], x[i]);
    }
#pragma unroll
    for (int i = 0; i < SIDE; i += 2) {
      const ulonglong2 l = l2[(blk * SIDE + i) / 2];
      x[i] = f2_fma(t[i], cap.c2, SLOPES ? f2_add(l.x, bias2) : l.x);
      x[i + 1] = f2_fma(t[i + 1], cap.c2, SLOPES ? f2_add(l.y, bias2) : l.y);
    }
#pragma unroll
    for (int i = 0; i < SIDE; ++i) {
      float x0, x1;
      f2_unpack(x[i], x0, x1);
      x[i] = f2_pack(ex2_approx(x0), ex2_approx(x1));
      if constexpr (MOD == MOD_CAP) t[i] = f2_fma(t[i], t[i], minus_one);
    }
#pragma unroll
    for (int i = 0; i < SIDE; ++i) {
      float p0, p1;
      f2_unpack(x[i], p0, p1);
      w[blk * SIDE + i] = pack_io2<F16>(p0, p1);
      P[blk * SIDE + i] = MOD == MOD_CAP ? f2_mul(x[i], t[i]) : x[i];
    }
  }
}

// ... and any other half, step by step.
template <int MOD, bool F16, bool SLOPES>
__device__ __forceinline__ void mod_replay_steps(const ModTile& tile, int h, bool small, const CapCoef& coef,
                                                 const ModCap& cap, const float* n_lse, uint32_t (&r)[32],
                                                 uint64_t (&P)[16], uint32_t (&w)[16]) {
  const ModHalf m = mod_half(tile, h);
  const ulonglong2* l2 = reinterpret_cast<const ulonglong2*>(n_lse) + h * 8;
  const uint64_t minus_one = f2_pack(-1.f, -1.f);
  if constexpr (MOD == MOD_CAP) {
    // r becomes the tanh.
#pragma unroll
    for (int blk = 0; blk < 16 / SIDE; ++blk) {
      uint64_t t[SIDE], x[SIDE];
#pragma unroll
      for (int i = 0; i < SIDE; ++i) t[i] = f2_pack(r[2 * (blk * SIDE + i)], r[2 * (blk * SIDE + i) + 1]);
      if (small) {
        tanh2_poly(t, coef, x);
#pragma unroll
        for (int i = 0; i < SIDE; ++i) t[i] = f2_mul(t[i], x[i]);
      } else {
        tanh2_any(t, cap.cap_in);
      }
#pragma unroll
      for (int i = 0; i < SIDE; ++i) f2_unpack(t[i], r[2 * (blk * SIDE + i)], r[2 * (blk * SIDE + i) + 1]);
    }
  }
#pragma unroll
  for (int i4 = 0; i4 < 8; ++i4) {
    const ulonglong2 l = l2[i4];
    P[2 * i4] = f2_fma(f2_pack(r[4 * i4], r[4 * i4 + 1]), cap.c2, l.x);
    P[2 * i4 + 1] = f2_fma(f2_pack(r[4 * i4 + 2], r[4 * i4 + 3]), cap.c2, l.y);
  }
  if (SLOPES && tile.slope2 != 0.f) {
    // -slope2 |dist + i| with the row statistics' -slope2 i taken back.
    const float i0 = h ? 32.f : 0.f;
#pragma unroll
    for (int i2 = 0; i2 < 16; ++i2) {
      const float i = i0 + (float)(2 * i2);
      float x0, x1;
      f2_unpack(P[i2], x0, x1);
      x0 = fmaf(tile.slope2, i - fabsf(tile.dist + i), x0);
      x1 = fmaf(tile.slope2, (i + 1.f) - fabsf(tile.dist + (i + 1.f)), x1);
      P[i2] = f2_pack(x0, x1);
    }
  }
#pragma unroll
  for (int i2 = 0; i2 < 16; ++i2) {
    float x0, x1;
    f2_unpack(P[i2], x0, x1);
    P[i2] = f2_pack(ex2_approx(x0), ex2_approx(x1));
  }
  if (!m.full) {
    // (r as well with a cap: a masked score may be an overflow or NaN, and 0 times that is
    // NaN, so its tanh is taken as 0.)
#pragma unroll
    for (int i2 = 0; i2 < 16; ++i2) {
      const bool see0 = (m.see >> (2 * i2)) & 1u, see1 = (m.see >> (2 * i2 + 1)) & 1u;
      float p0, p1;
      f2_unpack(P[i2], p0, p1);
      P[i2] = f2_pack(see0 ? p0 : 0.f, see1 ? p1 : 0.f);
      if constexpr (MOD == MOD_CAP) {
        r[2 * i2] = see0 ? r[2 * i2] : 0u;
        r[2 * i2 + 1] = see1 ? r[2 * i2 + 1] : 0u;
      }
    }
  }
#pragma unroll
  for (int i2 = 0; i2 < 16; ++i2) {
    float p0, p1;
    f2_unpack(P[i2], p0, p1);
    w[i2] = pack_io2<F16>(p0, p1);
    if constexpr (MOD == MOD_CAP) {
      const uint64_t t = f2_pack(r[2 * i2], r[2 * i2 + 1]);
      P[i2] = f2_mul(P[i2], f2_fma(t, t, minus_one));
    }
  }
}

// dS of half h's 32 query rows as io pairs, P (dP - delta), into the thread's row of the dS^T
// tile (16-byte pieces, XOR-swizzled by the row's `sw`); r holds the half's dP^T.
// CUT: some pairs are masked (not in `see`); theirs is 0, not 0 times a dP that may have
// overflowed.
template <bool F16, bool CUT>
__device__ __forceinline__ void mod_ds_pieces(uint32_t see, int h, const uint64_t (&P)[16], const float* n_delta,
                                              const uint32_t (&r)[32], uint8_t* ds_row, int sw) {
  const ulonglong2* d2 = reinterpret_cast<const ulonglong2*>(n_delta) + h * 8;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const ulonglong2 da = d2[2 * c], db = d2[2 * c + 1];
    const uint64_t d[4] = {da.x, da.y, db.x, db.y};
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = c * 8 + 2 * e;
      float s0, s1;
      f2_unpack(f2_mul(P[c * 4 + e], f2_add(f2_pack(r[i], r[i + 1]), d[e])), s0, s1);
      if constexpr (CUT) {
        s0 = (see >> i) & 1u ? s0 : 0.f;
        s1 = (see >> (i + 1)) & 1u ? s1 : 0.f;
      }
      w[e] = pack_io2<F16>(s0, s1);
    }
    *reinterpret_cast<uint4*>(ds_row + (((h * 4 + c) ^ sw) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace sdpa

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
  const float* slopes; // (Hq,) distance slopes, or null
  // Mask plan regions, or null. lo/hi are keys, clamped to [0, S_kv].
  const int2* ranges;  // [B][n_qt * 64] {lo, hi}; rows past S_q hold {0, 0}
  const int4* q_sum;   // [B][n_qt] {min lo, max hi, max lo, min hi} of the tile's rows (below)
  const int2* k_sum;   // [B][n_kt] {first, last} 64-row query tile that sees the 128-key tile
};

// Regions of a mask plan of n_qt 64-row and n_kt 128-key tiles, as byte offsets.
// q_sum: min lo and max hi over the rows with a key (INT_MAX and 0 when no row
// has one); max lo and min hi over all rows below S_q, where a row with no key
// counts as lo = INT_MAX, so that a tile is only taken as unmasked when every
// row sees all of it.
struct MaskPlanLayout {
  size_t ranges, q_sum, k_sum, bytes;
};
__host__ __device__ inline MaskPlanLayout mask_plan_layout(int B, int n_qt, int n_kt) {
  MaskPlanLayout l;
  l.ranges = 0;
  l.q_sum = (l.ranges + (size_t)B * n_qt * 64 * sizeof(int2) + 255) & ~(size_t)255;
  l.k_sum = (l.q_sum + (size_t)B * n_qt * sizeof(int4) + 255) & ~(size_t)255;
  l.bytes = (l.k_sum + (size_t)B * n_kt * sizeof(int2) + 255) & ~(size_t)255;
  return l;
}

// tanh over all reals, from 1 - 2 / (1 + e^(2|y|)) where |y| > 0.8 (there the
// subtraction loses nothing that matters: the result is above 0.66, the error
// a few units of its last place) and an odd polynomial of degree 11 below
// (relative error 5.8e-8 on [0, 0.8] before its roundings, a least-maximum fit
// of tanh(y) / y in y^2 made for this file): the quotient form alone would
// round small values to multiples of 2^-24, which a large cap multiplies.
constexpr float TANH_SMALL = 0.8f;
constexpr float TANH_C0 = 9.999999421e-01f, TANH_C1 = -3.333267492e-01f, TANH_C2 = 1.332104826e-01f, TANH_C3 = -5.311431475e-02f,
                TANH_C4 = 1.909329914e-02f, TANH_C5 = -4.355298764e-03f;

__device__ __forceinline__ float tanh_small(float y) {
  const float u = y * y;
  float r = fmaf(u, TANH_C5, TANH_C4);
  r = fmaf(u, r, TANH_C3);
  r = fmaf(u, r, TANH_C2);
  r = fmaf(u, r, TANH_C1);
  r = fmaf(u, r, TANH_C0);
  return y * r;
}
__device__ __forceinline__ float tanh_large(float y) {
  float q;
  const float e = ex2_approx(fabsf(y) * 2.8853900817779268f);  // e^(2 |y|), +inf for large y
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.f + e));
  return copysignf(fmaf(-2.f, q, 1.f), y);
}
__device__ __forceinline__ float tanh_any(float y) {
  return fabsf(y) <= TANH_SMALL ? tanh_small(y) : tanh_large(y);
}

// The backward's replay of one tile for one thread (its key k against 64 query
// rows): what the modified scores and the masks need besides S^T.
struct ModTile {
  float cap_in, cap_log2, scale_log2;
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
  float x[32];
  if (m.cap_in != 0.f) {
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) big = fmaxf(big, fabsf(__uint_as_float(r[i])));
    // r becomes tanh: one loop for a warp whose scores all stay below the
    // polynomial's bound, which is every warp unless scores come near the cap.
    if (__all_sync(0xffffffffu, big * m.cap_in <= TANH_SMALL)) {
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(tanh_small(__uint_as_float(r[i]) * m.cap_in));
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(tanh_any(__uint_as_float(r[i]) * m.cap_in));
    }
  }
  const float c = m.cap_in != 0.f ? m.cap_log2 : m.scale_log2;
#pragma unroll
  for (int i4 = 0; i4 < 8; ++i4) {
    const float4 l = lse4[i4];
    x[i4 * 4 + 0] = fmaf(__uint_as_float(r[i4 * 4 + 0]), c, -l.x);
    x[i4 * 4 + 1] = fmaf(__uint_as_float(r[i4 * 4 + 1]), c, -l.y);
    x[i4 * 4 + 2] = fmaf(__uint_as_float(r[i4 * 4 + 2]), c, -l.z);
    x[i4 * 4 + 3] = fmaf(__uint_as_float(r[i4 * 4 + 3]), c, -l.w);
  }
  if (m.slope2 != 0.f) {
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = fmaf(-m.slope2, fabsf(m.dist + (float)(H * 32 + i)), x[i]);
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) P[H * 32 + i] = ex2_approx(x[i]);
  if (m.masked) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (H * 32 + i < m.q_lo || H * 32 + i > m.q_hi) P[H * 32 + i] = 0.f;
    if (m.ranges != nullptr) {
      // Two rows per 16-byte load, the same address for the whole warp.
      const int4* rg = reinterpret_cast<const int4*>(m.ranges) + H * 16;
#pragma unroll
      for (int i2 = 0; i2 < 16; ++i2) {
        const int4 v = __ldg(rg + i2);
        if (m.k < v.x || m.k >= v.y) P[H * 32 + 2 * i2] = 0.f;
        if (m.k < v.z || m.k >= v.w) P[H * 32 + 2 * i2 + 1] = 0.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack_io2<F16>(P[H * 32 + 2 * i], P[H * 32 + 2 * i + 1]);
  if (m.cap_in != 0.f) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float t = __uint_as_float(r[i]);
      // (a masked place stays 0 whatever its score was)
      P[H * 32 + i] = P[H * 32 + i] == 0.f ? 0.f : P[H * 32 + i] * fmaf(-t, t, 1.f);
    }
  }
}

}  // namespace sdpa

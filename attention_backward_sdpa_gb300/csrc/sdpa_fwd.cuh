// sdpa_fwd.cuh -- what the three forward kernels share: the work-item decode of
// the persistent schedule, the bias row loader, a named barrier that also ORs a
// predicate, the constants of the schedule, and the launchers of the other two
// forward kernels, which launch_fwd (sdpa_fwd.cu) calls by head dims.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace sdpa {

namespace fwd_shared {
constexpr int BM = 128;  // query rows per item
constexpr int BK = 128;  // keys per tile
constexpr uint64_t WAIT_LIMIT_NS = 4000000000ull;
constexpr float RESCALE_THRESHOLD = 8.f;  // log2 units: P stays below 2^8 until a raise
// The same under modified scores: P below 2^15, within fp16 (at 8, one row in a warp of 32
// with a late maximum more often takes the tile off the common path: fwd_capped_gqa 170 us
// against 153).
constexpr float MOD_THRESHOLD = 15.f;
constexpr int FWD_SLOTS = 64;             // launch slots of the persistent tickets
}  // namespace fwd_shared

// One 32-byte streaming load (the address 32-byte aligned) into r[at .. at + 7].
__device__ __forceinline__ void ld_global_cs_32b(const void* ptr, uint32_t (&r)[64], int at) {
  asm volatile("ld.global.cs.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[at]), "=r"(r[at + 1]), "=r"(r[at + 2]), "=r"(r[at + 3]), "=r"(r[at + 4]),
                 "=r"(r[at + 5]), "=r"(r[at + 6]), "=r"(r[at + 7])
               : "l"(ptr));
}

// This row's bias for keys kb .. kb + 63 as 32-bit words: on the 16-byte path
// 16-bit pairs (`packed`, 32 words) or fp32 values (64 words); otherwise fp32
// values from scalar loads, 0 past S_kv.
__device__ __forceinline__ void load_fwd_bias_row(const FwdParams& p, long long row_off, int kb, bool live,
                                                  uint32_t (&raw)[64], bool& packed) {
  const bool vec = p.bias_vec && kb + 64 <= p.Skv;  // uniform across the warp
  packed = vec && !p.bias_fp32;
  if (!live) {
#pragma unroll
    for (int i = 0; i < 64; ++i) raw[i] = 0u;
    return;
  }
  const int esz = p.bias_fp32 ? 4 : 2;
  // 32-byte loads (a thread reads whole 32-byte sectors of its row) when every
  // row segment is 32-byte aligned: the base, and rows whose byte length is a
  // multiple of 32 (kb is a multiple of 64 keys). Uniform across the launch.
  const bool v32 = vec && (reinterpret_cast<uintptr_t>(p.bias) & 31u) == 0 && ((long long)p.Skv * esz) % 32 == 0;
  if (v32) {
    const char* src = static_cast<const char*>(p.bias) + (row_off + kb) * esz;
    if (p.bias_fp32) {
#pragma unroll
      for (int v = 0; v < 8; ++v) ld_global_cs_32b(src + 32 * v, raw, 8 * v);
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v) ld_global_cs_32b(src + 32 * v, raw, 8 * v);
#pragma unroll
      for (int i = 32; i < 64; ++i) raw[i] = 0u;
    }
  } else if (vec) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(p.bias) + (row_off + kb) * esz);
    if (p.bias_fp32) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const uint4 x = __ldcs(src + v);
        raw[4 * v] = x.x; raw[4 * v + 1] = x.y; raw[4 * v + 2] = x.z; raw[4 * v + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        const uint4 x = __ldcs(src + v);
        raw[4 * v] = x.x; raw[4 * v + 1] = x.y; raw[4 * v + 2] = x.z; raw[4 * v + 3] = x.w;
      }
#pragma unroll
      for (int i = 32; i < 64; ++i) raw[i] = 0u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      float x = 0.f;
      if (kb + i < p.Skv)
        x = p.bias_fp32 ? __ldcs(static_cast<const float*>(p.bias) + row_off + kb + i)
                        : bias16_to_f32(__ldcs(static_cast<const unsigned short*>(p.bias) + row_off + kb + i),
                                        p.bias_f16 != 0);
      raw[i] = __float_as_uint(x);
    }
  }
}

// A thread's scores of a tile rewritten as x = s * c + bias * log2e, the bias
// widened from 16-bit pairs (`packed`; fp16 when p.bias_f16, else bf16) or taken
// as fp32 words. One loop per element form (the choice is uniform across the
// warp), so that widening an element is a fixed instruction or two: a
// per-element choice between the bf16 and the fp16 widening cost the biased
// forward about a third of its speed.
__device__ __forceinline__ void add_bias_row(const FwdParams& p, float c, const uint32_t (&braw)[64], bool packed,
                                             uint32_t (&sr)[2][32]) {
  constexpr float LOG2E_F = 1.4426950408889634f;
  if (packed && p.bias_f16) {
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      const uint32_t wd = braw[i >> 1];
      const float bv = __half2float(__ushort_as_half((unsigned short)((i & 1) ? (wd >> 16) : (wd & 0xFFFFu))));
      sr[i >> 5][i & 31] = __float_as_uint(fmaf(__uint_as_float(sr[i >> 5][i & 31]), c, bv * LOG2E_F));
    }
  } else if (packed) {
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      const uint32_t wd = braw[i >> 1];
      const float bv = __uint_as_float((i & 1) ? (wd & 0xFFFF0000u) : (wd << 16));
      sr[i >> 5][i & 31] = __float_as_uint(fmaf(__uint_as_float(sr[i >> 5][i & 31]), c, bv * LOG2E_F));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 64; ++i)
      sr[i >> 5][i & 31] =
          __float_as_uint(fmaf(__uint_as_float(sr[i >> 5][i & 31]), c, __uint_as_float(braw[i]) * LOG2E_F));
  }
}

// ---- Modified scores (MOD): a thread's 64 keys of a tile in two chunks of 32. Which
// chunks are seen in full, in part or not at all is decided for a whole warp, so that a
// mask's edge costs the one chunk that it crosses, and a chunk that no row sees costs
// nothing but its zeros.
struct ModChunks {
  bool full[2];     // every row of the warp sees the whole chunk
  bool any[2];      // some row may see a key of it
  bool deferred[2]; // the scores are left to be capped with the exponentials
  bool large;       // ... with some past the polynomial (all within TANH_CLAMP caps)
  bool biased;      // all of them are left to be modified there, the distance bias included:
  float side;       // key i's is -side * (dist - i), side = +-slope2
  float big;        // the largest score of the chunks seen in full, as it is (a cap alone)
};

// A row's state under modified scores, for one item.
struct ModRow {
  int lo, hi;                          // its visible keys [lo, hi] (hi < lo: none)
  int lo_max, hi_min, lo_min, hi_max;  // the same over the warp's rows: what all and what any of them see
  int place;                           // q + diag
  float slope2;                        // the head's distance slope * log2(e)
  // Scores up to this one need no raise of the softmax reference (a cap alone): the cap
  // never widens a difference, so a score c x higher than the reference's is at most x
  // higher capped.
  float raw_ok;
};

// The chunk's scores as modified scores times log2(e): keys from kb, `dist` = q + diag - kb.
template <int MOD, bool SLOPES>
__device__ __forceinline__ void modify_chunk(const ScoreMods& m, const CapCoef& coef, float c, float slope2, float dist,
                                             bool small, uint32_t (&s)[32]) {
  // Every key at or before its row: the bias is -slope2 (dist - i), one multiply-add a
  // score without |.|.
  const bool biased = SLOPES && m.slopes != nullptr, ahead = biased && __all_sync(0xffffffffu, dist >= 31.f);
  const float base = -slope2 * dist;
  const uint64_t c2 = f2_pack(c, c), log2_cap = f2_pack(m.cap_log2, m.cap_log2);
#pragma unroll
  for (int blk = 0; blk < 16 / FWD_SIDE; ++blk) {
    uint64_t x[FWD_SIDE], b[FWD_SIDE];
    uint32_t* const sb = s + blk * FWD_SIDE * 2;
#pragma unroll
    for (int i = 0; i < FWD_SIDE; ++i) x[i] = f2_pack(sb[2 * i], sb[2 * i + 1]);
    if (biased && ahead) {
#pragma unroll
      for (int i = 0; i < FWD_SIDE; ++i) {
        const float i0 = (float)(2 * (blk * FWD_SIDE + i)), i1 = i0 + 1.f;
        b[i] = f2_pack(fmaf(slope2, i0, base), fmaf(slope2, i1, base));
      }
    } else if (biased) {
#pragma unroll
      for (int i = 0; i < FWD_SIDE; ++i) {
        const float i0 = (float)(2 * (blk * FWD_SIDE + i)), i1 = i0 + 1.f;
        b[i] = f2_pack(-slope2 * fabsf(dist - i0), -slope2 * fabsf(dist - i1));
      }
    } else {
#pragma unroll
      for (int i = 0; i < FWD_SIDE; ++i) b[i] = 0ull;
    }
    if constexpr (MOD == MOD_CAP) {
      if (small) {
        uint64_t r[FWD_SIDE];
        tanh2_poly(x, coef, r);
#pragma unroll
        for (int i = 0; i < FWD_SIDE; ++i) x[i] = f2_fma(x[i], r[i], b[i]);
      } else {
        tanh2_any(x, m.cap_in);
#pragma unroll
        for (int i = 0; i < FWD_SIDE; ++i) x[i] = f2_fma(x[i], log2_cap, b[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < FWD_SIDE; ++i) x[i] = f2_fma(x[i], c2, b[i]);
    }
#pragma unroll
    for (int i = 0; i < FWD_SIDE; ++i) f2_unpack(x[i], sb[2 * i], sb[2 * i + 1]);
  }
}

// One capped score in log2 units.
__device__ __forceinline__ float cap_score(float s, const CapCoef& coef) {
  const uint64_t x[1] = {f2_pack(s, s)};
  uint64_t r[1];
  tanh2_poly(x, coef, r);
  float y, z;
  f2_unpack(f2_mul(x[0], r[0]), y, z);
  return y;
}

// Which chunks of the 64 keys from kb the warp sees: from the item's bounds, no votes.
__device__ __forceinline__ void mod_chunks(const ModRow& r, int kb, ModChunks& ch) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c0 = kb + 32 * k;
    ch.full[k] = c0 >= r.lo_max && c0 + 31 <= r.hi_min;
    ch.any[k] = c0 + 31 >= r.lo_min && c0 <= r.hi_max;
    ch.deferred[k] = false;
  }
  ch.large = ch.biased = false;
  ch.big = -INFINITY;
}

// The largest score of a chunk and, in `least`, the smallest or 0.
__device__ __forceinline__ float chunk_extremes(const uint32_t (&s)[32], float& least) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, mn[4] = {least, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float s0 = __uint_as_float(s[i]), s1 = __uint_as_float(s[i + 1]);
    mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], s0, s1);
    mn[(i >> 1) & 3] = min3(mn[(i >> 1) & 3], s0, s1);
  }
  least = min3(mn[0], mn[1], fminf(mn[2], mn[3]));
  return max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
}

// The common tile: both chunks visible to the whole warp, with slopes all keys on one side of
// their rows, and no score that would raise its row's reference m by more than `slack`. The
// scores stay as they are for exp_chunk. (With a cap the maximum is of the sizes, which also
// tells whether the polynomial serves; a negative score that fails the test for a raise only
// costs the other path. The cap never raises a positive score, so that bounds it.) kb: the
// thread's first key; c: scale * log2(e).
template <int MOD, bool SLOPES>
__device__ __forceinline__ bool mod_tile_as_before(const ScoreMods& mods, const ModRow& r, float c, int kb, float m, float slack, const uint32_t (&sr)[2][32],
                                                   ModChunks& ch) {
  if ((MOD != MOD_CAP && !SLOPES) || !ch.full[0] || !ch.full[1]) return false;
  if constexpr (SLOPES) {
    const int first = r.place - (int)(threadIdx.x & 31u);  // the warp's first row's place
    if (first >= kb + 63) ch.side = r.slope2;
    else if (first + 31 <= kb) ch.side = -r.slope2;
    else return false;
  }
  const float d0 = (float)(r.place - kb);
  const float bias = SLOPES ? -fminf(ch.side * d0, ch.side * (d0 - 63.f)) : 0.f;  // the largest of the 64
  float mx[8];
#pragma unroll
  for (int a = 0; a < 8; ++a) mx[a] = -INFINITY;
#pragma unroll
  for (int i = 0; i < 64; i += 2) {
    float s0 = __uint_as_float(sr[i >> 5][i & 31]), s1 = __uint_as_float(sr[i >> 5][(i & 31) + 1]);
    if constexpr (MOD == MOD_CAP) s0 = fabsf(s0), s1 = fabsf(s1);
    mx[(i >> 1) & 7] = max3(mx[(i >> 1) & 7], s0, s1);
  }
  const float big = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
  bool fine = MOD == MOD_CAP && !SLOPES ? big <= r.raw_ok : fmaf(big, c, bias) <= m + slack;
  if (MOD != MOD_CAP) {
    if (!__all_sync(0xffffffffu, fine)) return false;
  } else if (!__all_sync(0xffffffffu, fine && big <= mods.cap_small)) {
    fine = fine && big * mods.cap_in <= TANH_CLAMP;
    if (!__all_sync(0xffffffffu, fine)) return false;
    ch.large = true;
  }
  ch.deferred[0] = ch.deferred[1] = true;
  ch.biased = SLOPES;
  return true;
}

// A tile's scores prepared for the exponentials: modified where `modified` (capped or
// biased; else they stay, and the exponent takes them times cs), -inf where masked. The
// thread's 64 keys start at kb. Returns the row's maximum in log2 units (-inf when it
// sees none).
template <int MOD, bool SLOPES = true>
__device__ __forceinline__ float mod_scores(const ScoreMods& m, const CapCoef& coef, float c, float cs, bool modified,
                                            const ModRow& r, int kb, uint32_t (&sr)[2][32], ModChunks& ch) {
  float big[2] = {-INFINITY, -INFINITY};  // the chunks' largest scores as they are
  bool small = false;
  if constexpr (MOD == MOD_CAP) {
    float least = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (ch.any[k]) big[k] = chunk_extremes(sr[k], least);
    small = __all_sync(0xffffffffu, max3(big[0], big[1], -least) <= m.cap_small);
  }
  float mt = -INFINITY;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!ch.any[k]) continue;
    if (MOD == MOD_CAP && ch.full[k] && (!SLOPES || m.slopes == nullptr)) {
      ch.big = fmaxf(ch.big, big[k]);
      if (small) {
        ch.deferred[k] = true;
        continue;
      }
    }
    const int c0 = kb + 32 * k;
    if (modified) modify_chunk<MOD, SLOPES>(m, coef, c, r.slope2, (float)(r.place - c0), small, sr[k]);
    if (!ch.full[k]) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < r.lo - c0 || i > r.hi - c0) sr[k][i] = 0xFF800000u;  // -inf
    }
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 32; i += 2)
      mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], __uint_as_float(sr[k][i]), __uint_as_float(sr[k][i + 1]));
    mt = fmaxf(mt, max3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * cs);  // cs > 0
  }
  if (MOD == MOD_CAP && (ch.deferred[0] || ch.deferred[1])) mt = fmaxf(mt, cap_score(ch.big, coef));
  return mt;
}

// The chunk's P = ex2(x * cs + neg_m) as io pairs, added to the row sum's partials. CAPPED 1:
// the polynomial's capped score instead of x * cs, 2: that of x up to TANH_CLAMP caps (cs = cap * log2(e));
// BIASED: key i adds slope2 * i (its bias, less what neg_m holds of it).
template <bool F16, int CAPPED, bool BIASED>
__device__ __forceinline__ void exp_chunk(const uint32_t (&s)[32], const CapCoef& coef, float cap_in, float cs,
                                          float neg_m, float slope2, float (&rs)[8], uint32_t (&w)[16]) {
  const uint64_t c2 = f2_pack(cs, cs), m2 = f2_pack(neg_m, neg_m);
  auto add = [&](int i) -> uint64_t {
    return BIASED ? f2_pack(fmaf(slope2, (float)(2 * i), neg_m), fmaf(slope2, (float)(2 * i + 1), neg_m)) : m2;
  };
  uint64_t sum[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) sum[a] = f2_pack(rs[2 * a], rs[2 * a + 1]);
#pragma unroll
  for (int blk = 0; blk < 16 / FWD_SIDE; ++blk) {
    uint64_t x[FWD_SIDE];
#pragma unroll
    for (int i = 0; i < FWD_SIDE; ++i) x[i] = f2_pack(s[2 * (blk * FWD_SIDE + i)], s[2 * (blk * FWD_SIDE + i) + 1]);
    if constexpr (CAPPED == 2) tanh2_any<FWD_SIDE, false>(x, cap_in);
    if constexpr (CAPPED == 1) {
      uint64_t r[FWD_SIDE];
      tanh2_poly(x, coef, r);
#pragma unroll
      for (int i = 0; i < FWD_SIDE; ++i) x[i] = f2_fma(x[i], r[i], add(blk * FWD_SIDE + i));
    } else {
#pragma unroll
      for (int i = 0; i < FWD_SIDE; ++i) x[i] = f2_fma(x[i], c2, add(blk * FWD_SIDE + i));
    }
#pragma unroll
    for (int i = 0; i < FWD_SIDE; ++i) {
      float x0, x1;
      f2_unpack(x[i], x0, x1);
      x[i] = f2_pack(ex2_approx(x0), ex2_approx(x1));
    }
#pragma unroll
    for (int i = 0; i < FWD_SIDE; ++i) {
      float p0, p1;
      f2_unpack(x[i], p0, p1);
      sum[i & 3] = f2_add(sum[i & 3], x[i]);
      w[blk * FWD_SIDE + i] = pack_io2<F16>(p0, p1);
    }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a) f2_unpack(sum[a], rs[2 * a], rs[2 * a + 1]);
}
// Chunk k (keys from kb) of the row; c: scale * log2(e).
template <bool F16, int MOD, bool SLOPES = true>
__device__ __forceinline__ void mod_exp_chunk(const ScoreMods& mods, const uint32_t (&s)[32], const ModChunks& ch,
                                              int k, const ModRow& r, int kb, const CapCoef& coef, float c, float cs,
                                              float neg_m, float (&rs)[8], uint32_t (&w)[16]) {
  if (!ch.any[k]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = 0u;
  } else if (SLOPES && ch.biased) {
    const float add = fmaf(-ch.side, (float)(r.place - kb), neg_m);
    if (MOD == MOD_CAP && ch.large) exp_chunk<F16, 2, true>(s, coef, mods.cap_in, mods.cap_log2, add, ch.side, rs, w);
    else exp_chunk<F16, MOD == MOD_CAP, true>(s, coef, 0.f, c, add, ch.side, rs, w);
  } else if (MOD == MOD_CAP && ch.deferred[k]) {
    if (ch.large) exp_chunk<F16, 2, false>(s, coef, mods.cap_in, mods.cap_log2, neg_m, 0.f, rs, w);
    else exp_chunk<F16, 1, false>(s, coef, 0.f, cs, neg_m, 0.f, rs, w);
  } else {
    exp_chunk<F16, 0, false>(s, coef, 0.f, cs, neg_m, 0.f, rs, w);
  }
}

// One work item: 128 query rows (query tile qt, descending so that under a
// causal mask the longest items come first) of one (batch, query head), and the
// range [kt_lo, kt_lo + n) of 128-key tiles that any of its live rows sees.
struct FwdItem {
  int qt, bh, h, kvh, q0, Lq, Lk, kt_lo, n;
  long long diag;
};

// What an item's bounds read from memory (the batch row's lengths, and under a mask plan
// the summaries of its two 64-row tiles), so that a caller can have the loads in flight.
struct FwdItemLoads {
  int Lq, Lk;
  int2 s;  // first key and end
};
template <int MOD>
__device__ __forceinline__ FwdItemLoads fwd_item_loads(const FwdParams& p, int it) {
  FwdItemLoads l;
  const int BH = p.B * p.Hq, qt = p.n_qt - 1 - it / BH, b = (it % BH) / p.Hq;
  l.Lq = p.Sq;
  l.Lk = p.Skv;
  if (p.seq_q_lens) l.Lq = min(max(p.seq_q_lens[b], 0), p.Sq);
  if (p.seq_kv_lens) l.Lk = min(max(p.seq_kv_lens[b], 0), p.Skv);
  l.s = make_int2(0, p.Skv);
  if constexpr (MOD) {
    if (p.mods.q_sum != nullptr) {  // the hull of the rows' ranges
      const int n64 = ceil_div(p.Sq, BQ);
      const int4* qs = p.mods.q_sum + (long long)b * n64 + 2 * qt;
      const int4 s0 = qs[0];
      l.s = make_int2(s0.x, s0.y);
      if (2 * qt + 1 < n64) {
        const int4 s1 = qs[1];
        l.s = make_int2(min(s0.x, s1.x), max(s0.y, s1.y));
      }
    }
  }
  return l;
}

template <int MOD = MOD_NONE>
__device__ __forceinline__ FwdItem fwd_item(const FwdParams& p, int it, const FwdItemLoads& l) {
  FwdItem w;
  const int BH = p.B * p.Hq;
  w.qt = p.n_qt - 1 - it / BH;
  w.bh = it % BH;
  const int b = w.bh / p.Hq;
  w.h = w.bh % p.Hq;
  w.kvh = b * p.Hkv + w.h / p.G;
  w.q0 = w.qt * fwd_shared::BM;
  w.Lq = l.Lq;
  w.Lk = l.Lk;
  w.diag = p.bottom_right ? (long long)w.Lk - w.Lq : 0;
  const long long Rp = p.window_right > 0 ? p.window_right : 0;
  int kt_lo = 0, kt_hi = -1;
  const long long q_last = min(w.q0 + fwd_shared::BM, w.Lq) - 1;
  if (w.q0 < w.Lq && w.Lk > 0) {
    long long k_hi = w.Lk - 1, k_lo = 0;
    if (p.causal) k_hi = min(k_hi, q_last + w.diag + Rp);
    if (p.window_left >= 0) k_lo = max(0ll, (long long)w.q0 + w.diag - p.window_left);
    if constexpr (MOD) {
      k_lo = max(k_lo, (long long)l.s.x);
      k_hi = min(k_hi, (long long)l.s.y - 1);
    }
    if (k_lo <= k_hi) {
      kt_lo = (int)(k_lo / fwd_shared::BK);
      kt_hi = (int)(k_hi / fwd_shared::BK);
    }
  }
  w.kt_lo = kt_lo;
  w.n = kt_hi - kt_lo + 1;  // may be 0
  return w;
}
template <int MOD = MOD_NONE>
__device__ __forceinline__ FwdItem fwd_item(const FwdParams& p, int it) {
  return fwd_item<MOD>(p, it, fwd_item_loads<MOD>(p, it));
}

// The item's j-th key tile. Under distance slopes from the last to the first: the bias grows
// towards the row's own place, so in ascending order nearly every tile would raise the
// softmax reference and rescale O.
template <bool SLOPES>
__device__ __forceinline__ int key_tile(const FwdItem& w, int j) {
  return SLOPES ? w.kt_lo + w.n - 1 - j : w.kt_lo + j;
}

// An item as the producer publishes it under modified scores, decoded and with the bounds
// that it has read, so that no other role divides indexes or waits for memory to know its
// item: two 16-byte words.
struct FwdItemMsg {
  int4 id;      // item (-1: the end), query tile, batch row, head
  int4 bounds;  // first key tile, number of them, L_q, L_k
};
__device__ __forceinline__ int4 ld_shared_16b(const void* p) {
  int4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(smem_u32(p)) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_16b(void* p, const int4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(smem_u32(p)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void put_msg(FwdItemMsg* at, const FwdItemMsg& m) {
  st_shared_16b(&at->id, m.id);
  st_shared_16b(&at->bounds, m.bounds);
}
__device__ __forceinline__ FwdItemMsg get_msg(const FwdItemMsg* at) {
  return FwdItemMsg{ld_shared_16b(&at->id), ld_shared_16b(&at->bounds)};
}
__device__ __forceinline__ FwdItem fwd_item(const FwdParams& p, const FwdItemMsg& m) {
  FwdItem w;
  w.qt = m.id.y;
  w.h = m.id.w;
  w.bh = m.id.z * p.Hq + w.h;
  w.kvh = 0;  // (the producer's alone)
  w.q0 = w.qt * fwd_shared::BM;
  w.Lq = m.bounds.z;
  w.Lk = m.bounds.w;
  w.diag = p.bottom_right ? (long long)w.Lk - w.Lq : 0;
  w.kt_lo = m.bounds.x;
  w.n = m.bounds.y;
  return w;
}

// What row q of an item reads from memory under modified scores.
struct ModRowLoads {
  int2 range;
  float slope, sink;
};
__device__ __forceinline__ ModRowLoads mod_row_loads(const FwdParams& p, const FwdItem& w, int b, int q) {
  ModRowLoads l;
  l.range = make_int2(0, p.Skv);
  if (p.mods.ranges != nullptr && q < p.Sq)
    l.range = p.mods.ranges[(long long)b * ceil_div(p.Sq, BQ) * BQ + q];
  l.slope = p.mods.slopes != nullptr ? p.mods.slopes[w.h] : 0.f;
  l.sink = p.sink != nullptr ? p.sink[w.h] : 0.f;
  return l;
}

// Row q's state under modified scores in item w: its visible keys by the causal, window,
// length and plan bounds.
__device__ __forceinline__ ModRow mod_row(const FwdParams& p, const FwdItem& w, int q, bool live, const ModRowLoads& l) {
  ModRow r;
  r.place = (int)(q + w.diag);
  long long lo = 0, hi = w.Lk - 1;
  if (p.causal) hi = min(hi, (long long)r.place + max(p.window_right, 0));
  if (p.window_left >= 0) lo = max(lo, (long long)r.place - p.window_left);
  lo = max(lo, (long long)l.range.x);
  hi = min(hi, (long long)l.range.y - 1);
  r.lo = (int)min(lo, (long long)w.Lk);
  r.hi = live ? (int)max(hi, -1ll) : -1;
  r.lo_max = __reduce_max_sync(0xffffffffu, r.lo);
  r.hi_min = __reduce_min_sync(0xffffffffu, r.hi);
  r.lo_min = __reduce_min_sync(0xffffffffu, r.lo);
  r.hi_max = __reduce_max_sync(0xffffffffu, r.hi);
  r.slope2 = l.slope * 1.4426950408889634f;
  r.raw_ok = -INFINITY;
  return r;
}

// One 32-byte global store of two 16-byte halves (the address 32-byte aligned):
// a thread writes a whole 32-byte sector of its O row at once.
__device__ __forceinline__ void st_global_32b(void* ptr, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(ptr), "r"(a.x), "r"(a.y),
               "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// Named barrier over nthreads threads that also ORs a predicate over them.
__device__ __forceinline__ bool named_bar_sync_or(uint32_t id, uint32_t nthreads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %1, 0;\n\tbar.red.or.pred po, %2, %3, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(id), "r"(nthreads)
      : "memory");
  return r != 0;
}


// The other forward kernels, each a persistent grid of `sms` CTAs taking items
// from ticket slot `slot`: the shared-O kernel for the MLA pair (D_qk = 192,
// D_v = 128; sdpa_fwd_shared.cu) and the head-dim-256 kernel (sdpa_fwd_wide.cu).
cudaError_t launch_fwd_shared(const FwdMaps& maps, const FwdParams& p, cudaStream_t s, int sms, int slot);
cudaError_t fwd_shared_setup();
cudaError_t launch_fwd_wide(const FwdMaps& maps, const FwdParams& p, cudaStream_t s, int sms, int slot);
cudaError_t fwd_wide_setup();

}  // namespace sdpa

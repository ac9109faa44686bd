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
// chunks a warp sees in full, in part or not at all is decided for the warp, so that a
// mask's edge costs the one chunk that it crosses, and a chunk that no row sees costs
// nothing but its zeros.
struct ModChunks {
  bool any[2];      // some row of the warp sees a key of the chunk
  bool deferred[2]; // the scores are left to be capped with the exponentials
};

// The chunk's scores as modified scores times log2(e): keys from kb, `dist` = q + diag - kb.
template <int MOD>
__device__ __forceinline__ void modify_chunk(const ScoreMods& m, const CapCoef& coef, float c, float slope2, float dist,
                                             bool small, uint32_t (&s)[32]) {
  // Every key at or before its row: the bias is -slope2 (dist - i), one multiply-add a
  // score without |.|.
  const bool biased = m.slopes != nullptr, ahead = __all_sync(0xffffffffu, dist >= 31.f);
  const float base = -slope2 * dist;
  const uint64_t c2 = f2_pack(c, c), log2_cap = f2_pack(m.cap_log2, m.cap_log2);
#pragma unroll
  for (int blk = 0; blk < 16 / SIDE; ++blk) {
    uint64_t x[SIDE], b[SIDE];
    uint32_t* const sb = s + blk * SIDE * 2;
#pragma unroll
    for (int i = 0; i < SIDE; ++i) x[i] = f2_pack(sb[2 * i], sb[2 * i + 1]);
    if (biased) {
#pragma unroll
      for (int i = 0; i < SIDE; ++i) {
        const float i0 = (float)(2 * (blk * SIDE + i)), i1 = i0 + 1.f;
        b[i] = ahead ? f2_pack(fmaf(slope2, i0, base), fmaf(slope2, i1, base))
                     : f2_pack(-slope2 * fabsf(dist - i0), -slope2 * fabsf(dist - i1));
      }
    } else {
#pragma unroll
      for (int i = 0; i < SIDE; ++i) b[i] = 0ull;
    }
    if constexpr (MOD == MOD_CAP) {
      if (small) {
        uint64_t r[SIDE];
        tanh2_poly(x, coef, r);
#pragma unroll
        for (int i = 0; i < SIDE; ++i) x[i] = f2_fma(x[i], r[i], b[i]);
      } else {
        tanh2_any(x, m.cap_in);
#pragma unroll
        for (int i = 0; i < SIDE; ++i) x[i] = f2_fma(x[i], log2_cap, b[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < SIDE; ++i) x[i] = f2_fma(x[i], c2, b[i]);
    }
#pragma unroll
    for (int i = 0; i < SIDE; ++i) f2_unpack(x[i], sb[2 * i], sb[2 * i + 1]);
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

// A tile's scores prepared for the exponentials: modified where `modified` (capped or
// biased; else they stay, and the exponent takes them times cs), -inf where masked.
// Keys [lo, hi] of the thread's 64 are visible to its row; `dist` = q + diag - its first
// key. Returns the row's maximum in log2 units (-inf when it sees none).
template <int MOD>
__device__ __forceinline__ float mod_scores(const ScoreMods& m, const CapCoef& coef, float c, float cs, bool modified,
                                            float slope2, float dist, int lo, int hi, uint32_t (&sr)[2][32],
                                            ModChunks& ch) {
  bool full[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int l = lo - 32 * k, h = hi - 32 * k;
    full[k] = __all_sync(0xffffffffu, l <= 0 && h >= 31);
    ch.any[k] = full[k] || __any_sync(0xffffffffu, l <= h && l <= 31 && h >= 0);
    ch.deferred[k] = false;
  }
  float big[2] = {-INFINITY, -INFINITY};  // the chunks' largest scores as they are
  bool small = false;
  if constexpr (MOD == MOD_CAP) {
    float least = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!ch.any[k]) continue;
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, mn[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float s0 = __uint_as_float(sr[k][i]), s1 = __uint_as_float(sr[k][i + 1]);
        mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], s0, s1);
        mn[(i >> 1) & 3] = min3(mn[(i >> 1) & 3], s0, s1);
      }
      big[k] = max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
      least = min3(least, fminf(mn[0], mn[1]), fminf(mn[2], mn[3]));
    }
    small = __all_sync(0xffffffffu, max3(big[0], big[1], -least) <= m.cap_small);
  }
  float mt = -INFINITY;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!ch.any[k]) continue;
    if (MOD == MOD_CAP && small && full[k] && m.slopes == nullptr) {
      ch.deferred[k] = true;
      mt = fmaxf(mt, cap_score(big[k], coef));
      continue;
    }
    if (modified) modify_chunk<MOD>(m, coef, c, slope2, dist - (float)(32 * k), small, sr[k]);
    if (!full[k]) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < lo - 32 * k || i > hi - 32 * k) sr[k][i] = 0xFF800000u;  // -inf
    }
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 32; i += 2)
      mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], __uint_as_float(sr[k][i]), __uint_as_float(sr[k][i + 1]));
    mt = fmaxf(mt, max3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * cs);  // cs > 0
  }
  return mt;
}

// The chunk's P = ex2(x * cs + neg_m) as io pairs, added to the row sum's partials.
template <bool F16, bool CAPPED>
__device__ __forceinline__ void exp_chunk(const uint32_t (&s)[32], const CapCoef& coef, float cs, float neg_m,
                                          float (&rs)[8], uint32_t (&w)[16]) {
  const uint64_t c2 = f2_pack(cs, cs), m2 = f2_pack(neg_m, neg_m);
  uint64_t sum[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) sum[a] = f2_pack(rs[2 * a], rs[2 * a + 1]);
#pragma unroll
  for (int blk = 0; blk < 16 / SIDE; ++blk) {
    uint64_t x[SIDE];
#pragma unroll
    for (int i = 0; i < SIDE; ++i) x[i] = f2_pack(s[2 * (blk * SIDE + i)], s[2 * (blk * SIDE + i) + 1]);
    if constexpr (CAPPED) {
      uint64_t r[SIDE];
      tanh2_poly(x, coef, r);
#pragma unroll
      for (int i = 0; i < SIDE; ++i) x[i] = f2_fma(x[i], r[i], m2);
    } else {
#pragma unroll
      for (int i = 0; i < SIDE; ++i) x[i] = f2_fma(x[i], c2, m2);
    }
#pragma unroll
    for (int i = 0; i < SIDE; ++i) {
      float x0, x1;
      f2_unpack(x[i], x0, x1);
      x[i] = f2_pack(ex2_approx(x0), ex2_approx(x1));
    }
#pragma unroll
    for (int i = 0; i < SIDE; ++i) {
      float p0, p1;
      f2_unpack(x[i], p0, p1);
      sum[i & 3] = f2_add(sum[i & 3], x[i]);
      w[blk * SIDE + i] = pack_io2<F16>(p0, p1);
    }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a) f2_unpack(sum[a], rs[2 * a], rs[2 * a + 1]);
}
template <bool F16, int MOD>
__device__ __forceinline__ void mod_exp_chunk(const uint32_t (&s)[32], const ModChunks& ch, int k, const CapCoef& coef,
                                              float cs, float neg_m, float (&rs)[8], uint32_t (&w)[16]) {
  if (!ch.any[k]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = 0u;
  } else if (MOD == MOD_CAP && ch.deferred[k]) {
    exp_chunk<F16, true>(s, coef, cs, neg_m, rs, w);
  } else {
    exp_chunk<F16, false>(s, coef, cs, neg_m, rs, w);
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

// What the modified scores add to row q's state of item w: its key range (a mask
// plan) joins the visible bounds [lo, hi], and the head's distance slope in log2 units.
__device__ __forceinline__ void mod_row(const FwdParams& p, const FwdItem& w, int q, bool live, long long& lo,
                                        long long& hi, float& slope2) {
  if (p.mods.ranges != nullptr && live) {
    const int2 r = p.mods.ranges[(long long)(w.bh / p.Hq) * ceil_div(p.Sq, BQ) * BQ + q];
    lo = max(lo, (long long)r.x);
    hi = min(hi, (long long)r.y - 1);
  }
  if (p.mods.slopes != nullptr) slope2 = p.mods.slopes[w.h] * 1.4426950408889634f;
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

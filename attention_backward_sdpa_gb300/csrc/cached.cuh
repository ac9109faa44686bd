// cached.cuh -- attention over a paged cache: what its two kernels (sdpa_cached_rows.cuh for few
// rows, sdpa_cached_tiles.cuh for many) and the merge of their parts share.
//
//   y = scale * (q . k),  x = cap tanh(y / cap) - slope |place - j|,  place = L - Lq + i,
//   row i sees key j < L when j <= place (causal) and (j >= place - W or j < F),
//   O = sum_j softmax(x [, sink])_j v_j,  LSE = log(sum_j exp(x_j) [+ exp(sink)]).
//
// Rows. The G query heads of a key/value head read the same keys, and the (B, Hq, Sq, D)
// queries of such a group are G * Sq consecutive rows: row r is query r % Sq of head r / Sq. A kernel takes
// them in tiles of `tile_rows`, whatever head and query they are.
//
// Schedule. A segment is one (batch row, row tile, key/value head); it visits n units of
// keys: those that some of its rows sees, the tiles of the first F keys and then those of the
// window, so nothing between them is read. All segments' units in a row are cut into equal shares, one
// a CTA (many rows) or one a warp (few rows): lengths as uneven as they come leave no SM idle, and one long
// sequence is shared by all. A segment inside one share is written at once; of one that is cut every share leaves
// a part (O / l in fp32, and log2 of its sum) in the workspace, two at most: of the segment that
// it begins in the middle of (slot 0), and of the one that it does not finish (slot 1). A note says which
// shares have parts of a segment, and the merge kernel weighs them in their order, so that results do not
// depend on timing. (A merge that found the cut segments by the schedule again took 10 to 28 us, most of
// it in scans and 64-bit divisions.)
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace sdpa {

struct CachedParams {
  KvCacheRef c;
  int B, Hq, G, Sq, R, D;  // R = G * Sq rows of a key/value head
  const void* q;           // (B, Hq, Sq, D)
  void* o;
  float* lse;              // (B, Hq, Sq)
  int f16;
  float scale_log2;        // scale * log2(e)
  int causal, window_left, first_keys;
  const int32_t* seq_q_lens;  // or null
  const float* sink;          // or null
  ScoreMods mods;             // cap and slopes
  int tile_rows, n_rt, tk_shift;  // rows of a tile, tiles of a key/value head, log2 of a unit's keys
  int n_ctas, n_shares, share_units;  // shares at most, and the fewest units of one past 512 of them
  int part_rows;              // rows of a part: those of a tile, or R
  float* part_o;              // [n_shares][2][part_rows][D]
  float* part_lse;            // [n_shares][2][part_rows], log2 units
  int4* cuts;                 // {segment (entry * Hkv + head), first share, last share, 0} or {-1, ..}: many rows,
                              // by the first share to begin in the middle of it; few rows, by segment
  int* status;
};

struct CachedBounds {
  int L, Lq;
  int k_lo, k_hi;  // keys that some row's window sees: [k_lo, k_hi)
  int n, nf, kt;   // units: nf tiles from 0, then n - nf from tile kt
};

// Units of 2^shift keys that hold the first `keys` of them, rounded up without passing 2^31 on the way:
// a page table may have up to 2^31 - 16 positions. (Sums like a key's + 16 are kept on the other side of
// their comparisons for the same reason.)
__host__ __device__ constexpr int cached_units(int keys, int shift) { return keys > 0 ? ((keys - 1) >> shift) + 1 : 0; }
static_assert(cached_units(0x7FFFFFF0, 7) == 1 << 24 && cached_units(0x7FFFFFF0, 5) == 1 << 26 &&
                  cached_units(0x7FFFFF80, 7) == (1 << 24) - 1 && cached_units(129, 7) == 2 && cached_units(128, 7) == 1 &&
                  cached_units(1, 7) == 1 && cached_units(0, 7) == 0,
              "units");

__device__ __forceinline__ CachedBounds cached_bounds(const CachedParams& p, int b, int rt) {
  CachedBounds s;
  s.L = cached_len(p.c, b);
  s.Lq = p.seq_q_lens ? min(max(p.seq_q_lens[b], 0), p.Sq) : p.Sq;
  const int r0 = rt * p.tile_rows, r1 = min(r0 + p.tile_rows, p.R) - 1;
  int i0 = 0, i1 = p.Sq - 1;
  if (p.Sq > 1 && r0 / p.Sq == r1 / p.Sq) i0 = r0 % p.Sq, i1 = r1 % p.Sq;
  i1 = min(i1, s.Lq - 1);
  const int place = s.L - s.Lq;  // of query 0
  s.k_hi = p.causal ? min(s.L, place + i1 + 1) : s.L;
  s.k_lo = p.window_left >= 0 ? (int)max(0ll, (long long)place + i0 - p.window_left) : 0;
  s.n = s.nf = s.kt = 0;
  if (i0 > i1 || s.k_hi <= 0) return s;
  s.kt = s.k_lo >> p.tk_shift;
  s.nf = min(cached_units(min(p.first_keys, s.k_hi), p.tk_shift), s.kt);
  s.n = s.nf + cached_units(s.k_hi, p.tk_shift) - s.kt;
  return s;
}
__device__ __forceinline__ int cached_tile(const CachedBounds& s, int j) { return j < s.nf ? j : s.kt + (j - s.nf); }

// T units (below 2^31) in n shares of q units, the first r of them one more. Few rows: every share of a cut segment costs the
// merge a part, so past 512 shares each has at least 8 units. The 512 is no optimum. With 256, 512, 1,024 and as many as there
// are warps or units: 8 sequences of up to 2,000 keys, 5 rows of 4 heads, fp16 and a cap 19.2, 16.4, 15.7, 16.1 us; one row of 32
// heads, bf16 25.2, 25.1, 16.7, 14.3, over codes 32.4, 20.4, 15.7, 14.6; one sequence of 20,000 over codes 17.7, 17.7, 16.1, 16.8.
struct CachedShares {
  int n, q, r;
  __device__ __forceinline__ CachedShares(const CachedParams& p, int T) {
    n = max(1, min(p.n_shares, max(T / p.share_units, min(T, 512))));
    q = T / n;
    r = T - q * n;
  }
  __device__ __forceinline__ int begin(int i) const { return i * q + min(i, r); }
  __device__ __forceinline__ int of(int t) const {  // the share that has unit t < T
    const int big = r * (q + 1);
    return t < big ? t / (q + 1) : r + (t - big) / q;
  }
};

// Where a share begins: its first unit and the one past its last, its entry e (b * n_rt + rt),
// and that entry's first unit. One call by every thread of the block; sh[W] and `warp_sum` are shared memory.
// W 1: the CTA is a share (and notes the segment that it cuts); else each of its W warps is one.
struct CachedStart {
  int begin, end, te, e;
};
template <int THREADS, int W>
__device__ __forceinline__ CachedStart cached_start(const CachedParams& p, CachedStart* sh, int* warp_sum, int& total) {
  const bool report = blockIdx.x == 0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // (entry e: batch row e / n_rt; few rows have one row tile)
  auto batch = [&](int e) { return W > 1 ? e : e / p.n_rt; };
  const int E = p.B * p.n_rt, per = ceil_div(E, THREADS), e0 = min(tid * per, E), e1 = min(e0 + per, E);
  int sum = 0;
  for (int e = e0; e < e1; ++e) {
    sum += cached_bounds(p, batch(e), e - batch(e) * p.n_rt).n * p.c.Hkv;
    if (report) {
      const int len = p.c.lens[batch(e)];
      if (len < 0 || len > (long long)p.c.max_pages * p.c.page) atomicOr(p.status, STATUS_PAGE);
    }
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int T = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) incl += T;
    T += warp_sum[w];
  }
  total = T;
  const CachedShares shares(p, T);
  const int te0 = incl - sum;
  const bool one = per == 1;  // the thread's sum is its entry's
#pragma unroll 1
  for (int w = 0; w < W; ++w) {
    const int i = blockIdx.x * W + w, begin = i < shares.n ? shares.begin(i) : T;
    if (begin >= te0 && begin < incl) {
      int te = te0;
      for (int e = e0; e < e1; ++e) {
        const int k = one ? sum : cached_bounds(p, batch(e), e - batch(e) * p.n_rt).n * p.c.Hkv;
        if (begin < te + k) {
          sh[w] = CachedStart{begin, shares.begin(i + 1), te, e};
          if constexpr (W == 1) {
            // A segment that the share begins in the middle of, and the share before does not.
            const int m = k / p.c.Hkv, h = (begin - te) / m, first = te + h * m;
            int4 cut = make_int4(-1, 0, 0, 0);
            if (begin > first && shares.begin(i - 1) <= first) cut = make_int4(e * p.c.Hkv + h, i - 1, shares.of(first + m - 1), 0);
            p.cuts[i] = cut;
          }
          break;
        }
        te += k;
      }
    }
    if (begin >= T && tid == 0) {
      sh[w] = CachedStart{T, T, T, -1};
      if (W == 1) p.cuts[i] = make_int4(-1, 0, 0, 0);
    }
  }
  __syncthreads();
  return sh[W == 1 ? 0 : warp];
}

// Rows that see no key: entries that visit no unit, each written by one of the CTAs.
template <int THREADS, bool NOTE>
__device__ __forceinline__ void cached_empty_rows(const CachedParams& p) {
  for (int e = blockIdx.x; e < p.B * p.n_rt; e += gridDim.x) {
    const int b = e / p.n_rt, rt = e % p.n_rt;
    if (cached_bounds(p, b, rt).n > 0) continue;
    if constexpr (NOTE)
      for (int h = threadIdx.x; h < p.c.Hkv; h += THREADS) p.cuts[e * p.c.Hkv + h] = make_int4(-1, 0, 0, 0);
    const int r0 = rt * p.tile_rows, rows = min(p.tile_rows, p.R - r0), pieces = p.D / 8;
    for (int i = threadIdx.x; i < p.c.Hkv * rows * pieces; i += THREADS) {
      const int c = i % pieces, r = r0 + i / pieces % rows, h = i / pieces / rows;
      const long long orow = ((long long)b * p.c.Hkv + h) * p.R + r;
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + orow * p.D + c * 8) = make_uint4(0u, 0u, 0u, 0u);
      if (c == 0) p.lse[orow] = p.sink ? p.sink[h * p.G + r / p.Sq] : -INFINITY;
    }
  }
}

// A share's walk over its portions of segments, the same for every thread that makes it.
struct CachedPortion {
  int b, rt, kvh, j0, j1;  // units [j0, j1) of the segment
  CachedBounds s;
  int slot;                // part slot, or -1: the whole segment
};
template <bool ONE_TILE>
struct CachedWalk {
  int u, end, te, e;
  __device__ __forceinline__ bool next(const CachedParams& p, CachedPortion& w) {
    if (u >= end) return false;
    for (;;) {
      w.b = ONE_TILE ? e : e / p.n_rt;
      w.rt = ONE_TILE ? 0 : e - w.b * p.n_rt;
      w.s = cached_bounds(p, w.b, w.rt);
      const int n = w.s.n * p.c.Hkv;
      if (u < te + n) break;
      te += n;
      ++e;
    }
    const int off = u - te;
    w.kvh = off / w.s.n;
    w.j0 = off - w.kvh * w.s.n;
    w.j1 = min(w.s.n, w.j0 + (end - u));
    w.slot = w.j0 > 0 ? 0 : w.j1 < w.s.n ? 1 : -1;
    u += w.j1 - w.j0;
    return true;
  }
};

// The keys that row r sees: [lo, hi], and below F those up to hi.
struct CachedRow {
  int lo, hi, place;
};
__device__ __forceinline__ CachedRow cached_row(const CachedParams& p, const CachedBounds& s, int r) {
  const int i = r % p.Sq;
  CachedRow w;
  w.place = s.L - s.Lq + i;
  w.hi = p.causal ? min(w.place, s.L - 1) : s.L - 1;
  if (i >= s.Lq) w.hi = -1;
  w.lo = p.window_left >= 0 ? (int)max(0ll, (long long)w.place - p.window_left) : 0;
  return w;
}

// The page of keys [k, k + 16) of batch row b as the table has it, and the page or -1 (reported) if
// that is none: apart, so that a lookup made ahead is not waited for before its use.
__device__ __forceinline__ int cached_lookup(const CachedParams& p, int b, int k) {
  return __ldg(p.c.table + (long long)b * p.c.max_pages + (k >> p.c.page_shift));
}
__device__ __forceinline__ int cached_page(const CachedParams& p, int entry) {
  if ((unsigned)entry < (unsigned)p.c.n_pages) return entry;
  atomicOr(p.status, STATUS_PAGE);
  return -1;
}

// Named barrier over nthreads threads that tells all of them whether `pred` holds for any.
__device__ __forceinline__ bool named_bar_any(uint32_t id, uint32_t nthreads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %1, 0;\n\tbar.red.or.pred po, %2, %3, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(id), "r"(nthreads)
      : "memory");
  return r != 0;
}

// A sink joins the sum 2^lse2: returns log2 of the whole and the factor on O.
__device__ __forceinline__ float cached_with_sink(const CachedParams& p, int head, float lse2, float& factor) {
  factor = 1.f;
  if (p.sink == nullptr) return lse2;
  const float s2 = p.sink[head] * 1.4426950408889634f;
  if (s2 == -INFINITY) return lse2;
  if (lse2 == -INFINITY) {
    factor = 0.f;
    return s2;
  }
  const float m = fmaxf(lse2, s2), all = m + __log2f(ex2_approx(lse2 - m) + ex2_approx(s2 - m));
  factor = ex2_approx(lse2 - all);
  return all;
}

cudaError_t launch_cached_rows_16(const CachedParams& p, int nr, cudaStream_t s);
cudaError_t launch_cached_rows_8(const CachedParams& p, int nr, cudaStream_t s);
cudaError_t cached_rows_16_setup();
cudaError_t cached_rows_8_setup();
cudaError_t launch_cached_tiles_16(const CachedParams& p, cudaStream_t s);
cudaError_t launch_cached_tiles_8(const CachedParams& p, cudaStream_t s);
cudaError_t cached_tiles_16_setup();
cudaError_t cached_tiles_8_setup();
cudaError_t launch_cached_merge(const CachedParams& p, cudaStream_t s);

// Keys of a unit of the few-rows kernel with 8 nr rows, a warp's piece.
__host__ __device__ constexpr int cached_rows_tk(bool f8, int nr) { return f8 && nr <= 2 ? 32 : 16; }
// CTAs of it that an SM holds.
__host__ __device__ constexpr int cached_rows_ctas(int nr) { return nr <= 2 ? 3 : 2; }

}  // namespace sdpa

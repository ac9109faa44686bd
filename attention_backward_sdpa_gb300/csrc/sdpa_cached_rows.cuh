// sdpa_cached_rows.cuh -- attention over a paged cache for few rows a key/value head: generated tokens.
//
// Bound by memory: each key and value is read once for all query heads of its group, 2 D sizes
// of bytes for 4 D flops a row. So the work is to keep enough reads in flight and everything
// else out of their way.
//
//   - A warp is a share of its own and has nothing to do with the others: it walks its share's units, pieces of 16
//     keys (in 8 bits with 16 rows, 32), through a ring of stages that it fills by 16-byte asynchronous
//     copies and waits for by itself.
//     Rows of a piece that no query sees are filled with zeros, so that what a recycled page
//     holds never meets a product.
//   - Both products on m16n8k16 with the softmax in registers: up to 32 rows are what such a call has (G heads, one
//     token or a few), and 16 rows of P against 16 keys of V take 2 clocks where the keys' bytes take 180; a
//     128-row tcgen05 tile would stand empty to seven eighths. With 16-bit pages the time is then that of the reads
//     (6.7 to 6.9 TB/s over long sequences); over codes it is a warp's chain of instructions, 740 a piece of 32 keys
//     with 16 rows, which 12 warps an SM hide less than the reads (issue slots 48 % full at 115 us for
//     decode_batch_8bit). Up to 8 rows have products of their own, half of them (below): 102 us.
//   - The maximum is a lazy reference: it is raised, and O rescaled, only when some score exceeds
//     it by 2^8; one vote a piece asks for that.
//   - 8 bits: codes become fp16 in registers (exact), the queries are fp16 times a power of two a row (exact
//     down to 2^-29 of the row's largest), and P is fp16. A page's key scale joins the
//     score's factor. Its value scale joins the weight's exponent, w = 2^(x + log2(vs) - reference), so that
//     O = sum w * code / sum w / vs: the reference is the largest weighted value's, whatever the scales are.
//     The contraction index is free to be permuted, so a thread's 16-byte piece of a key serves four steps,
//     and byte pairs of V go through the 16-bit transposing load as they are.
//   - Over 16-bit pages a weight meets the values as two numbers of the cache's type, itself rounded and what that
//     leaves, off by 2^-16 (bf16) or 2^-22 (fp16) of it in all: the second product waits for the same bytes. 64
//     sequences of up to 8,192 keys, with it and without: 184 and 184 us with 4 rows a head, 199 and 196 with 16, 122 and 117
//     with 32 of 64 columns; O of 500 keys is then off by 1.62e-3, what rounding it to bf16 alone gives, against 1.82e-3.
//     Over codes P is fp16, off by 2^-12 of a weight on average, where a second product would cost what a piece waits for.
//     P in fp16 is taken times 2^6, so that what falls below its smallest step is below 2^-30 of the row's largest.
#pragma once

#include "cached.cuh"

namespace sdpa {

namespace cached_rows {

constexpr int WARPS = 4, THREADS = 128;
constexpr float RAISE = 8.f;

enum : int { BF16 = 0, F16 = 1, E4M3 = 2 };

template <int CT, int DP, int NR>
struct Layout {
  static constexpr int GROUPS = CT == E4M3 && NR <= 2 ? 2 : 1;  // of 16 keys
  static constexpr int KS = 16 * GROUPS;                // keys of a piece
  static constexpr int RB = DP * (CT == E4M3 ? 1 : 2);  // bytes of a row
  static constexpr int CH = RB / 16;
  static constexpr int SIDE = KS * RB;                  // keys or values of a piece
  static constexpr int STAGE = 2 * SIDE;
  // Three CTAs an SM with up to 16 rows, two with 32, by their registers; what shared memory that leaves is stages.
  static constexpr int CTAS = cached_rows_ctas(NR);
  static constexpr int NST_FIT = (CTAS == 3 ? 2 : 3) * 8192 / STAGE, NST = NST_FIT < 6 ? NST_FIT : 6;
  static constexpr int META = 32;                       // {ks, ks, vs, vs, page bits}
  static constexpr int TR = 8 * NR;
  static constexpr int RING = NST * (STAGE + META);     // of a warp
  static constexpr int BYTES = WARPS * RING;
  static_assert(NST >= 2 && KS == cached_rows_tk(CT == E4M3, NR), "");
};

// 16-byte piece c of row r: rows of a piece lie on different banks for the eight rows of a
// matrix load, and neighbouring rows in different halves for 16-byte loads.
template <int CH>
__device__ __forceinline__ int phys(int r, int c) {
  if constexpr (CH == 4) return c ^ ((r >> 1) & 3);
  else return c ^ (((r & 1) << 2) | ((r >> 1) & 3));
}
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
// c += a (16 x 16) * b (16 x 8).
template <bool F>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  if constexpr (F)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
template <bool F>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  const uint32_t b[2] = {b0, b1};
  mma<F>(c, a, b);
}
// An 8 x 8 matrix of 16-bit elements, two neighbours of a row a lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Four codes as two fp16 pairs, exact.
__device__ __forceinline__ void codes_f16(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(four));
}

// NR: tiles of 8 rows. CT: type of the cache; IOF: the queries and O are fp16 (a 16-bit cache has their type). MOD: capped or
// distance-biased scores. FULL: D is DP, so that rows and copies lie at fixed distances.
template <int CT, bool IOF, int DP, int NR, bool MOD, bool FULL>
__global__ void __launch_bounds__(THREADS, Layout<CT, DP, NR>::CTAS) cached_rows_kernel(const CachedParams p) {
  using L = Layout<CT, DP, NR>;
  constexpr bool PF = CT != BF16;  // the products are fp16
  constexpr float BIAS = PF ? 6.f : 0.f;
  constexpr int KD = DP / 16, ESZ = CT == E4M3 ? 1 : 2;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ CachedStart sh_start[WARPS];
  __shared__ int sh_sum[WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (!FULL && p.D < DP)  // columns past D are never copied
    for (int i = tid; i < L::BYTES / 16; i += THREADS) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  int total;
  const CachedStart st = cached_start<THREADS, WARPS>(p, sh_start, sh_sum, total);
  cached_empty_rows<THREADS, true>(p);
  if (st.begin >= st.end) return;
  const int share = blockIdx.x * WARPS + warp;
  const uint32_t ring = smem_u32(smem) + warp * L::RING;
  const int copy_row = lane / L::CH, copy_c = lane % L::CH;
  const int D = FULL ? DP : p.D;
  const bool copy_in = FULL || copy_c * 16 < D * ESZ;
  const int row_bytes = D * ESZ;
  // A lane's place in rows copy_row + i * PASS of a group: the swizzle alternates from pass to pass at most.
  constexpr int PASS = 32 / L::CH;
  const uint32_t place[2] = {(uint32_t)(copy_row * L::RB + phys<L::CH>(copy_row, copy_c) * 16),
                             (uint32_t)(copy_row * L::RB + phys<L::CH>(copy_row + PASS, copy_c) * 16)};

  auto place_of = [&](int i) -> uint32_t {
    // (16 rows of CH pieces: PASS 2, 4 or 8; the swizzle repeats after 8 rows, and with CH 4 after 8 as well)
    const int x = (i * PASS) & 7;
    if (x == 0) return place[0] + i * PASS * L::RB;
    if (PASS == 4) return place[1] + i * PASS * L::RB;
    const int r = copy_row + i * PASS;
    return r * L::RB + phys<L::CH>(r, copy_c) * 16;
  };
  CachedWalk<true> walk{st.begin, st.end, st.te, st.e};
  CachedPortion w;
  while (walk.next(p, w)) {
    const CachedBounds& s = w.s;
    if (w.j0 == 0 && lane == 0) {  // the segment's first share
      int4 cut = make_int4(-1, 0, 0, 0);
      const int seg = (w.b * p.n_rt + w.rt) * p.c.Hkv + w.kvh;
      if (w.slot >= 0) cut = make_int4(seg, share, CachedShares(p, total).of(walk.u - w.j1 + s.n - 1), 0);
      p.cuts[seg] = cut;
    }
    auto group_seen = [&](int a) { return a < s.k_hi && (a + 15 >= s.k_lo || a < p.first_keys); };
    int next_entry[L::GROUPS];
    auto find_pages = [&](int j) {
      if (j >= w.j1) return;
      const int k0 = cached_tile(s, j) * L::KS;
#pragma unroll
      for (int u = 0; u < L::GROUPS; ++u)
        if (group_seen(k0 + 16 * u)) next_entry[u] = cached_lookup(p, w.b, k0 + 16 * u);
    };
    auto issue = [&](int j, int stage) {
      if (j < w.j1) {
        const uint32_t to = ring + stage * (L::STAGE + L::META), meta = to + L::STAGE;
        const int k0 = cached_tile(s, j) * L::KS;
        uint32_t ok = 0;
#pragma unroll
        for (int u = 0; u < L::GROUPS; ++u) {
          const int a = k0 + 16 * u, page = group_seen(a) ? cached_page(p, next_entry[u]) : -1;
          if (page >= 0) ok |= 1u << u;
          const bool all = page >= 0 && a <= s.k_hi - 16 && (a >= s.k_lo || a <= p.first_keys - 16);
          const long long head = (long long)max(page, 0) * p.c.Hkv + w.kvh;
          const long long at = ((head << p.c.page_shift) + (a & (p.c.page - 1)) + copy_row) * row_bytes + copy_c * 16;
          const char* kb = static_cast<const char*>(p.c.k) + at;
          const char* vb = static_cast<const char*>(p.c.v) + at;
          if (copy_in) {
            const uint32_t dst = to + 16 * u * L::RB;
            if (all) {
#pragma unroll
              for (int i = 0; i < 16 / PASS; ++i) {
                copy16(dst + place_of(i), kb + i * PASS * row_bytes, true);
                copy16(dst + L::SIDE + place_of(i), vb + i * PASS * row_bytes, true);
              }
            } else {  // rows that no query sees: zeros
#pragma unroll 1
              for (int i = 0; i < 16 / PASS; ++i) {
                const int r = copy_row + i * PASS, key = a + r;
                const bool take = page >= 0 && key < s.k_hi && (key >= s.k_lo || key < p.first_keys);
                const uint32_t at = dst + r * L::RB + phys<L::CH>(r, copy_c) * 16;
                copy16(at, take ? kb + i * PASS * row_bytes : static_cast<const char*>(p.c.k), take);
                copy16(at + L::SIDE, take ? vb + i * PASS * row_bytes : static_cast<const char*>(p.c.v), take);
              }
            }
          }
          if constexpr (CT == E4M3) {
            if (lane < 2) {
              if (page >= 0) copy4(meta + (2 * lane + u) * 4, (lane ? p.c.vs : p.c.ks) + head);
              else asm volatile("st.shared.f32 [%0], %1;" ::"r"(meta + (2 * lane + u) * 4), "f"(1.f) : "memory");
            }
          }
        }
        if (lane == 0) asm volatile("st.shared.b32 [%0], %1;" ::"r"(meta + 16), "r"(ok) : "memory");
      }
      copies_commit();
      find_pages(j + 1);
    };
    find_pages(w.j0);
#pragma unroll 1
    for (int i = 0; i < L::NST - 1; ++i) issue(w.j0 + i, i);

    if constexpr (NR == 1) {
      // Up to 8 rows a key/value head are the columns of the products' tiles, S^T = K Q^T and O^T += V^T P^T: the keys, and
      // the values' columns, fill the tiles' 16 rows. Against 16 rows there (below) that is half the products, scores
      // and accumulators: 111 -> 102 us for decode_batch_8bit (64 sequences of up to 8,192 keys, 4 rows a head).
      // Queries as B fragments: row g.
      uint32_t qf[KD][2];
      float back = 1.f;  // the row's score is its product times this
      {
        const bool in = g < p.R;
        const uint16_t* const q = static_cast<const uint16_t*>(p.q) + (((long long)w.b * p.c.Hkv + w.kvh) * p.R + g) * D;
        float amax = 0.f;
#pragma unroll
        for (int kd = 0; kd < KD; ++kd) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int d = CT == E4M3 ? 64 * (kd >> 2) + 16 * t + 4 * (kd & 3) + 2 * i : 16 * kd + 2 * t + 8 * i;
            qf[kd][i] = in && d < D ? *reinterpret_cast<const uint32_t*>(q + d) : 0u;
            if constexpr (CT == E4M3 && !IOF)
              amax = fmaxf(amax, fmaxf(fabsf(io_lo<false>(qf[kd][i])), fabsf(io_hi<false>(qf[kd][i]))));
          }
        }
        if constexpr (CT == E4M3 && !IOF) {
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          // 2^e brings the row's largest into [2^14, 2^15).
          const int e = amax > 0.f ? min(max(14 - ((int)(__float_as_uint(amax) >> 23) - 127), -113), 126) : 0;
          const float up = __uint_as_float((uint32_t)(127 + e) << 23);
          back = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
          for (int kd = 0; kd < KD; ++kd)
#pragma unroll
            for (int i = 0; i < 2; ++i) qf[kd][i] = pack_f16x2(io_lo<false>(qf[kd][i]) * up, io_hi<false>(qf[kd][i]) * up);
        }
      }
      // The state of this thread's rows of the scores, 2 t and 2 t + 1.
      float xmul[2], m[2], l[2], slope2[2];
      CachedRow rows[2];
      int lo_max = 0, hi_min = INT_MAX;
#pragma unroll
      for (int ri = 0; ri < 2; ++ri) {
        const int r = 2 * t + ri;
        const bool in = r < p.R;
        xmul[ri] = CT == E4M3 && !IOF ? __shfl_sync(0xffffffffu, back, 4 * r) : 1.f;
        if constexpr (!MOD) xmul[ri] *= p.scale_log2;
        rows[ri] = cached_row(p, s, r);
        if (!in) rows[ri].lo = 0, rows[ri].hi = s.L - 1;  // (not written; never the reason for a mask)
        lo_max = max(lo_max, rows[ri].lo);
        hi_min = min(hi_min, rows[ri].hi);
        slope2[ri] = MOD && p.mods.slopes && in ? p.mods.slopes[w.kvh * p.G + r / p.Sq] * 1.4426950408889634f : 0.f;
        m[ri] = -INFINITY;
        l[ri] = 0.f;
      }
      lo_max = __reduce_max_sync(0xffffffffu, lo_max);
      hi_min = __reduce_min_sync(0xffffffffu, hi_min);
      // O^T: element [i][e] is row 2 t + (e & 1), column 16 i + g + 8 (e >> 1), over codes 16 i + 2 g + (e >> 1).
      float o[KD][4];
#pragma unroll
      for (int i = 0; i < KD; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

      int stage = 0;
#pragma unroll 1
      for (int j = w.j0; j < w.j1; ++j) {
        copies_wait<L::NST - 2>();
        __syncwarp();  // every lane's copies of this stage have landed, and all are done with the one before
        issue(j + L::NST - 1, stage == 0 ? L::NST - 1 : stage - 1);
        const uint32_t at = ring + stage * (L::STAGE + L::META), meta = at + L::STAGE;
        if (++stage == L::NST) stage = 0;
        const int k0 = cached_tile(s, j) * L::KS;
        uint32_t ok;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(ok) : "r"(meta + 16) : "memory");
        if (ok == 0u) continue;
        const uint32_t sk = at, sv = at + L::SIDE;
        // ---- S^T = K Q^T: element [u][e]: key 16 u + g + 8 (e >> 1), row 2 t + (e & 1)
        // (in two sums each: half the chain of products)
        float sc[L::GROUPS][4], odd[L::GROUPS][4];
#pragma unroll
        for (int u = 0; u < L::GROUPS; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[u][e] = odd[u][e] = 0.f;
        if constexpr (CT == E4M3) {
#pragma unroll
          for (int h = 0; h < DP / 64; ++h) {
            uint4 v[2 * L::GROUPS];
#pragma unroll
            for (int n = 0; n < 2 * L::GROUPS; ++n) v[n] = lds16(sk + (8 * n + g) * L::RB + phys<L::CH>(8 * n + g, 4 * h + t) * 16);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj)
#pragma unroll
              for (int u = 0; u < L::GROUPS; ++u) {
                const uint4 &v0 = v[2 * u], &v1 = v[2 * u + 1];
                uint32_t a[4];
                codes_f16(jj == 0 ? v0.x : jj == 1 ? v0.y : jj == 2 ? v0.z : v0.w, a[0], a[2]);
                codes_f16(jj == 0 ? v1.x : jj == 1 ? v1.y : jj == 2 ? v1.z : v1.w, a[1], a[3]);
                mma<PF>(jj & 1 ? odd[u] : sc[u], a, qf[4 * h + jj]);
              }
          }
        } else {
          const int r = lane & 15, c = lane >> 4;
#pragma unroll
          for (int kd = 0; kd < KD; ++kd) {
            uint32_t a[4];
            ldm4(a, sk + r * L::RB + phys<L::CH>(r, 2 * kd + c) * 16);
            mma<PF>(kd & 1 ? odd[0] : sc[0], a, qf[kd]);
          }
        }
#pragma unroll
        for (int u = 0; u < L::GROUPS; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[u][e] += odd[u][e];
        // ---- scores in log2 units, masked
        // (unmodified ones stay as they are: their factor fx is part of the exponent)
        float lvs[L::GROUPS], inv_vs[L::GROUPS], fx[2][L::GROUPS];
#pragma unroll
        for (int u = 0; u < L::GROUPS; ++u) {
          lvs[u] = 0.f;
          inv_vs[u] = 1.f;
          float ks = 1.f;
          if constexpr (CT == E4M3) {
            float vs;
            asm volatile("ld.shared.b32 %0, [%1];" : "=f"(ks) : "r"(meta + u * 4) : "memory");
            asm volatile("ld.shared.b32 %0, [%1];" : "=f"(vs) : "r"(meta + 8 + u * 4) : "memory");
            lvs[u] = __log2f(vs);
            inv_vs[u] = __fdividef(1.f, vs);
          }
#pragma unroll
          for (int ri = 0; ri < 2; ++ri) {
            fx[ri][u] = fmaxf(xmul[ri] * ks, 1e-38f);  // (positive: a masked score stays -inf)
            if constexpr (MOD) {
              sc[u][ri] *= fx[ri][u];
              sc[u][2 + ri] *= fx[ri][u];
              fx[ri][u] = 1.f;
            }
          }
        }
        if constexpr (MOD) {
          const bool cap = p.mods.cap_in != 0.f;
          const float c = cap ? p.mods.cap_log2 : p.scale_log2;
          uint64_t y[2 * L::GROUPS];  // a key's two rows
#pragma unroll
          for (int i = 0; i < 2 * L::GROUPS; ++i) y[i] = f2_pack(sc[i >> 1][2 * (i & 1)], sc[i >> 1][2 * (i & 1) + 1]);
          if (cap) tanh2_any(y, p.mods.cap_in);
#pragma unroll
          for (int i = 0; i < 2 * L::GROUPS; ++i) {
            const int key = k0 + 8 * i + g;
            float x0, x1;
            f2_unpack(y[i], x0, x1);
            sc[i >> 1][2 * (i & 1)] = fmaf(-slope2[0], fabsf((float)(rows[0].place - key)), x0 * c);
            sc[i >> 1][2 * (i & 1) + 1] = fmaf(-slope2[1], fabsf((float)(rows[1].place - key)), x1 * c);
          }
        }
        constexpr uint32_t ALL = (1u << L::GROUPS) - 1u;
        if (!(ok == ALL && k0 + L::KS - 1 <= hi_min && (k0 >= lo_max || k0 <= p.first_keys - L::KS))) {
#pragma unroll
          for (int ri = 0; ri < 2; ++ri)
#pragma unroll
            for (int i = 0; i < 2 * L::GROUPS; ++i) {
              const int key = k0 + 8 * i + g;
              if (key > rows[ri].hi || (key < rows[ri].lo && key >= p.first_keys) || !((ok >> (i >> 1)) & 1u))
                sc[i >> 1][2 * (i & 1) + ri] = -INFINITY;
            }
        }
        // ---- the reference
        bool raise = false;
        float mx[2];
#pragma unroll
        for (int ri = 0; ri < 2; ++ri) {
          mx[ri] = -INFINITY;
#pragma unroll
          for (int u = 0; u < L::GROUPS; ++u) mx[ri] = fmaxf(mx[ri], fmaf(fmaxf(sc[u][ri], sc[u][2 + ri]), fx[ri][u], lvs[u]));
          raise |= mx[ri] > m[ri] + RAISE;
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int ri = 0; ri < 2; ++ri) {
            float v = mx[ri];
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, k));
            float fo = 1.f;
            if (v > m[ri] + RAISE) {
              fo = ex2_approx(m[ri] - v);  // 0 for the first key
              l[ri] *= fo;
              m[ri] = v;
            }
#pragma unroll
            for (int i = 0; i < KD; ++i) {
              o[i][ri] *= fo;
              o[i][2 + ri] *= fo;
            }
          }
        }
        // ---- P^T, transposed by eights into B fragments (16 bits: and what its rounding leaves)
        uint32_t pf[L::GROUPS][2];
        [[maybe_unused]] uint32_t rest[2];
        const float neg0 = m[0] == -INFINITY ? 0.f : BIAS - m[0], neg1 = m[1] == -INFINITY ? 0.f : BIAS - m[1];
#pragma unroll
        for (int u = 0; u < L::GROUPS; ++u) {
          const float n0 = neg0 + lvs[u], n1 = neg1 + lvs[u];
          const float p0 = ex2_approx(fmaf(sc[u][0], fx[0][u], n0)), p1 = ex2_approx(fmaf(sc[u][1], fx[1][u], n1));
          const float p2 = ex2_approx(fmaf(sc[u][2], fx[0][u], n0)), p3 = ex2_approx(fmaf(sc[u][3], fx[1][u], n1));
          const uint32_t h0 = pack_io2<PF>(p0, p1), h1 = pack_io2<PF>(p2, p3);
          pf[u][0] = transposed(h0);
          pf[u][1] = transposed(h1);
          if constexpr (CT != E4M3) {
            rest[0] = transposed(pack_io2<PF>(p0 - io_lo<PF>(h0), p1 - io_hi<PF>(h0)));
            rest[1] = transposed(pack_io2<PF>(p2 - io_lo<PF>(h1), p3 - io_hi<PF>(h1)));
          }
          l[0] = CT == E4M3 ? fmaf(p0 + p2, inv_vs[u], l[0]) : l[0] + (p0 + p2);
          l[1] = CT == E4M3 ? fmaf(p1 + p3, inv_vs[u], l[1]) : l[1] + (p1 + p3);
        }
        // ---- O^T += V^T P^T
        if constexpr (CT == E4M3) {
          const int r = (lane & 7) + (((lane >> 3) & 1) << 3), c = lane >> 4;
#pragma unroll
          for (int i = 0; i < KD; i += 2)
#pragma unroll
            for (int u = 0; u < L::GROUPS; ++u) {
              uint32_t b[4], a0[4], a1[4];
              ldm4t(b, sv + (16 * u + r) * L::RB + phys<L::CH>(16 * u + r, i + c) * 16);
              // A word has two columns of two keys: as a pair of keys of either column.
              codes_f16(__byte_perm(b[0], 0u, 0x3120), a0[0], a0[1]);
              codes_f16(__byte_perm(b[1], 0u, 0x3120), a0[2], a0[3]);
              codes_f16(__byte_perm(b[2], 0u, 0x3120), a1[0], a1[1]);
              codes_f16(__byte_perm(b[3], 0u, 0x3120), a1[2], a1[3]);
              mma<true>(o[i], a0, pf[u]);
              mma<true>(o[i + 1], a1, pf[u]);
            }
        } else {
          const int r = (lane & 7) + ((lane >> 4) << 3), c = (lane >> 3) & 1;
#pragma unroll
          for (int i = 0; i < KD; ++i) {
            uint32_t a[4];
            ldm4t(a, sv + r * L::RB + phys<L::CH>(r, 2 * i + c) * 16);
            mma<PF>(o[i], a, pf[0]);
            mma<PF>(o[i], a, rest);
          }
        }
      }

      // ---- the portion's rows as results, or as a part
      copies_wait<0>();
      __syncwarp();  // (and the ring is free for the next portion)
      const int b = w.b, kvh = w.kvh, slot = w.slot;
#pragma unroll
      for (int ri = 0; ri < 2; ++ri) {
        float lt = l[ri];
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, k);
        const int r = 2 * t + ri;
        if (r >= p.R) continue;
        const bool none = m[ri] == -INFINITY;
        float f = none ? 0.f : 1.f / lt;
        const float lse2 = none ? -INFINITY : m[ri] - BIAS + __log2f(lt);
        const long long part = ((long long)share * 2 + slot) * p.part_rows + r;
        const long long orow = ((long long)b * p.c.Hkv + kvh) * p.R + r;
        if (slot >= 0) {
          if (g == 0) p.part_lse[part] = lse2;
        } else {
          float fs;
          const float all = cached_with_sink(p, kvh * p.G + r / p.Sq, lse2, fs);
          f *= fs;
          if (g == 0) p.lse[orow] = all * 0.6931471805599453f;
        }
#pragma unroll
        for (int i = 0; i < KD; ++i) {
          if (16 * i >= D) continue;
          const float y0 = o[i][ri] * f, y1 = o[i][2 + ri] * f;
          if constexpr (CT == E4M3) {
            const int d = 16 * i + 2 * g;
            if (slot >= 0) *reinterpret_cast<float2*>(p.part_o + part * D + d) = make_float2(y0, y1);
            else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + orow * D + d) = pack_io2<IOF>(y0, y1);
          } else {
            const int d = 16 * i + g;
            if (slot >= 0) {
              p.part_o[part * D + d] = y0;
              p.part_o[part * D + d + 8] = y1;
            } else {
              const uint32_t both = pack_io2<IOF>(y0, y1);
              static_cast<uint16_t*>(p.o)[orow * D + d] = (uint16_t)both;
              static_cast<uint16_t*>(p.o)[orow * D + d + 8] = (uint16_t)(both >> 16);
            }
          }
        }
      }
    } else {
      // 16 MT rows are the tiles' rows, S = Q K^T and O += P V: P becomes an A fragment where it is. (Two tiles of 8 in
      // the form above take 154 us where one of 16 takes 127, the same batch with 16 rows a head; of 64 columns 81
      // against 75.)
      constexpr int MT = NR / 2, NT = DP / 8;
      const int r0 = w.rt * L::TR;
      // Queries as A fragments, and the rows' state. Thread rows: 16 m + g and 16 m + g + 8.
      uint32_t qf[MT][KD][4];
      float xmul[2 * MT], m[2 * MT], l[2 * MT], slope2[MOD ? 2 * MT : 1];
      CachedRow rows[2 * MT];
      int lo_max = 0, hi_min = INT_MAX;
#pragma unroll
      for (int ri = 0; ri < 2 * MT; ++ri) {
        const int mt = ri >> 1, half = ri & 1, r = r0 + 16 * mt + g + 8 * half;
        const bool in = r < p.R;
        const uint16_t* const q = static_cast<const uint16_t*>(p.q) + (((long long)w.b * p.c.Hkv + w.kvh) * p.R + r) * D;
        float amax = 0.f;
#pragma unroll
        for (int kd = 0; kd < KD; ++kd) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int d = CT == E4M3 ? 64 * (kd >> 2) + 16 * t + 4 * (kd & 3) + 2 * x : 16 * kd + 2 * t + 8 * x;
            uint32_t v = 0u;
            if (in && d < D) v = *reinterpret_cast<const uint32_t*>(q + d);
            qf[mt][kd][half + 2 * x] = v;
            if constexpr (CT == E4M3 && !IOF) amax = fmaxf(amax, fmaxf(fabsf(io_lo<false>(v)), fabsf(io_hi<false>(v))));
          }
        }
        xmul[ri] = 1.f;
        if constexpr (CT == E4M3 && !IOF) {
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          // 2^e brings the row's largest into [2^14, 2^15).
          const int e = amax > 0.f ? min(max(14 - ((int)(__float_as_uint(amax) >> 23) - 127), -113), 126) : 0;
          const float up = __uint_as_float((uint32_t)(127 + e) << 23);
          xmul[ri] = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
          for (int kd = 0; kd < KD; ++kd)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t& v = qf[mt][kd][half + 2 * x];
              v = pack_f16x2(io_lo<false>(v) * up, io_hi<false>(v) * up);
            }
        }
        if constexpr (!MOD) xmul[ri] *= p.scale_log2;
        rows[ri] = cached_row(p, s, r);
        if (!in) rows[ri].lo = 0, rows[ri].hi = s.L - 1;  // (not written; never the reason for a mask)
        lo_max = max(lo_max, rows[ri].lo);
        hi_min = min(hi_min, rows[ri].hi);
        if constexpr (MOD)
          slope2[ri] = p.mods.slopes && in ? p.mods.slopes[w.kvh * p.G + r / p.Sq] * 1.4426950408889634f : 0.f;
        m[ri] = -INFINITY;
        l[ri] = 0.f;
      }
      lo_max = __reduce_max_sync(0xffffffffu, lo_max);
      hi_min = __reduce_min_sync(0xffffffffu, hi_min);
      float o[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;

      int stage = 0;
#pragma unroll 1
      for (int j = w.j0; j < w.j1; ++j) {
        copies_wait<L::NST - 2>();
        __syncwarp();  // every lane's copies of this stage have landed, and all are done with the one before
        issue(j + L::NST - 1, stage == 0 ? L::NST - 1 : stage - 1);
        const uint32_t at = ring + stage * (L::STAGE + L::META), meta = at + L::STAGE;
        if (++stage == L::NST) stage = 0;
        const int k0 = cached_tile(s, j) * L::KS;
        uint32_t ok;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(ok) : "r"(meta + 16) : "memory");
        if (ok == 0u) continue;
        constexpr int KT = 2 * L::GROUPS;  // tiles of 8 keys
        const uint32_t sk = at, sv = at + L::SIDE;
        // ---- S = Q K^T: element [mt][n][e]: row g + 8 (e >> 1), key 8 n + 2 t + (e & 1)
        float sc[MT][KT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < KT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[mt][n][e] = 0.f;
        if constexpr (CT == E4M3) {
#pragma unroll
          for (int h = 0; h < DP / 64; ++h) {
            uint4 v[KT];
#pragma unroll
            for (int n = 0; n < KT; ++n) v[n] = lds16(sk + (8 * n + g) * L::RB + phys<L::CH>(8 * n + g, 4 * h + t) * 16);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj)
#pragma unroll
              for (int n = 0; n < KT; ++n) {
                uint32_t b0, b1;
                codes_f16(jj == 0 ? v[n].x : jj == 1 ? v[n].y : jj == 2 ? v[n].z : v[n].w, b0, b1);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) mma<true>(sc[mt][n], qf[mt][4 * h + jj], b0, b1);
              }
          }
        } else {
          const int r = (lane & 7) + ((lane >> 4) << 3), c = (lane >> 3) & 1;
#pragma unroll
          for (int kd = 0; kd < KD; ++kd) {
            uint32_t b[4];
            ldm4(b, sk + r * L::RB + phys<L::CH>(r, 2 * kd + c) * 16);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma<PF>(sc[mt][0], qf[mt][kd], b[0], b[1]);
              mma<PF>(sc[mt][1], qf[mt][kd], b[2], b[3]);
            }
          }
        }
        // ---- scores in log2 units, masked
        // (unmodified ones stay as they are: their factor fx is part of the exponent)
        float lvs[L::GROUPS], inv_vs[L::GROUPS], fx[2 * MT][L::GROUPS];
#pragma unroll
        for (int u = 0; u < L::GROUPS; ++u) {
          lvs[u] = 0.f;
          inv_vs[u] = 1.f;
          float ks = 1.f;
          if constexpr (CT == E4M3) {
            float vs;
            asm volatile("ld.shared.b32 %0, [%1];" : "=f"(ks) : "r"(meta + u * 4) : "memory");
            asm volatile("ld.shared.b32 %0, [%1];" : "=f"(vs) : "r"(meta + 8 + u * 4) : "memory");
            lvs[u] = __log2f(vs);
            inv_vs[u] = __fdividef(1.f, vs);
          }
#pragma unroll
          for (int ri = 0; ri < 2 * MT; ++ri) {
            fx[ri][u] = fmaxf(xmul[ri] * ks, 1e-38f);  // (positive: a masked score stays -inf)
            if constexpr (MOD) {
#pragma unroll
              for (int n = 2 * u; n < 2 * u + 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) sc[ri >> 1][n][2 * (ri & 1) + e] *= fx[ri][u];
              fx[ri][u] = 1.f;
            }
          }
        }
        if constexpr (MOD) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int u = 0; u < L::GROUPS; ++u) {
              uint64_t x[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                x[i] = f2_pack(sc[mt][2 * u + (i >> 1)][2 * (i & 1)], sc[mt][2 * u + (i >> 1)][2 * (i & 1) + 1]);
              const bool cap = p.mods.cap_in != 0.f;
              if (cap) tanh2_any(x, p.mods.cap_in);
              const float c = cap ? p.mods.cap_log2 : p.scale_log2;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float x0, x1;
                f2_unpack(x[i], x0, x1);
                const int ri = 2 * mt + (i & 1), n = 2 * u + (i >> 1), key = k0 + 8 * n + 2 * t;
                sc[mt][n][2 * (i & 1)] = fmaf(-slope2[ri], fabsf((float)(rows[ri].place - key)), x0 * c);
                sc[mt][n][2 * (i & 1) + 1] = fmaf(-slope2[ri], fabsf((float)(rows[ri].place - key - 1)), x1 * c);
              }
            }
        }
        constexpr uint32_t ALL = (1u << L::GROUPS) - 1u;
        if (!(ok == ALL && k0 + L::KS - 1 <= hi_min && (k0 >= lo_max || k0 <= p.first_keys - L::KS))) {
#pragma unroll
          for (int ri = 0; ri < 2 * MT; ++ri)
#pragma unroll
            for (int n = 0; n < KT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int key = k0 + 8 * n + 2 * t + e;
                if (key > rows[ri].hi || (key < rows[ri].lo && key >= p.first_keys) || !((ok >> (n >> 1)) & 1u))
                  sc[ri >> 1][n][2 * (ri & 1) + e] = -INFINITY;
              }
        }
        // ---- the reference
        bool raise = false;
        float mx[2 * MT];
#pragma unroll
        for (int ri = 0; ri < 2 * MT; ++ri) {
          const int e = 2 * (ri & 1);
          mx[ri] = -INFINITY;
#pragma unroll
          for (int u = 0; u < L::GROUPS; ++u) {
            const float(&a)[KT][4] = sc[ri >> 1];
            mx[ri] = fmaxf(mx[ri], fmaf(fmaxf(fmaxf(a[2 * u][e], a[2 * u][e + 1]), fmaxf(a[2 * u + 1][e], a[2 * u + 1][e + 1])), fx[ri][u], lvs[u]));
          }
          raise |= mx[ri] > m[ri] + RAISE;
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int ri = 0; ri < 2 * MT; ++ri) {
            float x = fmaxf(mx[ri], __shfl_xor_sync(0xffffffffu, mx[ri], 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            float fo = 1.f;
            if (x > m[ri] + RAISE) {
              fo = ex2_approx(m[ri] - x);  // 0 for the first key
              l[ri] *= fo;
              m[ri] = x;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              o[ri >> 1][n][2 * (ri & 1)] *= fo;
              o[ri >> 1][n][2 * (ri & 1) + 1] *= fo;
            }
          }
        }
        // ---- P, as A fragments (16 bits: and what its rounding leaves)
        uint32_t pf[MT][L::GROUPS][4];
        [[maybe_unused]] uint32_t rest[MT][4];
#pragma unroll
        for (int ri = 0; ri < 2 * MT; ++ri) {
          const float neg = m[ri] == -INFINITY ? 0.f : BIAS - m[ri];
#pragma unroll
          for (int u = 0; u < L::GROUPS; ++u) {
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const float x0 = sc[ri >> 1][2 * u + n][2 * (ri & 1)], x1 = sc[ri >> 1][2 * u + n][2 * (ri & 1) + 1];
              const float p0 = ex2_approx(fmaf(x0, fx[ri][u], neg + lvs[u])), p1 = ex2_approx(fmaf(x1, fx[ri][u], neg + lvs[u]));
              sum += p0 + p1;
              const uint32_t h = pack_io2<PF>(p0, p1);
              pf[ri >> 1][u][(ri & 1) + 2 * n] = h;
              if constexpr (CT != E4M3) rest[ri >> 1][(ri & 1) + 2 * n] = pack_io2<PF>(p0 - io_lo<PF>(h), p1 - io_hi<PF>(h));
            }
            l[ri] = CT == E4M3 ? fmaf(sum, inv_vs[u], l[ri]) : l[ri] + sum;
          }
        }
        // ---- O += P V
        {
          const int r = (lane & 7) + (((lane >> 3) & 1) << 3), c = lane >> 4;
          if constexpr (CT == E4M3) {
#pragma unroll
            for (int cp = 0; cp < DP / 32; ++cp)
#pragma unroll
              for (int u = 0; u < L::GROUPS; ++u) {
                uint32_t b[4], ev[4], od[4];
                ldm4t(b, sv + (16 * u + r) * L::RB + phys<L::CH>(16 * u + r, 2 * cp + c) * 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) codes_f16(__byte_perm(b[i], 0u, 0x3120), ev[i], od[i]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  mma<true>(o[mt][4 * cp], pf[mt][u], ev[0], ev[1]);
                  mma<true>(o[mt][4 * cp + 1], pf[mt][u], od[0], od[1]);
                  mma<true>(o[mt][4 * cp + 2], pf[mt][u], ev[2], ev[3]);
                  mma<true>(o[mt][4 * cp + 3], pf[mt][u], od[2], od[3]);
                }
              }
          } else {
#pragma unroll
            for (int dn = 0; dn < KD; ++dn) {
              uint32_t b[4];
              ldm4t(b, sv + r * L::RB + phys<L::CH>(r, 2 * dn + c) * 16);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma<PF>(o[mt][2 * dn], pf[mt][0], b[0], b[1]);
                mma<PF>(o[mt][2 * dn + 1], pf[mt][0], b[2], b[3]);
                mma<PF>(o[mt][2 * dn], rest[mt], b[0], b[1]);
                mma<PF>(o[mt][2 * dn + 1], rest[mt], b[2], b[3]);
              }
            }
          }
        }
      }

      // ---- the portion's rows as results, or as a part
      copies_wait<0>();
      __syncwarp();  // (and the ring is free for the next portion)
      const int b = w.b, kvh = w.kvh, slot = w.slot;
#pragma unroll
      for (int ri = 0; ri < 2 * MT; ++ri) {
        float lt = l[ri] + __shfl_xor_sync(0xffffffffu, l[ri], 1);
        lt += __shfl_xor_sync(0xffffffffu, lt, 2);
        const int row = 16 * (ri >> 1) + g + 8 * (ri & 1), r = r0 + row;
        if (r >= p.R) continue;
        const bool none = m[ri] == -INFINITY;
        float f = none ? 0.f : 1.f / lt;
        const float lse2 = none ? -INFINITY : m[ri] - BIAS + __log2f(lt);
        const long long part = ((long long)share * 2 + slot) * p.part_rows + row;
        const long long orow = ((long long)b * p.c.Hkv + kvh) * p.R + r;
        if (slot >= 0) {
          if (t == 0) p.part_lse[part] = lse2;
        } else {
          float fs;
          const float all = cached_with_sink(p, kvh * p.G + r / p.Sq, lse2, fs);
          f *= fs;
          if (t == 0) p.lse[orow] = all * 0.6931471805599453f;
        }
        const int e = 2 * (ri & 1);
        if constexpr (CT == E4M3) {  // tiles 2 n, 2 n + 1 hold the even and odd columns of 16-column piece n
#pragma unroll
          for (int n = 0; n < DP / 16; ++n) {
            if (16 * n >= D) continue;
            const float(&ev)[4] = o[ri >> 1][2 * n], (&od)[4] = o[ri >> 1][2 * n + 1];
            const float y0 = ev[e] * f, y1 = od[e] * f, y2 = ev[e + 1] * f, y3 = od[e + 1] * f;
            const int d = 16 * n + 4 * t;
            if (slot >= 0) *reinterpret_cast<float4*>(p.part_o + part * D + d) = make_float4(y0, y1, y2, y3);
            else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + orow * D + d) = make_uint2(pack_io2<IOF>(y0, y1), pack_io2<IOF>(y2, y3));
          }
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (8 * n >= D) continue;
            const float y0 = o[ri >> 1][n][e] * f, y1 = o[ri >> 1][n][e + 1] * f;
            const int d = 8 * n + 2 * t;
            if (slot >= 0) *reinterpret_cast<float2*>(p.part_o + part * D + d) = make_float2(y0, y1);
            else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + orow * D + d) = pack_io2<IOF>(y0, y1);
          }
        }
      }
    }
  }
}

template <int CT, bool IOF, int DP, int NR>
cudaError_t setup_one() {
  cudaError_t e = cudaSuccess;
  for (auto* k : {cached_rows_kernel<CT, IOF, DP, NR, false, true>, cached_rows_kernel<CT, IOF, DP, NR, false, false>,
                  cached_rows_kernel<CT, IOF, DP, NR, true, false>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<CT, DP, NR>::BYTES);
  return e;
}
template <int CT, bool IOF>
cudaError_t setup_type() {
  cudaError_t e = cudaSuccess;
  for (auto* f : {setup_one<CT, IOF, 64, 1>, setup_one<CT, IOF, 64, 2>, setup_one<CT, IOF, 64, 4>, setup_one<CT, IOF, 128, 1>,
                  setup_one<CT, IOF, 128, 2>})
    if (e == cudaSuccess) e = f();
  return e;
}
template <int CT, bool IOF, int DP, int NR>
cudaError_t launch_one(const CachedParams& p, cudaStream_t s) {
  auto* kernel = p.mods.cap_in != 0.f || p.mods.slopes != nullptr ? cached_rows_kernel<CT, IOF, DP, NR, true, false>
                 : p.D == DP ? cached_rows_kernel<CT, IOF, DP, NR, false, true> : cached_rows_kernel<CT, IOF, DP, NR, false, false>;
  return launch_kernel(kernel, dim3((unsigned)p.n_ctas), dim3(THREADS), Layout<CT, DP, NR>::BYTES, s, false, p);
}
template <int CT, bool IOF>
cudaError_t launch_type(const CachedParams& p, int nr, cudaStream_t s) {
  if (p.D > 64) return nr == 1 ? launch_one<CT, IOF, 128, 1>(p, s) : launch_one<CT, IOF, 128, 2>(p, s);
  return nr == 1 ? launch_one<CT, IOF, 64, 1>(p, s) : nr == 2 ? launch_one<CT, IOF, 64, 2>(p, s) : launch_one<CT, IOF, 64, 4>(p, s);
}

}  // namespace cached_rows

}  // namespace sdpa

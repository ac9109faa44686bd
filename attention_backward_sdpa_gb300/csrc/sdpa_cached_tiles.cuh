// sdpa_cached_tiles.cuh -- attention over a paged cache for many rows a key/value head: chunks of a
// prompt, or a few tokens of many heads.
//
// Bound by the tensor cores and the exponentials, as the forward (sdpa_fwd.cu), whose softmax this
// is: 128 rows against tiles of 128 keys, S = Q K^T and O += P V on tcgen05 with S, P
// and O in tensor memory, two softmax warpgroups that take half of a tile's keys each with a reference, a
// sum and an O of their own (raised lazily, joined at the end).
//
// What differs is where the tiles come from. Four loader warps fill the key tiles and four the
// value tiles, each side with a ring of its own (a key tile is free again as soon as its scores are there).
// 16-bit caches: by 16-byte asynchronous copies. 8 bits: a warp a side has bulk copies of the pages' rows, 16 at a
// time, land in two staging tiles, and the loaders widen the codes to fp16 (exact) on their way into the ring. (Codes through
// registers by plain loads waited for the small L1 that the rings leave: 445 us for 2,048 rows of 32 heads
// over 10,240 keys, 413 with rings of two stages.) Both write the 128-byte swizzle that the tensor core reads, take
// any page size, and put zeros where no query sees a row. (A tensor-map copy could bring 16-bit pages, but
// a page of 16 rows is a copy of 2 KB, and what a recycled page holds would have to be cleared.)
//
// 8 bits. All products are fp16. bf16 queries become fp16 times a power of two a row (exact down to 2^-29 of
// the row's largest). Scales stay out of the tiles: a page's key scale is in its scores' factor, and its
// value scale in the weight's exponent, w = 2^(x + log2(vs) - reference), so that
//   O = sum w * code / sum w / vs:
// the reference is the largest weighted value's, whatever the scales are. (bf16 tiles with the scales multiplied
// in took five instructions a pair of codes where fp16 takes one.)
//
// P is the products' type, each weight rounded once, as in the forward: fp16 results are off by 2.4e-4 where rounding O alone
// gives 2.1e-4 (3 chunks of up to 777 rows, D 80). (The few-rows kernel adds what the rounding leaves by a second product; here
// that would be half as many products again and as many conversions again as the softmax packs.)
//
// Under distance slopes keys still come from the first to the last, so the scores grow towards a row's own place and the
// reference is raised in nearly every tile of the steeper heads: those 3 chunks take 58 us, without slopes 47.
//
// Warps: 0-7 softmax, 8-11 key loaders (and queries), 12-15 value loaders, 16 issues S = Q K^T and owns the
// tensor memory, 17 issues O += P V, 18 and 19 have codes staged. Registers (launched with 96 a thread): 152 for
// softmax, 64 loaders, 48 the others: 256 x 152 + 256 x 64 + 128 x 48 = 640 x 96.
#pragma once

#include "cached.cuh"
#include "sdpa_fwd.cuh"

namespace sdpa {

namespace cached_tiles {

constexpr int THREADS = 640, BM = 128, BK = 128, NSLOT = 2;
constexpr uint32_t REGS_SOFTMAX = 152, REGS_LOAD = 64, REGS_CTRL = 48;
static_assert(256 * REGS_SOFTMAX + 256 * REGS_LOAD + 128 * REGS_CTRL <= THREADS * 96, "register split");
constexpr uint64_t WAIT_LIMIT_NS = 4000000000ull;
constexpr float RAISE = 8.f;  // P stays below 2^8 until its reference is raised

enum : int {
  BAR_QFULL = 0,                   // 128 arrivals: the portion's Q tile is there
  BAR_QEMPTY = 1,                  // its last S product is done
  BAR_SFULL = 2,                   // + slot
  BAR_PREADY = BAR_SFULL + NSLOT,  // + slot, 256 arrivals
  BAR_PVDONE = BAR_PREADY + NSLOT, // + slot
  BAR_RING = BAR_PVDONE + NSLOT    // keys: full (128 arrivals) + stage, empty (their S product is done) + stage; then values
};

template <int DP, bool F8>
struct Layout {
  static constexpr int BLK = 128 * 128;  // 64 columns of 128 rows
  static constexpr int TILE = BM * DP * 2;
  static constexpr int NS = DP == 64 ? 4 : F8 ? 2 : 3;
  static constexpr int STAGING = F8 ? 128 * DP : 0;   // codes of a tile; two a side
  static constexpr int NUM_BARS = BAR_RING + 4 * NS + (F8 ? 8 : 0);
  static constexpr int META = 160 + NS * 96;  // TileMeta
  static constexpr int OFF_KV = TILE;
  static constexpr int OFF_STAGING = OFF_KV + 2 * NS * TILE;  // key stages, then value stages
  static constexpr int OFF_BAR = OFF_STAGING + 4 * STAGING;
  static constexpr int OFF_XCH = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_META = OFF_XCH + 2 * 256 * 4;  // TileMeta
  static constexpr int OFF_QEXP = OFF_META + META;        // [3][128] exponents of the rows' factors, by portion
  static constexpr int OFF_MISC = OFF_QEXP + 3 * 128;
  static constexpr int BYTES_RAW = OFF_MISC + 16;
  static constexpr int BYTES = BYTES_RAW > 120 * 1024 ? BYTES_RAW : 120 * 1024;  // one CTA an SM
  static constexpr uint32_t COL_O = 128 * NSLOT;
  static_assert(BYTES <= 232448 && OFF_META % 16 == 0, "shared memory budget");
};

// Byte of 16-byte piece c (8 columns) of row r in a tile: blocks of 64 columns, 128-byte swizzle.
__device__ __forceinline__ int tile_at(int r, int c) { return (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4); }

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void codes_f16(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(four));
}

// What the loaders tell of a tile, by groups of 16 keys.
template <int NS>
struct TileMeta {
  // By side, by parity of the tile. 16 bits: the group's rows are 16 at of the cache, -1: none is read; every row of
  // the tile is. 8 bits: the staged groups' key scales and (in the second) value scales; the groups that are there,
  // and from bit 8 those without a page.
  int at[2][2][8];
  int full[2][2];
  int bad[4];       // by value stage: groups without a page
  float ks[NS][8], lvs[NS][8], inv[NS][8];  // by value stage, 8 bits: key scale, log2 and inverse of the value scale
};
static_assert(sizeof(TileMeta<3>) == Layout<128, false>::META && sizeof(TileMeta<4>) == Layout<64, true>::META, "");

// MOD (score.cuh): MOD_NONE, MOD_ROWS (distance slopes) or MOD_CAP (a cap, and slopes where given).
template <int DP, bool F8, bool F16, int MOD>
__global__ void __launch_bounds__(THREADS, 1) cached_tiles_kernel(const CachedParams p) {
  using L = Layout<DP, F8>;
  constexpr int NS = L::NS;
  constexpr bool PF = F8 || F16;          // the products are fp16
  constexpr float BIAS = PF ? 6.f : 0.f;  // weights times 2^6: what fp16's smallest step loses is below 2^-30 of the largest
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) atomicOr(p.status, STATUS_SMEM_ALIGN);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  TileMeta<NS>& meta = *reinterpret_cast<TileMeta<NS>*>(smem + L::OFF_META);
  int8_t* const q_exp = reinterpret_cast<int8_t*>(smem + L::OFF_QEXP);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  // (its shared memory: the place that the halves exchange their sums in later)
  int total;
  const CachedStart st0 = cached_start<THREADS, 1>(p, reinterpret_cast<CachedStart*>(smem + L::OFF_XCH),
                                                   reinterpret_cast<int*>(smem + L::OFF_XCH + 64), total);
  cached_empty_rows<THREADS, false>(p);
  CachedWalk<false> walk{st0.begin, st0.end, st0.te, st0.e};
  if (walk.u >= walk.end) return;
  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < L::NUM_BARS; ++i) {
      const bool full = i == BAR_QFULL || (i >= BAR_RING && i < BAR_RING + 4 * NS && (i - BAR_RING) % (2 * NS) < NS);
      mbar_init(&bars[i], full ? 128 : i >= BAR_PREADY && i < BAR_PREADY + NSLOT ? 256 : i >= BAR_RING + 4 * NS + 4 ? 4 : 1);
    }
    fence_mbar_init();
  }
  if (p.D < DP) {  // columns past D are never written
    for (int i = tid; i < L::OFF_BAR / 16; i += THREADS) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  if (warp == 16) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Every role makes the same walk and counts the tiles that it has passed (g) and the portions
  // (np), whose phases the stages, the S/P slots and the Q buffer go by.
  constexpr int K_FULL = BAR_RING, K_EMPTY = K_FULL + NS, V_FULL = K_EMPTY + NS, V_EMPTY = V_FULL + NS,
                STAGED = V_EMPTY + NS,   // 8 bits: + 2 side + parity, the staging tile's codes have landed
                STAGE_FREE = STAGED + 4; // and (an arrival a loader warp) have been read
  if (warp >= 16) {
    regs_decrease<REGS_CTRL>();
    if (warp < 18) {
      // ------------------------------------------------------------ MMA issuers
      constexpr uint32_t ID_S = idesc_io(BM, BK, false, false, PF);
      const uint32_t ID_O = idesc_io(BM, p.D, false, true, PF);  // (D is a multiple of 16)
      constexpr uint64_t T_KMAJ = sdesc_sw128_template(16, 1024);
      constexpr uint64_t T_MN_V = sdesc_sw128_template(L::BLK, 1024);
      int g = 0, np = 0;
      bool ok = true;
      CachedPortion w;
      while (ok && walk.next(p, w)) {
        const int n = w.j1 - w.j0;
        if (warp == 16) {
          ok = mbar_wait(&bars[BAR_QFULL], np & 1, abort_flag, WAIT_LIMIT_NS);
          for (int j = 0; j < n && ok; ++j, ++g) {
            const int st = g % NS, s = g % NSLOT;
            ok = mbar_wait(&bars[K_FULL + st], (g / NS) & 1, abort_flag, WAIT_LIMIT_NS);
            if (ok && g >= NSLOT)
              ok = mbar_wait(&bars[BAR_PVDONE + s], ((g - NSLOT) / NSLOT) & 1, abort_flag, WAIT_LIMIT_NS);
            if (!ok) break;
            __syncwarp();
            tc_fence_after();
            if (elect_one()) {
              const uint32_t aQ = smem_u32(smem), aK = smem_u32(smem + L::OFF_KV + st * L::TILE);
#pragma unroll
              for (int k = 0; k < DP / 16; ++k) {
                if (16 * k >= p.D) break;
                const uint32_t ko = (k >> 2) * L::BLK + (k & 3) * 32;
                mma_ss(tmem + 128u * s, sdesc_at(T_KMAJ, aQ + ko), sdesc_at(T_KMAJ, aK + ko), ID_S, k > 0);
              }
              mma_commit(&bars[BAR_SFULL + s]);
              mma_commit(&bars[K_EMPTY + st]);
              if (j == n - 1) mma_commit(&bars[BAR_QEMPTY]);
            }
            __syncwarp();
          }
        } else {
          for (int u = 0; u < n && ok; ++u, ++g) {
            const int su = g % NSLOT, stu = g % NS;
            ok = mbar_wait(&bars[BAR_PREADY + su], (g / NSLOT) & 1, abort_flag, WAIT_LIMIT_NS) &&
                 mbar_wait(&bars[V_FULL + stu], (g / NS) & 1, abort_flag, WAIT_LIMIT_NS);
            if (!ok) break;
            __syncwarp();
            tc_fence_after();
            if (elect_one()) {
              const uint32_t aV = smem_u32(smem + L::OFF_KV + (NS + stu) * L::TILE);
#pragma unroll
              for (int k = 0; k < BK / 16; ++k)
                mma_ts(tmem + L::COL_O + 128u * (k >> 2), tmem + 128u * su + 64u * (k >> 2) + 8 * (k & 3),
                       sdesc_at(T_MN_V, aV + k * 2048), ID_O, (u > 0 || (k & 3) > 0));
              mma_commit(&bars[BAR_PVDONE + su]);
              mma_commit(&bars[V_EMPTY + stu]);
            }
            __syncwarp();
          }
        }
        ++np;
      }
    } else if constexpr (F8) {
      // ------------------------------------------------------------ staging of codes
      const int side = warp - 18, group = lane & 7, bytes = 16 * p.D;
      const char* const codes = static_cast<const char*>(side ? p.c.v : p.c.k);
      uint8_t* const staging = smem + L::OFF_STAGING + side * 2 * L::STAGING + group * bytes;
      int t = 0;  // staging tiles taken
      bool ok = true;
      CachedPortion w;
      while (ok && walk.next(p, w)) {
        // Lanes 0-7 look up the pages of a tile's eight groups of 16 keys two tiles ahead, and the value side
        // their scales one tile ahead. Pages: -1 there is none, -2 no row sees the group.
        auto wanted = [&](int j) {
          const int a = cached_tile(w.s, j) * BK + 16 * group;
          return lane < 8 && j < w.j1 && a < w.s.k_hi && (a + 15 >= w.s.k_lo || a < p.first_keys);
        };
        auto entry_for = [&](int j) { return wanted(j) ? cached_lookup(p, w.b, cached_tile(w.s, j) * BK + 16 * group) : 0; };
        auto page_for = [&](int j, int entry) { return wanted(j) ? cached_page(p, entry) : -2; };
        float ks = 1.f, vs = 1.f;
        auto scales_for = [&](int page) {
          ks = vs = 1.f;
          if (side == 1 && page >= 0) {
            ks = p.c.ks[(long long)page * p.c.Hkv + w.kvh];
            vs = p.c.vs[(long long)page * p.c.Hkv + w.kvh];
          }
        };
        int page = page_for(w.j0, entry_for(w.j0)), entry = entry_for(w.j0 + 1);
        scales_for(page);
        for (int j = w.j0; j < w.j1 && ok; ++j, ++t) {
          const int x = t & 1;
          uint64_t* const full = &bars[STAGED + 2 * side + x];
          if (t >= 2) ok = __all_sync(0xffffffffu, mbar_wait(&bars[STAGE_FREE + 2 * side + x], ((t >> 1) - 1) & 1, abort_flag, WAIT_LIMIT_NS));
          if (!ok) break;
          const uint32_t there = __ballot_sync(0xffffffffu, page >= 0), bad = __ballot_sync(0xffffffffu, page == -1);
          if (side == 1 && lane < 8) {
            meta.at[0][x][lane] = __float_as_int(ks);
            meta.at[1][x][lane] = __float_as_int(vs);
          }
          if (lane == 0) meta.full[side][x] = (int)(there | (bad << 8));
          __syncwarp();
          if (lane == 0) {
            if (there) mbar_arrive_expect_tx(full, __popc(there) * bytes);
            else mbar_arrive(full);
          }
          __syncwarp();
          if (page >= 0) {
            const int a = cached_tile(w.s, j) * BK + 16 * group;
            const long long row = (((long long)page * p.c.Hkv + w.kvh) << p.c.page_shift) + (a & (p.c.page - 1));
            bulk_load(staging + x * L::STAGING, codes + row * p.D, bytes, full);
          }
          page = page_for(j + 1, entry);
          entry = entry_for(j + 2);
          scales_for(page);
        }
      }
      // No copy is in flight when the CTA ends, also where it has given up.
      volatile int never = 0;
      for (int k = max(t - 2, 0); k < t; ++k) mbar_wait(&bars[STAGED + 2 * side + (k & 1)], (k >> 1) & 1, &never, WAIT_LIMIT_NS);
    }
  } else if (warp >= 8) {
    regs_decrease<REGS_LOAD>();
    // ------------------------------------------------------------ loaders
    const int side = warp >= 12, lid = tid & 127;  // 0: keys, 1: values
    const int first_warp = 8 + 4 * side, bar_id = 2 + side;
    uint64_t* const full_bar = bars + (side ? V_FULL : K_FULL);
    uint64_t* const empty_bar = bars + (side ? V_EMPTY : K_EMPTY);
    uint8_t* const ring = smem + L::OFF_KV + side * NS * L::TILE;
    constexpr int ESZ = F8 ? 1 : 2, CHR = DP * ESZ / 16, STEP = 128 / CHR, N = CHR;  // pieces of a row, rows a pass, passes
    // Thread to piece c of row rl of a pass. 8 bits: a piece becomes two neighbouring ones of the tile; eight
    // lanes together take four pieces of an even row and the other four of the next one (or two whole rows
    // of 64), which lie on different banks both where they come from and, by the rows' swizzles, where they go.
    const int c = !F8 ? lid % CHR : CHR == 8 ? (lid & 3) | ((((lid >> 2) ^ (lid >> 3)) & 1) << 2) : lid & 3;
    const int rl = !F8 ? lid / CHR : CHR == 8 ? ((lid >> 2) & 1) | ((lid >> 3) & ~1) : lid >> 2;
    const bool in = c * 16 < p.D * ESZ;
    int g = 0, np = 0;
    bool ok = true;
    CachedPortion w;
    while (ok && walk.next(p, w)) {
      const CachedBounds& s = w.s;
      // (A wait that gives up leaves the portion going, so that all loaders meet at their barriers; they
      // end together after it.)
      if (side == 0 && np > 0) ok = mbar_wait(&bars[BAR_QEMPTY], (np - 1) & 1, abort_flag, WAIT_LIMIT_NS);
      if (side == 0) {
        __syncwarp();
        constexpr int CQ = DP / 8, SQ = 128 / CQ;  // a row's pieces on CQ neighbouring lanes
        const int cq = lid % CQ;
        const uint16_t* const q = static_cast<const uint16_t*>(p.q) + ((long long)w.b * p.c.Hkv + w.kvh) * p.R * p.D + cq * 8;
#pragma unroll 4
        for (int i = 0; i < CQ; ++i) {
          const int row = lid / CQ + i * SQ, r = w.rt * BM + row;
          if constexpr (!F8 || F16) {  // in a copy group of its own
            if (cq * 8 < p.D) copy16(smem_u32(smem) + tile_at(row, cq), q + (long long)min(r, p.R - 1) * p.D, r < p.R);
          } else {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (cq * 8 < p.D && r < p.R) v = __ldg(reinterpret_cast<const uint4*>(q + (long long)r * p.D));
            uint32_t x[4] = {v.x, v.y, v.z, v.w};
            float amax = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) amax = fmaxf(amax, fmaxf(fabsf(io_lo<false>(x[k])), fabsf(io_hi<false>(x[k]))));
#pragma unroll
            for (int k = 1; k < CQ; k <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, k));
            // 2^e brings the row's largest into [2^14, 2^15).
            const int e = amax > 0.f ? min(max(14 - ((int)(__float_as_uint(amax) >> 23) - 127), -113), 126) : 0;
            const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = pack_f16x2(io_lo<false>(x[k]) * up, io_hi<false>(x[k]) * up);
            *reinterpret_cast<uint4*>(smem + tile_at(row, cq)) = make_uint4(x[0], x[1], x[2], x[3]);
            if (cq == 0) q_exp[(np % 3) * 128 + row] = (int8_t)-e;
          }
        }
        copies_commit();
      }
      // What the softmax needs of the tile in stage st, told by the values' side: its stage is kept until the
      // softmax is done with the tile.
      auto tell_bad = [&](int st, uint32_t bad) {
        if (warp == 12 && lid == 0) meta.bad[st] = (int)bad;
      };
      const char* const rows = static_cast<const char*>(side ? p.c.v : p.c.k) + (long long)(rl & 15) * p.D * ESZ + c * 16;
      // Row rl + STEP i of a tile lies in group (rl + STEP i) / 16, the first
      // one of pass 0 in the place of the group that `rows` points to.
      const long long group_bytes = 16ll * p.D * ESZ;
      auto seen = [&](int k0, int i) {
        const int key = k0 + rl + STEP * i;
        return key < s.k_hi && (key >= s.k_lo || key < p.first_keys);
      };
      auto groups_of = [&](int x, int (&at)[8]) {
        const int4 u = *reinterpret_cast<const int4*>(meta.at[side][x]), v = *reinterpret_cast<const int4*>(meta.at[side][x] + 4);
        at[0] = u.x, at[1] = u.y, at[2] = u.z, at[3] = u.w, at[4] = v.x, at[5] = v.y, at[6] = v.z, at[7] = v.w;
      };
      if constexpr (F8) {
        const uint8_t* const staging = smem + L::OFF_STAGING + side * 2 * L::STAGING;
        for (int j = w.j0; j < w.j1; ++j, ++g) {  // (g counts the staging tiles too)
          const int st = g % NS, x = g & 1, k0 = cached_tile(s, j) * BK;
          if (ok) ok = mbar_wait(&bars[STAGED + 2 * side + x], (g >> 1) & 1, abort_flag, WAIT_LIMIT_NS);
          if (g >= NS && ok) ok = mbar_wait(&empty_bar[st], ((g / NS) - 1) & 1, abort_flag, WAIT_LIMIT_NS);
          const uint32_t about = (uint32_t)meta.full[side][x], there = about & 0xFFu;
          tell_bad(st, about >> 8);
          if (warp == 12 && lid < 8) {
            const float vs = __int_as_float(meta.at[1][x][lid]);
            meta.ks[st][lid] = __int_as_float(meta.at[0][x][lid]);
            meta.lvs[st][lid] = __log2f(vs);
            meta.inv[st][lid] = __fdividef(1.f, vs);
          }
          const bool full = there == 0xFFu && k0 <= s.k_hi - BK && (k0 >= s.k_lo || k0 <= p.first_keys - BK);
          const uint8_t* const from = staging + x * L::STAGING + rl * p.D + c * 16;
          uint8_t* const to = ring + st * L::TILE;
          if (in) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const int row = rl + STEP * i;
              uint4 v = *reinterpret_cast<const uint4*>(from + STEP * i * p.D);
              if (!full && !(((there >> (row >> 4)) & 1u) && seen(k0, i))) v = make_uint4(0u, 0u, 0u, 0u);
              uint4 a, b;
              codes_f16(v.x, a.x, a.y);
              codes_f16(v.y, a.z, a.w);
              codes_f16(v.z, b.x, b.y);
              codes_f16(v.w, b.z, b.w);
              *reinterpret_cast<uint4*>(to + tile_at(row, 2 * c)) = a;
              *reinterpret_cast<uint4*>(to + tile_at(row, 2 * c + 1)) = b;
            }
          }
          fence_proxy_async_smem();
          if (side == 0 && j == w.j0) {
            copies_wait<0>();  // Q
            fence_proxy_async_smem();
            mbar_arrive(&bars[BAR_QFULL]);
          }
          mbar_arrive(&full_bar[st]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[STAGE_FREE + 2 * side + x]);
        }
      } else {
        // Threads 0-7 look up the pages of a tile's eight groups of 16 keys one tile ahead. Pages: -1 there is none, -2 no
        // row sees the group.
        auto wanted = [&](int j) {
          const int a = cached_tile(s, j) * BK + 16 * lid;
          return lid < 8 && j < w.j1 && a < s.k_hi && (a + 15 >= s.k_lo || a < p.first_keys);
        };
        auto entry_for = [&](int j) { return wanted(j) ? cached_lookup(p, w.b, cached_tile(s, j) * BK + 16 * lid) : 0; };
        auto page_for = [&](int j, int entry) { return wanted(j) ? cached_page(p, entry) : -2; };
        // Where tile j's groups are, for its loads (parity x): the side's first warp.
        auto tell_places = [&](int x, int j, int page) {
          if (warp != first_warp) return;
          const int k0 = cached_tile(s, j) * BK, a = k0 + 16 * (lid & 7);
          if (lid < 8)
            meta.at[side][x][lid] = page < 0 ? -1 : ((page * p.c.Hkv + w.kvh) << (p.c.page_shift - 4)) + ((a & (p.c.page - 1)) >> 4);
          const bool all = __all_sync(0xffffffffu, lid >= 8 || page >= 0);
          if (lid == 0) meta.full[side][x] = all && k0 <= s.k_hi - BK && (k0 >= s.k_lo || k0 <= p.first_keys - BK);
        };
        int page = page_for(w.j0, entry_for(w.j0)), entry = entry_for(w.j0 + 1);
        int signalled = 0;  // tiles of this portion (and Q, before the first) that the others know of
        const int g0 = g;
        auto signal = [&](int upto) {
          fence_proxy_async_smem();
          if (side == 0 && signalled == 0 && upto > 0) mbar_arrive(&bars[BAR_QFULL]);
          for (; signalled < upto; ++signalled) mbar_arrive(&full_bar[(g0 + signalled) % NS]);
        };
        for (int j = w.j0; j < w.j1; ++j, ++g) {
          const int x = (j - w.j0) & 1, st = g % NS, k0 = cached_tile(s, j) * BK;
          if (j > w.j0) page = page_for(j, entry), entry = entry_for(j + 1);
          tell_places(x, j, page);
          if (g >= NS && ok) {
            if (!mbar_try_wait(&empty_bar[st], ((g / NS) - 1) & 1)) {
              copies_wait<0>();  // nothing to fill yet: what has been filled is handed over
              signal(j - w.j0);
              ok = mbar_wait(&empty_bar[st], ((g / NS) - 1) & 1, abort_flag, WAIT_LIMIT_NS);
            }
          }
          __syncwarp();
          if (warp == first_warp) tell_bad(st, __ballot_sync(0xffffffffu, page == -1));
          named_bar_sync(bar_id, 128);
          const uint32_t tile = smem_u32(ring + st * L::TILE);
          if (in) {
            int at[8];
            groups_of(x, at);
            if (meta.full[side][x]) {
#pragma unroll
              for (int i = 0; i < N; ++i)
                copy16(tile + tile_at(rl + STEP * i, c), rows + at[i * STEP / 16] * group_bytes + (i * STEP % 16) * p.D * ESZ, true);
            } else {
#pragma unroll
              for (int i = 0; i < N; ++i) {
                const bool take = at[i * STEP / 16] >= 0 && seen(k0, i);
                copy16(tile + tile_at(rl + STEP * i, c),
                       rows + (take ? at[i * STEP / 16] * group_bytes + (i * STEP % 16) * p.D * ESZ : 0), take);
              }
            }
          }
          copies_commit();
          copies_wait<1>();
          if (j > w.j0) signal(j - w.j0);  // the tile before, and Q
        }
        copies_wait<0>();
        signal(w.j1 - w.j0);
      }
      ++np;
      ok = !named_bar_any(bar_id, 128, !ok);  // (and the next portion's pages may replace these)
    }
    copies_wait<0>();
  } else {
    regs_increase<REGS_SOFTMAX>();
    // ------------------------------------------------------------ softmax
    const int half = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane, i0 = half * 64;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
    float* const xch = reinterpret_cast<float*>(smem + L::OFF_XCH);
    const uint32_t col_o = L::COL_O + 128u * half;
    CapCoef coef;
    if constexpr (MOD == MOD_CAP) coef = cap_coef(p.mods.cap_c, p.mods.cap_log2);
    int g = 0, np = 0;
    bool ok = true;
    CachedPortion w;
    while (ok && walk.next(p, w)) {
      const int r = w.rt * BM + row, n = w.j1 - w.j0;
      CachedRow rw = cached_row(p, w.s, r);
      if (r >= p.R) rw.lo = 0, rw.hi = w.s.L - 1;  // (not written; never the reason for a mask)
      const int head = w.kvh * p.G + min(r, p.R - 1) / p.Sq;
      const float slope2 = MOD != MOD_NONE && p.mods.slopes ? p.mods.slopes[head] * 1.4426950408889634f : 0.f;
      float m = -INFINITY, l = 0.f, unit = 1.f;  // unit: 8 bits, q . k of a product as it is
      for (int j = 0; j < n; ++j, ++g) {
        const int s = g % NSLOT, st = g % NS;
        const int kb = cached_tile(w.s, w.j0 + j) * BK + i0;
        // (the value stage's barrier too: what the loaders wrote beside the tile)
        ok = __all_sync(0xffffffffu, mbar_wait(&bars[V_FULL + st], (g / NS) & 1, abort_flag, WAIT_LIMIT_NS) &&
                                         mbar_wait(&bars[BAR_SFULL + s], (g / NSLOT) & 1, abort_flag, WAIT_LIMIT_NS));
        if (!ok) break;
        const uint32_t bad = ((uint32_t)meta.bad[st] >> (4 * half)) & 15u;
        // Factors of the four groups' scores (log2 units of a score as it is below), and what their weights'
        // exponents get and their sums are multiplied by.
        float cg[4], add[4], inv[4];
        if constexpr (F8) {
          if (!F16 && j == 0) unit = __uint_as_float((uint32_t)(127 + q_exp[(np % 3) * 128 + row]) << 23);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            cg[k] = fmaxf(meta.ks[st][4 * half + k] * unit * (MOD != MOD_NONE ? 1.f : p.scale_log2), 1e-38f);  // (positive: a masked score stays -inf)
            add[k] = meta.lvs[st][4 * half + k];
            inv[k] = meta.inv[st][4 * half + k];
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) cg[k] = MOD != MOD_NONE ? 1.f : p.scale_log2, add[k] = 0.f, inv[k] = 1.f;
        }
        tc_fence_after();
        uint32_t sr[2][32];
        tmem_ld32(t_lane + 128u * s + i0, sr[0]);
        tmem_ld32(t_lane + 128u * s + i0 + 32, sr[1]);
        tmem_ld_wait(sr[0]);
        tmem_ld_wait(sr[1]);
        if constexpr (MOD != MOD_NONE) {
          if constexpr (F8) {
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
              uint32_t& s0 = sr[i >> 5][i & 31];
              uint32_t& s1 = sr[i >> 5][(i & 31) + 1];
              f2_unpack(f2_mul(f2_pack(s0, s1), f2_pack(cg[i >> 4], cg[i >> 4])), s0, s1);
            }
          }
          bool small = false;
          if constexpr (MOD == MOD_CAP) {
            float big = 0.f;
#pragma unroll
            for (int i = 0; i < 64; i += 2)
              big = max3(big, fabsf(__uint_as_float(sr[i >> 5][i & 31])), fabsf(__uint_as_float(sr[i >> 5][(i & 31) + 1])));
            small = __all_sync(0xffffffffu, big <= p.mods.cap_small);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
            modify_chunk<MOD, true>(p.mods, coef, p.scale_log2, slope2, (float)(rw.place - kb - 32 * h), small, sr[h]);
#pragma unroll
          for (int k = 0; k < 4; ++k) cg[k] = 1.f;
        }
        // Masks, by halves of 32 keys and by what the warp's rows need: the last key, then the first
        // ones, then pages that there are not.
        const int hi = rw.hi - kb, lo = rw.lo - kb, first = p.first_keys - kb;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!__all_sync(0xffffffffu, hi >= 32 * h + 31)) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * h + i > hi) sr[h][i] = 0xFF800000u;  // -inf
          }
          if (!__all_sync(0xffffffffu, lo <= 32 * h || first > 32 * h + 31)) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * h + i < lo && 32 * h + i >= first) sr[h][i] = 0xFF800000u;
          }
          if ((bad >> (2 * h)) & 3u) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((bad >> (2 * h + (i >> 4))) & 1u) sr[h][i] = 0xFF800000u;
          }
        }
        float mp[8];
#pragma unroll
        for (int a = 0; a < 8; ++a) mp[a] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 64; i += 2)  // two partial maxima a group
          mp[2 * (i >> 4) + ((i >> 1) & 1)] = max3(mp[2 * (i >> 4) + ((i >> 1) & 1)], __uint_as_float(sr[i >> 5][i & 31]),
                                                   __uint_as_float(sr[i >> 5][(i & 31) + 1]));
        float mt;
        if constexpr (F8) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mp[k] = fmaf(fmaxf(mp[2 * k], mp[2 * k + 1]), cg[k], add[k]);
          mt = fmaxf(max3(mp[0], mp[1], mp[2]), mp[3]);
        } else {
          mt = max3(max3(mp[0], mp[1], mp[2]), max3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7])) * cg[0];
        }
        const bool raise = mt > m + RAISE || (m == -INFINITY && mt > -INFINITY);
        const float m_new = raise ? mt : m, alpha = raise ? ex2_approx(m - m_new) : 1.f;
        const bool rescale = raise && j > 0 && m > -INFINITY;
        if (__any_sync(0xffffffffu, rescale)) {
          ok = __all_sync(0xffffffffu, mbar_wait(&bars[BAR_PVDONE + (g - 1) % NSLOT], ((g - 1) / NSLOT) & 1, abort_flag, WAIT_LIMIT_NS));
          if (!ok) break;
          tc_fence_after();
          const float f = rescale ? alpha : 1.f;
#pragma unroll 1
          for (int c32 = 0; c32 < DP / 32; ++c32) {
            const uint32_t col = col_o + c32 * 32;
            uint32_t o[32];
            tmem_ld32(t_lane + col, o);
            tmem_ld_wait(o);
            uint32_t w0[16], w1[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              w0[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              w1[i] = __float_as_uint(__uint_as_float(o[16 + i]) * f);
            }
            tmem_st16(t_lane + col, w0);
            tmem_st16(t_lane + col + 16, w1);
          }
          tmem_st_wait();
        }
        l *= alpha;
        m = m_new;
        uint64_t rs[4];  // sums of the groups, in pairs
        const float neg_m = m == -INFINITY ? 0.f : BIAS - m;
#pragma unroll
        for (int c16 = 0; c16 < 2; ++c16) {
          uint32_t wv[16];
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2) {
            const int k = 2 * c16 + k2;
            const float f = F8 ? cg[k] : cg[0], a = F8 ? add[k] + neg_m : neg_m;
            const uint64_t f2 = f2_pack(f, f), a2 = f2_pack(a, a);
            uint64_t x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = f2_fma(f2_pack(sr[c16][16 * k2 + 2 * i], sr[c16][16 * k2 + 2 * i + 1]), f2, a2);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float x0, x1;
              f2_unpack(x[i], x0, x1);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              x[i] = f2_pack(p0, p1);
              wv[8 * k2 + i] = pack_io2<PF>(p0, p1);
            }
            rs[k] = f2_add(f2_add(f2_add(x[0], x[1]), f2_add(x[2], x[3])), f2_add(f2_add(x[4], x[5]), f2_add(x[6], x[7])));
          }
          __syncwarp();
          tmem_st16(t_lane + 128u * s + half * 64 + c16 * 16, wv);
        }
        if constexpr (F8) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float s0, s1;
            f2_unpack(rs[k], s0, s1);
            l = fmaf(s0 + s1, inv[k], l);
          }
        } else {
          float s0, s1;
          f2_unpack(f2_add(f2_add(rs[0], rs[1]), f2_add(rs[2], rs[3])), s0, s1);
          l += s0 + s1;
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars[BAR_PREADY + s]);
      }

      // ---- the halves together (as in sdpa_fwd.cu), written as results or as a part
      if (ok) ok = mbar_wait(&bars[BAR_PVDONE + (g - 1) % NSLOT], ((g - 1) / NSLOT) & 1, abort_flag, WAIT_LIMIT_NS);
      const bool warp_ok = __all_sync(0xffffffffu, ok);
      if (warp_ok) tc_fence_after();
      xch[half * 128 + row] = m;
      xch[256 + half * 128 + row] = l;
      ok = !named_bar_any(1, 256, !warp_ok);  // every softmax warp learns whether one gave up: they leave together
      const float m0 = xch[row], m1 = xch[128 + row], l0 = xch[256 + row], l1 = xch[384 + row];
      named_bar_sync(1, 256);
      const float M = fmaxf(m0, m1);
      const float a0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - M), a1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - M);
      const float lt = l0 * a0 + l1 * a1;
      const float inv = M == -INFINITY ? 0.f : 1.f / lt;
      const float lse2 = M == -INFINITY ? -INFINITY : M - BIAS + __log2f(lt);
      float f0 = a0 * inv, f1 = a1 * inv, all = lse2;
      const long long at = ((long long)blockIdx.x * 2 + max(w.slot, 0)) * p.part_rows + row;
      if (w.slot < 0) {
        float fs;
        all = cached_with_sink(p, head, lse2, fs);
        f0 *= fs;
        f1 *= fs;
      }
      const long long orow = ((long long)w.b * p.c.Hkv + w.kvh) * p.R + r;
#pragma unroll 1
      for (int c32 = 0; c32 < DP / 64; ++c32) {
        const int cbase = half * (DP / 2) + c32 * 32;
        uint32_t o0[32], o1[32];
        if (warp_ok) {
          tmem_ld32(t_lane + L::COL_O + cbase, o0);
          tmem_ld32(t_lane + L::COL_O + 128 + cbase, o1);
          tmem_ld_wait(o0);
          tmem_ld_wait(o1);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o0[i] = o1[i] = 0u;
        }
        if (r < p.R) {
#pragma unroll
          for (int v8 = 0; v8 < 4; ++v8) {
            if (cbase + v8 * 8 >= p.D) continue;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              y[e] = __uint_as_float(o0[v8 * 8 + e]) * f0 + __uint_as_float(o1[v8 * 8 + e]) * f1;
            if (w.slot >= 0) {  // (rows of a part are whole 32-byte sectors)
              float* const to = p.part_o + at * p.D + cbase + v8 * 8;
              asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(y[0]), "f"(y[1]), "f"(y[2]),
                           "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]) : "memory");
            } else {
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + orow * p.D + cbase + v8 * 8) =
                  make_uint4(pack_io2<F16>(y[0], y[1]), pack_io2<F16>(y[2], y[3]), pack_io2<F16>(y[4], y[5]),
                             pack_io2<F16>(y[6], y[7]));
            }
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      if (half == 0 && r < p.R) {
        if (w.slot >= 0) p.part_lse[at] = lse2;
        else p.lse[orow] = all * 0.6931471805599453f;
      }
      ++np;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag && tid == 0) atomicOr(p.status, STATUS_TIMEOUT);
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DP, bool F8, bool F16>
cudaError_t setup_width() {
  cudaError_t e = cudaSuccess;
  for (auto* k : {cached_tiles_kernel<DP, F8, F16, MOD_NONE>, cached_tiles_kernel<DP, F8, F16, MOD_ROWS>, cached_tiles_kernel<DP, F8, F16, MOD_CAP>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<DP, F8>::BYTES);
  return e;
}
template <bool F8, bool F16>
cudaError_t setup_type() {
  const cudaError_t e = setup_width<64, F8, F16>();
  return e != cudaSuccess ? e : setup_width<128, F8, F16>();
}
template <int DP, bool F8, bool F16>
cudaError_t launch_width(const CachedParams& p, cudaStream_t s) {
  auto* kernel = p.mods.cap_in != 0.f ? cached_tiles_kernel<DP, F8, F16, MOD_CAP>
                 : p.mods.slopes      ? cached_tiles_kernel<DP, F8, F16, MOD_ROWS> : cached_tiles_kernel<DP, F8, F16, MOD_NONE>;
  return launch_kernel(kernel, dim3((unsigned)p.n_ctas), dim3(THREADS), Layout<DP, F8>::BYTES, s, false, p);
}
template <bool F8>
cudaError_t launch_type(const CachedParams& p, cudaStream_t s) {
  if (p.f16) return p.D <= 64 ? launch_width<64, F8, true>(p, s) : launch_width<128, F8, true>(p, s);
  return p.D <= 64 ? launch_width<64, F8, false>(p, s) : launch_width<128, F8, false>(p, s);
}

}  // namespace cached_tiles

}  // namespace sdpa

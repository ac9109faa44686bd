// sdpa_cached_tiles.cuh -- attention over a paged cache for many rows a key/value head: chunks of a
// prompt, or a few tokens of many heads.
//
// Bound by the tensor cores and the exponentials, as the forward (sdpa_fwd.cu), whose softmax this
// is: 128 rows against tiles of 128 keys, S = Q K^T and O += P V on tcgen05 with S, P
// and O in tensor memory, two softmax warpgroups that take half of a tile's keys each with a reference, a
// sum and an O of their own (raised lazily, joined at the end).
//
// What differs is where the tiles come from. Four loader warps fill the stages: 16-byte asynchronous
// copies (16-bit caches), or loads that become io values on the way (8 bits: codes are widened
// and multiplied by their page's scale, exactly where that is a power of two). A thread keeps the next
// tile's codes in registers while it widens this one's. They write the 128-byte swizzle that the
// tensor core reads, take any page size, and fill rows that no query sees with zeros. (A bulk tensor
// copy could bring 16-bit pages, but not widen codes, and a page of 16 rows is a copy of 2 KB.)
//
// Warps: 0-7 softmax, 8-11 loaders, 12 issues S = Q K^T and owns the tensor memory, 13 issues
// O += P V. Registers (launched with 128 a thread): 184 for softmax, 104 loaders, 40 issuers:
// 256 x 184 + 128 x 104 + 128 x 40 = 512 x 128.
#pragma once

#include "cached.cuh"

namespace sdpa {

namespace cached_tiles {

constexpr int THREADS = 512, BM = 128, BK = 128, NSLOT = 2;
constexpr uint32_t REGS_SOFTMAX = 184, REGS_LOAD = 104, REGS_CTRL = 40;
static_assert(256 * REGS_SOFTMAX + 128 * REGS_LOAD + 128 * REGS_CTRL <= THREADS * 128, "register split");
constexpr uint64_t WAIT_LIMIT_NS = 4000000000ull;
constexpr float RAISE = 8.f;  // P stays below 2^8 until its reference is raised

enum : int {
  BAR_QFULL = 0,                   // 128 arrivals: the portion's Q tile is there
  BAR_QEMPTY = 1,                  // its last S product is done
  BAR_KVFULL = 2,                  // + stage (up to 4), 128 arrivals
  BAR_KVEMPTY = 6,                 // + stage: the tile's PV product is done
  BAR_SFULL = 10,                  // + slot
  BAR_PREADY = BAR_SFULL + NSLOT,  // + slot, 256 arrivals
  BAR_PVDONE = BAR_PREADY + NSLOT, // + slot
  NUM_BARS = BAR_PVDONE + NSLOT
};

template <int DP>
struct Layout {
  static constexpr int BLK = 128 * 128;  // 64 columns of 128 rows
  static constexpr int TILE = BM * DP * 2;
  static constexpr int STAGE = 2 * TILE;
  static constexpr int REST = NUM_BARS * 8 + 2 * 256 * 4 + 512 + 64;
  static constexpr int NS_FIT = (232448 - TILE - REST) / STAGE;
  static constexpr int NS = NS_FIT > 4 ? 4 : NS_FIT;
  static constexpr int OFF_KV = TILE;
  static constexpr int OFF_BAR = OFF_KV + NS * STAGE;
  static constexpr int OFF_XCH = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_META = OFF_XCH + 2 * 256 * 4;  // page[2][8], scales[2][16], bad[4]
  static constexpr int OFF_MISC = OFF_META + 512;
  static constexpr int BYTES_RAW = OFF_MISC + 64;
  static constexpr int BYTES = BYTES_RAW > 120 * 1024 ? BYTES_RAW : 120 * 1024;  // one CTA an SM
  static constexpr uint32_t COL_O = 128 * NSLOT;
  static_assert(NS >= 2 && BYTES <= 232448, "shared memory budget");
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
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void codes_f16(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(four));
}

// How a page's codes become io values: `fast`, one multiplication by `c` (a pair) after the bits
// of a code have been put where an io value has them; else through fp32.
struct Widen {
  bool fast;
  uint32_t c;
  float scale;
};
template <bool F16>
__device__ __forceinline__ Widen widen_by(float scale) {
  Widen w;
  const uint32_t u = __float_as_uint(scale), e = u >> 23;
  const bool two = (u & 0x7FFFFFu) == 0;
  w.scale = scale;
  if constexpr (F16) {  // e4m3 -> fp16 is exact; the scale as an fp16 number
    w.fast = two && e >= 127 - 14 && e <= 127 + 15;
    w.c = ((e - 127 + 15) << 10) * 0x10001u;
  } else {
    // A code's exponent and fraction bits as those of a bf16 number stand for 2^-120 of its
    // value (bias 127 against 7), the smallest ones included.
    w.fast = two && e >= 27 && e <= 127 + 7;
    w.c = ((e + 120) << 7) * 0x10001u;
  }
  return w;
}
// Four codes as two io pairs.
template <bool F16>
__device__ __forceinline__ void widen4(uint32_t four, const Widen& w, uint32_t& lo, uint32_t& hi) {
  if (w.fast) {
    if constexpr (F16) {
      codes_f16(four, lo, hi);
      lo = mul_f16x2(lo, w.c);
      hi = mul_f16x2(hi, w.c);
    } else {
      const uint32_t a = __byte_perm(four, 0u, 0x1404), b = __byte_perm(four, 0u, 0x3424);  // codes in the upper bytes
      lo = mul_bf16x2((a & 0x80008000u) | ((a >> 4) & 0x07F007F0u), w.c);
      hi = mul_bf16x2((b & 0x80008000u) | ((b >> 4) & 0x07F007F0u), w.c);
    }
  } else {
    codes_f16(four, lo, hi);
    lo = pack_io2<F16>(io_lo<true>(lo) * w.scale, io_hi<true>(lo) * w.scale);
    hi = pack_io2<F16>(io_lo<true>(hi) * w.scale, io_hi<true>(hi) * w.scale);
  }
}

template <int DP, bool F8, bool F16, bool MOD>
__global__ void __launch_bounds__(THREADS, 1) cached_tiles_kernel(const CachedParams p) {
  using L = Layout<DP>;
  constexpr int NS = L::NS;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) atomicOr(p.status, STATUS_SMEM_ALIGN);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  int* meta_page = reinterpret_cast<int*>(smem + L::OFF_META);        // [2][8]
  float* meta_scale = reinterpret_cast<float*>(smem + L::OFF_META + 64);  // [2][16]
  int* meta_bad = reinterpret_cast<int*>(smem + L::OFF_META + 192);   // [4] by stage: groups of 16 keys without a page
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  // (its shared memory: the place that the halves exchange their sums in later)
  const CachedStart st0 = cached_start<THREADS>(
      p, reinterpret_cast<CachedStart*>(smem + L::OFF_XCH), reinterpret_cast<long long*>(smem + L::OFF_XCH + 64),
      blockIdx.x == 0, [&](long long T) { return share_begin(T, p.n_ctas, blockIdx.x); });
  pdl_launch_dependents();  // (the merge waits for this grid before it reads the parts)
  CachedWalk walk{st0.at, share_begin(st0.T, p.n_ctas, blockIdx.x + 1), st0.te, st0.e};
  if (walk.u >= walk.end) return;
  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < NUM_BARS; ++i)
      mbar_init(&bars[i], i == BAR_QFULL || (i >= BAR_KVFULL && i < BAR_KVFULL + 4) ? 128
                          : i >= BAR_PREADY && i < BAR_PREADY + NSLOT ? 256 : 1);
    fence_mbar_init();
  }
  if (p.D < DP) {  // columns past D are never written
    for (int i = tid; i < L::OFF_BAR / 16; i += THREADS) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Every role makes the same walk and counts the tiles that it has passed (g) and the portions
  // (np), whose phases the stages, the S/P slots and the Q buffer go by.
  if (warp >= 12) {
    regs_decrease<REGS_CTRL>();
    if (warp < 14) {
      // ------------------------------------------------------------ MMA issuers
      constexpr uint32_t ID_S = idesc_io(BM, BK, false, false, F16);
      constexpr uint32_t ID_O = idesc_io(BM, DP, false, true, F16);
      constexpr uint64_t T_KMAJ = sdesc_sw128_template(16, 1024);
      constexpr uint64_t T_MN_V = sdesc_sw128_template(L::BLK, 1024);
      int g = 0, np = 0;
      bool ok = true;
      CachedPortion w;
      while (ok && walk.next(p, w)) {
        const int n = w.j1 - w.j0;
        if (warp == 12) {
          ok = mbar_wait(&bars[BAR_QFULL], np & 1, abort_flag, WAIT_LIMIT_NS);
          for (int j = 0; j < n && ok; ++j, ++g) {
            const int st = g % NS, s = g % NSLOT;
            ok = mbar_wait(&bars[BAR_KVFULL + st], (g / NS) & 1, abort_flag, WAIT_LIMIT_NS);
            if (ok && g >= NSLOT)
              ok = mbar_wait(&bars[BAR_PVDONE + s], ((g - NSLOT) / NSLOT) & 1, abort_flag, WAIT_LIMIT_NS);
            if (!ok) break;
            __syncwarp();
            tc_fence_after();
            if (elect_one()) {
              const uint32_t aQ = smem_u32(smem), aK = smem_u32(smem + L::OFF_KV + st * L::STAGE);
#pragma unroll
              for (int k = 0; k < DP / 16; ++k) {
                const uint32_t ko = (k >> 2) * L::BLK + (k & 3) * 32;
                mma_ss(tmem + 128u * s, sdesc_at(T_KMAJ, aQ + ko), sdesc_at(T_KMAJ, aK + ko), ID_S, k > 0);
              }
              mma_commit(&bars[BAR_SFULL + s]);
              if (j == n - 1) mma_commit(&bars[BAR_QEMPTY]);
            }
            __syncwarp();
          }
        } else {
          for (int u = 0; u < n && ok; ++u, ++g) {
            const int su = g % NSLOT, stu = g % NS;
            ok = mbar_wait(&bars[BAR_PREADY + su], (g / NSLOT) & 1, abort_flag, WAIT_LIMIT_NS) &&
                 mbar_wait(&bars[BAR_KVFULL + stu], (g / NS) & 1, abort_flag, WAIT_LIMIT_NS);
            if (!ok) break;
            __syncwarp();
            tc_fence_after();
            if (elect_one()) {
              const uint32_t aV = smem_u32(smem + L::OFF_KV + stu * L::STAGE + L::TILE);
#pragma unroll
              for (int k = 0; k < BK / 16; ++k)
                mma_ts(tmem + L::COL_O + 128u * (k >> 2), tmem + 128u * su + 64u * (k >> 2) + 8 * (k & 3),
                       sdesc_at(T_MN_V, aV + k * 2048), ID_O, (u > 0 || (k & 3) > 0));
              mma_commit(&bars[BAR_PVDONE + su]);
              mma_commit(&bars[BAR_KVEMPTY + stu]);
            }
            __syncwarp();
          }
        }
        ++np;
      }
    }
  } else if (warp >= 8) {
    regs_decrease<REGS_LOAD>();
    // ------------------------------------------------------------ loaders
    const int lid = tid - 256;
    constexpr int ESZ = F8 ? 1 : 2, CHR = DP * ESZ / 16, STEP = 128 / CHR, N = CHR;  // pieces of a row, rows a pass, passes
    const int c = lid % CHR, rl = lid / CHR;
    const bool in = c * 16 < p.D * ESZ;
    int g = 0, np = 0;
    bool ok = true;
    CachedPortion w;
    while (ok && walk.next(p, w)) {
      const CachedBounds& s = w.s;
      // Q, in a copy group of its own.
      // (A wait that gives up leaves the portion going, so that all loaders meet at their barriers; they
      // end together after it.)
      if (np > 0) ok = mbar_wait(&bars[BAR_QEMPTY], (np - 1) & 1, abort_flag, WAIT_LIMIT_NS);
      {
        constexpr int CQ = DP / 8, SQ = 128 / CQ;
        const int cq = lid % CQ;
        const uint16_t* const q = static_cast<const uint16_t*>(p.q) + ((long long)w.b * p.c.Hkv + w.kvh) * p.R * p.D + cq * 8;
        if (cq * 8 < p.D) {
#pragma unroll 4
          for (int i = 0; i < CQ; ++i) {
            const int row = lid / CQ + i * SQ, r = w.rt * BM + row;
            copy16(smem_u32(smem) + tile_at(row, cq), q + (long long)min(r, p.R - 1) * p.D, r < p.R);
          }
        }
        copies_commit();
      }
      // Threads 0-7 look up the pages of a tile's eight groups of 16 keys two tiles ahead, and their
      // scales one tile ahead.
      auto page_for = [&](int j) -> int {
        if (lid >= 8 || j >= w.j1) return -1;
        const int a = cached_tile(s, j) * BK + 16 * lid;
        return a < s.k_hi && (a + 15 >= s.k_lo || a < p.first_keys) ? cached_page(p, w.b, a) : -2;
      };
      auto scale_for = [&](int page, const float* scales) -> float {
        return F8 && lid < 8 && page >= 0 ? scales[(long long)page * p.c.Hkv + w.kvh] : 1.f;
      };
      int page0 = page_for(w.j0), page1 = page_for(w.j0 + 1);
      float ks = scale_for(page0, p.c.ks), vs = scale_for(page0, p.c.vs);
      auto row_from = [&](const int* pages, int j, int i, long long& off) -> bool {
        // row rl + STEP i of tile j: element offset of its piece, and whether some query sees it
        const int row = rl + STEP * i, key = cached_tile(s, j) * BK + row, page = pages[row >> 4];
        const bool take = in && page >= 0 && key < s.k_hi && (key >= s.k_lo || key < p.first_keys);
        off = take ? ((((long long)page * p.c.Hkv + w.kvh) << p.c.page_shift) + (key & (p.c.page - 1))) * p.D * ESZ + c * 16 : 0;
        return take;
      };
      const char* const kc = static_cast<const char*>(p.c.k);
      const char* const vc = static_cast<const char*>(p.c.v);
      auto bad_groups = [&](int page) -> uint32_t {  // (lanes 0-7 of warp 8)
        return __ballot_sync(0xffffffffu, lid < 8 && page == -1);
      };
      if constexpr (F8) {
        uint4 kr[N], vr[N];
        // Pages of the first tile, then its codes.
        if (lid < 8) meta_page[lid] = page0;
        uint32_t bad = warp == 8 ? bad_groups(page0) : 0u;
        named_bar_sync(2, 128);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          long long off;
          const bool take = row_from(meta_page, w.j0, i, off);
          kr[i] = take ? __ldg(reinterpret_cast<const uint4*>(kc + off)) : make_uint4(0u, 0u, 0u, 0u);
          vr[i] = take ? __ldg(reinterpret_cast<const uint4*>(vc + off)) : make_uint4(0u, 0u, 0u, 0u);
        }
        for (int j = w.j0; j < w.j1; ++j, ++g) {
          const int x = (j - w.j0) & 1, st = g % NS;
          // The scales of this tile, and the pages of the next one.
          if (lid < 8) {
            meta_scale[16 * x + lid] = ks;
            meta_scale[16 * x + 8 + lid] = vs;
            meta_page[8 * (x ^ 1) + lid] = page1;
          }
          const uint32_t bad_next = warp == 8 ? bad_groups(page1) : 0u;
          named_bar_sync(2, 128);
          ks = scale_for(page1, p.c.ks);
          vs = scale_for(page1, p.c.vs);
          page1 = page_for(j + 2);
          if (g >= NS && ok) ok = mbar_wait(&bars[BAR_KVEMPTY + st], ((g / NS) - 1) & 1, abort_flag, WAIT_LIMIT_NS);
          uint8_t* const tile = smem + L::OFF_KV + st * L::STAGE;
          if (lid == 0) meta_bad[st] = (int)bad;
          bad = bad_next;
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            uint8_t* const to = tile + side * L::TILE;
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const int row = rl + STEP * i;
              const uint4 v = side ? vr[i] : kr[i];
              long long off;
              const bool take = j + 1 < w.j1 && row_from(meta_page + 8 * (x ^ 1), j + 1, i, off);
              uint4& next = side ? vr[i] : kr[i];
              next = make_uint4(0u, 0u, 0u, 0u);
              if (take) next = __ldg(reinterpret_cast<const uint4*>((side ? vc : kc) + off));
              if (in) {
                const Widen wd = widen_by<F16>(meta_scale[16 * x + 8 * side + (row >> 4)]);
                uint4 a, b;
                widen4<F16>(v.x, wd, a.x, a.y);
                widen4<F16>(v.y, wd, a.z, a.w);
                widen4<F16>(v.z, wd, b.x, b.y);
                widen4<F16>(v.w, wd, b.z, b.w);
                // (Threads of the second block store their pieces in the other order: no bank twice.)
                const bool swap = c >= 4;
                *reinterpret_cast<uint4*>(to + tile_at(row, 2 * c + (swap ? 1 : 0))) = swap ? b : a;
                *reinterpret_cast<uint4*>(to + tile_at(row, 2 * c + (swap ? 0 : 1))) = swap ? a : b;
              }
            }
          }
          if (j == w.j0) copies_wait<0>();  // Q
          fence_proxy_async_smem();
          if (j == w.j0) mbar_arrive(&bars[BAR_QFULL]);
          mbar_arrive(&bars[BAR_KVFULL + st]);
        }
      } else {
        int signalled = 0;  // tiles of this portion (and Q, before the first) that the others know of
        auto signal = [&](int upto) {
          fence_proxy_async_smem();
          if (signalled == 0 && upto > 0) mbar_arrive(&bars[BAR_QFULL]);
          for (; signalled < upto; ++signalled) mbar_arrive(&bars[BAR_KVFULL + (g - (upto - signalled)) % NS]);
        };
        for (int j = w.j0; j < w.j1; ++j) {
          const int x = (j - w.j0) & 1, st = g % NS;
          if (lid < 8) meta_page[8 * x + lid] = page0;
          const uint32_t bad = warp == 8 ? bad_groups(page0) : 0u;
          page0 = page1;
          page1 = page_for(j + 2);
          named_bar_sync(2, 128);
          if (g >= NS && ok) {
            if (!mbar_try_wait(&bars[BAR_KVEMPTY + st], ((g / NS) - 1) & 1)) {
              copies_wait<0>();  // nothing to fill yet: what has been filled is handed over
              signal(j - w.j0);
              ok = mbar_wait(&bars[BAR_KVEMPTY + st], ((g / NS) - 1) & 1, abort_flag, WAIT_LIMIT_NS);
            }
          }
          const uint32_t tile = smem_u32(smem + L::OFF_KV + st * L::STAGE);
          if (lid == 0) meta_bad[st] = (int)bad;
          if (in) {
#pragma unroll 4
            for (int i = 0; i < N; ++i) {
              long long off;
              const bool take = row_from(meta_page + 8 * x, j, i, off);
              const int at = tile_at(rl + STEP * i, c);
              copy16(tile + at, kc + off, take);
              copy16(tile + L::TILE + at, vc + off, take);
            }
          }
          copies_commit();
          ++g;
          copies_wait<1>();
          if (j > w.j0) {
            // (tile j - 1 and Q have landed; g counts tile j too)
            --g;
            signal(j - w.j0);
            ++g;
          }
        }
        copies_wait<0>();
        signal(w.j1 - w.j0);
      }
      ++np;
      ok = !named_bar_any(2, 128, !ok);  // (and the next portion's pages may replace these)
    }
    copies_wait<0>();
  } else {
    regs_increase<REGS_SOFTMAX>();
    // ------------------------------------------------------------ softmax
    const int half = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane, i0 = half * 64;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
    float* const xch = reinterpret_cast<float*>(smem + L::OFF_XCH);
    const uint32_t col_o = L::COL_O + 128u * half;
    const float cs = MOD ? 1.f : p.scale_log2;  // log2 units of a score as it is below
    int g = 0;
    bool ok = true;
    CachedPortion w;
    while (ok && walk.next(p, w)) {
      const int r = w.rt * BM + row, n = w.j1 - w.j0;
      CachedRow rw = cached_row(p, w.s, r);
      if (r >= p.R) rw.lo = 0, rw.hi = w.s.L - 1;  // (not written; never the reason for a mask)
      const int head = w.kvh * p.G + min(r, p.R - 1) / p.Sq;
      const float slope2 = MOD && p.mods.slopes ? p.mods.slopes[head] * 1.4426950408889634f : 0.f;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++g) {
        const int s = g % NSLOT, st = g % NS;
        const int kb = cached_tile(w.s, w.j0 + j) * BK + i0;
        // (the stage's barrier too: what the loaders wrote beside the tile)
        ok = __all_sync(0xffffffffu, mbar_wait(&bars[BAR_KVFULL + st], (g / NS) & 1, abort_flag, WAIT_LIMIT_NS) &&
                                         mbar_wait(&bars[BAR_SFULL + s], (g / NSLOT) & 1, abort_flag, WAIT_LIMIT_NS));
        if (!ok) break;
        const uint32_t bad = ((uint32_t)meta_bad[st] >> (4 * half)) & 15u;
        tc_fence_after();
        uint32_t sr[2][32];
        tmem_ld32(t_lane + 128u * s + i0, sr[0]);
        tmem_ld32(t_lane + 128u * s + i0 + 32, sr[1]);
        tmem_ld_wait(sr[0]);
        tmem_ld_wait(sr[1]);
        if constexpr (MOD) {
          const bool cap = p.mods.cap_in != 0.f;
          const float c = cap ? p.mods.cap_log2 : p.scale_log2;
#pragma unroll
          for (int b8 = 0; b8 < 8; ++b8) {
            uint64_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = f2_pack(sr[b8 >> 2][(b8 & 3) * 8 + 2 * i], sr[b8 >> 2][(b8 & 3) * 8 + 2 * i + 1]);
            if (cap) tanh2_any(x, p.mods.cap_in);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float x0, x1;
              f2_unpack(x[i], x0, x1);
              const int key = kb + b8 * 8 + 2 * i;
              sr[b8 >> 2][(b8 & 3) * 8 + 2 * i] = __float_as_uint(fmaf(-slope2, fabsf((float)(rw.place - key)), x0 * c));
              sr[b8 >> 2][(b8 & 3) * 8 + 2 * i + 1] = __float_as_uint(fmaf(-slope2, fabsf((float)(rw.place - key - 1)), x1 * c));
            }
          }
        }
        const bool mine = kb + 63 <= rw.hi && (kb >= rw.lo || kb + 63 < p.first_keys);
        if (!__all_sync(0xffffffffu, mine) || bad != 0u) {
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            const int key = kb + i;
            if (key > rw.hi || (key < rw.lo && key >= p.first_keys) || ((bad >> (i >> 4)) & 1u))
              sr[i >> 5][i & 31] = 0xFF800000u;  // -inf
          }
        }
        float mp[8];
#pragma unroll
        for (int a = 0; a < 8; ++a) mp[a] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 64; i += 2)
          mp[(i >> 1) & 7] = max3(mp[(i >> 1) & 7], __uint_as_float(sr[i >> 5][i & 31]), __uint_as_float(sr[i >> 5][(i & 31) + 1]));
        const float mt = max3(max3(mp[0], mp[1], mp[2]), max3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7])) * cs;
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
        float rs[8];
#pragma unroll
        for (int a = 0; a < 8; ++a) rs[a] = 0.f;
        const float neg_m = m == -INFINITY ? 0.f : -m;
#pragma unroll
        for (int c16 = 0; c16 < 2; ++c16) {
          uint32_t wv[16];
#pragma unroll
          for (int i2 = 0; i2 < 16; ++i2) {
            const float p0 = ex2_approx(fmaf(__uint_as_float(sr[c16][2 * i2]), cs, neg_m));
            const float p1 = ex2_approx(fmaf(__uint_as_float(sr[c16][2 * i2 + 1]), cs, neg_m));
            rs[(2 * i2) & 7] += p0;
            rs[(2 * i2 + 1) & 7] += p1;
            wv[i2] = pack_io2<F16>(p0, p1);
          }
          __syncwarp();
          tmem_st16(t_lane + 128u * s + half * 64 + c16 * 16, wv);
        }
        l += ((rs[0] + rs[1]) + (rs[2] + rs[3])) + ((rs[4] + rs[5]) + (rs[6] + rs[7]));
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
      const float lse2 = M == -INFINITY ? -INFINITY : M + __log2f(lt);
      float f0 = a0 * inv, f1 = a1 * inv, all = lse2;
      const long long at = ((long long)blockIdx.x * 2 + max(w.slot, 0)) * BM + row;
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
            if (w.slot >= 0) {
              float4* to = reinterpret_cast<float4*>(p.part_o + at * p.D + cbase + v8 * 8);
              to[0] = make_float4(y[0], y[1], y[2], y[3]);
              to[1] = make_float4(y[4], y[5], y[6], y[7]);
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
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag && tid == 0) atomicOr(p.status, STATUS_TIMEOUT);
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DP, bool F8, bool F16, bool MOD>
cudaError_t setup_one() {
  return cudaFuncSetAttribute(cached_tiles_kernel<DP, F8, F16, MOD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<DP>::BYTES);
}
template <bool F8, bool F16>
cudaError_t setup_type() {
  cudaError_t e = cudaSuccess;
  for (auto* f : {setup_one<64, F8, F16, false>, setup_one<64, F8, F16, true>, setup_one<128, F8, F16, false>, setup_one<128, F8, F16, true>})
    if (e == cudaSuccess) e = f();
  return e;
}
template <int DP, bool F8, bool F16>
cudaError_t launch_width(const CachedParams& p, cudaStream_t s) {
  const bool mod = p.mods.cap_in != 0.f || p.mods.slopes != nullptr;
  return launch_kernel(mod ? cached_tiles_kernel<DP, F8, F16, true> : cached_tiles_kernel<DP, F8, F16, false>,
                       dim3((unsigned)p.n_ctas), dim3(THREADS), Layout<DP>::BYTES, s, false, p);
}
template <bool F8>
cudaError_t launch_type(const CachedParams& p, cudaStream_t s) {
  if (p.f16) return p.D <= 64 ? launch_width<64, F8, true>(p, s) : launch_width<128, F8, true>(p, s);
  return p.D <= 64 ? launch_width<64, F8, false>(p, s) : launch_width<128, F8, false>(p, s);
}

}  // namespace cached_tiles

}  // namespace sdpa

// sdpa_kv_cache.cu -- a paged cache of keys and values: appending rows, with the position
// rotation of queries and keys on the way, and reading rows back.
//
// Position j of a sequence is slot j % page of page table[j / page]. The new rows of a call
// are the last new_len positions of the sequence's length. A key is rotated in fp32 as by
// sdpa_rope.cu (what becomes a code, in twice that: angle_sin_cos_2) and rounded once, to the cache's type.
//
// 8 bits. e4m3 has the same 4 significant bits over 2^-6 .. 448, so what a scale is good for
// is the range, and a power of two serves as well as any: the smallest 2^e (e >= -64) that
// brings the largest new value of the page and head within 448. With powers of two a page whose
// scale has to grow loses nothing: its older codes are multiplied by a power of two, exact
// unless they fall below 2^-6, where they are rounded to the coarser steps. A page whose
// first slot is written starts anew; else its scale never falls.
// Values are rounded once, x / scale to nearest even. NaN stays NaN; an infinity saturates at
// 448 * scale and, like NaN, has no say in the scale.
//
// Work. `rows` blocks: a thread owns a token and eight column pairs and walks heads, as the
// rotary kernel does, with the row's place in the cache as its destination (queries, and keys
// and values of a 16-bit cache). `quant` blocks: one per page that the call touches, key/value
// heads (one, or a few that share the angles) and side (K, V), since a scale is one reduction over a page and
// head: rows to fp32, rotated, their largest value, then the codes. Both kinds run in one launch.
// Bound by memory: 2 bytes an element read, 1 or 2 written. For few tokens it is a chain of latencies (lengths, page,
// rows, angles; 4.1 us for 64 tokens of 32 + 8 + 8 heads, code fetched anew 9.8). For prompts it is the instructions, half
// of the issue slots: 5 prompts of up to 1,700 tokens into 8-bit pages, 92 MB with the cache read back, take 38 us, 28
// of them this launch (33 and 23 with sines, products and sums of fp32 alone, which put a few of 3 million codes a
// whole step off; eight library sines a thread in line waited for their code: 39). Into 16-bit pages prompts are bound by
// memory: 4 of 8,192 tokens, 32 + 8 + 8 heads of 128 columns, take 120 us, 6.7 TB/s (8 bits: 222, 3.3 TB/s); 5 of 1,700
// tokens, 16 + 4 + 4 heads, 20.9 us, 5.0 TB/s. Read back, 4 sequences of 8,192 positions take 43 us, 6.2 TB/s, from
// 16 bits and 38, 5.3 TB/s, from 8.
#include <cuda_fp16.h>

#include "common.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace sdpa {

namespace {

constexpr int THREADS = 256;

__device__ __forceinline__ int new_rows(const KvAppendArgs& a, int b) {
  return a.new_lens ? min(max(a.new_lens[b], 0), a.T) : a.T;
}
// The page of position pos of batch row b; -1 (and the status bit) when there is none.
__device__ __forceinline__ int page_of(const KvCacheRef& c, int b, long long pos, int* status) {
  int page = -1;
  if (pos >= 0 && (pos >> c.page_shift) < c.max_pages) page = c.table[(long long)b * c.max_pages + (pos >> c.page_shift)];
  if ((unsigned)page < (unsigned)c.n_pages) return page;
  atomicOr(status, STATUS_PAGE);
  return -1;
}
__device__ __forceinline__ int row_position(const KvAppendArgs& a, int b, int t, long long start, int axis) {
  return a.positions ? a.positions[axis * a.axis_stride + b * a.pos_bstride + t] : (int)(start + t);
}
// a / b for a >= 0 (64-bit only where it takes that).
__device__ __forceinline__ long long quotient(long long a, int b) {
  return (a >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}
__device__ __forceinline__ uint4 ld8(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void st8(uint16_t* p, const uint4& v) { *reinterpret_cast<uint4*>(p) = v; }
template <bool F16>
__device__ __forceinline__ void widen8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = io_lo<F16>(w[i]), f[2 * i + 1] = io_hi<F16>(w[i]);
}
template <bool F16>
__device__ __forceinline__ uint4 narrow8(const float* f) {
  return make_uint4(pack_io2<F16>(f[0], f[1]), pack_io2<F16>(f[2], f[3]), pack_io2<F16>(f[4], f[5]),
                    pack_io2<F16>(f[6], f[7]));
}
// Two pieces of eight columns turned: the pairs' first and second halves, or (interleaved) eight
// neighbouring pairs, four a piece.
template <bool F16>
__device__ __forceinline__ void turn16(const uint4& u, const uint4& w, bool interleaved, const float* sn, const float* cs,
                                       float (&f)[16]) {
  float p[8], r[8];
  widen8<F16>(u, p);
  widen8<F16>(w, r);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = p[2 * i] * cs[i] - p[2 * i + 1] * sn[i];
      f[2 * i + 1] = p[2 * i + 1] * cs[i] + p[2 * i] * sn[i];
      f[8 + 2 * i] = r[2 * i] * cs[4 + i] - r[2 * i + 1] * sn[4 + i];
      f[9 + 2 * i] = r[2 * i + 1] * cs[4 + i] + r[2 * i] * sn[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[i] = p[i] * cs[i] - r[i] * sn[i];
      f[8 + i] = r[i] * cs[i] + p[i] * sn[i];
    }
  }
}
struct AppendPlan {
  int quant_blocks;    // blocks [0, quant_blocks) write 8-bit pages, the others rows
  int pages_touched;   // pages a batch row may touch
  int page_heads, page_groups;  // key/value heads that a block of the former walks, groups of them
  int held;            // ... in registers (else through shared memory)
  int heads, head_groups;  // rows: heads a thread walks, groups of them in all (K's and V's with a 16-bit cache)
  int groups;          // column groups of a row: VW pairs each, or two pieces of VW pass-through columns
  int block_rows;      // tokens of a block at a time
  long long tokens;
  int item_blocks;
};

// The frequencies as fractions of a turn, and each pair's axis.
struct Turns {
  uint64_t turn[64];  // D <= 128
  SinCos2 nodes[33];
  uint8_t axis[64];
};
__device__ constexpr SinCosNodes NODES = sin_cos_nodes();
__device__ __forceinline__ void make_turns(const KvAppendArgs& a, Turns& m, int half, bool nodes) {
  for (int i = threadIdx.x; i < half; i += THREADS) {
    m.turn[i] = turn_fraction(a.freq[i]);
    m.axis[i] = a.pair_axis ? (uint8_t)min(max(a.pair_axis[i], 0), a.n_axes - 1) : (uint8_t)0;
  }
  if (nodes)
    for (int i = threadIdx.x; i < 33; i += THREADS) m.nodes[i] = NODES.at[i];
}

// VW 8: rot a multiple of 16, rows of 16-byte alignment; a group is eight pairs, or sixteen pass-through columns.
// VW 1: any rot, any alignment; a group is one pair, or two pass-through columns.
// A block takes a few heads of one tensor: queries, or (16-bit cache) keys or values.
template <bool F16, int VW>
__device__ __forceinline__ void append_rows(const KvAppendArgs& a, const AppendPlan& pl, int block, Turns& turns) {
  const KvCacheRef& c = a.c;
  const int D = c.D, tid = threadIdx.x;
  int hg = block % pl.head_groups;
  const int gq = ceil_div(a.Hq, pl.heads), gk = ceil_div(c.Hkv, pl.heads);
  const int which = hg < gq ? 0 : hg < gq + gk ? 1 : 2;
  hg -= which == 0 ? 0 : which == 1 ? gq : gq + gk;
  const int h0 = hg * pl.heads, nh = min(pl.heads, (which == 0 ? a.Hq : c.Hkv) - h0);
  const long long* const st = which == 0 ? a.qs : which == 1 ? a.kst : a.vst;
  const uint16_t* const x0 = static_cast<const uint16_t*>(which == 0 ? a.q : which == 1 ? a.k : a.v) + h0 * st[1];
  const long long xh = st[1], yh = which == 0 ? a.qos[1] : (long long)D << c.page_shift;
  const int rot = which == 2 ? 0 : a.rot, half = rot / 2;
  const int g = tid % pl.groups;
  const bool rotated = g < rot / (2 * VW);
  const int c0 = rotated ? (a.interleaved ? 2 * VW * g : VW * g) : 2 * VW * g;
  const int c1 = rotated && !a.interleaved ? half + VW * g : c0 + VW;  // D and rot are even: c1 < D
  const long long step = (long long)pl.item_blocks * pl.block_rows;
  long long tok = tid < pl.block_rows * pl.groups ? (long long)(block / pl.head_groups) * pl.block_rows + tid / pl.groups : pl.tokens;
  int b = 0, t = 0;
  const uint16_t* x = x0;
  auto token = [&]() {
    b = (int)quotient(tok, a.T), t = (int)(tok - (long long)b * a.T);
    x = x0 + b * st[0] + t * st[2];
  };
  constexpr int UNROLL = VW == 8 ? 4 : 1;  // heads whose loads are under way together
  uint4 u[UNROLL], w[UNROLL];
  auto load = [&](int h) {
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      if (h + k >= nh) continue;
      u[k] = ld8(x + (h + k) * xh + c0);
      w[k] = ld8(x + (h + k) * xh + c1);
    }
  };
  if (tok < pl.tokens) {  // (the first loads are on their way while the angles are made)
    token();
    if constexpr (VW == 8) load(0);
  }
  if (rot > 0) {
    make_turns(a, turns, half, false);
    __syncthreads();
  }
  while (tok < pl.tokens) {
    const int n_new = new_rows(a, b);
    const long long start = (long long)c.lens[b] - n_new;
    uint16_t* y = nullptr;
    if (which == 0) {
      y = static_cast<uint16_t*>(a.q_out) + b * a.qos[0] + h0 * a.qos[1] + t * a.qos[2];
    } else if (t < n_new) {
      const int page = page_of(c, b, start + t, a.status);
      if (page >= 0)
        y = static_cast<uint16_t*>(which == 1 ? c.k : c.v) +
            ((((long long)page * c.Hkv + h0) << c.page_shift) + ((start + t) & (c.page - 1))) * D;
    }
    float sn[VW], cs[VW];
    if (rotated) {
      int pos = 0, axis = -1;  // (neighbouring pairs mostly turn by the same axis)
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        const int ax = turns.axis[g * VW + i];
        if (ax != axis) axis = ax, pos = row_position(a, b, t, start, ax);
        angle_sin_cos_near(turns.turn[g * VW + i], pos, sn[i], cs[i]);
        sn[i] *= a.mult;
        cs[i] *= a.mult;
      }
    }
    if constexpr (VW == 8) {
      for (int h = 0; h < nh && y != nullptr;) {
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
          if (h + k >= nh) continue;
          if (rotated) {
            float f[16];
            turn16<F16>(u[k], w[k], a.interleaved != 0, sn, cs, f);
            u[k] = narrow8<F16>(f);
            w[k] = narrow8<F16>(f + 8);
          }
          st8(y + (h + k) * yh + c0, u[k]);
          st8(y + (h + k) * yh + c1, w[k]);
        }
        h += UNROLL;
        if (h < nh) load(h);
      }
    } else {
      for (int h = 0; h < nh && y != nullptr; ++h) {
        uint16_t p = x[h * xh + c0], r = x[h * xh + c1];
        if (rotated) {
          const float f = io_f32<F16>(p), z = io_f32<F16>(r);
          const uint32_t o = pack_io2<F16>(f * cs[0] - z * sn[0], z * cs[0] + f * sn[0]);
          p = (uint16_t)(o & 0xFFFFu);
          r = (uint16_t)(o >> 16);
        }
        y[h * yh + c0] = p;
        y[h * yh + c1] = r;
      }
    }
    tok += step;
    if (tok < pl.tokens) {
      token();
      if constexpr (VW == 8) load(0);
    }
  }
}

// turn16 for values that become codes.
template <bool F16>
__device__ __forceinline__ void turn16_odd(const uint4& u, const uint4& w, bool interleaved, const SinCos2 (&n)[8], float (&f)[16]) {
  float p[8], r[8];
  widen8<F16>(u, p);
  widen8<F16>(w, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = interleaved ? (i < 4 ? p[2 * (i & 3)] : r[2 * (i & 3)]) : p[i];
    const float y = interleaved ? (i < 4 ? p[2 * (i & 3) + 1] : r[2 * (i & 3) + 1]) : r[i];
    const float a = dot_odd(x, n[i].ch, n[i].cl, -y, n[i].sh, n[i].sl), b = dot_odd(y, n[i].ch, n[i].cl, x, n[i].sh, n[i].sl);
    if (interleaved) f[2 * i] = a, f[2 * i + 1] = b;
    else f[i] = a, f[8 + i] = b;
  }
}

// The smallest 2^e >= amax / 448, e >= -64 (448 = 1.75 * 2^8: the exponent less 8, one more
// where the fraction is above 1.75).
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(max(e, -64) + 127) << 23);
}
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void e4m3_widen(uint32_t four, float (&f)[4]) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(four));
  f[0] = io_lo<true>(lo), f[1] = io_hi<true>(lo), f[2] = io_lo<true>(hi), f[3] = io_hi<true>(hi);
}
// Eight values x / scale as codes: by its inverse, where that is exact (a power of two, as this kernel's own
// scales are; a page's scale may also be a caller's).
__device__ __forceinline__ uint2 codes8(const float* x, float inv) {
  return make_uint2(e4m3_pair(x[0] * inv, x[1] * inv) | (e4m3_pair(x[2] * inv, x[3] * inv) << 16),
                    e4m3_pair(x[4] * inv, x[5] * inv) | (e4m3_pair(x[6] * inv, x[7] * inv) << 16));
}
__device__ __noinline__ uint2 codes8_divided(float x0, float x1, float x2, float x3, float x4, float x5, float x6, float x7,
                                             float scale) {
  return make_uint2(e4m3_pair(__fdiv_rn(x0, scale), __fdiv_rn(x1, scale)) | (e4m3_pair(__fdiv_rn(x2, scale), __fdiv_rn(x3, scale)) << 16),
                    e4m3_pair(__fdiv_rn(x4, scale), __fdiv_rn(x5, scale)) | (e4m3_pair(__fdiv_rn(x6, scale), __fdiv_rn(x7, scale)) << 16));
}
__device__ __forceinline__ uint2 codes8(const float* x, float scale, float inv) {
  if (inv != 0.f) return codes8(x, inv);
  return codes8_divided(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], scale);
}
__device__ __forceinline__ float finite_max(float m, float x) { return fabsf(x) < INFINITY ? fmaxf(m, fabsf(x)) : m; }

constexpr int HELD = 2;  // items of 16 columns that a thread keeps

// A page's new rows of a few key/value heads of one side. `held`: a thread's items (16 columns of a row, in two
// pieces of eight as a rotation pairs them) stay in registers from their loads to their codes, the sines and cosines
// of its rows, which the heads share, in shared memory, and a head's loads are issued before the one before it is
// reduced. (Not all of it: three CTAs an SM leave 80 registers, and 96 bytes a thread, 176 with fp16 io, are stored to
// local memory and loaded again.) That takes at most HELD items a thread (64 rows of 128 columns); larger pages, and rows whose
// rotation or alignment does not go in pieces of eight, pass through shared memory in fp32.
template <bool F16, int VW>
__device__ __forceinline__ void append_page(const KvAppendArgs& a, const AppendPlan& pl, int block, float* smem, Turns& turns) {
  __shared__ float warp_max[2][THREADS / 32];
  const KvCacheRef& c = a.c;
  const int tid = threadIdx.x, D = c.D;
  const int side = block & 1;
  block >>= 1;
  const int h0 = block % pl.page_groups * pl.page_heads, h1 = min(h0 + pl.page_heads, c.Hkv);
  block /= pl.page_groups;
  const int b = block / pl.pages_touched;
  const int n_new = new_rows(a, b);
  const long long end = c.lens[b], start = end - n_new;
  if (n_new == 0) return;
  const long long pg = floor_div(start, c.page) + block % pl.pages_touched;
  const long long first = max(start, pg * c.page), last = min(end, (pg + 1) * c.page);
  if (first >= last) return;
  const int lo = (int)(first & (c.page - 1)), n = (int)(last - first);  // slots [lo, lo + n)
  const int t0 = (int)(first - start);
  const long long hs = side ? a.vst[1] : a.kst[1], xs = side ? a.vst[2] : a.kst[2];
  const uint16_t* x = side ? static_cast<const uint16_t*>(a.v) + b * a.vst[0] + h0 * hs + t0 * xs
                           : static_cast<const uint16_t*>(a.k) + b * a.kst[0] + h0 * hs + t0 * xs;
  const int rot = side ? 0 : a.rot, half = rot / 2;
  const bool held = VW == 8 && pl.held;
  const int groups = D / 16, items = n * groups;
  uint4 u[HELD], w[HELD];
  // Item k: row rk[k], columns [c0[k], c0[k] + 8) and [c1[k], c1[k] + 8).
  int rk[HELD], c0[HELD], c1[HELD];
  bool turned[HELD];
#pragma unroll
  for (int k = 0; k < HELD; ++k) {
    const int i = tid + k * THREADS, g = i % groups;
    const bool halves = g < rot / 16 && !a.interleaved;
    rk[k] = i / groups;
    turned[k] = g < rot / 16;
    c0[k] = halves ? 8 * g : 16 * g;
    c1[k] = halves ? half + 8 * g : c0[k] + 8;
  }
  auto load = [&]() {
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
      if (tid + k * THREADS >= items) continue;
      u[k] = ld8(x + rk[k] * xs + c0[k]);
      w[k] = ld8(x + rk[k] * xs + c1[k]);
    }
  };
  if (held) load();
  const int page = page_of(c, b, first, a.status);
  if (page < 0) return;
  if (rot > 0) make_turns(a, turns, half, true);
  // Angle j of a thread's item k is at [(8 k + j) * APART + tid] (apart so that neither side of it meets in a bank).
  constexpr int APART = THREADS + 1;
  SinCos2* const angles = reinterpret_cast<SinCos2*>(smem);
  if (rot > 0) {
    __syncthreads();
    if (held) {
#pragma unroll 2
      for (int i = tid; i < n * half; i += THREADS) {
        const int r = i / half, pair = i - r * half, item = r * groups + pair / 8;
        const SinCos2 n = angle_sin_cos_2(turns.turn[pair], row_position(a, b, t0 + r, start, turns.axis[pair]), turns.nodes, a.mult);
        *reinterpret_cast<float4*>(angles + (item / THREADS * 8 + (pair & 7)) * APART + item % THREADS) = make_float4(n.sh, n.sl, n.ch, n.cl);
      }
      __syncthreads();
    }
  }
#pragma unroll 1
  for (int h = h0; h < h1; ++h, x += hs) {
    float* const scale_at = (side ? c.vs : c.ks) + (long long)page * c.Hkv + h;
    const float was = *scale_at;
    float amax = 0.f;
    float f[HELD][16];
    if (held) {
#pragma unroll
      for (int k = 0; k < HELD; ++k) {
        if (tid + k * THREADS >= items) continue;
        if (turned[k]) {
          SinCos2 n[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 v = *reinterpret_cast<const float4*>(angles + (k * 8 + j) * APART + tid);
            n[j] = SinCos2{v.x, v.y, v.z, v.w};
          }
          turn16_odd<F16>(u[k], w[k], a.interleaved != 0, n, f[k]);
        } else {
          widen8<F16>(u[k], f[k]);
          widen8<F16>(w[k], f[k] + 8);
        }
        float m = 0.f;  // (fmaxf takes the other one of a NaN)
#pragma unroll
        for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(f[k][j]));
        if (m == INFINITY) {
          m = 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) m = finite_max(m, f[k][j]);
        }
        amax = fmaxf(amax, m);
      }
      if (h + 1 < h1) {
        x += hs;
        load();
        x -= hs;
      }
    } else {
      for (int i = tid; i < n * D; i += THREADS) {
        const int r = i / D, col = i - r * D;
        smem[i] = io_f32<F16>(x[r * xs + col]);
        if (col >= rot) amax = finite_max(amax, smem[i]);
      }
      __syncthreads();
      for (int i = tid; i < n * half; i += THREADS) {
        const int r = i / half, pair = i - r * half;
        const SinCos2 m = angle_sin_cos_2(turns.turn[pair], row_position(a, b, t0 + r, start, turns.axis[pair]), turns.nodes, a.mult);
        float* const p0 = smem + r * D + (a.interleaved ? 2 * pair : pair);
        float* const p1 = a.interleaved ? p0 + 1 : p0 + half;
        const float z0 = *p0, z1 = *p1, y0 = dot_odd(z0, m.ch, m.cl, -z1, m.sh, m.sl), y1 = dot_odd(z1, m.ch, m.cl, z0, m.sh, m.sl);
        *p0 = y0;
        *p1 = y1;
        amax = finite_max(finite_max(amax, y0), y1);
      }
    }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));  // (not negative: ordered as integers)
    float* const warps = warp_max[h & 1];  // two in turn: one barrier a head
    if ((tid & 31) == 0) warps[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) amax = fmaxf(amax, warps[i]);
    const float need = scale_for(amax), scale = lo == 0 ? need : fmaxf(need, was);
    const uint32_t bits = __float_as_uint(scale);  // (of a power of two below 2^127: the inverse has the exponent's negative)
    const float inv = (bits & 0x7FFFFFu) == 0 && bits - 1u < 0x7F000000u - 1u ? __uint_as_float(0x7F000000u - bits) : 0.f;
    uint8_t* const codes = static_cast<uint8_t*>(side ? c.v : c.k) + (((long long)page * c.Hkv + h) << c.page_shift) * D;
    if (held) {
#pragma unroll
      for (int k = 0; k < HELD; ++k) {
        if (tid + k * THREADS >= items) continue;
        uint8_t* const to = codes + (lo + rk[k]) * D;
        *reinterpret_cast<uint2*>(to + c0[k]) = codes8(f[k], scale, inv);
        *reinterpret_cast<uint2*>(to + c1[k]) = codes8(f[k] + 8, scale, inv);
      }
    } else {
      for (int i = tid; i < n * D / 8; i += THREADS)
        *reinterpret_cast<uint2*>(codes + lo * D + i * 8) = codes8(smem + i * 8, scale, inv);
      __syncthreads();
    }
    if (lo > 0 && scale != was) {  // the older slots in the new scale
#pragma unroll 1
      for (int i = tid; i < lo * D / 8; i += THREADS) {
        const uint2 v = *reinterpret_cast<const uint2*>(codes + i * 8);
        float y[8], z[4];
        e4m3_widen(v.x, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = z[e] * was;
        e4m3_widen(v.y, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[4 + e] = z[e] * was;
        *reinterpret_cast<uint2*>(codes + i * 8) = codes8(y, scale, inv);
      }
    }
    if (tid == 0) *scale_at = scale;  // (every thread has read it: before the barrier above)
  }
}

template <bool F16, int VW>
__global__ void __launch_bounds__(THREADS, 3) kv_append_kernel(const KvAppendArgs a, const AppendPlan pl) {
  extern __shared__ __align__(16) float smem[];
  __shared__ Turns turns;
  if ((int)blockIdx.x < pl.quant_blocks) append_page<F16, VW>(a, pl, blockIdx.x, smem, turns);
  else append_rows<F16, VW>(a, pl, blockIdx.x - pl.quant_blocks, turns);
}

// A block takes a (batch, head) and GATHER / pieces positions (pieces of 16 columns); a thread one row's piece of
// K and V, both loaded before the first store.
constexpr int GATHER = 256;
template <bool F8, bool F16>
__global__ void __launch_bounds__(GATHER) kv_gather_kernel(const KvGatherArgs a, int bh_count) {
  const KvCacheRef& c = a.c;
  const int pieces = c.D / 16, rows = GATHER / pieces;
  const int r = threadIdx.x / pieces, p = threadIdx.x - r * pieces;
  if (r >= rows) return;
  for (int bh = blockIdx.y; bh < bh_count; bh += gridDim.y) {
    const int b = bh / c.Hkv, h = bh - b * c.Hkv;
    for (long long s = (long long)blockIdx.x * rows + r; s < a.S; s += (long long)gridDim.x * rows) {
      int page = -1;
      if (s < cached_len(c, b)) page = page_of(c, b, s, a.status);
      if (p == 0 && h == 0 && s == 0 && (c.lens[b] < 0 || c.lens[b] > (long long)c.max_pages * c.page)) atomicOr(a.status, STATUS_PAGE);
      uint4 lo[2], hi[2];
      float scale[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        lo[j] = hi[j] = make_uint4(0u, 0u, 0u, 0u);
        scale[j] = 0.f;
        if (page < 0) continue;
        const void* const from = j ? c.v : c.k;
        const long long at = ((((long long)page * c.Hkv + h) << c.page_shift) + (s & (c.page - 1))) * c.D + p * 16;
        if constexpr (F8) {
          lo[j] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(from) + at));
          scale[j] = (j ? c.vs : c.ks)[(long long)page * c.Hkv + h];
        } else {
          const uint4* const q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(from) + at);
          lo[j] = __ldcs(q);
          hi[j] = __ldcs(q + 1);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (F8) {
          const uint32_t v[4] = {lo[j].x, lo[j].y, lo[j].z, lo[j].w};
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float f[4];
            e4m3_widen(v[e], f);
            o[2 * e] = pack_io2<F16>(f[0] * scale[j], f[1] * scale[j]);
            o[2 * e + 1] = pack_io2<F16>(f[2] * scale[j], f[3] * scale[j]);
          }
          lo[j] = make_uint4(o[0], o[1], o[2], o[3]);
          hi[j] = make_uint4(o[4], o[5], o[6], o[7]);
        }
        uint4* const to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(j ? a.v_out : a.k_out) +
                                                   ((long long)bh * a.S + s) * c.D + p * 16);
        to[0] = lo[j];
        to[1] = hi[j];
      }
    }
  }
}

bool rows_aligned(const void* base, const long long (&st)[3]) {
  return reinterpret_cast<uintptr_t>(base) % 16 == 0 && st[0] % 8 == 0 && st[1] % 8 == 0 && st[2] % 8 == 0;
}

}  // namespace

cudaError_t kv_cache_setup() {
  cudaError_t e = cudaSuccess;
  constexpr int most = 256 * 128 * 4;  // a page of 256 rows of 128 columns in fp32
  for (auto* k : {kv_append_kernel<false, 8>, kv_append_kernel<false, 1>, kv_append_kernel<true, 8>,
                  kv_append_kernel<true, 1>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  return e;
}

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t s, int num_sms) {
  AppendPlan pl{};
  const KvCacheRef& c = a.c;
  const bool wide = a.rot % 16 == 0 && rows_aligned(a.k, a.kst) && rows_aligned(a.v, a.vst) &&
                    (a.Hq == 0 || (rows_aligned(a.q, a.qs) && rows_aligned(a.q_out, a.qos)));
  size_t smem = 0;
  if (c.f8) {
    const int rows = a.T < c.page ? a.T : c.page;  // of a page at most
    const int items = ceil_div(rows * (c.D / 16), THREADS);
    pl.pages_touched = (a.T + c.page - 2) / c.page + 1;  // T rows from any slot
    pl.held = wide && items <= HELD;
    // Heads that share a page's angles, as long as there are some blocks for each SM.
    const long long pages = 2ll * a.B * pl.pages_touched;
    pl.page_heads = 1;
    while (pl.page_heads < 8 && pl.page_heads < c.Hkv && pages * ceil_div(c.Hkv, 2 * pl.page_heads) >= 4ll * num_sms)
      pl.page_heads *= 2;
    pl.page_groups = ceil_div(c.Hkv, pl.page_heads);
    pl.quant_blocks = (int)(pages * pl.page_groups);
    smem = !pl.held ? (size_t)rows * c.D * 4 : a.rot > 0 ? (size_t)items * 8 * (THREADS + 1) * sizeof(SinCos2) : 0;
  }
  pl.groups = c.D / (wide ? 16 : 2);
  pl.block_rows = THREADS / pl.groups;
  pl.tokens = (long long)a.B * a.T;
  const long long blocks = (pl.tokens + pl.block_rows - 1) / pl.block_rows;
  const auto head_groups = [&](int heads) { return ceil_div(a.Hq, heads) + (c.f8 ? 0 : 2 * ceil_div(c.Hkv, heads)); };
  pl.heads = blocks * head_groups(8) < num_sms ? 2 : 8;
  pl.head_groups = head_groups(pl.heads);
  pl.item_blocks = pl.head_groups == 0 ? 0 : (int)(blocks < num_sms * 16ll ? blocks : num_sms * 16ll);
  const unsigned grid = (unsigned)(pl.quant_blocks + pl.item_blocks * pl.head_groups);
  if (grid == 0) return cudaSuccess;
  auto* kernel = a.f16 ? (wide ? kv_append_kernel<true, 8> : kv_append_kernel<true, 1>)
                       : (wide ? kv_append_kernel<false, 8> : kv_append_kernel<false, 1>);
  return launch_kernel(kernel, dim3(grid), dim3(THREADS), smem, s, false, a, pl);
}

cudaError_t launch_kv_gather(const KvGatherArgs& a, cudaStream_t s, int num_sms) {
  if (a.B == 0 || a.S == 0) return cudaSuccess;
  const int bh = a.B * a.c.Hkv, rows = GATHER / (a.c.D / 16);
  const int across = (a.S - 1) / rows + 1;  // (S may be within `rows` of 2^31)
  const dim3 grid((unsigned)(across < num_sms * 64 ? across : num_sms * 64), (unsigned)(bh < 65535 ? bh : 65535));
  auto* kernel = a.c.f8 ? (a.f16 ? kv_gather_kernel<true, true> : kv_gather_kernel<true, false>)
                        : kv_gather_kernel<false, false>;
  return launch_kernel(kernel, grid, dim3(GATHER), 0, s, false, a, bh);
}

}  // namespace sdpa

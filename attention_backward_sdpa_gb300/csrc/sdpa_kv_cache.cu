// sdpa_kv_cache.cu -- a paged cache of keys and values: appending rows, with the position
// rotation of queries and keys on the way, and reading rows back.
//
// Position j of a sequence is slot j % page of page table[j / page]. The new rows of a call
// are the last new_len positions of the sequence's length. A key is rotated in fp32 as by
// sdpa_rope.cu and rounded once, to the cache's type.
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
// head and side (K, V), since a scale is one reduction over them: rows to fp32 in shared memory, rotated
// there pair by pair, their largest value, then the codes in 16-byte stores. Both kinds run in one launch.
// Bound by memory: 2 bytes an element read, 1 or 2 written.
#include <cuda_fp16.h>

#include "common.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace sdpa {

namespace {

constexpr int THREADS = 128;

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
__device__ __forceinline__ int axis_of(const KvAppendArgs& a, int pair) {
  return a.pair_axis ? min(max(a.pair_axis[pair], 0), a.n_axes - 1) : 0;
}

// Eight 16-bit values, in one access where the address allows it.
__device__ __forceinline__ uint4 ld8(const uint16_t* p, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void st8(uint16_t* p, const uint4& v, bool vec) {
  if (vec) {
    *reinterpret_cast<uint4*>(p) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) p[2 * i] = (uint16_t)w[i], p[2 * i + 1] = (uint16_t)(w[i] >> 16);
}
template <bool F16>
__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = io_lo<F16>(w[i]), f[2 * i + 1] = io_hi<F16>(w[i]);
}
template <bool F16>
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
  return make_uint4(pack_io2<F16>(f[0], f[1]), pack_io2<F16>(f[2], f[3]), pack_io2<F16>(f[4], f[5]),
                    pack_io2<F16>(f[6], f[7]));
}

struct AppendPlan {
  int quant_blocks;    // blocks [0, quant_blocks) write 8-bit pages, the others rows
  int pages_touched;   // pages a batch row may touch
  int heads, head_groups, n_heads;  // rows: heads a thread walks, groups of them, heads in all (K and V with a 16-bit cache)
  int groups;          // column groups of a row: VW pairs each, or two pieces of VW pass-through columns
  long long n_items;   // tokens * groups
  int item_blocks;
  int vec_q, vec_qo, vec_k, vec_v;  // rows of these are 16-byte aligned
};

// VW 8: rot a multiple of 16; a group is eight pairs, or sixteen pass-through columns.
// VW 1: any rot; a group is one pair, or two pass-through columns.
template <bool F16, int VW>
__device__ __forceinline__ void append_rows(const KvAppendArgs& a, const AppendPlan& pl, int block) {
  __shared__ uint64_t turns[ROPE_MAX_PAIRS];
  const KvCacheRef& c = a.c;
  const int half = a.rot / 2, D = c.D;
  for (int i = threadIdx.x; i < half; i += THREADS) turns[i] = turn_fraction(a.freq[i]);
  __syncthreads();
  const int h0 = (block % pl.head_groups) * pl.heads, h1 = min(h0 + pl.heads, pl.n_heads);
  const int rot_groups = a.rot / (2 * VW);
  for (long long it = (long long)(block / pl.head_groups) * THREADS + threadIdx.x; it < pl.n_items;
       it += (long long)pl.item_blocks * THREADS) {
    const int g = (int)(it % pl.groups);
    const long long tok = it / pl.groups;
    const int t = (int)(tok % a.T), b = (int)(tok / a.T);
    const bool rotated = g < rot_groups;
    const int c0 = rotated ? (a.interleaved ? 2 * VW * g : VW * g) : 2 * VW * g;
    const int c1 = rotated && !a.interleaved ? half + VW * g : c0 + VW;  // D and rot are even: c1 < D
    const int n_new = new_rows(a, b);
    const long long start = (long long)c.lens[b] - n_new;
    float sn[VW], cs[VW];
    if (rotated) {
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        const int pair = g * VW + i;
        angle_sin_cos_near(turns[pair], row_position(a, b, t, start, axis_of(a, pair)), sn[i], cs[i]);
        sn[i] *= a.mult;
        cs[i] *= a.mult;
      }
    }
    long long place = -1;  // element offset of the token's row of head 0 in the cache
    if (h1 > a.Hq && t < n_new) {
      const int page = page_of(c, b, start + t, a.status);
      if (page >= 0) place = (((long long)page * c.Hkv << c.page_shift) + ((start + t) & (c.page - 1))) * D;
    }
    for (int h = h0; h < h1; ++h) {
      const uint16_t* x;
      uint16_t* y;
      bool turn = rotated, vx, vy = true;
      if (h < a.Hq) {
        x = static_cast<const uint16_t*>(a.q) + b * a.qs[0] + h * a.qs[1] + t * a.qs[2];
        y = static_cast<uint16_t*>(a.q_out) + b * a.qos[0] + h * a.qos[1] + t * a.qos[2];
        vx = pl.vec_q, vy = pl.vec_qo;
      } else {
        if (place < 0) break;
        const bool val = h >= a.Hq + c.Hkv;
        const int hh = h - a.Hq - (val ? c.Hkv : 0);
        x = val ? static_cast<const uint16_t*>(a.v) + b * a.vst[0] + hh * a.vst[1] + t * a.vst[2]
                : static_cast<const uint16_t*>(a.k) + b * a.kst[0] + hh * a.kst[1] + t * a.kst[2];
        y = static_cast<uint16_t*>(val ? c.v : c.k) + place + ((long long)hh << c.page_shift) * D;
        vx = val ? pl.vec_v : pl.vec_k;
        turn = rotated && !val;
      }
      if constexpr (VW == 8) {
        uint4 u = ld8(x + c0, vx), w = ld8(x + c1, vx);
        if (turn) {
          float p[8], r[8], y0[8], y1[8];
          widen8<F16>(u, p);
          widen8<F16>(w, r);
          if (a.interleaved) {  // pairs are neighbours: p holds pairs 0-3, r pairs 4-7
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              y0[2 * i] = p[2 * i] * cs[i] - p[2 * i + 1] * sn[i];
              y0[2 * i + 1] = p[2 * i + 1] * cs[i] + p[2 * i] * sn[i];
              y1[2 * i] = r[2 * i] * cs[4 + i] - r[2 * i + 1] * sn[4 + i];
              y1[2 * i + 1] = r[2 * i + 1] * cs[4 + i] + r[2 * i] * sn[4 + i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              y0[i] = p[i] * cs[i] - r[i] * sn[i];
              y1[i] = r[i] * cs[i] + p[i] * sn[i];
            }
          }
          u = narrow8<F16>(y0);
          w = narrow8<F16>(y1);
        }
        st8(y + c0, u, vy);
        st8(y + c1, w, vy);
      } else {
        uint16_t u = x[c0], w = x[c1];
        if (turn) {
          const float p = io_f32<F16>(u), r = io_f32<F16>(w);
          const uint32_t o = pack_io2<F16>(p * cs[0] - r * sn[0], r * cs[0] + p * sn[0]);
          u = (uint16_t)(o & 0xFFFFu);
          w = (uint16_t)(o >> 16);
        }
        y[c0] = u;
        y[c1] = w;
      }
    }
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
// Sixteen values x * up / scale as codes (up: the older codes' scale, else 1; `inv` = 1 / scale
// where that is exact, else 0).
__device__ __forceinline__ uint4 codes16(const float (&x)[16], float up, float scale, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = x[4 * i + j] * up;
      y[j] = inv != 0.f ? v * inv : __fdiv_rn(v, scale);
    }
    w[i] = e4m3_pair(y[0], y[1]) | (e4m3_pair(y[2], y[3]) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool F16>
__device__ __forceinline__ void append_page(const KvAppendArgs& a, const AppendPlan& pl, int block, float* sx) {
  __shared__ float warp_max[THREADS / 32];
  __shared__ uint64_t turns[64];  // D <= 128
  const KvCacheRef& c = a.c;
  const int tid = threadIdx.x, D = c.D;
  const int side = block & 1;
  block >>= 1;
  const int h = block % c.Hkv;
  block /= c.Hkv;
  const int b = block / pl.pages_touched;
  const int n_new = new_rows(a, b);
  const long long end = c.lens[b], start = end - n_new;
  if (n_new == 0) return;
  const long long pg = floor_div(start, c.page) + block % pl.pages_touched;
  const long long first = max(start, pg * c.page), last = min(end, (pg + 1) * c.page);
  if (first >= last) return;
  const int page = page_of(c, b, first, a.status);
  if (page < 0) return;
  const int lo = (int)(first & (c.page - 1)), n = (int)(last - first);  // slots [lo, lo + n)
  const int t0 = (int)(first - start);
  // The new rows as fp32.
  const uint16_t* x = side ? static_cast<const uint16_t*>(a.v) + b * a.vst[0] + h * a.vst[1] + t0 * a.vst[2]
                           : static_cast<const uint16_t*>(a.k) + b * a.kst[0] + h * a.kst[1] + t0 * a.kst[2];
  const long long xs = side ? a.vst[2] : a.kst[2];
  const bool vec = side ? pl.vec_v : pl.vec_k;
  const int pieces = D / 8;
  float amax = 0.f;
  const bool turned = !side && a.rot > 0;
  const int rot = turned ? a.rot : 0;
  if (tid < rot / 2) turns[tid] = turn_fraction(a.freq[tid]);
  for (int i = tid; i < n * pieces; i += THREADS) {
    const int r = i / pieces, p = i % pieces;
    float f[8];
    widen8<F16>(ld8(x + r * xs + p * 8, vec), f);
    float4* to = reinterpret_cast<float4*>(sx + r * D + p * 8);
    to[0] = make_float4(f[0], f[1], f[2], f[3]);
    to[1] = make_float4(f[4], f[5], f[6], f[7]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (p * 8 + j >= rot && fabsf(f[j]) < INFINITY) amax = fmaxf(amax, fabsf(f[j]));
  }
  __syncthreads();
  if (turned) {
    const int half = rot / 2;
    for (int i = tid; i < n * half; i += THREADS) {
      const int r = i / half, pair = i % half;
      float sn, cs;
      angle_sin_cos_near(turns[pair], row_position(a, b, t0 + r, start, axis_of(a, pair)), sn, cs);
      sn *= a.mult;
      cs *= a.mult;
      float* p0 = sx + r * D + (a.interleaved ? 2 * pair : pair);
      float* p1 = a.interleaved ? p0 + 1 : p0 + half;
      const float u = *p0, w = *p1, y0 = u * cs - w * sn, y1 = w * cs + u * sn;
      *p0 = y0;
      *p1 = y1;
      if (fabsf(y0) < INFINITY) amax = fmaxf(amax, fabsf(y0));
      if (fabsf(y1) < INFINITY) amax = fmaxf(amax, fabsf(y1));
    }
  }
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));  // (not negative: ordered as integers)
  if ((tid & 31) == 0) warp_max[tid >> 5] = amax;
  float* const scale_at = (side ? c.vs : c.ks) + (long long)page * c.Hkv + h;
  const float was = *scale_at;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) amax = fmaxf(amax, warp_max[i]);
  const float need = scale_for(amax), scale = lo == 0 ? need : fmaxf(need, was);
  const bool exact = (__float_as_uint(scale) & 0x7FFFFFu) == 0;
  const float inv = exact ? __fdiv_rn(1.f, scale) : 0.f;
  uint8_t* const codes = static_cast<uint8_t*>(side ? c.v : c.k) + (((long long)page * c.Hkv + h) << c.page_shift) * D;
  for (int i = tid; i < n * D / 16; i += THREADS) {
    float f[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 v = reinterpret_cast<const float4*>(sx + i * 16)[j];
      f[4 * j] = v.x, f[4 * j + 1] = v.y, f[4 * j + 2] = v.z, f[4 * j + 3] = v.w;
    }
    *reinterpret_cast<uint4*>(codes + (long long)lo * D + i * 16) = codes16(f, 1.f, scale, inv);
  }
  if (lo > 0 && scale != was) {  // the older slots in the new scale
    for (int i = tid; i < lo * D / 16; i += THREADS) {
      const uint4 v = *reinterpret_cast<const uint4*>(codes + i * 16);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float f[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float g[4];
        e4m3_widen(w[j], g);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * j + e] = g[e];
      }
      *reinterpret_cast<uint4*>(codes + i * 16) = codes16(f, was, scale, inv);
    }
  }
  if (tid == 0) *scale_at = scale;  // (every thread has read it: before the barrier above)
}

template <bool F16, int VW>
__global__ void __launch_bounds__(THREADS) kv_append_kernel(const KvAppendArgs a, const AppendPlan pl) {
  extern __shared__ __align__(16) float sx[];
  if ((int)blockIdx.x < pl.quant_blocks) append_page<F16>(a, pl, blockIdx.x, sx);
  else append_rows<F16, VW>(a, pl, blockIdx.x - pl.quant_blocks);
}

// One thread per 16 columns of a (batch, head, position) row of K and the same of V.
template <bool F8, bool F16>
__global__ void __launch_bounds__(256) kv_gather_kernel(const KvGatherArgs a, long long n_items) {
  const KvCacheRef& c = a.c;
  const int pieces = c.D / 16;
  for (long long it = (long long)blockIdx.x * 256 + threadIdx.x; it < n_items; it += (long long)gridDim.x * 256) {
    const int p = (int)(it % pieces);
    const long long row = it / pieces;  // (b, h, s)
    const int s = (int)(row % a.S);
    const long long bh = row / a.S;
    const int h = (int)(bh % c.Hkv), b = (int)(bh / c.Hkv);
    int page = -1;
    if (s < cached_len(c, b)) page = page_of(c, b, s, a.status);
    if (p == 0 && h == 0 && s == 0 && c.lens[b] > (long long)c.max_pages * c.page) atomicOr(a.status, STATUS_PAGE);
    const long long at = page < 0 ? 0 : ((((long long)page * c.Hkv + h) << c.page_shift) + (s & (c.page - 1))) * c.D + p * 16;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
      if (page >= 0) {
        const void* from = side ? c.v : c.k;
        if constexpr (F8) {
          const uint4 v = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(from) + at));
          const float scale = (side ? c.vs : c.ks)[(long long)page * c.Hkv + h];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float f[4];
            e4m3_widen(w[j], f);
            o[2 * j] = pack_io2<F16>(f[0] * scale, f[1] * scale);
            o[2 * j + 1] = pack_io2<F16>(f[2] * scale, f[3] * scale);
          }
          lo = make_uint4(o[0], o[1], o[2], o[3]);
          hi = make_uint4(o[4], o[5], o[6], o[7]);
        } else {
          const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(from) + at);
          lo = __ldcs(q);
          hi = __ldcs(q + 1);
        }
      }
      uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(side ? a.v_out : a.k_out) + row * c.D + p * 16);
      to[0] = lo;
      to[1] = hi;
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
  size_t smem = 0;
  if (c.f8) {
    pl.pages_touched = (a.T + c.page - 2) / c.page + 1;  // T rows from any slot
    pl.quant_blocks = a.B * pl.pages_touched * c.Hkv * 2;
    smem = (size_t)(a.T < c.page ? a.T : c.page) * c.D * 4;
  }
  const bool wide = a.rot % 16 == 0;
  pl.n_heads = a.Hq + (c.f8 ? 0 : 2 * c.Hkv);
  pl.groups = c.D / (wide ? 16 : 2);
  pl.n_items = (long long)a.B * a.T * pl.groups;
  const long long blocks = (pl.n_items + THREADS - 1) / THREADS;
  pl.heads = blocks * ceil_div(pl.n_heads, 8) < num_sms ? 2 : 8;
  pl.head_groups = ceil_div(pl.n_heads, pl.heads);
  pl.item_blocks = pl.n_heads == 0 ? 0 : (int)(blocks < num_sms * 16ll ? blocks : num_sms * 16ll);
  pl.vec_q = a.Hq > 0 && rows_aligned(a.q, a.qs);
  pl.vec_qo = a.Hq > 0 && rows_aligned(a.q_out, a.qos);
  pl.vec_k = rows_aligned(a.k, a.kst);
  pl.vec_v = rows_aligned(a.v, a.vst);
  const unsigned grid = (unsigned)(pl.quant_blocks + pl.item_blocks * pl.head_groups);
  if (grid == 0) return cudaSuccess;
  auto* kernel = a.f16 ? (wide ? kv_append_kernel<true, 8> : kv_append_kernel<true, 1>)
                       : (wide ? kv_append_kernel<false, 8> : kv_append_kernel<false, 1>);
  return launch_kernel(kernel, dim3(grid), dim3(THREADS), smem, s, false, a, pl);
}

cudaError_t launch_kv_gather(const KvGatherArgs& a, cudaStream_t s, int num_sms) {
  const long long items = (long long)a.B * a.c.Hkv * a.S * (a.c.D / 16);
  if (items == 0) return cudaSuccess;
  const long long blocks = (items + 255) / 256;
  const unsigned grid = (unsigned)(blocks < num_sms * 64ll ? blocks : num_sms * 64ll);
  auto* kernel = a.c.f8 ? (a.f16 ? kv_gather_kernel<true, true> : kv_gather_kernel<true, false>)
                        : kv_gather_kernel<false, false>;
  return launch_kernel(kernel, dim3(grid), dim3(256), 0, s, false, a, items);
}

}  // namespace sdpa

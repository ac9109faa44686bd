// sdpa_rope.cu -- the rotary embedding of queries and keys, and its gradient.
//
// Column pairs (a, b) of the first rot_dim columns of a row at position t turn by
// the angle t * f[i] (i the pair's index, f in radians per position):
//   a' = mult * (a cos - b sin),   b' = mult * (b cos + a sin);
// the pair is columns (i, i + rot_dim / 2), or (2 i, 2 i + 1) when interleaved,
// and the columns past rot_dim pass through. The gradient is the transposed
// rotation: the same with -sin.
//
// Angles. A position times a frequency in fp32 loses the angle itself far into
// a context (at position 10^6 an fp32 angle is off by 0.03). Here each frequency
// becomes a 64-bit fraction of a turn, f / (2 pi) * 2^64 (taken from the fp64
// frequency: 53 bits), and the position multiplies it in wrapping 64-bit
// integers: the product's upper 32 bits are the angle in turns modulo 1, off by
// t * 2^-54 turns of f's own rounding and 2^-33 of the cut. They convert to fp32 in
// [-1/2, 1/2) turns (rounded once, 2^-25 relative) and go through sincospif.
//
// Cost. Every element is read once and written once; the angle work of a
// (token, pair) is shared by the heads a thread walks. So the bound is memory,
// 4 bytes an element.
//
// Layout. A thread owns one token's two pieces of 8 columns: eight pairs, two 16-byte loads
// and two 16-byte stores per head, and keeps their sines and cosines in registers while
// it walks its heads, whose loads it issues together. (Pieces of 4 or 2 columns where the
// rotated width or the rows' alignment does not allow 8.) Consecutive threads take
// consecutive column groups, then tokens. Tensors come with any strides of batch,
// head and position (the projection's (B, S, H, D) as a transposed view, say), so
// that no separate transposition is needed before or after.
#include <cuda.h>

#include "common.cuh"
#include "ptx.cuh"

namespace sdpa {

namespace {

constexpr int THREADS = 256;

struct RopeTensor {
  const uint16_t* x;
  uint16_t* y;
  long long xs[3], ys[3];  // element strides of batch, head, position
  int H;
};

struct RopeParams {
  RopeTensor t[2];         // queries, keys (t[1].H may be 0)
  const double* freq;      // (rot / 2,) radians per position
  const int32_t* positions;  // or null: offset + s
  long long pos_bstride;   // 0: one row of positions for every batch row
  int offset;
  int B, S, D, rot;
  int sign;                // +1, or -1 for the gradient
  float mult;
};

// 2^64 * f / (2 pi) modulo 2^64, for any finite f.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  double t = f * 0.15915494309189533577;
  t -= floor(t);
  // [0, 1] in two 32-bit pieces (a product by 2^64 may round to 2^64).
  const double hi = floor(t * 4294967296.0);
  const double lo = (t * 4294967296.0 - hi) * 4294967296.0;
  return ((uint64_t)hi << 32) + (uint64_t)lo;
}

__device__ __forceinline__ void angle_sin_cos(uint64_t turn, int pos, float& sn, float& cs) {
  const uint64_t a = turn * (uint64_t)(int64_t)pos;
  sincospif((float)(int32_t)(a >> 32) * 4.6566128730773926e-10f, &sn, &cs);  // 2^-31: half turns
}

template <bool F16>
__device__ __forceinline__ float io_f32(uint16_t v) {
  return F16 ? __half2float(__ushort_as_half(v)) : __uint_as_float((uint32_t)v << 16);
}

// Head h of the call's H0 + H1 heads: its tensor and the head's index there.
__device__ __forceinline__ const RopeTensor& rope_head(const RopeParams& p, int h, int& hh) {
  const bool second = h >= p.t[0].H;
  hh = second ? h - p.t[0].H : h;
  return p.t[second ? 1 : 0];
}

// A piece of VW columns (VW / 2 words), loaded and stored in one access.
template <int VW>
struct Piece {
  uint32_t w[VW / 2];
};
template <int VW>
__device__ __forceinline__ Piece<VW> ld_piece(const uint16_t* p) {
  Piece<VW> v;
  if constexpr (VW == 8) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    v.w[0] = x.x, v.w[1] = x.y, v.w[2] = x.z, v.w[3] = x.w;
  } else if constexpr (VW == 4) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    v.w[0] = x.x, v.w[1] = x.y;
  } else {
    v.w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
  return v;
}
template <int VW>
__device__ __forceinline__ void st_piece(uint16_t* p, const Piece<VW>& v) {
  if constexpr (VW == 8) *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
  else if constexpr (VW == 4) *reinterpret_cast<uint2*>(p) = make_uint2(v.w[0], v.w[1]);
  else *reinterpret_cast<uint32_t*>(p) = v.w[0];
}

// rot a multiple of 2 VW, D of VW, every row aligned to a piece. A work item is (token,
// column group), a group being VW pairs, or two pass-through pieces (one, at an odd end);
// blockIdx.y selects `heads` consecutive heads.
template <bool F16, bool INTER, int VW>
__global__ void __launch_bounds__(THREADS) rope_vec(const RopeParams p, int heads, long long n_items) {
  constexpr int UNROLL = 4, NW = VW / 2;
  __shared__ uint64_t turns[256];  // rot <= 512
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < half; i += THREADS) turns[i] = turn_fraction(p.freq[i]);
  __syncthreads();
  const int groups = (p.D + 2 * VW - 1) / (2 * VW), rot_groups = p.rot / (2 * VW);
  const int H = p.t[0].H + p.t[1].H;
  const int h0 = blockIdx.y * heads, h1 = min(h0 + heads, H);
  for (long long it = (long long)blockIdx.x * THREADS + threadIdx.x; it < n_items;
       it += (long long)gridDim.x * THREADS) {
    const int c = (int)(it % groups);
    const long long tok = it / groups;
    const int s = (int)(tok % p.S), b = (int)(tok / p.S);
    // This thread's two pieces: the pairs' first and second halves, or two neighbouring
    // pieces (interleaved, and past the rotated part).
    const bool rotated = c < rot_groups;
    const int c0 = (rotated && !INTER) ? c * VW : c * 2 * VW;
    const int c1 = (rotated && !INTER) ? half + c * VW : c * 2 * VW + VW;
    const bool two = c1 < p.D;
    float sn[VW], cs[VW];
    if (rotated) {
      const int pos = p.positions ? p.positions[b * p.pos_bstride + s] : p.offset + s;
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        angle_sin_cos(turns[c * VW + i], pos, sn[i], cs[i]);
        sn[i] *= p.sign > 0 ? p.mult : -p.mult;
        cs[i] *= p.mult;
      }
    }
    for (int h = h0; h < h1; h += UNROLL) {
      Piece<VW> u[UNROLL], w[UNROLL];
#pragma unroll
      for (int j = 0; j < UNROLL; ++j) {
        if (h + j >= h1) continue;
        int hh;
        const RopeTensor& t = rope_head(p, h + j, hh);
        const uint16_t* x = t.x + b * t.xs[0] + hh * t.xs[1] + s * t.xs[2];
        u[j] = ld_piece<VW>(x + c0);
        if (two) w[j] = ld_piece<VW>(x + c1);
      }
#pragma unroll
      for (int j = 0; j < UNROLL; ++j) {
        if (h + j >= h1) continue;
        int hh;
        const RopeTensor& t = rope_head(p, h + j, hh);
        uint16_t* y = t.y + b * t.ys[0] + hh * t.ys[1] + s * t.ys[2];
        if (rotated) {
          uint32_t(&a)[NW] = u[j].w;
          uint32_t(&z)[NW] = w[j].w;
#pragma unroll
          for (int i = 0; i < NW; ++i) {
            if (INTER) {  // a word is a pair
              const float a0 = io_lo<F16>(a[i]), b0 = io_hi<F16>(a[i]);
              const float a1 = io_lo<F16>(z[i]), b1 = io_hi<F16>(z[i]);
              a[i] = pack_io2<F16>(a0 * cs[i] - b0 * sn[i], b0 * cs[i] + a0 * sn[i]);
              z[i] = pack_io2<F16>(a1 * cs[NW + i] - b1 * sn[NW + i], b1 * cs[NW + i] + a1 * sn[NW + i]);
            } else {
              const float a0 = io_lo<F16>(a[i]), a1 = io_hi<F16>(a[i]);
              const float b0 = io_lo<F16>(z[i]), b1 = io_hi<F16>(z[i]);
              const int e = 2 * i;
              a[i] = pack_io2<F16>(a0 * cs[e] - b0 * sn[e], a1 * cs[e + 1] - b1 * sn[e + 1]);
              z[i] = pack_io2<F16>(b0 * cs[e] + a0 * sn[e], b1 * cs[e + 1] + a1 * sn[e + 1]);
            }
          }
        }
        st_piece<VW>(y + c0, u[j]);
        if (two) st_piece<VW>(y + c1, w[j]);
      }
    }
  }
}

// Any even rot, odd D and odd alignments: one pair (or two pass-through columns) a
// thread, element loads.
template <bool F16>
__global__ void __launch_bounds__(THREADS) rope_pairs(const RopeParams p, int interleaved, int heads,
                                                      long long n_items) {
  __shared__ uint64_t turns[256];
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < half; i += THREADS) turns[i] = turn_fraction(p.freq[i]);
  __syncthreads();
  const int per_row = half + (p.D - p.rot + 1) / 2;
  const int H = p.t[0].H + p.t[1].H;
  const int h0 = blockIdx.y * heads, h1 = min(h0 + heads, H);
  for (long long it = (long long)blockIdx.x * THREADS + threadIdx.x; it < n_items;
       it += (long long)gridDim.x * THREADS) {
    const int c = (int)(it % per_row);
    const long long tok = it / per_row;
    const int s = (int)(tok % p.S), b = (int)(tok / p.S);
    const bool rotated = c < half;
    const int c0 = rotated ? (interleaved ? 2 * c : c) : p.rot + 2 * (c - half);
    const int c1 = rotated ? (interleaved ? 2 * c + 1 : c + half) : c0 + 1;
    float sn = 0.f, cs = 0.f;
    if (rotated) {
      const int pos = p.positions ? p.positions[b * p.pos_bstride + s] : p.offset + s;
      angle_sin_cos(turns[c], pos, sn, cs);
      sn *= p.sign > 0 ? p.mult : -p.mult;
      cs *= p.mult;
    }
    for (int h = h0; h < h1; ++h) {
      int hh;
      const RopeTensor& t = rope_head(p, h, hh);
      const uint16_t* x = t.x + b * t.xs[0] + hh * t.xs[1] + s * t.xs[2];
      uint16_t* y = t.y + b * t.ys[0] + hh * t.ys[1] + s * t.ys[2];
      if (rotated) {
        const float a = io_f32<F16>(x[c0]), z = io_f32<F16>(x[c1]);
        const uint32_t w = pack_io2<F16>(a * cs - z * sn, z * cs + a * sn);
        y[c0] = (uint16_t)(w & 0xFFFFu);
        y[c1] = (uint16_t)(w >> 16);
      } else {
        const uint16_t a = x[c0], z = c1 < p.D ? x[c1] : (uint16_t)0;
        y[c0] = a;
        if (c1 < p.D) y[c1] = z;
      }
    }
  }
}

// The largest piece (8, 4 or 2 columns) that every row of the tensor is aligned to; 0: none.
int piece_of(const void* base, const long long (&st)[3]) {
  for (int vw = 8; vw >= 2; vw /= 2)
    if (reinterpret_cast<uintptr_t>(base) % (2 * vw) == 0 && st[0] % vw == 0 && st[1] % vw == 0 && st[2] % vw == 0)
      return vw;
  return 0;
}

template <bool F16, bool INTER>
void launch_vec(const RopeParams& p, int vw, int heads, long long items, dim3 grid, cudaStream_t s) {
  if (vw == 8) rope_vec<F16, INTER, 8><<<grid, THREADS, 0, s>>>(p, heads, items);
  else if (vw == 4) rope_vec<F16, INTER, 4><<<grid, THREADS, 0, s>>>(p, heads, items);
  else rope_vec<F16, INTER, 2><<<grid, THREADS, 0, s>>>(p, heads, items);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream, int num_sms) {
  RopeParams p{};
  int vw = 8;  // columns of a piece: 8, 4 or 2; 0: pair by pair
  while (vw > 1 && (a.rot % (2 * vw) != 0 || a.D % vw != 0)) vw /= 2;
  if (vw == 1) vw = 0;
  for (int i = 0; i < 2; ++i) {
    RopeTensor& t = p.t[i];
    t.H = a.H[i];
    if (t.H == 0) continue;
    t.x = static_cast<const uint16_t*>(a.x[i]);
    t.y = static_cast<uint16_t*>(a.y[i]);
    for (int j = 0; j < 3; ++j) {
      t.xs[j] = a.xs[3 * i + j];
      t.ys[j] = a.ys[3 * i + j];
    }
    for (const int fit : {piece_of(t.x, t.xs), piece_of(t.y, t.ys)}) vw = fit < vw ? fit : vw;
  }
  p.freq = a.freq;
  p.positions = a.positions;
  p.pos_bstride = a.pos_bstride;
  p.offset = a.offset;
  p.B = a.B;
  p.S = a.S;
  p.D = a.D;
  p.rot = a.rot;
  p.sign = a.inverse ? -1 : 1;
  p.mult = a.mult;
  const int H = a.H[0] + a.H[1];
  const long long tokens = (long long)a.B * a.S;
  const long long items = tokens * (vw ? (a.D + 2 * vw - 1) / (2 * vw) : a.rot / 2 + (a.D - a.rot + 1) / 2);
  const long long blocks = (items + THREADS - 1) / THREADS;
  // Heads a thread walks, sharing its sines and cosines: 8 (rope_batch 53.4 us, against
  // 58.1 with 4 and 80.4 with 2), but 2 where 8 leave SMs without a block, a short call's
  // time being that of one thread (16 tokens of 40 heads 3.3 us in a graph, against 5.0).
  const int heads = blocks * ceil_div(H, 8) < num_sms ? 2 : 8;
  const dim3 grid((unsigned)(blocks < num_sms * 64ll ? blocks : num_sms * 64ll), (unsigned)ceil_div(H, heads));
  if (vw == 0) {
    if (a.f16) rope_pairs<true><<<grid, THREADS, 0, stream>>>(p, a.interleaved, heads, items);
    else rope_pairs<false><<<grid, THREADS, 0, stream>>>(p, a.interleaved, heads, items);
  } else if (a.f16) {
    if (a.interleaved) launch_vec<true, true>(p, vw, heads, items, grid, stream);
    else launch_vec<true, false>(p, vw, heads, items, grid, stream);
  } else {
    if (a.interleaved) launch_vec<false, true>(p, vw, heads, items, grid, stream);
    else launch_vec<false, false>(p, vw, heads, items, grid, stream);
  }
  return cudaGetLastError();
}

}  // namespace sdpa

// sdpa_cached_rows_16.cu -- the few-rows attention (sdpa_cached_rows.cuh) over caches of bf16 and
// fp16, and the merge of the parts of cut segments (cached.cuh).
#include "sdpa_cached_rows.cuh"

namespace sdpa {

namespace {

// The parts of a cut segment weighed by their sums, in the shares' order. WARPS > 1 (few rows, which may be
// cut into very many parts): block (segment, row), the parts dealt out to its warps. WARPS 1 (many rows, in a few
// parts): block (x, y) has rows 4 y .. 4 y + 3, one a warp, of the segment that share x + 1 is the first to
// begin in the middle of.
template <bool IOF, int WARPS>
__global__ void __launch_bounds__(WARPS == 1 ? 128 : 32 * WARPS) cached_merge_kernel(const CachedParams p) {
  constexpr bool WIDE = WARPS > 1;
  __shared__ float4 sh_y[WARPS][32];
  __shared__ float sh_m[WARPS], sh_l[WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = WIDE ? blockIdx.y : blockIdx.y * 4 + warp;
  const int4 cut = p.cuts[WIDE ? blockIdx.x : blockIdx.x + 1];
  if (cut.x < 0) return;
  const int e = cut.x / p.c.Hkv, kvh = cut.x % p.c.Hkv, b = e / p.n_rt, r = (e % p.n_rt) * p.tile_rows + row;
  if (r >= p.R) return;
  const int n = cut.z - cut.y + 1, step = WARPS, c = lane * 4;
  auto part = [&](int i) {  // the first share left its part in slot 1: it does not finish the segment
    return ((long long)(cut.y + i) * 2 + (i == 0 ? 1 : 0)) * p.part_rows + row;
  };
  float m = -INFINITY, l = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i0 = WIDE ? warp : 0; i0 < n; i0 += 8 * step) {
    float lse[8];
    float4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {  // eight parts' loads at once
      const int i = i0 + k * step;
      lse[k] = -INFINITY;
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        lse[k] = p.part_lse[part(i)];
        if (c < p.D) v[k] = *reinterpret_cast<const float4*>(p.part_o + part(i) * p.D + c);
      }
    }
    float mx = m;
#pragma unroll
    for (int k = 0; k < 8; ++k) mx = fmaxf(mx, lse[k]);
    if (mx == -INFINITY) continue;
    const float a = ex2_approx(m - mx);
    l *= a;
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] *= a;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float f = ex2_approx(lse[k] - mx);
      l += f;
      y[0] = fmaf(f, v[k].x, y[0]), y[1] = fmaf(f, v[k].y, y[1]), y[2] = fmaf(f, v[k].z, y[2]), y[3] = fmaf(f, v[k].w, y[3]);
    }
    m = mx;
  }
  if constexpr (WIDE) {
    sh_y[warp][lane] = make_float4(y[0], y[1], y[2], y[3]);
    if (lane == 0) sh_m[warp] = m, sh_l[warp] = l;
    __syncthreads();
    if (warp != 0) return;
    m = sh_m[0];
#pragma unroll
    for (int k = 1; k < WARPS; ++k) m = fmaxf(m, sh_m[k]);
    l = y[0] = y[1] = y[2] = y[3] = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      const float f = sh_m[k] == -INFINITY ? 0.f : ex2_approx(sh_m[k] - m);
      const float4 v = sh_y[k][lane];
      l = fmaf(f, sh_l[k], l);
      y[0] = fmaf(f, v.x, y[0]), y[1] = fmaf(f, v.y, y[1]), y[2] = fmaf(f, v.z, y[2]), y[3] = fmaf(f, v.w, y[3]);
    }
  }
  float fs;
  const float lse2 = m == -INFINITY ? -INFINITY : m + __log2f(l);
  const float all = cached_with_sink(p, kvh * p.G + r / p.Sq, lse2, fs);
  const float f = m == -INFINITY ? 0.f : fs / l;
  const long long orow = ((long long)b * p.c.Hkv + kvh) * p.R + r;
  if (c < p.D)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + orow * p.D + c) =
        make_uint2(pack_io2<IOF>(y[0] * f, y[1] * f), pack_io2<IOF>(y[2] * f, y[3] * f));
  if (lane == 0) p.lse[orow] = all * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_cached_rows_16(const CachedParams& p, int mt, cudaStream_t s) {
  return p.f16 ? cached_rows::launch_type<cached_rows::F16, true>(p, mt, s)
               : cached_rows::launch_type<cached_rows::BF16, false>(p, mt, s);
}

cudaError_t cached_rows_16_setup() {
  const cudaError_t e = cached_rows::setup_type<cached_rows::F16, true>();
  return e != cudaSuccess ? e : cached_rows::setup_type<cached_rows::BF16, false>();
}

cudaError_t launch_cached_merge(const CachedParams& p, cudaStream_t s) {
  if (p.n_shares < 2) return cudaSuccess;  // one share: nothing is cut
  const int rows = p.R < p.tile_rows ? p.R : p.tile_rows;
  if (p.tile_rows > 32) {
    const dim3 grid((unsigned)(p.n_shares - 1), (unsigned)ceil_div(rows, 4));
    return launch_kernel(p.f16 ? cached_merge_kernel<true, 1> : cached_merge_kernel<false, 1>, grid, dim3(128), 0, s, false, p);
  }
  // Sixteen warps a row where there are few rows to merge: their parts are many then.
  const dim3 grid((unsigned)(p.B * p.n_rt * p.c.Hkv), (unsigned)rows);
  if ((long long)grid.x * rows <= 2 * 152)
    return launch_kernel(p.f16 ? cached_merge_kernel<true, 16> : cached_merge_kernel<false, 16>, grid, dim3(512), 0, s, false, p);
  return launch_kernel(p.f16 ? cached_merge_kernel<true, 4> : cached_merge_kernel<false, 4>, grid, dim3(128), 0, s, false, p);
}

}  // namespace sdpa

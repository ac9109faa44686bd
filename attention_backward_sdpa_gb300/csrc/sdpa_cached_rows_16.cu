// sdpa_cached_rows_16.cu -- the few-rows attention (sdpa_cached_rows.cuh) over caches of bf16 and
// fp16, and the merge of the parts of cut segments (cached.cuh).
#include "sdpa_cached_rows.cuh"

namespace sdpa {

namespace {

// Block (x, y): rows 4 y .. 4 y + 3 of a tile, one a warp. x < n_ctas - 1: the segment that share
// x + 1 begins in the middle of, if it is the first to do so; its parts weighed by their sums,
// in the shares' order. Past that, entry x - (n_ctas - 1): the rows of one that visits no unit.
template <bool IOF>
__global__ void __launch_bounds__(128) cached_merge_kernel(const CachedParams p) {
  __shared__ CachedStart sh_start;
  __shared__ long long sh_sum[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = blockIdx.y * 4 + warp;
  uint16_t* const out = static_cast<uint16_t*>(p.o);
  if ((int)blockIdx.x >= p.n_ctas - 1) {
    pdl_wait_prior_grid();
    const int e = blockIdx.x - (p.n_ctas - 1), b = e / p.n_rt, r = (e % p.n_rt) * p.tile_rows + row;
    if (r >= p.R || cached_bounds(p, b, e % p.n_rt).n > 0) return;
    for (int h = 0; h < p.c.Hkv; ++h) {
      const long long orow = ((long long)b * p.c.Hkv + h) * p.R + r;
      if (lane * 4 < p.D) *reinterpret_cast<uint2*>(out + orow * p.D + lane * 4) = make_uint2(0u, 0u);
      if (lane == 0) p.lse[orow] = p.sink ? p.sink[h * p.G + r / p.Sq] : -INFINITY;
    }
    return;
  }
  const int cta = blockIdx.x + 1;
  const CachedStart st = cached_start<128>(p, &sh_start, sh_sum, false,
                                           [&](long long T) { return share_begin(T, p.n_ctas, cta); });
  pdl_wait_prior_grid();
  if (st.e < 0) return;  // nothing from here on
  const int b = st.e / p.n_rt, rt = st.e % p.n_rt;
  const int n = cached_bounds(p, b, rt).n;
  const int kvh = (int)((st.at - st.te) / n);
  const long long begin = st.te + (long long)kvh * n;
  if (st.at == begin || share_begin(st.T, p.n_ctas, cta - 1) > begin) return;  // not cut here, or cut before
  const int r = rt * p.tile_rows + row;
  if (r >= p.R) return;
  // The segment's shares: cta - 1 (or, where that one is empty, the one that has its first unit) .. last.
  const int first = share_of(st.T, p.n_ctas, begin), last = share_of(st.T, p.n_ctas, begin + n - 1);
  auto part = [&](int i) {  // the first share left its part in slot 1: it does not finish the segment
    return ((long long)i * 2 + (i == first ? 1 : 0)) * p.tile_rows + row;
  };
  // (shares between first and last that hold no unit: none, as T >= n_ctas wherever a segment is cut twice or more,
  // and a share without units lies before a unit's begin)
  float M = -INFINITY;
  for (int i = first + lane; i <= last; i += 32)
    if (share_begin(st.T, p.n_ctas, i) < share_begin(st.T, p.n_ctas, i + 1)) M = fmaxf(M, p.part_lse[part(i)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float sum = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
  const int c = lane * 4;
  if (M != -INFINITY) {
    for (int i0 = first; i0 <= last; i0 += 32) {
      const int mine = i0 + lane;
      float wgt = 0.f;
      if (mine <= last && share_begin(st.T, p.n_ctas, mine) < share_begin(st.T, p.n_ctas, mine + 1))
        wgt = ex2_approx(p.part_lse[part(mine)] - M);
      sum += wgt;
      const int here = min(32, last - i0 + 1);
#pragma unroll 4
      for (int k = 0; k < here; ++k) {
        const float f = __shfl_sync(0xffffffffu, wgt, k);
        if (c < p.D && f != 0.f) {
          const float4 v = *reinterpret_cast<const float4*>(p.part_o + part(i0 + k) * p.D + c);
          y[0] = fmaf(f, v.x, y[0]), y[1] = fmaf(f, v.y, y[1]), y[2] = fmaf(f, v.z, y[2]), y[3] = fmaf(f, v.w, y[3]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  float fs;
  const float lse2 = M == -INFINITY ? -INFINITY : M + __log2f(sum);
  const float all = cached_with_sink(p, kvh * p.G + r / p.Sq, lse2, fs);
  const float f = M == -INFINITY ? 0.f : fs / sum;
  const long long orow = ((long long)b * p.c.Hkv + kvh) * p.R + r;
  if (c < p.D)
    *reinterpret_cast<uint2*>(out + orow * p.D + c) =
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
  const dim3 grid((unsigned)(p.n_ctas - 1 + p.B * p.n_rt), (unsigned)ceil_div(p.R < p.tile_rows ? p.R : p.tile_rows, 4));
  return p.f16 ? launch_kernel(cached_merge_kernel<true>, grid, dim3(128), 0, s, true, p)
               : launch_kernel(cached_merge_kernel<false>, grid, dim3(128), 0, s, true, p);
}

}  // namespace sdpa

// sdpa_cached_rows_16.cu -- the few-rows attention (sdpa_cached_rows.cuh) over caches of bf16 and
// fp16, and the merge of the parts of cut segments (cached.cuh).
#include "sdpa_cached_rows.cuh"

namespace sdpa {

namespace {

// The parts of a cut segment weighed by their sums, in the shares' order. A half-warp reads a part's row, eight
// columns a lane, four parts at once. GROUPS half-warps share a row's parts (and are joined in their order):
// 1: many rows, in a few parts: block (x, y) has rows 8 y .. 8 y + 7 of the segment that share x + 1 is the first to
// begin in the middle of; else block (x, y) has segment x, and rows 4 y .. 4 y + 3 with 2, row y with 8 or 32.
struct Weighed {
  float m, l, y[8];
};
__device__ __forceinline__ void join(Weighed& a, float m, float l, const float* y) {
  const float mx = fmaxf(a.m, m);
  if (mx == -INFINITY) return;
  const float fa = ex2_approx(a.m - mx), fb = ex2_approx(m - mx);
  a.m = mx;
  a.l = fmaf(fa, a.l, fb * l);
#pragma unroll
  for (int i = 0; i < 8; ++i) a.y[i] = fmaf(fa, a.y[i], fb * y[i]);
}
__device__ __forceinline__ void join_halves(Weighed& a) {  // (the first half's parts first)
  Weighed o;
  o.m = __shfl_xor_sync(0xffffffffu, a.m, 16);
  o.l = __shfl_xor_sync(0xffffffffu, a.l, 16);
#pragma unroll
  for (int i = 0; i < 8; ++i) o.y[i] = __shfl_xor_sync(0xffffffffu, a.y[i], 16);
  join(a, o.m, o.l, o.y);
}
template <bool IOF, int GROUPS>
__global__ void __launch_bounds__(GROUPS == 32 ? 512 : 128) cached_merge_kernel(const CachedParams p) {
  constexpr int WARPS = GROUPS > 2 ? GROUPS / 2 : 1;  // of a row
  __shared__ float4 sh_y[WARPS][2][16];
  __shared__ float2 sh_ml[WARPS];
  const int warp = threadIdx.x >> 5, half = threadIdx.x >> 4, c = (threadIdx.x & 15) * 8;
  const int row = GROUPS == 1 ? blockIdx.y * 8 + half : GROUPS == 2 ? blockIdx.y * 4 + warp : blockIdx.y;
  const int4 cut = p.cuts[GROUPS == 1 ? blockIdx.x + 1 : blockIdx.x];
  if (cut.x < 0) return;
  const int e = cut.x / p.c.Hkv, kvh = cut.x % p.c.Hkv, b = e / p.n_rt, r = (e % p.n_rt) * p.tile_rows + row;
  if (r >= p.R) return;  // (all of the threads that meet below)
  const int n = cut.z - cut.y + 1;
  const long long apart = 2ll * p.part_rows, at0 = cut.y * apart + row;  // part i: at0 + i * apart
  Weighed a{-INFINITY, 0.f, {}};
  for (int i0 = GROUPS == 1 ? 0 : half % GROUPS; i0 < n; i0 += 4 * GROUPS) {
    float lse[4];
    float4 v[4][2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * GROUPS;
      lse[k] = -INFINITY;
      v[k][0] = v[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        // (the first share left its part in slot 1: it does not finish the segment)
        const long long at = at0 + i * apart + (i == 0 ? p.part_rows : 0);
        lse[k] = p.part_lse[at];
        if (c < p.D) {
          const float4* const from = reinterpret_cast<const float4*>(p.part_o + at * p.D + c);
          v[k][0] = from[0];
          v[k][1] = from[1];
        }
      }
    }
    const float mx = fmaxf(fmaxf(fmaxf(lse[0], lse[1]), fmaxf(lse[2], lse[3])), a.m);
    if (mx == -INFINITY) continue;
    const float f = ex2_approx(a.m - mx);
    a.m = mx;
    a.l *= f;
#pragma unroll
    for (int q = 0; q < 8; ++q) a.y[q] *= f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i0 + k * GROUPS >= n) break;
      const float w = ex2_approx(lse[k] - mx);
      a.l += w;
      a.y[0] = fmaf(w, v[k][0].x, a.y[0]), a.y[1] = fmaf(w, v[k][0].y, a.y[1]);
      a.y[2] = fmaf(w, v[k][0].z, a.y[2]), a.y[3] = fmaf(w, v[k][0].w, a.y[3]);
      a.y[4] = fmaf(w, v[k][1].x, a.y[4]), a.y[5] = fmaf(w, v[k][1].y, a.y[5]);
      a.y[6] = fmaf(w, v[k][1].z, a.y[6]), a.y[7] = fmaf(w, v[k][1].w, a.y[7]);
    }
  }
  if constexpr (GROUPS >= 2) {
    __syncwarp();
    join_halves(a);
  }
  if constexpr (WARPS > 1) {
    const int lane16 = threadIdx.x & 15;
    sh_y[warp][half & 1][lane16] = half & 1 ? make_float4(a.y[4], a.y[5], a.y[6], a.y[7]) : make_float4(a.y[0], a.y[1], a.y[2], a.y[3]);
    if (lane16 == 0) sh_ml[warp] = make_float2(a.m, a.l);
    __syncthreads();
    if (warp != 0) return;
    float mx = sh_ml[0].x;  // (each half of the warp all of it: the loads are under way together)
#pragma unroll
    for (int k = 1; k < WARPS; ++k) mx = fmaxf(mx, sh_ml[k].x);
    a = Weighed{mx, 0.f, {}};
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      const float w = sh_ml[k].x == -INFINITY ? 0.f : ex2_approx(sh_ml[k].x - mx);
      const float4 u = sh_y[k][0][lane16], v = sh_y[k][1][lane16];
      a.l = fmaf(w, sh_ml[k].y, a.l);
      a.y[0] = fmaf(w, u.x, a.y[0]), a.y[1] = fmaf(w, u.y, a.y[1]), a.y[2] = fmaf(w, u.z, a.y[2]), a.y[3] = fmaf(w, u.w, a.y[3]);
      a.y[4] = fmaf(w, v.x, a.y[4]), a.y[5] = fmaf(w, v.y, a.y[5]), a.y[6] = fmaf(w, v.z, a.y[6]), a.y[7] = fmaf(w, v.w, a.y[7]);
    }
  }
  if (GROUPS >= 2 && (threadIdx.x & 16) != 0) return;
  float fs;
  const float lse2 = a.m == -INFINITY ? -INFINITY : a.m + __log2f(a.l);
  const float all = cached_with_sink(p, kvh * p.G + r / p.Sq, lse2, fs);
  const float f = a.m == -INFINITY ? 0.f : fs / a.l;
  const long long orow = ((long long)b * p.c.Hkv + kvh) * p.R + r;
  if (c < p.D)
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + orow * p.D + c) =
        make_uint4(pack_io2<IOF>(a.y[0] * f, a.y[1] * f), pack_io2<IOF>(a.y[2] * f, a.y[3] * f),
                   pack_io2<IOF>(a.y[4] * f, a.y[5] * f), pack_io2<IOF>(a.y[6] * f, a.y[7] * f));
  if (c == 0) p.lse[orow] = all * 0.6931471805599453f;
}

template <bool IOF>
cudaError_t launch_merge(const CachedParams& p, cudaStream_t s) {
  const int rows = p.R < p.tile_rows ? p.R : p.tile_rows;
  if (p.tile_rows > 32)
    return launch_kernel(cached_merge_kernel<IOF, 1>, dim3((unsigned)(p.n_shares - 1), (unsigned)ceil_div(rows, 8)), dim3(128),
                         0, s, false, p);
  // Few rows: the fewer there are of them the more parts each may have.
  const unsigned segments = (unsigned)(p.B * p.n_rt * p.c.Hkv);
  if ((long long)segments * rows <= 2 * 152)
    return launch_kernel(cached_merge_kernel<IOF, 32>, dim3(segments, (unsigned)rows), dim3(512), 0, s, false, p);
  if ((long long)segments * 8 <= p.n_shares)
    return launch_kernel(cached_merge_kernel<IOF, 8>, dim3(segments, (unsigned)rows), dim3(128), 0, s, false, p);
  return launch_kernel(cached_merge_kernel<IOF, 2>, dim3(segments, (unsigned)ceil_div(rows, 4)), dim3(128), 0, s, false, p);
}

}  // namespace

cudaError_t launch_cached_rows_16(const CachedParams& p, int nr, cudaStream_t s) {
  return p.f16 ? cached_rows::launch_type<cached_rows::F16, true>(p, nr, s)
               : cached_rows::launch_type<cached_rows::BF16, false>(p, nr, s);
}

cudaError_t cached_rows_16_setup() {
  const cudaError_t e = cached_rows::setup_type<cached_rows::F16, true>();
  return e != cudaSuccess ? e : cached_rows::setup_type<cached_rows::BF16, false>();
}

cudaError_t launch_cached_merge(const CachedParams& p, cudaStream_t s) {
  if (p.n_shares < 2) return cudaSuccess;  // one share: nothing is cut
  return p.f16 ? launch_merge<true>(p, s) : launch_merge<false>(p, s);
}

}  // namespace sdpa

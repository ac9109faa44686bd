// sdpa_cache_api.cu -- host side of the cache entry points of include/sdpa_bwd.h: arguments
// checked, then one launch (attention: two, the second merges the parts of what was cut).
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "sdpa_bwd.h"
#include "cached.cuh"
#include "common.cuh"
#include "rows.h"

using namespace sdpa;

namespace {

struct CacheArgs {
  int dtype;
  const void *k, *v, *k_scale, *v_scale;
  const int32_t *table, *lens;
  int n_pages, page, max_pages, H_kv, D;
};

bool misaligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

int fill_cache(const CacheArgs& a, int io_dtype, int B, KvCacheRef& c) {
  if (io_dtype != SDPA_DTYPE_BF16 && io_dtype != SDPA_DTYPE_F16) return SDPA_ERR_INVALID;
  if (a.dtype != SDPA_DTYPE_E4M3 && a.dtype != io_dtype) return SDPA_ERR_INVALID;
  if (B <= 0 || a.H_kv <= 0 || a.D <= 0 || a.n_pages <= 0 || a.max_pages <= 0) return SDPA_ERR_INVALID;
  if (a.D % 16 != 0 || a.D > 128) return SDPA_ERR_UNSUPPORTED;
  if (a.page < 16 || a.page > 256 || (a.page & (a.page - 1)) != 0) return SDPA_ERR_UNSUPPORTED;
  // Positions, table entries and groups of 16 rows are 32-bit; element offsets 64-bit.
  if ((long long)a.max_pages * a.page >= 1ll << 31 || (long long)a.n_pages * a.H_kv * (a.page / 16) >= 1ll << 31 ||
      (long long)B * a.max_pages >= 1ll << 31)
    return SDPA_ERR_INVALID;
  if (!a.k || !a.v || !a.table || !a.lens) return SDPA_ERR_INVALID;
  const bool f8 = a.dtype == SDPA_DTYPE_E4M3;
  if (f8 != (a.k_scale != nullptr) || f8 != (a.v_scale != nullptr)) return SDPA_ERR_INVALID;
  if (misaligned(a.k, 16) || misaligned(a.v, 16)) return SDPA_ERR_ALIGN;
  for (const void* p : {a.k_scale, a.v_scale, (const void*)a.table, (const void*)a.lens})
    if (misaligned(p, 4)) return SDPA_ERR_ALIGN;
  c.k = const_cast<void*>(a.k);
  c.v = const_cast<void*>(a.v);
  c.ks = static_cast<float*>(const_cast<void*>(a.k_scale));
  c.vs = static_cast<float*>(const_cast<void*>(a.v_scale));
  c.table = a.table;
  c.lens = a.lens;
  c.n_pages = a.n_pages;
  c.page = a.page;
  c.page_shift = 0;
  while ((1 << c.page_shift) < a.page) ++c.page_shift;
  c.max_pages = a.max_pages;
  c.Hkv = a.H_kv;
  c.D = a.D;
  c.f8 = f8 ? 1 : 0;
  return SDPA_OK;
}

struct Span {
  uintptr_t lo, hi;  // bytes [lo, hi)
};
bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }
Span span_of(const void* p, size_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return p ? Span{lo, lo + bytes} : Span{1, 0};  // (NULL meets nothing)
}
Span span_of(const RopeRows& r) { return {(uintptr_t)(r.base * 2), (uintptr_t)(r.end * 2)}; }
// Whether something written shares a byte with anything else that is written, or read (NULL: nothing).
bool writes_meet(std::initializer_list<Span> writes, std::initializer_list<Span> reads) {
  for (const Span& w : writes) {
    for (const Span& r : reads)
      if (meet(w, r)) return true;
    for (const Span& o : writes)
      if (&o < &w && meet(w, o)) return true;
  }
  return false;
}
size_t cache_bytes(const KvCacheRef& c) { return (size_t)c.n_pages * c.Hkv * c.page * c.D * (c.f8 ? 1 : 2); }

// How a call over the cache is cut, from its sizes alone (not from the device it runs on, so that
// neither the workspace nor any result depends on that).
struct CachedPlan {
  int tile_rows, n_rt, tk, n_ctas, n_shares, part_rows, nr;
  size_t o_bytes, lse_bytes, bytes;
};
constexpr int SHARE_SMS = 152;  // SMs of a GB300
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

CachedPlan cached_plan(long long B, int H_q, int H_kv, int S_q, int D, bool f8, long long max_keys) {
  CachedPlan c{};
  const long long R = (long long)(H_q / H_kv) * S_q;
  // 8-row tiles of the few-rows kernel; 0: the many-rows kernel. For 17 to 32 rows of more than 64 columns that one
  // is the faster, though its tiles are of 128 and the codes' bytes would take 89 us: 214 us against 252 for 32 rows a
  // head, 64 sequences of up to 8,192 keys (8 bits: 234, 246), 13.4 against 16.1 over 2,000 keys of one. Of 64
  // columns it is not where keys are many: 69 against 61 us over 131,072 keys, 135 against 121 for the batch (8 bits: 72
  // against 58, 144 against 120; over 2,000 keys 13.0 against 14.2). With 16 rows of 128 columns the few-rows kernel
  // takes 199 against 222 us for the batch and 98 against 91 over 131,072 keys (8 bits: 127 against 234, 60 against 80).
  c.nr = R <= 8 ? 1 : R <= 16 ? 2 : R <= 32 && D <= 64 ? 4 : 0;
  c.tile_rows = c.nr ? 8 * c.nr : 128;
  c.tk = c.nr ? cached_rows_tk(f8, c.nr) : 128;
  c.n_rt = (int)((R + c.tile_rows - 1) / c.tile_rows);
  // As many CTAs as the device holds at once (by their shared memory), fewer where there are
  // not that many units. A share is a CTA, or one of four warps of it.
  const long long units = B * c.n_rt * H_kv * ((max_keys + c.tk - 1) / c.tk), warps = c.nr ? 4 : 1;
  const long long ctas = (units + warps - 1) / warps, most = c.nr ? cached_rows_ctas(c.nr) * SHARE_SMS : SHARE_SMS;
  c.n_ctas = (int)(ctas < most ? ctas : most);
  c.n_shares = (int)(c.n_ctas * warps);
  c.part_rows = R < c.tile_rows ? (int)R : c.tile_rows;
  const size_t parts = (size_t)c.n_shares * 2 * c.part_rows;
  const size_t notes = c.nr ? (size_t)(B * c.n_rt * H_kv) : (size_t)c.n_shares;
  c.o_bytes = align256(parts * D * sizeof(float));
  c.lse_bytes = align256(parts * sizeof(float));
  c.bytes = c.o_bytes + c.lse_bytes + align256(notes * sizeof(int4));
  return c;
}

int cached_sizes(int B, int H_q, int H_kv, int S_q, int D) {
  if (B <= 0 || H_q <= 0 || H_kv <= 0 || S_q < 0 || D <= 0 || H_q % H_kv != 0) return SDPA_ERR_INVALID;
  if (D % 16 != 0 || D > 128) return SDPA_ERR_UNSUPPORTED;
  if ((long long)B * H_q * S_q * D >= 1ll << 31) return SDPA_ERR_INVALID;
  return SDPA_OK;
}

}  // namespace

extern "C" {

size_t sdpa_fwd_cached_workspace_size(int B, int H_q, int H_kv, int S_q, int D, int cache_dtype, int page_size,
                                      int max_pages) {
  if (cached_sizes(B, H_q, H_kv, S_q, D) != SDPA_OK || S_q == 0 || page_size <= 0 || max_pages <= 0) return 0;
  if ((long long)max_pages * page_size >= 1ll << 31) return 0;
  return cached_plan(B, H_q, H_kv, S_q, D, cache_dtype == SDPA_DTYPE_E4M3, (long long)max_pages * page_size).bytes;
}

int sdpa_fwd_cached(int io_dtype, int cache_dtype, const void* q, const void* k_cache, const void* v_cache,
                    const float* k_scale, const float* v_scale, const int32_t* page_table, const int32_t* seq_kv_lens,
                    const int32_t* seq_q_lens, void* o, float* lse, int B, int H_q, int H_kv, int S_q, int D,
                    int n_pages, int page_size, int max_pages, float scale, int causal, int window_left,
                    int first_keys, const float* sink, float softcap, const float* alibi_slopes, void* workspace,
                    size_t workspace_bytes, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  CachedParams p{};
  const CacheArgs ca{cache_dtype, k_cache, v_cache, k_scale, v_scale, page_table, seq_kv_lens,
                     n_pages, page_size, max_pages, H_kv, D};
  int rc = fill_cache(ca, io_dtype, B, p.c);
  if (rc == SDPA_OK) rc = cached_sizes(B, H_q, H_kv, S_q, D);
  if (rc != SDPA_OK) return rc;
  if (first_keys < 0) return SDPA_ERR_INVALID;
  if (!(scale > 0.f) || !std::isfinite(scale)) scale = 1.0f / std::sqrt((float)D);
  if (softcap != 0.f) {
    if (!(softcap > 0.f && std::isnormal(softcap))) return SDPA_ERR_INVALID;
    rc = fill_cap(softcap, scale, p.mods);
    if (rc != SDPA_OK) return rc;
  }
  if (S_q == 0) return SDPA_OK;  // no rows
  if (!q || !o || !lse) return SDPA_ERR_INVALID;
  if (misaligned(q, 16) || misaligned(o, 16)) return SDPA_ERR_ALIGN;
  for (const void* x : {(const void*)lse, (const void*)sink, (const void*)alibi_slopes, (const void*)seq_q_lens})
    if (misaligned(x, 4)) return SDPA_ERR_ALIGN;
  const CachedPlan plan = cached_plan(B, H_q, H_kv, S_q, D, p.c.f8 != 0, (long long)max_pages * page_size);
  // Units of the schedule are 32-bit.
  if ((double)B * plan.n_rt * H_kv * (((long long)max_pages * page_size + plan.tk - 1) / plan.tk) >= 2147483648.0)
    return SDPA_ERR_INVALID;
  if (workspace) {
    if (workspace_bytes < plan.bytes) return SDPA_ERR_WORKSPACE;
    if (misaligned(workspace, 256)) return SDPA_ERR_ALIGN;
  }
  const size_t rows = (size_t)B * H_q * S_q, scales = (size_t)n_pages * H_kv * 4;
  if (writes_meet({span_of(o, rows * D * 2), span_of(lse, rows * 4), span_of(workspace, plan.bytes)},
                  {span_of(q, rows * D * 2), span_of(k_cache, cache_bytes(p.c)), span_of(v_cache, cache_bytes(p.c)),
                   span_of(k_scale, scales), span_of(v_scale, scales), span_of(page_table, (size_t)B * max_pages * 4),
                   span_of(seq_kv_lens, (size_t)B * 4), span_of(seq_q_lens, (size_t)B * 4), span_of(sink, (size_t)H_q * 4),
                   span_of(alibi_slopes, (size_t)H_q * 4)}))
    return SDPA_ERR_INVALID;
  int sms = 0;
  rc = current_device_state(&p.status, &sms);
  if (rc != SDPA_OK) return rc;
  const bool own = workspace == nullptr;
  if (own && cudaMallocAsync(&workspace, plan.bytes, stream) != cudaSuccess) return SDPA_ERR_CUDA;
  p.B = B;
  p.Hq = H_q;
  p.G = H_q / H_kv;
  p.Sq = S_q;
  p.R = p.G * S_q;
  p.D = D;
  p.q = q;
  p.o = o;
  p.lse = lse;
  p.f16 = io_dtype == SDPA_DTYPE_F16 ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.causal = causal ? 1 : 0;
  p.window_left = window_left < 0 ? -1 : window_left;
  p.first_keys = window_left < 0 ? 0 : first_keys;
  p.seq_q_lens = seq_q_lens;
  p.sink = sink;
  p.mods.slopes = alibi_slopes;
  p.tile_rows = plan.tile_rows;
  p.n_rt = plan.n_rt;
  while ((1 << p.tk_shift) < plan.tk) ++p.tk_shift;
  p.n_ctas = plan.n_ctas;
  p.n_shares = plan.n_shares;
  p.share_units = plan.nr ? 8 : 1;
  p.part_rows = plan.part_rows;
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.o_bytes);
  p.cuts = reinterpret_cast<int4*>(static_cast<char*>(workspace) + plan.o_bytes + plan.lse_bytes);
  nvtxRangePushA("sdpa_fwd_cached");
  cudaError_t e = plan.nr ? (p.c.f8 ? launch_cached_rows_8(p, plan.nr, stream) : launch_cached_rows_16(p, plan.nr, stream))
                          : (p.c.f8 ? launch_cached_tiles_8(p, stream) : launch_cached_tiles_16(p, stream));
  if (e == cudaSuccess) e = launch_cached_merge(p, stream);
  nvtxRangePop();
  if (own) cudaFreeAsync(workspace, stream);
  return e == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

int sdpa_kv_append(int io_dtype, int cache_dtype, const void* q, void* q_out, const void* k, const void* v,
                   void* k_cache, void* v_cache, float* k_scale, float* v_scale, const int32_t* page_table,
                   const int32_t* seq_kv_lens, const int32_t* seq_q_lens, int B, int H_q, int H_kv, int S, int D,
                   int n_pages, int page_size, int max_pages, const long long* strides, const double* inv_freq,
                   int rot_dim, float mult, const int32_t* positions, int positions_per_batch, int n_axes,
                   const int32_t* pair_axis, int interleaved, void* stream) {
  KvAppendArgs a{};
  const CacheArgs ca{cache_dtype, k_cache, v_cache, k_scale, v_scale, page_table, seq_kv_lens,
                     n_pages, page_size, max_pages, H_kv, D};
  int rc = fill_cache(ca, io_dtype, B, a.c);
  if (rc != SDPA_OK) return rc;
  if (H_q < 0 || S < 0 || !strides || !std::isfinite(mult)) return SDPA_ERR_INVALID;
  if (rot_dim < 0 || rot_dim % 2 != 0 || rot_dim > D) return SDPA_ERR_INVALID;
  if (rot_dim > 0 && !inv_freq) return SDPA_ERR_INVALID;
  if (pair_axis && (!positions || n_axes <= 0 || n_axes > ROPE_MAX_AXES)) return SDPA_ERR_INVALID;
  if (S == 0) return SDPA_OK;  // no rows
  if (!k || !v || (H_q > 0 && (!q || !q_out))) return SDPA_ERR_INVALID;
  if ((long long)B * S * (H_q + 2ll * H_kv) >= 1ll << 31 ||
      (long long)B * (S / page_size + 2) * H_kv * 2 >= 1ll << 30)
    return SDPA_ERR_INVALID;
  for (const void* p : {q, (const void*)q_out, k, v})
    if (misaligned(p, 2)) return SDPA_ERR_ALIGN;
  if (misaligned(inv_freq, 8)) return SDPA_ERR_ALIGN;
  for (const void* p : {(const void*)positions, (const void*)pair_axis, (const void*)seq_q_lens})
    if (misaligned(p, 4)) return SDPA_ERR_ALIGN;
  long long(*const st[4])[3] = {&a.qs, &a.qos, &a.kst, &a.vst};
  const int heads[4] = {H_q, H_q, H_kv, H_kv};
  const int ext0 = B, ext2 = S;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 3; ++j) {
      (*st[i])[j] = strides[3 * i + j];
      if ((j == 0 ? ext0 : j == 1 ? heads[i] : ext2) > 1 && (*st[i])[j] < 0) return SDPA_ERR_INVALID;
    }
  // The rotated queries are the queries themselves, element by element, or share no element
  // with any tensor of the call; the cache shares none with any other.
  const RopeRows kr = rope_rows(k, a.kst, B, H_kv, S, D), vr = rope_rows(v, a.vst, B, H_kv, S, D);
  Span qs{1, 0}, qos{1, 0};
  if (H_q > 0) {
    if (!rows_apart(a.qos, B, H_q, S, D)) return SDPA_ERR_INVALID;
    const RopeRows qr = rope_rows(q, a.qs, B, H_q, S, D), qo = rope_rows(q_out, a.qos, B, H_q, S, D);
    if ((!same_rows(qr, qo) && rows_meet(qr, qo)) || rows_meet(kr, qo) || rows_meet(vr, qo)) return SDPA_ERR_INVALID;
    qs = span_of(qr);
    qos = span_of(qo);
  }
  const size_t scales = (size_t)n_pages * H_kv * 4;
  const Span kc = span_of(k_cache, cache_bytes(a.c)), vc = span_of(v_cache, cache_bytes(a.c)), ks = span_of(k_scale, scales),
             vs = span_of(v_scale, scales), table = span_of(page_table, (size_t)B * max_pages * 4),
             lens = span_of(seq_kv_lens, (size_t)B * 4), news = span_of(seq_q_lens, (size_t)B * 4),
             freq = span_of(rot_dim ? inv_freq : nullptr, (size_t)rot_dim * 4), axis = span_of(pair_axis, (size_t)rot_dim * 2),
             places = span_of(positions, (size_t)S * (positions_per_batch ? B : 1) * (pair_axis ? n_axes : 1) * 4);
  if (writes_meet({kc, vc, ks, vs}, {span_of(kr), span_of(vr), qs, qos, table, lens, news, freq, axis, places}) ||
      writes_meet({qos}, {table, lens, news, freq, axis, places}))
    return SDPA_ERR_INVALID;
  a.q = q;
  a.q_out = q_out;
  a.k = k;
  a.v = v;
  a.Hq = H_q;
  a.B = B;
  a.T = S;
  a.new_lens = seq_q_lens;
  a.freq = inv_freq;
  a.rot = rot_dim;
  a.mult = mult;
  a.positions = positions;
  a.pos_bstride = positions_per_batch ? S : 0;
  a.axis_stride = positions_per_batch ? (long long)B * S : S;
  a.pair_axis = pair_axis;
  a.n_axes = pair_axis ? n_axes : 1;
  a.f16 = io_dtype == SDPA_DTYPE_F16 ? 1 : 0;
  a.interleaved = interleaved ? 1 : 0;
  int sms = 0;
  rc = current_device_state(&a.status, &sms);
  if (rc != SDPA_OK) return rc;
  nvtxRangePushA("sdpa_kv_append");
  const cudaError_t e = launch_kv_append(a, static_cast<cudaStream_t>(stream), sms);
  nvtxRangePop();
  return e == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

int sdpa_kv_gather(int out_dtype, int cache_dtype, const void* k_cache, const void* v_cache, const float* k_scale,
                   const float* v_scale, const int32_t* page_table, const int32_t* seq_kv_lens, void* k_out,
                   void* v_out, int B, int H_kv, int S, int D, int n_pages, int page_size, int max_pages,
                   void* stream) {
  KvGatherArgs a{};
  const CacheArgs ca{cache_dtype, k_cache, v_cache, k_scale, v_scale, page_table, seq_kv_lens,
                     n_pages, page_size, max_pages, H_kv, D};
  int rc = fill_cache(ca, out_dtype, B, a.c);
  if (rc != SDPA_OK) return rc;
  if (S < 0 || S > (long long)max_pages * page_size || (long long)B * H_kv >= 1ll << 31) return SDPA_ERR_INVALID;
  if (S == 0) return SDPA_OK;  // no rows
  if (!k_out || !v_out) return SDPA_ERR_INVALID;
  if (misaligned(k_out, 16) || misaligned(v_out, 16)) return SDPA_ERR_ALIGN;
  const size_t bytes = (size_t)B * H_kv * S * D * 2;
  const size_t scales = (size_t)n_pages * H_kv * 4;
  if (writes_meet({span_of(k_out, bytes), span_of(v_out, bytes)},
                  {span_of(k_cache, cache_bytes(a.c)), span_of(v_cache, cache_bytes(a.c)), span_of(k_scale, scales),
                   span_of(v_scale, scales), span_of(page_table, (size_t)B * max_pages * 4), span_of(seq_kv_lens, (size_t)B * 4)}))
    return SDPA_ERR_INVALID;
  a.k_out = k_out;
  a.v_out = v_out;
  a.B = B;
  a.S = S;
  a.f16 = out_dtype == SDPA_DTYPE_F16 ? 1 : 0;
  int sms = 0;
  rc = current_device_state(&a.status, &sms);
  if (rc != SDPA_OK) return rc;
  nvtxRangePushA("sdpa_kv_gather");
  const cudaError_t e = launch_kv_gather(a, static_cast<cudaStream_t>(stream), sms);
  nvtxRangePop();
  return e == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

}  // extern "C"

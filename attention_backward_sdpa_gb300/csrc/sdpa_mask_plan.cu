// sdpa_mask_plan.cu -- the mask plan of document, prefix and row-range masks
// (layout in score.cuh): which keys each query row sees, as one range per row,
// with the summaries per 64-row query tile and per 128-key tile that the
// forward and backward kernels take their loop bounds from. A training step
// makes it once per batch; every layer and both directions read it.
//
//   row_ranges   the caller's lo / hi per row, clamped to [0, S_kv].
//   doc_ranges   document = maximal run of equal ids. A block scans one batch
//                row: ascending for the start of each position's run (a running
//                maximum of the positions where the id changes), descending
//                for its end (a running minimum). Row i of a document
//                [s, e) sees [s, e), or with `causal` [s, min(e, max(i + 1, s + prefix))).
//   q_summary    one warp per 64-row tile (two rows a lane, warp reductions).
//   k_summary    one warp per 128-key tile: the first and last query tile whose
//                [min lo, max hi) meets it.
//   k_exact      one block per batch row: whether lo and hi never decrease.
//   k_rows       per key, where they never do: the first row with hi above the key and
//                the last with lo at or below it, by bisection.
// A plan is 16 bytes a position and 24 per 64 of them (B 8, S 4096: 535 KB); the ids are read
// twice, and the ranges again by the last three kernels. Bound by five launches and, in the
// document form, by the scan's two passes over a batch row in one block: B 2 or 8, S 4096
// 18 and 19 us in a graph (explicit ranges 14 and 15); one row of S 16,384 35 us (17), of
// 131,072 233 us (45), 1.5 us more for every 1,024 positions of a row.
#include <climits>

#include "common.cuh"

namespace sdpa {

namespace {

constexpr int SCAN_THREADS = 1024;

__global__ void __launch_bounds__(256) mask_row_ranges(const int32_t* row_lo, const int32_t* row_hi, int Sq,
                                                       int Skv, int rows_pad, long long n_rows, int2* ranges) {
  const long long at = (long long)blockIdx.x * 256 + threadIdx.x;
  if (at >= n_rows) return;
  const int b = (int)(at / rows_pad), i = (int)(at % rows_pad);
  int lo = 0, hi = 0;
  if (i < Sq) {
    lo = min(max(row_lo[(long long)b * Sq + i], 0), Skv);
    hi = min(max(row_hi[(long long)b * Sq + i], 0), Skv);
    if (hi <= lo) lo = hi = 0;
  }
  ranges[at] = make_int2(lo, hi);
}

// Inclusive scan over the block (max when MAX, else min) of one value a thread.
template <bool MAX>
__device__ int block_scan(int v, int* warp_last) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = MAX ? max(v, u) : min(v, u);
  }
  if (lane == 31) warp_last[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = warp_last[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w = MAX ? max(w, u) : min(w, u);
    }
    warp_last[lane] = w;
  }
  __syncthreads();
  if (warp > 0) v = MAX ? max(v, warp_last[warp - 1]) : min(v, warp_last[warp - 1]);
  return v;
}

__global__ void __launch_bounds__(SCAN_THREADS)
    mask_doc_ranges(const int32_t* doc_ids, const int32_t* prefix_lens, int prefix_per_row, int causal, int S,
                    int rows_pad, int2* ranges) {
  static_assert(SCAN_THREADS == 1024, "block_scan takes 32 warps");
  __shared__ int warp_last[32];
  __shared__ int carry;
  const int b = blockIdx.x, t = threadIdx.x;
  const int32_t* ids = doc_ids ? doc_ids + (long long)b * S : nullptr;
  int2* out = ranges + (long long)b * rows_pad;
  const int chunks = (rows_pad + SCAN_THREADS - 1) / SCAN_THREADS;
  // Ascending: the start of each position's run, kept in .x until the second pass.
  if (t == 0) carry = 0;
  __syncthreads();
  for (int c = 0; c < chunks; ++c) {
    const int i = c * SCAN_THREADS + t;
    const bool edge = ids && i > 0 && i < S && ids[i] != ids[i - 1];
    const int start = max(block_scan<true>(edge ? i : 0, warp_last), carry);
    if (i < rows_pad) out[i].x = start;
    __syncthreads();  // every thread has read the carry
    if (t == SCAN_THREADS - 1) carry = start;
    __syncthreads();
  }
  // Descending: the end of each position's run (thread t takes the chunk's
  // position counted from its end, so that the same scan runs downwards).
  if (t == 0) carry = S;
  __syncthreads();
  for (int c = chunks - 1; c >= 0; --c) {
    const int i = c * SCAN_THREADS + (SCAN_THREADS - 1 - t);
    const bool edge = ids && i + 1 < S && ids[i + 1] != ids[i];
    const int end = min(block_scan<false>(edge ? i + 1 : S, warp_last), carry);
    if (i < rows_pad) {
      int lo = 0, hi = 0;
      if (i < S) {
        lo = out[i].x;
        hi = end;
        if (causal) {
          int pre = 0;
          if (prefix_lens) pre = prefix_lens[prefix_per_row ? (long long)b * S + i : b];
          pre = min(max(pre, 0), S);
          hi = min(hi, max(i + 1, lo + pre));  // lo + pre <= 2 S < 2^31
        }
      }
      out[i] = make_int2(lo, hi);
    }
    __syncthreads();
    if (t == SCAN_THREADS - 1) carry = end;
    __syncthreads();
  }
}

__global__ void __launch_bounds__(128) mask_q_summary(const int2* ranges, int Sq, int n_qt, int n_tiles,
                                                      int4* q_sum) {
  const int tile = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (tile >= n_tiles) return;
  const int rows = min(64, Sq - (tile % n_qt) * 64);
  int lo_min = INT_MAX, hi_max = 0, lo_max = 0, hi_min = INT_MAX;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = lane + 32 * j;
    if (i >= rows) continue;
    const int2 r = ranges[(long long)tile * 64 + i];
    if (r.x < r.y) {
      lo_min = min(lo_min, r.x);
      hi_max = max(hi_max, r.y);
      lo_max = max(lo_max, r.x);
      hi_min = min(hi_min, r.y);
    } else {
      lo_max = INT_MAX;
      hi_min = 0;
    }
  }
  lo_min = __reduce_min_sync(0xffffffffu, lo_min);
  hi_max = __reduce_max_sync(0xffffffffu, hi_max);
  lo_max = __reduce_max_sync(0xffffffffu, lo_max);
  hi_min = __reduce_min_sync(0xffffffffu, hi_min);
  if (lane == 0) q_sum[tile] = make_int4(lo_min, hi_max, lo_max, hi_min);
}

__global__ void __launch_bounds__(128) mask_k_summary(const int4* q_sum, int n_qt, int n_kt, int n_tiles,
                                                      int2* k_sum) {
  const int tile = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (tile >= n_tiles) return;
  const int b = tile / n_kt, k0 = (tile % n_kt) * BN;
  int first = INT_MAX, last = -1;
  for (int qt = lane; qt < n_qt; qt += 32) {
    const int4 s = q_sum[(long long)b * n_qt + qt];
    if (s.x < k0 + BN && s.y > k0) {
      first = min(first, qt);
      last = qt;
    }
  }
  first = __reduce_min_sync(0xffffffffu, first);
  last = __reduce_max_sync(0xffffffffu, last);
  if (lane == 0) k_sum[tile] = make_int2(first == INT_MAX ? 0 : first, last);
}

__global__ void __launch_bounds__(SCAN_THREADS) mask_k_exact(const int2* ranges, int Sq, int rows_pad, int* k_exact) {
  const int2* r = ranges + (long long)blockIdx.x * rows_pad;
  bool up = true;
  for (int i = threadIdx.x + 1; i < Sq; i += SCAN_THREADS) {
    const int2 a = r[i - 1], c = r[i];
    up = up && a.x <= c.x && a.y <= c.y;
  }
  const int all = __syncthreads_and(up);
  if (threadIdx.x == 0) k_exact[blockIdx.x] = all;
}

__global__ void __launch_bounds__(128) mask_k_rows(const int2* ranges, const int* k_exact, int Sq, int rows_pad,
                                                   int n_kt, int2* k_rows) {
  const int b = blockIdx.x / n_kt, k = (blockIdx.x % n_kt) * BN + threadIdx.x;
  const int2* r = ranges + (long long)b * rows_pad;
  int first = 0, past = Sq;  // the first row with hi > k, and the first with lo > k
  if (k_exact[b]) {
    for (int lo = 0, hi = Sq;;) {
      if (lo == hi) {
        first = lo;
        break;
      }
      const int mid = (lo + hi) / 2;
      if (r[mid].y > k) hi = mid;
      else lo = mid + 1;
    }
    for (int lo = 0, hi = Sq;;) {
      if (lo == hi) {
        past = lo;
        break;
      }
      const int mid = (lo + hi) / 2;
      if (r[mid].x > k) hi = mid;
      else lo = mid + 1;
    }
  }
  k_rows[((long long)b * n_kt) * BN + k] = make_int2(first, past - 1);
}

}  // namespace

cudaError_t launch_mask_plan(const MaskPlanArgs& a, void* plan, cudaStream_t s) {
  const int n_qt = ceil_div(a.Sq, BQ), n_kt = ceil_div(a.Skv, BN), rows_pad = n_qt * BQ;
  const MaskPlanLayout l = mask_plan_layout(a.B, n_qt, n_kt);
  char* base = static_cast<char*>(plan);
  int2* ranges = reinterpret_cast<int2*>(base + l.ranges);
  int4* q_sum = reinterpret_cast<int4*>(base + l.q_sum);
  int2* k_sum = reinterpret_cast<int2*>(base + l.k_sum);
  if (a.row_lo)
    mask_row_ranges<<<(unsigned)ceil_div(a.B * rows_pad, 256), 256, 0, s>>>(
        a.row_lo, a.row_hi, a.Sq, a.Skv, rows_pad, (long long)a.B * rows_pad, ranges);
  else
    mask_doc_ranges<<<(unsigned)a.B, SCAN_THREADS, 0, s>>>(a.doc_ids, a.prefix_lens, a.prefix_per_row,
                                                                 a.causal, a.Sq, rows_pad, ranges);
  mask_q_summary<<<(unsigned)ceil_div(a.B * n_qt, 4), 128, 0, s>>>(ranges, a.Sq, n_qt, a.B * n_qt, q_sum);
  mask_k_summary<<<(unsigned)ceil_div(a.B * n_kt, 4), 128, 0, s>>>(q_sum, n_qt, n_kt, a.B * n_kt, k_sum);
  int2* k_rows = reinterpret_cast<int2*>(base + l.k_rows);
  int* k_exact = reinterpret_cast<int*>(base + l.k_exact);
  mask_k_exact<<<(unsigned)a.B, SCAN_THREADS, 0, s>>>(ranges, a.Sq, rows_pad, k_exact);
  mask_k_rows<<<(unsigned)(a.B * n_kt), BN, 0, s>>>(ranges, k_exact, a.Sq, rows_pad, n_kt, k_rows);
  return cudaGetLastError();
}

}  // namespace sdpa

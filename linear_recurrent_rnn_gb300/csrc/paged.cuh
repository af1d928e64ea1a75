// Shared by the paged-cache kernels (include/paged_attn.h): the argument block of the attention,
// the division of its work over CTAs, and the partial results of rows whose keys are split.
//
// Work division.  Rows of a request: its q new tokens x the g = Hq / Hkv query heads of one
// key/value head, token-major; a row tile holds tb whole tokens.  An item is (request, key/value
// head, row tile); its keys are [lo, hi): from the first key its first token sees to its last
// token's own position.  Its weight is hi - lo + PG_OVERHEAD.  The items in order (requests,
// then heads, then row tiles) lie end to end on a line of U = sum of weights, and CTA i of G
// takes [U i / G, U (i + 1) / G): every CTA gets the same weight whatever the mix of lengths
// (one long request, many short ones, prefill among decode), and no host knowledge of lengths
// is needed.  An item cut by such a boundary is computed in parts, each over a range of whole
// key tiles, and joined by the last of its CTAs to finish.  Prefix sums over the row tiles of
// a request are sums of max(0, a + m tb) over m, so they have a closed form; only the sum over
// requests is a scan.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "../../include/paged_attn.h"

namespace rglru {

constexpr int PG_MAX_SEQS = 8192;
constexpr int PG_MAX_CTAS = 1024;
// Weight of an item beyond its keys (query load, epilogue): about one 128-key tile's time.
constexpr int PG_OVERHEAD = 128;
// Least weight of a CTA: one key tile and the overhead; below it splitting costs more than it
// saves.
constexpr int PG_MIN_WEIGHT = 128 + PG_OVERHEAD;

struct PagedArgs {
  int N, T, Hq, Hkv, g, D, P, ps_log2, table_width, window;
  int tb;      // tokens per row tile
  float scale_log2;  // scale * log2(e): scores in units of log2
  const void* q;
  const void* kc;
  const void* vc;
  const int32_t* table;
  const int32_t* cu;
  const int32_t* kv_lens;
  void* o;
  float* lse;
  int64_t q_token, q_head, o_token, o_head, kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;
  uint8_t* ws;
  size_t part_ml, part_o;  // workspace offsets (below)
  int rows;                // rows of a partial result
};

// Workspace: u32 status word, then at 256 one u32 counter per CTA (zero between calls), then the
// partial results, two slots a CTA (an item that began in an earlier CTA, one that goes on in
// a later CTA): row maxima and sums float2 [slot][rows], sums of weighted values float
// [slot][rows][Dp] (Dp: D rounded up to the kernel's head width).
struct PagedWs {
  size_t ml, o, total;
};
inline PagedWs paged_ws(int ctas, int rows, int Dp) {
  PagedWs w;
  w.ml = 256 + align_up((size_t)PG_MAX_CTAS * 4, 256);
  w.o = w.ml + align_up((size_t)2 * ctas * rows * 8, 256);
  w.total = w.o + (size_t)2 * ctas * rows * Dp * 4;
  return w;
}

struct PgReq {
  int first, q, kv;  // first token row, new tokens, keys
};

__device__ __forceinline__ PgReq pg_request(const PagedArgs& a, int n) {
  PgReq r;
  const int s = min(max(a.cu[n], 0), a.T), e = min(max(a.cu[n + 1], s), a.T);
  r.first = s;
  r.q = e - s;
  r.kv = min(max(a.kv_lens[n], 0), 1 << 30);
  return r;
}

// sum of max(0, x + m d) over 0 <= m < M (d > 0)
__device__ __forceinline__ int64_t pg_ramp(int64_t x, int d, int64_t M) {
  const int64_t m0 = x > 0 ? 0 : (-x) / d + 1;
  if (m0 >= M) return 0;
  return (M - m0) * x + (int64_t)d * ((M * (M - 1) - m0 * (m0 - 1)) / 2);
}

// Key range of row tile m.
__device__ __forceinline__ void pg_range(const PagedArgs& a, const PgReq& r, int m, int& lo, int& hi) {
  const int64_t base = (int64_t)r.kv - r.q, t0 = (int64_t)m * a.tb;
  const int64_t t1 = min(t0 + a.tb, (int64_t)r.q);
  hi = (int)max(base + t1, (int64_t)0);
  lo = a.window ? (int)max(base + t0 - a.window + 1, (int64_t)0) : 0;
  if (lo > hi) lo = hi;
}
__device__ __forceinline__ int64_t pg_weight(const PagedArgs& a, const PgReq& r, int m) {
  int lo, hi;
  pg_range(a, r, m, lo, hi);
  return hi - lo + PG_OVERHEAD;
}
__device__ __forceinline__ int pg_tiles(const PagedArgs& a, const PgReq& r) {
  return (r.q + a.tb - 1) / a.tb;
}
// Weight of the first M row tiles of one head, none of them the request's last.
__device__ __forceinline__ int64_t pg_prefix(const PagedArgs& a, const PgReq& r, int64_t M) {
  const int64_t base = (int64_t)r.kv - r.q;
  int64_t w = M * PG_OVERHEAD + pg_ramp(base + a.tb, a.tb, M);
  if (a.window) {
    // lo is at most hi: the keys before the window of a tile that ends past position 0
    const int64_t x = base - a.window + 1;
    w -= pg_ramp(x, a.tb, M);
  }
  return w;
}
__device__ __forceinline__ int64_t pg_head_weight(const PagedArgs& a, const PgReq& r) {
  const int M = pg_tiles(a, r);
  if (M == 0) return 0;
  return pg_prefix(a, r, M - 1) + pg_weight(a, r, M - 1);
}

// CTA i's range of the line and the owner of a place on it.
__device__ __forceinline__ int64_t pg_cut(int64_t U, int i, int G) { return U * i / G; }
__device__ __forceinline__ int pg_owner(int64_t x, int64_t U, int G) {
  return (int)(((x + 1) * G - 1) / U);
}

// Sum over the requests by the whole CTA: prefix[n] = weight of the requests before n (n <= N).
// `prefix` and the 33-entry `scratch` in shared memory; ends with a CTA barrier.
__device__ __forceinline__ void pg_scan(const PagedArgs& a, int64_t* prefix, int64_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  int64_t carry = 0;
  for (int n0 = 0; n0 < a.N; n0 += blockDim.x) {
    const int n = n0 + tid;
    int64_t w = 0;
    if (n < a.N) w = pg_head_weight(a, pg_request(a, n)) * a.Hkv;
    int64_t s = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += u;
    }
    if (lane == 31) scratch[warp] = s;
    __syncthreads();
    int64_t before = carry, all = 0;
    for (int k = 0; k < nw; ++k) {
      const int64_t u = scratch[k];
      if (k < warp) before += u;
      all += u;
    }
    if (n < a.N) prefix[n] = before + s - w;
    carry += all;
    __syncthreads();
  }
  if (tid == 0) prefix[a.N] = carry;
  __syncthreads();
}

// An item of this CTA's range and how much of it is the CTA's.
struct PgItem {
  int n, h, m;       // request, key/value head, row tile
  PgReq r;
  int lo, hi;        // the row tile's keys
  int64_t at, w;     // place on the line, weight
};

// Walks the items that meet [w0, w1).  All state is per thread; every thread that walks sees
// the same items.
struct PgWalk {
  int64_t U, w0, w1;
  int G, cta;
  PgItem it;

  // `prefix` as left by pg_scan.  Returns false if the CTA has no work.
  __device__ __forceinline__ bool start(const PagedArgs& a, const int64_t* prefix) {
    U = prefix[a.N];
    cta = blockIdx.x;
    G = (int)min((int64_t)gridDim.x, (U + PG_MIN_WEIGHT - 1) / PG_MIN_WEIGHT);
    if (cta >= G) return false;
    w0 = pg_cut(U, cta, G);
    w1 = pg_cut(U, cta + 1, G);
    // the request, head and row tile that hold w0
    int l = 0, h = a.N - 1;
    while (l < h) {
      const int mid = (l + h + 1) >> 1;
      if (prefix[mid] <= w0) l = mid; else h = mid - 1;
    }
    // (requests without rows have no weight: l is the last one that starts at or before w0)
    it.n = l;
    it.r = pg_request(a, l);
    const int64_t hw = pg_head_weight(a, it.r);
    int64_t x = w0 - prefix[l];
    it.h = (int)(x / hw);
    x -= it.h * hw;
    int ml = 0, mh = pg_tiles(a, it.r) - 1;
    while (ml < mh) {
      const int mid = (ml + mh + 1) >> 1;
      if (pg_prefix(a, it.r, mid) <= x) ml = mid; else mh = mid - 1;
    }
    it.m = ml;
    it.at = prefix[l] + it.h * hw + pg_prefix(a, it.r, ml);
    fill(a);
    return true;
  }
  __device__ __forceinline__ void fill(const PagedArgs& a) {
    pg_range(a, it.r, it.m, it.lo, it.hi);
    it.w = it.hi - it.lo + PG_OVERHEAD;
  }
  // The next item; false past the CTA's range.
  __device__ __forceinline__ bool next(const PagedArgs& a) {
    it.at += it.w;
    if (it.at >= w1) return false;
    if (++it.m == pg_tiles(a, it.r)) {
      it.m = 0;
      if (++it.h == a.Hkv) {
        it.h = 0;
        do {
          it.r = pg_request(a, ++it.n);
        } while (it.r.q == 0);  // ends: weight is left on the line
      }
    }
    fill(a);
    return true;
  }
  // The CTA's key tiles [j0, j1) of the item, tiles of `bn` keys counted from position 0.
  // A cut at x of the item's weight w gives the parts floor(tiles x / w) of its tiles.
  __device__ __forceinline__ void tiles(int bn, int& j0, int& j1) const {
    const int t0 = it.lo / bn, nt = (it.hi + bn - 1) / bn - t0;
    const int64_t x0 = max(w0, it.at) - it.at, x1 = min(w1, it.at + it.w) - it.at;
    j0 = t0 + (int)(x0 * nt / it.w);
    j1 = t0 + (int)(x1 * nt / it.w);
  }
  __device__ __forceinline__ bool whole() const { return w0 <= it.at && it.at + it.w <= w1; }
  // CTAs [first, last] that share the item.
  __device__ __forceinline__ void owners(int& first, int& last) const {
    first = pg_owner(it.at, U, G);
    last = pg_owner(it.at + it.w - 1, U, G);
  }
  // Partial-result slot of CTA c for an item whose first CTA is `first`.
  __device__ __forceinline__ static int slot(int c, int first) { return 2 * c + (c == first); }
};

// Tensor-core attention (paged_attn_tc.cu, bf16 I/O).
cudaError_t launch_paged_attn_tc(PagedArgs a, int num_pages, int page_size, cudaStream_t s);
size_t paged_attn_tc_ws_bytes(const paged_shape* s);
// CUDA-core attention (paged_attn_simt.cu, float32 I/O).
cudaError_t launch_paged_attn_simt(PagedArgs a, cudaStream_t s);
size_t paged_attn_simt_ws_bytes(const paged_shape* s);

// One kernel on `s` with programmatic stream serialisation (and clusters of `cluster` CTAs).
cudaError_t launch_pdl(const void* f, dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       void** args, int cluster);

}  // namespace rglru

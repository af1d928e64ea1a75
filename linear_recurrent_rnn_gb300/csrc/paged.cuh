// Shared by the paged-cache kernels (include/paged_attn.h): the argument block of the attention,
// the division of its work over CTAs, and the partial results of rows whose keys are split.
//
// Work division.  Rows of a request: its q new tokens x the g = Hq / Hkv query heads of one
// key/value head, token-major; a row tile holds tb whole tokens.  An item is (request, key/value
// head, row tile); its keys are [lo, hi): from the first key its first token sees to its last
// token's own position.  Its weight is hi - lo + overhead.  The items in order (requests,
// then heads, then row tiles) lie end to end on a line of U = sum of weights, and CTA i takes
// [W i, W (i + 1)), W = U / CTAs rounded up: every CTA gets the same weight whatever the mix of lengths
// (one long request, many short ones, prefill among decode), and no host knowledge of lengths
// is needed.  An item cut by such a boundary is computed in parts, each over a range of whole
// key tiles, and joined by the last of its CTAs to finish; a cut that would leave a part of less
// than `snap` moves to the item's end, as parts cost more than a small difference of weight.  Prefix sums over the row tiles of
// a request are sums of max(0, a + m tb) over m, so they have a closed form; only the sum over
// requests is a scan.  All of it is done by every CTA for itself (no kernel before, no host
// synchronisation), so it is in the way of the first load and kept short: no 64-bit division.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "../../include/paged_attn.h"

namespace rglru {

constexpr int PG_MAX_SEQS = 8192;
constexpr int PG_MAX_TOKENS = 1 << 30;  // rows and lengths up to 2^30: sums of two, or a step past the end, fit 32 bits
constexpr int PG_MAX_CTAS = 1024;
constexpr int PG_WARP_SEQS = 32;  // requests that one warp scans alone

struct PagedArgs {
  int N, T, Hq, Hkv, g, D, P, ps_log2, table_width, window;
  int tb;          // tokens per row tile
  uint32_t g_inv;  // 2^16 / g, rounded up
  int overhead;    // weight of an item beyond its keys: its switch, in keys' time
  uint64_t grid_inv;
  int min_weight;  // least weight of a CTA: below it splitting costs more than it saves
  int snap;        // least weight of a part (at most a quarter of a CTA's)
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
  uint64_t wait_ns;        // limit of a device wait; CTA that hands out no work (tests; -1: none)
  int drop_cta;
  int o_32;                // rows of o are multiples of 32 bytes on 32-byte boundaries
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

// The division's constants: CTAs of the launch, an item's weight beyond its keys, a CTA's and a
// part's least.
inline void pg_division(PagedArgs& a, int grid, int overhead, int min_weight, int snap) {
  a.grid_inv = ~0ull / grid + 1;
  a.overhead = overhead;
  a.min_weight = min_weight;
  a.snap = snap;
}

struct PgReq {
  int first, q, kv;  // first token row, new tokens, keys
};

// r / g for a row r < 2^16 / g
__device__ __forceinline__ int pg_token(const PagedArgs& a, int r) { return (int)((uint32_t)r * a.g_inv >> 16); }

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
  const int64_t m0 = x > 0 ? 0 : (uint32_t)(-x) / (uint32_t)d + 1;  // (|x| < 2^32)
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
  return hi - lo + a.overhead;
}
__device__ __forceinline__ int pg_tiles(const PagedArgs& a, const PgReq& r) {
  return r.q <= a.tb ? (r.q > 0) : (r.q + a.tb - 1) / a.tb;
}
// Weight of the first M row tiles of one head, none of them the request's last.
__device__ __forceinline__ int64_t pg_prefix(const PagedArgs& a, const PgReq& r, int64_t M) {
  const int64_t base = (int64_t)r.kv - r.q;
  int64_t w = M * a.overhead + pg_ramp(base + a.tb, a.tb, M);
  if (a.window) {
    // lo is at most hi: the keys before the window of a tile that ends past position 0
    const int64_t x = base - a.window + 1;
    w -= pg_ramp(x, a.tb, M);
  }
  return w;
}
__device__ __forceinline__ int64_t pg_head_weight(const PagedArgs& a, const PgReq& r) {
  const int M = pg_tiles(a, r);
  if (M <= 1) return M == 0 ? 0 : pg_weight(a, r, 0);
  return pg_prefix(a, r, M - 1) + pg_weight(a, r, M - 1);
}

__device__ __forceinline__ float pg_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// floor(x / y) for a quotient below 2^20, x < 2^62: the float32 quotient is at most one off.
__device__ __forceinline__ int pg_div(int64_t x, int64_t y) {
  int q = (int)__fmul_rn((float)x, pg_rcp((float)y));
  while (q * y > x) --q;
  while ((q + 1) * y <= x) ++q;
  return q;
}

// The last n < count with f(n) true, f true up to there and f(0) true; by a converged warp, 32
// places at a time.
template <class F>
__device__ __forceinline__ int pg_last(int count, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = count;
  while (n > 1) {
    const int step = (n + 31) >> 5, at = lane * step;
    const int k = __popc(__ballot_sync(0xffffffffu, at < n && f(lo + at))) - 1;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
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
  int64_t W, w0, w1;
  int cta, snap;
  PgItem it;

  // The CTA's range of a line of weight U; false if there is none.
  __device__ __forceinline__ bool range(const PagedArgs& a, int64_t U) {
    cta = blockIdx.x;
    // U / grid, rounded up: grid_inv is 2^64 / grid, rounded up (exact for U grid < 2^64)
    W = gridDim.x == 1 ? U : (int64_t)__umul64hi((uint64_t)U + gridDim.x - 1, a.grid_inv);
    W = max(W, (int64_t)a.min_weight);
    snap = (int)min((int64_t)a.snap, W >> 2);
    w0 = W * cta;
    w1 = min(w0 + W, U);
    return w0 < U;
  }
  // The request that holds w0 (r.q = 0: the CTA has no work), its place and one head's weight;
  // `prefix` as left by pg_scan.
  struct Found {
    int n;
    PgReq r;
    int64_t at, hw;
  };
  __device__ __forceinline__ Found find(const PagedArgs& a, const int64_t* prefix) {
    Found f = {0, {0, 0, 0}, 0, 0};
    if (!range(a, prefix[a.N])) return f;
    const int l = pg_last(a.N, [&](int n) { return prefix[n] <= w0; });
    // (requests without rows have no weight: l is the last one that starts at or before w0)
    f.n = l;
    f.r = pg_request(a, l);
    f.at = prefix[l];
    f.hw = pg_head_weight(a, f.r);
    return f;
  }
  // The same for up to 32 requests, one a lane, by a whole warp without shared memory.
  __device__ __forceinline__ Found find_warp(const PagedArgs& a) {
    const int lane = threadIdx.x & 31;
    Found f = {0, {0, 0, 0}, 0, 0};
    if (lane < a.N) {
      f.r = pg_request(a, lane);
      f.hw = pg_head_weight(a, f.r);
    }
    const int64_t w = f.hw * a.Hkv;
    int64_t s = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += u;
    }
    const bool any = range(a, __shfl_sync(0xffffffffu, s, 31));
    const uint32_t before = __ballot_sync(0xffffffffu, w > 0 && s - w <= w0);
    f.n = before ? 31 - __clz(before) : 0;
    f.at = __shfl_sync(0xffffffffu, s - w, f.n);
    f.hw = __shfl_sync(0xffffffffu, f.hw, f.n);
    f.r.first = __shfl_sync(0xffffffffu, f.r.first, f.n);
    f.r.kv = __shfl_sync(0xffffffffu, f.r.kv, f.n);
    f.r.q = __shfl_sync(0xffffffffu, f.r.q, f.n);
    if (!any) f.r.q = 0;
    return f;
  }
  // Begins at w0.  False if the CTA has no work.
  __device__ __forceinline__ bool enter(const PagedArgs& a, const Found& f) {
    if (f.r.q == 0) return false;
    it.n = f.n;
    it.r = f.r;
    int64_t x = w0 - f.at;
    it.h = pg_div(x, f.hw);
    x -= it.h * f.hw;
    it.m = 0;
    it.at = w0 - x;
    if (it.r.q > a.tb) {
      it.m = pg_last(pg_tiles(a, it.r), [&](int m) { return pg_prefix(a, it.r, m) <= x; });
      it.at += pg_prefix(a, it.r, it.m);
    }
    fill(a);
    const int64_t d = w0 - it.at;
    if (d > 0) {  // the cut is inside the item
      if (d < snap)
        w0 = it.at;
      else if (it.w - d < snap)
        w0 = it.at + it.w;  // the item is the neighbour's
    }
    return it.at + it.w > w0 ? it.at < w1 : next(a);
  }
  __device__ __forceinline__ void fill(const PagedArgs& a) {
    pg_range(a, it.r, it.m, it.lo, it.hi);
    it.w = it.hi - it.lo + a.overhead;
    const int64_t d = w1 - it.at;
    if (d > 0 && d < it.w) {  // the CTA's other cut
      if (d < snap)
        w1 = it.at;
      else if (it.w - d < snap)
        w1 = it.at + it.w;
    }
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
    return it.at < w1;
  }
  // The CTA's key tiles [j0, j1) of the item, tiles of `bn` keys counted from position 0.
  // A cut at x of the item's weight w gives the parts about tiles x / w of its tiles, rounded in
  // one way for the CTAs on both sides of the cut.
  __device__ __forceinline__ void tiles(int bn, int& j0, int& j1) const {
    const int t0 = it.lo / bn, nt = (it.hi + bn - 1) / bn - t0;
    j0 = t0 + place(max(w0, it.at) - it.at, nt);
    j1 = t0 + place(min(w1, it.at + it.w) - it.at, nt);
  }
  __device__ __forceinline__ int place(int64_t x, int nt) const {
    if (x <= 0) return 0;
    if (x >= it.w) return nt;
    return min((int)__fmul_rn(__fmul_rn((float)x, pg_rcp((float)it.w)), (float)nt), nt);
  }
  __device__ __forceinline__ bool whole() const { return w0 <= it.at && it.at + it.w <= w1; }
  // CTAs [first, last] that share the item: where it begins and ends on the line, but for a cut
  // that has moved to its end.
  __device__ __forceinline__ void owners(int& first, int& last) const {
    first = last = cta;
    if (it.at < w0) {
      first = pg_div(it.at, W);
      if ((first + 1) * W - it.at < snap) ++first;
    }
    if (it.at + it.w > w1) {
      last = pg_div(it.at + it.w - 1, W);
      if (it.at + it.w - last * W < snap) --last;
    }
  }
  // Partial-result slot of CTA c for an item whose first CTA is `first`.
  __device__ __forceinline__ static int slot(int c, int first) { return 2 * c + (c == first); }
};

// Tensor-core attention (bf16 I/O): many rows a request (paged_attn_tc.cu), few rows a request,
// `rows` in the mean (paged_attn_few.cu, up to PG_FEW_ROWS).
cudaError_t launch_paged_attn_tc(PagedArgs a, cudaStream_t s);
size_t paged_attn_tc_ws_bytes(const paged_shape* s);
constexpr int PG_FEW_ROWS = 32;
cudaError_t launch_paged_attn_few(PagedArgs a, int rows, cudaStream_t s);
size_t paged_attn_few_ws_bytes(const paged_shape* s, int rows);
// CUDA-core attention (paged_attn_simt.cu, float32 I/O), `rows` a request in the mean.
cudaError_t launch_paged_attn_simt(PagedArgs a, int rows, cudaStream_t s);
size_t paged_attn_simt_ws_bytes(const paged_shape* s, int rows);

// Host checks that every call over a paged cache makes.
inline int pg_log2(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}
inline bool pg_aligned(const void* p, size_t n) { return p && reinterpret_cast<uintptr_t>(p) % n == 0; }
rglru_status pg_check_cache(const paged_shape* s);

// One kernel on `s` with programmatic stream serialisation (and clusters of `cluster` CTAs).  Such a
// kernel's lifetime overlaps the one before it, which may be writing what this one reads: what
// comes after griddep_wait are ordinary loads, none through the non-coherent path (__ldg).
cudaError_t launch_pdl(const void* f, dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       void** args, int cluster);

}  // namespace rglru

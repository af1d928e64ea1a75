// The pages of the cache as requests come and go (include/paged_pages.h): rows forked, pages
// released and copied, the pool compacted.
//
// Page numbers are few and the work on them short: what counts is the number of launches and of
// dependent round trips.  Every CTA works out what it needs of the whole for itself (a scan of the
// children, the set bits before its own words), as the plan does (paged.cu), so nothing waits for
// another CTA; where all of a phase has to be done before the next, the next is a kernel of its
// own, begun early by programmatic stream serialisation.
#include <algorithm>

#include "host_util.h"
#include "paged_tc.cuh"

namespace rglru {

namespace {

constexpr int PP_THREADS = 512;
constexpr int PP_WARPS = PP_THREADS / 32;
constexpr int PP_CLUSTER = 8;   // CTAs of a fork in place
constexpr int PP_MAX_CTAS = 152;
constexpr int PP_COLS = 128;    // table entries that a warp takes at once

// Exclusive sum over the CTA's threads (a multiple of 32); `all` is the total.  `s_warp`: 32 entries in
// shared memory, free again after the next barrier.
__device__ __forceinline__ int pp_scan(int x, int32_t* s_warp, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += u;
  }
  if (lane == 31) s_warp[warp] = s;
  __syncthreads();
  int before = 0;
  all = 0;
  for (int k = 0; k < nw; ++k) {
    const int u = s_warp[k];
    all += u;
    if (k < warp) before += u;
  }
  return before + s - x;
}

// The ring's head and count as they are used: within the ring.
__device__ __forceinline__ void pp_ring(const int32_t* state, int P, int& head, int& count) {
  head = state[0];
  if ((uint32_t)head >= (uint32_t)P) head = (head % P + P) % P;
  count = min(max(state[1], 0), P);
}
__device__ __forceinline__ int pp_wrap(int64_t i, int P) { return (int)(i < P ? i : i - P); }

// ---------------------------------------------------------------- a copy of page counts
__global__ void __launch_bounds__(PP_THREADS) k_paged_counts(const int32_t* from, int32_t* to, int n) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  for (int64_t i = (int64_t)blockIdx.x * PP_THREADS + threadIdx.x; i < n; i += (int64_t)gridDim.x * PP_THREADS) to[i] = from[i];
}

// ---------------------------------------------------------------- fork
struct ForkArgs {
  int N, M, P, s_log2, width, cluster;
  const int32_t *parents, *children, *table, *lens, *ring, *state;
  int32_t *table_out, *lens_out, *holders, *moves, *state_out;
};

// Every CTA scans the children for their places on the ring; then a warp takes a child and PP_COLS
// entries of its row.  In place the CTAs are one cluster, which meets between reading and
// writing.
__global__ void __launch_bounds__(PP_THREADS) k_paged_fork(const ForkArgs a) {
  extern __shared__ int32_t pp_sm[];
  int32_t* s_len = pp_sm;        // [M] tokens; -1: passed over
  int32_t* s_at = s_len + a.M;   // [M] place on the ring
  __shared__ int32_t s_warp[32];
  const int tid = threadIdx.x, lane = tid & 31, s = 1 << a.s_log2;
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  int head, count;
  pp_ring(a.state, a.P, head, count);
  const int per = (a.M + PP_THREADS - 1) / PP_THREADS;
  const int i0 = min(tid * per, a.M), i1 = min(i0 + per, a.M);
  auto part = [&](int L) { return L >= 0 && (L & (s - 1)) && L >> a.s_log2 < a.width; };  // a page of its own
  int mine = 0;
  for (int i = i0; i < i1; ++i) {
    const int p = a.parents[i], c = a.children[i];
    const bool ok = (uint32_t)p < (uint32_t)a.N && (uint32_t)c < (uint32_t)a.N;
    s_len[i] = ok ? max(a.lens[p], 0) : -1;
    mine += part(s_len[i]);
  }
  int wanted, at = pp_scan(mine, s_warp, wanted);
  for (int i = i0; i < i1; ++i) {
    s_at[i] = at;
    at += part(s_len[i]);
  }
  if (a.cluster > 1) {
    __syncwarp();  // the barrier's form is the warp-aligned one
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    const int taken = min(wanted, count);
    a.state_out[0] = pp_wrap((int64_t)head + taken, a.P);
    a.state_out[1] = count - taken;
    a.state_out[2] = wanted - taken;
  }
  const int chunks = (a.width + PP_COLS - 1) / PP_COLS;
  const int64_t tasks = (int64_t)a.M * chunks, step = (int64_t)gridDim.x * PP_WARPS;
  for (int64_t t = (int64_t)blockIdx.x * PP_WARPS + (tid >> 5); t < tasks; t += step) {
    const int i = (int)(t / chunks), c0 = (int)(t - (int64_t)i * chunks) * PP_COLS, L = s_len[i];
    const bool own = part(L);
    const int child = a.children[i], full = min(L >> a.s_log2, a.width);
    if (c0 == 0 && lane == 0) {
      if (L >= 0) a.lens_out[child] = L;
      if (!own) a.moves[2 * i] = a.moves[2 * i + 1] = -1;
    }
    if (L < 0 || c0 > full) continue;
    const int32_t* row = a.table + (int64_t)a.parents[i] * a.width;
    int32_t* out = a.table_out + (int64_t)child * a.width;
    int id[PP_COLS / 32];
#pragma unroll
    for (int e = 0; e < PP_COLS / 32; ++e) {
      const int col = c0 + e * 32 + lane;
      id[e] = col < full + own ? row[col] : -1;
    }
#pragma unroll
    for (int e = 0; e < PP_COLS / 32; ++e) {
      const int col = c0 + e * 32 + lane;
      if (col < full) {
        out[col] = id[e];
        if ((uint32_t)id[e] < (uint32_t)a.P) atomicAdd(a.holders + id[e], 1);
      } else if (col == full && own) {
        const int f = s_at[i] < count ? a.ring[pp_wrap((int64_t)head + s_at[i], a.P)] : -1;
        const bool move = (uint32_t)f < (uint32_t)a.P && (uint32_t)id[e] < (uint32_t)a.P;
        out[col] = f;
        a.moves[2 * i] = move ? id[e] : -1;
        a.moves[2 * i + 1] = move ? f : -1;
      }
    }
  }
}

// ---------------------------------------------------------------- release and compact: a bit a page
// Workspace: a counter of CTAs, at 256 a bit a page; all zero between calls, so pools of any size may share
// one.  Nothing else is kept there: numbers by page, left behind by a call over a small pool, would be
// set bits to one over a larger pool.
size_t pages_ws_bytes(int P) { return 256 + align_up(((size_t)P + 31) / 32 * 4, 256); }

struct PagesArgs {
  int N, P, s_log2, width, words;
  const int32_t *first, *end, *lens;  // entries of a row: from first to end, or those in use of a length
  const int32_t *table, *state, *holders;
  int32_t *table_out, *holders_out, *ring, *state_out, *moves;
  uint32_t *counter, *bits;
};

// One bit for every page that the entries free (RELEASE) or use.  A warp takes a row and PP_COLS
// entries, one such task where the GPU holds as many warps (1024 requests of up to 1000 pages: 15.2 us a
// release; with a CTA an SM, and three tasks a warp one after another, 19.0).  A page without other holders is
// free at once; the others count down, and the one that finds none left frees the page: which of them does not
// matter, as the ring's order is the pages' own.
template <bool RELEASE>
__global__ void __launch_bounds__(PP_THREADS) k_paged_mark(const PagesArgs a) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, s = 1 << a.s_log2;
  const int chunks = (a.width + PP_COLS - 1) / PP_COLS;
  const int64_t tasks = (int64_t)a.N * chunks, step = (int64_t)gridDim.x * PP_WARPS;
  for (int64_t t = (int64_t)blockIdx.x * PP_WARPS + (threadIdx.x >> 5); t < tasks; t += step) {
    const int n = (int)(t / chunks), c0 = (int)(t - (int64_t)n * chunks) * PP_COLS;
    const int lo = RELEASE ? max(a.first[n], 0) : 0;
    const int hi = min(RELEASE ? a.end[n] : (int)(((int64_t)max(a.lens[n], 0) + s - 1) >> a.s_log2), a.width);
    if (c0 >= hi || c0 + PP_COLS <= lo) continue;
    const int64_t row = (int64_t)n * a.width;
    int id[PP_COLS / 32], held[PP_COLS / 32];
#pragma unroll
    for (int e = 0; e < PP_COLS / 32; ++e) {
      const int col = c0 + e * 32 + lane;
      id[e] = col >= lo && col < hi ? a.table[row + col] : -1;
    }
#pragma unroll
    for (int e = 0; e < PP_COLS / 32; ++e) {
      const int col = c0 + e * 32 + lane;
      const bool page = (uint32_t)id[e] < (uint32_t)a.P;
      if (RELEASE) {
        if (col >= lo && col < hi) a.table_out[row + col] = -1;
        held[e] = page ? __ldcg(a.holders_out + id[e]) : 1;
      } else {  // seen already by another row?
        held[e] = page ? (int)(__ldcg(a.bits + (id[e] >> 5)) >> (id[e] & 31) & 1u) : 1;
      }
    }
#pragma unroll
    for (int e = 0; e < PP_COLS / 32; ++e) {
      if ((uint32_t)id[e] >= (uint32_t)a.P) continue;
      bool mark = held[e] <= 0;
      if (RELEASE && !mark) mark = atomicSub(a.holders_out + id[e], 1) <= 0;
      if (mark) atomicOr(a.bits + (id[e] >> 5), 1u << (id[e] & 31));
    }
  }
}

// This CTA's words [w0, w1).
__device__ __forceinline__ void pp_words(const PagesArgs& a, int& w0, int& w1) {
  const int per = (a.words + gridDim.x - 1) / gridDim.x;
  w0 = min((int)blockIdx.x * per, a.words);
  w1 = min(w0 + per, a.words);
}

// Calls f(page, bit, set bits before it) for the 32 pages of each word, a lane a page; by the whole CTA.
// `before`: set bits before word w0.
template <class F>
__device__ __forceinline__ void pp_pages(const PagesArgs& a, int w0, int w1, int before, int32_t* s_warp, F f) {
  __shared__ uint32_t s_bits[PP_THREADS];
  __shared__ int32_t s_before[PP_THREADS];
  const int tid = threadIdx.x, lane = tid & 31;
  for (int w = w0; w < w1; w += PP_THREADS) {
    __syncthreads();
    const uint32_t x = w + tid < w1 ? a.bits[w + tid] : 0u;
    int all;
    const int at = pp_scan(__popc(x), s_warp, all);
    s_bits[tid] = x;
    s_before[tid] = before + at;
    before += all;
    __syncthreads();
    for (int k = tid >> 5; k < min(PP_THREADS, w1 - w); k += PP_WARPS) {
      const uint32_t y = s_bits[k];
      const int64_t p = (int64_t)(w + k) * 32 + lane;
      if (p < a.P) f((int)p, y >> lane & 1u, s_before[k] + __popc(y & ((1u << lane) - 1)));
    }
  }
}

// The freed pages onto the ring.  The CTA that is done last clears the bits and writes the ring's state
// (which may be where the others have read it).
__global__ void __launch_bounds__(PP_THREADS) k_paged_freed(const PagesArgs a) {
  __shared__ int32_t s_warp[32];
  __shared__ uint32_t s_last;
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  int head, count, w0, w1, before = 0, all;
  pp_ring(a.state, a.P, head, count);
  pp_words(a, w0, w1);
  for (int w = threadIdx.x; w < w0; w += PP_THREADS) before += __popc(a.bits[w]);
  pp_scan(before, s_warp, all);
  before = all;
  __syncthreads();
  const int tail = pp_wrap((int64_t)head + count, a.P);
  pp_pages(a, w0, w1, before, s_warp, [&](int p, uint32_t bit, int at) {
    if (!bit) return;
    a.ring[pp_wrap((int64_t)tail + at, a.P)] = p;
    a.holders_out[p] = 0;  // (entries beyond its holders have counted on)
  });
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(a.counter, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  int total = 0;
  for (int w = threadIdx.x; w < a.words; w += PP_THREADS) {
    total += __popc(a.bits[w]);
    a.bits[w] = 0u;
  }
  pp_scan(total, s_warp, all);
  if (threadIdx.x == 0) {
    *a.counter = 0u;
    a.state_out[0] = head;
    a.state_out[1] = (int)min((int64_t)count + all, (int64_t)a.P);
    a.state_out[2] = 0;
  }
}

// The pages that move: sources and destinations by their places among either, the ring, and the
// holders of the pages that do not move.
__global__ void __launch_bounds__(PP_THREADS) k_paged_moves(const PagesArgs a) {
  __shared__ int32_t s_warp[32];
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  int w0, w1, before = 0, some = 0, used, kept;
  pp_words(a, w0, w1);
  for (int w = threadIdx.x; w < a.words; w += PP_THREADS) {
    const int n = __popc(a.bits[w]);
    some += n;
    if (w < w0) before += n;
  }
  pp_scan(some, s_warp, used);
  __syncthreads();
  int all;
  pp_scan(before, s_warp, all);
  before = all;
  __syncthreads();
  some = 0;  // pages in use that stay: the bits below `used`
  for (int w = threadIdx.x; w * 32 < used; w += PP_THREADS) {
    const int left = used - w * 32;
    some += __popc(a.bits[w] & (left >= 32 ? ~0u : (1u << left) - 1));
  }
  pp_scan(some, s_warp, kept);
  const int most = a.P / 2, move = used - kept;
  pp_pages(a, w0, w1, before, s_warp, [&](int p, uint32_t bit, int at) {
    if (p < used) {
      if (bit) {
        a.holders_out[p] = a.holders[p];
      } else {
        const int r = p - at;  // free pages before it
        a.moves[2 * r + 1] = p;
      }
    } else if (bit) {
      a.moves[2 * (at - kept)] = p;
    } else {
      a.holders_out[p] = 0;
    }
    if (p < a.P - used) a.ring[p] = used + p;
    if (p >= move && p < most) a.moves[2 * p] = a.moves[2 * p + 1] = -1;
  });
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.state_out[0] = 0;
    a.state_out[1] = a.P - used;
    a.state_out[2] = 0;
  }
}

// The table's entries and the moved pages' holders by the new numbers.  A moved page's place is looked for among the moves,
// which are in ascending order (an unused one, -1, is the largest as an unsigned number): every stride-th, the CTA has in
// shared memory, between those by quarters, three loads at once.  These are scattered, a cycle of L1 each, so tasks go to
// as many SMs as there are.  96 requests of 100 to 8000 tokens: 12.3 us the call, 234 with its copies (16 tasks a CTA 13.9;
// quarters alone, without the samples, 236 with the copies; places kept in an array by page 10.1, but that array had to
// be cleared by another kernel).
__global__ void __launch_bounds__(PP_THREADS) k_paged_renumber(const PagesArgs a) {
  __shared__ uint32_t s_from[PP_THREADS + PP_THREADS / 32];  // (a place more after 32: the halves meet in no bank)
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, s = 1 << a.s_log2, most = a.P / 2;
  const int stride = (most + PP_THREADS - 1) / PP_THREADS;
  const uint32_t sample = (int64_t)tid * stride < most ? (uint32_t)a.moves[2 * tid * stride] : ~0u;
  const int used = a.P - a.state_out[1];
  const int64_t first = (int64_t)blockIdx.x * PP_THREADS + tid, all = (int64_t)gridDim.x * PP_THREADS;
  const int chunks = (a.width + PP_COLS - 1) / PP_COLS;
  const int64_t tasks = (int64_t)a.N * chunks, step = (int64_t)gridDim.x * PP_WARPS;
  int64_t t = (int64_t)(tid >> 5) * gridDim.x + blockIdx.x, row = 0;
  int c0 = 0, hi = 0, id[PP_COLS / 32];
  auto load = [&] {  // of task t
    if (t >= tasks) return;
    const int n = (int)(t / chunks);
    c0 = (int)(t - (int64_t)n * chunks) * PP_COLS;
    row = (int64_t)n * a.width;
    hi = min((int)(((int64_t)max(a.lens[n], 0) + s - 1) >> a.s_log2), a.width);
#pragma unroll
    for (int e = 0; e < PP_COLS / 32; ++e) id[e] = c0 + e * 32 + lane < a.width ? a.table[row + c0 + e * 32 + lane] : -1;
  };
  load();
  s_from[tid + (tid >> 5)] = sample;
  __syncthreads();
  for (; t < tasks; t += step, load()) {
    int r[PP_COLS / 32];
    bool moved[PP_COLS / 32];
#pragma unroll
    for (int e = 0; e < PP_COLS / 32; ++e) {
      moved[e] = c0 + e * 32 + lane < hi && id[e] >= used && id[e] < a.P;
      int at = 0;
#pragma unroll
      for (int d = PP_THREADS / 2; d; d >>= 1)
        if (s_from[at + d + ((at + d) >> 5)] <= (uint32_t)id[e]) at += d;
      r[e] = moved[e] ? at * stride : 0;
    }
    int d = 1;
    while (d * 4 < stride) d *= 4;
#pragma unroll 1
    for (; d && stride > 1; d >>= 2) {
      uint32_t from[PP_COLS / 32][3];
#pragma unroll
      for (int e = 0; e < PP_COLS / 32; ++e)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const int at = r[e] + (k + 1) * d;
          from[e][k] = moved[e] && at < most ? (uint32_t)a.moves[2 * at] : ~0u;
        }
#pragma unroll
      for (int e = 0; e < PP_COLS / 32; ++e) {
        int below = 0;
#pragma unroll
        for (int k = 0; k < 3; ++k) below += from[e][k] <= (uint32_t)id[e];
        r[e] += below * d;
      }
    }
#pragma unroll
    for (int e = 0; e < PP_COLS / 32; ++e) {
      const int col = c0 + e * 32 + lane;
      if (col < a.width) a.table_out[row + col] = moved[e] ? a.moves[2 * r[e] + 1] : id[e];
    }
  }
  for (int64_t i = first; i < a.P / 2; i += all) {
    const int from = a.moves[2 * i], to = a.moves[2 * i + 1];
    if (from < 0) break;  // (the moves come first)
    a.holders_out[to] = a.holders[from];
    a.holders_out[from] = 0;
  }
  for (int64_t w = first; w < a.words; w += all) a.bits[w] = 0u;
}

// ---------------------------------------------------------------- copy
// CTAs: a few moves each (x) of one piece of one cache's pages (y); moves that are none cost a read.
constexpr int COPY_THREADS = 256;
constexpr int COPY_MOVES = 4;     // of a CTA
constexpr int COPY_PIECE = 8192;  // bytes of a page that a CTA takes
constexpr int COPY_CACHES = 64;

struct CopyArgs {
  int M, P, n;
  const int32_t* moves;
  uint8_t* base[COPY_CACHES];
  int64_t stride[COPY_CACHES], bytes[COPY_CACHES];
  uint8_t vec[COPY_CACHES];      // log2 of the bytes of one access
  int32_t piece[COPY_CACHES + 1];  // first piece of each cache
};

template <class V>
__device__ __forceinline__ void copy_piece(const uint8_t* from, uint8_t* to, int64_t bytes) {
  constexpr int BATCH = COPY_PIECE / COPY_THREADS / 16;
  const int n = (int)(min(bytes, (int64_t)COPY_PIECE) / (int64_t)sizeof(V));
  for (int i0 = threadIdx.x; i0 < n; i0 += COPY_THREADS * BATCH) {
    V v[BATCH];
#pragma unroll
    for (int e = 0; e < BATCH; ++e)
      if (i0 + e * COPY_THREADS < n) v[e] = reinterpret_cast<const V*>(from)[i0 + e * COPY_THREADS];
#pragma unroll
    for (int e = 0; e < BATCH; ++e)
      if (i0 + e * COPY_THREADS < n) reinterpret_cast<V*>(to)[i0 + e * COPY_THREADS] = v[e];
  }
  // a page's last bytes, where they are no whole access
  for (int i = n * (int)sizeof(V) + threadIdx.x; i < min(bytes, (int64_t)COPY_PIECE); i += COPY_THREADS) to[i] = from[i];
}

__global__ void __launch_bounds__(COPY_THREADS) k_paged_copy(const __grid_constant__ CopyArgs a) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  int c = 0;
  while (c + 1 < a.n && a.piece[c + 1] <= (int)blockIdx.y) ++c;
  const int64_t off = (int64_t)((int)blockIdx.y - a.piece[c]) * COPY_PIECE;
  const int i0 = blockIdx.x * COPY_MOVES;
  for (int i = i0; i < min(i0 + COPY_MOVES, a.M); ++i) {
    const int from = a.moves[2 * i], to = a.moves[2 * i + 1];
    if ((uint32_t)from >= (uint32_t)a.P || (uint32_t)to >= (uint32_t)a.P) continue;
    const uint8_t* src = a.base[c] + from * a.stride[c] + off;
    uint8_t* dst = a.base[c] + to * a.stride[c] + off;
    const int64_t left = a.bytes[c] - off;
    if (a.vec[c] == 4)
      copy_piece<uint4>(src, dst, left);
    else if (a.vec[c] == 2)
      copy_piece<uint32_t>(src, dst, left);
    else
      copy_piece<uint8_t>(src, dst, left);
  }
}

// ---------------------------------------------------------------- host
int ctas_for(int64_t work, int per, int most = PP_MAX_CTAS) { return (int)std::min<int64_t>(std::max<int64_t>((work + per - 1) / per, 1), most); }

// holders_out = holders, where they are two
cudaError_t copy_counts(const int32_t* from, int32_t* to, int n, cudaStream_t stream) {
  if (from == to) return cudaSuccess;
  void* args[] = {&from, &to, &n};
  return launch_pdl(reinterpret_cast<const void*>(k_paged_counts), dim3(ctas_for(n, PP_THREADS)), dim3(PP_THREADS), 0, stream, args, 1);
}

template <class A>
cudaError_t launch(void (*f)(const A), int ctas, A& a, cudaStream_t stream) {
  void* args[] = {&a};
  return launch_pdl(reinterpret_cast<const void*>(f), dim3(ctas), dim3(PP_THREADS), 0, stream, args, 1);
}

}  // namespace

}  // namespace rglru

using namespace rglru;

extern "C" rglru_status paged_fork(const paged_shape* s, int32_t num_children, const int32_t* parents, const int32_t* children,
                                   const int32_t* block_table, const int32_t* kv_lens, const int32_t* holders,
                                   const int32_t* free_pages, const int32_t* free_state, int32_t* block_table_out,
                                   int32_t* kv_lens_out, int32_t* holders_out, int32_t* moves, int32_t* free_state_out,
                                   rglru_stream stream) {
  const rglru_status st = pg_check_cache(s);
  if (st != RGLRU_OK) return st;
  if (num_children < 0) return RGLRU_ERR_INVALID_ARG;
  if (num_children > PG_MAX_SEQS) return RGLRU_ERR_UNSUPPORTED;
  for (const void* p : {(const void*)block_table, (const void*)kv_lens, (const void*)holders, (const void*)free_pages,
                        (const void*)free_state, (const void*)block_table_out, (const void*)kv_lens_out,
                        (const void*)holders_out, (const void*)free_state_out})
    if (!pg_aligned(p, 4)) return RGLRU_ERR_INVALID_ARG;
  if (num_children > 0 && (!pg_aligned(parents, 4) || !pg_aligned(children, 4) || !pg_aligned(moves, 4)))
    return RGLRU_ERR_INVALID_ARG;
  ForkArgs a;
  a.N = s->num_seqs;
  a.M = num_children;
  a.P = s->num_pages;
  a.s_log2 = pg_log2(s->page_size);
  a.width = s->table_width;
  a.parents = parents;
  a.children = children;
  a.table = block_table;
  a.lens = kv_lens;
  a.ring = free_pages;
  a.state = free_state;
  a.table_out = block_table_out;
  a.lens_out = kv_lens_out;
  a.holders = holders_out;
  a.moves = moves;
  a.state_out = free_state_out;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = ta_prepare(reinterpret_cast<const void*>(k_paged_fork), (size_t)PG_MAX_SEQS * 8, 0, ready);
  if (e != cudaSuccess) return cuda_status(e);
  e = copy_counts(holders, holders_out, a.P, stream);
  if (e != cudaSuccess) return cuda_status(e);
  const int64_t tasks = (int64_t)a.M * ((a.width + PP_COLS - 1) / PP_COLS);
  const bool in_place = block_table_out == block_table || kv_lens_out == kv_lens || free_state_out == free_state;
  int ctas = ctas_for(tasks, PP_WARPS);
  a.cluster = 1;
  if (in_place && ctas > 1) ctas = a.cluster = PP_CLUSTER;
  void* args[] = {&a};
  return cuda_status(launch_pdl(reinterpret_cast<const void*>(k_paged_fork), dim3(ctas), dim3(PP_THREADS), (size_t)a.M * 8,
                                stream, args, a.cluster));
}

extern "C" size_t paged_pages_workspace_bytes(const paged_shape* s) {
  return pg_check_cache(s) == RGLRU_OK ? pages_ws_bytes(s->num_pages) : 0;
}

extern "C" rglru_status paged_release(const paged_shape* s, const int32_t* first_pages, const int32_t* end_pages,
                                      const int32_t* block_table, const int32_t* holders, int32_t* free_pages,
                                      const int32_t* free_state, int32_t* block_table_out, int32_t* holders_out,
                                      int32_t* free_state_out, void* workspace, rglru_stream stream) {
  const rglru_status st = pg_check_cache(s);
  if (st != RGLRU_OK) return st;
  for (const void* p : {(const void*)first_pages, (const void*)end_pages, (const void*)block_table, (const void*)holders,
                        (const void*)free_pages, (const void*)free_state, (const void*)block_table_out,
                        (const void*)holders_out, (const void*)free_state_out})
    if (!pg_aligned(p, 4)) return RGLRU_ERR_INVALID_ARG;
  if (!req(workspace)) return RGLRU_ERR_INVALID_ARG;
  PagesArgs a = {};
  a.N = s->num_seqs;
  a.P = s->num_pages;
  a.s_log2 = pg_log2(s->page_size);
  a.width = s->table_width;
  a.words = (a.P + 31) / 32;
  a.first = first_pages;
  a.end = end_pages;
  a.table = block_table;
  a.state = free_state;
  a.table_out = block_table_out;
  a.holders_out = holders_out;
  a.ring = free_pages;
  a.state_out = free_state_out;
  a.counter = static_cast<uint32_t*>(workspace);
  a.bits = a.counter + 64;
  cudaError_t e = copy_counts(holders, holders_out, a.P, stream);
  const int64_t tasks = (int64_t)a.N * ((a.width + PP_COLS - 1) / PP_COLS);
  if (e == cudaSuccess) e = launch(k_paged_mark<true>, ctas_for(tasks, PP_WARPS, 4 * PP_MAX_CTAS), a, stream);
  if (e == cudaSuccess) e = launch(k_paged_freed, ctas_for(a.words, PP_WARPS), a, stream);
  return cuda_status(e);
}

extern "C" rglru_status paged_compact(const paged_shape* s, const int32_t* kv_lens, const int32_t* block_table,
                                      const int32_t* holders, int32_t* block_table_out, int32_t* holders_out,
                                      int32_t* free_pages, int32_t* free_state_out, int32_t* moves, void* workspace,
                                      rglru_stream stream) {
  const rglru_status st = pg_check_cache(s);
  if (st != RGLRU_OK) return st;
  for (const void* p : {(const void*)kv_lens, (const void*)block_table, (const void*)holders, (const void*)block_table_out,
                        (const void*)holders_out, (const void*)free_pages, (const void*)free_state_out})
    if (!pg_aligned(p, 4)) return RGLRU_ERR_INVALID_ARG;
  if ((s->num_pages > 1 && !pg_aligned(moves, 4)) || !req(workspace)) return RGLRU_ERR_INVALID_ARG;
  PagesArgs a = {};
  a.N = s->num_seqs;
  a.P = s->num_pages;
  a.s_log2 = pg_log2(s->page_size);
  a.width = s->table_width;
  a.words = (a.P + 31) / 32;
  a.lens = kv_lens;
  a.table = block_table;
  a.holders = holders;
  a.table_out = block_table_out;
  a.holders_out = holders_out;
  a.ring = free_pages;
  a.state_out = free_state_out;
  a.moves = moves;
  a.counter = static_cast<uint32_t*>(workspace);
  a.bits = a.counter + 64;
  const int64_t tasks = (int64_t)a.N * ((a.width + PP_COLS - 1) / PP_COLS);
  cudaError_t e = launch(k_paged_mark<false>, ctas_for(tasks, PP_WARPS, 4 * PP_MAX_CTAS), a, stream);
  if (e == cudaSuccess) e = launch(k_paged_moves, ctas_for(a.words, PP_WARPS), a, stream);
  if (e == cudaSuccess) e = launch(k_paged_renumber, ctas_for(tasks, 1, 4 * PP_MAX_CTAS), a, stream);
  return cuda_status(e);
}

extern "C" rglru_status paged_copy(const paged_shape* s, int32_t num_moves, const int32_t* moves, int32_t num_caches,
                                   void* const* caches, const int64_t* page_strides, const int64_t* page_bytes,
                                   rglru_stream stream) {
  const rglru_status st = pg_check_cache(s);
  if (st != RGLRU_OK) return st;
  if (num_moves < 0 || num_caches < 0) return RGLRU_ERR_INVALID_ARG;
  if (num_moves > 0 && !pg_aligned(moves, 4)) return RGLRU_ERR_INVALID_ARG;
  if (num_caches > 0 && (!caches || !page_strides || !page_bytes)) return RGLRU_ERR_INVALID_ARG;
  for (int c = 0; c < num_caches; ++c) {
    if (!caches[c] || page_bytes[c] < 1 || page_strides[c] < page_bytes[c]) return RGLRU_ERR_INVALID_ARG;
    if (page_bytes[c] > 1 << 28) return RGLRU_ERR_UNSUPPORTED;
  }
  if (num_moves > 1 << 30) return RGLRU_ERR_UNSUPPORTED;  // (places in the list are counted in 32 bits)
  if (num_moves == 0) return RGLRU_OK;
  CopyArgs a;
  a.M = num_moves;
  a.P = s->num_pages;
  a.moves = moves;
  for (int c = 0; c < num_caches;) {
    int pieces = 0;
    for (a.n = 0; a.n < COPY_CACHES && c < num_caches; ++a.n, ++c) {
      const int more = (int)((page_bytes[c] + COPY_PIECE - 1) / COPY_PIECE);
      if (a.n > 0 && pieces + more > 65535) break;  // the grid's height
      const uint64_t all = reinterpret_cast<uintptr_t>(caches[c]) | (uint64_t)page_strides[c];
      a.base[a.n] = static_cast<uint8_t*>(caches[c]);
      a.stride[a.n] = page_strides[c];
      a.bytes[a.n] = page_bytes[c];
      a.vec[a.n] = all % 16 == 0 ? 4 : all % 4 == 0 ? 2 : 0;
      a.piece[a.n] = pieces;
      pieces += more;
    }
    a.piece[a.n] = pieces;
    void* args[] = {&a};
    const cudaError_t e = launch_pdl(reinterpret_cast<const void*>(k_paged_copy), dim3((a.M + COPY_MOVES - 1) / COPY_MOVES, pieces),
                                     dim3(COPY_THREADS), 0, stream, args, 1);
    if (e != cudaSuccess) return cuda_status(e);
  }
  return RGLRU_OK;
}

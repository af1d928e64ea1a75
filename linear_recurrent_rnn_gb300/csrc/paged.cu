// The paged key/value cache (include/paged_attn.h): the step's plan, the write of new keys and
// values, and the host side of the attention.
#include <math.h>

#include <algorithm>

#include "host_util.h"
#include "paged_tc.cuh"

namespace rglru {

namespace {

// ---------------------------------------------------------------- plan
// One launch.  Every CTA scans all requests (new tokens and pages wanted) into its own shared
// memory and then writes its share of the table entries and token rows: nothing waits for another
// CTA's result, as the page of a token in a new page is read from the ring itself, not from the
// table.  Updated in place (kv_lens = cached_lens or free_state_out = free_state) the CTAs must
// all have read before one writes, so they are then one cluster, which meets in between.
// Tokens: a warp takes 32 in a row and searches the offsets for the first; the others are mostly
// in the same request.  Latency-bound: the floor is a launch, two dependent reads (lengths, then
// table or ring) and the writes.  Measured (GB300): 3.0 us for 8 requests, 4.8 for 512, 6.0 for 1024
// requests with 83 000 new tokens; the last one in place, on the cluster's 8 CTAs, 23.
struct PlanArgs {
  int N, T, P, s, s_log2, width, cluster;
  const int32_t* cached;
  const int32_t* fresh;
  const int32_t* ring;
  const int32_t* state;
  int32_t* table;
  int32_t* cu;
  int32_t* kv_lens;
  int32_t* positions;
  int64_t* slots;
  int32_t* state_out;
};

constexpr int PLAN_THREADS = 512;
constexpr int PLAN_CLUSTER = 8;   // CTAs in place
constexpr int PLAN_CTAS = 128;    // CTAs otherwise, at most

constexpr size_t plan_smem(int N) { return (size_t)(3 * N + 2) * 4; }

__device__ __forceinline__ int plan_ceil(int64_t x, const PlanArgs& a) { return (int)((x + a.s - 1) >> a.s_log2); }

__global__ void __launch_bounds__(PLAN_THREADS) k_paged_plan(const PlanArgs a) {
  // per request: first row, first of its places in the ring's order, tokens cached
  extern __shared__ int32_t plan_sm[];
  int32_t* s_cu = plan_sm;
  int32_t* s_off = s_cu + a.N + 1;
  int32_t* s_c = s_off + a.N + 1;
  __shared__ int64_t s_warp[3][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int head = a.state[0], count = min(max(a.state[1], 0), a.P);
  // a thread's requests are neighbours: one scan over the CTA whatever their number
  const int per = a.N <= (int)blockDim.x ? 1 : (a.N + blockDim.x - 1) / blockDim.x;
  const int n0 = min(tid * per, a.N), n1 = min(n0 + per, a.N);
  int64_t q_sum = 0, p_sum = 0, over = 0;  // over: pages wanted past the table's width
  for (int n = n0; n < n1; ++n) {
    const int c = max(a.cached[n], 0), q = max(a.fresh[n], 0);
    const int held = plan_ceil(c, a), want = plan_ceil((int64_t)c + q, a);
    const int need = max(min(want, a.width) - min(held, a.width), 0);
    over += max(want - max(held, a.width), 0);
    s_c[n] = c;
    s_cu[n] = q;
    s_off[n] = need;
    q_sum += q;
    p_sum += need;
  }
  int64_t sq = q_sum, sp = p_sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, sq, d), v = __shfl_up_sync(0xffffffffu, sp, d);
    if (lane >= d) {
      sq += u;
      sp += v;
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) over += __shfl_xor_sync(0xffffffffu, over, d);
  if (lane == 31) {
    s_warp[0][warp] = sq;
    s_warp[1][warp] = sp;
    s_warp[2][warp] = over;
  }
  __syncthreads();
  int64_t all_q = 0, all_p = 0, all_over = 0;
  sq -= q_sum;
  sp -= p_sum;
  for (int k = 0; k < nw; ++k) {
    const int64_t u = s_warp[0][k], v = s_warp[1][k];
    all_q += u;
    all_p += v;
    all_over += s_warp[2][k];
    if (k < warp) {
      sq += u;
      sp += v;
    }
  }
  for (int n = n0; n < n1; ++n) {
    const int q = s_cu[n], need = s_off[n];
    s_cu[n] = (int)min(sq, (int64_t)0x7fffffff);
    s_off[n] = (int)min(sp, (int64_t)0x7fffffff);
    sq += q;
    sp += need;
  }
  if (tid == 0) {
    s_cu[a.N] = (int)min(all_q, (int64_t)0x7fffffff);
    s_off[a.N] = (int)min(all_p, (int64_t)0x7fffffff);
  }
  // in place: every CTA has read its inputs before any CTA writes
  if (a.cluster > 1) {
    __syncwarp();  // the barrier's form is the warp-aligned one
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  __syncthreads();
  const int h0 = (uint32_t)head < (uint32_t)a.P ? head : (head % a.P + a.P) % a.P;
  const int stride = gridDim.x * blockDim.x, first = blockIdx.x * blockDim.x + tid;
  if (first == 0) {
    const int taken = min(s_off[a.N], count);
    const int64_t next = (int64_t)h0 + taken;  // (taken <= P: at most once around)
    a.state_out[0] = (int)(next < a.P ? next : next - a.P);
    a.state_out[1] = count - taken;
    a.state_out[2] = (int)min((int64_t)s_off[a.N] - taken + all_over, (int64_t)0x7fffffff);
  }
  auto owner = [&](const int32_t* v, int x) {  // the last n with v[n] <= x
    int l = 0, h = a.N - 1;
    while (l < h) {
      const int mid = (l + h + 1) >> 1;
      if (v[mid] <= x) l = mid; else h = mid - 1;
    }
    return l;
  };
  auto ring = [&](int i) { return i < count ?  // (count <= P: at most once around)
                          a.ring[h0 + i < a.P ? h0 + i : h0 + i - a.P] : -1; };
  for (int n = first; n <= a.N; n += stride) {
    a.cu[n] = s_cu[n];
    if (n < a.N)
      a.kv_lens[n] = (int)min((int64_t)s_c[n] + (s_cu[n + 1] - s_cu[n]), (int64_t)0x7fffffff);
  }
  for (int64_t k = first; k < s_off[a.N]; k += stride) {  // (a step past the end may pass 2^31)
    const int i = (int)k, n = owner(s_off, i);
    a.table[(size_t)n * a.width + plan_ceil(s_c[n], a) + (i - s_off[n])] = ring(i);
  }
  const int total = s_cu[a.N];
  constexpr int BATCH = 4;  // rows of a thread whose pages are looked up at once
  for (int64_t t0 = first; t0 - lane < a.T; t0 += (int64_t)BATCH * stride) {
    int pos[BATCH], id[BATCH];
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const int64_t t = t0 + (int64_t)b * stride;
      pos[b] = 0;
      id[b] = -1;
      const int64_t w = t - lane;  // the warp's first row
      if (w >= a.T || w >= total) continue;
      int n = owner(s_cu, (int)w);
      if (s_cu[n + 1] < w + 32 && t < total) n = owner(s_cu, (int)t);
      if (t >= total) continue;
      const int c = s_c[n];
      pos[b] = (int)min((int64_t)c + (t - s_cu[n]), (int64_t)0x7fffffff);
      const int pg = pos[b] >> a.s_log2, held = plan_ceil(c, a);
      if (pg < a.width) id[b] = pg < held ? a.table[(size_t)n * a.width + pg] : ring(s_off[n] + pg - held);
    }
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const int64_t t = t0 + (int64_t)b * stride;
      if (t >= a.T) continue;
      a.positions[t] = pos[b];
      a.slots[t] = id[b] >= 0 ? ((int64_t)id[b] << a.s_log2) + (pos[b] & (a.s - 1)) : -1;
    }
  }
}

// ---------------------------------------------------------------- write
// A copy whose destination rows are chosen by the slots: a warp takes a token, its lanes the
// 16-byte pieces of the token's keys and then its values, so that a warp has all of a token's
// loads in flight at once (as many as its registers hold: stores may not be passed by later loads).
// Bound by memory bandwidth (and by latency for few tokens).  Measured (GB300): 16384 tokens of 8
// heads of 128, slices of a fused projection: 22.0 us, 6.1 TB/s read and written (one piece at a
// time: 23.9); 64 tokens: 2.0 us.
struct WriteArgs {
  int T, pieces, head_pieces, s_log2;  // 16-byte pieces of a token's keys, of one head
  int64_t slots_end;                   // num_pages * page_size
  const uint8_t* src[2];
  uint8_t* dst[2];
  int64_t src_token[2], src_head[2], dst_page[2], dst_token[2], dst_head[2];  // bytes
  const int64_t* slots;
};

constexpr int WRITE_THREADS = 256;
constexpr int WRITE_BATCH = 4;  // 16-byte pieces of a lane in flight

__global__ void __launch_bounds__(WRITE_THREADS) k_paged_write(const WriteArgs a) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int nwarps = gridDim.x * (WRITE_THREADS / 32);
  for (int t = blockIdx.x * (WRITE_THREADS / 32) + (threadIdx.x >> 5); t < a.T; t += nwarps) {
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.slots_end) continue;
    const int64_t page = slot >> a.s_log2, off = slot & ((1 << a.s_log2) - 1);
    for (int i0 = lane; i0 < 2 * a.pieces; i0 += 32 * WRITE_BATCH) {
      uint4 x[WRITE_BATCH];
      uint8_t* to[WRITE_BATCH];
#pragma unroll
      for (int e = 0; e < WRITE_BATCH; ++e) {
        const int i = i0 + 32 * e;
        to[e] = nullptr;
        if (i >= 2 * a.pieces) continue;
        const int kv = i >= a.pieces, c = kv ? i - a.pieces : i;
        const int h = c / a.head_pieces, b = (c - h * a.head_pieces) * 16;
        x[e] = *reinterpret_cast<const uint4*>(a.src[kv] + t * a.src_token[kv] + h * a.src_head[kv] + b);
        to[e] = a.dst[kv] + page * a.dst_page[kv] + off * a.dst_token[kv] + h * a.dst_head[kv] + b;
      }
#pragma unroll
      for (int e = 0; e < WRITE_BATCH; ++e)
        if (to[e]) *reinterpret_cast<uint4*>(to[e]) = x[e];
    }
  }
}

// ---------------------------------------------------------------- host
int elem_bytes(const paged_shape* s) { return s->io == RGLRU_BF16 ? 2 : 4; }

int log2_exact(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

rglru_status check_cache(const paged_shape* s) {
  if (!s || s->num_seqs < 1 || s->tokens < 0 || s->num_pages < 1 || s->page_size < 1 ||
      s->table_width < 1)
    return RGLRU_ERR_INVALID_ARG;
  if ((s->page_size & (s->page_size - 1)) || s->page_size < 8 || s->page_size > 4096 ||
      s->num_seqs > PG_MAX_SEQS || (int64_t)s->num_pages * s->page_size > 0x7fffffffLL ||
      s->tokens > PG_MAX_TOKENS || (int64_t)s->num_seqs * s->table_width > 0x7fffffffLL)
    return RGLRU_ERR_UNSUPPORTED;
  return RGLRU_OK;
}

rglru_status check_heads(const paged_shape* s) {
  if (s->Hkv < 1 || s->D < 1 || (s->io != RGLRU_F32 && s->io != RGLRU_BF16))
    return RGLRU_ERR_INVALID_ARG;
  if (s->D < 8 || s->D > 256 || s->D * elem_bytes(s) % 16) return RGLRU_ERR_UNSUPPORTED;
  return RGLRU_OK;
}

rglru_status check_queries(const paged_shape* s) {
  if (s->Hq < 1 || s->Hq % s->Hkv || s->window < 0) return RGLRU_ERR_INVALID_ARG;
  if (s->Hq / s->Hkv > 64) return RGLRU_ERR_UNSUPPORTED;
  return RGLRU_OK;
}

// Rows (tokens x query heads of a key/value head) of a request in the mean, rounded up to whole
// tokens: what the host knows of the lengths.  Every kernel is right for any lengths; the mean
// chooses among them.  bf16, 64 requests of 500 to 4096 keys, 32 heads on 8 of 128, few-rows kernel
// (tiles of 16 or 32 rows) against 128-row tiles: 4 rows a request 85 : 99 us, 16 rows 87 : 100,
// 20 rows 92 : 100, 32 rows 100 : 100, 40 rows (two tiles, keys read twice) 174 : 101.  These are
// batches of equal requests; the mean serves one long chunk among many decodes badly: 255 decodes of
// 64 to 8192 keys (292 us) and a chunk of 512 tokens on 4096 (50 us) take 561 us in one call, as the
// chunk's keys are read for every 4 of its tokens: better two calls.
int mean_rows(const paged_shape* s) {
  return (int)std::min<int64_t>(((int64_t)s->tokens + s->num_seqs - 1) / s->num_seqs * (s->Hq / s->Hkv), 1 << 30);
}

bool aligned(const void* p, size_t n) { return p && reinterpret_cast<uintptr_t>(p) % n == 0; }

paged_strides strides_of(const paged_shape* s, const paged_strides* given) {
  if (given) return *given;
  paged_strides t;
  t.q_token = t.o_token = (int64_t)s->Hq * s->D;
  t.k_token = t.v_token = t.kc_token = t.vc_token = (int64_t)s->Hkv * s->D;
  t.q_head = t.o_head = t.k_head = t.v_head = t.kc_head = t.vc_head = s->D;
  t.kc_page = t.vc_page = (int64_t)s->page_size * s->Hkv * s->D;
  return t;
}

// Strides are positive multiples of 16 bytes (16-byte loads, tensor maps).
bool strides_ok(const paged_shape* s, std::initializer_list<int64_t> v) {
  for (int64_t x : v)
    if (x <= 0 || x * elem_bytes(s) % 16) return false;
  return true;
}

}  // namespace

cudaError_t launch_pdl(const void* f, dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       void** args, int cluster) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cudaError_t e = cudaLaunchKernelExC(&cfg, f, args);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace rglru

using namespace rglru;

extern "C" rglru_status paged_plan(const paged_shape* s, const int32_t* cached_lens,
                                   const int32_t* new_lens, const int32_t* free_pages,
                                   const int32_t* free_state, int32_t* block_table,
                                   int32_t* cu_seqlens, int32_t* kv_lens, int32_t* positions,
                                   int64_t* slots, int32_t* free_state_out, rglru_stream stream) {
  const rglru_status st = check_cache(s);
  if (st != RGLRU_OK) return st;
  if (!aligned(cached_lens, 4) || !aligned(new_lens, 4) || !aligned(free_pages, 4) ||
      !aligned(free_state, 4) || !aligned(block_table, 4) || !aligned(cu_seqlens, 4) ||
      !aligned(kv_lens, 4) || !aligned(free_state_out, 4))
    return RGLRU_ERR_INVALID_ARG;
  if (s->tokens > 0 && (!aligned(positions, 4) || !aligned(slots, 8))) return RGLRU_ERR_INVALID_ARG;
  PlanArgs a;
  a.N = s->num_seqs;
  a.T = s->tokens;
  a.P = s->num_pages;
  a.s = s->page_size;
  a.s_log2 = log2_exact(s->page_size);
  a.width = s->table_width;
  a.cached = cached_lens;
  a.fresh = new_lens;
  a.ring = free_pages;
  a.state = free_state;
  a.table = block_table;
  a.cu = cu_seqlens;
  a.kv_lens = kv_lens;
  a.positions = positions;
  a.slots = slots;
  a.state_out = free_state_out;
  // once a device, to what the most requests take: a limit set call by call would be another
  // thread's too, between its own setting and its launch
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = ta_prepare(reinterpret_cast<const void*>(k_paged_plan), plan_smem(PG_MAX_SEQS), 0, ready);
  if (e != cudaSuccess) return cuda_status(e);
  const size_t smem = plan_smem(a.N);
  // one CTA up to a row a thread; beyond, one to two rows a thread, or the cluster
  const bool in_place = kv_lens == cached_lens || free_state_out == free_state;
  int ctas = 1, cluster = 1;
  if (s->tokens > PLAN_THREADS) {
    ctas = in_place ? PLAN_CLUSTER : std::min(PLAN_CTAS, (s->tokens + PLAN_THREADS - 1) / PLAN_THREADS);
    cluster = in_place ? PLAN_CLUSTER : 1;
  }
  a.cluster = cluster;
  // no more warps than requests and rows ask for: every warp reads every other's sums
  const int threads = (std::min(PLAN_THREADS, std::max(s->num_seqs, s->tokens)) + 31) / 32 * 32;
  void* args[] = {&a};
  return cuda_status(launch_pdl(reinterpret_cast<const void*>(k_paged_plan), dim3(ctas),
                                dim3(threads), smem, stream, args, cluster));
}

extern "C" rglru_status paged_kv_write(const paged_shape* s, const paged_strides* strides,
                                       const void* k, const void* v, const int64_t* slots,
                                       void* k_cache, void* v_cache, rglru_stream stream) {
  rglru_status st = check_cache(s);
  if (st == RGLRU_OK) st = check_heads(s);
  if (st != RGLRU_OK) return st;
  if (s->tokens == 0) return RGLRU_OK;
  if (!req(k) || !req(v) || !aligned(slots, 8) || !req(k_cache) || !req(v_cache))
    return RGLRU_ERR_INVALID_ARG;
  const paged_strides t = strides_of(s, strides);
  if (!strides_ok(s, {t.k_token, t.k_head, t.v_token, t.v_head, t.kc_page, t.kc_token, t.kc_head,
                      t.vc_page, t.vc_token, t.vc_head}))
    return RGLRU_ERR_UNSUPPORTED;
  const int es = elem_bytes(s);
  WriteArgs a;
  a.T = s->tokens;
  a.head_pieces = s->D * es / 16;
  a.pieces = s->Hkv * a.head_pieces;
  a.s_log2 = log2_exact(s->page_size);
  a.slots_end = (int64_t)s->num_pages * s->page_size;
  a.src[0] = static_cast<const uint8_t*>(k);
  a.src[1] = static_cast<const uint8_t*>(v);
  a.dst[0] = static_cast<uint8_t*>(k_cache);
  a.dst[1] = static_cast<uint8_t*>(v_cache);
  const int64_t str[2][5] = {{t.k_token, t.k_head, t.kc_page, t.kc_token, t.kc_head},
                             {t.v_token, t.v_head, t.vc_page, t.vc_token, t.vc_head}};
  for (int i = 0; i < 2; ++i) {
    a.src_token[i] = str[i][0] * es;
    a.src_head[i] = str[i][1] * es;
    a.dst_page[i] = str[i][2] * es;
    a.dst_token[i] = str[i][3] * es;
    a.dst_head[i] = str[i][4] * es;
  }
  a.slots = slots;
  const int per = WRITE_THREADS / 32;
  const int blocks = (int)std::min<int64_t>(((int64_t)a.T + per - 1) / per, 1 << 16);
  void* args[] = {&a};
  return cuda_status(launch_pdl(reinterpret_cast<const void*>(k_paged_write), dim3(blocks),
                                dim3(WRITE_THREADS), 0, stream, args, 1));
}

extern "C" size_t paged_attention_workspace_bytes(const paged_shape* s) {
  if (check_cache(s) != RGLRU_OK || check_heads(s) != RGLRU_OK || check_queries(s) != RGLRU_OK)
    return 0;
  const int rows = mean_rows(s);
  if (s->io == RGLRU_F32) return paged_attn_simt_ws_bytes(s, rows);
  return rows <= PG_FEW_ROWS ? paged_attn_few_ws_bytes(s, rows) : paged_attn_tc_ws_bytes(s);
}

extern "C" rglru_status paged_attention(const paged_shape* s, const paged_strides* strides,
                                        const void* q, const void* k_cache, const void* v_cache,
                                        const int32_t* block_table, const int32_t* cu_seqlens,
                                        const int32_t* kv_lens, float scale, void* o, float* lse,
                                        void* workspace, rglru_stream stream) {
  rglru_status st = check_cache(s);
  if (st == RGLRU_OK) st = check_heads(s);
  if (st == RGLRU_OK) st = check_queries(s);
  if (st != RGLRU_OK) return st;
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!(scale > 0.0f) || !isfinite(scale_log2)) return RGLRU_ERR_INVALID_ARG;
  if (s->tokens == 0) return RGLRU_OK;
  if (!req(q) || !req(k_cache) || !req(v_cache) || !aligned(block_table, 4) ||
      !aligned(cu_seqlens, 4) || !aligned(kv_lens, 4) || !req(o) ||
      (lse && !aligned(lse, 4)) || !req(workspace))
    return RGLRU_ERR_INVALID_ARG;
  const paged_strides t = strides_of(s, strides);
  if (!strides_ok(s, {t.q_token, t.q_head, t.o_token, t.o_head, t.kc_page, t.kc_token, t.kc_head,
                      t.vc_page, t.vc_token, t.vc_head}))
    return RGLRU_ERR_UNSUPPORTED;
  PagedArgs a = {};
  a.N = s->num_seqs;
  a.T = s->tokens;
  a.Hq = s->Hq;
  a.Hkv = s->Hkv;
  a.g = s->Hq / s->Hkv;
  a.g_inv = (65536u + a.g - 1) / a.g;
  a.D = s->D;
  a.P = s->num_pages;
  a.ps_log2 = log2_exact(s->page_size);
  a.table_width = s->table_width;
  a.window = s->window < 1 << 30 ? s->window : 0;  // (lengths are clamped to 2^30)
  a.scale_log2 = scale_log2;
  a.q = q;
  a.kc = k_cache;
  a.vc = v_cache;
  a.table = block_table;
  a.cu = cu_seqlens;
  a.kv_lens = kv_lens;
  a.o = o;
  a.lse = lse;
  a.q_token = t.q_token;
  a.q_head = t.q_head;
  a.o_token = t.o_token;
  a.o_head = t.o_head;
  a.kc_page = t.kc_page;
  a.kc_token = t.kc_token;
  a.kc_head = t.kc_head;
  a.vc_page = t.vc_page;
  a.vc_token = t.vc_token;
  a.vc_head = t.vc_head;
  a.ws = static_cast<uint8_t*>(workspace);
  // rglru_debug_lookback: the limit in polls, taken as 100 ns each, and the CTA without work
  a.drop_cta = debug_drop_tile();
  a.wait_ns = a.drop_cta >= 0 ? (uint64_t)debug_spin_limit() * 100 : TA_WAIT_NS;
  const int rows = mean_rows(s);
  if (s->io == RGLRU_F32) return cuda_status(launch_paged_attn_simt(a, rows, stream));
  return cuda_status(rows <= PG_FEW_ROWS ? launch_paged_attn_few(a, rows, stream)
                                         : launch_paged_attn_tc(a, stream));
}

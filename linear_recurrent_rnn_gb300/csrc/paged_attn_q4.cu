// Attention over the paged cache held in 4 bits (include/paged_q4.h), R rows a row tile (whole tokens x
// the query heads of one key/value head).
//
// As in the kernel for few rows over a bf16 cache (paged_attn_few.cu), keys lie along the 128 rows of the
// tensor core's tile:
//   S^T = K Q^T       128 keys x the rows; S^T in TMEM, float32
//   P^T = 2^(c S^T - c m)     one key a thread, to shared memory as f16
//   O^T += V^T P^T    D x the rows; V read transposed by the tensor core, O^T in TMEM, float32
// What is new is the way of keys and values to the tensor core.  Codes and scales come to shared memory
// by cp.async, a quarter of bf16's bytes, and dequantising warps write the numbers that they stand for to
// a second ring as f16.  A code times its scale has 6 significant bits at most, so f16 holds it
// exactly (2^-10 to 2688).  Rows that no row of the item sees, and pages that are not there, are copied
// as zeros (cp.async with fewer source bytes), so nothing stale reaches a product.
//
// Queries are f16 too, as the tensor core takes two operands of one type: each row is multiplied by
// the power of two that brings its largest element to [2^14, 2^15), and its scores by the inverse.
// bf16's 8 significant bits fit f16's 11.  float32 queries and weights are split into two f16 numbers
// (22 bits), rows of their own in the products, added in float32.  Weights are held times 2^11, so
// that f16's range, 2^-25 to 2^15, is used from the largest weight down; the reference m is moved when a
// weight would pass 2^15.
//
// Warps: 4 softmax, 2 that copy codes, MMA issuer (one thread), one that walks the items and loads
// queries, 8 that dequantise.
#include <float.h>

#include <algorithm>

#include "host_util.h"
#include "paged_q4.cuh"

namespace rglru {

namespace {

constexpr int TQ_SOFT = 128;
constexpr int TQ_LOAD = 64;     // threads that copy
constexpr int TQ_DEQ = 256;     // threads that dequantise
constexpr int TQ_THREADS = TQ_SOFT + 128 + TQ_DEQ;
constexpr size_t TQ_SMEM_MAX = 232448 - 4096;  // 227 KB less the static part
constexpr float TQ_SHIFT = 11.0f;  // weights are held times 2^TQ_SHIFT
constexpr float TQ_TOP = 15.0f;    // and stay below 2^TQ_TOP

template <int DP, int R_, bool F32_>
struct Tq {
  static constexpr int R = R_;
  static constexpr bool F32 = F32_;
  static constexpr int NR = F32 ? 2 * R : R;          // columns of the products
  static constexpr int SLABS = DP / 64;
  static constexpr int UPT = DP == 256 ? 2 : 1;       // ring units of a key (or value) tile
  static constexpr uint32_t UB = DP == 64 ? TA_SLAB : 2 * TA_SLAB;
  static constexpr int VROWS = TA_BN / UPT;           // rows of V in a unit
  static constexpr int MH = DP == 256 ? 2 : 1;        // products of 128 columns of V
  static constexpr uint32_t RB = DP / 2, SP = DP / 16;  // bytes of a row's codes, of its scales
  static constexpr uint32_t SB = 1024 * ((TA_BN * (RB + SP) + 1023) / 1024);  // a tile's
  static constexpr uint32_t QSLAB = NR * 128;         // 64 columns of the rows of Q
  static constexpr uint32_t QB = SLABS * QSLAB;
  static constexpr int QBUF = QB <= 8192 ? 4 : 2;
  static constexpr uint32_t PROW = NR * 2;            // a key's weights
  static constexpr uint32_t PB = TA_BN * PROW;
  static constexpr uint32_t P_LAYOUT = NR == 16 ? tc::LAYOUT_SW32 : tc::LAYOUT_SW64;
  static constexpr int STAGES = 3;                    // units as f16
  static constexpr int FIT = (int)((TQ_SMEM_MAX - 1024 - QBUF * QB - 2 * PB - STAGES * UB - 1024) / SB);
  static constexpr int COPIES = FIT < 16 ? FIT : 16;  // tiles of codes on their way
  static constexpr uint32_t S_COL = 0, O_COL = 128;   // TMEM: S^T buffers, O^T buffers
  static constexpr size_t smem = 1024 + STAGES * UB + (size_t)COPIES * SB + QBUF * QB + 2 * PB + 1024;
  // slabs of 64 columns, 128-byte swizzle, a slab's rows together
  static constexpr uint32_t K_SLAB = TA_SLAB, V_SLAB = VROWS * 128;
  static_assert(COPIES >= 4, "shared memory");
};

__device__ __forceinline__ uint32_t tq_pack(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return reinterpret_cast<const uint32_t&>(v);
}
// what is left of a pair after its rounding to f16
__device__ __forceinline__ uint32_t tq_rest(float lo, float hi, uint32_t rounded) {
  const float2 v = __half22float2(reinterpret_cast<const __half2&>(rounded));
  return tq_pack(lo - v.x, hi - v.y);
}

// `bytes` of 16 (or 4) copied, zeros behind them; nothing is read where it is 0.
__device__ __forceinline__ void tq_copy16(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tq_copy4(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
// Arrives on `bar` once this thread's copies so far are done.
__device__ __forceinline__ void tq_copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}

// A row's 16-byte pieces of codes lie where neither the copies nor the dequantising threads, a row a thread,
// meet in a bank.
template <class C>
__device__ __forceinline__ uint32_t tq_code(int r, int piece) {
  const int x = C::RB == 128 ? r & 7 : C::RB == 64 ? r >> 1 & 3 : r >> 2 & 1;
  return r * C::RB + ((piece ^ x) << 4);
}

// Copies tiles of codes and scales into the ring, by two warps, each half of a tile's rows.
template <class C>
struct TqLoader {
  const PagedArgs& a;
  const Q4Cache& c;
  const TaAbort& ctl;
  uint8_t* ring;
  uint64_t* full;
  uint64_t* empty;
  int* kinds;
  int half;
  uint32_t st = 0, ph = 1;  // next stage, parity of its `empty`

  // This lane's page of key tile j, for the 8 rows from row 64 half + 8 lane on (-1: zeros).
  __device__ __forceinline__ int page_of(const TaItem& it, int j) const {
    const int lane = threadIdx.x & 31, pos = j * TA_BN + 64 * half + 8 * lane, pg = pos >> a.ps_log2;
    if (j >= it.j1 || lane >= 8 || pos >= it.hi || pos + 8 <= it.lo || pg >= a.table_width) return -1;
    const int id = a.table[(int64_t)it.n * a.table_width + pg];
    return id >= 0 && id < a.P ? id : -1;
  }
  __device__ __forceinline__ bool tile(bool v, int j, int id, int h, int lo, int hi) {
    if (!ctl.wait(&empty[st], ph)) return false;
    const int lane = threadIdx.x & 31;
    uint8_t* dst = ring + st * C::SB;
    const int64_t token = v ? c.vc_token : c.kc_token, s_token = v ? c.vs_token : c.ks_token;
    const uint8_t* codes = v ? c.vc : c.kc;
    const uint8_t* scales = v ? c.vs : c.ks;
    // where this lane's 8 rows begin
    const int off = (j * TA_BN + 64 * half + 8 * lane) & ((1 << a.ps_log2) - 1);
    const int64_t at = max(id, 0) * (v ? c.vc_page : c.kc_page) + h * (v ? c.vc_head : c.kc_head) + off * token;
    const int64_t s_at = max(id, 0) * (v ? c.vs_page : c.ks_page) + h * (v ? c.vs_head : c.ks_head) + off * s_token;
    constexpr int CPR = C::RB / 16, RPI = 32 / CPR;  // pieces of a row, rows of an instruction
    const int piece = lane % CPR;
#pragma unroll
    for (int i = 0; i < 64 / RPI; ++i) {
      const int r = i * RPI + lane / CPR, row = 64 * half + r, pos = j * TA_BN + row;
      const int64_t base = __shfl_sync(0xffffffffu, at, r >> 3);
      const bool there = __shfl_sync(0xffffffffu, id, r >> 3) >= 0 && pos >= lo && pos < hi;
      const int bytes = there ? min(max(a.D / 2 - piece * 16, 0), 16) : 0;
      tq_copy16(dst + tq_code<C>(row, piece), bytes ? codes + base + (r & 7) * token + piece * 16 : codes, bytes);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 32 * i + lane, row = 64 * half + r, pos = j * TA_BN + row;
      const int64_t base = __shfl_sync(0xffffffffu, s_at, r >> 3);
      const bool there = __shfl_sync(0xffffffffu, id, r >> 3) >= 0 && pos >= lo && pos < hi;
#pragma unroll
      for (int w = 0; w < (int)C::SP / 4; ++w) {
        const int bytes = there ? min(max(a.D / 16 - 4 * w, 0), 4) : 0;
        tq_copy4(dst + TA_BN * C::RB + row * C::SP + 4 * w, bytes ? scales + base + (r & 7) * s_token + 4 * w : scales, bytes);
      }
    }
    if (half == 0 && lane == 0) {
      kinds[st] = v;
      tc::mbar_arrive(&full[st]);
    }
    tq_copies_arrive(&full[st]);
    advance();
    return true;
  }
  __device__ __forceinline__ void advance() {
    __syncwarp();
    if (++st == C::COPIES) {
      st = 0;
      ph ^= 1;
    }
  }
  // No more tiles.
  __device__ __forceinline__ void end() {
    if (!ctl.wait(&empty[st], ph)) return;
    if (half == 0 && (threadIdx.x & 31) == 0) {
      kinds[st] = -1;
      tc::mbar_arrive(&full[st]);
    }
    tc::mbar_arrive(&full[st]);
  }
};

template <int DP, int R, bool F32>
__global__ void __launch_bounds__(TQ_THREADS, 1)
    k_paged_attn_q4(const __grid_constant__ PagedArgs a, const __grid_constant__ Q4Cache cache) {
  using C = Tq<DP, R, F32>;
  constexpr int NR = C::NR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* s_ring = smem;
  uint8_t* s_copy = s_ring + (size_t)C::STAGES * C::UB;
  uint8_t* s_q = s_copy + (size_t)C::COPIES * C::SB;
  uint8_t* s_p = s_q + C::QBUF * C::QB;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_p + 2 * C::PB);
  uint64_t* empty = full + C::STAGES;
  uint64_t* c_full = empty + C::STAGES;    // [COPIES] a tile's codes are there
  uint64_t* c_empty = c_full + C::COPIES;  // [COPIES] and have been read
  uint64_t* q_full = c_empty + C::COPIES;  // [QBUF]
  uint64_t* q_empty = q_full + C::QBUF;    // [QBUF]
  uint64_t* s_full = q_empty + C::QBUF;    // [2] S^T of buffer b complete
  uint64_t* p_full = s_full + 2;           // [2] P^T of buffer b written (and O^T scaled)
  uint64_t* pv_done = p_full + 2;          // [2] the product with P^T of buffer b complete
  uint64_t* o_empty = pv_done + 2;         // [2] O^T buffer read
  uint64_t* i_full = o_empty + 2;          // [TA_ITEMS] item records
  uint64_t* i_empty = i_full + TA_ITEMS;
  uint64_t* r_full = i_empty + TA_ITEMS;   // [TA_ITEMS] the factors of an item's rows
  uint64_t* drain = r_full + TA_ITEMS;
  __shared__ int64_t scratch[33];
  __shared__ TaItem s_item[TA_ITEMS];
  __shared__ uint32_t tmem_holder, s_flag, s_last;
  __shared__ int s_kind[C::COPIES];                          // of a tile: 0 keys, 1 values, -1 no more
  __shared__ float s_red[4][R];                              // a value a softmax warp and row
  __shared__ __align__(16) float s_ref[R], s_scale[R];       // the rows' references; factors of a change
  __shared__ __align__(16) float s_factor[TA_ITEMS][R];      // of the rows' scores
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // < 0: softmax; 0, 1: copies, 2: MMA, 3: walk and queries, 4 and on: dequantising
  const int role = warp - TQ_SOFT / 32;
  const TaAbort ctl{&s_flag, reinterpret_cast<uint32_t*>(a.ws), a.wait_ns};

  // up to griddep_wait nothing touches global memory
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      tc::mbar_init(&full[i], TQ_DEQ / 32);
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::COPIES; ++i) {
      tc::mbar_init(&c_full[i], TQ_LOAD + 1);
      tc::mbar_init(&c_empty[i], TQ_DEQ / 32);
    }
    for (int i = 0; i < C::QBUF; ++i) {
      tc::mbar_init(&q_full[i], 1);
      tc::mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s_full[i], 1);
      tc::mbar_init(&p_full[i], TQ_SOFT / 32);
      tc::mbar_init(&pv_done[i], 1);
      tc::mbar_init(&o_empty[i], TQ_SOFT / 32);
    }
    for (int i = 0; i < TA_ITEMS; ++i) {
      tc::mbar_init(&i_full[i], 1);
      tc::mbar_init(&i_empty[i], TQ_SOFT / 32 + 3);
      tc::mbar_init(&r_full[i], 1);
    }
    tc::mbar_init(drain, 1);
    s_flag = 0u;
    tc::fence_barrier_init();
  }
  if (role == 2) {
    tc::tmem_alloc(&tmem_holder, 512);
    tc::tmem_relinquish();
  }
  tc::griddep_wait();
  // By the warp that holds the TMEM, not before: a CTA of the next grid that takes TMEM keeps it until
  // this grid has ended.
  if (role == 2) tc::griddep_launch_dependents();
  PgWalk w;
  PgWalk::Found start;
  if (a.N <= PG_WARP_SEQS) {
    if (role == 3) start = w.find_warp(a);
  } else {
    int64_t* prefix = reinterpret_cast<int64_t*>(s_ring);  // before the ring is in use
    pg_scan(a, prefix, scratch);
    if (role == 3) start = w.find(a, prefix);
  }
  tc::fence_proxy_async_smem();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_holder;

  if (role < 0) {
    // ------------------------------------------------------------ softmax, one key a thread
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    uint32_t step = 0, no = 0;  // key tiles, items with an O^T so far
    bool ok = true;
    for (uint32_t ni = 0;; ++ni) {
      ok = ctl.wait(&i_full[ni % TA_ITEMS], ni / TA_ITEMS & 1);
      if (tf_any(!ok)) break;
      const TaItem& it = s_item[ni % TA_ITEMS];
      if (it.n < 0) break;
      const int j0 = it.j0, j1 = it.j1;
      const int rows = min(a.tb, it.q - it.tok) * a.g;
      const int p_first = it.kv - it.q + it.tok, p_last = p_first + min(a.tb, it.q - it.tok) - 1;
      const uint32_t ob = no & 1, t_o = lanes + C::O_COL + ob * (C::MH * NR);
      float ref[R], l[R];  // the rows' references (scores in log2 units), this thread's sums
#pragma unroll
      for (int c = 0; c < R; ++c) l[c] = ref[c] = 0.0f;
      const float* factor = s_factor[ni % TA_ITEMS];
      ok = ctl.wait(&r_full[ni % TA_ITEMS], ni / TA_ITEMS & 1);
      bool out = false;
      for (int j = j0; j < j1; ++j, ++step) {
        const uint32_t b = step & 1;
        ok = ctl.wait(&s_full[b], step >> 1 & 1) && ok;
        tc::tc_fence_after();
        float x[NR];
#pragma unroll
        for (int c = 0; c < NR; c += 16)
          tc::tmem_ld16(lanes + C::S_COL + b * NR + c, *reinterpret_cast<float(*)[16]>(x + c));
        tc::tmem_ld_wait();
        tc::reg_fence(x);
        if (F32)
#pragma unroll
          for (int c = 0; c < R; ++c) x[c] += x[NR - R + c];
        const int k0 = j * TA_BN;
        float worst = -INFINITY;
#pragma unroll
        for (int c = 0; c < R; c += 4) {
          const float4 f = *reinterpret_cast<const float4*>(factor + c);
          x[c] *= f.x;
          x[c + 1] *= f.y;
          x[c + 2] *= f.z;
          x[c + 3] *= f.w;
        }
        if (k0 + TA_BN - 1 > p_first || (a.window && k0 < p_last - a.window + 1)) {
          int p = p_first, h = 0;  // row c's position
#pragma unroll
          for (int c = 0; c < R; ++c) {
            if (k0 + tid > p || (a.window && k0 + tid <= p - a.window)) x[c] = -INFINITY;
            if (++h == a.g) {
              h = 0;
              ++p;
            }
          }
        }
#pragma unroll
        for (int c = 0; c < R; ++c) worst = fmaxf(worst, x[c] - ref[c]);
        if (tf_any(!ok || j == j0 || worst > TQ_TOP)) {
          // new references: the rows' maxima so far, less the shift
          float v[R];
#pragma unroll
          for (int c = 0; c < R; ++c) v[c] = x[c];
          tf_combine<R>(v, [](float p, float q) { return fmaxf(p, q); });
          s_red[warp][tf_column<R>()] = v[0];
          if (j > j0) ok = ctl.wait(&pv_done[b ^ 1], (step - 1) >> 1 & 1) && ok;
          if (tf_any(!ok)) {
            out = true;
            break;
          }
          if (tid < R) {
            // the lowest finite number: no score is below it, and a key that is not seen (-inf) weighs 0
            const float m0 = j == j0 ? -FLT_MAX : s_ref[tid];
            const float seen = fmaxf(fmaxf(s_red[0][tid], s_red[1][tid]), fmaxf(s_red[2][tid], s_red[3][tid]));
            // Rows that the tile has to spare see stale keys' zeros: with an infinite reference they weigh
            // nothing and never ask for a change.
            const float m = tid < rows ? fmaxf(seen - TQ_SHIFT, m0) : INFINITY;
            s_scale[tid] = m0 == m ? 1.0f : ta_ex2(m0 - m);
            s_ref[tid] = m;
          }
          tf_any(false);
#pragma unroll
          for (int c = 0; c < R; c += 4)
            *reinterpret_cast<float4*>(ref + c) = *reinterpret_cast<const float4*>(s_ref + c);
          if (j > j0) {
            tc::tc_fence_after();
#pragma unroll
            for (int c = 0; c < R; ++c) l[c] *= s_scale[c];
#pragma unroll 1
            for (int c = 0; c < C::MH * NR; c += 4) {
              float o[4];
              tc::tmem_ld4(t_o + c, o);
              tc::tmem_ld_wait();
              tc::reg_fence(o);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[e] *= s_scale[c % R + e];
              tc::tmem_st4(t_o + c, o);
            }
            tc::tmem_st_wait();
          }
        }
        uint32_t pk[NR / 2];
#pragma unroll
        for (int c = 0; c < R; c += 2) {
          const float p0 = ta_ex2(x[c] - ref[c]), p1 = ta_ex2(x[c + 1] - ref[c + 1]);
          l[c] += p0;
          l[c + 1] += p1;
          pk[c / 2] = tq_pack(p0, p1);
          if (F32) pk[(NR - R + c) / 2] = tq_rest(p0, p1, pk[c / 2]);
        }
        ok = ctl.wait(&pv_done[b], (step >> 1 & 1) ^ 1) && ok;  // P^T of two steps ago is used up
        // key tid's row of P^T: 16-byte pieces where the tensor core's swizzle has them
        uint8_t* row = s_p + b * C::PB + tid * C::PROW;
        const int sw = NR == 16 ? tid >> 2 & 1 : tid >> 1 & 3;
#pragma unroll
        for (int c = 0; c < NR / 8; ++c)
          *reinterpret_cast<uint4*>(row + ((c ^ sw) << 4)) =
              make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&p_full[b]);
      }
      if (out) break;
      const bool any = j1 > j0;
      // the rows' sums over the threads
      tf_combine<R>(l, [](float p, float q) { return p + q; });
      s_red[warp][tf_column<R>()] = l[0];
      if (any) {
        ok = ctl.wait(&pv_done[(step - 1) & 1], (step - 1) >> 1 & 1) && ok;
        tc::tc_fence_after();
        ++no;
      }
      if (tf_any(!ok)) break;
      const bool whole = it.c0 == it.c1;
      const int tok0 = it.first + it.tok;
      auto row_sum = [&](int c) { return (s_red[0][c] + s_red[1][c]) + (s_red[2][c] + s_red[3][c]); };
      if (tid < rows) {
        const float sum = row_sum(tid);
        if (!whole)
          reinterpret_cast<float2*>(a.ws + a.part_ml)[(size_t)it.slot * R + tid] = make_float2(s_ref[tid], sum);
        else if (a.lse)
          a.lse[(int64_t)(tok0 + pg_token(a, tid)) * a.Hq + it.h * a.g + tid - pg_token(a, tid) * a.g] =
              tf_lse(s_ref[tid], sum);
      }
      {
        int64_t dst = tok0 * a.o_token + (int64_t)it.h * a.g * a.o_head + tid;
        float* po = reinterpret_cast<float*>(a.ws + a.part_o) + (size_t)it.slot * R * DP + tid;
        int h = 0;
#pragma unroll 1
        for (int c = 0; c < rows; c += 4) {
          __syncwarp();  // (TMEM is read by whole warps)
          float o[C::MH][4], o2[C::MH][4];
#pragma unroll
          for (int hm = 0; hm < C::MH; ++hm) {
            if (any) tc::tmem_ld4(t_o + hm * NR + c, o[hm]);
            if (any && F32) tc::tmem_ld4(t_o + hm * NR + R + c, o2[hm]);
          }
          if (any) tc::tmem_ld_wait();
#pragma unroll
          for (int hm = 0; hm < C::MH; ++hm) {
            tc::reg_fence(o[hm]);
            if (F32) {
              tc::reg_fence(o2[hm]);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[hm][e] += o2[hm][e];
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (c + e >= rows) break;
            if (whole) {
              const float sum = row_sum(c + e), inv = __fdividef(1.0f, sum);
#pragma unroll
              for (int hm = 0; hm < C::MH; ++hm) {
                const float y = sum == 0.0f ? 0.0f : o[hm][e] * inv;
                if (hm * 128 + tid >= a.D) continue;
                if (F32)
                  static_cast<float*>(a.o)[dst + hm * 128] = y;
                else
                  static_cast<bf16*>(a.o)[dst + hm * 128] = __float2bfloat16_rn(y);
              }
              dst += a.o_head;
              if (++h == a.g) {
                h = 0;
                dst += a.o_token - a.g * a.o_head;
              }
            } else if (any) {
#pragma unroll
              for (int hm = 0; hm < C::MH; ++hm)
                if (hm * 128 + tid < DP) po[(c + e) * DP + hm * 128] = o[hm][e];
            }
          }
        }
      }
      if (any) tc::tc_fence_before();
      if (!whole) {
        tf_any(false);
        if (tid == 0) {
          __threadfence();  // cumulative: the other threads' parts, ordered before by the barrier
          uint32_t* cnt = reinterpret_cast<uint32_t*>(a.ws + 256) + it.c0;
          const bool last = atomicAdd(cnt, 1u) == (uint32_t)(it.c1 - it.c0);
          if (last) *cnt = 0u;  // as it was found: zero between calls
          s_last = last;
        }
        tf_any(false);
        if (s_last) {
          // The item's last CTA joins its parts, up to PARTS at a time: first their weights (in the
          // buffers of P^T, which nothing uses now), then the sums, a thread four columns of every
          // RP-th row.
          __threadfence();
          float2* wt = reinterpret_cast<float2*>(s_p);  // [part][row]
          constexpr int PARTS = 2 * C::PB / (R * 8), RP = 512 / DP, PASSES = R / RP;
          constexpr int BATCH = PASSES >= 16 ? 1 : 16 / PASSES;  // parts loaded at once
          const int col = tid % (DP / 4) * 4, r0 = tid / (DP / 4);
          float4 o[PASSES];
#pragma unroll
          for (int k = 0; k < PASSES; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          float m = -INFINITY, sum = 0.0f;  // of row tid
          for (int q0 = it.c0; q0 <= it.c1; q0 += PARTS) {
            const int nq = min(PARTS, it.c1 - q0 + 1);
            // the first parts' sums are on their way while their weights are worked out
            const float* po = reinterpret_cast<const float*>(a.ws + a.part_o) + r0 * DP + col;
            float4 v[BATCH][PASSES];
            auto load = [&](int qb) {
#pragma unroll
              for (int b = 0; b < BATCH; ++b) {
                const float* pq = po + (size_t)PgWalk::slot(q0 + min(qb + b, nq - 1), it.c0) * R * DP;
#pragma unroll
                for (int k = 0; k < PASSES; ++k) v[b][k] = __ldcg(reinterpret_cast<const float4*>(pq + k * RP * DP));
              }
            };
            load(0);
#pragma unroll 1
            for (int i = tid; i < nq * R; i += TQ_SOFT)
              wt[i] = i % R < rows ? __ldcg(reinterpret_cast<const float2*>(a.ws + a.part_ml) +
                                            (size_t)PgWalk::slot(q0 + i / R, it.c0) * R + i % R)
                                   : make_float2(0.0f, 0.0f);
            tf_any(false);
            if (tid < R) {
              const float m0 = m;
#pragma unroll 4
              for (int q = 0; q < nq; ++q) m = fmaxf(m, wt[q * R + tid].y != 0.0f ? wt[q * R + tid].x : -INFINITY);
              const float f = m0 == m ? 1.0f : ta_ex2(m0 - m);
              sum *= f;
#pragma unroll 4
              for (int q = 0; q < nq; ++q) {
                const float2 x = wt[q * R + tid];  // a part that saw nothing did not write its sums
                const float e = x.y != 0.0f ? ta_ex2(x.x - m) : 0.0f;
                sum += x.y * e;
                wt[q * R + tid].x = e;
              }
              s_scale[tid] = f;
              s_ref[tid] = sum;
            }
            tf_any(false);
            if (q0 > it.c0)
#pragma unroll
              for (int k = 0; k < PASSES; ++k) {
                const float f = s_scale[r0 + k * RP];
                o[k] = make_float4(o[k].x * f, o[k].y * f, o[k].z * f, o[k].w * f);
              }
#pragma unroll 1
            for (int q = 0; q < nq; q += BATCH) {
              if (q > 0) load(q);
#pragma unroll
              for (int b = 0; b < BATCH; ++b)
#pragma unroll
                for (int k = 0; k < PASSES; ++k) {
                  const float e = q + b < nq ? wt[(q + b) * R + r0 + k * RP].x : 0.0f;
                  if (e != 0.0f)
                    o[k] = make_float4(fmaf(e, v[b][k].x, o[k].x), fmaf(e, v[b][k].y, o[k].y),
                                       fmaf(e, v[b][k].z, o[k].z), fmaf(e, v[b][k].w, o[k].w));
                }
            }
            tf_any(false);
          }
          if (tid < rows && a.lse)
            a.lse[(int64_t)(tok0 + pg_token(a, tid)) * a.Hq + it.h * a.g + tid - pg_token(a, tid) * a.g] =
                tf_lse(m, sum);
#pragma unroll
          for (int k = 0; k < PASSES; ++k) {
            const int r = r0 + k * RP;
            if (r >= rows || col >= a.D) continue;
            const float sum_r = s_ref[r], inv = sum_r == 0.0f ? 0.0f : __fdividef(1.0f, sum_r);
            const int tok = pg_token(a, r);
            const int64_t dst = (int64_t)(tok0 + tok) * a.o_token + (int64_t)(it.h * a.g + r - tok * a.g) * a.o_head + col;
            const float4 y = make_float4(o[k].x * inv, o[k].y * inv, o[k].z * inv, o[k].w * inv);
            if (F32)
              *reinterpret_cast<float4*>(static_cast<float*>(a.o) + dst) = y;
            else
              *reinterpret_cast<uint2*>(static_cast<bf16*>(a.o) + dst) = make_uint2(ta_pack(y.x, y.y), ta_pack(y.z, y.w));
          }
        }
      }
      __syncwarp();
      if (lane == 0) {
        if (any) tc::mbar_arrive(&o_empty[ob]);
        tc::mbar_arrive(&i_empty[ni % TA_ITEMS]);
      }
    }
  } else if (role < 2) {
    // ------------------------------------------------------------ codes and scales
    TqLoader<C> ld{a, cache, ctl, s_copy, c_full, c_empty, s_kind, role};
    bool ok = true, pend = false;
    int pj = 0, pid = 0, ph = 0, plo = 0, phi = 0;  // the values still to be loaded
    for (uint32_t ni = 0; ok; ++ni) {
      ok = ctl.wait(&i_full[ni % TA_ITEMS], ni / TA_ITEMS & 1);
      if (!ok) break;
      TaItem it = s_item[ni % TA_ITEMS];
      if (it.n < 0) break;
      it.h /= cache.split;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&i_empty[ni % TA_ITEMS]);
      if (it.j1 <= it.j0 && pend) {  // (as the MMA issuer does)
        ok = ld.tile(true, pj, pid, ph, plo, phi);
        pend = false;
      }
      int id = ld.page_of(it, it.j0);
      for (int j = it.j0; j < it.j1 && ok; ++j) {
        const int id_next = ld.page_of(it, j + 1);
        ok = ld.tile(false, j, id, it.h, it.lo, it.hi);
        if (pend) ok = ok && ld.tile(true, pj, pid, ph, plo, phi);
        pend = true;
        pj = j;
        pid = id;
        ph = it.h;
        plo = it.lo;
        phi = it.hi;
        id = id_next;
      }
    }
    if (pend && ok) ok = ld.tile(true, pj, pid, ph, plo, phi);
    if (ok) ld.end();
    asm volatile("cp.async.wait_all;" ::: "memory");  // none is in flight when the CTA leaves
  } else if (role == 2) {
    // ------------------------------------------------------------ MMA issuer: one thread
    if (tc::elect_one()) {
      constexpr uint32_t id_s = tc::idesc_f16(128, NR, 0, 0);
      constexpr uint32_t id_o = tc::idesc_f16(128, NR, 1, 1);
      const uint64_t d_k = tc::smem_desc(tc::smem_u32(s_ring), 16, 1024, tc::LAYOUT_SW128);
      const uint64_t d_q = tc::smem_desc(tc::smem_u32(s_q), 16, 1024, tc::LAYOUT_SW128);
      // V^T: 64 columns a slab; D <= 64 has one, read twice for the 128 rows of the product
      const uint64_t d_v = tc::smem_desc(tc::smem_u32(s_ring), DP == 64 ? 0 : C::V_SLAB, 1024, tc::LAYOUT_SW128);
      const uint64_t d_p = tc::smem_desc(tc::smem_u32(s_p), 16, 8 * C::PROW, C::P_LAYOUT);
      uint32_t st = 0, par = 0;   // next ring unit, parity of its `full`
      uint32_t step = 0, nq = 0;  // S^T begun; items with keys
      bool ok = true, pend = false;
      struct {
        uint32_t step, item;
        bool first;
      } pv = {};
      // (a unit's arrival is waited for where it is used)
      auto take = [&](uint32_t (&at)[C::UPT], uint32_t (&arr)[C::UPT]) {
#pragma unroll
        for (int u = 0; u < C::UPT; ++u) {
          at[u] = st;
          arr[u] = par;
          if (++st == C::STAGES) {
            st = 0;
            par ^= 1;
          }
        }
      };
      auto product = [&] {  // O^T += V^T P^T of the step before
        uint32_t at[C::UPT], arr[C::UPT];
        take(at, arr);
        const uint32_t b = pv.step & 1, ob = pv.item & 1;
        ok = ok && ctl.wait1(&p_full[b], pv.step >> 1 & 1);
        if (pv.first) ok = ok && ctl.wait1(&o_empty[ob], (pv.item >> 1 & 1) ^ 1);
        if (!ok) return;
        tc::tc_fence_after();
#pragma unroll
        for (int k = 0; k < TA_BN / 16; ++k) {
          if (k * 16 % C::VROWS == 0) {
            ok = ctl.wait1(&full[at[k * 16 / C::VROWS]], arr[k * 16 / C::VROWS]);
            if (!ok) return;
            tc::tc_fence_after();
          }
#pragma unroll
          for (int hm = 0; hm < C::MH; ++hm)
            tc::mma_bf16(tmem + C::O_COL + (ob * C::MH + hm) * NR,
                         d_v + ((at[k * 16 / C::VROWS] * C::UB + 2 * hm * C::V_SLAB + k % (C::VROWS / 16) * 2048) >> 4),
                         d_p + ((b * C::PB + k * 16 * C::PROW) >> 4), id_o, k > 0 ? 1u : (uint32_t)!pv.first);
          if ((k + 1) * 16 % C::VROWS == 0) tc::mma_commit(&empty[at[k * 16 / C::VROWS]]);
        }
        tc::mma_commit(&pv_done[b]);
      };
      for (uint32_t ni = 0; ok; ++ni) {
        ok = ctl.wait1(&i_full[ni % TA_ITEMS], ni / TA_ITEMS & 1);
        if (!ok) break;
        const TaItem& it = s_item[ni % TA_ITEMS];
        if (it.n < 0) break;
        const int j0 = it.j0, j1 = it.j1;
        tc::mbar_arrive(&i_empty[ni % TA_ITEMS]);
        if (j1 <= j0 && pend) {  // no step to wait for: items without keys may follow one another
          product();
          pend = false;
        }
        const uint32_t qb = nq % C::QBUF;
        for (int j = j0; j < j1 && ok; ++j, ++step) {
          uint32_t at[C::UPT], arr[C::UPT];
          take(at, arr);
          if (j == j0) ok = ok && ctl.wait1(&q_full[qb], nq / C::QBUF & 1);
          if (!ok) break;
          tc::tc_fence_after();
          const uint32_t b = step & 1;
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            if (k % 8 == 0) {
              ok = ctl.wait1(&full[at[k / 8]], arr[k / 8]);
              if (!ok) break;
              tc::tc_fence_after();
            }
            tc::mma_bf16(tmem + C::S_COL + b * NR,
                         d_k + ((at[k / 8] * C::UB + k % 8 / 4 * C::K_SLAB + k % 4 * 32) >> 4),
                         d_q + ((qb * C::QB + k / 4 * C::QSLAB + k % 4 * 32) >> 4), id_s, k > 0);
            if (k % 8 == 7 || k == DP / 16 - 1) tc::mma_commit(&empty[at[k / 8]]);
          }
          if (!ok) break;
          tc::mma_commit(&s_full[b]);
          if (j == j1 - 1) tc::mma_commit(&q_empty[qb]);
          if (pend) product();
          pend = true;
          pv.step = step;
          pv.item = nq;
          pv.first = j == j0;
        }
        nq += j1 > j0;
      }
      if (pend && ok) product();
      tc::mma_commit(drain);  // arrives when all MMAs are done
    }
  } else if (role == 3) {
    // ------------------------------------------------------------ walk, and queries
    uint32_t n = 0;  // items with keys
    bool more = w.enter(a, start);
    bool ok = true;
    for (uint32_t ni = 0; ok; ++ni) {
      ok = ctl.wait(&i_empty[ni % TA_ITEMS], (ni / TA_ITEMS & 1) ^ 1);
      if (!ok) break;
      TaItem x;
      x.n = -1;
      if (more) {
        x.n = w.it.n;
        x.h = w.it.h;
        x.first = w.it.r.first;
        x.q = w.it.r.q;
        x.kv = w.it.r.kv;
        x.tok = w.it.m * a.tb;
        w.tiles(TA_BN, x.j0, x.j1);
        x.lo = w.it.lo;
        x.hi = w.it.hi;
        w.owners(x.c0, x.c1);
        x.slot = PgWalk::slot(w.cta, x.c0);
      }
      if (lane == 0) {
        s_item[ni % TA_ITEMS] = x;
        if (a.drop_cta != (int)blockIdx.x) tc::mbar_arrive(&i_full[ni % TA_ITEMS]);
      }
      __syncwarp();
      if (!more) break;
      if (x.j1 > x.j0) {
        // Queries: LPR lanes a row, 8 channels a lane.
        const uint32_t qb = n % C::QBUF;
        ok = ctl.wait(&q_empty[qb], (n / C::QBUF & 1) ^ 1);
        if (!ok) break;
        constexpr int LPR = DP / 8, RPP = 32 / LPR, PASSES = R / RPP, BATCH = PASSES < 4 ? PASSES : 4;
        const int c0 = lane % LPR * 8, rows = min(a.tb, x.q - x.tok) * a.g;
        uint8_t* dst = s_q + qb * C::QB + c0 / 64 * C::QSLAB;
#pragma unroll 1
        for (int p0 = 0; p0 < PASSES; p0 += BATCH) {
          float v[BATCH][8];
#pragma unroll
          for (int e = 0; e < BATCH; ++e) {
            const int r = (p0 + e) * RPP + lane / LPR, tok = pg_token(a, r);
            const int64_t at = (int64_t)(x.first + x.tok + tok) * a.q_token + (int64_t)(x.h * a.g + r - tok * a.g) * a.q_head + c0;
            const bool there = r < rows && c0 < a.D;
            if (F32) {
              const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
              const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
              *reinterpret_cast<float4*>(v[e]) = there ? q[0] : zero;
              *reinterpret_cast<float4*>(v[e] + 4) = there ? q[1] : zero;
            } else {
              const uint4 q = there ? *reinterpret_cast<const uint4*>(static_cast<const bf16*>(a.q) + at) : make_uint4(0u, 0u, 0u, 0u);
              const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                v[e][2 * k] = __uint_as_float(u[k] << 16);
                v[e][2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
              }
            }
          }
#pragma unroll
          for (int e = 0; e < BATCH; ++e) {
            const int r = (p0 + e) * RPP + lane / LPR;
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(v[e][k]) & 0x7fffffffu);
#pragma unroll
            for (int d = 1; d < LPR; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
            // the row's power of two, within what float32 holds; 1 where the row is not finite
            const int ex = top >= 0x7f800000u ? 14 : max((int)(top >> 23) - 127, -112);
            const float f = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float y0 = v[e][2 * k] * f, y1 = v[e][2 * k + 1] * f;
              hi[k] = tq_pack(y0, y1);
              lo[k] = F32 ? tq_rest(y0, y1, hi[k]) : 0u;
            }
            uint8_t* at = dst + r * 128 + ((c0 / 8 % 8 ^ (r & 7)) << 4);
            *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if (F32) *reinterpret_cast<uint4*>(at + R * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            if (lane % LPR == 0)
              s_factor[ni % TA_ITEMS][r] = fminf(a.scale_log2 * __uint_as_float((uint32_t)max(ex - 14 + 127, 1) << 23), FLT_MAX);
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&q_full[qb]);
        ++n;
      }
      if (lane == 0) tc::mbar_arrive(&r_full[ni % TA_ITEMS]);
      __syncwarp();
      more = w.next(a);
    }
  } else {
    // ------------------------------------------------------------ dequantising, a row a thread
    const int t = tid - TQ_SOFT - 128;
    uint32_t cst = 0, cpar = 0;  // next tile of codes, parity of its `full`
    uint32_t st = 0, par = 1;    // next unit, parity of its `empty`
    for (bool ok = true; ok;) {
      ok = ctl.wait_long(&c_full[cst], cpar);
      if (!ok) break;
      const int v = s_kind[cst];
      if (v < 0) break;
      const uint8_t* src = s_copy + cst * C::SB;
#pragma unroll 1
      for (int u = 0; u < C::UPT && ok; ++u) {
        // this thread's row, and its pieces of 32 channels
        constexpr int PPT = DP == 64 ? 1 : 2;
        const bool deep = C::UPT == 2 && v;
        const int r = deep ? 64 * u + (t & 63) : t & 127;
        const int p0 = deep ? (t >> 6) * 2 : (t >> 7) * PPT + (C::UPT == 2 ? 4 * u : 0);
        uint4 codes[PPT];
        uint32_t two[PPT];
#pragma unroll
        for (int e = 0; e < PPT; ++e) {
          codes[e] = *reinterpret_cast<const uint4*>(src + tq_code<C>(r, p0 + e));
          two[e] = *reinterpret_cast<const uint16_t*>(src + TA_BN * C::RB + r * C::SP + (p0 + e) * 2);
        }
        ok = ctl.wait(&empty[st], par);
        if (!ok) break;
        uint8_t* dst = s_ring + st * C::UB;
#pragma unroll
        for (int e = 0; e < PPT; ++e) {
          const int p = p0 + e - (!deep && C::UPT == 2 ? 4 * u : 0);  // within the unit
          const int row = deep ? r - 64 * u : r;
          uint8_t* line = dst + p / 2 * (deep ? C::V_SLAB : C::K_SLAB) + row * 128;
          const uint32_t s2 = q4_scales(two[e]);
          const uint32_t s_lo = __byte_perm(s2, s2, 0x1010), s_hi = __byte_perm(s2, s2, 0x3232);
          const uint32_t word[4] = {codes[e].x, codes[e].y, codes[e].z, codes[e].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t y[4];
            q4_pairs(word[c], y);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = q4_mul2(y[k], c < 2 ? s_lo : s_hi);
            *reinterpret_cast<uint4*>(line + ((((p & 1) * 4 + c) ^ (row & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(&full[st]);
          if (u == C::UPT - 1) tc::mbar_arrive(&c_empty[cst]);
        }
        if (++st == C::STAGES) {
          st = 0;
          par ^= 1;
        }
      }
      if (++cst == C::COPIES) {
        cst = 0;
        cpar ^= 1;
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (s_flag && tid < 32) tc::mbar_wait(drain, 0, a.wait_ns);  // a wait ran out: products in flight end
  __syncthreads();
  if (role == 2) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int DP, int R, bool F32>
cudaError_t run(PagedArgs& a, const Q4Cache& c, cudaStream_t s, int sms) {
  using C = Tq<DP, R, F32>;
  const void* f = reinterpret_cast<const void*>(k_paged_attn_q4<DP, R, F32>);
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = ta_prepare(f, C::smem, 0, ready);
  if (e != cudaSuccess) return e;
  a.tb = R / a.g;
  const PagedWs L = paged_ws(sms, R, DP);
  a.part_ml = L.ml;
  a.part_o = L.o;
  a.rows = R;
  pg_division(a, sms, 128, 192, 256);
  Q4Cache cache = c;
  void* args[] = {&a, &cache};
  return launch_pdl(f, dim3(sms), dim3(TQ_THREADS), C::smem, s, args, 1);
}

// Rows of a tile: 16, or 32 where a request has more in the mean.
int tile_rows(bool f32, int rows) { return f32 || rows <= 16 ? 16 : 32; }

template <int DP>
cudaError_t run_rows(PagedArgs& a, const Q4Cache& c, bool f32, int rows, cudaStream_t s, int sms) {
  if (f32) return run<DP, 16, true>(a, c, s, sms);
  return rows == 16 ? run<DP, 16, false>(a, c, s, sms) : run<DP, 32, false>(a, c, s, sms);
}

}  // namespace

cudaError_t launch_paged_attn_q4(PagedArgs a, const Q4Cache& cache, bool f32, int rows, cudaStream_t s) {
  const int sms = sm_count();
  if (sms < 1 || sms > PG_MAX_CTAS) return cudaErrorNotSupported;
  const int R = tile_rows(f32, rows);
  // More query heads on a key/value head than rows in a tile: the head counts as several, of as many of
  // its query heads each as fit and divide them.
  Q4Cache c = cache;
  int g = std::min(a.g, R);
  while (a.g % g) --g;
  c.split = a.g / g;
  if ((int64_t)a.Hkv * c.split > 0x7fffffff) return cudaErrorNotSupported;
  a.Hkv *= c.split;
  a.g = g;
  a.g_inv = (65536u + g - 1) / g;
  switch (ta_width(a.D)) {
    case 64: return run_rows<64>(a, c, f32, R, s, sms);
    case 128: return run_rows<128>(a, c, f32, R, s, sms);
    default: return run_rows<256>(a, c, f32, R, s, sms);
  }
}

size_t paged_attn_q4_ws_bytes(const paged_shape* s, int rows) {
  const int sms = sm_count();
  return paged_ws(sms > 0 ? sms : 256, tile_rows(s->io == RGLRU_F32, rows), ta_width(s->D)).total;
}

}  // namespace rglru

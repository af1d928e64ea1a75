// Attention over the paged cache for requests with few rows (bf16 I/O): decode steps and drafted
// tokens, at most NR = 16 or 32 rows (whole tokens x the query heads of one key/value head) a
// row tile.
//
// Such calls read every key and value once for a handful of rows and are bound by memory
// bandwidth: the products have to be kept off the critical path, not fast.  So they are turned
// around, keys along the 128 rows of the tensor core's tile:
//   S^T = K Q^T       128 keys x NR rows; K, Q from shared memory, S^T in TMEM, float32
//   P^T = 2^(c S^T - c m)     one key a thread, to shared memory as bf16
//   O^T += V^T P^T    D x NR; V read transposed by the tensor core, O^T in TMEM, float32
// which costs an eighth of the products of a 128-row tile and spreads the softmax over all
// threads.  The statistics of a row now lie across threads.  Its reference m is the same number in
// every thread; a tile's weights are taken at the m of the tile before it, and only if one of them
// would pass 2^8 (one reducing barrier tells) is the maximum found, by exchanges in halves between
// lanes and through shared memory, and O^T scaled.  The sums l stay apart, one a thread, until
// the item ends.  Rounding: weights to bf16 for the second product (8-bit significand, relative
// 2^-8 at most, as the output's own), l and all else in float32.
//
// The steps (key tiles) of all of a CTA's items form one stream: loads, products and softmax run
// on across the items' ends, with two buffers of S^T, P^T and O^T and several of Q, so that the
// ring of key and value tiles never runs dry.  Step i's S^T is computed before step i - 1's O^T,
// behind whose softmax it runs; an item without keys (rows before position 0, a request without
// any) has no step to put the last O^T behind, so there it is computed at once: the softmax warps
// keep an item's record until its O^T is done, and records are few.  Warps: 4 softmax, key/value loader, MMA issuer (one thread), one
// that clears rows of V that no row sees, and one that walks the items and loads queries.
//
// Measured (GB300): 64 requests of 4096 keys, 16 heads of 128: 314 us, 6.7 TB/s, the copy
// bandwidth.  256 requests of 64 to 8192 keys, 32 query heads on 8 (1.78 GB): 284 us, 6.3 TB/s;
// what is missing is the switch from item to item where they have one or two key tiles, and the
// start.  128 requests with a window of 2048, 10 query heads of 256 on one (227 MB): 48.4 us, 4.7
// TB/s: 14 key tiles a CTA, of which one is a rounding loss, 3 us of start and 4 us of joining
// parts.  One request of 1000 keys: 10.7 us, all latency: 4 us to the first product (lengths,
// division of work, table entry, copy: each a round trip), 3 to the parts, 3 to their join.
#include <float.h>

#include <algorithm>

#include "host_util.h"
#include "paged_tc.cuh"

namespace rglru {

namespace {

constexpr int TF_SOFT = 128;
constexpr int TF_THREADS = TF_SOFT + 128;
constexpr size_t TF_SMEM_MAX = 232448 - 4096;  // 227 KB less the static part

template <int DP, int NR, bool W>
struct Tf {
  static constexpr bool WIDE = W;                     // TaLay
  static constexpr int SLABS = DP / 64;
  static constexpr int UPT = DP == 256 ? 2 : 1;       // ring units of a key (or value) tile
  static constexpr uint32_t UB = DP == 64 ? TA_SLAB : 2 * TA_SLAB;
  static constexpr int VROWS = TA_BN / UPT;           // rows of V in a unit
  static constexpr int MH = DP == 256 ? 2 : 1;        // products of 128 columns of V
  static constexpr uint32_t QSLAB = NR * 128;         // 64 columns of the rows of Q
  static constexpr uint32_t QB = SLABS * QSLAB;
  static constexpr int QBUF = QB <= 8192 ? 4 : 2;
  static constexpr uint32_t PROW = NR * 2;            // a key's weights
  static constexpr uint32_t PB = TA_BN * PROW;
  static constexpr uint32_t P_LAYOUT = NR == 16 ? tc::LAYOUT_SW32 : tc::LAYOUT_SW64;
  static constexpr int FIT = (int)((TF_SMEM_MAX - 1024 - QBUF * QB - 2 * PB - 1024) / UB);
  static constexpr int STAGES = FIT < 16 ? FIT : 16;
  static constexpr uint32_t S_COL = 0, O_COL = 128;   // TMEM: S^T buffers, O^T buffers
  static constexpr size_t smem = 1024 + QBUF * QB + 2 * PB + (size_t)STAGES * UB + 1024;
};

// Or over the softmax threads.
__device__ __forceinline__ bool tf_any(bool x) {
  uint32_t y;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y)
      : "r"((uint32_t)x)
      : "memory");
  return y != 0;
}

// Combines NR values over a warp's lanes in halves: lane l is left with the result of value
// tf_column(l) in v[0].
template <int NR, class F>
__device__ __forceinline__ void tf_combine(float (&v)[NR], F f) {
  const int lane = threadIdx.x & 31;
  int n = NR;
#pragma unroll
  for (int bit = 16; bit; bit >>= 1) {
    if (n > 1) {
      n >>= 1;
#pragma unroll
      for (int k = 0; k < NR / 2; ++k) {
        if (k >= n) break;
        const float keep = lane & bit ? v[k + n] : v[k], give = lane & bit ? v[k] : v[k + n];
        v[k] = f(keep, __shfl_xor_sync(0xffffffffu, give, bit));
      }
    } else {
      v[0] = f(v[0], __shfl_xor_sync(0xffffffffu, v[0], bit));
    }
  }
}
template <int NR>
__device__ __forceinline__ int tf_column() {
  const int lane = threadIdx.x & 31;
  return NR == 32 ? lane : lane >> 1;
}

__device__ __forceinline__ float tf_lse(float ref, float sum) {
  return sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
}

template <int DP, int NR, bool W>
__global__ void __launch_bounds__(TF_THREADS, 1)
    k_paged_attn_few(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedArgs a) {
  using C = Tf<DP, NR, W>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* s_ring = smem;
  uint8_t* s_q = s_ring + (size_t)C::STAGES * C::UB;
  uint8_t* s_p = s_q + C::QBUF * C::QB;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_p + 2 * C::PB);
  uint64_t* empty = full + C::STAGES;
  uint64_t* q_full = empty + C::STAGES;  // [QBUF]
  uint64_t* q_empty = q_full + C::QBUF;  // [QBUF]
  uint64_t* s_full = q_empty + C::QBUF;  // [2] S^T of buffer b complete
  uint64_t* p_full = s_full + 2;         // [2] P^T of buffer b written (and O^T scaled)
  uint64_t* pv_done = p_full + 2;        // [2] the product with P^T of buffer b complete
  uint64_t* o_empty = pv_done + 2;       // [2] O^T buffer read
  uint64_t* i_full = o_empty + 2;        // [TA_ITEMS] item records
  uint64_t* i_empty = i_full + TA_ITEMS;
  uint64_t* v_come = i_empty + TA_ITEMS;  // [TA_CLEARS] a value tile to clear is on its way
  uint64_t* v_clean = v_come + TA_CLEARS; // [TA_CLEARS] it is cleared
  uint64_t* drain = v_clean + TA_CLEARS;
  __shared__ int64_t scratch[33];
  __shared__ TaItem s_item[TA_ITEMS];
  __shared__ uint32_t tmem_holder, s_flag, s_last;
  __shared__ uint32_t s_issued[2];       // loads issued: queries, ring units
  __shared__ TaClear s_clear[TA_CLEARS];
  __shared__ float s_red[4][NR];                        // a value a softmax warp and row
  __shared__ __align__(16) float s_ref[NR], s_scale[NR];  // the rows' references; factors of a change
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int role = warp - TF_SOFT / 32;  // < 0: softmax; 0: loader, 1: MMA, 2: clearing, 3: walk and queries
  const TaAbort ctl{&s_flag, reinterpret_cast<uint32_t*>(a.ws), a.wait_ns};

  // up to griddep_wait nothing touches global memory
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::QBUF; ++i) {
      tc::mbar_init(&q_full[i], 1);
      tc::mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s_full[i], 1);
      tc::mbar_init(&p_full[i], TF_SOFT / 32);
      tc::mbar_init(&pv_done[i], 1);
      tc::mbar_init(&o_empty[i], TF_SOFT / 32);
      s_issued[i] = 0u;
    }
    for (int i = 0; i < TA_ITEMS; ++i) {
      tc::mbar_init(&i_full[i], 1);
      tc::mbar_init(&i_empty[i], TF_SOFT / 32 + 2);
    }
    for (int i = 0; i < TA_CLEARS; ++i) {
      tc::mbar_init(&v_come[i], 1);
      tc::mbar_init(&v_clean[i], 1);
    }
    tc::mbar_init(drain, 1);
    s_flag = 0u;
    tc::fence_barrier_init();
    tc::prefetch_tmap(&tm_q);
    tc::prefetch_tmap(&tm_k);
    tc::prefetch_tmap(&tm_v);
  }
  if (role == 1) {
    tc::tmem_alloc(&tmem_holder, 512);
    tc::tmem_relinquish();
  }
  // rows of the query buffers that no copy fills stay zero
  for (uint32_t i = tid; i < C::QBUF * C::QB / 16; i += TF_THREADS)
    reinterpret_cast<uint4*>(s_q)[i] = make_uint4(0, 0, 0, 0);
  tc::griddep_wait();
  // By the warp that holds the TMEM, not before: a CTA of the next grid that takes TMEM (a decode
  // step's fits beside this one) keeps it until this grid has ended.
  if (role == 1) tc::griddep_launch_dependents();
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
    // What runs once an item is written as loops over rows kept in shared memory: a call with one
    // item a CTA pays for every instruction it fetches for the first time.
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    const float sc = a.scale_log2;
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
      float ref[NR], l[NR];  // the rows' references (scores in log2 units), this thread's sums
#pragma unroll
      for (int c = 0; c < NR; ++c) l[c] = ref[c] = 0.0f;
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
        const int k0 = j * TA_BN;
        if (k0 + TA_BN - 1 > p_first || (a.window && k0 < p_last - a.window + 1)) {
          int p = p_first, h = 0;  // row c's position
#pragma unroll
          for (int c = 0; c < NR; ++c) {
            if (k0 + tid > p || (a.window && k0 + tid <= p - a.window)) x[c] = -INFINITY;
            if (++h == a.g) {
              h = 0;
              ++p;
            }
          }
        }
        float worst = -INFINITY;
#pragma unroll
        for (int c = 0; c < NR; ++c) {
          x[c] *= sc;
          worst = fmaxf(worst, x[c] - ref[c]);
        }
        if (tf_any(!ok || j == j0 || worst > 8.0f)) {
          // new references: the rows' maxima so far
          float v[NR];
#pragma unroll
          for (int c = 0; c < NR; ++c) v[c] = x[c];
          tf_combine<NR>(v, [](float p, float q) { return fmaxf(p, q); });
          s_red[warp][tf_column<NR>()] = v[0];
          if (j > j0) ok = ctl.wait(&pv_done[b ^ 1], (step - 1) >> 1 & 1) && ok;
          if (tf_any(!ok)) {
            out = true;
            break;
          }
          if (tid < NR) {
            // the lowest finite number: no score is below it, and a key that is not seen (-inf) weighs 0
            const float m0 = j == j0 ? -FLT_MAX : s_ref[tid];
            const float top = fmaxf(fmaxf(fmaxf(s_red[0][tid], s_red[1][tid]), fmaxf(s_red[2][tid], s_red[3][tid])), m0);
            // Rows that the tile has to spare hold other requests' queries and see stale keys: with
            // an infinite reference they weigh nothing and never ask for a change, which would move
            // the item's own references (and so the rounding of its weights) too.
            const float m = tid < rows ? top : INFINITY;
            s_scale[tid] = m0 == m ? 1.0f : ta_ex2(m0 - m);
            s_ref[tid] = m;
          }
          tf_any(false);
#pragma unroll
          for (int c = 0; c < NR; c += 4)
            *reinterpret_cast<float4*>(ref + c) = *reinterpret_cast<const float4*>(s_ref + c);
          if (j > j0) {
            tc::tc_fence_after();
#pragma unroll
            for (int c = 0; c < NR; ++c) l[c] *= s_scale[c];
#pragma unroll 1
            for (int c = 0; c < C::MH * NR; c += 4) {
              float o[4];
              tc::tmem_ld4(t_o + c, o);
              tc::tmem_ld_wait();
              tc::reg_fence(o);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[e] *= s_scale[c % NR + e];
              tc::tmem_st4(t_o + c, o);
            }
            tc::tmem_st_wait();
          }
        }
        uint32_t pk[NR / 2];
#pragma unroll
        for (int c = 0; c < NR; c += 2) {
          const float p0 = ta_ex2(x[c] - ref[c]), p1 = ta_ex2(x[c + 1] - ref[c + 1]);
          l[c] += p0;
          l[c + 1] += p1;
          pk[c / 2] = ta_pack(p0, p1);
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
      tf_combine<NR>(l, [](float p, float q) { return p + q; });
      s_red[warp][tf_column<NR>()] = l[0];
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
          reinterpret_cast<float2*>(a.ws + a.part_ml)[(size_t)it.slot * NR + tid] = make_float2(s_ref[tid], sum);
        else if (a.lse)
          a.lse[(int64_t)(tok0 + pg_token(a, tid)) * a.Hq + it.h * a.g + tid - pg_token(a, tid) * a.g] =
              tf_lse(s_ref[tid], sum);
      }
      {
        bf16* dst = static_cast<bf16*>(a.o) + tok0 * a.o_token + (int64_t)it.h * a.g * a.o_head + tid;
        float* po = reinterpret_cast<float*>(a.ws + a.part_o) + (size_t)it.slot * NR * DP + tid;
        int h = 0;
#pragma unroll 1
        for (int c = 0; c < rows; c += 4) {
          __syncwarp();  // (TMEM is read by whole warps)
          float o[C::MH][4];
#pragma unroll
          for (int hm = 0; hm < C::MH; ++hm)
            if (any) tc::tmem_ld4(t_o + hm * NR + c, o[hm]);
          if (any) tc::tmem_ld_wait();
#pragma unroll
          for (int hm = 0; hm < C::MH; ++hm) tc::reg_fence(o[hm]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (c + e >= rows) break;
            if (whole) {
              const float sum = row_sum(c + e), inv = __fdividef(1.0f, sum);
#pragma unroll
              for (int hm = 0; hm < C::MH; ++hm)
                if (hm * 128 + tid < a.D) dst[hm * 128] = __float2bfloat16_rn(sum == 0.0f ? 0.0f : o[hm][e] * inv);
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
          constexpr int PARTS = 2 * C::PB / (NR * 8), RP = 512 / DP, PASSES = NR / RP;
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
                const float* pq = po + (size_t)PgWalk::slot(q0 + min(qb + b, nq - 1), it.c0) * NR * DP;
#pragma unroll
                for (int k = 0; k < PASSES; ++k) v[b][k] = __ldcg(reinterpret_cast<const float4*>(pq + k * RP * DP));
              }
            };
            load(0);
#pragma unroll 1
            for (int i = tid; i < nq * NR; i += TF_SOFT)
              wt[i] = i % NR < rows ? __ldcg(reinterpret_cast<const float2*>(a.ws + a.part_ml) +
                                             (size_t)PgWalk::slot(q0 + i / NR, it.c0) * NR + i % NR)
                                    : make_float2(0.0f, 0.0f);
            tf_any(false);
            if (tid < NR) {
              const float m0 = m;
#pragma unroll 4
              for (int q = 0; q < nq; ++q) m = fmaxf(m, wt[q * NR + tid].y != 0.0f ? wt[q * NR + tid].x : -INFINITY);
              const float f = m0 == m ? 1.0f : ta_ex2(m0 - m);
              sum *= f;
#pragma unroll 4
              for (int q = 0; q < nq; ++q) {
                const float2 x = wt[q * NR + tid];  // a part that saw nothing did not write its sums
                const float e = x.y != 0.0f ? ta_ex2(x.x - m) : 0.0f;
                sum += x.y * e;
                wt[q * NR + tid].x = e;
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
                  const float e = q + b < nq ? wt[(q + b) * NR + r0 + k * RP].x : 0.0f;
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
            const float l = s_ref[r], inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
            const int tok = pg_token(a, r);
            bf16* dst = static_cast<bf16*>(a.o) + (int64_t)(tok0 + tok) * a.o_token +
                        (int64_t)(it.h * a.g + r - tok * a.g) * a.o_head + col;
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(ta_pack(o[k].x * inv, o[k].y * inv), ta_pack(o[k].z * inv, o[k].w * inv));
          }
        }
      }
      __syncwarp();
      if (lane == 0) {
        if (any) tc::mbar_arrive(&o_empty[ob]);
        tc::mbar_arrive(&i_empty[ni % TA_ITEMS]);
      }
    }
  } else if (role == 0) {
    // ------------------------------------------------------------ key / value loader
    TaLoader<C> ld{a, ctl, s_ring, full, empty, s_clear, v_come};
    bool ok = true, pend = false;
    int pj = 0, pid = 0, ph = 0, plo = 0, phi = 0;  // the values still to be loaded
    for (uint32_t ni = 0; ok; ++ni) {
      ok = ctl.wait(&i_full[ni % TA_ITEMS], ni / TA_ITEMS & 1);
      if (!ok) break;
      const TaItem it = s_item[ni % TA_ITEMS];
      if (it.n < 0) break;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&i_empty[ni % TA_ITEMS]);
      if (it.j1 <= it.j0 && pend) {  // (as the MMA issuer does)
        ok = ld.values(&tm_v, pj, pid, ph, plo, phi);
        pend = false;
      }
      int id = ld.page_of(it, it.j0);
      for (int j = it.j0; j < it.j1 && ok; ++j) {
        const int id_next = ld.page_of(it, j + 1);
        ok = ld.keys(&tm_k, j, id, it.h);
        if (pend) ok = ok && ld.values(&tm_v, pj, pid, ph, plo, phi);
        pend = true;
        pj = j;
        pid = id;
        ph = it.h;
        plo = it.lo;
        phi = it.hi;
        id = id_next;
      }
    }
    if (pend && ok) ld.values(&tm_v, pj, pid, ph, plo, phi);
    ld.end();
    if (lane == 0) s_issued[1] = ld.issued;
  } else if (role == 1) {
    // ------------------------------------------------------------ MMA issuer: one thread
    if (tc::elect_one()) {
      constexpr uint32_t id_s = tc::idesc_bf16(128, NR, 0, 0);
      constexpr uint32_t id_o = tc::idesc_bf16(128, NR, 1, 1);
      const TaLay<C> lay(a);
      const uint64_t d_k = tc::smem_desc(tc::smem_u32(s_ring), 16, TaLay<C>::K_GROUP, tc::LAYOUT_SW128);
      const uint64_t d_q = tc::smem_desc(tc::smem_u32(s_q), 16, 1024, tc::LAYOUT_SW128);
      // V^T: 64 columns a slab; D <= 64 has one, read twice for the 128 rows of the product
      const uint64_t d_v = tc::smem_desc(tc::smem_u32(s_ring), DP == 64 ? 0 : lay.v_slab(), lay.v_group(), tc::LAYOUT_SW128);
      const uint32_t v_slab = lay.v_slab() >> 4;
      const uint64_t d_p = tc::smem_desc(tc::smem_u32(s_p), 16, 8 * C::PROW, C::P_LAYOUT);
      uint32_t st = 0, par = 0;          // next ring unit, parity of its `full`
      uint32_t step = 0, nq = 0, nc = 0; // S^T begun; items with keys; value tiles cleared
      bool ok = true, pend = false;
      struct {
        uint32_t step, item;
        bool first, cut;
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
        if (pv.cut) {
          ok = ok && ctl.wait1(&v_clean[nc % TA_CLEARS], nc / TA_CLEARS & 1);
          ++nc;
        }
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
                         d_v + (at[k * 16 / C::VROWS] * (C::UB >> 4) +
                                2 * hm * v_slab + (k % (C::VROWS / 16) * TaLay<C>::V_16 >> 4)),
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
        const int j0 = it.j0, j1 = it.j1, lo = it.lo, hi = it.hi;
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
                         d_k + (at[k / 8] * (C::UB >> 4) + ((k % 8 / 4 * TaLay<C>::K_SLAB + k % 4 * 32) >> 4)),
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
          pv.cut = ta_cut(j, lo, hi);
        }
        nq += j1 > j0;
      }
      if (pend && ok) product();
      tc::mma_commit(drain);  // arrives when all MMAs are done
    }
  } else if (role == 2) {
    // ------------------------------------------------------------ rows of V that no row sees
    ta_clear_rows<C>(a, ctl, s_clear, v_come, v_clean, full, s_ring);
  } else {
    // ------------------------------------------------------------ walk, and queries
    uint32_t n = 0;  // query loads
    bool more = w.enter(a, start);
    const uint32_t bytes = C::SLABS * a.tb * a.g * 128;
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
        const uint32_t qb = n % C::QBUF;
        ok = ctl.wait(&q_empty[qb], (n / C::QBUF & 1) ^ 1);
        if (ok) {
          if (lane == 0) {
            tc::mbar_expect_tx(&q_full[qb], bytes);
            for (int s = 0; s < C::SLABS; ++s)
              tc::tma_load_3d(s_q + qb * C::QB + s * C::QSLAB, &tm_q, &q_full[qb], s * 64, x.h * a.g, x.first + x.tok);
          }
          ++n;
        }
        __syncwarp();
      }
      more = w.next(a);
    }
    if (lane == 0) s_issued[0] = n;
  }
  tc::tc_fence_before();
  __syncthreads();
  if (s_flag && tid < 32) {
    // a wait ran out: copies and products in flight end (or run out too) before the CTA leaves
    for (uint32_t i = lane; i < min(s_issued[1], (uint32_t)C::STAGES); i += 32) {
      const uint32_t n = s_issued[1] - 1 - i;
      tc::mbar_wait(&full[n % C::STAGES], n / C::STAGES & 1, a.wait_ns);
    }
    for (uint32_t i = lane; i < min(s_issued[0], (uint32_t)C::QBUF); i += 32) {
      const uint32_t n = s_issued[0] - 1 - i;
      tc::mbar_wait(&q_full[n % C::QBUF], n / C::QBUF & 1, a.wait_ns);
    }
    tc::mbar_wait(drain, 0, a.wait_ns);
  }
  __syncthreads();
  if (role == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int DP, int NR, bool W>
cudaError_t run(PagedArgs& a, cudaStream_t s, int sms) {
  using C = Tf<DP, NR, W>;
  a.tb = NR / a.g;
  CUtensorMap mq, mk, mv;
  cudaError_t e = ta_maps<C>(a, a.tb, &mq, &mk, &mv);
  if (e != cudaSuccess) return e;
  const void* f = reinterpret_cast<const void*>(k_paged_attn_few<DP, NR, W>);
  static std::atomic<uint64_t> ready{0};
  e = ta_prepare(f, C::smem, 0, ready);
  if (e != cudaSuccess) return e;
  const PagedWs L = paged_ws(sms, NR, DP);
  a.part_ml = L.ml;
  a.part_o = L.o;
  a.rows = NR;
  // an item's switch costs about a key tile's time, a part's hand-over and join more
  pg_division(a, sms, 128, 192, 256);
  void* args[] = {&mq, &mk, &mv, &a};
  return launch_pdl(f, dim3(sms), dim3(TF_THREADS), C::smem, s, args, 1);
}

template <int DP, bool W>
cudaError_t run_rows(PagedArgs& a, int rows, cudaStream_t s, int sms) {
  return rows <= 16 ? run<DP, 16, W>(a, s, sms) : run<DP, 32, W>(a, s, sms);
}

}  // namespace

cudaError_t launch_paged_attn_few(PagedArgs a, int rows, cudaStream_t s) {
  const int sms = sm_count();
  if (sms < 1 || sms > PG_MAX_CTAS) return cudaErrorNotSupported;
  switch (ta_width(a.D)) {
    case 64: return run_rows<64, false>(a, rows, s, sms);
    case 128: return ta_wide(a) ? run_rows<128, true>(a, rows, s, sms) : run_rows<128, false>(a, rows, s, sms);
    default: return ta_wide(a) ? run_rows<256, true>(a, rows, s, sms) : run_rows<256, false>(a, rows, s, sms);
  }
}

size_t paged_attn_few_ws_bytes(const paged_shape* s, int rows) {
  const int sms = sm_count();
  return paged_ws(sms > 0 ? sms : 256, rows <= 16 ? 16 : 32, ta_width(s->D)).total;
}

}  // namespace rglru

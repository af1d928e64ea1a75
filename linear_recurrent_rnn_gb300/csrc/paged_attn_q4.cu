// Attention over the paged cache held in 4 bits (include/paged_q4.h), R rows a row tile (whole tokens x
// the query heads of one key/value head).
//
// As in the kernel for few rows over a bf16 cache (paged_attn_few.cu), keys lie along the 128 rows of the
// tensor core's tile:
//   S^T = K Q^T       128 keys x the rows; S^T in TMEM, float32
//   P^T = 2^(c S^T - c m)     one key a thread, to shared memory as f16
//   O^T += V^T P^T    D x the rows; V read transposed by the tensor core, O^T in TMEM, float32
// What is new is the way of keys and values to the tensor core.  Codes and scales come to shared memory by
// cp.async, a quarter of bf16's bytes; the warpgroup that copied them writes the numbers that they stand
// for as f16, keys to TMEM (the products' A operand, a row a lane), values to shared memory.  A code times its
// scale has 6 significant bits at most, so f16 holds it exactly (2^-10 to 2688).  Rows that no row of the
// item sees, and pages that are not there, are copied as zeros (cp.async with fewer source bytes), so
// nothing stale reaches a product.
//
// Queries are f16 too, as the tensor core takes two operands of one type: each row is multiplied by
// the power of two that brings its largest element to [2^14, 2^15), and its scores by the inverse.
// bf16's 8 significant bits fit f16's 11.  float32 queries and weights are split into two f16 numbers
// (22 bits), rows of their own in the products, added in float32.  Weights are held times 2^11, so
// that f16's range, 2^-25 to 2^15, is used from 2^4 times the first maximum down to 2^-36 of it; the reference m
// is moved when a weight would pass 2^15.
//
// The tensor core cuts what it adds to a sum where it would have to round: outputs of values of one sign come out 2.8e-9
// too small for each key of a sum, 1.8e-4 for 65536 (bf16 rounds by up to 2e-3).  So float32's products are summed a step of 256
// keys at a time; the softmax's threads add the steps up, a step behind, in registers, where the references' changes are
// applied too (256 requests decoding, 32 heads on 8 of 128, 258 us without, 267 with it; 128 requests, 16 heads on one
// of 128, 34.6 and 37.7).  Sums of 512 keys and more, and tiles of 128 keys a step with all in registers, were slower.
//
// Warpgroups: softmax; control (a thread that issues S's products, one that issues O's, a warp that walks the
// items, one that brings queries); 2 that bring keys and 2 that bring values, a unit each in turn.
// Bound by the warps that dequantise: 1390 cycles a key tile of one head of 128, in which a scheduler issues some 780
// instructions (56 % of its slots); each of its six warps issues in order, ten cycles an instruction, and more warps
// have no registers.  That is 3.8 TB/s of codes on long sequences, where bf16's kernel reaches 6.1 TB/s of 3.6 times
// the bytes.
// Measured (GB300): 256 requests of 64 to 8192 keys, 32 heads on 8 of 128, 195 us (the kernel over bf16
// caches: 287); 64 of 4096 keys, 16 heads on 16, 164 us (314); 152 of 16384 keys on one head, 94 us.
// Other ways that were measured: keys from shared memory (a product of 128 x 16 x 16 takes the tensor core 39
// cycles then, from TMEM 9); TMA and bulk copies of the codes (84 cycles a copy and SM, and a page's codes
// are 1 KB); warps that only copy, with a barrier between them and those that dequantise (420 us).
#include <float.h>

#include <algorithm>

#include "host_util.h"
#include "paged_q4.cuh"

namespace rglru {

namespace {

// Warpgroups: softmax; scores' and outputs' MMA, walk, queries; TQ_KEYS that bring keys, a unit each in
// turn, TQ_VALUES that bring values.
constexpr int TQ_KEYS = 2, TQ_VALUES = 2;
constexpr int TQ_THREADS = 128 * (2 + TQ_KEYS + TQ_VALUES);
constexpr size_t TQ_SMEM_MAX = 232448 - 4096;  // 227 KB less the static part
constexpr float TQ_SHIFT = 11.0f;  // weights are held times 2^TQ_SHIFT
constexpr float TQ_TOP = 15.0f;    // and stay below 2^TQ_TOP
constexpr uint32_t TQ_JOIN = 4096; // bytes of the weights of parts that are joined

template <int DP, int R_, bool F32_>
struct Tq {
  static constexpr int R = R_;
  static constexpr bool F32 = F32_;
  static constexpr int COLS = F32 ? 2 * R : R;        // columns in use of the products
  static constexpr int NR = COLS < 16 ? 16 : COLS;    // columns
  // Units: 128 keys (or values) of up to 128 columns; what is copied, dequantised and multiplied at once.
  static constexpr int UNITS = DP == 256 ? 2 : 1;     // of a tile
  static constexpr int COL = DP / UNITS;              // columns of one
  static constexpr int KT = R == 32 ? 1 : F32 || R == 16 || DP == 256 ? 2 : 4;  // key tiles of a step
  static constexpr int SCORES = (KT * COLS + 15) / 16 * 16;  // of a thread and step as they are read from TMEM, 16 at once
  static constexpr uint32_t RB = COL / 2, SP = COL / 16;  // bytes of a row's codes, of its scales
  static constexpr uint32_t SB = 1024 * ((TA_BN * (RB + SP) + 1023) / 1024);  // a unit's
  static constexpr uint32_t VB = TA_BN * COL * 2;     // of a unit of values as f16
  static constexpr uint32_t QSLAB = NR * 128;         // 64 columns of the rows of Q
  static constexpr uint32_t QB = DP / 64 * QSLAB;
  static constexpr int QBUF = 2;
  static constexpr uint32_t PROW = NR * 2;            // a key's weights
  static constexpr uint32_t PT = TA_BN * PROW;        // a tile's
  static constexpr uint32_t PB = KT * PT;             // a step's
  static constexpr uint32_t P_LAYOUT = NR == 16 ? tc::LAYOUT_SW32 : tc::LAYOUT_SW64;
  static constexpr int VBUF = DP == 256 && F32 && NR == 32 ? 2 : 3;  // units of V
  static constexpr int FIT = (int)((TQ_SMEM_MAX - 1024 - QBUF * QB - 2 * PB - VBUF * VB - TQ_JOIN - 1024) / SB);
  // units of codes on their way: of each warpgroup that brings them
  static constexpr int DEPTH = FIT / (TQ_KEYS + TQ_VALUES) < 6 ? FIT / (TQ_KEYS + TQ_VALUES) : 6;
  // TMEM: S^T buffers, O^T buffers, units of keys as f16 (a row a lane).  A step's tiles lie COLS columns
  // apart in S^T: a product's columns beyond those in use are overwritten by the next tile's.
  static constexpr uint32_t S_WIDTH = 64;  // of a buffer
  static constexpr uint32_t S_COL = 0, O_COL = 128, K_COL = 256;
  static constexpr int KBUF = 4;
  static constexpr uint32_t V_SLAB = TA_SLAB;         // 64 columns, 128-byte swizzle
  static constexpr size_t smem = 1024 + VBUF * VB + (size_t)(TQ_KEYS + TQ_VALUES) * DEPTH * SB + QBUF * QB + 2 * PB + TQ_JOIN + 1024;
  static_assert(SCORES % 16 == 0 && SCORES >= KT * COLS && SCORES <= (int)S_WIDTH, "reads of S");
  static_assert(KT * COLS + NR - COLS <= S_WIDTH && 2 * UNITS * NR <= 128 && KBUF * COL / 2 <= 256, "TMEM");
  static_assert(DEPTH >= 2, "shared memory");
  static_assert(KBUF >= TQ_KEYS && VBUF >= TQ_VALUES, "a stage at least for each that fills them in turn");
  static_assert(VBUF * VB + (size_t)(TQ_KEYS + TQ_VALUES) * DEPTH * SB >= (PG_MAX_SEQS + 1) * 8, "the scan of the requests");
};

template <int DP, int R, bool F32>
__global__ void __launch_bounds__(TQ_THREADS, 1)
    k_paged_attn_q4(const __grid_constant__ PagedArgs a, const __grid_constant__ Q4Cache cache) {
  using C = Tq<DP, R, F32>;
  constexpr int NR = C::NR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* s_v = smem;
  uint8_t* s_copy = s_v + (size_t)C::VBUF * C::VB;
  uint8_t* s_q = s_copy + (size_t)(TQ_KEYS + TQ_VALUES) * C::DEPTH * C::SB;
  uint8_t* s_p = s_q + C::QBUF * C::QB;
  float2* s_join = reinterpret_cast<float2*>(s_p + 2 * C::PB);
  uint64_t* v_full = reinterpret_cast<uint64_t*>(s_p + 2 * C::PB + TQ_JOIN);
  uint64_t* v_empty = v_full + C::VBUF;    // [VBUF] units of V
  uint64_t* k_full = v_empty + C::VBUF;    // [KBUF] units of K in TMEM
  uint64_t* k_empty = k_full + C::KBUF;
  uint64_t* q_full = k_empty + C::KBUF;    // [QBUF]
  uint64_t* q_empty = q_full + C::QBUF;    // [QBUF]
  uint64_t* s_full = q_empty + C::QBUF;    // [2] S^T of buffer b complete
  uint64_t* s_empty = s_full + 2;          // [2] and read
  uint64_t* p_full = s_empty + 2;          // [2] P^T of buffer b written (and O^T scaled)
  uint64_t* pv_done = p_full + 2;          // [2] the products with P^T of buffer b complete
  uint64_t* o_empty = pv_done + 2;         // [2] O^T buffer read
  uint64_t* i_full = o_empty + 2;          // [TA_ITEMS] item records
  uint64_t* i_empty = i_full + TA_ITEMS;
  uint64_t* r_full = i_empty + TA_ITEMS;   // [TA_ITEMS] the factors of an item's rows
  uint64_t* drain = r_full + TA_ITEMS;
  __shared__ int64_t scratch[33];
  __shared__ TaItem s_item[TA_ITEMS];
  __shared__ uint32_t tmem_holder, s_flag, s_last;
  __shared__ __align__(16) float s_red[4][R];                // a value a softmax warp and row
  __shared__ __align__(16) float s_ref[R], s_scale[R];       // the rows' references; factors of a change
  __shared__ __align__(16) float s_factor[TA_ITEMS][R];      // of the rows' scores
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = warp >> 2, role = warp - 4;  // warpgroup; of the second: 0, 2: MMA, 1: walk, 3: queries
  const TqAbort ctl{&s_flag, reinterpret_cast<uint32_t*>(a.ws), (uint32_t)(a.wait_ns >> 10) + 1};

  // up to griddep_wait nothing touches global memory
  if (tid == 0) {
    for (int i = 0; i < C::VBUF; ++i) {
      tc::mbar_init(&v_full[i], 4);
      tc::mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < C::KBUF; ++i) {
      tc::mbar_init(&k_full[i], 4);
      tc::mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::QBUF; ++i) {
      tc::mbar_init(&q_full[i], 1);
      tc::mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s_full[i], 1);
      tc::mbar_init(&s_empty[i], 4);
      tc::mbar_init(&p_full[i], 4);
      tc::mbar_init(&pv_done[i], 1);
      tc::mbar_init(&o_empty[i], 4);
    }
    for (int i = 0; i < TA_ITEMS; ++i) {
      tc::mbar_init(&i_full[i], 1);
      tc::mbar_init(&i_empty[i], 4 * (1 + TQ_KEYS + TQ_VALUES) + 3);
      tc::mbar_init(&r_full[i], 1);
    }
    tc::mbar_init(drain, 2);
    s_flag = 0u;
    tc::fence_barrier_init();
  }
  if (role == 0) {
    tc::tmem_alloc(&tmem_holder, 512);
    tc::tmem_relinquish();
  }
  // columns that no row uses stay zero, of queries and of weights
  for (uint32_t i = tid; i < (C::QBUF * C::QB + 2 * C::PB) / 16; i += TQ_THREADS)
    reinterpret_cast<uint4*>(s_q)[i] = make_uint4(0u, 0u, 0u, 0u);
  tc::griddep_wait();
  // By the warp that holds the TMEM, not before: a CTA of the next grid that takes TMEM keeps it until
  // this grid has ended.
  if (role == 0) tc::griddep_launch_dependents();
  PgWalk w;
  PgWalk::Found start;
  if (a.N <= PG_WARP_SEQS) {
    if (role == 1) start = w.find_warp(a);
  } else {
    int64_t* prefix = reinterpret_cast<int64_t*>(s_v);  // before the rings are in use
    pg_scan(a, prefix, scratch);
    if (role == 1) start = w.find(a, prefix);
  }
  tc::fence_proxy_async_smem();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_holder;

  // Registers: 768 threads x 80 at launch = 128 x (144 + 80 + 4 x 64).
  if (group == 0) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    // ------------------------------------------------------------ softmax, a key of each tile a thread
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    uint32_t step = 0, no = 0;  // steps, items with an O^T so far
    bool ok = true;
    for (uint32_t ni = 0;; ++ni) {
      ok = ctl.wait(&i_full[ni % TA_ITEMS], ni / TA_ITEMS & 1);
      if (tf_any(!ok)) break;
      const TaItem& it = s_item[ni % TA_ITEMS];
      if (it.n < 0) break;
      const int j0 = it.j0, j1 = it.j1;
      const int rows = min(a.tb, it.q - it.tok) * a.g;
      const int p_first = it.kv - it.q + it.tok, p_last = p_first + min(a.tb, it.q - it.tok) - 1;
      uint32_t ob = no & 1, t_o = lanes + C::O_COL + ob * (C::UNITS * NR);
      // the rows' factors, references (scores in log2 units), this thread's sums; in pairs of rows.  Of 32
      // rows, and of 16 in float32, only the sums are kept in registers.
      constexpr bool KEEP = R <= 16 && !(F32 && R == 16);
      float2 factors[KEEP ? R / 2 : 1], refs[KEEP ? R / 2 : 1], l[R / 2];
      float2 acc[F32 ? C::UNITS : 1][R / 2];  // float32: O^T, but for the products that are still to be added
      ok = ctl.wait(&r_full[ni % TA_ITEMS], ni / TA_ITEMS & 1);
      const float2* s_f2 = reinterpret_cast<const float2*>(s_factor[ni % TA_ITEMS]);
      if (!KEEP) {
        if (tid < R) s_ref[tid] = 0.0f;
        tf_any(false);
      }
#pragma unroll
      for (int c = 0; c < R / 2; ++c) {
        if (KEEP) factors[c] = s_f2[c];
        if (KEEP) refs[c] = make_float2(0.0f, 0.0f);
        l[c] = make_float2(0.0f, 0.0f);
        if (F32)
#pragma unroll
          for (int hm = 0; hm < C::UNITS; ++hm) acc[hm][c] = make_float2(0.0f, 0.0f);
      }
      auto factor = [&](int c) { return KEEP ? factors[KEEP ? c : 0] : s_f2[c]; };
      auto ref = [&](int c) { return KEEP ? refs[KEEP ? c : 0] : reinterpret_cast<const float2*>(s_ref)[c]; };
      bool out = false;
      // (float32: once more behind the last step, for its product)
      for (int j = j0; F32 || j < j1; j += C::KT, ++step) {
        const uint32_t b = step & 1;
        constexpr bool ALL = R <= 8;  // more rows would cost the registers that the steps need
        float2 scale[ALL ? R / 2 : 1];
        auto factor_of = [&](int c) { return ALL ? scale[ALL ? c : 0] : reinterpret_cast<const float2*>(s_scale)[c]; };
        bool grown = false;
        if (!F32 || j < j1) {
          ok = ctl.wait(&s_full[b], step >> 1 & 1) && ok;
          tc::tc_fence_after();
          float x[C::SCORES];
#pragma unroll
          for (int c = 0; c < C::SCORES; c += 16)
            tc::tmem_ld16(lanes + C::S_COL + b * C::S_WIDTH + c, *reinterpret_cast<float(*)[16]>(x + c));
          tc::tmem_ld_wait();
          tc::reg_fence(x);
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&s_empty[b]);
          // scores, and those times their factors less the references (rounded once)
          float2 z[C::KT][R / 2], y[C::KT][R / 2];
#pragma unroll
          for (int t = 0; t < C::KT; ++t)
#pragma unroll
            for (int c = 0; c < R / 2; ++c) {
              z[t][c] = make_float2(x[t * C::COLS + 2 * c], x[t * C::COLS + 2 * c + 1]);
              if (F32)
                z[t][c] = ta_add2(z[t][c], make_float2(x[t * C::COLS + (C::COLS - R) + 2 * c], x[t * C::COLS + (C::COLS - R) + 2 * c + 1]));
              y[t][c] = ta_fma2(z[t][c], factor(c), make_float2(-ref(c).x, -ref(c).y));
            }
          // positions that rows do not see, and tiles past the part's last (their scores are stale)
          const int k0 = j * TA_BN, k1 = j1 * TA_BN;
          if (k0 + C::KT * TA_BN > min(p_first + 1, k1) || (a.window && k0 < p_last - a.window + 1)) {
            int p = p_first, h = 0;  // the row's position
#pragma unroll
            for (int c = 0; c < R; ++c) {
              const int lo = a.window ? p - k0 - tid - a.window : -1, hi = min(p, k1 - 1) - k0 - tid;  // lo < 128 t <= hi
#pragma unroll
              for (int t = 0; t < C::KT; ++t) {
                float& w = c & 1 ? y[t][c / 2].y : y[t][c / 2].x;
                if (t * TA_BN > hi || t * TA_BN <= lo) w = -INFINITY;
              }
              if (++h == a.g) {
                h = 0;
                ++p;
              }
            }
          }
          float worst = -INFINITY;
#pragma unroll
          for (int t = 0; t < C::KT; ++t)
#pragma unroll
            for (int c = 0; c < R / 2; ++c) worst = ta_max3(worst, y[t][c].x, y[t][c].y);
          if (j == j0 || tf_any(!ok || worst > TQ_TOP)) {
            // new references: the rows' maxima so far, less the shift
            // (from the scores themselves: y has lost them where the reference was far off)
            auto score = [&](float w, float p, float f, float m) { return w == -INFINITY ? w : fmaf(p, f, -m); };
            float v[R];
#pragma unroll
            for (int c = 0; c < R / 2; ++c) {
              v[2 * c] = v[2 * c + 1] = -INFINITY;
#pragma unroll
              for (int t = 0; t < C::KT; ++t) {
                v[2 * c] = fmaxf(v[2 * c], score(y[t][c].x, z[t][c].x, factor(c).x, 0.0f));
                v[2 * c + 1] = fmaxf(v[2 * c + 1], score(y[t][c].y, z[t][c].y, factor(c).y, 0.0f));
              }
            }
            tf_combine<R>(v, [](float p, float q) { return fmaxf(p, q); });
            s_red[warp][tf_column<R>()] = v[0];
            if (j > j0) ok = ctl.wait(&pv_done[b ^ 1], (step - 1) >> 1 & 1) && ok;
            if (tf_any(!ok)) {
              out = true;
              break;
            }
            // the lowest finite number: no score is below it, and a key that is not seen (-inf) weighs 0.
            // Rows that the tile has to spare: with an infinite reference they weigh nothing and never ask
            // for a change.
            auto moved = [&](int c, float seen, float m0) { return c < rows ? fmaxf(seen - TQ_SHIFT, m0) : INFINITY; };
            if constexpr (ALL) {  // each thread all rows: one barrier
#pragma unroll
              for (int c = 0; c < R; c += 4) {
                float4 t4 = *reinterpret_cast<const float4*>(&s_red[0][c]);
#pragma unroll
                for (int w = 1; w < 4; ++w) {
                  const float4 u = *reinterpret_cast<const float4*>(&s_red[w][c]);
                  t4 = make_float4(fmaxf(t4.x, u.x), fmaxf(t4.y, u.y), fmaxf(t4.z, u.z), fmaxf(t4.w, u.w));
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float2 m0 = j == j0 ? make_float2(-FLT_MAX, -FLT_MAX) : refs[c / 2 + e];
                  const float2 m = make_float2(moved(c + 2 * e, e ? t4.z : t4.x, m0.x), moved(c + 2 * e + 1, e ? t4.w : t4.y, m0.y));
                  scale[c / 2 + e] = make_float2(m0.x == m.x ? 1.0f : ta_ex2(m0.x - m.x), m0.y == m.y ? 1.0f : ta_ex2(m0.y - m.y));
                  refs[c / 2 + e] = m;
                }
              }
            } else {
              if (tid < R) {
                const float m0 = j == j0 ? -FLT_MAX : s_ref[tid];
                const float m = moved(tid, fmaxf(fmaxf(s_red[0][tid], s_red[1][tid]), fmaxf(s_red[2][tid], s_red[3][tid])), m0);
                s_scale[tid] = m0 == m ? 1.0f : ta_ex2(m0 - m);
                s_ref[tid] = m;
              }
              tf_any(false);
              if constexpr (KEEP)
#pragma unroll
                for (int c = 0; c < R / 2; ++c) refs[c] = reinterpret_cast<const float2*>(s_ref)[c];
            }
#pragma unroll
            for (int c = 0; c < R / 2; ++c)
#pragma unroll
              for (int t = 0; t < C::KT; ++t)
                y[t][c] = make_float2(score(y[t][c].x, z[t][c].x, factor(c).x, ref(c).x), score(y[t][c].y, z[t][c].y, factor(c).y, ref(c).y));
            if (j > j0) {
              tc::tc_fence_after();
              grown = true;
#pragma unroll
              for (int c = 0; c < R / 2; ++c) l[c] = make_float2(l[c].x * factor_of(c).x, l[c].y * factor_of(c).y);
              auto rescale = [&](uint32_t at, float2 f0, float2 f1) {
                float o[4];
                tc::tmem_ld4(at, o);
                tc::tmem_ld_wait();
                tc::reg_fence(o);
                o[0] *= f0.x;
                o[1] *= f0.y;
                o[2] *= f1.x;
                o[3] *= f1.y;
                tc::tmem_st4(at, o);
              };
#pragma unroll 1
              for (int hm = 0; hm < (F32 ? 0 : C::UNITS); ++hm) {
                if constexpr (ALL) {
#pragma unroll
                  for (int c = 0; c < C::COLS; c += 4) rescale(t_o + hm * NR + c, factor_of(c % R / 2), factor_of(c % R / 2 + 1));
                } else {
#pragma unroll 1
                  for (int c = 0; c < C::COLS; c += 4) {
                    const float2* f = reinterpret_cast<const float2*>(s_scale) + c % R / 2;
                    rescale(t_o + hm * NR + c, f[0], f[1]);
                  }
                }
              }
              if (!F32) tc::tmem_st_wait();
            }
          }
          ok = ctl.wait(&pv_done[b], (step >> 1 & 1) ^ 1) && ok;  // P^T of two steps ago is used up
#pragma unroll
          for (int t = 0; t < C::KT; ++t) {
            uint32_t pk[C::COLS / 2];
#pragma unroll
            for (int c = 0; c < R / 2; ++c) {
              const float2 w = make_float2(ta_ex2(y[t][c].x), ta_ex2(y[t][c].y));
              l[c] = ta_add2(l[c], w);
              pk[c] = tq_pack(w.x, w.y);
              if (F32) pk[(C::COLS - R) / 2 + c] = tq_rest(w.x, w.y, pk[c]);
            }
            // the key's row of P^T: 16-byte pieces where the tensor core's swizzle has them
            uint8_t* row = s_p + b * C::PB + t * C::PT + tid * C::PROW;
            const int sw = NR == 16 ? tid >> 2 & 1 : tid >> 1 & 3;
            if constexpr (C::COLS == 4) {
              *reinterpret_cast<uint2*>(row + (sw << 4)) = make_uint2(pk[0], pk[1]);
            } else {
#pragma unroll
              for (int c = 0; c < C::COLS / 8; ++c)
                *reinterpret_cast<uint4*>(row + ((c ^ sw) << 4)) =
                    make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
            }
          }
          tc::fence_proxy_async_smem();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&p_full[b]);
        }
        if (F32 && j > j0) {  // the product of the step before
          ok = ctl.wait(&pv_done[b ^ 1], (step - 1) >> 1 & 1) && ok;
          tc::tc_fence_after();
          const uint32_t t_b = lanes + C::O_COL + (b ^ 1) * (C::UNITS * NR);
#pragma unroll
          for (int hm = 0; hm < (F32 ? C::UNITS : 0); ++hm) {
            float o[F32 ? C::COLS : 16];
#pragma unroll
            for (int c = 0; c < C::COLS; c += 16) tc::tmem_ld16(t_b + hm * NR + c, *reinterpret_cast<float(*)[16]>(o + c));
            tc::tmem_ld_wait();
            tc::reg_fence(o);
#pragma unroll
            for (int c = 0; c < R / 2; ++c) {
              acc[hm][c] = ta_add2(acc[hm][c], ta_add2(make_float2(o[2 * c], o[2 * c + 1]), make_float2(o[C::COLS - R + 2 * c], o[C::COLS - R + 2 * c + 1])));
              if (grown) acc[hm][c] = make_float2(acc[hm][c].x * factor_of(c).x, acc[hm][c].y * factor_of(c).y);
            }
            if (j >= j1)  // the sums back to where they are written out from, as other types' are
#pragma unroll
              for (int c = 0; c < R; c += 4) {
                const float4 v = make_float4(acc[hm][c / 2].x, acc[hm][c / 2].y, acc[hm][c / 2 + 1].x, acc[hm][c / 2 + 1].y);
                tc::tmem_st4(t_b + hm * NR + c, *reinterpret_cast<const float(*)[4]>(&v));
              }
          }
          if (j >= j1) tc::tmem_st_wait();
          tc::tc_fence_before();
          __syncwarp();
          if (j < j1 && lane == 0) tc::mbar_arrive(&o_empty[b ^ 1]);
        }
        if (F32 && j >= j1) break;
      }
      if (out) break;
      const bool any = j1 > j0;
      // the rows' sums over the threads
      float v[R];
#pragma unroll
      for (int c = 0; c < R / 2; ++c) {
        v[2 * c] = l[c].x;
        v[2 * c + 1] = l[c].y;
      }
      tf_combine<R>(v, [](float p, float q) { return p + q; });
      if (any) {
        ok = ctl.wait(&pv_done[(step - 1) & 1], (step - 1) >> 1 & 1) && ok;
        tc::tc_fence_after();
        ++no;
      }
      if (F32) {  // the last product's
        ob = (step - 1) & 1;
        t_o = lanes + C::O_COL + ob * (C::UNITS * NR);
      }
      // Not before the wait: it ends once all four warps have handed in the last step's weights, and until then one
      // of them may still read that step's maxima from s_red.  (Without keys nothing has been read since the barrier
      // at the item's start.)
      s_red[warp][tf_column<R>()] = v[0];
      if (R <= 8 && tid == 0)
#pragma unroll
        for (int c = 0; c < R / 2; ++c) reinterpret_cast<float2*>(s_ref)[c] = ref(c);
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
          float o[C::UNITS][4];
#pragma unroll
          for (int hm = 0; hm < C::UNITS; ++hm)
            if (any) tc::tmem_ld4(t_o + hm * NR + c, o[hm]);
          if (any) tc::tmem_ld_wait();
#pragma unroll
          for (int hm = 0; hm < C::UNITS; ++hm) tc::reg_fence(o[hm]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (c + e >= rows) break;
            if (whole) {
              const float sum = row_sum(c + e), inv = __fdividef(1.0f, sum);
#pragma unroll
              for (int hm = 0; hm < C::UNITS; ++hm) {
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
              for (int hm = 0; hm < C::UNITS; ++hm)
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
          // The item's last CTA joins its parts, up to PARTS at a time: first their weights, then the
          // sums, a thread four columns of every RP-th row.
          __threadfence();
          float2* wt = s_join;  // [part][row]
          constexpr int PARTS = TQ_JOIN / (R * 8), RP = 512 / DP, PASSES = R < RP ? 1 : R / RP;
          constexpr int BATCH = PASSES >= 16 ? 1 : 16 / PASSES;  // parts loaded at once
          const int col = tid % (DP / 4) * 4, r0 = min(tid / (DP / 4), R - 1);
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
            for (int i = tid; i < nq * R; i += 128)
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
            if (r >= rows || col >= a.D || tid / (DP / 4) >= R) continue;
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
  } else if (group >= 2 && group < 2 + TQ_KEYS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    // ------------------------------------------------------------ keys: a row a thread, to its lane of TMEM
    const int r = tid & 127, g = group - 2;
    const uint32_t lanes = tmem + ((uint32_t)(r & ~31) << 16) + C::K_COL;
    TqStream<C, TQ_KEYS, 0> str{a, cache, ctl, s_item, i_full, i_empty, s_copy + g * C::DEPTH * C::SB, (uint32_t)g};
    uint32_t s = g;  // unit
    while (str.issue()) {
      if (__builtin_expect(!str.come(), 0)) continue;
      const uint32_t kb = s % C::KBUF;
      if (!ctl.wait(&k_empty[kb], (s / C::KBUF & 1) ^ 1)) break;
      tc::tc_fence_after();
      tq_row<C>(str.ring + str.stage, r, [&](int p, const uint32_t (&y)[16]) {
        tc::tmem_st16(lanes + kb * (C::COL / 2) + p * 16, *reinterpret_cast<const float(*)[16]>(y));
      });
      tc::tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&k_full[kb]);
      s += TQ_KEYS;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // none is in flight when the CTA leaves
  } else if (group >= 2 + TQ_KEYS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    // ------------------------------------------------------------ values: to shared memory
    const int r = tid & 127, g = group - 2 - TQ_KEYS;
    uint8_t* ring = s_copy + (TQ_KEYS + g) * C::DEPTH * C::SB;
    uint32_t o[4];  // where the row's 16-byte pieces lie
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = (c ^ (r & 7)) << 4;
    TqStream<C, TQ_VALUES, 1> str{a, cache, ctl, s_item, i_full, i_empty, ring, (uint32_t)g};
    uint32_t vb = g, par = 1;  // (C::VBUF >= TQ_VALUES)
    while (str.issue()) {
      if (__builtin_expect(!str.come(), 0)) continue;
      if (!ctl.wait(&v_empty[vb], par)) break;
      uint8_t* line = s_v + vb * C::VB + r * 128;
      tq_row<C>(ring + str.stage, r, [&](int p, const uint32_t (&y)[16]) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(line + p / 2 * C::V_SLAB + (o[c] ^ (p & 1) << 6)) = make_uint4(y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]);
      });
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&v_full[vb]);
      vb += TQ_VALUES;
      if (vb >= C::VBUF) {
        vb -= C::VBUF;
        par ^= 1;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (role == 0) {
    // ------------------------------------------------------------ S^T = K Q^T: one thread
    // The two kinds of products have a thread each, which sleeps where what it needs is not there: one
    // thread that looked for either took a quarter of the SM's issue slots.
    if (tc::elect_one()) {
      constexpr uint32_t id_s = tc::idesc_f16(128, NR, 0, 0);
      const uint64_t d_q = tc::smem_desc(tc::smem_u32(s_q), 16, 1024, tc::LAYOUT_SW128);
      uint32_t ks = 0, step = 0, nq = 0;  // units of K used, steps, items with keys
      bool ok = true;
      for (uint32_t ni = 0; ok; ++ni) {
        ok = ctl.wait1(&i_full[ni % TA_ITEMS], ni / TA_ITEMS & 1);
        if (!ok) break;
        const TaItem& it = s_item[ni % TA_ITEMS];
        if (it.n < 0) break;
        const int j0 = it.j0, j1 = it.j1;
        tc::mbar_arrive(&i_empty[ni % TA_ITEMS]);
        if (j1 <= j0) continue;
        const uint32_t qb = nq % C::QBUF;
        ok = ctl.wait1(&q_full[qb], nq / C::QBUF & 1);
        ++nq;
        for (int j = j0; j < j1 && ok; j += C::KT, ++step) {
          const uint32_t b = step & 1;
          ok = ctl.wait1(&s_empty[b], (step >> 1 & 1) ^ 1);
          const int kt = min(C::KT, j1 - j);
#pragma unroll 1
          for (int t = 0; t < kt && ok; ++t)
#pragma unroll
            for (int u = 0; u < C::UNITS; ++u, ++ks) {
              const uint32_t kb = ks % C::KBUF;
              ok = ok && ctl.wait1(&k_full[kb], ks / C::KBUF & 1);
              if (!ok) break;
              tc::tc_fence_after();
#pragma unroll
              for (int k = 0; k < C::COL / 16; ++k)
                tc::mma_ts(tmem + C::S_COL + b * C::S_WIDTH + t * C::COLS, tmem + C::K_COL + kb * (C::COL / 2) + k * 8,
                           d_q + ((qb * C::QB + (u * C::COL / 64 + k / 4) * C::QSLAB + k % 4 * 32) >> 4), id_s, u > 0 || k > 0);
              tc::mma_commit(&k_empty[kb]);
            }
          if (!ok) break;
          tc::mma_commit(&s_full[b]);
          if (j + C::KT >= j1) tc::mma_commit(&q_empty[qb]);
        }
      }
      tc::mma_commit(drain);  // arrives when all of this thread's products are done
    }
  } else if (role == 2) {
    // ------------------------------------------------------------ O^T += V^T P^T: one thread
    if (tc::elect_one()) {
      constexpr uint32_t id_o = tc::idesc_f16(128, NR, 1, 1);
      // V^T: 64 columns a slab; D <= 64 has one, read twice for the 128 rows of the product
      const uint64_t d_v = tc::smem_desc(tc::smem_u32(s_v), DP == 64 ? 0 : C::V_SLAB, 1024, tc::LAYOUT_SW128);
      const uint64_t d_p = tc::smem_desc(tc::smem_u32(s_p), 16, 8 * C::PROW, C::P_LAYOUT);
      uint32_t vn = 0, step = 0, no = 0;  // units of V used, steps, items with keys
      bool ok = true;
      for (uint32_t ni = 0; ok; ++ni) {
        ok = ctl.wait1(&i_full[ni % TA_ITEMS], ni / TA_ITEMS & 1);
        if (!ok) break;
        const TaItem& it = s_item[ni % TA_ITEMS];
        if (it.n < 0) break;
        const int j0 = it.j0, j1 = it.j1;
        tc::mbar_arrive(&i_empty[ni % TA_ITEMS]);
        if (j1 <= j0) continue;
        // O^T's buffer is an item's, of float32 a step's
        if (!F32) ok = ctl.wait1(&o_empty[no & 1], (no >> 1 & 1) ^ 1);
        ++no;
        uint32_t more = 0;  // not the buffer's first product
        for (int j = j0; j < j1 && ok; j += C::KT, ++step) {
          const uint32_t b = step & 1, ob = F32 ? b : (no - 1) & 1;
          if (F32) {
            ok = ctl.wait1(&o_empty[b], (step >> 1 & 1) ^ 1);
            more = 0;
          }
          ok = ok && ctl.wait1(&p_full[b], step >> 1 & 1);
          const int kt = min(C::KT, j1 - j);
#pragma unroll 1
          for (int t = 0; t < kt && ok; ++t, more = 1)
#pragma unroll
            for (int u = 0; u < C::UNITS; ++u, ++vn) {
              const uint32_t vb = vn % C::VBUF;
              ok = ok && ctl.wait1(&v_full[vb], vn / C::VBUF & 1);
              if (!ok) break;
              tc::tc_fence_after();
#pragma unroll
              for (int k = 0; k < TA_BN / 16; ++k)
                tc::mma_bf16(tmem + C::O_COL + (ob * C::UNITS + u) * NR, d_v + ((vb * C::VB + k * 2048) >> 4),
                             d_p + ((b * C::PB + t * C::PT + k * 16 * C::PROW) >> 4), id_o, k > 0 ? 1u : more);
              tc::mma_commit(&v_empty[vb]);
            }
          if (ok) tc::mma_commit(&pv_done[b]);
        }
      }
      tc::mma_commit(drain);
    }
  } else if (role == 1) {
    // ------------------------------------------------------------ walk
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
      more = w.next(a);
    }
  } else if (role == 3) {
    // ------------------------------------------------------------ queries
    uint32_t n = 0;  // items with keys
    bool ok = true;
    for (uint32_t ni = 0; ok; ++ni) {
      ok = ctl.wait(&i_full[ni % TA_ITEMS], ni / TA_ITEMS & 1);
      if (!ok) break;
      const TaItem x = s_item[ni % TA_ITEMS];
      if (x.n < 0) break;
      if (x.j1 > x.j0) {
        // Queries: LPR lanes a row, 8 channels a lane.
        const uint32_t qb = n % C::QBUF;
        ok = ctl.wait(&q_empty[qb], (n / C::QBUF & 1) ^ 1);
        if (!ok) break;
        constexpr int LPR = DP / 8, RPP = 32 / LPR, PASSES = R < RPP ? 1 : R / RPP, BATCH = PASSES < 4 ? PASSES : 4;
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
            if (r >= R) continue;
            *reinterpret_cast<uint4*>(dst + r * 128 + ((c0 / 8 % 8 ^ (r & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if (F32)
              *reinterpret_cast<uint4*>(dst + (r + R) * 128 + ((c0 / 8 % 8 ^ ((r + R) & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            if (lane % LPR == 0)
              s_factor[ni % TA_ITEMS][r] =
                  fminf(fmaxf(a.scale_log2 * __uint_as_float((uint32_t)max(ex - 14 + 127, 1) << 23), FLT_MIN), FLT_MAX);  // (0 times infinity is none)
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&q_full[qb]);
        ++n;
      }
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&r_full[ni % TA_ITEMS]);
        tc::mbar_arrive(&i_empty[ni % TA_ITEMS]);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (s_flag && tid < 32) tc::mbar_wait(drain, 0, a.wait_ns);  // a wait ran out: products in flight end
  __syncthreads();
  if (role == 0) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int DP, int R, bool F32>
cudaError_t run(PagedArgs& a, const Q4Cache& c, cudaStream_t s, int sms) {
  using C = Tq<DP, R, F32>;
  const void* f = reinterpret_cast<const void*>(k_paged_attn_q4<DP, R, F32>);
  static std::atomic<uint64_t> ready{0};
  // the register split draws on what the launch gives
  const cudaError_t e = ta_prepare(f, C::smem, 80, ready);
  if (e != cudaSuccess) return e;
  a.tb = R / a.g;
  const PagedWs L = paged_ws(sms, R, DP);
  a.part_ml = L.ml;
  a.part_o = L.o;
  a.rows = R;
  pg_division(a, sms, 640, 192, 256);
  Q4Cache cache = c;
  void* args[] = {&a, &cache};
  return launch_pdl(f, dim3(sms), dim3(TQ_THREADS), C::smem, s, args, 1);
}

// Rows of a tile: no more than a request's in the mean ask for.
int tile_rows(bool f32, int rows) {
  if (f32) return rows <= 8 ? 8 : 16;
  return rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
}

template <int DP>
cudaError_t run_rows(PagedArgs& a, const Q4Cache& c, bool f32, int rows, cudaStream_t s, int sms) {
  if (f32) return rows == 8 ? run<DP, 8, true>(a, c, s, sms) : run<DP, 16, true>(a, c, s, sms);
  if constexpr (DP == 256)  // (narrower heads have their many rows elsewhere)
    if (rows == 32) return run<DP, 32, false>(a, c, s, sms);
  return rows == 4 ? run<DP, 4, false>(a, c, s, sms) : rows == 8 ? run<DP, 8, false>(a, c, s, sms) : run<DP, 16, false>(a, c, s, sms);
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
  c.s_whole = q4_whole_scales(a, c);
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

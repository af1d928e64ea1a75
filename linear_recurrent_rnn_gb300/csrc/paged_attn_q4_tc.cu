// Attention over the paged cache held in 4 bits (include/paged_q4.h), many rows a request.
//
// The products and the softmax are those of the kernel for many rows over a bf16 cache (paged_attn_tc.cu):
//   S = Q K^T, P = 2^(c S - c m), O += P V, rows along the 128 lanes, one thread a row.
// What is new: a warpgroup copies codes and scales (cp.async, its own 32 rows a warp) and writes the
// numbers that they stand for to the ring of key and value tiles as f16, which holds them exactly; rows that no
// row of the item sees, and pages that are not there, are zeros there.  Queries come by TMA and are rewritten in
// place as f16, each row times the power of two that brings its largest element to [2^14, 2^15) (bf16's 8
// significant bits fit f16's 11); its scores are multiplied by the inverse.  Weights are f16 and held times a
// power of two; the maximum is moved when a weight would pass 2^15.  float32 queries and weights are sums of two f16
// (22 bits): each of the two is multiplied with the same keys or values into the same sums, twice the products, the small
// halves first.  The tensor core cuts what it adds to a sum (paged_attn_q4.cu has the figures), so float32's product of a
// key tile's unit is a sum of its own in TMEM, and the row's thread adds it to the sums there, a tile behind; heads of 256 leave
// TMEM for one S only then, and their two products take turns with the softmax (122 -> 157 us below; heads of 128 120 -> 128).
//
// Widths up to 128: one row tile a CTA and two warpgroups that bring keys and values, or, for long prompts in bf16, two
// row tiles and one (row_tiles below; a second beside two tiles needs registers that softmax has: reading the
// scores twice, so as not to hold 128 of them, took 2161 us where this takes 1822, of 8 chunks of 2048 tokens in 8192, 32
// heads on 8 of 128).  Width 256: one row tile and three (8 chunks of 2048 tokens in 8192, 10 heads on 1, window 2048:
// 590 us with one, 377 with two, 340 with three), or one where float32 queries take the shared memory.
// Measured (GB300): those chunks 1.05 PFLOP/s (1.41 over bf16 caches), with heads of 256 1.01; 20 decode rows and 4
// chunks of 300 to 777 tokens in up to 8192, 104 us.  What bounds it: a warpgroup's 2250 cycles a unit, of which a key
// tile has two, against 1024 of products a row tile; a lone warp a scheduler issues in order, ten cycles an
// instruction.  float32, 4 chunks of 700 tokens in 1000 to 4096, 16 heads on 4 of 128: 128 us, 10 on 1 of 256:
// 157 (the kernel for few rows, before it added steps up: four and six times as much).
#include <float.h>

#include <algorithm>
#include <type_traits>

#include "host_util.h"
#include "paged_q4.cuh"

namespace rglru {

namespace {

template <int DP, bool F32, int NT_>
struct Tm {
  static constexpr int NT = NT_;                      // row tiles
  // weights are held times 2^SHIFT, and may grow to 2^15 before a row's sums are scaled anew: rarer with 7, but the
  // numbers then end at 2^-32 of the largest, with 11 at 2^-36
  static constexpr float SHIFT = F32 ? 11.0f : 7.0f;
  static constexpr int NUM = F32 ? 2 : 1;             // f16 numbers for one of a query or weight
  static constexpr int SLABS = NUM * DP / 64;         // 64 columns of f16, of either number in turn
  // Units: 128 keys (or values) of up to 128 columns; what is copied, dequantised and multiplied at once.
  static constexpr int UNITS = DP == 256 ? 2 : 1;     // of a tile
  static constexpr int COL = DP / UNITS;              // columns of one
  static constexpr uint32_t RB = COL / 2, SP = COL / 16;  // bytes of a row's codes, of its scales
  static constexpr uint32_t SB = 1024 * ((TA_BN * (RB + SP) + 1023) / 1024);  // a unit's
  static constexpr uint32_t UB = TA_BN * COL * 2;     // of a unit as f16
  static constexpr int STAGES = DP == 64 ? 6 : DP == 256 && F32 ? 2 : 3;  // units as f16
  static constexpr int SOFT = NT * 128;               // softmax threads
  // warpgroups that bring keys and values, a unit each in turn
  static constexpr int GROUPS = NT == 2 || (DP == 256 && F32) ? 1 : DP == 256 ? 3 : 2;
  static constexpr int THREADS = SOFT + 128 + GROUPS * 128;
  // Registers of a thread: at launch, and after the softmax's warpgroups have taken what the others give up.
  static constexpr int REGS = 65536 / THREADS / 8 * 8;
  static constexpr int SOFT_REGS = NT == 2 ? 184 : GROUPS == 3 ? 192 : 224;
  static constexpr int OTHER_REGS = (REGS * THREADS - SOFT_REGS * SOFT) / (THREADS - SOFT) / 8 * 8;
  // TMEM: S/P buffers b at 128 b, O tiles; of float32 O's sums, and the product of a key tile's unit that is added to
  // them (heads of 256 leave room for one S/P)
  static constexpr int S_BUF = F32 && DP == 256 ? 1 : 2;
  static constexpr uint32_t S_COL = 0, O_COL = 256, STEP_COL = DP == 256 ? 128 : 256 + DP;
  static_assert(!F32 || NT == 1, "one row tile");
  static constexpr size_t Q_BYTES = (size_t)NT * SLABS * TA_SLAB;
  static constexpr int FIT = (int)((232448 - 4096 - 1024 - Q_BYTES - STAGES * UB - 1024) / SB);
  static constexpr int DEPTH = FIT / GROUPS < 6 ? FIT / GROUPS : 6;  // units of codes on their way, of a group
  static constexpr size_t smem = 1024 + Q_BYTES + STAGES * UB + (size_t)GROUPS * DEPTH * SB + 1024;
  static_assert(DEPTH >= 2 && GROUPS <= STAGES, "shared memory");
  static_assert(STAGES * UB + (size_t)GROUPS * DEPTH * SB >= (PG_MAX_SEQS + 1) * 8, "the scan of the requests");
};

template <int DP, bool F32, int NT_>
__global__ void __launch_bounds__(Tm<DP, F32, NT_>::THREADS, 1)
    k_paged_attn_q4_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ PagedArgs a,
                       const __grid_constant__ Q4Cache cache) {
  using C = Tm<DP, F32, NT_>;
  using IO = std::conditional_t<F32, float, bf16>;
  constexpr int NT = C::NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* s_q = smem;
  uint8_t* s_ring = s_q + C::Q_BYTES;
  uint8_t* s_copy = s_ring + C::STAGES * C::UB;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_copy + (size_t)C::GROUPS * C::DEPTH * C::SB);
  uint64_t* empty = full + C::STAGES;
  uint64_t* q_full = empty + C::STAGES;  // [NT]
  uint64_t* q_empty = q_full + NT;       // [NT]
  uint64_t* q_ready = q_empty + NT;      // [NT] rewritten as f16, the rows' factors there
  uint64_t* f_empty = q_ready + NT;      // [NT] the factors read
  uint64_t* s_full = f_empty + NT;       // [2]  S of buffer b complete
  uint64_t* p_full = s_full + 2;         // [2]  P of buffer b written (and O scaled)
  uint64_t* pv_done = p_full + 2;        // [NT] a product P V of tile t complete
  uint64_t* o_empty = pv_done + NT;      // [NT] O of tile t read
  uint64_t* j_full = o_empty + NT;       // a part of an item is in the workspace
  uint64_t* j_go = j_full + 1;           // s_last says whether this CTA joins the item
  uint64_t* j_here = j_go + 1;           // [TA_ITEMS] s_here says whether this CTA has the last part
  uint64_t* i_full = j_here + TA_ITEMS;           // [TA_ITEMS] item records
  uint64_t* i_empty = i_full + TA_ITEMS;
  uint64_t* drain = i_empty + TA_ITEMS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  uint32_t* s_flag = tmem_holder + 1;
  uint32_t* s_last = tmem_holder + 2;
  __shared__ int64_t scratch[33];
  __shared__ TaItem s_item[TA_ITEMS];
  __shared__ float s_factor[NT * 128];   // of the rows' scores
  __shared__ uint32_t s_here[TA_ITEMS];
  __shared__ uint32_t s_issued[NT];      // loads issued: queries of each tile
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tb1 = max(1, 128 / a.g);  // tokens of a row tile
  const TqAbort ctl{s_flag, reinterpret_cast<uint32_t*>(a.ws), (uint32_t)(a.wait_ns >> 10) + 1};

  // up to griddep_wait nothing touches global memory
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      tc::mbar_init(&full[i], 4);
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NT; ++i) {
      tc::mbar_init(&q_full[i], 1);
      tc::mbar_init(&q_empty[i], 1);
      tc::mbar_init(&q_ready[i], NT == 2 ? 1 : 2);
      tc::mbar_init(&f_empty[i], 4);
      tc::mbar_init(&pv_done[i], 1);
      tc::mbar_init(&o_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s_full[i], 1);
      tc::mbar_init(&p_full[i], 4);
    }
    tc::mbar_init(j_full, C::SOFT / 32);
    tc::mbar_init(j_go, 1);
    for (int i = 0; i < TA_ITEMS; ++i) {
      tc::mbar_init(&j_here[i], 1);
      tc::mbar_init(&i_full[i], 1);
      tc::mbar_init(&i_empty[i], C::SOFT / 32 + 1 + 2 + 4 * C::GROUPS);
    }
    tc::mbar_init(drain, 1);
    for (int i = 0; i < NT; ++i) s_issued[i] = 0u;
    *s_flag = 0u;
    tc::fence_barrier_init();
    tc::prefetch_tmap(&tm_q);
  }
  if (warp == C::SOFT / 32 + 1) {
    tc::tmem_alloc(tmem_holder, 512);
    tc::tmem_relinquish();
  }
  // < 0: softmax; 0, 2: queries to f16, 1: MMA, 3: walk and queries; 4 and on: keys and values
  const int role = warp - C::SOFT / 32;
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  PgWalk w;
  PgWalk::Found start;
  if (a.N <= PG_WARP_SEQS) {
    if (role == 3) start = w.find_warp(a);
  } else {
    int64_t* prefix = reinterpret_cast<int64_t*>(s_ring);  // before the ring is in use
    pg_scan(a, prefix, scratch);
    if (role == 3) start = w.find(a, prefix);
    tc::fence_proxy_async_smem();
    __syncthreads();
  }
  const uint32_t tmem = *tmem_holder;

  uint32_t ni = 0;  // items so far
  // the next item, or null at the end of the work (or of a wait); done() hands its record back
  auto next_item = [&]() -> const TaItem* {
    if (!ctl.wait(&i_full[ni % TA_ITEMS], ni / TA_ITEMS & 1)) return nullptr;
    const TaItem* it = &s_item[ni % TA_ITEMS];
    return it->n < 0 ? nullptr : it;
  };
  auto done_item = [&] {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&i_empty[ni % TA_ITEMS]);
    ++ni;
  };
  if (role < 0) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFT_REGS));
    // ------------------------------------------------------------ softmax, one row a thread
    const int t = NT == 2 ? warp >> 2 : 0, wq = warp & 3, r = wq * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t t_o = lanes + C::O_COL + t * DP;
    uint32_t cs = 0, npv = 0, nj = 0, nf = 0;  // S taken, products P V of this tile (float32: of its units), parts handed over
    // float32: the product in STEP_COL is added to the sums of unit u, or is the first of them.  The sums so far are multiplied by
    // f, and with `old` the product too: it is of a tile before the sums' growth.
    constexpr int ADD = 64;  // columns at once
    auto add_product = [&](int u, bool first, bool old, float f, bool live) {
      tc::tc_fence_after();
      if (live) {
        const float fx = old ? f : 1.0f;
#pragma unroll 1
        for (int c = 0; c < C::COL && u * C::COL + c < a.D; c += ADD) {
          __syncwarp();
          float x[ADD], y[ADD];
#pragma unroll
          for (int e = 0; e < ADD; e += 16) {
            tc::tmem_ld16(lanes + C::STEP_COL + c + e, *reinterpret_cast<float(*)[16]>(x + e));
            tc::tmem_ld16(t_o + u * C::COL + c + e, *reinterpret_cast<float(*)[16]>(y + e));
          }
          tc::tmem_ld_wait();
          tc::reg_fence(x);
          tc::reg_fence(y);
#pragma unroll
          for (int e = 0; e < ADD; ++e) x[e] = first ? x[e] * fx : fmaf(y[e], f, x[e] * fx);
#pragma unroll
          for (int e = 0; e < ADD; e += 16) tc::tmem_st16(t_o + u * C::COL + c + e, *reinterpret_cast<const float(*)[16]>(x + e));
        }
        tc::tmem_st_wait();
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&o_empty[0]);
    };
    uint32_t here_par = 0;             // parities of j_here
    bool ok = true;
    const TaItem* rec;
    while (ok && (rec = next_item())) {
      const TaItem& it = *rec;
      const TaTile tl = ta_tile(a, it, t, tb1);
      const bool live = wq * 32 < tl.rows;  // any row of the warp
      const int base = it.kv - it.q + tl.tok;
      const int my_tok = pg_token(a, min(r, max(tl.rows - 1, 0))), pos = base + my_tok;
      // positions of the warp's first and last row: tiles between need no mask
      const int p_first = base + pg_token(a, wq * 32), p_last = base + pg_token(a, min(wq * 32 + 31, max(tl.rows - 1, 0)));
      float m = -INFINITY, l = 0.0f;  // in units of the scores; the sum at that maximum
      float sc = 0.0f;                // the row's factor
      if (tl.jb > tl.ja) {
        ok = ctl.wait(&q_ready[t], nf++ & 1);
        if (!ok) break;
        sc = s_factor[t * 128 + r];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&f_empty[t]);
      }
      for (int j = tl.ja; j < tl.jb; ++j) {
        const int b = NT == 2 ? t : C::S_BUF == 1 ? 0 : cs & 1;
        ok = ctl.wait(&s_full[b], (NT == 2 || C::S_BUF == 1 ? cs : cs >> 1) & 1);
        ++cs;
        if (!ok) break;
        tc::tc_fence_after();
        bool waited = j == tl.ja;  // NT = 1: for the product before this one
        float grown = 1.0f;        // float32: what the sums so far are to be multiplied by
        if (live) {
          float s[128];
          const uint32_t t_s = lanes + C::S_COL + b * 128;
#pragma unroll
          for (int c = 0; c < 8; ++c) tc::tmem_ld16(t_s + 16 * c, *reinterpret_cast<float(*)[16]>(s + 16 * c));
          tc::tmem_ld_wait();
          tc::reg_fence(s);
          const int k0 = j * TA_BN;
          if (k0 + TA_BN - 1 > p_first || (a.window && k0 < p_last - a.window + 1)) {
            const int hi = pos - k0, lo = a.window ? hi - a.window : -1;  // lo < column <= hi
            uint32_t bits[4];  // one a column: a test and a select a score
#pragma unroll
            for (int w = 0; w < 4; ++w) bits[w] = ta_bits(hi - 32 * w) & ~ta_bits(lo - 32 * w);
#pragma unroll
            for (int c = 0; c < 128; ++c) s[c] = bits[c / 32] & (1u << c % 32) ? s[c] : -INFINITY;
          }
          float mx[4] = {m, s[1], s[2], s[3]};
          mx[0] = fmaxf(m, s[0]);
#pragma unroll
          for (int c = 4; c < 124; c += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = ta_max3(mx[e], s[c + e], s[c + 4 + e]);
          const float top = ta_max3(ta_max3(mx[0], s[124], s[125]), ta_max3(mx[1], s[126], s[127]),
                                    fmaxf(mx[2], mx[3]));
          if (j == tl.ja) {
            m = top;
          } else if (__any_sync(0xffffffffu, r < tl.rows && (top - m) * sc > 15.0f - C::SHIFT)) {  // (of rows in use)
            const float f = top == m ? 1.0f : ta_ex2((top - m) * -sc);
            l *= f;
            m = top;
            grown = f;
            if (NT == 1 && !F32) {
              ok = ctl.wait(&pv_done[0], (npv + (j - tl.ja) - 1) & 1);
              waited = true;
              if (!ok) break;
              tc::tc_fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < (F32 ? 0 : DP); c += 16) {
              float o[16];
              tc::tmem_ld16(t_o + c, o);
              tc::tmem_ld_wait();
              tc::reg_fence(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= f;
              tc::tmem_st16(t_o + c, o);
            }
          }
          const float off = m == -INFINITY ? 0.0f : fmaf(-m, sc, C::SHIFT);
          float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            float pk[16], pl[16];  // and what is left of float32 ones
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 x = ta_fma2(make_float2(s[c + 2 * e], s[c + 2 * e + 1]), make_float2(sc, sc),
                                       make_float2(off, off));
              const float2 p = make_float2(ta_ex2(x.x), ta_ex2(x.y));
              sum[e & 1] = ta_add2(sum[e & 1], p);
              const uint32_t hi = tq_pack(p.x, p.y);
              pk[e] = __uint_as_float(hi);
              if (F32) pl[e] = __uint_as_float(tq_rest(p.x, p.y, hi));
            }
            tc::tmem_st16(t_s + c / 2, pk);
            if (F32) tc::tmem_st16(t_s + 64 + c / 2, pl);
          }
          const float2 s2 = ta_add2(sum[0], sum[1]);
          l += s2.x + s2.y;
          tc::tmem_st_wait();
        }
        if (NT == 1 && !F32 && !waited) {
          ok = ctl.wait(&pv_done[0], (npv + (j - tl.ja) - 1) & 1);
          if (!ok) break;
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&p_full[b]);
        if constexpr (F32) {
          // the last unit's product of the tile before, then this tile's, but for its last unit's
#pragma unroll 1
          for (int u = -1; u < C::UNITS - 1 && ok; ++u) {
            if (u < 0 && j == tl.ja) continue;
            ok = ctl.wait(&pv_done[0], npv++ & 1);
            if (ok) add_product(u < 0 ? C::UNITS - 1 : u, j == tl.ja + (u < 0 ? 1 : 0), u < 0, grown, live);
          }
          if (!ok) break;
        }
      }
      if (!ok) break;
      const bool any = tl.jb > tl.ja;
      // If all other parts of an item are there by now, this CTA joins them to its own in TMEM.
      const int parts = it.c1 - it.c0 + 1;
      bool here = parts == 1;
      if (parts > 1 && parts <= TA_HERE) {
        const uint32_t k = ni % TA_ITEMS;
        if (tid == 0) {
          uint32_t* cnt = reinterpret_cast<uint32_t*>(a.ws + 256) + it.c0;
          uint32_t had;
          asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(had) : "l"(cnt) : "memory");
          const bool all = had == (uint32_t)(parts - 1);
          if (all) *cnt = 0u;  // as it was found: zero between calls
          *reinterpret_cast<volatile uint32_t*>(&s_here[k]) = all;
          tc::mbar_arrive(&j_here[k]);
        }
        __syncwarp();
        ok = ctl.wait(&j_here[k], here_par >> k & 1);
        if (!ok) break;
        here_par ^= 1u << k;
        here = *reinterpret_cast<volatile uint32_t*>(&s_here[k]);
      }
      if (any) {
        npv += F32 ? 1 : tl.jb - tl.ja;
        ok = ctl.wait(&pv_done[t], (npv - 1) & 1);
        if (!ok) break;
        tc::tc_fence_after();
        if (F32) add_product(C::UNITS - 1, tl.jb == tl.ja + 1, false, 1.0f, live);
      }
      const bool mine = r < tl.rows;
      const int row = t * 128 + r;
      constexpr int R = NT * 128;
      const float2* g_ml = reinterpret_cast<const float2*>(a.ws + a.part_ml);
      const float* g_o = reinterpret_cast<const float*>(a.ws + a.part_o);
      // (rounded here as in memory, whichever of the two it is joined from)
      const float2 own = make_float2(m == -INFINITY ? m : fmaf(m, sc, -C::SHIFT), l);
      if (here) {
        if (live) {
          const int64_t tok = it.first + tl.tok + my_tok;
          const int hq = it.h * a.g + min(r, tl.rows - 1) - my_tok * a.g;
          IO* o = static_cast<IO*>(a.o) + tok * a.o_token + hq * a.o_head;
          float top = own.x, sum = l;
          auto part = [&](int q) { return q == (int)blockIdx.x ? own : __ldcg(g_ml + (size_t)PgWalk::slot(q, it.c0) * R + row); };
          if (parts > 1) {
            top = -INFINITY;
            for (int q = it.c0; q <= it.c1; ++q)
              if (part(q).y != 0.0f) top = fmaxf(top, part(q).x);
            sum = 0.0f;
            for (int q = it.c0; q <= it.c1; ++q)
              if (part(q).y != 0.0f) sum = fmaf(part(q).y, ta_ex2(part(q).x - top), sum);
          }
          const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll 1
          for (int c = 0; c < DP && c < a.D; c += 32) {
            __syncwarp();  // (TMEM is read by whole warps)
            float v[32];
            if (any) {
              tc::tmem_ld16(t_o + c, *reinterpret_cast<float(*)[16]>(v));
              tc::tmem_ld16(t_o + c + 16, *reinterpret_cast<float(*)[16]>(v + 16));
              tc::tmem_ld_wait();
              tc::reg_fence(v);
            }
            if (parts > 1) {
              float acc[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) acc[e] = 0.0f;
#pragma unroll 1
              for (int q = it.c0; q <= it.c1; ++q) {
                const float2 x = part(q);
                if (x.y == 0.0f) continue;  // saw nothing: its sums were not written
                const float f = ta_ex2(x.x - top);
                if (q == (int)blockIdx.x) {
#pragma unroll
                  for (int e = 0; e < 32; ++e) acc[e] = fmaf(v[e], f, acc[e]);
                } else {
                  const float* po = g_o + ((size_t)PgWalk::slot(q, it.c0) * DP + c) * R + row;
                  float u[32];
#pragma unroll
                  for (int e = 0; e < 32; ++e) u[e] = __ldcg(po + e * R);
#pragma unroll
                  for (int e = 0; e < 32; ++e) acc[e] = fmaf(u[e], f, acc[e]);
                }
              }
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = acc[e];
            }
            if constexpr (F32) {
              if (mine)
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                  if (c + e < a.D)
                    *reinterpret_cast<float4*>(o + c + e) = sum == 0.0f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                                                        : make_float4(v[e] * inv, v[e + 1] * inv, v[e + 2] * inv, v[e + 3] * inv);
            } else {
              uint32_t u[16];
#pragma unroll
              for (int e = 0; e < 16; ++e)
                u[e] = sum == 0.0f ? 0u : ta_pack(v[2 * e] * inv, v[2 * e + 1] * inv);
              if (mine) {
                if (a.o_32) {  // whole 32-byte sectors a store: half as many passes through L1
                  ta_store32(o + c, u);
                  if (c + 16 < a.D) ta_store32(o + c + 16, u + 8);
                } else {
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    if (c + 8 * e < a.D)
                      *reinterpret_cast<uint4*>(o + c + 8 * e) =
                          make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
                }
              }
            }
          }
          if (mine && a.lse)
            a.lse[tok * a.Hq + hq] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
        }
        if (any) {
          tc::tc_fence_before();
          __syncwarp();
          if (!F32 && lane == 0) tc::mbar_arrive(&o_empty[t]);
        }
      } else {
        // a part: maxima, sums and unscaled O to the workspace; the last CTA of the item joins them
        if (live) {
          if (mine) const_cast<float2*>(g_ml)[(size_t)it.slot * R + row] = own;
          if (any) {
            float* po = const_cast<float*>(g_o) + (size_t)it.slot * DP * R + row;
#pragma unroll 1
            for (int c = 0; c < DP; c += 32) {
              __syncwarp();
              float v[32];
              tc::tmem_ld16(t_o + c, *reinterpret_cast<float(*)[16]>(v));
              tc::tmem_ld16(t_o + c + 16, *reinterpret_cast<float(*)[16]>(v + 16));
              tc::tmem_ld_wait();
              tc::reg_fence(v);
              if (mine)
#pragma unroll
                for (int e = 0; e < 32; ++e) po[(size_t)(c + e) * R] = v[e];
            }
          }
        }
        if (any) tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (any && !F32) tc::mbar_arrive(&o_empty[t]);
          tc::mbar_arrive(j_full);
        }
        if (warp == 0) {
          ok = ctl.wait(j_full, nj & 1);
          if (!ok) break;
          if (lane == 0) {
            __threadfence();  // cumulative: the other threads' parts, ordered before by the barrier
            uint32_t* cnt = reinterpret_cast<uint32_t*>(a.ws + 256) + it.c0;
            const bool last = atomicAdd(cnt, 1u) == (uint32_t)(it.c1 - it.c0);
            if (last) *cnt = 0u;  // as it was found: zero between calls
            *reinterpret_cast<volatile uint32_t*>(s_last) = last;
            tc::mbar_arrive(j_go);
          }
          __syncwarp();
        }
        ok = ctl.wait(j_go, nj & 1);
        if (!ok) break;
        ++nj;
        if (*reinterpret_cast<volatile uint32_t*>(s_last)) {
          __threadfence();
          ta_join<DP, IO, NT>(a, it, tb1, tid);
        }
      }
      done_item();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    if (role == 3) {
      // ------------------------------------------------------------ walk, and queries
      uint32_t n[NT] = {};  // query loads
      bool more = w.enter(a, start);
      const uint32_t bytes = C::SLABS * tb1 * a.g * 128;
      for (bool ok = true; ok;) {
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
        ++ni;
        if (!more) break;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const TaTile tl = ta_tile(a, x, t, tb1);
          if (tl.jb == tl.ja || !ok) continue;
          ok = ctl.wait(&q_empty[t], (n[t] & 1) ^ 1);
          if (ok) {
            if (lane == 0) {
              tc::mbar_expect_tx(&q_full[t], bytes);
              for (int s = 0; s < C::SLABS; ++s)
                tc::tma_load_3d(s_q + (t * C::SLABS + s) * TA_SLAB, &tm_q, &q_full[t], s * (F32 ? 32 : 64), x.h * a.g,
                                x.first + tl.tok);
            }
            ++n[t];
          }
          __syncwarp();
        }
        more = w.next(a);
      }
      if (lane == 0)
        for (int t = 0; t < NT; ++t) s_issued[t] = n[t];
    } else if (role == 0 || role == 2) {
      // ------------------------------------------------------------ queries to f16, each lane whole rows
      const int t = NT == 2 ? role / 2 : 0, first = NT == 2 ? 0 : role * 32, rows = NT == 2 ? 128 : 64;
      uint32_t n = 0;  // items of this tile
      const TaItem* rec;
      bool ok = true;
      while (ok && (rec = next_item())) {
        const TaTile tl = ta_tile(a, *rec, t, tb1);
        done_item();
        if (tl.jb == tl.ja) continue;
        ok = ctl.wait(&q_full[t], n & 1) && ctl.wait(&f_empty[t], (n & 1) ^ 1);
        ++n;
        if (!ok) break;
#pragma unroll 1
        for (int r = first + lane; r < first + rows; r += 32) {
          uint8_t* row = s_q + (size_t)t * C::SLABS * TA_SLAB + r * 128;
          auto at = [&](int c) { return reinterpret_cast<uint4*>(row + c / 8 * TA_SLAB + ((c % 8 ^ (r & 7)) << 4)); };
          uint32_t top = 0;  // the largest, as a float's bits without the sign
#pragma unroll 4
          for (int c = 0; c < C::SLABS * 8; ++c) {
            const uint4 v = *at(c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t x = (&v.x)[e] & (F32 ? 0x7fffffffu : 0x7fff7fffu);
              top = max(top, F32 ? x : max(x << 16, x & 0xffff0000u));
            }
          }
          // the row's power of two, within what float32 holds; 1 where the row is not finite
          const int ex = top >= 0x7f800000u ? 14 : max((int)(top >> 23) - 127, -112);
          const float f = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
          if constexpr (F32) {
            // 64 columns: two slabs of float32 become one of f16 numbers and one of what is left of them
#pragma unroll 1
            for (int c0 = 0; c0 < C::SLABS * 8; c0 += 16) {
              uint32_t y[64];
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                const uint4 v = *at(c0 + c);
                const float x[4] = {__uint_as_float(v.x) * f, __uint_as_float(v.y) * f, __uint_as_float(v.z) * f, __uint_as_float(v.w) * f};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  y[2 * c + e] = tq_pack(x[2 * e], x[2 * e + 1]);
                  y[32 + 2 * c + e] = tq_rest(x[2 * e], x[2 * e + 1], y[2 * c + e]);
                }
              }
#pragma unroll
              for (int c = 0; c < 16; ++c) *at(c0 + c) = make_uint4(y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]);
            }
          } else {
#pragma unroll 4
            for (int c = 0; c < C::SLABS * 8; ++c) {
              uint4 v = *at(c);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t& x = (&v.x)[e];
                x = tq_pack(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f);
              }
              *at(c) = v;
            }
          }
          s_factor[t * 128 + r] =
              fminf(fmaxf(a.scale_log2 * __uint_as_float((uint32_t)max(ex - 14 + 127, 1) << 23), FLT_MIN), FLT_MAX);  // (0 times infinity is none)
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&q_ready[t]);
      }
    } else if (role == 1) {
      // ------------------------------------------------------------ MMA issuer: one thread
      // Products are issued as their operands come; a product of 128 x 128 x 16 takes the tensor
      // cores 64 cycles, so the thread must spend less than that on each: descriptors are one
      // base and constant offsets, waits are its own.
      if (tc::elect_one()) {
        constexpr uint32_t id_qk = tc::idesc_f16(128, TA_BN, 0, 0);
        constexpr uint32_t id_pv = tc::idesc_f16(128, C::COL, 0, 1);
        const uint64_t d_q = tc::smem_desc(tc::smem_u32(s_q), 16, 1024, tc::LAYOUT_SW128);
        const uint64_t d_k = tc::smem_desc(tc::smem_u32(s_ring), 16, 1024, tc::LAYOUT_SW128);
        const uint64_t d_v = tc::smem_desc(tc::smem_u32(s_ring), TA_SLAB, 1024, tc::LAYOUT_SW128);
        uint32_t st = 0, ph = 0;            // next ring unit, parity of its `full`
        uint32_t nq[NT] = {}, no[NT] = {};  // items of tile t so far: queries taken, O begun (float32: products of units)
        uint32_t cs[NT] = {}, cp[NT] = {};  // S of tile t issued, P taken
        bool ok = true;
        for (; ok; ++ni) {
          if (!ctl.wait1(&i_full[ni % TA_ITEMS], ni / TA_ITEMS & 1)) break;
          const TaItem& it = s_item[ni % TA_ITEMS];
          if (it.n < 0) break;
          const int j0 = it.j0, j1 = it.j1;
          TaTile tl[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) tl[t] = ta_tile(a, it, t, tb1);
          tc::mbar_arrive(&i_empty[ni % TA_ITEMS]);
          // step j: the products P V of key tile j - 1 and Q K^T of key tile j (in the order in
          // which the loader fills the ring)
          for (int j = j0; j <= j1 && ok && j0 < j1; ++j) {
            uint32_t v_st[C::UNITS], k_st[C::UNITS], v_par[C::UNITS], k_par[C::UNITS];
            bool v_in = false, k_in = false;
            // (NT = 1: the units' arrival is waited for where they are used, one by one)
            auto take = [&](uint32_t (&at)[C::UNITS], uint32_t (&par)[C::UNITS]) {
#pragma unroll
              for (int u = 0; u < C::UNITS; ++u) {
                at[u] = st;
                par[u] = ph;
                if (NT == 2) ok = ok && ctl.wait1(&full[st], ph);
                if (++st == C::STAGES) {
                  st = 0;
                  ph ^= 1;
                }
              }
            };
            auto take_v = [&] {
              if (v_in) return;
              take(v_st, v_par);
              v_in = true;
            };
            auto take_k = [&] {
              if (!k_in) take(k_st, k_par);
              k_in = true;
            };
            auto qk = [&](int t) {
              take_k();
              if (j == tl[t].ja) ok = ok && ctl.wait1(&q_ready[t], nq[t]++ & 1);
              if (!ok) return;
              const uint32_t b = NT == 2 ? t : C::S_BUF == 1 ? 0 : cs[t] & 1;
              ++cs[t];
              tc::tc_fence_after();
#pragma unroll
              for (int u = 0; u < C::UNITS; ++u) {
                if (NT == 1) {
                  ok = ctl.wait1(&full[k_st[u]], k_par[u]);
                  if (!ok) return;
                  tc::tc_fence_after();
                }
                // (the small halves first: a product is cut to the bits of the sum that it meets)
#pragma unroll
                for (int x = C::NUM - 1; x >= 0; --x)
#pragma unroll
                  for (int k = 0; k < C::COL / 16; ++k)
                    tc::mma_bf16(tmem + C::S_COL + b * 128,
                                 d_q + (((t * C::SLABS + (u * C::COL / 64 + k / 4) * C::NUM + x) * TA_SLAB + k % 4 * 32) >> 4),
                                 d_k + ((k_st[u] * C::UB + k / 4 * TA_SLAB + k % 4 * 32) >> 4), id_qk, u > 0 || x < C::NUM - 1 || k > 0);
                if (NT == 1) tc::mma_commit(&empty[k_st[u]]);  // a unit is free once read
              }
              tc::mma_commit(&s_full[b]);
              if (j == tl[t].jb - 1) tc::mma_commit(&q_empty[t]);
            };
            auto pv = [&](int t) {
              take_v();
              const uint32_t b = NT == 2 ? t : C::S_BUF == 1 ? 0 : cp[t] & 1;
              ok = ok && ctl.wait1(&p_full[b], (NT == 2 || C::S_BUF == 1 ? cp[t] : cp[t] >> 1) & 1);
              ++cp[t];
              if (!F32 && j - 1 == tl[t].ja) ok = ok && ctl.wait1(&o_empty[t], (no[t]++ & 1) ^ 1);
              if (!ok) return;
              tc::tc_fence_after();
              const uint32_t more = j - 1 > tl[t].ja;
#pragma unroll
              for (int u = 0; u < C::UNITS; ++u) {
                if (NT == 1) {
                  ok = ctl.wait1(&full[v_st[u]], v_par[u]);
                  if (F32) ok = ok && ctl.wait1(&o_empty[t], (no[t]++ & 1) ^ 1);
                  if (!ok) return;
                  tc::tc_fence_after();
                }
#pragma unroll
                for (int x = C::NUM - 1; x >= 0; --x)
#pragma unroll
                  for (int k = 0; k < TA_BN / 16; ++k)
                    tc::mma_ts(tmem + (F32 ? C::STEP_COL : C::O_COL + t * DP + u * C::COL), tmem + C::S_COL + b * 128 + x * 64 + k * 8,
                               d_v + ((v_st[u] * C::UB + k * 2048) >> 4), id_pv, x < C::NUM - 1 || k > 0 ? 1u : F32 ? 0u : more);
                if (NT == 1) tc::mma_commit(&empty[v_st[u]]);
                if (F32) tc::mma_commit(&pv_done[t]);
              }
              if (!F32) tc::mma_commit(&pv_done[t]);
            };
            if (NT == 1) {
              if (C::S_BUF == 1 && j > j0) pv(0);
              if (j < j1 && ok) qk(0);
              if (C::S_BUF == 2 && j > j0 && ok) pv(0);
            } else {
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                if (ok && j > tl[t].ja && j <= tl[t].jb) pv(t);
                if (ok && t == NT - 1 && v_in) tc::mma_commit(&empty[v_st[0]]);  // the values' last use
                if (ok && j >= tl[t].ja && j < tl[t].jb) qk(t);
              }
            }
            // two row tiles: what neither used is passed over, so that the ring stays in step
            if (NT == 2 && ok && j > j0 && !v_in) {
              take_v();
              if (ok) tc::mma_commit(&empty[v_st[0]]);
            }
            if (NT == 2 && ok && j < j1) {
              take_k();
              if (ok) tc::mma_commit(&empty[k_st[0]]);
            }
          }
        }
        tc::mma_commit(drain);  // arrives when all MMAs are done
      }
    } else {
      // ------------------------------------------------------------ keys and values, a row a thread
      const int r = tid & 127, g = role / 4 - 1;
      uint32_t o[4];  // where the row's 16-byte pieces lie
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] = (c ^ (r & 7)) << 4;
      TqStream<C, C::GROUPS, NT == 2 || C::S_BUF == 1 ? 2 : 3> str{a, cache, ctl, s_item, i_full, i_empty, s_copy + g * C::DEPTH * C::SB, (uint32_t)g};
      uint32_t rb = g, par = 1;
      while (str.issue()) {
        if (__builtin_expect(!str.come(), 0)) continue;
        if (!ctl.wait(&empty[rb], par)) break;
        uint8_t* line = s_ring + rb * C::UB + r * 128;
        tq_row<C>(str.ring + str.stage, r, [&](int p, const uint32_t (&y)[16]) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(line + p / 2 * TA_SLAB + (o[c] ^ (p & 1) << 6)) = make_uint4(y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]);
        });
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&full[rb]);
        rb += C::GROUPS;
        if (rb >= C::STAGES) {
          rb -= C::STAGES;
          par ^= 1;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");  // none is in flight when the CTA leaves
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (*s_flag && tid < 32) {
    // a wait ran out: copies and products in flight end (or run out too) before the CTA leaves
    for (int t = 0; t < NT; ++t)
      if (s_issued[t]) tc::mbar_wait(&q_full[t], (s_issued[t] - 1) & 1, a.wait_ns);
    tc::mbar_wait(drain, 0, a.wait_ns);
  }
  __syncthreads();
  if (warp == C::SOFT / 32 + 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int DP, bool F32, int NT>
cudaError_t run(PagedArgs& a, const Q4Cache& c, cudaStream_t s, int sms) {
  using C = Tm<DP, F32, NT>;
  const int tb1 = std::max(1, 128 / a.g);
  CUtensorMap mq;
  const uint64_t dq[3] = {(uint64_t)a.D, (uint64_t)a.Hq, (uint64_t)a.T};
  constexpr uint64_t size = F32 ? 4 : 2;
  const uint64_t sq[2] = {(uint64_t)a.q_head * size, (uint64_t)a.q_token * size};
  const uint32_t bq[3] = {F32 ? 32 : 64, (uint32_t)a.g, (uint32_t)tb1};
  cudaError_t e = encode_tmap(&mq, F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.q, dq, sq, bq, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  const void* f = reinterpret_cast<const void*>(k_paged_attn_q4_tc<DP, F32, NT>);
  static std::atomic<uint64_t> ready{0};
  // the register split draws on what the launch gives
  e = ta_prepare(f, C::smem, C::REGS, ready);
  if (e != cudaSuccess) return e;
  const PagedWs L = paged_ws(sms, C::NT * 128, DP);
  a.part_ml = L.ml;
  a.part_o = L.o;
  a.rows = C::NT * 128;
  a.tb = C::NT * tb1;
  a.o_32 = reinterpret_cast<uintptr_t>(a.o) % 32 == 0 && a.o_token % 16 == 0 && a.o_head % 16 == 0 && a.D % 16 == 0;
  // (an item's own cost 256 to 1536 keys, its least part, what a part is a multiple of: within 5 % from 384 to 768)
  pg_division(a, sms, C::NT == 2 ? 512 : 256, 896, C::NT == 2 ? 512 : 384);
  Q4Cache cache = c;
  cache.s_whole = q4_whole_scales(a, c);
  void* args[] = {&mq, &a, &cache};
  return launch_pdl(f, dim3(sms), dim3(C::THREADS), C::smem, s, args, 1);
}

// Row tiles of a CTA.  Measured (bf16, one against two): heads of 128, mean rows of a request 48 98 and 145 us, 717 104 and
// 116, 1024 155 and 156, 5200 135 and 129, 8192 1919 and 1822; heads of 64, 358 98 and 99, 1536 189 and 159, 8192 845 and 694.
int row_tiles(bool f32, int D, int rows) { return !f32 && D <= 128 && rows > 1024 ? 2 : 1; }

}  // namespace

cudaError_t launch_paged_attn_q4_tc(PagedArgs a, const Q4Cache& c, bool f32, int rows, cudaStream_t s) {
  const int sms = sm_count();
  if (sms < 1 || sms > PG_MAX_CTAS) return cudaErrorNotSupported;
  const bool two = row_tiles(f32, a.D, rows) == 2;
  switch (ta_width(a.D)) {
    case 64: return f32 ? run<64, true, 1>(a, c, s, sms) : two ? run<64, false, 2>(a, c, s, sms) : run<64, false, 1>(a, c, s, sms);
    case 128: return f32 ? run<128, true, 1>(a, c, s, sms) : two ? run<128, false, 2>(a, c, s, sms) : run<128, false, 1>(a, c, s, sms);
    default: return f32 ? run<256, true, 1>(a, c, s, sms) : run<256, false, 1>(a, c, s, sms);
  }
}

size_t paged_attn_q4_tc_ws_bytes(const paged_shape* s, int rows) {
  const int sms = sm_count();
  return paged_ws(sms > 0 ? sms : 256, row_tiles(s->io == RGLRU_F32, s->D, rows) * 128, ta_width(s->D)).total;
}

}  // namespace rglru

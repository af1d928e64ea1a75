// Attention over the paged cache on the tensor cores (bf16 I/O), many rows a request: tcgen05
// MMAs with accumulators and softmax weights in TMEM, operands by TMA.
//
// One pass over the keys with a running maximum and sum.  Per row tile (up to 128 rows: whole
// tokens x the g query heads of one key/value head) and per tile of 128 keys
//   S = Q K^T               Q, K from shared memory, S in TMEM, float32
//   P = 2^(c S - c m)       c = scale log2 e; one thread a row, P back to TMEM as bf16
//   O += P V                P from TMEM, V from shared memory, O in TMEM, float32
// with l the float32 sum of P before its rounding to bf16.  The rounding of P (8-bit significand,
// relative 2^-8 at most, as V's own storage) is what lets the second product run on the tensor
// cores; sums and statistics stay in float32.  m is moved only when a row's maximum has grown by
// more than 2^8 in weight (O and l are then scaled): weights up to 2^8 keep bf16's relative
// precision, and the rescaling of O, a round trip through TMEM, becomes rare.
//
// Width D <= 128: two row tiles a CTA share every key tile and alternate on the tensor cores, so
// that one's softmax runs behind the other's products (TMEM: two S/P of 128 columns, two O of
// D: full).  D <= 256: one row tile, two S buffers, the next tile's S computed behind this one's
// softmax.  Warps: 4 softmax warps a row tile, then key/value loader, MMA issuer (one thread), one
// that clears rows of V, and one that walks the CTA's items and loads queries.
//
// Pages: a key tile is copied page by page, one box of rows per page and 64 columns (128-byte
// swizzle).  A page that the tile does not need, or whose table entry is outside the cache,
// is copied from outside the tensor map, which gives zeros: the byte count of a stage is
// always the same, and nothing outside the cache is read.  Rows of V past the request's keys
// (or before its window) are cleared in shared memory, so that stale or non-finite cache
// contents cannot reach a product with a zero weight; scores of such keys are replaced.
//
// Work is divided over the CTAs by weight (paged.cuh): one CTA per SM, each with a list of
// items of which the first and the last may be shared with its neighbours.
//
// Measured (GB300): two prompts of 8192 tokens, 16 query heads on 4 of 128, 550 GFLOP: 390 us,
// 1.41 PFLOP/s (the tensor pipe 59 % of its cycles).  What bounds it: a 128 x 128 x 16 product
// takes the pipe 64 cycles, and Q K^T, both operands from shared memory, takes shared memory's
// whole 128 bytes a cycle meanwhile, so the key tiles' arrival delays it; a tile's softmax (1200
// cycles) and the latencies of its hand-overs are a little longer than the other tile's products
// (1024).  Without any softmax the same call takes 334 us.  Heads of 256 (S two tiles ahead):
// 1.50 PFLOP/s.  Heads of 64: 0.87 PFLOP/s, bound by the softmax (154 us of 235 without it).  Not
// faster: weights handed over in halves, and taken at the last maximum beside the new one.
#include <algorithm>

#include "host_util.h"
#include "paged_tc.cuh"

namespace rglru {

namespace {

template <int DP, bool W>
struct Ta {
  static constexpr bool WIDE = W;                     // TaLay
  static constexpr int NT = DP == 256 ? 1 : 2;        // row tiles
  static constexpr int SLABS = DP / 64;
  static constexpr int UPT = DP == 256 ? 2 : 1;       // ring units of a key (or value) tile
  static constexpr uint32_t UB = DP == 64 ? TA_SLAB : 2 * TA_SLAB;
  static constexpr int STAGES = DP == 64 ? 10 : 5;
  static constexpr int VROWS = TA_BN / UPT;           // rows of V in a unit
  static constexpr int SOFT = NT * 128;               // softmax threads
  static constexpr int THREADS = SOFT + 128;
  static constexpr uint32_t S_COL = 0, O_COL = 256;   // TMEM: S/P buffers b at 128 b, O tiles
  static constexpr size_t Q_BYTES = (size_t)NT * SLABS * TA_SLAB;
  static constexpr size_t smem = 1024 + Q_BYTES + STAGES * UB + 768;
};

constexpr int TA_HERE = 4;  // parts that are joined without handing over the last one

// Row tile t of an item and its key tiles within the CTA's part.
struct TaTile {
  int tok, rows, ja, jb;
};
__device__ __forceinline__ TaTile ta_tile(const PagedArgs& a, const TaItem& it, int t, int tb1) {
  TaTile x;
  x.tok = it.tok + t * tb1;
  const int nt = min(tb1, it.q - x.tok);
  x.rows = max(nt, 0) * a.g;
  const int base = it.kv - it.q + x.tok;
  const int hi = max(base + nt, 0);
  const int lo = a.window && base >= a.window ? base - a.window + 1 : 0;
  x.ja = max(it.j0, lo / TA_BN);
  x.jb = min(it.j1, (hi + TA_BN - 1) / TA_BN);
  if (x.rows == 0 || x.jb < x.ja) x.jb = x.ja;
  return x;
}

__device__ __forceinline__ void ta_store32(bf16* p, const uint32_t* u) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]),
               "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}

// Bits 0 to h, none for a negative h.
__device__ __forceinline__ uint32_t ta_bits(int h) { return h < 0 ? 0u : h >= 31 ? ~0u : (2u << h) - 1; }

// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void ta_mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}

// One row's results joined over the CTAs [c0, c1] of an item, by all softmax threads: a thread
// takes one row and a run of columns.
template <int DP>
__device__ __noinline__ void ta_join(const PagedArgs& a, const TaItem& it, int tb1, int tid) {
  const int c0 = it.c0, c1 = it.c1;
  using C = Ta<DP, false>;
  const float2* ml = reinterpret_cast<const float2*>(a.ws + a.part_ml);
  const float* po = reinterpret_cast<const float*>(a.ws + a.part_o);
  const int R = C::NT * 128;
  // rows in use: of tile 0, and past 128 of tile 1
  const int n1 = min(it.q - it.tok, tb1) * a.g;
  const int n2 = C::NT == 2 ? max(min(it.q - it.tok - tb1, tb1), 0) * a.g : 0;
  const int used = n2 > 0 ? 128 + n2 : n1;
  int rp = C::SOFT * 16 / DP;
  while (rp < used) rp <<= 1;
  const int groups = C::SOFT / rp, cols = DP / groups;
  const int row = tid & (rp - 1), col0 = tid / rp * cols;
  if (row >= used || (row < 128 && row >= n1)) return;
  float m = -INFINITY;
  for (int c = c0; c <= c1; ++c) {
    const float2 x = __ldcg(ml + (size_t)PgWalk::slot(c, c0) * R + row);
    if (x.y != 0.0f) m = fmaxf(m, x.x);
  }
  float l = 0.0f;
  for (int c = c0; c <= c1; ++c) {
    const float2 x = __ldcg(ml + (size_t)PgWalk::slot(c, c0) * R + row);
    if (x.y != 0.0f) l = fmaf(x.y, ta_ex2(x.x - m), l);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int t = row >> 7, r = row & 127;
  const int64_t tok = it.first + it.tok + t * tb1 + pg_token(a, r);
  const int hq = it.h * a.g + r - pg_token(a, r) * a.g;
  bf16* o = static_cast<bf16*>(a.o) + tok * a.o_token + hq * a.o_head;
  constexpr int W = 16;  // columns at a time: with two parts, 32 loads in flight
#pragma unroll 1
  for (int k = col0; k < col0 + cols && k < a.D; k += W) {
    float acc[W];
#pragma unroll
    for (int e = 0; e < W; ++e) acc[e] = 0.0f;
#pragma unroll 2
    for (int c = c0; c <= c1; ++c) {
      const size_t s = (size_t)PgWalk::slot(c, c0);
      const float2 x = __ldcg(ml + s * R + row);
      float v[W];
#pragma unroll
      for (int e = 0; e < W; ++e) v[e] = __ldcg(po + (s * DP + k + e) * R + row);
      const float f = x.y == 0.0f ? 0.0f : ta_ex2(x.x - m);  // a part that saw nothing did not write its sums
#pragma unroll
      for (int e = 0; e < W; ++e) acc[e] = f != 0.0f ? fmaf(v[e], f, acc[e]) : acc[e];
    }
#pragma unroll
    for (int e = 0; e < W; e += 8)
      if (k + e < a.D && k + e < col0 + cols)
        *reinterpret_cast<uint4*>(o + k + e) =
            make_uint4(ta_pack(acc[e] * inv, acc[e + 1] * inv), ta_pack(acc[e + 2] * inv, acc[e + 3] * inv),
                       ta_pack(acc[e + 4] * inv, acc[e + 5] * inv), ta_pack(acc[e + 6] * inv, acc[e + 7] * inv));
  }
  if (a.lse && col0 == 0)
    a.lse[tok * a.Hq + hq] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

template <int DP, bool W>
__global__ void __launch_bounds__(Ta<DP, W>::THREADS, 1)
    k_paged_attn(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedArgs a) {
  using C = Ta<DP, W>;
  constexpr int NT = C::NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* s_q = smem;
  uint8_t* s_ring = s_q + C::Q_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_ring + C::STAGES * C::UB);
  uint64_t* empty = full + C::STAGES;
  uint64_t* q_full = empty + C::STAGES;  // [NT]
  uint64_t* q_empty = q_full + NT;       // [NT]
  uint64_t* s_full = q_empty + NT;       // [2]  S of buffer b complete
  uint64_t* p_full = s_full + 2;         // [2]  P of buffer b written (and O scaled)
  uint64_t* pv_done = p_full + 2;        // [NT] a product P V of tile t complete
  uint64_t* o_empty = pv_done + NT;      // [NT] O of tile t read
  uint64_t* j_full = o_empty + NT;       // a part of an item is in the workspace
  uint64_t* j_go = j_full + 1;           // s_last says whether this CTA joins the item
  uint64_t* j_here = j_go + 1;           // [TA_ITEMS] s_here says whether this CTA has the last part
  uint64_t* i_full = j_here + TA_ITEMS;           // [TA_ITEMS] item records
  uint64_t* i_empty = i_full + TA_ITEMS;
  uint64_t* v_come = i_empty + TA_ITEMS;  // [TA_CLEARS] a value tile to clear is on its way
  uint64_t* v_clean = v_come + TA_CLEARS; // [TA_CLEARS] it is cleared
  uint64_t* drain = v_clean + TA_CLEARS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  uint32_t* s_flag = tmem_holder + 1;
  uint32_t* s_last = tmem_holder + 2;
  __shared__ int64_t scratch[33];
  __shared__ TaItem s_item[TA_ITEMS];
  __shared__ TaClear s_clear[TA_CLEARS];
  __shared__ uint32_t s_here[TA_ITEMS];
  __shared__ uint32_t s_issued[NT + 1];  // loads issued: queries of each tile, ring units
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tb1 = max(1, 128 / a.g);  // tokens of a row tile
  const TaAbort ctl{s_flag, reinterpret_cast<uint32_t*>(a.ws), a.wait_ns};

  // up to griddep_wait nothing touches global memory
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NT; ++i) {
      tc::mbar_init(&q_full[i], 1);
      tc::mbar_init(&q_empty[i], 1);
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
      tc::mbar_init(&i_empty[i], C::SOFT / 32 + 2);
    }
    for (int i = 0; i < TA_CLEARS; ++i) {
      tc::mbar_init(&v_come[i], 1);
      tc::mbar_init(&v_clean[i], 1);
    }
    tc::mbar_init(drain, 1);
    for (int i = 0; i <= NT; ++i) s_issued[i] = 0u;
    *s_flag = 0u;
    tc::fence_barrier_init();
    tc::prefetch_tmap(&tm_q);
    tc::prefetch_tmap(&tm_k);
    tc::prefetch_tmap(&tm_v);
  }
  if (warp == C::SOFT / 32 + 1) {
    tc::tmem_alloc(tmem_holder, 512);
    tc::tmem_relinquish();
  }
  const int role = warp - C::SOFT / 32;  // < 0: softmax; 0: keys and values, 1: MMA, 2: clearing, 3: walk and queries
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
  // Registers: 384 threads x 168 at launch = 256 x 208 + 128 x 88 after the two warpgroups of
  // softmax have taken what the other one gives up.
  if (role < 0) {
    if (NT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------------------ softmax, one row a thread
    const int t = NT == 2 ? warp >> 2 : 0, wq = warp & 3, r = wq * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t t_o = lanes + C::O_COL + t * DP;
    const float sc = a.scale_log2;
    uint32_t cs = 0, npv = 0, nj = 0;  // S taken, products P V of this tile, parts handed over
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
      for (int j = tl.ja; j < tl.jb; ++j) {
        const int b = NT == 2 ? t : cs & 1;
        ok = ctl.wait(&s_full[b], (NT == 2 ? cs : cs >> 1) & 1);
        ++cs;
        if (!ok) break;
        tc::tc_fence_after();
        bool waited = j == tl.ja;  // NT = 1: for the product before this one
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
          } else if (__any_sync(0xffffffffu, r < tl.rows && (top - m) * sc > 8.0f)) {  // (of rows in use)
            const float f = top == m ? 1.0f : ta_ex2((top - m) * -sc);
            l *= f;
            m = top;
            if (NT == 1) {
              ok = ctl.wait(&pv_done[0], (npv + (j - tl.ja) - 1) & 1);
              waited = true;
              if (!ok) break;
              tc::tc_fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < DP; c += 16) {
              float o[16];
              tc::tmem_ld16(t_o + c, o);
              tc::tmem_ld_wait();
              tc::reg_fence(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= f;
              tc::tmem_st16(t_o + c, o);
            }
          }
          const float off = m == -INFINITY ? 0.0f : -m * sc;
          float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            float pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 x = ta_fma2(make_float2(s[c + 2 * e], s[c + 2 * e + 1]), make_float2(sc, sc),
                                       make_float2(off, off));
              const float2 p = make_float2(ta_ex2(x.x), ta_ex2(x.y));
              sum[e & 1] = ta_add2(sum[e & 1], p);
              pk[e] = __uint_as_float(ta_pack(p.x, p.y));
            }
            tc::tmem_st16(t_s + c / 2, pk);
          }
          const float2 s2 = ta_add2(sum[0], sum[1]);
          l += s2.x + s2.y;
          tc::tmem_st_wait();
        }
        if (NT == 1 && !waited) {
          ok = ctl.wait(&pv_done[0], (npv + (j - tl.ja) - 1) & 1);
          if (!ok) break;
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&p_full[b]);
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
        npv += tl.jb - tl.ja;
        ok = ctl.wait(&pv_done[t], (npv - 1) & 1);
        if (!ok) break;
        tc::tc_fence_after();
      }
      const bool mine = r < tl.rows;
      const int row = t * 128 + r;
      constexpr int R = NT * 128;
      const float2* g_ml = reinterpret_cast<const float2*>(a.ws + a.part_ml);
      const float* g_o = reinterpret_cast<const float*>(a.ws + a.part_o);
      // (rounded here as in memory, whichever of the two it is joined from)
      const float2 own = make_float2(m == -INFINITY ? m : __fmul_rn(m, sc), l);
      if (here) {
        if (live) {
          const int64_t tok = it.first + tl.tok + my_tok;
          const int hq = it.h * a.g + min(r, tl.rows - 1) - my_tok * a.g;
          bf16* o = static_cast<bf16*>(a.o) + tok * a.o_token + hq * a.o_head;
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
          if (mine && a.lse)
            a.lse[tok * a.Hq + hq] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
        }
        if (any) {
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&o_empty[t]);
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
          if (any) tc::mbar_arrive(&o_empty[t]);
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
          ta_join<DP>(a, it, tb1, tid);
        }
      }
      done_item();
    }
  } else {
    if (NT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
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
                tc::tma_load_3d(s_q + (t * C::SLABS + s) * TA_SLAB, &tm_q, &q_full[t], s * 64, x.h * a.g,
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
    } else if (role == 0) {
      // ------------------------------------------------------------ key / value loader
      TaLoader<C> ld{a, ctl, s_ring, full, empty, s_clear, v_come};
      const TaItem* rec;
      bool ok = true;
      while (ok && (rec = next_item())) {
        const TaItem it = *rec;
        done_item();
        const int j0 = it.j0, j1 = it.j1;
        int id_prev = a.P, id = ld.page_of(it, j0);
        for (int j = j0; j <= j1 && ok && j0 < j1; ++j) {
          const int id_next = ld.page_of(it, j + 1);
          if (NT == 1 && j < j1) ok = ld.keys(&tm_k, j, id, it.h);
          if (j > j0) ok = ok && ld.values(&tm_v, j - 1, id_prev, it.h, it.lo, it.hi);
          if (NT == 2 && j < j1) ok = ok && ld.keys(&tm_k, j, id, it.h);
          id_prev = id;
          id = id_next;
        }
      }
      ld.end();
      if (lane == 0) s_issued[NT] = ld.issued;
    } else if (role == 1) {
      // ------------------------------------------------------------ MMA issuer: one thread
      // Products are issued as their operands come; a product of 128 x 128 x 16 takes the tensor
      // cores 64 cycles, so the thread must spend less than that on each: descriptors are one
      // base and constant offsets, waits are its own.
      if (tc::elect_one()) {
        constexpr uint32_t id_qk = tc::idesc_bf16(128, TA_BN, 0, 0);
        constexpr uint32_t id_pv = tc::idesc_bf16(128, DP, 0, 1);
        const uint64_t d_q = tc::smem_desc(tc::smem_u32(s_q), 16, 1024, tc::LAYOUT_SW128);
        const TaLay<C> lay(a);
        const uint64_t d_k = tc::smem_desc(tc::smem_u32(s_ring), 16, TaLay<C>::K_GROUP, tc::LAYOUT_SW128);
        const uint64_t d_v = tc::smem_desc(tc::smem_u32(s_ring), lay.v_slab(), lay.v_group(), tc::LAYOUT_SW128);
        uint32_t st = 0, ph = 0;            // next ring unit, parity of its `full`
        uint32_t nq[NT] = {}, no[NT] = {};  // items of tile t so far: queries taken, O begun
        uint32_t cs[NT] = {}, cp[NT] = {};  // S of tile t issued, P taken
        uint32_t nc = 0;                    // value tiles cleared
        bool ok = true;
        for (; ok; ++ni) {
          if (!ctl.wait1(&i_full[ni % TA_ITEMS], ni / TA_ITEMS & 1)) break;
          const TaItem& it = s_item[ni % TA_ITEMS];
          if (it.n < 0) break;
          const int j0 = it.j0, j1 = it.j1, k_lo = it.lo, k_hi = it.hi;
          TaTile tl[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) tl[t] = ta_tile(a, it, t, tb1);
          tc::mbar_arrive(&i_empty[ni % TA_ITEMS]);
          // step j: the products P V of key tile j - 1 and Q K^T of key tile j (in the order in
          // which the loader fills the ring)
          for (int j = j0; j <= j1 && ok && j0 < j1; ++j) {
            uint32_t v_st[C::UPT], k_st[C::UPT], v_par[C::UPT], k_par[C::UPT];
            bool v_in = false, k_in = false;
            // (NT = 1: the units' arrival is waited for where they are used, one by one)
            auto take = [&](uint32_t (&at)[C::UPT], uint32_t (&par)[C::UPT]) {
#pragma unroll
              for (int u = 0; u < C::UPT; ++u) {
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
              if (ta_cut(j - 1, k_lo, k_hi)) {
                ok = ok && ctl.wait1(&v_clean[nc % TA_CLEARS], nc / TA_CLEARS & 1);
                ++nc;
              }
            };
            auto take_k = [&] {
              if (!k_in) take(k_st, k_par);
              k_in = true;
            };
            auto qk = [&](int t) {
              take_k();
              if (j == tl[t].ja) ok = ok && ctl.wait1(&q_full[t], nq[t]++ & 1);
              if (!ok) return;
              const uint32_t b = NT == 2 ? t : cs[t] & 1;
              ++cs[t];
              tc::tc_fence_after();
#pragma unroll
              for (int k = 0; k < DP / 16; ++k) {
                if (NT == 1 && k % 8 == 0) {
                  ok = ctl.wait1(&full[k_st[k / 8]], k_par[k / 8]);
                  if (!ok) return;
                  tc::tc_fence_after();
                }
                tc::mma_bf16(tmem + C::S_COL + b * 128,
                             d_q + (((t * C::SLABS + k / 4) * TA_SLAB + k % 4 * 32) >> 4),
                             d_k + (k_st[k / 8] * (C::UB >> 4) + ((k % 8 / 4 * TaLay<C>::K_SLAB + k % 4 * 32) >> 4)),
                             id_qk, k > 0);
                if (NT == 1 && k % 8 == 7) tc::mma_commit(&empty[k_st[k / 8]]);  // a unit is free once read
              }
              tc::mma_commit(&s_full[b]);
              if (j == tl[t].jb - 1) tc::mma_commit(&q_empty[t]);
            };
            auto pv = [&](int t) {
              take_v();
              const uint32_t b = NT == 2 ? t : cp[t] & 1;
              ok = ok && ctl.wait1(&p_full[b], (NT == 2 ? cp[t] : cp[t] >> 1) & 1);
              ++cp[t];
              if (j - 1 == tl[t].ja) ok = ok && ctl.wait1(&o_empty[t], (no[t]++ & 1) ^ 1);
              if (!ok) return;
              tc::tc_fence_after();
              const uint32_t more = j - 1 > tl[t].ja;
#pragma unroll
              for (int k = 0; k < TA_BN / 16; ++k) {
                if (NT == 1 && k * 16 % C::VROWS == 0) {
                  ok = ctl.wait1(&full[v_st[k * 16 / C::VROWS]], v_par[k * 16 / C::VROWS]);
                  if (!ok) return;
                  tc::tc_fence_after();
                }
                ta_mma_ts(tmem + C::O_COL + t * DP, tmem + C::S_COL + b * 128 + k * 8,
                          d_v + (v_st[k * 16 / C::VROWS] * (C::UB >> 4) + (k % (C::VROWS / 16) * TaLay<C>::V_16 >> 4)),
                          id_pv, k > 0 ? 1u : more);
                if (NT == 1 && (k + 1) * 16 % C::VROWS == 0) tc::mma_commit(&empty[v_st[k * 16 / C::VROWS]]);
              }
              tc::mma_commit(&pv_done[t]);
            };
            if (NT == 1) {
              if (j < j1) qk(0);
              if (j > j0 && ok) pv(0);
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
    } else if (role == 2) {
      // ------------------------------------------------------------ rows of V that no row sees
      ta_clear_rows<C>(a, ctl, s_clear, v_come, v_clean, full, s_ring);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (*s_flag && tid < 32) {
    // a wait ran out: copies and products in flight end (or run out too) before the CTA leaves
    for (uint32_t i = lane; i < min(s_issued[NT], (uint32_t)C::STAGES); i += 32) {
      const uint32_t n = s_issued[NT] - 1 - i;
      tc::mbar_wait(&full[n % C::STAGES], n / C::STAGES & 1, a.wait_ns);
    }
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

template <int DP, bool W>
cudaError_t run(PagedArgs& a, cudaStream_t s, int sms) {
  using C = Ta<DP, W>;
  const int tb1 = std::max(1, 128 / a.g);
  CUtensorMap mq, mk, mv;
  cudaError_t e = ta_maps<C>(a, tb1, &mq, &mk, &mv);
  if (e != cudaSuccess) return e;
  const void* f = reinterpret_cast<const void*>(k_paged_attn<DP, W>);
  static std::atomic<uint64_t> ready{0};
  // the register split draws on what the launch gives
  e = ta_prepare(f, C::smem, C::NT == 2 ? (256 * 208 + 128 * 88) / C::THREADS : 0, ready);
  if (e != cudaSuccess) return e;
  const PagedWs L = paged_ws(sms, C::NT * 128, DP);
  a.part_ml = L.ml;
  a.part_o = L.o;
  a.rows = C::NT * 128;
  a.tb = C::NT * tb1;
  a.o_32 = reinterpret_cast<uintptr_t>(a.o) % 32 == 0 && a.o_token % 16 == 0 && a.o_head % 16 == 0 && a.D % 16 == 0;
  // the switch of an item costs two row tiles about 9000 cycles, three key tiles' time
  pg_division(a, sms, C::NT == 2 ? 384 : 256, 896, C::NT == 2 ? 768 : 384);
  void* args[] = {&mq, &mk, &mv, &a};
  return launch_pdl(f, dim3(sms), dim3(C::THREADS), C::smem, s, args, 1);
}

}  // namespace

cudaError_t launch_paged_attn_tc(PagedArgs a, cudaStream_t s) {
  const int sms = sm_count();
  if (sms < 1 || sms > PG_MAX_CTAS) return cudaErrorNotSupported;
  switch (ta_width(a.D)) {
    case 64: return run<64, false>(a, s, sms);
    case 128: return ta_wide(a) ? run<128, true>(a, s, sms) : run<128, false>(a, s, sms);
    default: return ta_wide(a) ? run<256, true>(a, s, sms) : run<256, false>(a, s, sms);
  }
}

size_t paged_attn_tc_ws_bytes(const paged_shape* s) {
  const int sms = sm_count(), dp = ta_width(s->D);
  return paged_ws(sms > 0 ? sms : 256, dp == 256 ? 128 : 256, dp).total;
}

}  // namespace rglru

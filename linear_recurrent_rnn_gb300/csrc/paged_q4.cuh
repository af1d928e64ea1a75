// Shared by the kernels of the cache held in 4 bits (include/paged_q4.h): its arrays, and the numbers
// that codes stand for.
#pragma once

#include <cuda_fp16.h>

#include "../../include/paged_q4.h"
#include "paged_tc.cuh"

namespace rglru {

// Codes and scales of keys and values; strides in bytes.
struct Q4Cache {
  const uint8_t* kc;
  const uint8_t* ks;
  const uint8_t* vc;
  const uint8_t* vs;
  int64_t kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;
  int64_t ks_page, ks_token, ks_head, vs_page, vs_token, vs_head;
  int s_whole;  // nothing of a row is cut off: its scales lie on boundaries of their size, D fills its columns, pages of 16 and more
  int split;  // heads of the attention's work division a key/value head
};

// The eight values of a word of codes, as four pairs of f16.
__device__ __forceinline__ void q4_pairs(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// Two neighbouring scales as a pair of f16.
__device__ __forceinline__ uint32_t q4_scales(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ uint32_t q4_mul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(reinterpret_cast<const __half2&>(a), reinterpret_cast<const __half2&>(b));
  return reinterpret_cast<const uint32_t&>(r);
}

// Bounded waits as TaAbort's, in less code: there are some forty, and five roles share the instruction
// cache of a quarter of the SM.
struct TqAbort {
  uint32_t* flag;    // shared: set once a wait has run out
  uint32_t* status;  // global
  uint32_t limit;    // of a wait, in units of 1024 ns
  __device__ __forceinline__ static uint32_t now() { return (uint32_t)(tc::global_ns() >> 10); }
  __device__ __forceinline__ bool over(uint32_t t0) const {
    if (!*reinterpret_cast<volatile uint32_t*>(flag) && now() - t0 <= limit) return false;
    *reinterpret_cast<volatile uint32_t*>(flag) = 1u;
    *reinterpret_cast<volatile uint32_t*>(status) = 1u;
    return true;
  }
  // By one thread.
  __device__ __forceinline__ bool wait1(uint64_t* bar, uint32_t parity) const {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const uint32_t t0 = now();
    while (!tc::mbar_try_wait_sleep(bar, parity, 20000u))
      if (over(t0)) return false;
    return true;
  }
  // By a converged warp; the answer is the same in all its lanes.
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait1(bar, parity));
  }
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
__device__ __forceinline__ void tq_copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void tq_copy4(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
// A row's scales, on a boundary of their size.
template <int N>
__device__ __forceinline__ void tq_copy_row(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "n"(N) : "memory");
}
// A row's 16-byte pieces of codes lie where neither the copies nor the dequantising threads, a row a thread,
// meet in a bank.
template <class C>
__device__ __forceinline__ uint32_t tq_code(int r, int piece) {
  const int x = C::RB == 128 ? r & 7 : C::RB == 64 ? r >> 1 & 3 : r >> 2 & 1;
  return r * C::RB + ((piece ^ x) << 4);
}

// The units of codes that a warpgroup brings: every G-th of the CTA's stream of keys (KIND 0) or of values
// (1), or all of both in the order in which a kernel uses them: the values of a tile after its keys (2), or
// after the next tile's (3).  Each of its warps copies its own 32 rows, waits for them and dequantises
// them, so that no other warp is asked: units in flight are the warp's own groups of cp.async, one an iteration
// (an empty one where there is no unit to copy).  A lane reads the page of its own row, an iteration before it is
// used.  What little state is kept matters: addresses of an item's head, worked out once and kept, cost 64 bits each of
// 64 registers and were slower than working them out for every unit (256 requests decoding 209 us, 197 without).
template <class C, int G, int KIND>
struct TqStream {
  static constexpr int CPR = C::RB / 16, RPI = 32 / CPR;  // 16-byte pieces of a row, rows of an instruction
  const PagedArgs& a;
  const Q4Cache& c;
  const TqAbort& ctl;
  const TaItem* items;
  uint64_t* i_full;
  uint64_t* i_empty;
  uint8_t* ring;  // this warpgroup's
  uint32_t g;     // which of the G it is
  uint32_t stage = 0;  // offset of the stage that is copied to next, and of the oldest copy
  uint32_t ni = 0, next = 0;  // item; number of its first unit
  int q = 0, part = 0, end = 0, j0 = 0, lo = 0, hi = 0;  // the place in the item's stream of what is copied next (q < end), its keys
  int pos = 0;                 // its first position of this warp's rows
  const int32_t* table = nullptr;  // the item's row of the table
  int h = 0;
  int mine = -1;               // the page of the lane's row (-1: zeros)
  bool more = true, ok = true; // there are items left
  uint32_t real = 0;           // a bit an iteration: a unit was copied (the last one: bit 0)

  // Whether values come at the place, and the tile.
  __device__ __forceinline__ bool values() const { return KIND == 1 || (KIND == 2 && (q & 1)) || (KIND == 3 && q > 0 && (!(q & 1) || q + 1 == end)); }
  __device__ __forceinline__ int tile() const {
    return j0 + (KIND < 2 ? q : KIND == 2 ? q >> 1 : !values() ? (q + 1) >> 1 : q + 1 == end ? (q >> 1) : (q >> 1) - 1);
  }
  // (read an iteration before they are used)
  __device__ __forceinline__ void page() {
    pos = tile() * TA_BN + (threadIdx.x & 96);
    const int at = pos + (threadIdx.x & 31);
    mine = -1;
    if ((q < end) & (at < hi) & (at >= lo)) mine = table[at >> a.ps_log2];
  }
  __device__ __forceinline__ void forward(uint32_t units) {
    if (C::UNITS == 1) {
      q += units;
    } else {
      part += units;
      q += part / C::UNITS;
      part %= C::UNITS;
    }
  }
  // The next item, if its record is there (or waiting for it); its first unit that is this group's.
  __device__ __forceinline__ void item(bool wait) {
    uint64_t* come = &i_full[ni % TA_ITEMS];
    const uint32_t par = ni / TA_ITEMS & 1;
    if (wait) {
      ok = ctl.wait(come, par);
      if (!ok) return;
    } else if (!__all_sync(0xffffffffu, tc::mbar_test(come, par))) {
      return;
    }
    const TaItem& it = items[ni % TA_ITEMS];
    more = it.n >= 0;
    if (!more) return;
    const int lane = threadIdx.x & 31;
    h = it.h / c.split;
    table = a.table + (int64_t)it.n * a.table_width;
    j0 = it.j0;
    q = 0;
    end = max(it.j1 - j0, 0) * (KIND < 2 ? 1 : 2);
    lo = it.lo;
    hi = (int)min((int64_t)it.hi, (int64_t)a.table_width << a.ps_log2);  // (beyond the table: zeros)
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&i_empty[ni % TA_ITEMS]);
    ++ni;
    const uint32_t skip = (g + G - next % G) % G;
    next += end * C::UNITS;
    part = 0;
    forward(skip);
    page();
  }
  // One iteration: copies the next unit; false once nothing is left to copy or on its way.
  __device__ __forceinline__ bool issue() {
    real <<= 1;
    while (__builtin_expect((q >= end) & more & ok, 0)) {
      const uint32_t had = ni;
      item((real & ((1u << C::DEPTH) - 1)) == 0);
      if (ni == had) break;
    }
    if (__builtin_expect(!ok, 0)) return false;
    if (__builtin_expect(q < end, 1)) {
      // whole rows of pages of 16 and more, as nearly all are: nothing to cut off
      const bool v = values();
      if (__builtin_expect(__all_sync(0xffffffffu, (uint32_t)mine < (uint32_t)a.P) & c.s_whole, 1)) {
        if (v) whole<true>();
        else whole<false>();
      } else {
        cut(v);
      }
      real |= 1u;
      forward(G);
      page();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    stage = stage + C::SB == C::DEPTH * C::SB ? 0u : stage + C::SB;
    return more | (q < end) | ((real & ((1u << C::DEPTH) - 1)) != 0);
  }
  template <bool V>
  __device__ __forceinline__ void whole() {
    const int lane = threadIdx.x & 31, r0 = threadIdx.x & 96, in = (1 << a.ps_log2) - 1;
    const uint32_t token = V ? c.vc_token : c.kc_token, s_token = V ? c.vs_token : c.ks_token;
    uint8_t* dst = ring + stage;
    const uint32_t id[2] = {__shfl_sync(0xffffffffu, (uint32_t)mine, 0), __shfl_sync(0xffffffffu, (uint32_t)mine, 16)};
    const uint32_t o[2] = {(uint32_t)(pos & in), (uint32_t)((pos + 16) & in)};
    const uint8_t* codes = (V ? c.vc + h * c.vc_head : c.kc + h * c.kc_head) + part * C::RB + lane % CPR * 16;
    const uint8_t* scales = (V ? c.vs + h * c.vs_head : c.ks + h * c.ks_head) + part * C::SP;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint8_t* row = codes + (uint64_t)id[e] * (uint32_t)(V ? c.vc_page : c.kc_page) + (uint64_t)(o[e] + lane / CPR) * token;
      uint8_t* to = dst + r0 * C::RB + tq_code<C>(lane / CPR, lane % CPR);
#pragma unroll
      for (int i = 0; i < 16 / RPI; ++i) {
        tq_copy16(to + (16 * e + i * RPI) * C::RB, row);
        row += (uint64_t)RPI * token;
      }
    }
    tq_copy_row<C::SP>(dst + TA_BN * C::RB + (r0 + lane) * C::SP,
                       scales + (uint64_t)(uint32_t)mine * (uint32_t)(V ? c.vs_page : c.ks_page) +
                           (uint64_t)((lane < 16 ? o[0] : o[1]) + (lane & 15)) * s_token);
  }
  __device__ __forceinline__ void cut(bool v) {
    const int lane = threadIdx.x & 31, r0 = threadIdx.x & 96, piece = lane % CPR;
    uint8_t* dst = ring + stage;
    const int in = (1 << a.ps_log2) - 1, left = a.D - part * C::COL;  // columns
    const uint32_t page = v ? c.vc_page : c.kc_page, token = v ? c.vc_token : c.kc_token;
    const uint32_t s_page = v ? c.vs_page : c.ks_page, s_token = v ? c.vs_token : c.ks_token;
    const uint8_t* from = (v ? c.vc : c.kc) + h * (v ? c.vc_head : c.kc_head) + part * C::RB + piece * 16;
    const uint8_t* s_from = (v ? c.vs : c.ks) + h * (v ? c.vs_head : c.ks_head) + part * C::SP;
    uint8_t* to = dst + TA_BN * C::RB + (r0 + lane) * C::SP;
    const bool there = (uint32_t)mine < (uint32_t)a.P;
    const uint64_t off = (uint32_t)((pos + lane) & in);
    const uint64_t row = there ? (uint64_t)(uint32_t)mine * page + off * token : ~0ull;  // of the lane's own row
    const int wide = min(max(left / 2 - piece * 16, 0), 16);
#pragma unroll
    for (int i = 0; i < 32 / RPI; ++i) {
      const int r = i * RPI + lane / CPR;
      const uint64_t at = __shfl_sync(0xffffffffu, row, r);
      const int bytes = at == ~0ull ? 0 : wide;
      tq_copy16(dst + tq_code<C>(r0 + r, piece), bytes ? from + at : c.kc, bytes);
    }
    s_from += (uint64_t)(uint32_t)mine * s_page + off * s_token;
#pragma unroll
    for (int w = 0; w < (int)C::SP / 4; ++w) {
      const int bytes = there ? min(max(left / 16 - 4 * w, 0), 4) : 0;
      tq_copy4(to + 4 * w, bytes ? s_from + 4 * w : c.ks, bytes);
    }
  }
  // Waits for the unit that was copied DEPTH - 1 iterations ago, at `ring + stage` (issue() has moved it on);
  // false if there was none.
  __device__ __forceinline__ bool come() const {
    asm volatile("cp.async.wait_group %0;" ::"n"(C::DEPTH - 1) : "memory");
    __syncwarp();
    return real >> (C::DEPTH - 1) & 1;
  }
};

// The pairs of f16 that 32 codes and their two scales stand for: 16 registers, four of 8 channels each.
__device__ __forceinline__ void tq_values(const uint4& codes, uint32_t two, uint32_t (&y)[16]) {
  const uint32_t s2 = q4_scales(two);
  const uint32_t s_lo = __byte_perm(s2, s2, 0x1010), s_hi = __byte_perm(s2, s2, 0x3232);
  const uint32_t word[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t p[4];
    q4_pairs(word[c], p);
#pragma unroll
    for (int k = 0; k < 4; ++k) y[4 * c + k] = q4_mul2(p[k], c < 2 ? s_lo : s_hi);
  }
}

// Calls f(p, values) for a row's pieces of 32 channels, two in a turn of a loop: five roles' code has to
// fit the instruction cache of a quarter of the SM (all unrolled, a third of all stalls were for instructions).
template <class C, class F>
__device__ __forceinline__ void tq_row(const uint8_t* src, int r, F f) {
  const uint32_t base = tc::smem_u32(src + tq_code<C>(r, 0));
  auto codes = [&](int p) {  // (where tq_code has them)
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(base ^ (uint32_t)(p << 4)) : "memory");
    return v;
  };
  uint32_t two[C::SP / 4];
#pragma unroll
  for (int w = 0; w < (int)C::SP / 4; ++w) two[w] = reinterpret_cast<const uint32_t*>(src + TA_BN * C::RB + r * C::SP)[w];
  uint4 x = codes(0), y = codes(1);
#pragma unroll 1
  for (int p = 0; p < C::COL / 32; p += 2) {
    uint32_t v[16];
    tq_values(x, two[0], v);
    if (C::COL > 64) x = codes(2);
    f(p, v);
    tq_values(y, two[0] >> 16, v);
    if (C::COL > 64) y = codes(3);
    f(p + 1, v);
    two[0] = two[C::SP / 4 - 1];
  }
}

// Attention over the cache in 4 bits: few rows a request, `rows` in the mean (paged_attn_q4.cu), many rows
// (paged_attn_q4_tc.cu).  Rows up to which the first is taken.  Measured (64 requests of 500 to 4096 keys, few against
// many), 32 heads on 8: bf16, heads of 128, 16 rows 79 and 95 us, 20 rows 118 and 95; heads of 64 67 and 76, 97 and 76;
// float32, heads of 128, 88 and 143, 166 and 143; heads of 64 73 and 107, 137 and 108.  10 heads on 1 of 256: bf16 30 rows
// 50 and 54, 40 rows 59 and 52; float32 20 rows 44 and 61, 40 rows 70 and 60, 50 rows 84 and 62 (1 to 7 tokens, 40 rows in
// the mean, window 2048: 46 and 56).
constexpr int TQ_FEW_ROWS = 16, TQ_FEW_ROWS_WIDE = 32, TQ_FEW_ROWS_WIDE_F32 = 40;  // (wide: D above 128)
cudaError_t launch_paged_attn_q4(PagedArgs a, const Q4Cache& c, bool f32, int rows, cudaStream_t s);
size_t paged_attn_q4_ws_bytes(const paged_shape* s, int rows);
cudaError_t launch_paged_attn_q4_tc(PagedArgs a, const Q4Cache& c, bool f32, int rows, cudaStream_t s);
size_t paged_attn_q4_tc_ws_bytes(const paged_shape* s, int rows);
// Q4Cache::s_whole (a row that is cut off is copied piece by piece, with what lies behind it as zeros).
inline int q4_whole_scales(const PagedArgs& a, const Q4Cache& c) {
  const uint64_t on = reinterpret_cast<uintptr_t>(c.ks) | reinterpret_cast<uintptr_t>(c.vs) | c.ks_page | c.ks_token | c.ks_head |
                      c.vs_page | c.vs_token | c.vs_head;
  return on % (a.D <= 64 ? 4 : 8) == 0 && (a.D == 64 || a.D == 128 || a.D == 256) && a.ps_log2 >= 4;
}

}  // namespace rglru

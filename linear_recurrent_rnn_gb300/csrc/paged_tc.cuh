// Shared by the tensor-core attention kernels over the paged cache: bounded waits, the item
// records that a CTA's warps read, the copy of key and value tiles, and arithmetic of the softmax.
#pragma once

#include <atomic>

#include "host_util.h"
#include "paged.cuh"
#include "tc.cuh"

namespace rglru {

constexpr int TA_BN = 128;                     // keys of a tile
constexpr uint64_t TA_WAIT_NS = 2000000000ull;  // a wait's limit: far above any time it can take
constexpr uint32_t TA_SLAB = 128 * 128;        // 64 columns of 128 rows

struct TaAbort {
  uint32_t* flag;     // shared: set once a wait has run out
  uint32_t* status;   // global
  uint64_t limit_ns;  // of a wait
  // By a converged warp; the answer is the same in all its lanes.
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
    bool ok = tc::mbar_try_wait(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) ok = __all_sync(0xffffffffu, ok || slow(bar, parity));
    return ok;
  }
  // The same for what may not come for most of a long call.
  __device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t parity) const {
    const TaAbort longer{flag, status, 100 * limit_ns};
    return longer.wait(bar, parity);
  }
  // By one thread.
  __device__ __forceinline__ bool wait1(uint64_t* bar, uint32_t parity) const {
    return tc::mbar_try_wait(bar, parity) || slow(bar, parity);
  }
  __device__ bool slow(uint64_t* bar, uint32_t parity) const {
    const uint64_t t0 = tc::global_ns();
    while (!tc::mbar_try_wait_sleep(bar, parity, 20000u)) {
      if (*reinterpret_cast<volatile uint32_t*>(flag)) return false;
      if (tc::global_ns() - t0 > limit_ns) {
        *reinterpret_cast<volatile uint32_t*>(flag) = 1u;
        *reinterpret_cast<volatile uint32_t*>(status) = 1u;
        return false;
      }
    }
    return true;
  }
};

// An item of the CTA's work as its warps read it: written by the walking warp into a ring in
// shared memory, so that the walk's state costs the other warps no registers.
struct TaItem {
  int n, h;           // request (-1: no more items), key/value head
  int first, q, kv;   // its first token row, new tokens, keys
  int tok;            // the item's first token
  int j0, j1;         // key tiles of the CTA's part
  int lo, hi;         // keys that the item's rows see
  int c0, c1, slot;   // CTAs that share the item, this one's partial-result slot
};
constexpr int TA_ITEMS = 4;

// Key tile j has positions that no row of the item sees (keys [lo, hi)).
__device__ __forceinline__ bool ta_cut(int j, int lo, int hi) {
  return (j + 1) * TA_BN > hi || j * TA_BN < lo;
}

// Value tiles with rows that no row of their item sees (past the request's keys, before the
// window) are cleared there before they are used: the loader leaves a record, a warp of its own
// clears, the MMA issuer waits for it at such a tile.  More records than value tiles fit the ring.
struct TaClear {
  int p0, lo, hi;         // the tile's first position (-1: no more tiles), the keys that are seen
  uint32_t st[2], par[2]; // the units' stages and their parity
};
constexpr int TA_CLEARS = 16;

// How a unit lies in shared memory, as slabs of 64 columns in the 128-byte swizzle.  Keys: 128 rows of
// NS slabs, values: VROWS rows of SLABS slabs.  A box has a cost of its own (measured: some 40 cycles
// beside 13 a KB), so with pages of up to 16 rows it holds all of a unit's slabs of 8 rows (keys,
// whose groups of 8 rows have to lie evenly spaced) or up to 16 rows (values, read 16 rows a product);
// otherwise a box is the rows of a page of one slab, and a slab's rows lie together.  Heads
// whose width is not a multiple of 64 stay with the latter, as zeros fill their last slab at the
// map's inner edge.  Measured (2 prompts of 4096, 16 heads on 4; pages of 8 and 16 rows, and of 64):
// heads of 128: 123 and 120 us (single slabs 167 and 121), 119; heads of 256: 291 and 265 (571 and
// 356), 212.  64 requests decoding on 4096 keys: heads of 128: 102 and 97 (143 and 95), 90; heads of
// 256: 170 and 168 (247 and 172), 165.  A template parameter, as offsets that are not constants
// cost the thread that issues the products 4 to 20 % of the kernel.
template <class C>
struct TaLay {
  static constexpr int NS = C::SLABS / C::UPT;
  int v_log2;  // rows of a box of values
  __device__ __forceinline__ explicit TaLay(const PagedArgs& a)
      : v_log2(C::WIDE ? min(a.ps_log2, 4) : C::VROWS == 128 ? 7 : 6) {}
  // bytes from one slab to the next, from one group of 8 rows to the next, from 16 rows to the next
  static constexpr uint32_t K_SLAB = C::WIDE ? 1024 : TA_SLAB;
  static constexpr uint32_t K_GROUP = C::WIDE ? NS * 1024 : 1024;
  static constexpr uint32_t V_16 = C::WIDE ? C::SLABS * 2048 : 2048;
  __device__ __forceinline__ uint32_t v_slab() const { return 128u << v_log2; }
  __device__ __forceinline__ uint32_t v_group() const { return v_log2 == 3 ? C::SLABS * 1024 : 1024; }
  __device__ __forceinline__ uint32_t v_row(int r) const {
    return ((r >> v_log2) * (C::SLABS << v_log2) + (r & ((1 << v_log2) - 1))) * 128;
  }
};
inline bool ta_wide(const PagedArgs& a) { return a.D > 64 && a.D % 64 == 0 && a.ps_log2 <= 4; }

template <class C>
__device__ __forceinline__ void ta_clear_rows(const PagedArgs& a, const TaAbort& ctl, const TaClear* rec, uint64_t* come, uint64_t* clean,
                                              uint64_t* full, uint8_t* ring) {
  constexpr int PIECES = C::SLABS * 8;  // 16-byte pieces of a row
  const int lane = threadIdx.x & 31;
  const int piece = lane % PIECES, sub = lane / PIECES;
  const TaLay<C> lay(a);
  for (uint32_t n = 0; ctl.wait_long(&come[n % TA_CLEARS], n / TA_CLEARS & 1); ++n) {
    const TaClear x = rec[n % TA_CLEARS];
    if (x.p0 < 0) break;
#pragma unroll
    for (int u = 0; u < C::UPT; ++u) {
      if (!ctl.wait(&full[x.st[u]], x.par[u])) return;
      uint8_t* dst = ring + x.st[u] * C::UB + piece / 8 * lay.v_slab() + piece % 8 * 16;
      const int p = x.p0 + u * C::VROWS;
      for (int r = sub; r < min(x.lo - p, C::VROWS); r += 32 / PIECES)
        *reinterpret_cast<uint4*>(dst + lay.v_row(r)) = make_uint4(0, 0, 0, 0);
      for (int r = max(x.hi - p, 0) + sub; r < C::VROWS; r += 32 / PIECES)
        *reinterpret_cast<uint4*>(dst + lay.v_row(r)) = make_uint4(0, 0, 0, 0);
    }
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&clean[n % TA_CLEARS]);
  }
}

// Copies key and value tiles into the ring, by one warp.  A tile is UPT units of UB bytes: keys
// 128 rows of 128 (or 64) columns a unit, values VROWS rows of all columns, page by page (TaLay).
// C: the kernel's constants.
template <class C>
struct TaLoader {
  const PagedArgs& a;
  const TaAbort& ctl;
  uint8_t* ring;
  uint64_t* full;
  uint64_t* empty;
  TaClear* rec;
  uint64_t* come;
  uint32_t st = 0, ph = 1;  // next stage, parity of its `empty`
  uint32_t issued = 0, clears = 0;

  // This lane's page of key tile j (a.P, outside the tensor map and so zeros, where the tile needs
  // none).  Lanes from the number of a tile's pages on have none.
  __device__ __forceinline__ int page_of(const TaItem& it, int j) const {
    const int lane = threadIdx.x & 31;
    if (j >= it.j1 || lane >= max(1, TA_BN >> a.ps_log2)) return a.P;
    const int pos = j * TA_BN + (lane << a.ps_log2), pg = pos >> a.ps_log2;
    if (pos >= it.hi || pos + min(1 << a.ps_log2, TA_BN) <= it.lo || pg >= a.table_width) return a.P;
    const int id = a.table[(int64_t)it.n * a.table_width + pg];
    return id >= 0 && id < a.P ? id : a.P;
  }
  // Rows [r0, r0 + NR) of tile j, NS slabs from s0 on (wide: in boxes of 2^box_log2 rows; else a slab's
  // rows together).
  template <int NR, int NS>
  __device__ __forceinline__ bool unit(const CUtensorMap* tm, int j, int id, int h, int r0, int s0, int box_log2) {
    constexpr uint32_t SB = NR * 128;
    const int lane = threadIdx.x & 31, ps = 1 << a.ps_log2;
    if (!ctl.wait(&empty[st], ph)) return false;
    if (lane == 0) tc::mbar_expect_tx(&full[st], C::UB);
    __syncwarp();
    if (C::WIDE) {
      const int r = r0 + (lane << box_log2);  // this lane's box: its first row, its page's entry
      const int page = __shfl_sync(0xffffffffu, id, (r & (TA_BN - 1)) >> a.ps_log2);
      if (lane < NR >> box_log2)
        tc::tma_load_5d(ring + st * C::UB + lane * (NS * 128 << box_log2), tm, &full[st], 0, r & (ps - 1), s0, h, page);
      return advance();
    }
    const int bx = min(ps, NR);                                    // rows of a box
    const int i = lane - (ps >= TA_BN ? 0 : r0 >> a.ps_log2);      // box of this lane's page
    if (i >= 0 && i < max(1, NR >> a.ps_log2)) {
      uint8_t* dst = ring + st * C::UB + i * bx * 128;
      const int off = ps > NR ? (j * TA_BN + r0) & (ps - 1) : 0;
#pragma unroll
      for (int s = 0; s < NS; ++s) tc::tma_load_4d(dst + s * SB, tm, &full[st], (s0 + s) * 64, off, h, id);
    }
    return advance();
  }
  __device__ __forceinline__ bool advance() {
    __syncwarp();
    ++issued;
    if (++st == C::STAGES) {
      st = 0;
      ph ^= 1;
    }
    return true;
  }
  __device__ __forceinline__ bool keys(const CUtensorMap* tm, int j, int id, int h) {
    constexpr int NS = C::SLABS / C::UPT;
#pragma unroll
    for (int u = 0; u < C::UPT; ++u)
      if (!unit<TA_BN, NS>(tm, j, id, h, 0, NS * u, 3)) return false;
    return true;
  }
  // Keys [lo, hi) are seen by the tile's item.
  __device__ __forceinline__ bool values(const CUtensorMap* tm, int j, int id, int h, int lo, int hi) {
    TaClear x;
    x.p0 = j * TA_BN;
    x.lo = lo;
    x.hi = hi;
#pragma unroll
    for (int u = 0; u < C::UPT; ++u) {
      x.st[u] = st;
      x.par[u] = ph ^ 1;
      if (!unit<C::VROWS, C::SLABS>(tm, j, id, h, u * C::VROWS, 0, min(a.ps_log2, 4))) return false;
    }
    if (ta_cut(j, lo, hi)) clear(x);
    return true;
  }
  __device__ __forceinline__ void clear(const TaClear& x) {
    if ((threadIdx.x & 31) == 0) {
      rec[clears % TA_CLEARS] = x;
      tc::mbar_arrive(&come[clears % TA_CLEARS]);
    }
    __syncwarp();
    ++clears;
  }
  // No more tiles.
  __device__ __forceinline__ void end() {
    TaClear x;
    x.p0 = -1;
    clear(x);
  }
};

// Columns of the kernels' tiles.
inline int ta_width(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

// Tensor maps: queries in boxes of tb tokens x g heads x 64 columns, the caches in boxes of one
// page's rows (at most a tile's, for values VROWS) x 64 columns, or of several slabs (TaLay).
template <class C>
cudaError_t ta_maps(const PagedArgs& a, int tb, CUtensorMap* mq, CUtensorMap* mk, CUtensorMap* mv) {
  const int ps = 1 << a.ps_log2;
  const uint64_t dq[3] = {(uint64_t)a.D, (uint64_t)a.Hq, (uint64_t)a.T};
  const uint64_t sq[2] = {(uint64_t)a.q_head * 2, (uint64_t)a.q_token * 2};
  const uint32_t bq[3] = {64, (uint32_t)a.g, (uint32_t)tb};
  const uint64_t dk[4] = {(uint64_t)a.D, (uint64_t)ps, (uint64_t)a.Hkv, (uint64_t)a.P};
  const uint64_t sk[3] = {(uint64_t)a.kc_token * 2, (uint64_t)a.kc_head * 2, (uint64_t)a.kc_page * 2};
  const uint64_t sv[3] = {(uint64_t)a.vc_token * 2, (uint64_t)a.vc_head * 2, (uint64_t)a.vc_page * 2};
  const uint32_t bk[4] = {64, (uint32_t)(ps < TA_BN ? ps : TA_BN), 1, 1};
  const uint32_t bv[4] = {64, (uint32_t)(ps < C::VROWS ? ps : C::VROWS), 1, 1};
  cudaError_t e = encode_tmap(mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.q, dq, sq, bq, CU_TENSOR_MAP_SWIZZLE_128B);
  if (C::WIDE) {
    const uint64_t dw[5] = {64, (uint64_t)ps, (uint64_t)a.D / 64, (uint64_t)a.Hkv, (uint64_t)a.P};
    const uint64_t wk[4] = {sk[0], 128, sk[1], sk[2]}, wv[4] = {sv[0], 128, sv[1], sv[2]};
    const uint32_t xk[5] = {64, 8, C::SLABS / C::UPT, 1, 1}, xv[5] = {64, (uint32_t)ps, C::SLABS, 1, 1};
    if (e == cudaSuccess)
      e = encode_tmap(mk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, a.kc, dw, wk, xk, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
      e = encode_tmap(mv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, a.vc, dw, wv, xv, CU_TENSOR_MAP_SWIZZLE_128B);
    return e;
  }
  if (e == cudaSuccess)
    e = encode_tmap(mk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, a.kc, dk, sk, bk, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e == cudaSuccess)
    e = encode_tmap(mv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, a.vc, dk, sv, bv, CU_TENSOR_MAP_SWIZZLE_128B);
  return e;
}

// Once a device and kernel: its shared memory, and that it has at least `regs` registers a thread
// at launch.  `ready` has a bit a device.
inline cudaError_t ta_prepare(const void* f, size_t smem, int regs, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || ready.load(std::memory_order_relaxed) >> dev & 1) return e;
  e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes at;
  e = cudaFuncGetAttributes(&at, f);
  if (e != cudaSuccess) return e;
  if (at.numRegs < regs) return cudaErrorInvalidConfiguration;
  ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  return cudaSuccess;
}

__device__ __forceinline__ float ta_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float ta_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// two float32 operations in one instruction
__device__ __forceinline__ float2 ta_fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 ta_add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ uint32_t ta_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace rglru

// Attention over the paged cache on the CUDA cores (float32 I/O: its 1e-5 bound).
//
// One pass over the keys with a running maximum and sum: per tile of keys
//   S = Q K^T (scores in units of log2), m' = max(m, max S), P = 2^(S - m'),
//   l = l 2^(m - m') + sum P,  O = O 2^(m - m') + P V
// and at the end o = O / l, lse = (m + log2 l) ln 2.
//
// A row tile is BM rows (whole tokens x the query heads of one key/value head).  Half a warp
// owns 4 rows: 16 lanes side by side along the keys for S and along the columns for O, so that
// maxima, sums and the exchange of P stay within 16 lanes, and only the key and value tiles
// are shared by the CTA.  With many rows (BM = 64) all warps work on one tile of keys and the
// kernel is bound by the float32 pipe; two products an instruction (fma.f32x2) and 4 x 4 (S) or
// 4 x DP / 16 (O) outputs a thread keep shared memory below it.  With few (BM = 32, 16, 8:
// drafts, decode) it is bound by memory, and groups of BM / 8 warps take a part of the tile's keys
// each, with maxima and sums of their own that are joined when the item ends.
// Tiles are gathered by 16-byte asynchronous copies, row by row through the block table (whose
// entries are looked up one tile ahead): values land behind the scores, the next keys behind P V.
// Keys that no row of the item sees are not read, their rows are zero.  Products
// run over the columns in use, not the tile's width (heads of 192, 64 requests with a window of 256: 137 -> 116
// us; heads of 96, 249 requests decoding: 408 -> 368).  Work is divided over CTAs
// by weight (paged.cuh).
//
// Measured (GB300): 64 requests of 500 to 4096 keys, 16 query heads on 4 of 128 (452 MB): 111 us,
// 4.1 TB/s: eight warps an SM do not cover the latencies of a tile's phases.  Two chunks of 1024 tokens over 2048
// keys, the same heads: 651 us, 40 TFLOP/s of 74: shared-memory reads and the two barriers a tile
// with 8 warps an SM (row tiles of 128 and 16 warps: 590 us here, but slower for short calls, as
// 128 registers a thread spill).
#include <algorithm>

#include "host_util.h"
#include "paged.cuh"
#include "tc.cuh"

namespace rglru {

namespace {

template <int BM, int DP>
struct Sa {
  static constexpr int THREADS = BM == 8 ? 128 : 256;
  static constexpr int SPLIT = THREADS / 4 / BM;  // key ranges of a tile
  // keys of a range: 64, or what lets a tile of all ranges fit
  static constexpr int BN = SPLIT == 1 ? 64 : SPLIT == 2 ? (DP == 256 ? 32 : 64)
                            : BM == 16 ? (DP == 64 ? 64 : 4096 / DP) : 2048 / DP;
  static constexpr int TILE = SPLIT * BN;
  static constexpr int KS = BN / 16;     // keys a thread
  static constexpr int C4 = DP / 64;     // times four columns of O a thread
  static constexpr int DS = KS > 2 ? 16 : 32;  // columns of Q K^T at a time
  static constexpr int LD = DP + 4;      // row stride: 16-byte reads of 8 rows meet all banks
  static constexpr int CTAS = (BM == 64 && DP == 64) || BM == 8 ? 2 : 1;  // per SM
  // shared memory, in floats: queries, keys, values, P^T of each warp; then row offsets
  static constexpr int Q = 0, K = Q + BM * LD, V = K + TILE * LD, P = V + TILE * LD, OFF = P + THREADS / 32 * BN * 8;
  static constexpr size_t smem = (size_t)OFF * 4 + (size_t)4 * TILE * 8;
};

__device__ __forceinline__ void sa_copy16(float* dst, const float* src, bool read) {
  const int n = read ? 16 : 0;  // 0: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void sa_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void sa_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ float2 sa_fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}

template <int BM, int DP>
__global__ void __launch_bounds__(Sa<BM, DP>::THREADS, Sa<BM, DP>::CTAS) k_paged_attn_simt(const PagedArgs a) {
  using C = Sa<BM, DP>;
  extern __shared__ __align__(16) float sa_sm[];
  float* s_q = sa_sm + C::Q;
  float* s_k = sa_sm + C::K;
  float* s_v = sa_sm + C::V;
  int64_t* s_off = reinterpret_cast<int64_t*>(sa_sm + C::OFF);  // [2 tiles][keys, values][TILE]
  __shared__ int64_t scratch[33];
  __shared__ float2 s_ml[C::SPLIT][BM];  // maxima and sums of the key ranges
  __shared__ float s_f[BM], s_sum[BM];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sp = warp / (BM / 8), tx = lane & 15;
  const int r0 = warp % (BM / 8) * 8 + (lane >> 4) * 4;  // first of this thread's rows
  float* s_p = sa_sm + C::P + warp * (C::BN * 8) + (lane >> 4) * 4;

  tc::griddep_wait();
  tc::griddep_launch_dependents();
  PgWalk w;
  PgWalk::Found start;
  if (a.N <= PG_WARP_SEQS) {
    start = w.find_warp(a);
  } else {
    int64_t* prefix = reinterpret_cast<int64_t*>(sa_sm);  // before the tiles are in use
    pg_scan(a, prefix, scratch);
    start = w.find(a, prefix);
    __syncthreads();
  }
  if (!w.enter(a, start)) return;
  do {
    const PgItem& it = w.it;
    int j0, j1;
    w.tiles(C::TILE, j0, j1);
    const int t0 = it.m * a.tb, rows = min(a.tb, it.r.q - t0) * a.g;
    const int base = it.r.kv - it.r.q + t0;  // position of row 0
    int pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) pos[i] = base + pg_token(a, min(r0 + i, rows - 1));

    // offsets of tile j's rows (negative: not seen, or no page)
    auto look_up = [&](int j) {
      if (j >= j1 || tid >= C::TILE) return;
      const int p = j * C::TILE + tid;
      int64_t ko = -1, vo = -1;
      if (p >= it.lo && p < it.hi) {
        const int pg = p >> a.ps_log2, off = p & ((1 << a.ps_log2) - 1);
        const int id = pg < a.table_width ? a.table[(int64_t)it.n * a.table_width + pg] : -1;
        if (id >= 0 && id < a.P) {
          ko = id * a.kc_page + off * a.kc_token;
          vo = id * a.vc_page + off * a.vc_token;
        }
      }
      s_off[(j & 1) * 2 * C::TILE + tid] = ko;
      s_off[((j & 1) * 2 + 1) * C::TILE + tid] = vo;
    };
    auto load = [&](int j, int kv) {
      const int64_t* off = s_off + ((j & 1) * 2 + kv) * C::TILE;
      float* dst = kv ? s_v : s_k;
      const float* src = static_cast<const float*>(kv ? a.vc : a.kc) + it.h * (kv ? a.vc_head : a.kc_head);
#pragma unroll 4
      for (int i = tid; i < C::TILE * (DP / 4); i += C::THREADS) {
        const int r = i / (DP / 4), c = i % (DP / 4) * 4;
        const int64_t o = off[r];
        const bool read = o >= 0 && c < a.D;
        sa_copy16(dst + r * C::LD + c, read ? src + o + c : src, read);
      }
      sa_commit();
    };

    look_up(j0);
    for (int i = tid; i < BM * (DP / 4); i += C::THREADS) {
      const int r = i / (DP / 4), c = i % (DP / 4) * 4, t = pg_token(a, r);
      const bool read = r < rows && c < a.D;
      const float* src = static_cast<const float*>(a.q);
      if (read)
        src += (int64_t)(it.r.first + t0 + t) * a.q_token + (int64_t)(it.h * a.g + r - t * a.g) * a.q_head + c;
      sa_copy16(s_q + r * C::LD + c, src, read);
    }
    sa_commit();
    __syncthreads();
    if (j0 < j1) load(j0, 0);

    float m[4], l[4];
    float2 acc[4][2 * C::C4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.0f;
#pragma unroll
      for (int c = 0; c < 2 * C::C4; ++c) acc[i][c] = make_float2(0.0f, 0.0f);
    }
    for (int j = j0; j < j1; ++j) {
      sa_wait();        // the keys are there,
      __syncthreads();  // for everyone, and the values before are used
      load(j, 1);
      look_up(j + 1);
      float2 s2[4][C::KS];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < C::KS; ++k) s2[i][k] = make_float2(0.0f, 0.0f);
      const float* kp = s_k + (sp * C::BN + tx) * C::LD;
      const float* qp = s_q + r0 * C::LD;
      // (columns past D are zero up to the next multiple of DS)
#pragma unroll 1
      for (int d0 = 0; d0 < a.D; d0 += C::DS)
#pragma unroll
        for (int d = d0; d < d0 + C::DS; d += 4) {
          float4 q[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const float4*>(qp + i * C::LD + d);
#pragma unroll
          for (int k = 0; k < C::KS; ++k) {
            const float4 x = *reinterpret_cast<const float4*>(kp + k * 16 * C::LD + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              s2[i][k] = sa_fma2(make_float2(q[i].x, q[i].y), make_float2(x.x, x.y), s2[i][k]);
              s2[i][k] = sa_fma2(make_float2(q[i].z, q[i].w), make_float2(x.z, x.w), s2[i][k]);
            }
          }
        }
      float p[4][C::KS];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < C::KS; ++k) {
          const int key = j * C::TILE + sp * C::BN + tx + 16 * k;
          const bool seen = key <= pos[i] && (!a.window || key > pos[i] - a.window);
          p[i][k] = seen ? (s2[i][k].x + s2[i][k].y) * a.scale_log2 : -INFINITY;
          top = fmaxf(top, p[i][k]);
        }
#pragma unroll
        for (int b = 8; b; b >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, b));
        const float m1 = fmaxf(m[i], top);
        // a row that has seen nothing yet keeps m = -inf; its weights are zero
        const float sub = m1 == -INFINITY ? 0.0f : m1, f = exp2f(m[i] - sub);
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < C::KS; ++k) {
          p[i][k] = exp2f(p[i][k] - sub);
          sum += p[i][k];
        }
        m[i] = m1;
        l[i] = l[i] * f + sum;  // over this lane's keys; over the lanes when the item ends
#pragma unroll
        for (int c = 0; c < 2 * C::C4; ++c) acc[i][c] = make_float2(acc[i][c].x * f, acc[i][c].y * f);
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < C::KS; ++k)
        *reinterpret_cast<float4*>(s_p + (tx + 16 * k) * 8) = make_float4(p[0][k], p[1][k], p[2][k], p[3][k]);
      sa_wait();        // the values are there,
      __syncthreads();  // for everyone, and the keys are used
      if (j + 1 < j1) load(j + 1, 0);
      const float* vp = s_v + sp * C::BN * C::LD + tx * 4;
#pragma unroll (C::C4 > 1 || BM == 64 ? 4 : 8)
      for (int k = 0; k < C::BN; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(s_p + k * 8);
        const float pr[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int c = 0; c < C::C4; ++c) {
          if (c > C::C4 / 2 && 64 * c >= a.D) break;  // (D is above DP / 2)
          const float4 v = *reinterpret_cast<const float4*>(vp + k * C::LD + 64 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 pp = make_float2(pr[i], pr[i]);
            acc[i][2 * c] = sa_fma2(pp, make_float2(v.x, v.y), acc[i][2 * c]);
            acc[i][2 * c + 1] = sa_fma2(pp, make_float2(v.z, v.w), acc[i][2 * c + 1]);
          }
        }
      }
    }
    sa_wait();
    __syncthreads();  // the tiles' memory is free
    // the rows' parts over the key ranges to shared memory
    float* s_o = s_k;  // [SPLIT][BM][DP]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int b = 8; b; b >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], b);
      if (tx == 0) s_ml[sp][r0 + i] = make_float2(m[i], l[i]);
#pragma unroll
      for (int c = 0; c < C::C4; ++c)
        *reinterpret_cast<float4*>(s_o + ((sp * BM + r0 + i) * DP + tx * 4 + 64 * c)) =
            make_float4(acc[i][2 * c].x, acc[i][2 * c].y, acc[i][2 * c + 1].x, acc[i][2 * c + 1].y);
    }
    __syncthreads();
    const bool whole = w.whole();
    int c0 = w.cta, c1 = w.cta;
    if (!whole) w.owners(c0, c1);
    float2* g_ml = reinterpret_cast<float2*>(a.ws + a.part_ml);
    float* g_o = reinterpret_cast<float*>(a.ws + a.part_o);
    // one weight a range and row: 2^(m - top)
    if (tid < BM) {
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int q = 0; q < C::SPLIT; ++q)
        if (s_ml[q][tid].y != 0.0f) top = fmaxf(top, s_ml[q][tid].x);
#pragma unroll
      for (int q = 0; q < C::SPLIT; ++q) {
        const float f = s_ml[q][tid].y != 0.0f ? exp2f(s_ml[q][tid].x - top) : 0.0f;
        sum += s_ml[q][tid].y * f;
        s_ml[q][tid].x = f;
      }
      if (tid < rows) {
        if (!whole)
          g_ml[(size_t)PgWalk::slot(w.cta, c0) * BM + tid] = make_float2(top, sum);
        else if (a.lse)
          a.lse[(int64_t)(it.r.first + t0 + pg_token(a, tid)) * a.Hq + it.h * a.g + tid - pg_token(a, tid) * a.g] =
              sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
      }
      s_f[tid] = !whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
    }
    __syncthreads();
    auto write = [&](int r, int c, float4 x) {
      const int t = pg_token(a, r);
      *reinterpret_cast<float4*>(static_cast<float*>(a.o) + (int64_t)(it.r.first + t0 + t) * a.o_token +
                                 (int64_t)(it.h * a.g + r - t * a.g) * a.o_head + c) = x;
    };
    for (int i = tid; i < rows * (DP / 4); i += C::THREADS) {
      const int r = i / (DP / 4), c = i % (DP / 4) * 4;
      if (c >= a.D) continue;
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int q = 0; q < C::SPLIT; ++q) {
        const float4 o = *reinterpret_cast<const float4*>(s_o + (q * BM + r) * DP + c);
        const float f = s_ml[q][r].x * s_f[r];
        if (f != 0.0f) {
          x.x = fmaf(o.x, f, x.x);
          x.y = fmaf(o.y, f, x.y);
          x.z = fmaf(o.z, f, x.z);
          x.w = fmaf(o.w, f, x.w);
        }
      }
      if (whole)
        write(r, c, x);
      else
        *reinterpret_cast<float4*>(g_o + ((size_t)PgWalk::slot(w.cta, c0) * BM + r) * DP + c) = x;
    }
    __syncthreads();
    if (!whole) {
      if (tid == 0) {
        __threadfence();  // cumulative: the other threads' parts, ordered before by the barrier
        uint32_t* cnt = reinterpret_cast<uint32_t*>(a.ws + 256) + c0;
        const bool last = atomicAdd(cnt, 1u) == (uint32_t)(c1 - c0);
        if (last) *cnt = 0u;  // as it was found: zero between calls
        s_last = last;
      }
      __syncthreads();
      if (s_last) {
        // the item's last CTA joins its parts, up to PARTS at a time: their weights, then the sums
        __threadfence();
        float2* wt = reinterpret_cast<float2*>(s_k);  // [part][row]
        constexpr int PARTS = C::TILE * C::LD / (BM * 2), RP = C::THREADS * 4 / DP, PASSES = (BM + RP - 1) / RP;
        constexpr int BATCH = PASSES >= 16 ? 1 : 16 / PASSES;  // parts loaded at once
        const int c = tid % (DP / 4) * 4, rr = tid / (DP / 4);
        float4 o[PASSES];
#pragma unroll
        for (int k = 0; k < PASSES; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        float top = -INFINITY, sum = 0.0f;  // of row tid
        for (int q0 = c0; q0 <= c1; q0 += PARTS) {
          const int nq = min(PARTS, c1 - q0 + 1);
          for (int i = tid; i < nq * BM; i += C::THREADS)
            wt[i] = i % BM < rows ? __ldcg(g_ml + (size_t)PgWalk::slot(q0 + i / BM, c0) * BM + i % BM)
                                  : make_float2(0.0f, 0.0f);
          __syncthreads();
          if (tid < BM) {
            const float m0 = top;
            for (int q = 0; q < nq; ++q) top = fmaxf(top, wt[q * BM + tid].y != 0.0f ? wt[q * BM + tid].x : -INFINITY);
            const float f = m0 == top ? 1.0f : exp2f(m0 - top);
            sum *= f;
            for (int q = 0; q < nq; ++q) {
              const float2 x = wt[q * BM + tid];
              const float e = x.y != 0.0f ? exp2f(x.x - top) : 0.0f;
              sum += x.y * e;
              wt[q * BM + tid].x = e;
            }
            s_f[tid] = f;
            s_sum[tid] = sum;
          }
          __syncthreads();
          if (q0 > c0)
#pragma unroll
            for (int k = 0; k < PASSES; ++k) {
              const float f = s_f[min(rr + k * RP, BM - 1)];
              o[k] = make_float4(o[k].x * f, o[k].y * f, o[k].z * f, o[k].w * f);
            }
#pragma unroll 1
          for (int q = 0; q < nq; q += BATCH) {
            float4 v[BATCH][PASSES];
#pragma unroll
            for (int b = 0; b < BATCH; ++b)
#pragma unroll
              for (int k = 0; k < PASSES; ++k)
                v[b][k] = __ldcg(reinterpret_cast<const float4*>(
                    g_o + ((size_t)PgWalk::slot(q0 + min(q + b, nq - 1), c0) * BM + min(rr + k * RP, BM - 1)) * DP + c));
#pragma unroll
            for (int b = 0; b < BATCH; ++b)
#pragma unroll
              for (int k = 0; k < PASSES; ++k) {
                const float e = q + b < nq ? wt[(q + b) * BM + min(rr + k * RP, BM - 1)].x : 0.0f;
                if (e != 0.0f)  // (a part that saw nothing did not write its sums)
                  o[k] = make_float4(fmaf(e, v[b][k].x, o[k].x), fmaf(e, v[b][k].y, o[k].y),
                                     fmaf(e, v[b][k].z, o[k].z), fmaf(e, v[b][k].w, o[k].w));
              }
          }
          __syncthreads();
        }
        if (tid < rows && a.lse)
          a.lse[(int64_t)(it.r.first + t0 + pg_token(a, tid)) * a.Hq + it.h * a.g + tid - pg_token(a, tid) * a.g] =
              sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
#pragma unroll
        for (int k = 0; k < PASSES; ++k) {
          const int r = rr + k * RP;
          if (r >= rows || c >= a.D) break;
          const float inv = s_sum[r] == 0.0f ? 0.0f : 1.0f / s_sum[r];
          write(r, c, make_float4(o[k].x * inv, o[k].y * inv, o[k].z * inv, o[k].w * inv));
        }
        __syncthreads();
      }
    }
  } while (w.next(a));
}

template <int BM, int DP>
cudaError_t run(PagedArgs& a, cudaStream_t s, int sms) {
  using C = Sa<BM, DP>;
  static_assert(C::TILE <= C::THREADS, "a thread looks one row up");
  static_assert(C::SPLIT * BM * DP <= C::TILE * C::LD, "the parts of the key ranges fit the key tile");
  const size_t smem = std::max(C::smem, (size_t)(a.N + 1) * 8);
  const void* f = reinterpret_cast<const void*>(k_paged_attn_simt<BM, DP>);
  const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int ctas = std::min(sms * C::CTAS, PG_MAX_CTAS);
  const PagedWs L = paged_ws(ctas, BM, DP);
  a.part_ml = L.ml;
  a.part_o = L.o;
  a.rows = BM;
  a.tb = BM / a.g;
  pg_division(a, ctas, 128, 128, 128);
  void* args[] = {&a};
  return launch_pdl(f, dim3(ctas), dim3(C::THREADS), smem, s, args, 1);
}

template <int BM>
cudaError_t run_d(PagedArgs& a, cudaStream_t s, int sms) {
  if (a.D <= 64) return run<BM, 64>(a, s, sms);
  if (a.D <= 128) return run<BM, 128>(a, s, sms);
  return run<BM, 256>(a, s, sms);
}

}  // namespace

cudaError_t launch_paged_attn_simt(PagedArgs a, int rows, cudaStream_t s) {
  const int sms = sm_count();
  if (sms < 1) return cudaErrorNotSupported;
  // The row tile is the least that holds the mean's rows.  64 requests of 500 to 4096 keys, 16 heads
  // on 4 of 128: 4 rows in tiles of 8, 16, 64: 112, 155, 379 us; 16 rows: 226 (twice), 156, 379;
  // 20 rows: 333, 296, 223, 380 in tiles of 8, 16, 32, 64.  (Eight ranges of 256 columns do not fit.)
  if (rows <= 8 && a.D <= 128) return a.D <= 64 ? run<8, 64>(a, s, sms) : run<8, 128>(a, s, sms);
  return rows <= 16 ? run_d<16>(a, s, sms) : rows <= 32 ? run_d<32>(a, s, sms) : run_d<64>(a, s, sms);
}

size_t paged_attn_simt_ws_bytes(const paged_shape* s, int rows) {
  const int sms = sm_count();
  return paged_ws(std::min(2 * (sms > 0 ? sms : 256), PG_MAX_CTAS), rows <= 16 ? 16 : rows <= 32 ? 32 : 64,
                  s->D <= 64 ? 64 : s->D <= 128 ? 128 : 256).total;
}

}  // namespace rglru

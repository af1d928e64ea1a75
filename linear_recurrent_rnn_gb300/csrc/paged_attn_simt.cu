// Attention over the paged cache on the CUDA cores (float32 I/O: its 1e-5 bound).
//
// One pass over the keys with a running maximum and sum: per tile of BN keys
//   S = Q K^T (scores in units of log2), m' = max(m, max S), P = 2^(S - m'),
//   l = l 2^(m - m') + sum P,  O = O 2^(m - m') + P V
// and at the end o = O / l, lse = (m + log2 l) ln 2.  The row tile (BM rows: whole tokens x the
// query heads of one key/value head) stays in shared memory, O in registers, and the key tile is
// gathered page by page; work is divided over CTAs by weight (paged.cuh).
#include <algorithm>

#include "host_util.h"
#include "paged.cuh"
#include "tc.cuh"

namespace rglru {

namespace {

constexpr int SA_THREADS = 256;
constexpr int SA_BN = 64;

__device__ __forceinline__ float4 sa_load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
// BM rows, DP columns (D rounded up).  Threads: TX along keys / columns, TY along rows, 4 rows a
// thread.
template <int BM, int DP>
struct Sa {
  static constexpr int TY = BM / 4, TX = SA_THREADS / TY;
  static constexpr int KS = SA_BN / TX;        // keys a thread
  static constexpr int CS = DP / TX;           // columns of O a thread
  static constexpr int LD = DP + 4;            // row stride: 16-byte reads of 8 rows meet all banks
  static constexpr int LS = SA_BN + 4;
  static constexpr size_t smem = (size_t)((BM + 2 * SA_BN) * LD + BM * LS + 3 * BM) * 4;
};

template <int BM, int DP>
__global__ void __launch_bounds__(SA_THREADS) k_paged_attn_simt(const PagedArgs a) {
  using C = Sa<BM, DP>;
  extern __shared__ float sa_sm[];
  float* s_q = sa_sm;
  float* s_k = s_q + BM * C::LD;
  float* s_v = s_k + SA_BN * C::LD;
  float* s_p = s_v + SA_BN * C::LD;
  float* s_m = s_p + BM * C::LS;
  float* s_l = s_m + BM;
  float* s_a = s_l + BM;
  __shared__ int64_t scratch[33];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tx = tid % C::TX, ty = tid / C::TX;

  tc::griddep_wait();
  tc::griddep_launch_dependents();
  PgWalk w;
  {
    int64_t* prefix = reinterpret_cast<int64_t*>(sa_sm);  // before the tiles are in use
    pg_scan(a, prefix, scratch);
    const bool any = w.start(a, prefix);
    __syncthreads();
    if (!any) return;
  }
  const int dv = a.D / 4;
  do {
    const PgItem& it = w.it;
    int j0, j1;
    w.tiles(SA_BN, j0, j1);
    const int t0 = it.m * a.tb, rows = min(a.tb, it.r.q - t0) * a.g;
    const int64_t base = (int64_t)it.r.kv - it.r.q;
    for (int i = tid; i < BM * (DP / 4); i += SA_THREADS) {
      const int r = i / (DP / 4), c = i % (DP / 4);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows && c < dv)
        x = sa_load4(static_cast<const float*>(a.q) + (int64_t)(it.r.first + t0 + r / a.g) * a.q_token +
                     (int64_t)(it.h * a.g + r % a.g) * a.q_head + 4 * c);
      *reinterpret_cast<float4*>(s_q + r * C::LD + 4 * c) = x;
    }
    for (int r = tid; r < BM; r += SA_THREADS) {
      s_m[r] = -INFINITY;
      s_l[r] = 0.0f;
    }
    float acc[4][C::CS];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < C::CS; ++c) acc[i][c] = 0.0f;

    for (int j = j0; j < j1; ++j) {
      __syncthreads();
      for (int i = tid; i < SA_BN * (DP / 4); i += SA_THREADS) {
        const int r = i / (DP / 4), c = i % (DP / 4);
        const int64_t pos = (int64_t)j * SA_BN + r;
        float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
        if (pos >= it.lo && pos < it.hi && c < dv) {
          const int64_t pg = pos >> a.ps_log2, off = pos & ((1 << a.ps_log2) - 1);
          const int id = pg < a.table_width ? a.table[(int64_t)it.n * a.table_width + pg] : -1;
          if (id >= 0 && id < a.P) {
            k = sa_load4(static_cast<const float*>(a.kc) + id * a.kc_page + off * a.kc_token + it.h * a.kc_head + 4 * c);
            v = sa_load4(static_cast<const float*>(a.vc) + id * a.vc_page + off * a.vc_token + it.h * a.vc_head + 4 * c);
          }
        }
        *reinterpret_cast<float4*>(s_k + r * C::LD + 4 * c) = k;
        *reinterpret_cast<float4*>(s_v + r * C::LD + 4 * c) = v;
      }
      __syncthreads();
      // S: rows ty * 4 + i, keys tx + TX * k
      float s[4][C::KS];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < C::KS; ++k) s[i][k] = 0.0f;
      for (int d = 0; d < DP; d += 4) {
        float4 qv[4], kv[C::KS];
#pragma unroll
        for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(s_q + (ty * 4 + i) * C::LD + d);
#pragma unroll
        for (int k = 0; k < C::KS; ++k) kv[k] = *reinterpret_cast<const float4*>(s_k + (tx + C::TX * k) * C::LD + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < C::KS; ++k) {
            s[i][k] = fmaf(qv[i].x, kv[k].x, s[i][k]);
            s[i][k] = fmaf(qv[i].y, kv[k].y, s[i][k]);
            s[i][k] = fmaf(qv[i].z, kv[k].z, s[i][k]);
            s[i][k] = fmaf(qv[i].w, kv[k].w, s[i][k]);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        const int64_t p = base + t0 + r / a.g;
#pragma unroll
        for (int k = 0; k < C::KS; ++k) {
          const int64_t pos = (int64_t)j * SA_BN + tx + C::TX * k;
          const bool seen = r < rows && pos <= p && (!a.window || pos > p - a.window);
          s_p[r * C::LS + tx + C::TX * k] = seen ? s[i][k] * a.scale_log2 : -INFINITY;
        }
      }
      __syncthreads();
      // a warp takes BM / 8 rows, a lane two keys
#pragma unroll
      for (int rr = 0; rr < BM / 8; ++rr) {
        const int r = warp * (BM / 8) + rr;
        const float2 x = *reinterpret_cast<const float2*>(s_p + r * C::LS + 2 * lane);
        float mx = fmaxf(x.x, x.y);
#pragma unroll
        for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float m0 = s_m[r], m1 = fmaxf(m0, mx);
        // a row that has seen nothing yet keeps m = -inf; its weights are zero
        const float sub = m1 == -INFINITY ? 0.0f : m1;
        const float2 p = make_float2(exp2f(x.x - sub), exp2f(x.y - sub));
        float sum = p.x + p.y;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        *reinterpret_cast<float2*>(s_p + r * C::LS + 2 * lane) = p;
        __syncwarp();
        if (lane == 0) {
          const float al = exp2f(m0 - sub);
          s_a[r] = al;
          s_m[r] = m1;
          s_l[r] = s_l[r] * al + sum;
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float al = s_a[ty * 4 + i];
#pragma unroll
        for (int c = 0; c < C::CS; ++c) acc[i][c] *= al;
      }
      for (int k = 0; k < SA_BN; ++k) {
        float p[4], v[C::CS];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = s_p[(ty * 4 + i) * C::LS + k];
#pragma unroll
        for (int c = 0; c < C::CS; ++c) v[c] = s_v[k * C::LD + tx + C::TX * c];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < C::CS; ++c) acc[i][c] = fmaf(p[i], v[c], acc[i][c]);
      }
    }
    __syncthreads();
    float m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = s_m[ty * 4 + i];
      l[i] = s_l[ty * 4 + i];
    }
    bool last = true;
    if (!w.whole()) {
      int c0, c1;
      w.owners(c0, c1);
      float2* ml = reinterpret_cast<float2*>(a.ws + a.part_ml);
      float* po = reinterpret_cast<float*>(a.ws + a.part_o);
      const int slot = PgWalk::slot(w.cta, c0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        if (r >= rows) continue;
        if (tx == 0) ml[(size_t)slot * a.rows + r] = make_float2(m[i], l[i]);
#pragma unroll
        for (int c = 0; c < C::CS; ++c)
          po[((size_t)slot * a.rows + r) * DP + tx + C::TX * c] = acc[i][c];
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        uint32_t* cnt = reinterpret_cast<uint32_t*>(a.ws + 256) + c0;
        const uint32_t had = atomicAdd(cnt, 1u);
        s_last = had == (uint32_t)(c1 - c0);
        if (s_last) *cnt = 0u;  // as it was found: zero between calls
      }
      __syncthreads();
      last = s_last;
      if (last) {
        __threadfence();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          m[i] = -INFINITY;
          l[i] = 0.0f;
#pragma unroll
          for (int c = 0; c < C::CS; ++c) acc[i][c] = 0.0f;
          const int r = ty * 4 + i;
          if (r >= rows) continue;
          for (int q = c0; q <= c1; ++q) {
            const size_t at = (size_t)PgWalk::slot(q, c0) * a.rows + r;
            const float2 x = __ldcg(ml + at);
            if (x.y == 0.0f) continue;  // saw nothing
            const float m1 = fmaxf(m[i], x.x), f0 = exp2f(m[i] - m1), f1 = exp2f(x.x - m1);
            m[i] = m1;
            l[i] = l[i] * f0 + x.y * f1;
#pragma unroll
            for (int c = 0; c < C::CS; ++c)
              acc[i][c] = acc[i][c] * f0 + __ldcg(po + at * DP + tx + C::TX * c) * f1;
          }
        }
      }
    }
    if (last) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        if (r >= rows) continue;
        const int64_t t = it.r.first + t0 + r / a.g;
        const int hq = it.h * a.g + r % a.g;
        const float inv = l[i] > 0.0f ? 1.0f / l[i] : l[i] == 0.0f ? 0.0f : l[i];
        float* o = static_cast<float*>(a.o) + t * a.o_token + hq * a.o_head;
#pragma unroll
        for (int c = 0; c < C::CS; ++c) {
          const int col = tx + C::TX * c;
          if (col < a.D) o[col] = acc[i][c] * inv;
        }
        if (a.lse && tx == 0)
          a.lse[t * a.Hq + hq] = l[i] == 0.0f ? -INFINITY : (m[i] + log2f(l[i])) * 0.69314718055994531f;
      }
    }
    __syncthreads();
  } while (w.next(a));
}

template <int BM, int DP>
cudaError_t run(PagedArgs& a, cudaStream_t s, int sms) {
  using C = Sa<BM, DP>;
  const size_t smem = std::max(C::smem, (size_t)(a.N + 1) * 8);
  const void* f = reinterpret_cast<const void*>(k_paged_attn_simt<BM, DP>);
  cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const PagedWs L = paged_ws(sms, BM, DP);
  a.part_ml = L.ml;
  a.part_o = L.o;
  a.rows = BM;
  a.tb = std::max(1, BM / a.g);
  pg_division(a, sms, 128, 256);
  void* args[] = {&a};
  return launch_pdl(f, dim3(sms), dim3(SA_THREADS), smem, s, args, 1);
}

template <int BM>
cudaError_t run_d(PagedArgs& a, cudaStream_t s, int sms) {
  if (a.D <= 64) return run<BM, 64>(a, s, sms);
  if (a.D <= 128) return run<BM, 128>(a, s, sms);
  return run<BM, 256>(a, s, sms);
}

}  // namespace

cudaError_t launch_paged_attn_simt(PagedArgs a, cudaStream_t s) {
  const int sms = sm_count();
  if (sms < 1 || sms > PG_MAX_CTAS) return cudaErrorNotSupported;
  return run_d<64>(a, s, sms);
}

size_t paged_attn_simt_ws_bytes(const paged_shape* s) {
  const int sms = sm_count();
  return paged_ws(sms > 0 ? sms : 256, 64, s->D <= 64 ? 64 : s->D <= 128 ? 128 : 256).total;
}

}  // namespace rglru

// The cache held in 4 bits (include/paged_q4.h): the write of new keys and values, the read, and
// the host side of the attention.
#include <math.h>

#include <algorithm>

#include "host_util.h"
#include "paged_q4.cuh"

namespace rglru {

namespace {

// ---------------------------------------------------------------- write and read
// A lane has a group, 16 channels of a head of the keys or of the values, and takes it of several tokens at
// once: where the group lies is worked out once, and the tokens' loads are in flight together.  A token's
// groups are spread over the lanes of a warp, or of a part of one where it has few; more than 32 of them, and keys
// and values, are blocks of their own (blockIdx.y).
// Measured (GB300): 16384 tokens of 8 heads of 128 in bf16, written and read back, 33.9 us, 5.1 TB/s of what must
// move (with a lane's place worked out anew for each group, 16-byte loads and a division: 50.6); in float32 55, 5.5 TB/s.  Under
// ncu no part is full: issue slots 57 and 53 %, the read's way from L1 to L2 56 %.  Bound by latency for few tokens: 64
// of 1 head 5.4 us.
struct Q4RowArgs {
  int T, groups, s_log2, lanes_log2;  // groups of a token's keys; lanes of a token
  int head_groups, units;             // groups of a head; blocks of lanes for a token's keys and values
  int wide;                           // rows lie on 32 bytes
  int64_t slots_end;
  const int64_t* slots;
  uint8_t* row[2];  // k and v
  uint8_t* codes[2];
  uint8_t* scales[2];
  int64_t row_token[2], row_head[2], c_page[2], c_token[2], c_head[2], s_page[2], s_token[2], s_head[2];  // bytes
};

constexpr int Q4_THREADS = 256;

// 16 channels as they are stored
template <class T>
struct Q4Group {
  static constexpr int WORDS = 16 * sizeof(T) / 16;
  uint4 w[WORDS];
};
__device__ __forceinline__ float q4_get(const Q4Group<bf16>& g, int i) {
  const uint32_t x = (&g.w[i / 8].x)[i / 2 % 4];
  return __uint_as_float(i & 1 ? x & 0xffff0000u : x << 16);
}
__device__ __forceinline__ float q4_get(const Q4Group<float>& g, int i) { return __uint_as_float((&g.w[i / 4].x)[i % 4]); }

__device__ __forceinline__ void q4_put(Q4Group<bf16>& g, int i, float lo, float hi) { (&g.w[i / 8].x)[i / 2 % 4] = ta_pack(lo, hi); }
__device__ __forceinline__ void q4_put(Q4Group<float>& g, int i, float lo, float hi) {
  (&g.w[i / 4].x)[i % 4] = __float_as_uint(lo);
  (&g.w[i / 4].x)[i % 4 + 1] = __float_as_uint(hi);
}
// The largest of the group, without its sign, as bits: an infinity's are above all finite ones', a NaN's above those.
__device__ __forceinline__ uint32_t q4_top(const Q4Group<bf16>& g) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = __vmaxu2(top, (&g.w[i / 4].x)[i % 4] & 0x7fff7fffu);
  return max(top & 0xffff0000u, top << 16);
}
__device__ __forceinline__ uint32_t q4_top(const Q4Group<float>& g) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, (&g.w[i / 4].x)[i % 4] & 0x7fffffffu);
  return top;
}
// Whole sectors an instruction: half as many passes through L1.
__device__ __forceinline__ void q4_load32(uint4* u, const uint8_t* p) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(u[0].x), "=r"(u[0].y), "=r"(u[0].z), "=r"(u[0].w), "=r"(u[1].x), "=r"(u[1].y), "=r"(u[1].z), "=r"(u[1].w)
               : "l"(p)
               : "memory");
}

// A group's codes and scale.  x / s is needed to the last bit only near a border between two codes, s times
// a number b of at most 3 bits.  With r the reciprocal of s cut to 16 bits (never above it, so that a zero keeps its
// sign) and d = (1 - r s) / s, where r s is exact: x / s = x r + x d.  That sum, rounded once, is off by less than
// 2^-37 of it before its rounding; where x = s b it rounds to b, and the next float32 x on either side is
// at least 2^-24 / 1.875 of b away from it, more than half of the last bit by 2^-28: the code is that of the exact
// quotient.  The same for the largest by 6, of which no float32 quotient lies within 2^-27 of a rounding's border.
template <class T>
__device__ __forceinline__ uint2 q4_quantise(const Q4Group<T>& g, uint8_t& scale) {
  const uint32_t bits = q4_top(g);
  if (bits >= 0x7f800000u) {
    scale = 0x7f;  // NaN
    return make_uint2(0u, 0u);
  }
  const float top = __uint_as_float(bits);
  constexpr float SIXTH = 0x1.5554p-3f, REST = 0x1.555556p-19f;  // 1/6 in 16 bits, and what is left of it
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(fmaf(top, SIXTH, top * REST)));
  const uint32_t code = max((uint32_t)two & 0xffu, 1u);  // 1: 2^-9
  const uint32_t h = q4_scales(code);
  const float s = __half2float(reinterpret_cast<const __half2&>(h).x);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  const float cut = __uint_as_float(__float_as_uint(r) & 0xffffff00u), d = fmaf(-cut, s, 1.0f) * r;
  scale = (uint8_t)code;
  uint32_t out[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float2 q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = make_float2(q4_get(g, 8 * w + 2 * k), q4_get(g, 8 * w + 2 * k + 1));
      q[k] = make_float2(fmaf(x.x, cut, x.x * d), fmaf(x.y, cut, x.y * d));
    }
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(out[w])
        : "f"(q[0].x), "f"(q[0].y), "f"(q[1].x), "f"(q[1].y), "f"(q[2].x), "f"(q[2].y), "f"(q[3].x), "f"(q[3].y));
  }
  return make_uint2(out[0], out[1]);
}

// The lane's group of token 0 and slot 0: `kv` keys or values, its row, its codes and its scale.
struct Q4Place {
  int kv;
  bool in;
  uint8_t *row, *codes, *scale;
};
template <class T>
__device__ __forceinline__ Q4Place q4_place(const Q4RowArgs& a, int unit) {
  Q4Place p;
  p.kv = unit & 1;
  const int lanes = 1 << a.lanes_log2, c = (unit >> 1) * lanes + (threadIdx.x & (lanes - 1)), h = c / a.head_groups, b = c - h * a.head_groups;
  p.in = c < a.groups;
  p.row = a.row[p.kv] + h * a.row_head[p.kv] + b * (16 * (int)sizeof(T));
  p.codes = a.codes[p.kv] + h * a.c_head[p.kv] + b * 8;
  p.scale = a.scales[p.kv] + h * a.s_head[p.kv] + b;
  return p;
}
// tokens of a lane in flight
template <class T>
constexpr int Q4_BATCH = sizeof(T) == 2 ? 4 : 2;

template <class T>
__global__ void __launch_bounds__(Q4_THREADS) k_paged_q4_write(const __grid_constant__ Q4RowArgs a) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  constexpr int BATCH = Q4_BATCH<T>;
  const int64_t step = (int64_t)gridDim.x * Q4_THREADS >> a.lanes_log2;
  for (int unit = blockIdx.y; unit < a.units; unit += gridDim.y) {
    const Q4Place p = q4_place<T>(a, unit);
    if (!p.in) continue;
    for (int64_t t0 = ((int64_t)blockIdx.x * Q4_THREADS + threadIdx.x) >> a.lanes_log2; t0 < a.T; t0 += step * BATCH) {
      Q4Group<T> g[BATCH];
      int64_t slot[BATCH];
#pragma unroll
      for (int e = 0; e < BATCH; ++e) {
        const int64_t t = t0 + e * step;
        slot[e] = -1;
        if (t >= a.T) continue;
        slot[e] = a.slots[t];
        const uint8_t* src = p.row + t * a.row_token[p.kv];
        if (a.wide) {
#pragma unroll
          for (int w = 0; w < Q4Group<T>::WORDS; w += 2) q4_load32(g[e].w + w, src + 16 * w);
        } else {
#pragma unroll
          for (int w = 0; w < Q4Group<T>::WORDS; ++w) g[e].w[w] = reinterpret_cast<const uint4*>(src)[w];
        }
      }
#pragma unroll
      for (int e = 0; e < BATCH; ++e) {
        if (slot[e] < 0 || slot[e] >= a.slots_end) continue;
        const int64_t page = slot[e] >> a.s_log2, off = slot[e] & ((1 << a.s_log2) - 1);
        uint8_t scale;
        const uint2 codes = q4_quantise(g[e], scale);
        *reinterpret_cast<uint2*>(p.codes + page * a.c_page[p.kv] + off * a.c_token[p.kv]) = codes;
        p.scale[page * a.s_page[p.kv] + off * a.s_token[p.kv]] = scale;
      }
    }
  }
}

template <class T>
__global__ void __launch_bounds__(Q4_THREADS) k_paged_q4_read(const __grid_constant__ Q4RowArgs a) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  constexpr int BATCH = Q4_BATCH<T>;
  const int64_t step = (int64_t)gridDim.x * Q4_THREADS >> a.lanes_log2;
  for (int unit = blockIdx.y; unit < a.units; unit += gridDim.y) {
    const Q4Place p = q4_place<T>(a, unit);
    if (!p.in) continue;
    for (int64_t t0 = ((int64_t)blockIdx.x * Q4_THREADS + threadIdx.x) >> a.lanes_log2; t0 < a.T; t0 += step * BATCH) {
      int64_t slot[BATCH];
#pragma unroll
      for (int e = 0; e < BATCH; ++e) slot[e] = t0 + e * step < a.T ? a.slots[t0 + e * step] : -1;
      uint2 codes[BATCH];
      uint32_t scale[BATCH];
#pragma unroll
      for (int e = 0; e < BATCH; ++e) {
        codes[e] = make_uint2(0u, 0u);
        scale[e] = 0u;
        if (slot[e] < 0 || slot[e] >= a.slots_end) continue;
        const int64_t page = slot[e] >> a.s_log2, off = slot[e] & ((1 << a.s_log2) - 1);
        codes[e] = *reinterpret_cast<const uint2*>(p.codes + page * a.c_page[p.kv] + off * a.c_token[p.kv]);
        scale[e] = p.scale[page * a.s_page[p.kv] + off * a.s_token[p.kv]];
      }
#pragma unroll
      for (int e = 0; e < BATCH; ++e) {
        const int64_t t = t0 + e * step;
        if (t >= a.T) continue;
        const uint32_t s = q4_scales(scale[e]), s2 = __byte_perm(s, s, 0x1010);
        Q4Group<T> g;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t r[4];
          q4_pairs(w ? codes[e].y : codes[e].x, r);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t y = q4_mul2(r[k], s2);  // (exact)
            const float2 v = __half22float2(reinterpret_cast<const __half2&>(y));
            q4_put(g, 8 * w + 2 * k, v.x, v.y);
          }
        }
        uint8_t* dst = p.row + t * a.row_token[p.kv];
        if (a.wide) {
#pragma unroll
          for (int w = 0; w < Q4Group<T>::WORDS; w += 2) ta_store32(reinterpret_cast<bf16*>(dst + 16 * w), &g.w[w].x);
        } else {
#pragma unroll
          for (int w = 0; w < Q4Group<T>::WORDS; ++w) reinterpret_cast<uint4*>(dst)[w] = g.w[w];
        }
      }
    }
  }
}

// ---------------------------------------------------------------- host
int io_bytes(const paged_shape* s) { return s->io == RGLRU_BF16 ? 2 : 4; }

rglru_status check_heads(const paged_shape* s) {
  if (s->Hkv < 1 || s->D < 1 || (s->io != RGLRU_F32 && s->io != RGLRU_BF16)) return RGLRU_ERR_INVALID_ARG;
  if (s->D < 16 || s->D > 256 || s->D % 16) return RGLRU_ERR_UNSUPPORTED;
  return RGLRU_OK;
}

rglru_status check_queries(const paged_shape* s) {
  if (s->Hq < 1 || s->Hq % s->Hkv || s->window < 0) return RGLRU_ERR_INVALID_ARG;
  if (s->Hq / s->Hkv > 64) return RGLRU_ERR_UNSUPPORTED;
  return RGLRU_OK;
}

paged_q4_strides strides_of(const paged_shape* s, const paged_q4_strides* given) {
  if (given) return *given;
  paged_q4_strides t;
  t.q_token = t.o_token = (int64_t)s->Hq * s->D;
  t.k_token = t.v_token = (int64_t)s->Hkv * s->D;
  t.q_head = t.o_head = t.k_head = t.v_head = s->D;
  t.kc_token = t.vc_token = (s->D / 2 + 15) / 16 * 16;
  t.ks_token = t.vs_token = (s->D / 16 + 3) / 4 * 4;
  t.kc_head = t.vc_head = s->page_size * t.kc_token;
  t.ks_head = t.vs_head = s->page_size * t.ks_token;
  t.kc_page = t.vc_page = s->Hkv * t.kc_head;
  t.ks_page = t.vs_page = s->Hkv * t.ks_head;
  return t;
}

// Strides are positive multiples of `n` bytes.
bool strides_ok(int64_t size, int64_t n, std::initializer_list<int64_t> v) {
  for (int64_t x : v)
    if (x <= 0 || x * size % n) return false;
  return true;
}

bool cache_strides_ok(const paged_q4_strides& t) {
  for (int64_t x : {t.kc_page, t.kc_token, t.vc_page, t.vc_token, t.ks_page, t.ks_token, t.vs_page, t.vs_token})
    if (x >= (int64_t)1 << 32) return false;  // (multiplied in 32 bits, to 64)
  return strides_ok(1, 16, {t.kc_page, t.kc_token, t.kc_head, t.vc_page, t.vc_token, t.vc_head}) &&
         strides_ok(1, 4, {t.ks_page, t.ks_token, t.ks_head, t.vs_page, t.vs_token, t.vs_head});
}

int mean_rows(const paged_shape* s) {
  return (int)std::min<int64_t>(((int64_t)s->tokens + s->num_seqs - 1) / s->num_seqs * (s->Hq / s->Hkv), 1 << 30);
}

// Which of the two kernels.
bool many_rows(const paged_shape* s) {
  return mean_rows(s) > (s->D <= 128 ? TQ_FEW_ROWS : s->io == RGLRU_BF16 ? TQ_FEW_ROWS_WIDE : TQ_FEW_ROWS_WIDE_F32);
}

// Write (k and v read) and read (k and v written).
rglru_status rows_call(const paged_shape* s, const paged_q4_strides* strides, const void* k, const void* v, const int64_t* slots,
                       const void* kc, const void* ks, const void* vc, const void* vs, bool write, cudaStream_t stream) {
  rglru_status st = pg_check_cache(s);
  if (st == RGLRU_OK) st = check_heads(s);
  if (st != RGLRU_OK) return st;
  if (s->tokens == 0) return RGLRU_OK;
  if (!req(k) || !req(v) || !pg_aligned(slots, 8) || !req(kc) || !pg_aligned(ks, 4) || !req(vc) || !pg_aligned(vs, 4))
    return RGLRU_ERR_INVALID_ARG;
  const paged_q4_strides t = strides_of(s, strides);
  const int es = io_bytes(s);
  if (!strides_ok(es, 16, {t.k_token, t.k_head, t.v_token, t.v_head}) || !cache_strides_ok(t)) return RGLRU_ERR_UNSUPPORTED;
  Q4RowArgs a;
  a.T = s->tokens;
  a.head_groups = s->D / 16;
  if ((int64_t)s->Hkv * a.head_groups > 1 << 24) return RGLRU_ERR_UNSUPPORTED;  // (groups are counted in 32 bits)
  a.groups = s->Hkv * (int)a.head_groups;
  a.s_log2 = pg_log2(s->page_size);
  for (a.lanes_log2 = 0; a.lanes_log2 < 5 && 1 << a.lanes_log2 < a.groups;) ++a.lanes_log2;
  a.units = 2 * ((a.groups + (1 << a.lanes_log2) - 1) >> a.lanes_log2);
  a.wide = 1;
  a.slots_end = (int64_t)s->num_pages * s->page_size;
  a.slots = slots;
  const void* ptr[2][3] = {{k, kc, ks}, {v, vc, vs}};
  const int64_t str[2][8] = {{t.k_token, t.k_head, t.kc_page, t.kc_token, t.kc_head, t.ks_page, t.ks_token, t.ks_head},
                             {t.v_token, t.v_head, t.vc_page, t.vc_token, t.vc_head, t.vs_page, t.vs_token, t.vs_head}};
  for (int i = 0; i < 2; ++i) {
    a.row[i] = const_cast<uint8_t*>(static_cast<const uint8_t*>(ptr[i][0]));
    a.codes[i] = const_cast<uint8_t*>(static_cast<const uint8_t*>(ptr[i][1]));
    a.scales[i] = const_cast<uint8_t*>(static_cast<const uint8_t*>(ptr[i][2]));
    a.wide = a.wide && (reinterpret_cast<uintptr_t>(ptr[i][0]) | str[i][0] * es | str[i][1] * es) % 32 == 0;
    a.row_token[i] = str[i][0] * es;
    a.row_head[i] = str[i][1] * es;
    a.c_page[i] = str[i][2];
    a.c_token[i] = str[i][3];
    a.c_head[i] = str[i][4];
    a.s_page[i] = str[i][5];
    a.s_token[i] = str[i][6];
    a.s_head[i] = str[i][7];
  }
  // few tokens: one a lane, over many SMs
  const int64_t per = Q4_THREADS >> a.lanes_log2, batch = es == 2 ? Q4_BATCH<bf16> : Q4_BATCH<float>;
  const int y = std::min(a.units, 1 << 15);
  const int64_t most = (a.T + per - 1) / per, least = (a.T + per * batch - 1) / (per * batch);
  const int blocks = (int)std::max(least, std::min<int64_t>(most, (608 + y - 1) / y));
  const void* f = write ? (es == 2 ? reinterpret_cast<const void*>(k_paged_q4_write<bf16>) : reinterpret_cast<const void*>(k_paged_q4_write<float>))
                        : (es == 2 ? reinterpret_cast<const void*>(k_paged_q4_read<bf16>) : reinterpret_cast<const void*>(k_paged_q4_read<float>));
  void* args[] = {&a};
  return cuda_status(launch_pdl(f, dim3(blocks, y), dim3(Q4_THREADS), 0, stream, args, 1));
}

}  // namespace

}  // namespace rglru

using namespace rglru;

extern "C" rglru_status paged_q4_write(const paged_shape* s, const paged_q4_strides* strides, const void* k, const void* v,
                                       const int64_t* slots, void* k_codes, void* k_scales, void* v_codes, void* v_scales,
                                       rglru_stream stream) {
  return rows_call(s, strides, k, v, slots, k_codes, k_scales, v_codes, v_scales, true, stream);
}

extern "C" rglru_status paged_q4_read(const paged_shape* s, const paged_q4_strides* strides, const int64_t* slots,
                                      const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                                      void* k, void* v, rglru_stream stream) {
  return rows_call(s, strides, k, v, slots, k_codes, k_scales, v_codes, v_scales, false, stream);
}

extern "C" size_t paged_q4_attention_workspace_bytes(const paged_shape* s) {
  if (pg_check_cache(s) != RGLRU_OK || check_heads(s) != RGLRU_OK || check_queries(s) != RGLRU_OK) return 0;
  return many_rows(s) ? paged_attn_q4_tc_ws_bytes(s, mean_rows(s)) : paged_attn_q4_ws_bytes(s, mean_rows(s));
}

extern "C" rglru_status paged_q4_attention(const paged_shape* s, const paged_q4_strides* strides, const void* q,
                                           const void* k_codes, const void* k_scales, const void* v_codes,
                                           const void* v_scales, const int32_t* block_table, const int32_t* cu_seqlens,
                                           const int32_t* kv_lens, float scale, void* o, float* lse, void* workspace,
                                           rglru_stream stream) {
  rglru_status st = pg_check_cache(s);
  if (st == RGLRU_OK) st = check_heads(s);
  if (st == RGLRU_OK) st = check_queries(s);
  if (st != RGLRU_OK) return st;
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!(scale > 0.0f) || !isfinite(scale_log2)) return RGLRU_ERR_INVALID_ARG;
  if (s->tokens == 0) return RGLRU_OK;
  if (!req(q) || !req(k_codes) || !pg_aligned(k_scales, 4) || !req(v_codes) || !pg_aligned(v_scales, 4) ||
      !pg_aligned(block_table, 4) || !pg_aligned(cu_seqlens, 4) || !pg_aligned(kv_lens, 4) || !req(o) ||
      (lse && !pg_aligned(lse, 4)) || !req(workspace))
    return RGLRU_ERR_INVALID_ARG;
  const paged_q4_strides t = strides_of(s, strides);
  if (!strides_ok(io_bytes(s), 16, {t.q_token, t.q_head, t.o_token, t.o_head}) || !cache_strides_ok(t)) return RGLRU_ERR_UNSUPPORTED;
  PagedArgs a = {};
  a.N = s->num_seqs;
  a.T = s->tokens;
  a.Hq = s->Hq;
  a.Hkv = s->Hkv;
  a.g = s->Hq / s->Hkv;
  a.g_inv = (65536u + a.g - 1) / a.g;
  a.D = s->D;
  a.P = s->num_pages;
  a.ps_log2 = pg_log2(s->page_size);
  a.table_width = s->table_width;
  a.window = s->window < 1 << 30 ? s->window : 0;  // (lengths are clamped to 2^30)
  a.scale_log2 = scale_log2;
  a.q = q;
  a.table = block_table;
  a.cu = cu_seqlens;
  a.kv_lens = kv_lens;
  a.o = o;
  a.lse = lse;
  a.q_token = t.q_token;
  a.q_head = t.q_head;
  a.o_token = t.o_token;
  a.o_head = t.o_head;
  a.ws = static_cast<uint8_t*>(workspace);
  // rglru_debug_lookback: the limit in polls, taken as 100 ns each, and the CTA without work
  a.drop_cta = debug_drop_tile();
  a.wait_ns = a.drop_cta >= 0 ? (uint64_t)debug_spin_limit() * 100 : TA_WAIT_NS;
  const Q4Cache c = {static_cast<const uint8_t*>(k_codes), static_cast<const uint8_t*>(k_scales), static_cast<const uint8_t*>(v_codes),
                     static_cast<const uint8_t*>(v_scales), t.kc_page, t.kc_token, t.kc_head, t.vc_page, t.vc_token, t.vc_head,
                     t.ks_page, t.ks_token, t.ks_head, t.vs_page, t.vs_token, t.vs_head, 0, 1};
  if (many_rows(s)) return cuda_status(launch_paged_attn_q4_tc(a, c, s->io == RGLRU_F32, mean_rows(s), stream));
  return cuda_status(launch_paged_attn_q4(a, c, s->io == RGLRU_F32, mean_rows(s), stream));
}

// The cache held in 4 bits (include/paged_q4.h): the write of new keys and values, the read, and
// the host side of the attention.
#include <math.h>

#include <algorithm>

#include "host_util.h"
#include "paged_q4.cuh"

namespace rglru {

namespace {

// ---------------------------------------------------------------- write and read
// A lane takes a group: 16 channels of a token's head, keys' groups first, then values'.  A token's
// groups are spread over the lanes of a warp, or of a part of one where it has few.  Bound by memory
// bandwidth, and by latency for few tokens.
struct Q4RowArgs {
  int T, Hkv, groups, s_log2, lanes_log2;  // groups of a token's keys; lanes of a token
  uint32_t head_groups;                    // groups of a head
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

// A group's codes and scale.  The largest is found among the bits without signs: an infinity's are
// above all finite ones', a NaN's above those.  x / s is needed to the last bit only near a border
// between two codes, s times a number of at most 3 bits, which x may equal; so it is rounded
// correctly, by one step of Newton's method on the product with 1 / s (Markstein, 1990).
template <class T>
__device__ __forceinline__ uint2 q4_quantise(const Q4Group<T>& g, uint8_t& scale) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(q4_get(g, i)) & 0x7fffffffu);
  if (top >= 0x7f800000u) {
    scale = 0x7f;  // NaN
    return make_uint2(0u, 0u);
  }
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(__fdiv_rn(__uint_as_float(top), 6.0f)));
  const uint32_t code = max((uint32_t)two & 0xffu, 1u);  // 1: 2^-9
  const uint32_t h = q4_scales(code);
  const float s = __half2float(reinterpret_cast<const __half2&>(h).x), r = __frcp_rn(s);
  scale = (uint8_t)code;
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    float q[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float x = q4_get(g, i + e), y = x * r;
      q[e] = copysignf(fmaf(fmaf(-y, s, x), r, y), x);  // (a zero keeps its sign)
    }
    uint32_t b;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(b) : "f"(q[1]), "f"(q[0]));
    out[i / 8] |= b << i % 8 * 4;
  }
  return make_uint2(out[0], out[1]);
}

// Where group i of a token lies: keys or values, its row's bytes, its code's and scale's in the slot.
struct Q4Place {
  int kv, b;
  int64_t row, code, scale;
};
template <class T>
__device__ __forceinline__ Q4Place q4_place(const Q4RowArgs& a, int64_t t, int64_t page, int64_t off, int i) {
  Q4Place p;
  p.kv = i >= a.groups;
  const int c = p.kv ? i - a.groups : i, h = c / a.head_groups, b = c - h * a.head_groups;
  p.b = b;
  p.row = t * a.row_token[p.kv] + h * a.row_head[p.kv] + b * (16 * (int)sizeof(T));
  p.code = page * a.c_page[p.kv] + off * a.c_token[p.kv] + h * a.c_head[p.kv] + b * 8;
  p.scale = page * a.s_page[p.kv] + off * a.s_token[p.kv] + h * a.s_head[p.kv] + b;
  return p;
}

template <class T>
__global__ void __launch_bounds__(Q4_THREADS) k_paged_q4_write(const __grid_constant__ Q4RowArgs a) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  constexpr int BATCH = sizeof(T) == 2 ? 4 : 2;  // groups of a lane in flight
  const int lanes = 1 << a.lanes_log2, lane = threadIdx.x & (lanes - 1);
  const int64_t step = (int64_t)gridDim.x * Q4_THREADS >> a.lanes_log2;
  for (int64_t t = ((int64_t)blockIdx.x * Q4_THREADS + threadIdx.x) >> a.lanes_log2; t < a.T; t += step) {
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.slots_end) continue;
    const int64_t page = slot >> a.s_log2, off = slot & ((1 << a.s_log2) - 1);
    for (int i0 = lane; i0 < 2 * a.groups; i0 += lanes * BATCH) {
      Q4Group<T> g[BATCH];
      Q4Place p[BATCH];
#pragma unroll
      for (int e = 0; e < BATCH; ++e) {
        const int i = i0 + lanes * e;
        if (i >= 2 * a.groups) continue;
        p[e] = q4_place<T>(a, t, page, off, i);
        const uint4* src = reinterpret_cast<const uint4*>(a.row[p[e].kv] + p[e].row);
#pragma unroll
        for (int w = 0; w < Q4Group<T>::WORDS; ++w) g[e].w[w] = src[w];
      }
#pragma unroll
      for (int e = 0; e < BATCH; ++e) {
        if (i0 + lanes * e >= 2 * a.groups) continue;
        uint8_t scale;
        const uint2 codes = q4_quantise(g[e], scale);
        *reinterpret_cast<uint2*>(a.codes[p[e].kv] + p[e].code) = codes;
        a.scales[p[e].kv][p[e].scale] = scale;
      }
    }
  }
}

__device__ __forceinline__ void q4_put(Q4Group<bf16>& g, int i, float lo, float hi) { (&g.w[i / 8].x)[i / 2 % 4] = ta_pack(lo, hi); }
__device__ __forceinline__ void q4_put(Q4Group<float>& g, int i, float lo, float hi) {
  (&g.w[i / 4].x)[i % 4] = __float_as_uint(lo);
  (&g.w[i / 4].x)[i % 4 + 1] = __float_as_uint(hi);
}

template <class T>
__global__ void __launch_bounds__(Q4_THREADS) k_paged_q4_read(const __grid_constant__ Q4RowArgs a) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  constexpr int BATCH = 4;
  const int lanes = 1 << a.lanes_log2, lane = threadIdx.x & (lanes - 1);
  const int64_t step = (int64_t)gridDim.x * Q4_THREADS >> a.lanes_log2;
  for (int64_t t = ((int64_t)blockIdx.x * Q4_THREADS + threadIdx.x) >> a.lanes_log2; t < a.T; t += step) {
    const int64_t slot = a.slots[t];
    const bool there = slot >= 0 && slot < a.slots_end;
    const int64_t page = there ? slot >> a.s_log2 : 0, off = there ? slot & ((1 << a.s_log2) - 1) : 0;
    for (int i0 = lane; i0 < 2 * a.groups; i0 += lanes * BATCH) {
      uint2 codes[BATCH];
      uint32_t scale[BATCH];
      Q4Place p[BATCH];
#pragma unroll
      for (int e = 0; e < BATCH; ++e) {
        const int i = i0 + lanes * e;
        codes[e] = make_uint2(0u, 0u);
        scale[e] = 0u;
        if (i >= 2 * a.groups) continue;
        p[e] = q4_place<T>(a, t, page, off, i);
        if (!there) continue;
        codes[e] = *reinterpret_cast<const uint2*>(a.codes[p[e].kv] + p[e].code);
        scale[e] = a.scales[p[e].kv][p[e].scale];
      }
#pragma unroll
      for (int e = 0; e < BATCH; ++e) {
        if (i0 + lanes * e >= 2 * a.groups) continue;
        const uint32_t h = q4_scales(scale[e]);
        const float s = __half2float(reinterpret_cast<const __half2&>(h).x);
        Q4Group<T> g;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t r[4];
          q4_pairs(w ? codes[e].y : codes[e].x, r);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 v = __half22float2(reinterpret_cast<const __half2&>(r[k]));
            q4_put(g, 8 * w + 2 * k, v.x * s, v.y * s);
          }
        }
        uint4* dst = reinterpret_cast<uint4*>(a.row[p[e].kv] + p[e].row);
#pragma unroll
        for (int w = 0; w < Q4Group<T>::WORDS; ++w) dst[w] = g.w[w];
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

// Which of the two kernels (paged_attention's rule for a bf16 cache, at half as many rows).
bool many_rows(const paged_shape* s) { return s->io == RGLRU_BF16 && mean_rows(s) > TQ_FEW_ROWS; }

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
  a.Hkv = s->Hkv;
  a.head_groups = s->D / 16;
  if ((int64_t)s->Hkv * a.head_groups > 1 << 24) return RGLRU_ERR_UNSUPPORTED;  // (groups are counted in 32 bits)
  a.groups = s->Hkv * (int)a.head_groups;
  a.s_log2 = pg_log2(s->page_size);
  a.lanes_log2 = std::min(5, pg_log2(2 * a.groups));
  a.slots_end = (int64_t)s->num_pages * s->page_size;
  a.slots = slots;
  const void* ptr[2][3] = {{k, kc, ks}, {v, vc, vs}};
  const int64_t str[2][8] = {{t.k_token, t.k_head, t.kc_page, t.kc_token, t.kc_head, t.ks_page, t.ks_token, t.ks_head},
                             {t.v_token, t.v_head, t.vc_page, t.vc_token, t.vc_head, t.vs_page, t.vs_token, t.vs_head}};
  for (int i = 0; i < 2; ++i) {
    a.row[i] = const_cast<uint8_t*>(static_cast<const uint8_t*>(ptr[i][0]));
    a.codes[i] = const_cast<uint8_t*>(static_cast<const uint8_t*>(ptr[i][1]));
    a.scales[i] = const_cast<uint8_t*>(static_cast<const uint8_t*>(ptr[i][2]));
    a.row_token[i] = str[i][0] * es;
    a.row_head[i] = str[i][1] * es;
    a.c_page[i] = str[i][2];
    a.c_token[i] = str[i][3];
    a.c_head[i] = str[i][4];
    a.s_page[i] = str[i][5];
    a.s_token[i] = str[i][6];
    a.s_head[i] = str[i][7];
  }
  const int per = Q4_THREADS >> a.lanes_log2;
  const int blocks = (int)std::min<int64_t>(((int64_t)a.T + per - 1) / per, 1 << 16);
  const void* f = write ? (es == 2 ? reinterpret_cast<const void*>(k_paged_q4_write<bf16>) : reinterpret_cast<const void*>(k_paged_q4_write<float>))
                        : (es == 2 ? reinterpret_cast<const void*>(k_paged_q4_read<bf16>) : reinterpret_cast<const void*>(k_paged_q4_read<float>));
  void* args[] = {&a};
  return cuda_status(launch_pdl(f, dim3(blocks), dim3(Q4_THREADS), 0, stream, args, 1));
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
  return many_rows(s) ? paged_attn_q4_tc_ws_bytes(s) : paged_attn_q4_ws_bytes(s, mean_rows(s));
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
  if (many_rows(s)) return cuda_status(launch_paged_attn_q4_tc(a, c, stream));
  return cuda_status(launch_paged_attn_q4(a, c, s->io == RGLRU_F32, mean_rows(s), stream));
}

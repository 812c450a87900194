// Device and host helpers shared by the attention and cache kernels
// (entro_attn_prompt.hip, entro_kv.hip, entro_attn_cache.hip): element types,
// matrix-core fragments, reductions, and the search that turns a workgroup's
// number into a place in one of the call's sequences.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "entro_attn.h"
#include "entro_device.h"

namespace entro {

typedef __bf16 bf16v8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16v8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.4426950408889634f;

// The two 16-bit element types.  pack2 rounds two floats to nearest even into
// one word, the first in the low half; add2 adds both values of a word to a
// float, in 32 bits.  kInf: the magnitude bits from which a
// value is infinite or NaN.
template <entro_dtype T>
struct Elem;
template <>
struct Elem<ENTRO_BF16> {
  typedef __bf16 type;
  typedef bf16v8 v8;
  static constexpr uint32_t kInf = 0x7F80u;
  __device__ static float lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
  __device__ static float hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
  __device__ static uint32_t pack2(float a, float b) {
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, v2));
  }
  __device__ static float add2(uint32_t w, float c) {
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2, w), __builtin_bit_cast(v2, 0x3F803F80u), c, false);
  }
  __device__ static f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
};
template <>
struct Elem<ENTRO_F16> {
  typedef _Float16 type;
  typedef f16v8 v8;
  typedef _Float16 v2 __attribute__((ext_vector_type(2)));
  static constexpr uint32_t kInf = 0x7C00u;
  __device__ static float lo(uint32_t w) { return (float)__builtin_bit_cast(v2, w).x; }
  __device__ static float hi(uint32_t w) { return (float)__builtin_bit_cast(v2, w).y; }
  __device__ static uint32_t pack2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, v2));
  }
  __device__ static float add2(uint32_t w, float c) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(v2, w), __builtin_bit_cast(v2, 0x3C003C00u), c, false);
  }
  __device__ static f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
};

// 2^x in one instruction (x below -126 gives a denormal or 0)
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Maximum or sum over the lane pairs 32 (16) apart, in both lanes.
__device__ __forceinline__ float max32(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float add32(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}
__device__ __forceinline__ float max16(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float add16(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// Factor of a part with maximum m where the parts' is `all`: parts without
// tokens (both -inf) count with their zeros, NaN passes through.
__device__ __forceinline__ float join_factor(float m, float all) { return m == all ? 1.0f : exp2_fast(m - all); }

// Inclusive running sum (maximum) over the wavefront's lanes: within rows of 16
// by shifts, then the rows' ends to the rows after (vector instructions only;
// all lanes active).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp0(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += dpp0<0x111, 0xF>(v);   // row_shr:1, 2, 4, 8
  v += dpp0<0x112, 0xF>(v);
  v += dpp0<0x114, 0xF>(v);
  v += dpp0<0x118, 0xF>(v);
  v += dpp0<0x142, 0xA>(v);   // row_bcast:15 into rows 1 and 3
  v += dpp0<0x143, 0xC>(v);   // row_bcast:31 into rows 2 and 3
  return v;
}
__device__ __forceinline__ uint32_t wave_max_scan(uint32_t v) {
  v = max(v, dpp0<0x111, 0xF>(v));
  v = max(v, dpp0<0x112, 0xF>(v));
  v = max(v, dpp0<0x114, 0xF>(v));
  v = max(v, dpp0<0x118, 0xF>(v));
  v = max(v, dpp0<0x142, 0xA>(v));
  v = max(v, dpp0<0x143, 0xC>(v));
  return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) { return __builtin_amdgcn_readlane(wave_max_scan(v), 63); }

// The sequence whose items include number `item` when the sequences' items are
// numbered one after another, and the item's number within it.  Every lane of the
// wavefront returns the same; seq = n_seq where there are fewer items.  64
// sequences a step: count(b0) is the number of items of sequence b0 + lane (0 past
// the last), b0 = 0, 64, ... in turn, all lanes active; all of them together are
// below 2^32.
struct Found {
  uint32_t seq, local;
};
template <typename Count>
__device__ __forceinline__ Found find_item(uint32_t item, uint32_t n_seq, uint32_t lane, Count count) {
  uint32_t before = 0;
  for (uint32_t b0 = 0; b0 < n_seq; b0 += 64u) {
    const uint32_t own = count(b0);
    const uint32_t run = wave_scan(own);
    const uint64_t past = __ballot(before + run > item);
    if (past) {
      const uint32_t at = (uint32_t)__builtin_ctzll(past);
      return {rfl(b0 + at), rfl(item - before - __builtin_amdgcn_readlane(run - own, at))};
    }
    before += __builtin_amdgcn_readlane(run, 63);
  }
  return {n_seq, 0u};
}

// All sequences' items together.
template <typename Count>
__device__ __forceinline__ uint32_t count_items(uint32_t n_seq, Count count) {
  uint32_t sum = 0;
  for (uint32_t b0 = 0; b0 < n_seq; b0 += 64u) sum += __builtin_amdgcn_readlane(wave_scan(count(b0)), 63);
  return sum;
}

// Rows of sequence b from its running sums, with what is wrong with them.
struct Span {
  uint32_t begin, count;
  bool ok;
};
__device__ __forceinline__ Span span_of(const int32_t *cu, uint32_t b, uint32_t total) {
  const int32_t lo = cu[b], hi = cu[b + 1];
  const bool ok = lo >= 0 && hi >= lo && (uint32_t)hi <= total;
  return {ok ? (uint32_t)lo : 0u, ok ? (uint32_t)(hi - lo) : 0u, ok};
}

// Rows of the sequences b0 + lane (b0 = 0, 64, ... in turn, all lanes active) that
// are written or taken as new: no row belongs to two sequences, so one that begins
// before an earlier one's end is wrong, and the rows of all others together are no
// more than there are (which bounds the items that are counted from them).
struct Spans {
  const int32_t *cu;
  uint32_t total, n_seq, lane, end;   // end: the largest sum so far
  __device__ Spans(const int32_t *sums, uint32_t rows, uint32_t n, uint32_t lane_)
      : cu(sums), total(rows), n_seq(n), lane(lane_), end(0u) {}
  // b0 + lane or, past the last sequence, the last: what is read of it without a
  // branch is on its way together with what else the caller reads
  __device__ uint32_t place(uint32_t b0) const { return min(b0 + lane, n_seq - 1u); }
  __device__ Span at(uint32_t b0) {
    if (b0 == 0u) end = 0u;
    const uint32_t b = place(b0);
    const uint32_t lo = (uint32_t)cu[b], hi = (uint32_t)cu[b + 1u];   // negative: past all rows
    const uint32_t run = max(end, wave_max_scan(lo <= total ? lo : 0u));
    end = __builtin_amdgcn_readlane(run, 63);
    const bool ok = b0 + lane < n_seq && lo <= hi && hi <= total && lo >= run;
    return {ok ? lo : 0u, ok ? hi - lo : 0u, ok};
  }
};

// Workgroup cap of the attention's and cache's launches
// (entro_attn_set_max_workgroups; 0: none).
inline std::atomic<uint32_t> g_attn_max_workgroups{0};

// host side: a grid of x by y workgroups (x going fastest), fewer where the
// cap says so or the launch cannot have as many: the kernels step through both
// by the grid's extent.
inline dim3 grid2(uint64_t x, uint64_t y) {
  const uint64_t gx = std::min<uint64_t>(std::max<uint64_t>(x, 1), 1u << 24);
  const uint64_t gy = std::min<uint64_t>(std::max<uint64_t>(y, 1), 65535u);
  const uint32_t cap = g_attn_max_workgroups.load(std::memory_order_relaxed);
  const uint64_t most = cap ? std::min<uint64_t>(gx * gy, cap) : gx * gy, cx = std::min(gx, most);
  return dim3((uint32_t)cx, (uint32_t)std::min(gy, std::max<uint64_t>(most / cx, 1)));
}

// host side: one 16-bit operand
inline entro_status check_rows(const entro_rows &r, uint32_t rows) {
  if (rows == 0) return ENTRO_OK;
  if (!r.d || (reinterpret_cast<uintptr_t>(r.d) & 15u)) return ENTRO_E_INVAL;
  if ((r.stride_t & 7) || (r.stride_h & 7)) return ENTRO_E_INVAL;
  if (r.stride_t < 0 || r.stride_h < 0) return ENTRO_E_INVAL;
  return ENTRO_OK;
}

inline bool head_dim_ok(uint32_t d) { return d == 64u || d == 96u || d == 128u; }

inline entro_status check_heads(uint32_t n_heads, uint32_t n_kv, uint32_t dim, int dtype) {
  if (n_heads == 0 || n_kv == 0 || n_heads % n_kv) return ENTRO_E_INVAL;
  if (dtype != ENTRO_BF16 && dtype != ENTRO_F16) return ENTRO_E_INVAL;
  if (!head_dim_ok(dim) || n_heads > 65535u) return ENTRO_E_UNSUPPORTED;
  return ENTRO_OK;
}

inline entro_status check_cache(const entro_kv_cache *c, const entro_kv_table *t) {
  if (!c || !t) return ENTRO_E_INVAL;
  if (t->n_seq == 0) return ENTRO_OK;
  if (c->page_tokens != 16u && c->page_tokens != 32u && c->page_tokens != 64u && c->page_tokens != 128u)
    return ENTRO_E_FORMAT;
  if (!head_dim_ok(c->head_dim) || c->n_kv_heads > 65535u) return ENTRO_E_UNSUPPORTED;
  if (c->n_kv_heads == 0 || c->n_pages == 0 || c->n_pages > 0x7FFFFFFFu) return ENTRO_E_INVAL;
  if (!c->d_k_codes || !c->d_v_codes || !c->d_k_scales || !c->d_v_scales || !t->d_table) return ENTRO_E_INVAL;
  if ((reinterpret_cast<uintptr_t>(c->d_k_codes) | reinterpret_cast<uintptr_t>(c->d_v_codes)) & 15u)
    return ENTRO_E_INVAL;
  if (t->table_pages == 0 || t->table_pages > t->table_stride) return ENTRO_E_INVAL;
  // positions are 31-bit numbers
  if ((uint64_t)t->table_pages * c->page_tokens > 0x7FFFFFFFull || t->n_seq > 0x7FFFFFFFu) return ENTRO_E_UNSUPPORTED;
  return ENTRO_OK;
}

}  // namespace entro

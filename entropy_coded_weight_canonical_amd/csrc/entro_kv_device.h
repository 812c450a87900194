// Device code that the kernels which write or read pages of the 8-bit cache share
// (entro_kv.hip, entro_rope.hip): a workgroup's page, and the arithmetic of its
// codes.  The cache's layout and definition are in entro_attn.h.
#pragma once

#include "entro_attn_device.h"
#include "entro_internal.h"

namespace entro {

// Keys or values.
struct KvSide {
  int8_t *codes;
  float *scales;
  char *x;                     // rows of the call's type (written by the load)
  int64_t stride_t, stride_h;  // bytes
};
struct KvArg {
  KvSide side[2];              // keys, values
  const int32_t *table;
  uint64_t table_stride;
  uint32_t table_pages, n_seq, n_pages, n_kv;
  uint64_t items;              // pages that the call can have
  const int32_t *pos;          // [n_seq] tokens held (store), first position (load)
  const int32_t *cu;           // [n_seq + 1]
  uint32_t total;
  uint32_t *status;
};

// A sequence's part in a call: rows begin .. begin + count - 1 of the packed
// operands are its positions pos .. pos + count - 1.
struct KvSpan {
  uint32_t begin, count, pos;
  bool ok;
};
// of sequence b0 + lane, 64 in turn
__device__ __forceinline__ KvSpan kv_span(const KvArg &a, Spans &spans, uint32_t b0, uint32_t page) {
  const int32_t p = a.pos[spans.place(b0)];
  const Span s = spans.at(b0);
  const bool ok = s.ok && p >= 0 && (uint64_t)p + s.count <= (uint64_t)a.table_pages * page;
  return {s.begin, ok ? s.count : 0u, ok ? (uint32_t)p : 0u, ok};
}
__device__ __forceinline__ uint32_t kv_pages(const KvSpan &s, uint32_t page) {
  return s.count ? (s.pos + s.count - 1u) / page - s.pos / page + 1u : 0u;
}

// Marks the sequences whose lengths do not fit (one wavefront of the call).
__device__ __forceinline__ void kv_check(const KvArg &a, uint32_t page) {
  if (threadIdx.x >= 64u) return;
  Spans spans(a.cu, a.total, a.n_seq, threadIdx.x);
  for (uint32_t b0 = 0; b0 < a.n_seq; b0 += 64u) {
    const bool ok = kv_span(a, spans, b0, page).ok;
    if (b0 + threadIdx.x < a.n_seq && !ok) atomicOr(a.status + b0 + threadIdx.x, ENTRO_F_LENGTH);
  }
}

// What a workgroup does: one page (the sequences' pages that take part are
// numbered one after another) for one head, keys and values.  In the store and the load
// neighbouring workgroups take the pages of one head: with the heads of one page side by
// side, reading 58371 tokens back took 98 us instead of 74.  (The append, which has
// queries between them, takes the heads of one page: see kv_append_kernel.)
struct KvItem {
  bool any;            // whether there is an item, and a page
  uint32_t head;
  uint32_t r0, r1;     // rows of the page that take part
  int64_t first;       // packed row of page row 0
  uint32_t place;      // place in its sequence of page row 0
  uint64_t at;         // place of the page's and head's scale
};
__device__ __forceinline__ KvItem kv_item(const KvArg &a, uint32_t page, uint32_t item, uint32_t head, uint32_t lane) {
  KvItem it{};
  KvSpan own{};   // of the sequence this lane looked at last
  Spans spans(a.cu, a.total, a.n_seq, lane);
  const Found f = find_item(item, a.n_seq, lane, [&](uint32_t b0) {
    own = kv_span(a, spans, b0, page);
    return kv_pages(own, page);
  });
  if (f.seq == a.n_seq) return it;
  const auto there = [&](uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, (int)(f.seq % 64u)); };
  const KvSpan s{there(own.begin), there(own.count), there(own.pos), true};
  const uint32_t index = s.pos / page + f.local;
  const int32_t page_id = a.table[(uint64_t)f.seq * a.table_stride + index];
  if (page_id < 0 || (uint32_t)page_id >= a.n_pages) {
    if (threadIdx.x == 0u && head == 0u) atomicOr(a.status + f.seq, ENTRO_F_PAGE);
    return it;
  }
  it.any = true;
  it.head = head;
  it.at = (uint64_t)page_id * a.n_kv + head;
  it.r0 = f.local == 0u ? s.pos % page : 0u;
  it.r1 = min(page, s.pos + s.count - index * page);
  it.place = index * page;
  it.first = (int64_t)s.begin + ((int64_t)index * page - (int64_t)s.pos);
  return it;
}

// Value of one code after x * r: rounded to even and limited; NaN gives 0.
// The code's two's complement is the low byte of what is returned.
__device__ __forceinline__ uint32_t code_of(float y) {
  y = y == y ? y : 0.0f;
  y = fminf(fmaxf(y, -127.0f), 127.0f);
  return __builtin_bit_cast(uint32_t, y + 12582912.0f);   // 1.5 * 2^23: rounds at the integer
}
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x0C0C0400u);
  const uint32_t cd = __builtin_amdgcn_perm(d, c, 0x0C0C0400u);
  return __builtin_amdgcn_perm(cd, ab, 0x05040100u);
}
__device__ __forceinline__ float byte_of(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

// Four codes multiplied by `ratio` and rounded again.
__device__ __forceinline__ uint32_t again4(uint32_t w, float ratio) {
  return pack4(code_of(byte_of(w, 0) * ratio), code_of(byte_of(w, 1) * ratio), code_of(byte_of(w, 2) * ratio),
               code_of(byte_of(w, 3) * ratio));
}

// Largest magnitude of the 16-bit values in w (their bits without the sign);
// FINITE leaves out infinities and NaN.
template <entro_dtype T, bool FINITE>
__device__ __forceinline__ uint32_t top_of(uint32_t w, uint32_t top) {
  uint32_t a = w & 0x7FFFu, b = (w >> 16) & 0x7FFFu;
  if (FINITE) {
    a = a < Elem<T>::kInf ? a : 0u;
    b = b < Elem<T>::kInf ? b : 0u;
  }
  return max(top, max(a, b));
}

constexpr uint32_t kWavesMost = 8;   // wavefronts of a workgroup, at most

// Largest of v over the workgroup.
__device__ __forceinline__ uint32_t wg_max(uint32_t v, uint32_t *red) {
  v = wave_max(v);
  const uint32_t waves = blockDim.x >> 6;
  if (waves > 1u) {
    __syncthreads();
    if ((threadIdx.x & 63u) == 0u) red[threadIdx.x >> 6] = v;
    __syncthreads();
    for (uint32_t w = 0; w < waves; ++w) v = max(v, red[w]);
  }
  return v;
}

// Four rows of four bytes turned to four columns of four.
__device__ __forceinline__ u32x4 turn4(uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  const uint32_t a = __builtin_amdgcn_perm(r1, r0, 0x05010400u), b = __builtin_amdgcn_perm(r1, r0, 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(r3, r2, 0x05010400u), d = __builtin_amdgcn_perm(r3, r2, 0x07030602u);
  return (u32x4){__builtin_amdgcn_perm(c, a, 0x05040100u), __builtin_amdgcn_perm(c, a, 0x07060302u),
                 __builtin_amdgcn_perm(d, b, 0x05040100u), __builtin_amdgcn_perm(d, b, 0x07060302u)};
}

// New scale of a page and the factors of new values and of codes held.
struct Grow {
  float scale, fresh, again;
};
__device__ __forceinline__ Grow grow(float before, float top) {
  const float s = fmaxf(before, top * (1.0f / 127.0f));
  const bool some = s >= 1.17549435e-38f;
  return {s, some ? 1.0f / s : 0.0f, some ? before / s : 0.0f};
}

}  // namespace entro

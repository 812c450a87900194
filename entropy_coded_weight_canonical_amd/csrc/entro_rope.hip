// HIP kernels (gfx950) and entry points of the rotary positions: entro_rope, and
// entro_kv_append, which writes rotated keys and values to the 8-bit cache.
// Definitions and the cache's layout are in entro_attn.h.
//
// Bound by memory; small calls by the launch and the chain of reads (lengths, table,
// operands).  Cosine and sine are computed where they are used, once for all heads that a
// thread takes: a table of them would be read and kept beside what it turns.  Measured on
// an MI355X (copy 4.8 TB/s): 32768 tokens, 32 / 32 heads of 96 in f16, 160 us, 5.0 TB/s;
// 32768 tokens appended with their queries, 32 / 8 heads of 128 in bf16, 154 us, 4.8 TB/s;
// 12 sequences of up to 1001 tokens, 32 heads of 96, pages of 32, 46 us, 3.0 TB/s; one
// token for each of 5 sequences turned 3.3 us, for each of 16 appended 10 us.  From 32 bits:
// 32768 tokens, 32 / 8 heads of 128, turned 190 us, 5.3 TB/s, appended 209 us, 5.5 TB/s (in
// pages of 128 233 us, 4.9).
#include <algorithm>
#include <type_traits>

#include "entro_kv_device.h"

namespace entro {

__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

struct RotArg {
  const float *freqs;
  uint32_t axes[4];
  uint32_t units;       // pairs / 8
  uint32_t n_axes;
  float gain;
  const int32_t *pos;   // null: a token's place in its sequence
  int64_t pos_stride;
};

// Input element types: eight operands' bits, and each as a float (after anew, computed
// again: floats from before are not kept in registers).
template <entro_dtype T>
struct In {
  static constexpr int kSize = 2;
  typedef u32x4 raw;
  __device__ static void anew(raw &r) { asm volatile("" : "+v"(r)); }
  __device__ static raw load(const char *p) { return *reinterpret_cast<const u32x4 *>(p); }
  __device__ static float get(const raw &r, int i) {
    return i & 1 ? Elem<T>::hi(r[i >> 1]) : Elem<T>::lo(r[i >> 1]);
  }
};
template <>
struct In<ENTRO_F32> {
  static constexpr int kSize = 4;
  struct raw {
    u32x4 a, b;
  };
  __device__ static void anew(raw &r) { asm volatile("" : "+v"(r.a), "+v"(r.b)); }
  __device__ static raw load(const char *p) {
    return {*reinterpret_cast<const u32x4 *>(p), *reinterpret_cast<const u32x4 *>(p + 16)};
  }
  __device__ static float get(const raw &r, int i) { return __builtin_bit_cast(float, i < 4 ? r.a[i & 3] : r.b[i & 3]); }
};

template <entro_dtype T>
__device__ __forceinline__ u32x4 pack8(const float *x) {
  return (u32x4){Elem<T>::pack2(x[0], x[1]), Elem<T>::pack2(x[2], x[3]), Elem<T>::pack2(x[4], x[5]),
                 Elem<T>::pack2(x[6], x[7])};
}

// A thread takes a head's elements in units of eight pairs: two pieces of eight
// neighbouring elements, x[j] of the one and x[8 + j] of the other being a pair
// (with INTER both pieces together hold the pairs side by side).  Units past the
// rotated pairs are two neighbouring pieces that stay as they are.
struct Unit {
  uint32_t c0, c1;   // first element of the pieces
  bool turned;
};
template <bool INTER>
__device__ __forceinline__ Unit unit_of(const RotArg &r, uint32_t u) {
  const bool turned = u < r.units;
  if (!INTER && turned) return {8u * u, 8u * (u + r.units), true};
  return {16u * u, 16u * u + 8u, turned};
}

// Cosine and sine of a unit's eight pairs at one token.  Whole turns are taken out of
// position * (freqs / (2 pi)) in 64 bits by a fused product, so that the rest, -1/2 ..
// 1/2, is off by no more than the factor is: 1.56 * 2^-53 of the angle, 2^-53 for its
// rounding and 0.56 * 2^-53 for that of 1 / (2 pi).  (With the factor as two 64-bit
// numbers it would be off by 2^-52 of a turn wherever, and rope_kernel take 4 % more where
// a thread has one head: 64-bit angles have the former error in any case.)  The cosine
// instruction takes the rest in 32 bits, off by 2^-26 of a turn (2^-23.3 as an angle), and
// is off by 2^-22.9 itself (over all 32-bit numbers of the range): together below 2^-22.
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ void turn_at(Turn &t, const RotArg &r, uint32_t u, int64_t row, uint32_t place) {
  constexpr double kTurn = 0.15915494309189533577;   // 1 / (2 pi)
  int32_t p[4];
  p[0] = r.pos ? r.pos[row] : (int32_t)place;
  if (r.n_axes > 1u)
#pragma unroll
    for (uint32_t a = 1; a < 4u; ++a) p[a] = r.pos ? r.pos[min(a, r.n_axes - 1u) * r.pos_stride + row] : p[0];
  const uint32_t bits = r.axes[u >> 1] >> (16u * (u & 1u));   // of pairs 8 u .. 8 u + 7
  const f32x4 f0 = *reinterpret_cast<const f32x4 *>(r.freqs + 8u * u), f1 = *reinterpret_cast<const f32x4 *>(r.freqs + 8u * u + 4u);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    int32_t at = p[0];
    if (r.n_axes > 1u) {
      const uint32_t a = (bits >> (2 * j)) & 3u;
      at = a == 0u ? p[0] : a == 1u ? p[1] : a == 2u ? p[2] : p[3];
    }
    const double by = (double)(j < 4 ? f0[j & 3] : f1[j & 3]) * kTurn, way = (double)at;
    const float y = (float)__builtin_fma(way, by, -__builtin_rint(way * by));
    t.c[j] = __builtin_amdgcn_cosf(y) * r.gain;
    t.s[j] = __builtin_amdgcn_sinf(y) * r.gain;
    if (j % 2) in_order();   // (eight at once take registers for eight products of 64 bits)
  }
}

// The unit's 16 elements rotated.
template <entro_dtype T, bool INTER>
__device__ __forceinline__ void turned16(float *x, const typename In<T>::raw &p0, const typename In<T>::raw &p1, const Turn &t,
                                         bool turned) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = In<T>::get(p0, j);
    x[8 + j] = In<T>::get(p1, j);
  }
  if (!turned) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int a = INTER ? 2 * j : j, b = INTER ? 2 * j + 1 : 8 + j;
    const float xa = x[a], xb = x[b];
    x[a] = xa * t.c[j] - xb * t.s[j];
    x[b] = xb * t.c[j] + xa * t.s[j];
  }
}

// Rows of queries and keys, a few heads at a time, a thread's own unit and token: cosine and sine are taken once for all its heads.
struct RowsArg {
  const char *x[2];         // queries, keys
  char *out[2];
  int64_t x_t[2], x_h[2], o_t[2], o_h[2];   // bytes
  uint32_t heads[2];
};
template <entro_dtype T, entro_dtype O, bool INTER>
__device__ __forceinline__ void turn_rows(const RowsArg &a, const RotArg &r, uint32_t u, int64_t row, uint32_t place,
                                          uint32_t head0, uint32_t step) {
  constexpr uint32_t kHeadsAhead = 8 / In<T>::kSize;   // heads whose loads go out together
  const Unit un = unit_of<INTER>(r, u);
  Turn t;
  if (un.turned) turn_at(t, r, u, row, place);
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const uint32_t heads = a.heads[side];
    const char *x = a.x[side] + row * a.x_t[side];
    char *out = a.out[side] + row * a.o_t[side];
    for (uint32_t h0 = head0; h0 < heads; h0 += step * kHeadsAhead) {
      typename In<T>::raw p0[kHeadsAhead], p1[kHeadsAhead];
#pragma unroll
      for (uint32_t i = 0; i < kHeadsAhead; ++i) {
        const char *from = x + min(h0 + i * step, heads - 1u) * a.x_h[side];
        p0[i] = In<T>::load(from + un.c0 * In<T>::kSize);
        p1[i] = In<T>::load(from + un.c1 * In<T>::kSize);
      }
#pragma unroll
      for (uint32_t i = 0; i < kHeadsAhead; ++i) {
        const uint32_t h = h0 + i * step;
        if (h >= heads) break;
        float v[16];
        turned16<T, INTER>(v, p0[i], p1[i], t, un.turned);
        char *to = out + h * a.o_h[side];
        *reinterpret_cast<u32x4 *>(to + un.c0 * 2u) = pack8<O>(v);
        *reinterpret_cast<u32x4 *>(to + un.c1 * 2u) = pack8<O>(v + 8);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// rope
// ---------------------------------------------------------------------------
struct RopeArg {
  RowsArg rows;
  RotArg rot;
  uint32_t total, tokens;   // tokens of a workgroup
};

constexpr uint32_t kRopeThreads = 256;

template <entro_dtype T, entro_dtype O, int D, bool INTER>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArg a) {
  constexpr uint32_t U = D / 16, S = kRopeThreads / U;   // units of a head, places for (token, head)
  const uint32_t u = threadIdx.x % U, slot = threadIdx.x / U;
  const uint32_t step = S / a.tokens, token = slot / step, head0 = slot % step;
  if (token >= a.tokens) return;
  for (uint64_t t0 = (uint64_t)blockIdx.x * a.tokens; t0 < a.total; t0 += (uint64_t)gridDim.x * a.tokens)
    if (t0 + token < a.total) turn_rows<T, O, INTER>(a.rows, a.rot, u, (int64_t)(t0 + token), 0u, head0, step);
}

// ---------------------------------------------------------------------------
// append: a workgroup takes one page and head as the cache's store does (there:
// four rows x eight columns a thread, one pass), here for the keys two rows x two
// pieces of eight columns a thread, whose pairs it holds; further workgroups
// rotate the queries.
// ---------------------------------------------------------------------------
struct AppendArg {
  KvArg kv;
  RotArg rot;
  RowsArg rows;             // queries at [0]
  uint32_t tokens;          // of a workgroup that rotates queries
  uint64_t q_items;         // such workgroups that the call can have
};

// The largest of a and of b over the workgroup.
__device__ __forceinline__ void wg_max2(uint32_t &a, uint32_t &b, uint32_t *red) {
  a = wave_max(a);
  b = wave_max(b);
  const uint32_t waves = blockDim.x >> 6;
  if (waves > 1u) {
    __syncthreads();
    if ((threadIdx.x & 63u) == 0u) {
      red[threadIdx.x >> 6] = a;
      red[kWavesMost + (threadIdx.x >> 6)] = b;
    }
    __syncthreads();
    for (uint32_t w = 0; w < waves; ++w) {
      a = max(a, red[w]);
      b = max(b, red[kWavesMost + w]);
    }
  }
}

__device__ __forceinline__ uint32_t bits_of(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu; }
// (infinities and NaN do not count)
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t b = bits_of(x);
  return b < 0x7F800000u ? b : 0u;
}

template <entro_dtype T, int D, bool INTER>
__device__ __forceinline__ void append_page(const AppendArg &arg, const KvItem &it, uint32_t page) {
  constexpr uint32_t U = D / 16, C = D / 8;
  const KvArg &a = arg.kv;
  uint8_t *vt = reinterpret_cast<uint8_t *>(dyn_lds);   // [D][page + 4]
  const uint32_t tid = threadIdx.x, vs = page + 4u;
  uint32_t *red = reinterpret_cast<uint32_t *>(vt + D * vs);   // [2][kWavesMost]
  // (rows before r0 are held, by these scales)
  const float k_before = it.r0 ? a.side[0].scales[it.at] : 0.0f, v_before = it.r0 ? a.side[1].scales[it.at] : 0.0f;
  // A place that is no new row gets the nearest one: it changes no maximum, and
  // what is made of it is not written; all loads go out together.
  const auto near = [&](uint32_t r) { return min(max(r, it.r0), it.r1 - 1u); };
  const uint32_t u = tid % U, pair = tid / U, c = tid % C, quad = tid / C;
  const Unit un = unit_of<INTER>(arg.rot, u);
  typename In<T>::raw k0[2], k1[2], vx[4];
  {
    const char *k = a.side[0].x + it.head * a.side[0].stride_h, *v = a.side[1].x + it.head * a.side[1].stride_h;
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) {
      const char *row = k + (it.first + near(2u * pair + i)) * a.side[0].stride_t;
      k0[i] = In<T>::load(row + un.c0 * In<T>::kSize);
      k1[i] = In<T>::load(row + un.c1 * In<T>::kSize);
    }
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
      vx[i] = In<T>::load(v + (it.first + near(4u * quad + i)) * a.side[1].stride_t + c * (8u * In<T>::kSize));
  }
  float kx[2][16];
  uint32_t k_top = 0, v_top = 0;
#pragma unroll
  for (uint32_t i = 0; i < 2; ++i) {
    Turn t;
    if (un.turned) {
      const uint32_t r = near(2u * pair + i);
      turn_at(t, arg.rot, u, it.first + r, it.place + r);
    }
    turned16<T, INTER>(kx[i], k0[i], k1[i], t, un.turned);
    in_order();
#pragma unroll
    for (int j = 0; j < 16; ++j) k_top = max(k_top, bits_of(kx[i][j]));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 8; ++j) v_top = max(v_top, bits_of(In<T>::get(vx[i], j)));
  wg_max2(k_top, v_top, red);
#pragma unroll
  for (int i = 0; i < 4; ++i) In<T>::anew(vx[i]);
  if (max(k_top, v_top) >= 0x7F800000u) {   // the same in every thread
    k_top = v_top = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 16; ++j) k_top = max(k_top, finite_bits(kx[i][j]));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 8; ++j) v_top = max(v_top, finite_bits(In<T>::get(vx[i], j)));
    wg_max2(k_top, v_top, red);
#pragma unroll
    for (int i = 0; i < 4; ++i) In<T>::anew(vx[i]);
  }
  const Grow kg = grow(k_before, __builtin_bit_cast(float, k_top)), vg = grow(v_before, __builtin_bit_cast(float, v_top));
  if (tid == 0u) {
    a.side[0].scales[it.at] = kg.scale;
    a.side[1].scales[it.at] = vg.scale;
  }
  int8_t *kc = a.side[0].codes + it.at * (page * D), *vc = a.side[1].codes + it.at * (page * D);
  // keys
#pragma unroll
  for (uint32_t i = 0; i < 2; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = pack4(code_of(kx[i][4 * j] * kg.fresh), code_of(kx[i][4 * j + 1] * kg.fresh), code_of(kx[i][4 * j + 2] * kg.fresh),
                   code_of(kx[i][4 * j + 3] * kg.fresh));
    const uint32_t r = 2u * pair + i;
    if (r >= it.r0 && r < it.r1) {
      *reinterpret_cast<u32x2 *>(kc + r * D + un.c0) = (u32x2){w[0], w[1]};
      *reinterpret_cast<u32x2 *>(kc + r * D + un.c1) = (u32x2){w[2], w[3]};
    }
  }
  if (kg.again != 1.0f)   // the range grew
#pragma unroll 1
    for (uint32_t i = tid; i < it.r0 * (D / 16u); i += blockDim.x) {
      u32x4 *to = reinterpret_cast<u32x4 *>(kc) + i;
      u32x4 w = *to;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = again4(w[e], kg.again);
      *to = w;
    }
  // values, turned to four tokens a word and collected in LDS
  if (quad * 4u < page) {
    u32x2 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = code_of(In<T>::get(vx[i], j) * vg.fresh);
      q[i] = (u32x2){pack4(e[0], e[1], e[2], e[3]), pack4(e[4], e[5], e[6], e[7])};
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 w = turn4(q[0][h], q[1][h], q[2][h], q[3][h]);
      uint8_t *to = vt + (c * 8u + h * 4u) * vs + quad * 4u;
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) *reinterpret_cast<uint32_t *>(to + e * vs) = w[e];
    }
  }
  __syncthreads();
  const uint32_t pieces = page / 16u;
#pragma unroll 1
  for (uint32_t p = tid; p < D * pieces; p += blockDim.x) {
    const uint32_t t0 = p % pieces * 16u;
    const uint8_t *from = vt + p / pieces * vs + t0;
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const uint32_t *>(from + 4 * e);
    u32x4 *to = reinterpret_cast<u32x4 *>(vc + p * 16u);   // of dimension p / pieces
    if (t0 < it.r0 || t0 + 16u > it.r1) {
      if (t0 >= it.r1 || (t0 + 16u <= it.r0 && vg.again == 1.0f)) continue;
      const u32x4 was = *to;
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) {
        const uint32_t re = vg.again == 1.0f ? was[e] : again4(was[e], vg.again);
        uint32_t out = 0;
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
          const uint32_t r = t0 + 4u * e + j;
          const uint32_t src = r < it.r0 ? re : r < it.r1 ? w[e] : was[e];
          out |= src & (0xFFu << (8u * j));
        }
        w[e] = out;
      }
    }
    *to = w;
  }
  __syncthreads();   // vt and red are written again
}

// A workgroup's queries: the sequences' new tokens in groups of arg.tokens,
// numbered one after another.
template <entro_dtype T, entro_dtype O, int D, bool INTER>
__device__ __forceinline__ void append_queries(const AppendArg &arg, uint32_t page, uint32_t item, uint32_t lane) {
  constexpr uint32_t U = D / 16;
  const KvArg &a = arg.kv;
  KvSpan own{};
  Spans spans(a.cu, a.total, a.n_seq, lane);
  const Found f = find_item(item, a.n_seq, lane, [&](uint32_t b0) {
    own = kv_span(a, spans, b0, page);
    return (own.count + arg.tokens - 1u) / arg.tokens;
  });
  if (f.seq == a.n_seq) return;
  const auto there = [&](uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, (int)(f.seq % 64u)); };
  const uint32_t begin = there(own.begin), count = there(own.count), pos = there(own.pos);
  const uint32_t u = threadIdx.x % U, slot = threadIdx.x / U;
  const uint32_t step = (blockDim.x / U) / arg.tokens, token = slot / step, head0 = slot % step;
  const uint32_t i = f.local * arg.tokens + token;
  if (token < arg.tokens && i < count)
    turn_rows<T, O, INTER>(arg.rows, arg.rot, u, (int64_t)begin + i, pos + i, head0, step);
}

template <entro_dtype T, entro_dtype O, int D, bool INTER>
__global__ __launch_bounds__(512, T == ENTRO_F32 ? 2 : 4) void kv_append_kernel(AppendArg arg, uint32_t page) {
  const KvArg &a = arg.kv;
  const uint32_t lane = threadIdx.x & 63u;
  if (blockIdx.x == 0u && blockIdx.y == 0u) kv_check(a, page);
  // rows of the grid: the heads' pages and the queries' items, as many a row as there
  // are pages, the heads spread evenly among them: pages wait (for their largest values,
  // for their turn through LDS) while queries stream
  const uint64_t rows = a.n_kv + (arg.q_items + a.items - 1u) / a.items;
  for (uint64_t y = blockIdx.y; y < rows; y += gridDim.y)
    for (uint64_t x = blockIdx.x; x < a.items; x += gridDim.x) {
      const uint64_t head = y * a.n_kv / rows;   // heads before row y
      if ((y + 1u) * a.n_kv / rows != head) {
        // a page's heads are neighbours: 12 sequences of up to 1001 tokens, 32 heads of 96,
        // 46.2 us instead of 47.7 with the pages of one head side by side
        const uint64_t place = head * a.items + x;
        const KvItem it = kv_item(a, page, (uint32_t)(place / a.n_kv), (uint32_t)(place % a.n_kv), lane);
        if (it.any) append_page<T, D, INTER>(arg, it, page);
      } else {
        const uint64_t item = (y - head) * a.items + x;
        if (item < arg.q_items) append_queries<T, O, D, INTER>(arg, page, (uint32_t)item, lane);
      }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

static entro_status check_rotary(const entro_rotary *r, uint32_t dim) {
  if (!r || !r->d_freqs || (reinterpret_cast<uintptr_t>(r->d_freqs) & 15u)) return ENTRO_E_INVAL;
  if (!head_dim_ok(dim)) return ENTRO_E_UNSUPPORTED;
  if (r->pairs == 0 || r->pairs > dim / 2u || r->n_axes == 0 || r->interleaved > 1u || !std::isfinite(r->gain))
    return ENTRO_E_INVAL;
  if (r->pairs % 8u || r->n_axes > 4u) return ENTRO_E_UNSUPPORTED;
  for (uint32_t i = 0; i < r->pairs; ++i)
    if (((r->axes[i / 16u] >> (2u * (i % 16u))) & 3u) >= r->n_axes) return ENTRO_E_INVAL;
  return ENTRO_OK;
}

static entro_status check_types(int in, int out) {
  if (in != ENTRO_BF16 && in != ENTRO_F16 && in != ENTRO_F32) return ENTRO_E_INVAL;
  return out == ENTRO_BF16 || out == ENTRO_F16 ? ENTRO_OK : ENTRO_E_INVAL;
}

static RotArg rot_arg(const entro_rotary &r, const int32_t *pos, int64_t stride) {
  RotArg a{};
  a.freqs = r.d_freqs;
  for (int i = 0; i < 4; ++i) a.axes[i] = r.axes[i];
  a.units = r.pairs / 8u;
  a.n_axes = r.n_axes;
  a.gain = r.gain;
  a.pos = pos;
  a.pos_stride = stride;
  return a;
}

static void rows_arg(RowsArg &a, int side, const entro_rows &x, const entro_rows &out, uint32_t heads, int in) {
  const int64_t size = in == ENTRO_F32 ? 4 : 2;
  a.x[side] = static_cast<const char *>(x.d);
  a.out[side] = static_cast<char *>(out.d);
  a.x_t[side] = size * x.stride_t;
  a.x_h[side] = size * x.stride_h;
  a.o_t[side] = 2 * out.stride_t;
  a.o_h[side] = 2 * out.stride_h;
  a.heads[side] = heads;
}

// Tokens of a workgroup that rotates rows: as many as leave 1024 workgroups, four a CU,
// since each takes its cosines and sines once for all its heads.
static uint32_t tokens_of(uint32_t rows) { return rows >= 8192u ? 8u : rows >= 4096u ? 4u : rows >= 2048u ? 2u : 1u; }

// f(constants of the input's and the output's type, the head dimension, the layout)
template <typename F>
static entro_status with_types(int in, int out, uint32_t dim, bool inter, F f) {
  const auto layout = [&](auto i, auto o, auto d) {
    return inter ? f(i, o, d, std::true_type{}) : f(i, o, d, std::false_type{});
  };
  const auto dims = [&](auto i, auto o) {
    return dim == 64u   ? layout(i, o, std::integral_constant<int, 64>{})
           : dim == 96u ? layout(i, o, std::integral_constant<int, 96>{})
                        : layout(i, o, std::integral_constant<int, 128>{});
  };
  const auto outs = [&](auto i) {
    return out == ENTRO_BF16 ? dims(i, std::integral_constant<entro_dtype, ENTRO_BF16>{})
                             : dims(i, std::integral_constant<entro_dtype, ENTRO_F16>{});
  };
  return in == ENTRO_BF16  ? outs(std::integral_constant<entro_dtype, ENTRO_BF16>{})
         : in == ENTRO_F16 ? outs(std::integral_constant<entro_dtype, ENTRO_F16>{})
                           : outs(std::integral_constant<entro_dtype, ENTRO_F32>{});
}

}  // namespace entro

using namespace entro;

extern "C" entro_status entro_rope(const entro_rotary *r, const entro_rope_args *a, hipStream_t stream) {
  if (!a) return ENTRO_E_INVAL;
  entro_status st = check_rotary(r, a->head_dim);
  if (st != ENTRO_OK) return st;
  st = check_types(a->in, a->out);
  if (st != ENTRO_OK) return st;
  if (a->n_heads > 65535u || a->n_kv_heads > 65535u) return ENTRO_E_UNSUPPORTED;
  if (a->rows == 0 || (a->n_heads == 0 && a->n_kv_heads == 0)) return ENTRO_OK;
  if (!a->d_pos || a->pos_stride < 0 || a->rows > 0x7FFFFFFFu) return ENTRO_E_INVAL;
  for (const entro_rows *x : {&a->q, &a->q_out, &a->k, &a->k_out}) {
    st = check_rows(*x, (x == &a->q || x == &a->q_out ? a->n_heads : a->n_kv_heads) ? a->rows : 0u);
    if (st != ENTRO_OK) return st;
  }
  RopeArg k{};
  rows_arg(k.rows, 0, a->q, a->q_out, a->n_heads, a->in);
  rows_arg(k.rows, 1, a->k, a->k_out, a->n_kv_heads, a->in);
  k.rot = rot_arg(*r, a->d_pos, a->pos_stride);
  k.total = a->rows;
  k.tokens = tokens_of(a->rows);
  return with_types(a->in, a->out, a->head_dim, r->interleaved != 0u, [&](auto i, auto o, auto d, auto inter) {
    (void)hipGetLastError();
    hipLaunchKernelGGL((rope_kernel<decltype(i)::value, decltype(o)::value, decltype(d)::value, decltype(inter)::value>),
                       grid2(((uint64_t)k.total + k.tokens - 1u) / k.tokens, 1), dim3(kRopeThreads), 0, stream, k);
    return hipGetLastError() == hipSuccess ? ENTRO_OK : ENTRO_E_HIP;
  });
}

extern "C" entro_status entro_kv_append(const entro_kv_cache *c, const entro_kv_table *t, const entro_rotary *r,
                                        const entro_kv_append_args *a, uint32_t *d_status, hipStream_t stream) {
  if (!a) return ENTRO_E_INVAL;
  entro_status st = check_cache(c, t);
  if (st != ENTRO_OK) return st;
  st = check_rotary(r, c->head_dim);
  if (st != ENTRO_OK && (t->n_seq || !r)) return st;
  st = check_types(a->in, a->out);
  if (st != ENTRO_OK) return st;
  if (a->n_heads > 65535u) return ENTRO_E_UNSUPPORTED;
  if (t->n_seq == 0) return ENTRO_OK;
  if (!a->d_held || !a->d_cu_new || !d_status || a->total_new > 0x7FFFFFFFu) return ENTRO_E_INVAL;
  if (a->d_pos && a->pos_stride < 0) return ENTRO_E_INVAL;
  for (const entro_rows *x : {&a->k, &a->v, &a->q, &a->q_out}) {
    st = check_rows(*x, x == &a->k || x == &a->v || a->n_heads ? a->total_new : 0u);
    if (st != ENTRO_OK) return st;
  }
  const uint32_t page = c->page_tokens;
  const int64_t size = a->in == ENTRO_F32 ? 4 : 2;
  AppendArg k{};
  k.kv.side[0] = {c->d_k_codes, c->d_k_scales, static_cast<char *>(a->k.d), size * a->k.stride_t, size * a->k.stride_h};
  k.kv.side[1] = {c->d_v_codes, c->d_v_scales, static_cast<char *>(a->v.d), size * a->v.stride_t, size * a->v.stride_h};
  k.kv.table = t->d_table;
  k.kv.table_stride = t->table_stride;
  k.kv.table_pages = t->table_pages;
  k.kv.n_seq = t->n_seq;
  k.kv.n_pages = c->n_pages;
  k.kv.n_kv = c->n_kv_heads;
  // every page that takes part has a token of the call, and at most two pages of a
  // sequence are not full
  const uint64_t total = a->total_new;
  k.kv.items = std::max<uint64_t>(1u, std::min<uint64_t>(total, total / page + 2ull * t->n_seq));
  k.kv.pos = a->d_held;
  k.kv.cu = a->d_cu_new;
  k.kv.total = a->total_new;
  k.kv.status = d_status;
  k.rot = rot_arg(*r, a->d_pos, a->pos_stride);
  const uint32_t dim = c->head_dim, threads = (dim / 8u * (page / 4u) + 63u) & ~63u;
  if (a->n_heads) {
    rows_arg(k.rows, 0, a->q, a->q_out, a->n_heads, a->in);
    k.tokens = std::min(tokens_of(a->total_new), threads / (dim / 16u));
    k.q_items = std::min<uint64_t>(total, total / k.tokens + t->n_seq);
  } else {
    k.tokens = 1u;
  }
  const uint64_t rows = k.kv.n_kv + (k.q_items + k.kv.items - 1u) / k.kv.items;
  const size_t lds = (size_t)dim * (page + 4u) + 8u * kWavesMost;
  return with_types(a->in, a->out, dim, r->interleaved != 0u, [&](auto i, auto o, auto d, auto inter) {
    (void)hipGetLastError();
    hipLaunchKernelGGL((kv_append_kernel<decltype(i)::value, decltype(o)::value, decltype(d)::value, decltype(inter)::value>),
                       grid2(k.kv.items, rows), dim3(threads), lds, stream, k, page);
    return hipGetLastError() == hipSuccess ? ENTRO_OK : ENTRO_E_HIP;
  });
}

// HIP kernels (gfx950) and entry points of the 8-bit key/value cache:
// entro_kv_store, entro_kv_load.  The cache's layout and the arithmetic of a
// page's codes are in entro_attn.h.
#include <algorithm>

#include "entro_kv_device.h"

namespace entro {

// ---------------------------------------------------------------------------
// store: a thread holds four rows x eight columns of the new rows (one pass over
// the inputs: the largest magnitude is taken from registers before the codes are
// made there), of keys and values.  Key codes go out as they lie; value codes are turned in
// registers to four tokens a word and collected in LDS, from where a thread
// writes 16 tokens of one dimension.  Pieces of 16 tokens that are not all new
// are merged with what the page holds.  Memory bound: 2 bytes in and 1 out per
// value.  32768 tokens of 8 heads of 128: 46 us, 4.4 TB/s of both together (a copy
// in that proportion reaches 5.6); 4522 tokens of 12 sequences, 32 heads of 96 in
// pages of 32: 24 us, 3.5 TB/s.  One token for each of 16 sequences: 7.4 us, 0.3 more
// where the range grows: a chain of reads (sums, page, rows and scale, codes held).
// Reading the codes held with the rows takes registers: it spills and costs the
// large calls 10%.
// ---------------------------------------------------------------------------
template <entro_dtype T, int D>
__global__ __launch_bounds__(512, 5) void kv_store_kernel(KvArg a, uint32_t page) {
  constexpr uint32_t C = D / 8;           // column groups of eight
  uint8_t *vt = reinterpret_cast<uint8_t *>(dyn_lds);   // [D][page + 4]
  const uint32_t tid = threadIdx.x, lane = tid & 63u;
  const uint32_t vs = page + 4u, c = tid % C, quad = tid / C;
  uint32_t *red = reinterpret_cast<uint32_t *>(vt + D * vs);   // [kWavesMost]
  if (blockIdx.x == 0u && blockIdx.y == 0u) kv_check(a, page);
  for (uint32_t head = blockIdx.y; head < a.n_kv; head += gridDim.y)
    for (uint64_t item = blockIdx.x; item < a.items; item += gridDim.x) {
      const KvItem it = kv_item(a, page, (uint32_t)item, head, lane);
      if (!it.any) continue;
      const bool mine = quad * 4u < page;
      // rows before r0 are held, by these scales
      const float k_before = it.r0 ? a.side[0].scales[it.at] : 0.0f, v_before = it.r0 ? a.side[1].scales[it.at] : 0.0f;
      u32x4 kx[4], vx[4];
      // (a place that is no new row gets the nearest one: it changes no maximum,
      // and what is made of it is not written; all loads go out together)
      auto rows = [&](u32x4 (&x)[4], const KvSide &s) {
        const char *from = s.x + it.first * s.stride_t + it.head * s.stride_h + c * 16u;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
          x[i] = *reinterpret_cast<const u32x4 *>(from + min(max(quad * 4u + i, it.r0), it.r1 - 1u) * s.stride_t);
      };
      rows(kx, a.side[0]);
      rows(vx, a.side[1]);
      // the new scale, written, and the codes of the thread's rows in place of them
      auto quantize = [&](u32x4 (&x)[4], u32x2 (&q)[4], float before, float *scale) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          for (int e = 0; e < 4; ++e) top = top_of<T, false>(x[i][e], top);
        top = wg_max(top, red);
        if (top >= Elem<T>::kInf) {   // the same in every thread
          top = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            for (int e = 0; e < 4; ++e) top = top_of<T, true>(x[i][e], top);
          top = wg_max(top, red);
        }
        const Grow g = grow(before, Elem<T>::lo(top));
        if (tid == 0u) *scale = g.scale;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t e[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            e[2 * j] = code_of(Elem<T>::lo(x[i][j]) * g.fresh);
            e[2 * j + 1] = code_of(Elem<T>::hi(x[i][j]) * g.fresh);
          }
          q[i] = (u32x2){pack4(e[0], e[1], e[2], e[3]), pack4(e[4], e[5], e[6], e[7])};
          __builtin_amdgcn_sched_barrier(0);   // one row after another: registers are occupancy here
        }
        return g.again;
      };
      u32x2 q[4];
      {
        int8_t *codes = a.side[0].codes + it.at * (page * D);
        const float again = quantize(kx, q, k_before, a.side[0].scales + it.at);
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
          const uint32_t r = quad * 4u + i;
          if (mine && r >= it.r0 && r < it.r1) *reinterpret_cast<u32x2 *>(codes + r * D + c * 8u) = q[i];
        }
        if (again != 1.0f)   // the range grew
#pragma unroll 1
          for (uint32_t i = tid; i < it.r0 * (D / 16u); i += blockDim.x) {
            u32x4 *to = reinterpret_cast<u32x4 *>(codes) + i;
            u32x4 w = *to;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              w[e] = again4(w[e], again);
              __builtin_amdgcn_sched_barrier(0);
            }
            *to = w;
          }
      }
      {
        int8_t *codes = a.side[1].codes + it.at * (page * D);
        const float again = quantize(vx, q, v_before, a.side[1].scales + it.at);
        if (mine)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x4 w = turn4(q[0][h], q[1][h], q[2][h], q[3][h]);
            uint8_t *to = vt + (c * 8u + h * 4u) * vs + quad * 4u;
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) *reinterpret_cast<uint32_t *>(to + e * vs) = w[e];
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
          u32x4 *to = reinterpret_cast<u32x4 *>(codes + p * 16u);   // of dimension p / pieces
          if (t0 < it.r0 || t0 + 16u > it.r1) {
            if (t0 >= it.r1 || (t0 + 16u <= it.r0 && again == 1.0f)) continue;
            const u32x4 was = *to;
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) {
              const uint32_t re = again == 1.0f ? was[e] : again4(was[e], again);
              uint32_t out = 0;
#pragma unroll
              for (uint32_t j = 0; j < 4; ++j) {
                const uint32_t r = t0 + 4u * e + j;
                const uint32_t src = r < it.r0 ? re : r < it.r1 ? w[e] : was[e];
                out |= src & (0xFFu << (8u * j));
              }
              w[e] = out;
              __builtin_amdgcn_sched_barrier(0);
            }
          }
          *to = w;
        }
      }
      __syncthreads();   // vt and red are written again
    }
}

// ---------------------------------------------------------------------------
// load: the same four rows x eight columns a thread, keys and values of a head
// on their way together.  Value codes come in as 16 tokens of one dimension and
// are turned over LDS.  Memory bound, 1 byte in and 2 out: 58371 tokens of 8
// heads of 128 (24 sequences) 71 us, 5.05 TB/s (a copy in that proportion: 5.2); 700 tokens of 32 heads of 64 in
// pages of 16 5.2 us.
// ---------------------------------------------------------------------------
template <entro_dtype T>
__device__ __forceinline__ u32x4 values8(uint32_t lo, uint32_t hi, float s) {
  return (u32x4){Elem<T>::pack2(byte_of(lo, 0) * s, byte_of(lo, 1) * s), Elem<T>::pack2(byte_of(lo, 2) * s, byte_of(lo, 3) * s),
                 Elem<T>::pack2(byte_of(hi, 0) * s, byte_of(hi, 1) * s), Elem<T>::pack2(byte_of(hi, 2) * s, byte_of(hi, 3) * s)};
}

template <entro_dtype T, int D>
__global__ __launch_bounds__(512, 8) void kv_load_kernel(KvArg a, uint32_t page) {
  constexpr uint32_t C = D / 8;
  uint8_t *vt = reinterpret_cast<uint8_t *>(dyn_lds);   // [D][page + 4]
  const uint32_t tid = threadIdx.x, lane = tid & 63u;
  const uint32_t vs = page + 4u, c = tid % C, quad = tid / C;
  if (blockIdx.x == 0u && blockIdx.y == 0u) kv_check(a, page);
  for (uint32_t head = blockIdx.y; head < a.n_kv; head += gridDim.y)
    for (uint64_t item = blockIdx.x; item < a.items; item += gridDim.x) {
      const KvItem it = kv_item(a, page, (uint32_t)item, head, lane);
      if (!it.any) continue;
      const bool mine = quad * 4u < page;
      const uint32_t pieces = page / 16u;
      const int8_t *kc = a.side[0].codes + it.at * (page * D), *vc = a.side[1].codes + it.at * (page * D);
      const float k_scale = a.side[0].scales[it.at], v_scale = a.side[1].scales[it.at];
      u32x2 w[4];
      if (mine)
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const u32x2 *>(kc + (quad * 4u + i) * D + c * 8u);
      for (uint32_t p = tid; p < D * pieces; p += blockDim.x) {
        const u32x4 x = *reinterpret_cast<const u32x4 *>(vc + p * 16u);   // of dimension p / pieces
        uint8_t *to = vt + p / pieces * vs + p % pieces * 16u;
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t *>(to + 4 * e) = x[e];
      }
      auto put = [&](const KvSide &s, float scale) {
        char *to = s.x + (it.first + quad * 4u) * s.stride_t + it.head * s.stride_h + c * 16u;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
          const uint32_t r = quad * 4u + i;
          if (mine && r >= it.r0 && r < it.r1)
            *reinterpret_cast<u32x4 *>(to + i * s.stride_t) = values8<T>(w[i].x, w[i].y, scale);
        }
      };
      put(a.side[0], k_scale);
      __syncthreads();
      if (mine)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t *from = vt + (c * 8u + h * 4u) * vs + quad * 4u;
          uint32_t b[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) b[e] = *reinterpret_cast<const uint32_t *>(from + e * vs);
          const u32x4 r = turn4(b[0], b[1], b[2], b[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e][h] = r[e];
        }
      put(a.side[1], v_scale);
      __syncthreads();   // vt is written again
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

template <bool STORE, entro_dtype T, int D>
static entro_status launch_kv(KvArg &a, uint32_t page, hipStream_t s) {
  // every page that takes part has a token of the call, and at most two pages
  // of a sequence are not full
  const uint64_t items = std::min<uint64_t>(a.total, (uint64_t)a.total / page + 2ull * a.n_seq);
  a.items = items;
  const uint32_t threads = (D / 8u * (page / 4u) + 63u) & ~63u;
  const size_t lds = (size_t)D * (page + 4u) + (STORE ? 4u * kWavesMost : 0u);
  (void)hipGetLastError();
  hipLaunchKernelGGL((STORE ? kv_store_kernel<T, D> : kv_load_kernel<T, D>), grid2(items, a.n_kv), dim3(threads), lds, s,
                     a, page);
  return hipGetLastError() == hipSuccess ? ENTRO_OK : ENTRO_E_HIP;
}

template <bool STORE>
static entro_status run_kv(const entro_kv_cache *c, const entro_kv_table *t, const entro_rows &k, const entro_rows &v,
                           const int32_t *pos, const int32_t *cu, uint32_t total, int dtype, uint32_t *d_status,
                           hipStream_t s) {
  const entro_status bad = check_cache(c, t);
  if (bad != ENTRO_OK) return bad;
  if (dtype != ENTRO_BF16 && dtype != ENTRO_F16) return ENTRO_E_INVAL;
  if (t->n_seq == 0) return ENTRO_OK;
  if (!pos || !cu || !d_status || total > 0x7FFFFFFFu) return ENTRO_E_INVAL;
  for (const entro_rows *r : {&k, &v}) {
    const entro_status e = check_rows(*r, total);
    if (e != ENTRO_OK) return e;
  }
  KvArg a{};
  a.side[0] = {c->d_k_codes, c->d_k_scales, static_cast<char *>(k.d), 2 * k.stride_t, 2 * k.stride_h};
  a.side[1] = {c->d_v_codes, c->d_v_scales, static_cast<char *>(v.d), 2 * v.stride_t, 2 * v.stride_h};
  a.table = t->d_table;
  a.table_stride = t->table_stride;
  a.table_pages = t->table_pages;
  a.n_seq = t->n_seq;
  a.n_pages = c->n_pages;
  a.n_kv = c->n_kv_heads;
  a.pos = pos;
  a.cu = cu;
  a.total = total;
  a.status = d_status;
  const uint32_t p = c->page_tokens;
  if (dtype == ENTRO_BF16)
    return c->head_dim == 64u   ? launch_kv<STORE, ENTRO_BF16, 64>(a, p, s)
           : c->head_dim == 96u ? launch_kv<STORE, ENTRO_BF16, 96>(a, p, s)
                                : launch_kv<STORE, ENTRO_BF16, 128>(a, p, s);
  return c->head_dim == 64u   ? launch_kv<STORE, ENTRO_F16, 64>(a, p, s)
         : c->head_dim == 96u ? launch_kv<STORE, ENTRO_F16, 96>(a, p, s)
                              : launch_kv<STORE, ENTRO_F16, 128>(a, p, s);
}

}  // namespace entro

using namespace entro;

extern "C" entro_status entro_kv_store(const entro_kv_cache *c, const entro_kv_table *t, const entro_kv_store_args *a,
                                       uint32_t *d_status, hipStream_t stream) {
  if (!a) return ENTRO_E_INVAL;
  return run_kv<true>(c, t, a->k, a->v, a->d_held, a->d_cu_new, a->total_new, a->dtype, d_status, stream);
}

extern "C" entro_status entro_kv_load(const entro_kv_cache *c, const entro_kv_table *t, const entro_kv_load_args *a,
                                      uint32_t *d_status, hipStream_t stream) {
  if (!a) return ENTRO_E_INVAL;
  return run_kv<false>(c, t, a->k, a->v, a->d_first, a->d_cu_out, a->total_out, a->dtype, d_status, stream);
}

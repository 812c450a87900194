// HIP kernels (gfx950) and entry points of the 8-bit key/value cache:
// entro_kv_store, entro_kv_load.  The cache's layout and the arithmetic of a
// page's codes are in entro_attn.h.
#include <algorithm>

#include "entro_attn_device.h"
#include "entro_internal.h"

namespace entro {

struct KvArg {
  int8_t *k_codes, *v_codes;
  float *k_scales, *v_scales;
  const int32_t *table;
  uint64_t table_stride;
  uint32_t table_pages, n_seq, n_pages, n_kv;
  const char *k, *v;           // 16-bit rows (written by the load)
  int64_t k_t, k_h, v_t, v_h;  // strides in bytes
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
__device__ __forceinline__ KvSpan kv_span(const KvArg &a, uint32_t b, uint32_t page) {
  const Span s = span_of(a.cu, b, a.total);
  const int32_t p = a.pos[b];
  const bool ok = s.ok && p >= 0 && (uint64_t)p + s.count <= (uint64_t)a.table_pages * page;
  return {s.begin, ok ? s.count : 0u, ok ? (uint32_t)p : 0u, ok};
}
__device__ __forceinline__ uint32_t kv_pages(const KvSpan &s, uint32_t page) {
  return s.count ? (s.pos + s.count - 1u) / page - s.pos / page + 1u : 0u;
}

// Marks the sequences whose lengths do not fit (one workgroup of the call).
__device__ __forceinline__ void kv_check(const KvArg &a, uint32_t page) {
  for (uint32_t b = threadIdx.x; b < a.n_seq; b += blockDim.x)
    if (!kv_span(a, b, page).ok) atomicOr(a.status + b, ENTRO_F_LENGTH);
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

// Largest of v over the workgroup, for keys and values at once.
__device__ __forceinline__ void wg_max(uint32_t &k, uint32_t &v, uint32_t *red) {
  for (int s = 32; s >= 1; s >>= 1) {
    k = max(k, (uint32_t)__shfl_xor((int)k, s, 64));
    v = max(v, (uint32_t)__shfl_xor((int)v, s, 64));
  }
  const uint32_t waves = blockDim.x >> 6;
  if (waves > 1u) {
    __syncthreads();
    if ((threadIdx.x & 63u) == 0u) {
      red[threadIdx.x >> 6] = k;
      red[8u + (threadIdx.x >> 6)] = v;
    }
    __syncthreads();
    for (uint32_t w = 0; w < waves; ++w) {
      k = max(k, red[w]);
      v = max(v, red[8u + w]);
    }
  }
}

template <entro_dtype T>
__device__ __forceinline__ float value_of(uint32_t bits) {
  return Elem<T>::lo(bits);
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

// ---------------------------------------------------------------------------
// store: one workgroup per page that gets tokens and head.  A thread holds
// four rows x eight columns of the page's new keys and of its new values (8
// loads of 16 bytes in flight, one pass over the inputs: the largest
// magnitude is taken from registers before the codes are made there).  Key
// codes go out as they lie; value codes are turned in registers to four
// tokens a word and collected in LDS, from where a thread writes 16 tokens of
// one dimension.  Pieces of 16 tokens that are not all new are merged with
// what the page holds.  Memory bound (2 bytes in, 1 out per value).
// ---------------------------------------------------------------------------
template <entro_dtype T, int D>
__global__ __launch_bounds__(512) void kv_store_kernel(KvArg a, uint32_t page) {
  constexpr uint32_t C = D / 8;           // column groups of eight
  __shared__ uint32_t red[16];
  uint8_t *vt = reinterpret_cast<uint8_t *>(dyn_lds);   // [D][page + 4]
  const uint32_t tid = threadIdx.x, lane = tid & 63u, head = blockIdx.y;
  const uint32_t vs = page + 4u;
  if (blockIdx.x == 0u && head == 0u) kv_check(a, page);
  for (uint32_t item = blockIdx.x;; item += gridDim.x) {
    const Found f = find_item(item, a.n_seq, lane, [&](uint32_t b) { return kv_pages(kv_span(a, b, page), page); });
    if (f.seq == a.n_seq) break;
    const KvSpan s = kv_span(a, f.seq, page);
    const uint32_t index = s.pos / page + f.local;
    const int32_t id = a.table[(uint64_t)f.seq * a.table_stride + index];
    if (id < 0 || (uint32_t)id >= a.n_pages) {
      if (tid == 0u && head == 0u) atomicOr(a.status + f.seq, ENTRO_F_PAGE);
      continue;
    }
    const uint64_t at = (uint64_t)id * a.n_kv + head;
    int8_t *kc = a.k_codes + at * (page * D), *vc = a.v_codes + at * (page * D);
    // page rows r0 .. r1 - 1 are new, rows before r0 are held
    const uint32_t r0 = f.local == 0u ? s.pos % page : 0u;
    const uint32_t r1 = min(page, s.pos + s.count - index * page);
    const uint32_t c = tid % C, quad = tid / C;
    const bool mine = quad * 4u < page;
    u32x4 kx[4], vx[4];
    const int64_t first = (int64_t)s.begin + ((int64_t)index * page - (int64_t)s.pos);   // packed row of page row 0
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t r = quad * 4u + i;
      kx[i] = vx[i] = (u32x4){0u, 0u, 0u, 0u};
      if (mine && r >= r0 && r < r1) {
        kx[i] = *reinterpret_cast<const u32x4 *>(a.k + (first + r) * a.k_t + head * a.k_h + c * 16u);
        vx[i] = *reinterpret_cast<const u32x4 *>(a.v + (first + r) * a.v_t + head * a.v_h + c * 16u);
      }
    }
    const float k_before = r0 ? a.k_scales[at] : 0.0f, v_before = r0 ? a.v_scales[at] : 0.0f;
    uint32_t kt = 0, vtop = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      for (int e = 0; e < 4; ++e) {
        kt = top_of<T, false>(kx[i][e], kt);
        vtop = top_of<T, false>(vx[i][e], vtop);
      }
    wg_max(kt, vtop, red);
    if (kt >= Elem<T>::kInf || vtop >= Elem<T>::kInf) {   // the same in every thread
      kt = vtop = 0;
      for (int i = 0; i < 4; ++i)
        for (int e = 0; e < 4; ++e) {
          kt = top_of<T, true>(kx[i][e], kt);
          vtop = top_of<T, true>(vx[i][e], vtop);
        }
      wg_max(kt, vtop, red);
    }
    const Grow gk = grow(k_before, value_of<T>(kt)), gv = grow(v_before, value_of<T>(vtop));
    if (mine) {
      uint32_t vq[4][2];
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t r = quad * 4u + i;
        uint32_t q[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          q[2 * e] = code_of(Elem<T>::lo(kx[i][e]) * gk.fresh);
          q[2 * e + 1] = code_of(Elem<T>::hi(kx[i][e]) * gk.fresh);
        }
        if (r >= r0 && r < r1)
          *reinterpret_cast<u32x2 *>(kc + r * D + c * 8u) =
              (u32x2){pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7])};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          q[2 * e] = code_of(Elem<T>::lo(vx[i][e]) * gv.fresh);
          q[2 * e + 1] = code_of(Elem<T>::hi(vx[i][e]) * gv.fresh);
        }
        vq[i][0] = pack4(q[0], q[1], q[2], q[3]);
        vq[i][1] = pack4(q[4], q[5], q[6], q[7]);
      }
      // four rows of eight columns to eight words of four rows
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t ab = __builtin_amdgcn_perm(vq[1][h], vq[0][h], 0x05010400u), ab2 = __builtin_amdgcn_perm(vq[1][h], vq[0][h], 0x07030602u);
        const uint32_t cd = __builtin_amdgcn_perm(vq[3][h], vq[2][h], 0x05010400u), cd2 = __builtin_amdgcn_perm(vq[3][h], vq[2][h], 0x07030602u);
        uint8_t *to = vt + (c * 8u + h * 4u) * vs + quad * 4u;
        *reinterpret_cast<uint32_t *>(to) = __builtin_amdgcn_perm(cd, ab, 0x05040100u);
        *reinterpret_cast<uint32_t *>(to + vs) = __builtin_amdgcn_perm(cd, ab, 0x07060302u);
        *reinterpret_cast<uint32_t *>(to + 2u * vs) = __builtin_amdgcn_perm(cd2, ab2, 0x05040100u);
        *reinterpret_cast<uint32_t *>(to + 3u * vs) = __builtin_amdgcn_perm(cd2, ab2, 0x07060302u);
      }
    }
    if (tid == 0u) {
      a.k_scales[at] = gk.scale;
      a.v_scales[at] = gv.scale;
    }
    // keys held, where the range grew
    if (gk.again != 1.0f)
      for (uint32_t i = tid; i < r0 * (D / 4u); i += blockDim.x) {
        uint32_t *w = reinterpret_cast<uint32_t *>(kc) + i;
        *w = again4(*w, gk.again);
      }
    __syncthreads();
    const uint32_t pieces = page / 16u;
    for (uint32_t i = tid; i < D * pieces; i += blockDim.x) {
      const uint32_t d = i / pieces, t0 = (i % pieces) * 16u;
      const uint8_t *from = vt + d * vs + t0;
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const uint32_t *>(from + 4 * e);
      u32x4 *to = reinterpret_cast<u32x4 *>(vc + d * page + t0);
      if (t0 < r0 || t0 + 16u > r1) {
        if (t0 >= r1 || (t0 + 16u <= r0 && gv.again == 1.0f)) continue;
        const u32x4 was = *to;
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
          const uint32_t re = gv.again == 1.0f ? was[e] : again4(was[e], gv.again);
          uint32_t out = 0;
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t r = t0 + 4u * e + j;
            const uint32_t src = r < r0 ? re : r < r1 ? w[e] : was[e];
            out |= src & (0xFFu << (8u * j));
          }
          w[e] = out;
        }
      }
      *to = w;
    }
    __syncthreads();   // vt and red are written again
  }
}

// ---------------------------------------------------------------------------
// load: one workgroup per page that holds wanted tokens and head; the same
// four rows x eight columns a thread.  Value codes come in as 16 tokens of one
// dimension and are turned over LDS.
// ---------------------------------------------------------------------------
template <entro_dtype T>
__device__ __forceinline__ u32x4 values8(uint32_t lo, uint32_t hi, float s) {
  return (u32x4){Elem<T>::pack2(byte_of(lo, 0) * s, byte_of(lo, 1) * s), Elem<T>::pack2(byte_of(lo, 2) * s, byte_of(lo, 3) * s),
                 Elem<T>::pack2(byte_of(hi, 0) * s, byte_of(hi, 1) * s), Elem<T>::pack2(byte_of(hi, 2) * s, byte_of(hi, 3) * s)};
}

template <entro_dtype T, int D>
__global__ __launch_bounds__(512) void kv_load_kernel(KvArg a, uint32_t page) {
  constexpr uint32_t C = D / 8;
  uint8_t *vt = reinterpret_cast<uint8_t *>(dyn_lds);   // [D][page + 4]
  const uint32_t tid = threadIdx.x, lane = tid & 63u, head = blockIdx.y;
  const uint32_t vs = page + 4u;
  if (blockIdx.x == 0u && head == 0u) kv_check(a, page);
  for (uint32_t item = blockIdx.x;; item += gridDim.x) {
    const Found f = find_item(item, a.n_seq, lane, [&](uint32_t b) { return kv_pages(kv_span(a, b, page), page); });
    if (f.seq == a.n_seq) break;
    const KvSpan s = kv_span(a, f.seq, page);
    const uint32_t index = s.pos / page + f.local;
    const int32_t id = a.table[(uint64_t)f.seq * a.table_stride + index];
    if (id < 0 || (uint32_t)id >= a.n_pages) {
      if (tid == 0u && head == 0u) atomicOr(a.status + f.seq, ENTRO_F_PAGE);
      continue;
    }
    const uint64_t at = (uint64_t)id * a.n_kv + head;
    const int8_t *kc = a.k_codes + at * (page * D), *vc = a.v_codes + at * (page * D);
    const uint32_t r0 = f.local == 0u ? s.pos % page : 0u;
    const uint32_t r1 = min(page, s.pos + s.count - index * page);
    const uint32_t c = tid % C, quad = tid / C;
    const bool mine = quad * 4u < page;
    const int64_t first = (int64_t)s.begin + ((int64_t)index * page - (int64_t)s.pos);
    const float ks = a.k_scales[at], vsc = a.v_scales[at];
    u32x2 kq[4];
    if (mine)
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) kq[i] = *reinterpret_cast<const u32x2 *>(kc + (quad * 4u + i) * D + c * 8u);
    const uint32_t pieces = page / 16u;
    for (uint32_t i = tid; i < D * pieces; i += blockDim.x) {
      const uint32_t d = i / pieces, t0 = (i % pieces) * 16u;
      const u32x4 w = *reinterpret_cast<const u32x4 *>(vc + d * page + t0);
      uint8_t *to = vt + d * vs + t0;
#pragma unroll
      for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t *>(to + 4 * e) = w[e];
    }
    if (mine)
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t r = quad * 4u + i;
        if (r >= r0 && r < r1)
          *reinterpret_cast<u32x4 *>(const_cast<char *>(a.k) + (first + r) * a.k_t + head * a.k_h + c * 16u) =
              values8<T>(kq[i].x, kq[i].y, ks);
      }
    __syncthreads();
    if (mine) {
      uint32_t rows[4][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t *from = vt + (c * 8u + h * 4u) * vs + quad * 4u;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const uint32_t *>(from + e * vs);
        const uint32_t ab = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), ab2 = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
        const uint32_t cd = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), cd2 = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
        rows[0][h] = __builtin_amdgcn_perm(cd, ab, 0x05040100u);
        rows[1][h] = __builtin_amdgcn_perm(cd, ab, 0x07060302u);
        rows[2][h] = __builtin_amdgcn_perm(cd2, ab2, 0x05040100u);
        rows[3][h] = __builtin_amdgcn_perm(cd2, ab2, 0x07060302u);
      }
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t r = quad * 4u + i;
        if (r >= r0 && r < r1)
          *reinterpret_cast<u32x4 *>(const_cast<char *>(a.v) + (first + r) * a.v_t + head * a.v_h + c * 16u) =
              values8<T>(rows[i][0], rows[i][1], vsc);
      }
    }
    __syncthreads();   // vt is written again
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

template <bool STORE, entro_dtype T, int D>
static entro_status launch_kv(const KvArg &a, uint32_t page, hipStream_t s) {
  // every page that takes part has a token of the call, and at most two pages
  // of a sequence are not full
  const uint64_t items = std::min<uint64_t>(a.total, (uint64_t)a.total / page + 2ull * a.n_seq);
  uint64_t grid = std::min<uint64_t>(items, 1u << 20);
  grid = std::max<uint64_t>(1, cap_grid(grid * a.n_kv) / a.n_kv);
  const uint32_t threads = (D / 8u * (page / 4u) + 63u) & ~63u;
  const size_t lds = (size_t)D * (page + 4u);
  (void)hipGetLastError();
  hipLaunchKernelGGL((STORE ? kv_store_kernel<T, D> : kv_load_kernel<T, D>), dim3((uint32_t)grid, a.n_kv), dim3(threads), lds, s,
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
  a.k_codes = c->d_k_codes;
  a.v_codes = c->d_v_codes;
  a.k_scales = c->d_k_scales;
  a.v_scales = c->d_v_scales;
  a.table = t->d_table;
  a.table_stride = t->table_stride;
  a.table_pages = t->table_pages;
  a.n_seq = t->n_seq;
  a.n_pages = c->n_pages;
  a.n_kv = c->n_kv_heads;
  a.k = static_cast<const char *>(k.d);
  a.v = static_cast<const char *>(v.d);
  a.k_t = 2 * k.stride_t;
  a.k_h = 2 * k.stride_h;
  a.v_t = 2 * v.stride_t;
  a.v_h = 2 * v.stride_h;
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

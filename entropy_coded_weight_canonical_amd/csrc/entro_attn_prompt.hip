// HIP kernel (gfx950) and entry point of the causal attention of packed
// prompts: entro_attn_prompt.  Definition in entro_attn.h.
#include <algorithm>

#include "entro_attn_device.h"
#include "entro_internal.h"

namespace entro {

struct PromptArg {
  const char *q, *k, *v;
  char *out;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;   // bytes
  const int32_t *cu_q, *cu_k;
  uint32_t n_seq, total_q, total_k, n_heads, n_kv;
  float scale;                                      // times log2(e)
  uint32_t *status;
};

constexpr uint32_t kRows = 32;   // queries of a workgroup

// Weights are held as 2^(score - maximum + kLift): f16 has 11 bits down to
// 2^-14 only, and many small weights can outweigh the largest together.
template <entro_dtype T>
constexpr float kLift = T == ENTRO_F16 ? 15.0f : 0.0f;

// Whether one of the eight 16-bit values is infinite or NaN.
template <entro_dtype T>
__device__ __forceinline__ bool special(u32x4 w) {
  constexpr uint32_t exps = Elem<T>::kInf * 0x10001u, one = (0x8000u - Elem<T>::kInf) * 0x10001u;
  uint32_t any = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) any |= (w[e] & exps) + one;   // a full exponent carries into bit 15
  return (any & 0x80008000u) != 0u;
}

// acc + w p for 16 tokens (token 8 (j / 4) + 4 half + j % 4 is element j of a
// half) that hold infinities or NaN, where some queries must not see some of
// the tokens: 0 * inf would reach them.  One product a token, added where the
// lane's query sees it (`seen`: its tokens here, from the first on).
template <entro_dtype T>
__device__ f32x16 mfma_seen(u32x4 w, u32x4 p, f32x16 acc, uint32_t half, int64_t seen) {
#pragma unroll 1
  for (uint32_t t = 0; t < 16u; ++t) {
    const uint32_t j = (t & 3u) + 4u * (t >> 3);
    const bool mine = half == ((t >> 2) & 1u);
    u32x4 x;
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) x[e] = mine && e == j / 2u ? w[e] & (0xFFFFu << (16u * (j & 1u))) : 0u;
    f32x16 add;
#pragma unroll
    for (int r = 0; r < 16; ++r) add[r] = 0.0f;
    add = Elem<T>::mfma32(x, p, add);
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] += (int64_t)t < seen ? add[r] : 0.0f;
  }
  return acc;
}

template <entro_dtype T, int D>
__global__ __launch_bounds__(64) void attn_prompt_kernel(PromptArg a) {
  constexpr int KS = D / 16, DT = D / 32;
  const uint32_t lane = threadIdx.x, n = lane & 31u, half = lane >> 5;
  const uint32_t head = blockIdx.y, kvh = head / (a.n_heads / a.n_kv);
  if (blockIdx.x == 0u && head == 0u)
    for (uint32_t b = lane; b < a.n_seq; b += 64u)
      if (!span_of(a.cu_q, b, a.total_q).ok || !span_of(a.cu_k, b, a.total_k).ok) atomicOr(a.status + b, ENTRO_F_LENGTH);
  for (uint32_t item = blockIdx.x;; item += gridDim.x) {
    const Found f = find_item(item, a.n_seq, lane, [&](uint32_t b) {
      return span_of(a.cu_k, b, a.total_k).ok ? (span_of(a.cu_q, b, a.total_q).count + kRows - 1u) / kRows : 0u;
    });
    if (f.seq == a.n_seq) break;
    const Span sq = span_of(a.cu_q, f.seq, a.total_q), sk = span_of(a.cu_k, f.seq, a.total_k);
    const uint32_t q0 = f.local * kRows;
    const uint32_t qi = q0 + n;
    const int64_t last = (int64_t)qi + sk.count - sq.count;   // last key of this lane's query
    const char *kb = a.k + sk.begin * a.k_t + kvh * a.k_h, *vb = a.v + sk.begin * a.v_t + kvh * a.v_h;
    u32x4 qf[KS];
    const char *qp = a.q + (int64_t)(sq.begin + min(qi, sq.count - 1u)) * a.q_t + head * a.q_h;
#pragma unroll
    for (int s = 0; s < KS; ++s) qf[s] = *reinterpret_cast<const u32x4 *>(qp + s * 32 + half * 16);
    f32x16 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
      for (int r = 0; r < 16; ++r) o[d][r] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    const int64_t end = min((int64_t)sk.count, (int64_t)min(q0 + kRows, sq.count) + sk.count - sq.count);
    for (int64_t k0 = 0; k0 < end; k0 += 32) {
      f32x16 s;
      for (int r = 0; r < 16; ++r) s[r] = 0.0f;
      const char *kp = kb + min(k0 + n, (int64_t)sk.count - 1) * a.k_t;
#pragma unroll
      for (int i = 0; i < KS; ++i)
        s = Elem<T>::mfma32(*reinterpret_cast<const u32x4 *>(kp + i * 32 + half * 16), qf[i], s);
      float mx = -INFINITY;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t j = k0 + 8 * (r / 4) + 4 * half + r % 4;
        s[r] = j <= last && j < sk.count ? s[r] * a.scale : -INFINITY;
        mx = fmaxf(mx, s[r]);
      }
      mx = max32(mx);
      const float mn = fmaxf(m, mx);
      const float off = mn == -INFINITY ? 0.0f : mn - kLift<T>;
      const float k = mn == -INFINITY ? 1.0f : exp2_fast(m - mn);
      m = mn;
      l *= k;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= k;
      u32x4 p[2];
#pragma unroll
      for (int r = 0; r < 16; r += 2) {
        const float x = exp2_fast(s[r] - off), y = exp2_fast(s[r + 1] - off);
        l += x + y;
        p[r / 8][r % 8 / 2] = Elem<T>::pack2(x, y);
      }
      // values of the tokens that the weights' places stand for, one by one
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          u32x4 w;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t x[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int r = 8 * c + 2 * e + z;
              const int64_t j = k0 + 8 * (r / 4) + 4 * half + r % 4;
              x[z] = j < sk.count ? *reinterpret_cast<const uint16_t *>(vb + j * a.v_t + (32 * d + n) * 2u) : 0u;
            }
            w[e] = x[0] | x[1] << 16;
          }
          const int64_t seen = last + 1 - (k0 + 16 * c);
          if (__any(special<T>(w)) && __any(seen < 16))
            o[d] = mfma_seen<T>(w, p[c], o[d], half, seen);
          else
            o[d] = Elem<T>::mfma32(w, p[c], o[d]);
        }
    }
    l = add32(l);
    const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
    if (qi < sq.count) {
      char *op = a.out + (int64_t)(sq.begin + qi) * a.o_t + head * a.o_h;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
          *reinterpret_cast<u32x2 *>(op + (32 * d + 8 * (r / 4) + 4 * half) * 2) =
              (u32x2){Elem<T>::pack2(o[d][r] * inv, o[d][r + 1] * inv), Elem<T>::pack2(o[d][r + 2] * inv, o[d][r + 3] * inv)};
    }
  }
}

template <entro_dtype T, int D>
static entro_status launch_prompt(const PromptArg &a, hipStream_t s) {
  uint64_t grid = std::min<uint64_t>(a.total_q, (uint64_t)a.total_q / kRows + a.n_seq);
  grid = std::max<uint64_t>(1, cap_grid(grid * a.n_heads) / a.n_heads);
  (void)hipGetLastError();
  hipLaunchKernelGGL((attn_prompt_kernel<T, D>), dim3((uint32_t)grid, a.n_heads), dim3(64), 0, s, a);
  return hipGetLastError() == hipSuccess ? ENTRO_OK : ENTRO_E_HIP;
}

}  // namespace entro

using namespace entro;

extern "C" entro_status entro_attn_prompt(const entro_attn_prompt_args *a, uint32_t *d_status, hipStream_t stream) {
  if (!a) return ENTRO_E_INVAL;
  entro_status st = check_heads(a->n_heads, a->n_kv_heads, a->head_dim, a->dtype);
  if (st != ENTRO_OK) return st;
  if (!std::isfinite(a->scale)) return ENTRO_E_INVAL;
  if (a->n_seq == 0) return ENTRO_OK;
  if (!a->d_cu_q || !a->d_cu_k || !d_status) return ENTRO_E_INVAL;
  if (a->total_q > 0x7FFFFFFFu || a->total_k > 0x7FFFFFFFu || a->n_seq > 0x7FFFFFFFu) return ENTRO_E_INVAL;
  if ((st = check_rows(a->q, a->total_q)) != ENTRO_OK || (st = check_rows(a->out, a->total_q)) != ENTRO_OK ||
      (st = check_rows(a->k, a->total_k)) != ENTRO_OK || (st = check_rows(a->v, a->total_k)) != ENTRO_OK)
    return st;
  PromptArg p{};
  p.q = static_cast<const char *>(a->q.d);
  p.k = static_cast<const char *>(a->k.d);
  p.v = static_cast<const char *>(a->v.d);
  p.out = static_cast<char *>(a->out.d);
  p.q_t = 2 * a->q.stride_t;
  p.q_h = 2 * a->q.stride_h;
  p.k_t = 2 * a->k.stride_t;
  p.k_h = 2 * a->k.stride_h;
  p.v_t = 2 * a->v.stride_t;
  p.v_h = 2 * a->v.stride_h;
  p.o_t = 2 * a->out.stride_t;
  p.o_h = 2 * a->out.stride_h;
  p.cu_q = a->d_cu_q;
  p.cu_k = a->d_cu_k;
  p.n_seq = a->n_seq;
  p.total_q = a->total_q;
  p.total_k = a->total_k;
  p.n_heads = a->n_heads;
  p.n_kv = a->n_kv_heads;
  p.scale = a->scale * kLog2e;
  p.status = d_status;
  if (a->dtype == ENTRO_BF16)
    return a->head_dim == 64u   ? launch_prompt<ENTRO_BF16, 64>(p, stream)
           : a->head_dim == 96u ? launch_prompt<ENTRO_BF16, 96>(p, stream)
                                : launch_prompt<ENTRO_BF16, 128>(p, stream);
  return a->head_dim == 64u   ? launch_prompt<ENTRO_F16, 64>(p, stream)
         : a->head_dim == 96u ? launch_prompt<ENTRO_F16, 96>(p, stream)
                              : launch_prompt<ENTRO_F16, 128>(p, stream);
}

// HIP kernel (gfx950) and entry point of the causal attention of packed
// prompts: entro_attn_prompt.  Definition in entro_attn.h.
#include <algorithm>
#include <type_traits>

#include "entro_attn_device.h"
#include "entro_internal.h"

namespace entro {

struct PromptArg {
  const char *q, *k, *v;
  char *out;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;   // bytes
  const int32_t *cu_q, *cu_k;
  uint32_t n_seq, total_q, total_k, n_heads, n_kv;
  float scale;                                      // magnitude, times log2(e); 1 where the scale is 0
  uint32_t q_and, q_xor;                            // on a pair of q: the scale's sign, and 0 where the scale is 0
  uint32_t *status;
};

constexpr uint32_t kTile = 64;     // keys of a step
constexpr uint32_t kWaves4 = 4;    // wavefronts of a workgroup

// Weights are held as 2^(score - maximum + kLift), the maximum being behind by
// at most kLag (in powers of two): raising it means a pass over the outputs,
// and most tiles raise it by little.  f16 has 11 bits down to 2^-14 only, and
// many small weights can outweigh the largest together: its weights go up to
// 2^15, so that those down to 2^-26 of the largest have all their bits.
template <entro_dtype T>
constexpr float kLift = T == ENTRO_F16 ? 12.0f : 0.0f;
template <entro_dtype T>
constexpr float kLag = T == ENTRO_F16 ? 3.0f : 8.0f;

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
__device__ __forceinline__ f32x16 mfma_seen(u32x4 w, u32x4 p, f32x16 acc, uint32_t half, int seen) {
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
    for (int r = 0; r < 16; ++r) acc[r] += (int)t < seen ? add[r] : 0.0f;
  }
  return acc;
}

// LDS place (16-byte piece) of piece c of row r of a tile of keys or values.
// Rows are 2 D bytes, and a wavefront reads one piece of 32 rows (keys), or two
// neighbouring pieces of 8 rows (values), at once: the pieces' order within a
// row varies with the row so that these spread over all banks.
template <int D>
__device__ __forceinline__ uint32_t key_piece(uint32_t r, uint32_t c) {
  return D == 128 ? c ^ (r & 15u) : D == 64 ? c ^ ((r >> 1) & 7u) : c ^ ((r >> 2) & 3u);
}
template <int D>
__device__ __forceinline__ uint32_t value_piece(uint32_t r, uint32_t c) {
  return D == 128 ? c ^ (2u * (r & 7u)) : D == 64 ? c ^ (2u * ((r >> 1) & 3u)) : c;
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;

// Four rows (tokens) of 16 columns turned: a lane of a group of 16 gives the
// address of row lane / 4, columns 4 (lane % 4) on, and receives the four rows
// of column lane % 16.
__device__ __forceinline__ u32x2 read_turned(uint32_t at) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)at));
}

// ---------------------------------------------------------------------------
// One workgroup takes 128 QB queries of one sequence and head, a wavefront 32 QB
// of them; the keys come in tiles of 64 that all four wavefronts read from
// LDS, two tiles in turn: the next one's copies (global memory to LDS, 16
// bytes a lane) are in flight while one is computed, one barrier a tile.
// Copies go through a buffer resource that ends with the sequence's last row,
// so rows past it arrive as zeros.
//
// Scores are K Q^T and outputs V^T P^T with the queries as columns: a lane and
// the one 32 further hold one query's softmax, whose statistics need one
// exchange between them a tile, and the weights leave the first product in
// the order in which the second takes them (row 8 (r / 4) + 4 half + r % 4 of a
// product is element r of a half; the values' tokens are read in that order).
// Values are turned on the way from LDS to registers.
// ---------------------------------------------------------------------------
template <entro_dtype T, int D, int QB>
__global__ __launch_bounds__(256, QB == 1 ? 2 : 1) void attn_prompt_kernel(PromptArg a) {
  constexpr int KS = D / 16, DT = D / 32, N = D / 32;
  constexpr uint32_t kBytes = kTile * D * 2u, kPieces = D / 8u;   // of a tile, of a row
  constexpr uint32_t kQueries = 32u * QB, kRows = kQueries * kWaves4;
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = rfl(tid >> 6), n = lane & 31u, half = lane >> 5;
  if (blockIdx.x == 0u)
    for (uint32_t b = tid; b < a.n_seq; b += 256u)
      if (!span_of(a.cu_q, b, a.total_q).ok || !span_of(a.cu_k, b, a.total_k).ok) atomicOr(a.status + b, ENTRO_F_LENGTH);

  // this lane's part of a tile's copies: N pieces of keys and N of values
  uint32_t k_off[N], v_off[N];
#pragma unroll
  for (uint32_t s = 0; s < (uint32_t)N; ++s) {
    const uint32_t i = (wave * N + s) * 64u + lane, r = i / kPieces, c = i % kPieces;
    k_off[s] = r * (uint32_t)a.k_t + key_piece<D>(r, c) * 16u;
    v_off[s] = r * (uint32_t)a.v_t + value_piece<D>(r, c) * 16u;
  }
  // and of its reads: keys of row n, values of rows 4 half + (lane / 4) % 4
  const uint32_t k_row = n * (2u * D);
  const uint32_t v_r = 4u * half + ((lane >> 2) & 3u), v_c = 2u * ((lane >> 4) & 1u) + ((lane >> 1) & 1u);
  const uint32_t v_row = v_r * (2u * D) + (lane & 1u) * 8u;

  for (uint64_t id = blockIdx.x;; id += gridDim.x) {
    // a key/value head's query heads and tiles stay on one XCD (workgroups go
    // around the 8 in turn) where n_kv is a multiple of 8
    const uint32_t slot = (uint32_t)(id % a.n_heads);
    const uint32_t kvh = slot % a.n_kv, head = kvh * (a.n_heads / a.n_kv) + slot / a.n_kv;
    const Found f = find_item((uint32_t)(id / a.n_heads), a.n_seq, lane, [&](uint32_t b) {
      return span_of(a.cu_k, b, a.total_k).ok ? (span_of(a.cu_q, b, a.total_q).count + kRows - 1u) / kRows : 0u;
    });
    if (f.seq == a.n_seq) break;
    const Span sq = span_of(a.cu_q, f.seq, a.total_q), sk = span_of(a.cu_k, f.seq, a.total_k);
    const uint32_t count_q = rfl(sq.count), count_k = rfl(sk.count), begin_q = rfl(sq.begin), begin_k = rfl(sk.begin);
    // the last queries first: they have the most keys
    const uint32_t wg0 = ((count_q + kRows - 1u) / kRows - 1u - f.local) * kRows;
    const uint32_t q0 = wg0 + wave * kQueries;
    const int64_t shift = (int64_t)count_k - count_q;       // query i sees keys up to i + shift
    const char *kb = a.k + begin_k * a.k_t + kvh * a.k_h, *vb = a.v + begin_k * a.v_t + kvh * a.v_h;

    u32x4 qf[QB][KS];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      const char *qp = a.q + (int64_t)(begin_q + min(q0 + 32u * b + n, count_q - 1u)) * a.q_t + head * a.q_h;
#pragma unroll
      for (int s = 0; s < KS; ++s)
        qf[b][s] = (*reinterpret_cast<const u32x4 *>(qp + s * 32 + half * 16) & a.q_and) ^ a.q_xor;
    }
    f32x16 o[QB][DT];
    float m[QB], l[QB];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      m[b] = -INFINITY;
      l[b] = 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d)
        for (int r = 0; r < 16; ++r) o[b][d][r] = 0.0f;
    }
    // keys that the workgroup, and this wavefront, see
    const int64_t wg_end = max((int64_t)0, (int64_t)min(wg0 + kRows, count_q) + shift);
    const int64_t my_end = q0 < count_q ? max((int64_t)0, (int64_t)min(q0 + kQueries, count_q) + shift) : 0;
    const int64_t full_end = (int64_t)q0 + shift + 1;       // keys that every query of the wavefront sees
    const uint32_t tiles = (uint32_t)((wg_end + kTile - 1) / kTile);

    auto copy = [&](uint32_t tile, uint32_t buf) {
      const uint32_t rows = min(kTile, count_k - tile * kTile);
      const __amdgpu_buffer_rsrc_t rk = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<char *>(kb + (int64_t)(tile * kTile) * a.k_t), 0, (int)((rows - 1u) * (uint32_t)a.k_t + 2u * D), 0x00020000);
      const __amdgpu_buffer_rsrc_t rv = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<char *>(vb + (int64_t)(tile * kTile) * a.v_t), 0, (int)((rows - 1u) * (uint32_t)a.v_t + 2u * D), 0x00020000);
      const uint32_t to = buf * (2u * kBytes) + wave * N * 1024u;
#pragma unroll
      for (uint32_t s = 0; s < (uint32_t)N; ++s)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rk, (lds_void *)(uintptr_t)(to + s * 1024u), 16, (int)k_off[s], 0, 0, 0);
#pragma unroll
      for (uint32_t s = 0; s < (uint32_t)N; ++s)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rv, (lds_void *)(uintptr_t)(to + kBytes + s * 1024u), 16, (int)v_off[s], 0, 0, 0);
    };
    __syncthreads();   // the last item's tiles have been read
    if (tiles) copy(0, 0);

    // keys of a tile that the lane's query of block b sees
    auto sees = [&](int b, uint32_t tile) {
      const int64_t k = (int64_t)(q0 + 32u * b + n) + shift + 1 - (int64_t)tile * kTile;
      return (int)min(max(k, (int64_t)0), (int64_t)kTile);
    };
    auto compute = [&](uint32_t tile, uint32_t buf, auto masked) {
      constexpr bool MASKED = decltype(masked)::value;
      const uint32_t kt = buf * (2u * kBytes), vt = kt + kBytes;
      f32x16 s[QB][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int b = 0; b < QB; ++b)
          for (int r = 0; r < 16; ++r) s[b][i][r] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const u32x4 w = *(lds_u32x4 *)(uintptr_t)(kt + i * 64u * D + k_row + key_piece<D>(n, 2 * k + half) * 16u);
#pragma unroll
          for (int b = 0; b < QB; ++b) s[b][i] = Elem<T>::mfma32(w, qf[b][k], s[b][i]);
        }
      }
      u32x4 p[QB][4];
#pragma unroll
      for (int b = 0; b < QB; ++b) {
        if (MASKED) {
          const int seen = sees(b, tile) - 4 * (int)half;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            for (int r = 0; r < 16; ++r) s[b][i][r] = 32 * i + 8 * (r / 4) + r % 4 < seen ? s[b][i][r] : -INFINITY;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[b][i][r]);
        mx = max32(mx);
        const bool raise = mx * a.scale > m[b] * a.scale + kLag<T>;
        if (__any(raise)) {
          const float mn = raise ? mx : m[b];
          const float k = mn == -INFINITY ? 1.0f : exp2_fast((m[b] - mn) * a.scale);
          m[b] = mn;
          l[b] *= k;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[b][d] *= k;
        }
        const float off = m[b] == -INFINITY ? 0.0f : kLift<T> - m[b] * a.scale;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          for (int r = 0; r < 16; r += 2) {
            const float x = exp2_fast(__builtin_fmaf(s[b][i][r], a.scale, off));
            const float y = exp2_fast(__builtin_fmaf(s[b][i][r + 1], a.scale, off));
            l[b] += x + y;
            p[b][2 * i + r / 8][r % 8 / 2] = Elem<T>::pack2(x, y);
          }
      }
      auto value = [&](uint32_t c, int d) {
        const uint32_t at = vt + c * 32u * D + v_row + value_piece<D>(v_r, 4 * d + v_c) * 16u;
        const u32x2 lo = read_turned(at), hi = read_turned(at + 16u * D);
        return (u32x4){lo.x, lo.y, hi.x, hi.y};
      };
      if (MASKED) {
        bool any = false;
#pragma unroll 1
        for (uint32_t c = 0; c < 4; ++c)
#pragma unroll
          for (int d = 0; d < DT; ++d) any |= special<T>(value(c, d));
        if (__any(any)) {
#pragma unroll 1
          for (uint32_t c = 0; c < 4; ++c)
#pragma unroll
            for (int b = 0; b < QB; ++b) {
              const int seen = sees(b, tile) - 16 * (int)c;
              const u32x4 w = c == 0u ? p[b][0] : c == 1u ? p[b][1] : c == 2u ? p[b][2] : p[b][3];
#pragma unroll
              for (int d = 0; d < DT; ++d) o[b][d] = mfma_seen<T>(value(c, d), w, o[b][d], half, seen);
            }
          return;
        }
      }
#pragma unroll
      for (uint32_t c = 0; c < 4; ++c)
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const u32x4 w = value(c, d);
#pragma unroll
          for (int b = 0; b < QB; ++b) o[b][d] = Elem<T>::mfma32(w, p[b][c], o[b][d]);
        }
    };
    for (uint32_t t = 0; t < tiles; ++t) {
      wait_lds_copy();
      __syncthreads();   // tile t is there; the buffer of tile t - 1 is free
      if (t + 1u < tiles) copy(t + 1u, (t + 1u) & 1u);
      const int64_t k0 = (int64_t)t * kTile;
      if (k0 + kTile <= full_end) compute(t, t & 1u, std::false_type{});
      else if (k0 < my_end) compute(t, t & 1u, std::true_type{});
    }
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      const uint32_t qi = q0 + 32u * b + n;
      const float sum = add32(l[b]);
      const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;   // NaN stays
      if (qi < count_q) {
        char *op = a.out + (int64_t)(begin_q + qi) * a.o_t + head * a.o_h;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int r = 0; r < 16; r += 4)
            *reinterpret_cast<u32x2 *>(op + (32 * d + 8 * (r / 4) + 4 * half) * 2) =
                (u32x2){Elem<T>::pack2(o[b][d][r] * inv, o[b][d][r + 1] * inv),
                        Elem<T>::pack2(o[b][d][r + 2] * inv, o[b][d][r + 3] * inv)};
      }
    }
  }
}

template <entro_dtype T, int D>
static entro_status launch_prompt(const PromptArg &a, hipStream_t s) {
  constexpr int QB = 1;
  constexpr uint32_t rows = 32u * QB * kWaves4;
  uint64_t grid = std::min<uint64_t>(a.total_q, (uint64_t)a.total_q / rows + a.n_seq);
  grid = std::min<uint64_t>(grid * a.n_heads, 1u << 30);
  grid = std::max<uint64_t>(1, cap_grid(grid));
  (void)hipGetLastError();
  hipLaunchKernelGGL((attn_prompt_kernel<T, D, QB>), dim3((uint32_t)grid), dim3(256), 2u * 2u * kTile * D * 2u, s, a);
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
  // the copies of a tile reach 64 rows with 32-bit offsets
  if (a->k.stride_t > (1 << 23) || a->v.stride_t > (1 << 23)) return ENTRO_E_UNSUPPORTED;
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
  p.scale = a->scale == 0.0f ? 1.0f : std::fabs(a->scale) * kLog2e;
  p.q_and = a->scale == 0.0f ? 0u : 0xFFFFFFFFu;
  p.q_xor = a->scale < 0.0f ? 0x80008000u : 0u;
  p.status = d_status;
  if (a->dtype == ENTRO_BF16)
    return a->head_dim == 64u   ? launch_prompt<ENTRO_BF16, 64>(p, stream)
           : a->head_dim == 96u ? launch_prompt<ENTRO_BF16, 96>(p, stream)
                                : launch_prompt<ENTRO_BF16, 128>(p, stream);
  return a->head_dim == 64u   ? launch_prompt<ENTRO_F16, 64>(p, stream)
         : a->head_dim == 96u ? launch_prompt<ENTRO_F16, 96>(p, stream)
                              : launch_prompt<ENTRO_F16, 128>(p, stream);
}

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
  uint32_t turned;                                  // this many of the first items in reverse order
  uint32_t heads;                                   // query heads of a workgroup: 1, 2 or 4 of one key/value head
  uint32_t parts;                                   // workgroups that share an item's keys
  float *part_o;                                    // parts > 1: [parts][total_q][n_heads][D]
  f32x2 *part_ml;                                   // [parts][total_q][n_heads]: maximum (of q . k), sum
  float scale;                                      // magnitude, times log2(e); 1 where the scale is 0
  float lift;                                       // see lift_of
  uint32_t q_and, q_xor;                            // on a pair of q: the scale's sign, and 0 where the scale is 0
  uint32_t *status;
};

constexpr uint32_t kTile = 64;     // keys of a step
constexpr uint32_t kWaves4 = 4;    // wavefronts of a workgroup

// Weights are held as 2^(score - maximum + lift), the maximum being behind by
// at most kLag (in powers of two): raising it means a pass over the outputs,
// and most tiles raise it by little.  f16 has 11 bits down to 2^-14 only, and
// many small weights can outweigh the largest together: its weights go up to
// 2^15, so that those down to 2^-26 of the largest have all their bits.  bf16 has
// all its bits down to 2^-126, and values up to the 32-bit sums' own largest: its
// weights are held so small that those of all keys are at most 1 together, and the
// sums stay finite wherever the values are.
template <entro_dtype T>
constexpr float kLag = T == ENTRO_F16 ? 3.0f : 8.0f;
template <entro_dtype T>
static float lift_of(uint32_t total_k) {
  return T == ENTRO_F16 ? 12.0f : -kLag<T> - std::ceil(std::log2((float)std::max(total_k, 1u)));
}

// The 16-bit values of w that are infinite or NaN: 0x8000 in their places.
template <entro_dtype T>
__device__ __forceinline__ uint32_t special(uint32_t w) {
  constexpr uint32_t exps = Elem<T>::kInf * 0x10001u, one = (0x8000u - Elem<T>::kInf) * 0x10001u;
  return ((w & exps) + one) & 0x80008000u;   // a full exponent carries into bit 15
}

// w with zeros in the place of infinities and NaN.
template <entro_dtype T>
__device__ __forceinline__ u32x4 without_special(u32x4 w) {
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] &= ~((special<T>(w[e]) >> 15) * 0xFFFFu);
  return w;
}

// Weights are 2^(s scale + (lift - maximum scale)), one instruction before the
// exponential, and what the second term is rounded by is the same for all keys of a
// maximum.  With maxima above this (in powers of two) it would show between tiles,
// or push weights out of their type: the maximum then is taken from the scores first.
constexpr float kFar = 256.0f;

// LDS place (16-byte piece) of piece c of row r of a tile of keys or values.
// Rows are 2 D bytes, and 256 bytes are read at once: one piece of 16 rows
// (keys), or four neighbouring pieces of 4 rows (values).  The pieces' order
// within a row varies with the row so that these lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t key_piece(uint32_t r, uint32_t c) {
  return D == 128 ? c ^ (r & 15u) : D == 64 ? c ^ ((r >> 1) & 7u) : c ^ ((r >> 2) & 3u);
}
template <int D>
__device__ __forceinline__ uint32_t value_piece(uint32_t r, uint32_t c) {
  return D == 128 ? c ^ (4u * (r & 3u)) : D == 64 ? c ^ (4u * ((r >> 1) & 1u)) : c;
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// o *= k in the registers that hold o: written as a product, the two ways
// through the (rare) branch around it get registers of their own, and the
// common way copies all outputs every tile.
__device__ __forceinline__ void scale_in_place(f32x16 &o, float k) {
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    float x = o[r];
    asm volatile("v_mul_f32 %0, %1, %0" : "+v"(x) : "v"(k));
    o[r] = x;
  }
}

// s -= x likewise.
__device__ __forceinline__ void less_in_place(f32x16 &s, float x) {
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    float y = s[r];
    asm volatile("v_sub_f32 %0, %0, %1" : "+v"(y) : "v"(x));
    s[r] = y;
  }
}

// The lane's number, not known to be the one it was: what follows from it is
// worked out at its use, or it would take registers from the loop over tiles.
__device__ __forceinline__ uint32_t fresh(uint32_t lane) {
  asm volatile("" : "+v"(lane));
  return lane;
}

// Instructions stay on their side of this place.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// Four rows (tokens) of 16 columns turned: a lane of a group of 16 gives the
// address of row lane / 4, columns 4 (lane % 4) on, and receives the four rows
// of column lane % 16.
__device__ __forceinline__ u32x2 read_turned(const void *at) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at));
}

// ---------------------------------------------------------------------------
// One workgroup takes 128 rows of one sequence and key/value head, a wavefront
// 32 of them: 128 queries of one query head or, for short prompts that would
// leave wavefronts empty, 32 (64) queries of four (two).  The keys come in
// tiles of 64 that all four wavefronts read from LDS, two tiles in turn: the
// next one's copies (global memory to LDS, 16 bytes a lane) are in flight while
// one is computed, one barrier a tile.  Copies go through a buffer resource
// that ends with the sequence's last row, so rows past it arrive as zeros.
//
// Scores are K Q^T and outputs V^T P^T with the queries as columns: a lane and
// the one 32 further hold one query's softmax, whose statistics they exchange
// where its maximum rises and at the end, and the weights leave the first product in
// the order in which the second takes them (row 8 (r / 4) + 4 half + r % 4 of a
// product is element r of a half; the values' tokens are read in that order).
// Values are turned on the way from LDS to registers.
//
// Weights are rounded to the element type, that of the values, which is what the
// matrix cores multiply; their sum is taken of the rounded ones, so that an output
// is a mean of values whose weights are each off by half a step and sum to 1.
//
// Values that a query must not see have weight 0, and 0 times an infinity
// would reach it: a tile that some queries see in part is looked over by the
// wavefronts that copied it, and where it holds infinities or NaN these are
// left out of the product and added at the end, to the queries that see them.
//
// Few queries with many keys (a piece of a prompt behind a long prefix) are too
// few workgroups, each with a long way: `parts` of them then take an equal
// share of an item's tiles each and leave their sums, which a second kernel
// joins.
//
// Bound by the matrix cores, and on them by the card's power: 16384 tokens of
// 32 / 8 heads of 128 (bf16, normal values) take 2.0 to 2.1 ms by the card, 1080
// TFLOP/s, at a clock of 1.5 to 1.7 GHz with the matrix cores busy 61% of it; with all values
// zero the same work runs at 1480 TFLOP/s (a library product of 8192^3: 1150 and
// 1690).  8192 tokens of 32 heads: of 96 462 us, 890 TFLOP/s; of 64 306 us, 900, with
// 7.7 vector instructions (the exponentials at a quarter of the rate among
// them) a matrix product at 96.  4096 tokens (32 / 8 heads of 128) 148 us, 2048
// 47 us, 8 sequences of 512 40 us.  37 tokens 6.5 us a call, which is latency: sums,
// the first tile, the queries, one tile's work, the outputs.
//
// Measured and not taken: the scores of the next tile between the exponentials
// of this one (their registers do not fit at 128; 2048 tokens 52 -> 66 us, 8192
// tokens of 96 5% slower), wavefront priorities, eight LDS reads ahead instead
// of six (nothing), 12 packed sequences longest first (131 -> 136 us), heads in
// groups of eight, whose keys an XCD's L2 holds (8192 tokens of 32 heads of 96
// 464 -> 482 us).
// ---------------------------------------------------------------------------
constexpr int wavefronts_per_simd(int d) { return d == 64 ? 3 : 2; }   // what the registers allow

template <entro_dtype T, int D>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(wavefronts_per_simd(D), wavefronts_per_simd(D)))) void
attn_prompt_kernel(PromptArg a) {
  constexpr int KS = D / 16, DT = D / 32, N = D / 32;
  constexpr uint32_t kBytes = kTile * D * 2u, kPieces = D / 8u;   // of a tile, of a row
  constexpr uint32_t kQueries = 32u;
  // four arrays: the compiler then knows that copies into one tile's need not
  // be waited for before the other's are read
  __shared__ u32x4 lds_k0[kBytes / 16u], lds_k1[kBytes / 16u], lds_v0[kBytes / 16u], lds_v1[kBytes / 16u];
  __shared__ uint32_t lds_special[2];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = rfl(tid >> 6), n = lane & 31u, half = lane >> 5;
  const uint32_t rows = kQueries * kWaves4 / a.heads;   // queries of a workgroup
  Spans spans(a.cu_q, a.total_q, a.n_seq, lane);
  if (blockIdx.x == 0u && blockIdx.y == 0u && wave == 0u)
    for (uint32_t b0 = 0; b0 < a.n_seq; b0 += 64u) {
      const Span k = span_of(a.cu_k, spans.place(b0), a.total_k), s = spans.at(b0);
      if (b0 + lane < a.n_seq && !(s.ok && k.ok)) atomicOr(a.status + b0 + lane, ENTRO_F_LENGTH);
    }

  // this lane's part of a tile's copies: N pieces of keys and N of values
  uint32_t k_off[N], v_off[N];
#pragma unroll
  for (uint32_t s = 0; s < (uint32_t)N; ++s) {
    const uint32_t i = (wave * N + s) * 64u + lane, r = i / kPieces, c = i % kPieces;
    k_off[s] = r * (uint32_t)a.k_t + key_piece<D>(r, c) * 16u;
    v_off[s] = r * (uint32_t)a.v_t + value_piece<D>(r, c) * 16u;
  }

  Span lq{}, lk{};                  // of the sequence this lane looked at last
  auto items = [&](uint32_t b0) {   // workgroups of sequence b0 + lane for a key/value head
    lk = span_of(a.cu_k, spans.place(b0), a.total_k);
    lq = spans.at(b0);
    return lk.ok ? (lq.count + rows - 1u) / rows : 0u;
  };
  const uint32_t turned = a.turned ? min(a.turned, count_items(a.n_seq, items)) : 0u;
  for (uint32_t slot = blockIdx.x; slot < a.n_heads / a.heads; slot += gridDim.x)
    for (uint32_t y = blockIdx.y;; y += gridDim.y) {
      const uint32_t at = y / a.parts, share = y % a.parts;
      // a key/value head's query heads and tiles stay on one XCD (workgroups go
      // around the 8 in turn) where n_kv is a multiple of 8
      const uint32_t kvh = slot % a.n_kv, head = kvh * (a.n_heads / a.n_kv) + slot / a.n_kv * a.heads + wave % a.heads;
      const uint32_t item = at < turned ? turned - 1u - at : at;
      const Found f = find_item(item, a.n_seq, lane, items);
      if (f.seq == a.n_seq) break;
      const uint32_t in = f.seq % 64u;   // the lane that has the sequence
      const uint32_t count_q = __builtin_amdgcn_readlane(lq.count, in), count_k = __builtin_amdgcn_readlane(lk.count, in);
      const uint32_t begin_q = __builtin_amdgcn_readlane(lq.begin, in), begin_k = __builtin_amdgcn_readlane(lk.begin, in);
      // the last queries first: they have the most keys
      const uint32_t wg0 = ((count_q + rows - 1u) / rows - 1u - f.local) * rows;
      const uint32_t q0 = wg0 + wave / a.heads * kQueries, qi = q0 + n;
      const int64_t shift = (int64_t)count_k - count_q;       // query i sees keys up to i + shift
      const char *kb = a.k + begin_k * a.k_t + kvh * a.k_h, *vb = a.v + begin_k * a.v_t + kvh * a.v_h;

      f32x16 o[DT];
      float m = -INFINITY, l = 0.0f;   // l: this lane's keys only
      bool far = false;                // some of the wavefront's maxima are, see kFar
#pragma unroll
      for (int d = 0; d < DT; ++d)
        for (int r = 0; r < 16; ++r) o[d][r] = 0.0f;
      // keys that the workgroup, and this wavefront, see
      const int64_t wg_end = max((int64_t)0, (int64_t)min(wg0 + rows, count_q) + shift);
      const int64_t my_end = q0 < count_q ? max((int64_t)0, (int64_t)min(q0 + kQueries, count_q) + shift) : 0;
      const uint32_t all_tiles = rfl((uint32_t)((wg_end + kTile - 1) / kTile)), pairs = (all_tiles + 1u) / 2u;
      const uint32_t mine = (uint32_t)((my_end + kTile - 1) / kTile);
      // this workgroup's tiles: `begin`, even, to `tiles`
      const uint32_t begin = rfl((uint32_t)((uint64_t)pairs * share / a.parts) * 2u);
      const uint32_t tiles = rfl(min(all_tiles, (uint32_t)((uint64_t)pairs * (share + 1u) / a.parts) * 2u));
      // tiles that every query of the workgroup sees whole, an even number
      const uint32_t full = (uint32_t)min((int64_t)tiles, max((int64_t)0, (int64_t)wg0 + shift + 1) / kTile) & ~1u;

      // 32 rows for this wavefront in a tile's place
      auto quarter = [&](u32x4 *k, u32x4 *v) { return (wave < 2u ? k : v) + (wave & 1u) * (kBytes / 32u); };
      // A tile's rows (none past the last tile: the copies then write zeros), and
      // piece s of this wavefront's N copies.
      auto rows_at = [&](const char *from, int64_t stride, uint32_t tile) {
        const uint32_t n_rows = tile < tiles ? min(kTile, count_k - tile * kTile) : 0u;
        const uint32_t bytes = n_rows ? (n_rows - 1u) * (uint32_t)stride + 2u * D : 0u;
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(from + (int64_t)(tile * kTile) * stride), 0, (int)rfl(bytes),
                                                 0x00020000);
      };
      auto copy = [&](__amdgpu_buffer_rsrc_t r, const uint32_t (&off)[N], u32x4 *to, uint32_t s) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(to + (wave * N + s) * 64u), 16, (int)off[s], 0, 0, 0);
      };
      auto copy_all = [&](uint32_t tile, u32x4 *to_k, u32x4 *to_v) {
        const __amdgpu_buffer_rsrc_t rk = rows_at(kb, a.k_t, tile), rv = rows_at(vb, a.v_t, tile);
#pragma unroll
        for (uint32_t s = 0; s < (uint32_t)N; ++s) copy(rk, k_off, to_k, s);
#pragma unroll
        for (uint32_t s = 0; s < (uint32_t)N; ++s) copy(rv, v_off, to_v, s);
      };
      __syncthreads();   // the last item's tiles and marks have been read
      if (tid < 2u) lds_special[tid] = 0u;
      __syncthreads();   // no mark is set before
      if (begin < tiles) copy_all(begin, lds_k0, lds_v0);
      // the wavefront's queries, by way of its quarter of the other tile's place
      // (whole rows a copy; rows past the end are zeros)
      u32x4 qf[KS];
      {
        const uint32_t ln = fresh(lane);
        u32x4 *at = quarter(lds_k1, lds_v1);
        const uint32_t n_rows = q0 < count_q ? min(kQueries, count_q - q0) : 0u;
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char *>(a.q + (int64_t)(begin_q + q0) * a.q_t + head * a.q_h), 0,
            (int)rfl(n_rows ? (n_rows - 1u) * (uint32_t)a.q_t + 2u * D : 0u), 0x00020000);
#pragma unroll
        for (uint32_t s = 0; s < (uint32_t)KS; ++s) {
          const uint32_t i = s * 64u + ln, row = i / kPieces;
          __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(at + s * 64u), 16,
                                                   (int)(row * (uint32_t)a.q_t + key_piece<D>(row, i % kPieces) * 16u), 0, 0, 0);
        }
        wait_lds_copy();
#pragma unroll
        for (int s = 0; s < KS; ++s)
          qf[s] = (at[(ln & 31u) * kPieces + key_piece<D>(ln & 31u, 2 * s + (ln >> 5))] & a.q_and) ^ a.q_xor;
      }

      // The two products are written in the order in which their instructions
      // should run, which the barriers keep the compiler to: LDS reads several
      // products ahead of their use, and the exponentials of the next 16 keys
      // between the products of the last.  (Its own order waited for each read.)
      auto key = [&](const u32x4 *kt, uint32_t ln, int i) {   // keys 32 (i / KS) on, dimensions 16 (i % KS) on
        const uint32_t r = ln & 31u;
        const uint32_t at = r * (2u * D) + (uint32_t)(i / KS * 64 * D) + key_piece<D>(r, 2 * (i % KS) + (ln >> 5)) * 16u;
        return *reinterpret_cast<const u32x4 *>(reinterpret_cast<const char *>(kt) + at);
      };
      auto scores = [&](f32x16 (&s)[2], const u32x4 *kt, uint32_t ln, auto between) {
        constexpr int AHEAD = 6;
        u32x4 w[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) w[i] = key(kt, ln, i);
        in_order();
#pragma unroll
        for (int i = 0; i < 2 * KS; ++i) {
          if (i % KS == 0)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[i / KS][r] = 0.0f;
          s[i / KS] = Elem<T>::mfma32(w[i % AHEAD], qf[i % KS], s[i / KS]);
          if (i + AHEAD < 2 * KS) w[i % AHEAD] = key(kt, ln, i + AHEAD);
          between(i);
          in_order();
        }
      };
      // Maximum of the lane's query up to this tile.
      auto raise_to = [&](f32x16 (&s)[2]) {
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[i][r]);
        if (far || __any((mx - m) * a.scale > kLag<T>)) {
          mx = max32(mx);
          const float mn = (mx - m) * a.scale > kLag<T> ? mx : m;
          const float k = mn == -INFINITY ? 1.0f : exp2_fast((m - mn) * a.scale);
          m = mn;
          l *= k;
#pragma unroll
          for (int d = 0; d < DT; ++d) scale_in_place(o[d], k);
          far = __any(m != -INFINITY && fabsf(m) * a.scale > kFar);
          if (far) {
            const float less = m == -INFINITY ? 0.0f : m;
            less_in_place(s[0], less);
            less_in_place(s[1], less);
          }
        }
      };
      // Values of 16 tokens from 16 c on, of dimensions 32 d on: the lane gives
      // the place of row 4 half + (lane / 4) % 4 and the one 8 further.
      auto value = [&](const u32x4 *vt, uint32_t ln, int c, int d) {
        const uint32_t r = 4u * (ln >> 5) + ((ln >> 2) & 3u), piece = 2u * ((ln >> 4) & 1u) + ((ln >> 1) & 1u);
        // (one step from the array: further ones, and the compiler loses track
        // of which it is)
        const uint32_t at = (uint32_t)(c * 32 * D) + r * (2u * D) + (ln & 1u) * 8u + value_piece<D>(r, 4 * d + piece) * 16u;
        const u32x2 lo = read_turned(reinterpret_cast<const char *>(vt) + at),
                    hi = read_turned(reinterpret_cast<const char *>(vt) + (at + 16u * D));
        return (u32x4){lo.x, lo.y, hi.x, hi.y};
      };
      // Outputs of a tile; kept(w): w, or what is left of it.
      auto outputs = [&](const f32x16 (&s)[2], const u32x4 *vt, uint32_t ln, auto kept) {
        const float off = m == -INFINITY ? 0.0f : far ? a.lift : a.lift - m * a.scale;
        u32x4 p[2], w[DT];
        auto pair = [&](int c, int e) {   // weights of keys 16 c + 2 e, 2 e + 1 (in the products' order)
          const float x = exp2_fast(__builtin_fmaf(s[c / 2][c % 2 * 8 + 2 * e], a.scale, off));
          const float y = exp2_fast(__builtin_fmaf(s[c / 2][c % 2 * 8 + 2 * e + 1], a.scale, off));
          p[c % 2][e] = Elem<T>::pack2(x, y);
          l = Elem<T>::add2(p[c % 2][e], l);
        };
#pragma unroll
        for (int d = 0; d < DT; ++d) w[d] = value(vt, ln, 0, d);
        in_order();
#pragma unroll
        for (int e = 0; e < 4; ++e) pair(0, e);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            o[d] = Elem<T>::mfma32(kept(w[d]), p[c % 2], o[d]);
            if (c < 3) {
              w[d] = value(vt, ln, c + 1, d);
#pragma unroll
              for (int e = 4 * d / DT; e < 4 * (d + 1) / DT; ++e) pair(c + 1, e);
            }
            in_order();
          }
      };

      auto whole = [&](uint32_t t, const u32x4 *kt, const u32x4 *vt, u32x4 *next_k, u32x4 *next_v) {
        wait_lds_copy();
        __syncthreads();   // tile t is there; the other buffer has been read
        // the next tile's copies between the products: one after another they
        // keep the wavefront from anything else
        const __amdgpu_buffer_rsrc_t rk = rows_at(kb, a.k_t, t + 1u), rv = rows_at(vb, a.v_t, t + 1u);
        f32x16 s[2];
        scores(s, kt, lane, [&](int i) {
          if (i % 2) return;
          if (i / 2 < N) copy(rk, k_off, next_k, i / 2);
          else if (i / 2 < 2 * N) copy(rv, v_off, next_v, i / 2 - N);
        });
        raise_to(s);
        outputs(s, vt, lane, [](u32x4 w) { return w; });
      };
      bool left_out = false;   // infinities or NaN among the values of a tile seen in part
      auto part = [&](uint32_t t, const u32x4 *kt, const u32x4 *vt, u32x4 *next_k, u32x4 *next_v) {
        wait_lds_copy();
        uint32_t any = 0;
#pragma unroll
        for (uint32_t i = 0; i < (uint32_t)N; ++i) {
          const u32x4 w = vt[(wave * N + i) * 64u + lane];
          for (int e = 0; e < 4; ++e) any |= special<T>(w[e]);
        }
        if (any) lds_special[t & 1u] = 1u;
        __syncthreads();
        if (t + 1u < tiles) copy_all(t + 1u, next_k, next_v);
        // (a mark stays for the tiles after: they take the longer way for nothing)
        const bool special_here = lds_special[t & 1u] != 0u;
        if (t >= mine) return;
        const uint32_t ln = fresh(lane);
        f32x16 s[2];
        scores(s, kt, ln, [](int) {});
        const int64_t keys = (int64_t)(q0 + (ln & 31u)) + shift + 1 - (int64_t)t * kTile;   // of this tile, seen by the query
        const int seen = (int)min(max(keys, (int64_t)0), (int64_t)kTile) - 4 * (int)(ln >> 5);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          for (int r = 0; r < 16; ++r) s[i][r] = 32 * i + 8 * (r / 4) + r % 4 < seen ? s[i][r] : -INFINITY;
        raise_to(s);
        if (special_here) {
          left_out = true;
          outputs(s, vt, ln, [](u32x4 w) { return without_special<T>(w); });
        } else {
          outputs(s, vt, ln, [](u32x4 w) { return w; });
        }
      };
      uint32_t t = begin;
      for (; t < full; t += 2u) {
        whole(t, lds_k0, lds_v0, lds_k1, lds_v1);
        whole(t + 1u, lds_k1, lds_v1, lds_k0, lds_v0);
      }
      for (; t < tiles; ++t) {
        const bool odd = t & 1u;
        part(t, odd ? lds_k1 : lds_k0, odd ? lds_v1 : lds_v0, odd ? lds_k0 : lds_k1, odd ? lds_v0 : lds_v1);
      }
      // the last tile was seen whole: the copies (of zeros) sent out during it
      // may still be on their way to the place that the outputs pass through
      if (full == tiles) {
        wait_lds_copy();
        __syncthreads();
      }
      const int64_t at_row = (int64_t)begin_q + q0;

      const float sum = add32(l);
      const float inv = a.parts > 1u ? 1.0f : sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;   // NaN stays
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= inv;
      if (left_out)
        for (int64_t j = (int64_t)max(begin, full) * kTile; j < min(my_end, (int64_t)tiles * kTile); ++j) {
          const char *vp = vb + j * a.v_t + half * 8u;
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
              const u32x2 w = *reinterpret_cast<const u32x2 *>(vp + (32 * d + 2 * r) * 2);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t x = e & 1 ? w[e / 2] >> 16 : w[e / 2];
                const bool add = j <= (int64_t)qi + shift && (x & Elem<T>::kInf) == Elem<T>::kInf;
                o[d][r + e] += add ? Elem<T>::lo(x) : 0.0f;
              }
            }
        }
      if (a.parts > 1u) {
        const uint32_t ln = fresh(lane);
        if (q0 + (ln & 31u) < count_q) {
          const uint64_t row = ((uint64_t)share * a.total_q + (uint64_t)(at_row + (ln & 31u))) * a.n_heads + head;
          float *to = a.part_o + row * D + (ln >> 5) * 4u;
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
              *reinterpret_cast<f32x4 *>(to + 32 * d + 2 * r) = (f32x4){o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]};
          if (ln < 32u) a.part_ml[row] = (f32x2){m, sum};
        }
        continue;
      }
      // rows out by way of the place of the tile before the last, which every
      // wavefront has left, so that a store writes whole rows
      {
        const uint32_t ln = fresh(lane);
        u32x4 *at = tiles & 1u ? quarter(lds_k1, lds_v1) : quarter(lds_k0, lds_v0);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int r = 0; r < 16; r += 4)
            reinterpret_cast<u32x2 *>(at)[2u * ((ln & 31u) * kPieces + key_piece<D>(ln & 31u, 4 * d + r / 4)) + (ln >> 5)] =
                (u32x2){Elem<T>::pack2(o[d][r], o[d][r + 1]), Elem<T>::pack2(o[d][r + 2], o[d][r + 3])};
#pragma unroll
        for (uint32_t s = 0; s < (uint32_t)KS; ++s) {
          const uint32_t i = s * 64u + ln, row = i / kPieces, c = i % kPieces;
          const u32x4 w = at[row * kPieces + key_piece<D>(row, c)];
          if (q0 + row < count_q)
            *reinterpret_cast<u32x4 *>(a.out + (int64_t)(begin_q + q0 + row) * a.o_t + head * a.o_h + c * 16u) = w;
        }
      }
    }
}

// Joins the parts of split items: D / 4 threads a row and head, as many rows of
// a sequence a workgroup as it has threads for, eight parts' reads at once.
template <entro_dtype T, int D>
__global__ __launch_bounds__(256) void attn_prompt_join_kernel(PromptArg a) {
  constexpr uint32_t L = D / 4u, R = 256u / L, kBatch = 8u;
  const uint32_t tid = threadIdx.x, lane = tid & 63u, d = tid % L * 4u;
  const auto factor = [&](float m, float all) { return m == all ? 1.0f : exp2_fast((m - all) * a.scale); };   // as join_factor
  Span lq{}, lk{};
  Spans spans(a.cu_q, a.total_q, a.n_seq, lane);
  auto items = [&](uint32_t b0) {
    lk = span_of(a.cu_k, spans.place(b0), a.total_k);
    lq = spans.at(b0);
    return lk.ok ? (lq.count + R - 1u) / R : 0u;
  };
  for (uint32_t head = blockIdx.x; head < a.n_heads; head += gridDim.x)
    for (uint32_t y = blockIdx.y;; y += gridDim.y) {
      const Found f = find_item(y, a.n_seq, lane, items);
      if (f.seq == a.n_seq) break;
      const uint32_t in = f.seq % 64u;
      const uint32_t count_q = __builtin_amdgcn_readlane(lq.count, in), begin_q = __builtin_amdgcn_readlane(lq.begin, in);
      const uint32_t i = f.local * R + tid / L;
      if (tid < R * L && i < count_q) {
        const uint64_t row = (uint64_t)(begin_q + i) * a.n_heads + head, step = (uint64_t)a.total_q * a.n_heads;
        float m = -INFINITY, l = 0.0f;
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
        for (uint32_t p0 = 0; p0 < a.parts; p0 += kBatch) {
          f32x2 ml[kBatch];
          f32x4 o[kBatch];
#pragma unroll
          for (uint32_t j = 0; j < kBatch; ++j) {
            const uint64_t at = row + min(p0 + j, a.parts - 1u) * step;
            ml[j] = a.part_ml[at];
            o[j] = *reinterpret_cast<const f32x4 *>(a.part_o + at * D + d);
          }
          float mn = m;
#pragma unroll
          for (uint32_t j = 0; j < kBatch; ++j) mn = fmaxf(mn, ml[j].x);
          const float k = factor(m, mn);
          x *= k;
          l *= k;
          m = mn;
#pragma unroll
          for (uint32_t j = 0; j < kBatch; ++j) {
            if (p0 + j >= a.parts) break;
            const float kj = factor(ml[j].x, m);
            x += kj * o[j];
            l += kj * ml[j].y;
          }
        }
        const float r = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;   // NaN stays
        *reinterpret_cast<u32x2 *>(a.out + (int64_t)(begin_q + i) * a.o_t + head * a.o_h + d * 2u) =
            (u32x2){Elem<T>::pack2(x[0] * r, x[1] * r), Elem<T>::pack2(x[2] * r, x[3] * r)};
      }
    }
}

// A call's workgroups: `slots` times `items` (at most) times `parts`.
struct PromptGrid {
  uint32_t heads, slots, parts;
  uint64_t items;
};
static PromptGrid prompt_grid(uint32_t n_seq, uint32_t total_q, uint32_t total_k, uint32_t n_heads, uint32_t n_kv,
                              uint32_t head_dim) {
  PromptGrid g{};
  const uint32_t group = n_heads / n_kv;
  // sequences of 64 queries on average: 256 x 64 (32 / 8 heads of 128) 215 us
  // by queries, 140 by heads; 128 x 128 the same; 16 x 1024 212 and 220
  const bool small = total_q <= 64ull * n_seq;
  g.heads = !small ? 1u : group % 4u == 0u ? 4u : group % 2u == 0u ? 2u : 1u;
  g.slots = n_heads / g.heads;
  const uint32_t rows = 32u * kWaves4 / g.heads;
  g.items = std::min<uint64_t>(total_q, (total_q + (uint64_t)n_seq * (rows - 1u)) / rows);
  g.parts = 1u;
  const uint64_t all = g.items * g.slots, tiles = total_k / n_seq / kTile;
  if (all == 0u || all > 256u || tiles < 16u) return g;
  // Too few workgroups for the CUs: with n parts the way through the tiles takes
  // a share of n less (0.6, 0.8, 0.9 us a tile at head dimension 64, 96, 128; the
  // longest of several sequences is taken to be half longer than the average,
  // which is all the host knows), the sums of all rows are written and read n
  // times (about 6 bytes a picosecond), and the second kernel takes some 6 us.
  // The n with the least of both, from 4 tiles a part and 32 parts (the second
  // kernel's own way) on down.  32 / 8 heads of 128, split and not: one query,
  // 16000 keys 30 and 216 us, 1100 keys 17 and 23; 128 queries behind 4000 keys 30
  // and 64; 9 x 13 with 3506 keys each 44 and 71; 512 behind 4000 54 and 70; 6 of up
  // to 45 queries with up to 3664 keys 27 and 57; one query of 16000 keys beside 15 of
  // 200 83 and 271 (all get the parts of their average).  The guess is off for 12 x 20
  // behind 1300: 31 and 29.
  const double way = (0.3 + 0.005 * head_dim) * (n_seq > 1u ? 1.5 : 1.0) * (double)tiles;
  const double sums = (double)total_q * n_heads * head_dim * 8.0 / 6e6;
  uint64_t parts = std::min<uint64_t>({512u / all, tiles / 4u, 32u, (uint64_t)std::sqrt(way / sums)});
  if (parts > 8u) parts &= ~7ull;   // the second kernel reads eight at once: 9 parts 28 us where 8 take 26
  if (parts > 1u && way - way / (double)parts > 6.0 + sums * (double)parts) g.parts = (uint32_t)parts;
  return g;
}

template <entro_dtype T, int D>
static entro_status launch_prompt(PromptArg &a, const PromptGrid &g, hipStream_t s) {
  a.lift = lift_of<T>(a.total_k);
  // Where all workgroups run at once, the 256 first get a CU each and the rest
  // follow in the same order: the first ones' order is turned around, so that
  // the CUs with the least of them to do get the most of the rest.
  a.turned = a.parts == 1u && g.items * g.slots <= 512u ? 256u / g.slots : 0u;
  if (a.parts > 1u) a.part_ml = reinterpret_cast<f32x2 *>(a.part_o + (uint64_t)a.parts * a.total_q * a.n_heads * D);
  (void)hipGetLastError();
  hipLaunchKernelGGL((attn_prompt_kernel<T, D>), grid2(g.slots, g.items * a.parts), dim3(256), 0, s, a);
  if (hipGetLastError() != hipSuccess) return ENTRO_E_HIP;
  if (a.parts > 1u) {
    const uint32_t rows = 256u / (D / 4u);
    const uint64_t items = std::min<uint64_t>(a.total_q, (uint64_t)a.total_q / rows + a.n_seq);
    hipLaunchKernelGGL((attn_prompt_join_kernel<T, D>), grid2(a.n_heads, items), dim3(256), 0, s, a);
    if (hipGetLastError() != hipSuccess) return ENTRO_E_HIP;
  }
  return ENTRO_OK;
}

}  // namespace entro

using namespace entro;

extern "C" uint64_t entro_attn_prompt_work_bytes(uint32_t n_seq, uint32_t total_q, uint32_t total_k, uint32_t n_heads,
                                                 uint32_t n_kv_heads, uint32_t head_dim) {
  if (n_seq == 0 || check_heads(n_heads, n_kv_heads, head_dim, ENTRO_BF16) != ENTRO_OK) return 0;
  const uint64_t parts = prompt_grid(n_seq, total_q, total_k, n_heads, n_kv_heads, head_dim).parts;
  return parts > 1u ? parts * total_q * n_heads * (head_dim + 2ull) * 4ull : 0u;
}

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
  if (a->d_work && ((reinterpret_cast<uintptr_t>(a->d_work) & 15u) ||
                    a->work_bytes < entro_attn_prompt_work_bytes(a->n_seq, a->total_q, a->total_k, a->n_heads,
                                                                 a->n_kv_heads, a->head_dim)))
    return ENTRO_E_INVAL;
  // copies reach up to 64 rows with 32-bit offsets
  if (a->q.stride_t > (1 << 23) || a->k.stride_t > (1 << 23) || a->v.stride_t > (1 << 23)) return ENTRO_E_UNSUPPORTED;
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
  const PromptGrid g = prompt_grid(a->n_seq, a->total_q, a->total_k, a->n_heads, a->n_kv_heads, a->head_dim);
  p.heads = g.heads;
  p.parts = a->d_work ? g.parts : 1u;
  p.part_o = static_cast<float *>(a->d_work);
  if (a->dtype == ENTRO_BF16)
    return a->head_dim == 64u   ? launch_prompt<ENTRO_BF16, 64>(p, g, stream)
           : a->head_dim == 96u ? launch_prompt<ENTRO_BF16, 96>(p, g, stream)
                                : launch_prompt<ENTRO_BF16, 128>(p, g, stream);
  return a->head_dim == 64u   ? launch_prompt<ENTRO_F16, 64>(p, g, stream)
         : a->head_dim == 96u ? launch_prompt<ENTRO_F16, 96>(p, g, stream)
                              : launch_prompt<ENTRO_F16, 128>(p, g, stream);
}

extern "C" uint32_t entro_attn_set_max_workgroups(uint32_t n) { return g_attn_max_workgroups.exchange(n); }

// HIP kernels (gfx950) and entry points of the attention of chunks over the 8-bit
// cache: entro_attn_chunk.  Layout and definition are in entro_attn.h.
#include <algorithm>
#include <type_traits>

#include "entro_attn_device.h"
#include "entro_internal.h"

namespace entro {

constexpr uint32_t kTile = 64;          // tokens of a step
constexpr uint32_t kShareTiles = 4;     // least tiles of a workgroup's share
constexpr float kFloatMax = 3.40282347e38f;

struct ChunkArg {
  const int8_t *k_codes, *v_codes;
  const float *k_scales, *v_scales;
  const int32_t *table;
  uint64_t table_stride;
  uint32_t table_pages, n_seq, n_pages, n_kv;
  uint32_t page_log2;
  const char *q;
  char *out;
  int64_t q_t, q_h, o_t, o_h;   // bytes
  const int32_t *cu, *lens;
  uint32_t total_q;
  uint32_t n_heads, group;      // group: query heads per key/value head
  uint32_t heads, parts;        // query heads of a workgroup, workgroups per key/value head for all of them
  uint32_t block_log2;          // tokens of a workgroup
  uint32_t shares;              // that the tiles of a key/value head are split into at most
  float scale;                  // magnitude, times log2(e)
  uint32_t q_xor;               // on a pair of q: the scale's sign
  float *part_o;                // [n_kv parts][shares][2][rows][D]
  f32x4 *part_s;                // [n_kv parts][shares][2][rows]: a row's State
  uint32_t *status;
};

// A sequence's part in a call: queries begin .. begin + count - 1, the last of len
// tokens.
struct Seq {
  uint32_t begin, count, len;
};
// of sequence b0 + lane, 64 in turn (none: all 0)
__device__ __forceinline__ Seq chunk_seq(const ChunkArg &a, Spans &spans, uint32_t b0, bool *fine = nullptr) {
  const int32_t n = a.lens[spans.place(b0)];
  const Span s = spans.at(b0);
  const bool ok = s.ok && n >= 0 && (uint64_t)n <= ((uint64_t)a.table_pages << a.page_log2);
  if (fine) *fine = ok;
  return {ok ? s.begin : 0u, ok ? s.count : 0u, ok ? (uint32_t)n : 0u};
}

// The blocks of a sequence: 2^L tokens each, the last one maybe fewer.  A block
// has the tiles that its last token sees, and one at least.  L is a whole number so
// that the tiles of a sequence's first blocks can be written down.
struct Blocks {
  uint32_t L, n, count;
  int64_t ahead;   // tokens in front of the first query; below 0 where the first ones see none
  __device__ Blocks(uint32_t log2, const Seq &s)
      : L(log2), n((uint32_t)(((uint64_t)s.count + (1ull << log2) - 1u) >> log2)), count(s.count),
        ahead((int64_t)s.len - (int64_t)s.count) {}
  // tiles of the first x blocks, all of them full: the sum over y = 1 .. x of
  // max(1, ceil((ahead + 2^L y) / 64))
  __device__ uint64_t full(uint32_t blocks) const {
    const int64_t x = blocks;
    if (L <= 6u) {   // ceil(ceil((ahead + 2^L y) / 2^L) / 2^(6 - L))
      const uint32_t j = 6u - L;
      const int64_t s = (ahead + (1 << L) - 1) >> L;
      const auto sum = [&](int64_t m) {   // of ceil(y / 2^j) over y = 1 .. m
        const int64_t e = m >> j, r = m & ((1 << j) - 1);
        return ((e * (e + 1) / 2) << j) + r * (e + 1);
      };
      if (s >= 0) return (uint64_t)(sum(x + s) - sum(s));
      return (uint64_t)(x + s > 0 ? -s + sum(x + s) : x);
    }
    const uint32_t j = L - 6u;
    const int64_t s = (ahead + 63) >> 6, z = s < 0 ? min(x, -s >> j) : 0;   // z blocks see nothing
    return (uint64_t)(z + (x - z) * s + (((x * (x + 1) - z * (z + 1)) / 2) << j));
  }
  __device__ uint32_t tiles(uint32_t b) const {
    const int64_t end = ahead + (int64_t)min(((uint64_t)b + 1u) << L, (uint64_t)count);
    return end > 0 ? (uint32_t)((end + kTile - 1) / kTile) : 1u;
  }
  __device__ uint64_t all() const { return n ? full(n - 1u) + tiles(n - 1u) : 0u; }
  // the block of tile t
  __device__ uint32_t of(uint64_t t) const {
    uint32_t lo = 0, hi = n - 1u;
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1u) / 2u;
      if (full(mid) <= t) lo = mid;
      else hi = mid - 1u;
    }
    return lo;
  }
};

__device__ __forceinline__ uint64_t wave_scan64(uint64_t v) {
  const auto step = [&](uint32_t lo, uint32_t hi) { v += ((uint64_t)hi << 32) | lo; };
#define ENTRO_STEP(CTRL, ROWS) step(dpp0<CTRL, ROWS>((uint32_t)v), dpp0<CTRL, ROWS>((uint32_t)(v >> 32)))
  ENTRO_STEP(0x111, 0xF);
  ENTRO_STEP(0x112, 0xF);
  ENTRO_STEP(0x114, 0xF);
  ENTRO_STEP(0x118, 0xF);
  ENTRO_STEP(0x142, 0xA);
  ENTRO_STEP(0x143, 0xC);
#undef ENTRO_STEP
  return v;
}
__device__ __forceinline__ uint32_t lane_of(uint32_t v, uint32_t lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, (int)lane);
}
__device__ __forceinline__ uint64_t lane_of(uint64_t v, uint32_t lane) {
  return ((uint64_t)lane_of((uint32_t)(v >> 32), lane) << 32) | lane_of((uint32_t)v, lane);
}
__device__ __forceinline__ float lane_of(float v, uint32_t lane) {
  return __builtin_bit_cast(float, lane_of(__builtin_bit_cast(uint32_t, v), lane));
}

// A place among the tiles of all sequences' blocks, one after another.
struct Place {
  const ChunkArg &a;
  uint32_t lane;
  Spans spans;
  uint32_t b0;       // own: of sequence b0 + lane
  Seq own;
  uint32_t seq;      // n_seq: past the last
  uint32_t block;
  uint64_t before;   // tiles before the block
  __device__ Place(const ChunkArg &arg, uint32_t lane_)
      : a(arg), lane(lane_), spans(arg.cu, arg.total_q, arg.n_seq, lane_) {}
  __device__ uint64_t count_all() {
    uint64_t sum = 0;
    for (b0 = 0; b0 < a.n_seq; b0 += 64u) {
      own = chunk_seq(a, spans, b0);
      sum += lane_of(wave_scan64(Blocks(a.block_log2, own).all()), 63u);
    }
    return sum;
  }
  __device__ void find(uint64_t tile) {
    uint64_t sum = 0;
    for (b0 = 0; b0 < a.n_seq; b0 += 64u) {
      own = chunk_seq(a, spans, b0);
      const uint64_t mine = Blocks(a.block_log2, own).all(), run = wave_scan64(mine);
      const uint64_t past = __ballot(sum + run > tile);
      if (past) {
        const uint32_t at = (uint32_t)__builtin_ctzll(past);
        seq = rfl(b0 + at);
        sum += lane_of(run - mine, at);
        const Blocks b(a.block_log2, here());
        block = rfl(b.of(tile - sum));
        before = rfl64(sum + b.full(block));
        return;
      }
      sum += lane_of(run, 63u);
    }
    seq = a.n_seq;
  }
  __device__ Seq here() const {
    const uint32_t at = seq - b0;
    return {lane_of(own.begin, at), lane_of(own.count, at), lane_of(own.len, at)};
  }
  // to the next block
  __device__ void next() {
    const Blocks b(a.block_log2, here());
    before += b.tiles(block);
    if (++block < b.n) return;
    block = 0u;
    while (++seq < a.n_seq) {
      if (seq - b0 == 64u) own = chunk_seq(a, spans, b0 += 64u);
      if (here().count) return;
    }
  }
};

// All tiles of a key/value head in equal shares (to one tile), one workgroup each and
// as many as the GPU holds at once: share w has tiles begin(w) .. begin(w + 1) - 1.  A
// share's part of one block is a piece; a block in one piece is finished by its
// workgroup, the others' pieces are joined by the second kernel.  A share has at most
// two pieces of blocks that it does not finish: one that lacks the block's first
// tile, always the share's first (place 0), and one that has it, always its last
// (place 1).
struct Shares {
  uint64_t tiles;
  uint32_t n;
  __device__ uint64_t begin(uint32_t w) const { return w * tiles / n; }
};
__device__ __forceinline__ Shares shares_of(const ChunkArg &a, uint64_t tiles) {
  return {tiles, (uint32_t)min((uint64_t)a.shares, max((uint64_t)1, tiles / kShareTiles))};
}

// What is known of a row (one query of one head) beside its outputs, in powers of
// two: the largest score m, the weights' sum l relative to 2^m, and the exponent g
// of the outputs' unit, relative to 2^m too.  top: the largest exponent, less m, with
// which values have been added (their scale's times their weight's); the unit stays
// near it, so that outputs keep their bits whatever the pages' scales are.
struct State {
  float m, l, g, top;
};
constexpr float kUnit = 11.5f;   // the unit lies by about as much below top

// log2 of a page's value scale (below 2^-126: 0)
struct Scale {
  float whole, part, log;   // scale = part * 2^whole
  __device__ explicit Scale(float s) {
    int e;
    part = s >= 1.17549435e-38f || !(s == s) ? __builtin_frexpf(s, &e) : 0.0f;
    if (!(s >= 1.17549435e-38f) || s == INFINITY) e = 0;
    whole = (float)e;
    log = part == 0.0f ? -INFINITY : whole + __log2f(part);
  }
};

// A value of each four lanes in another order (0: the first one's), and the largest.
template <int CTRL>
__device__ __forceinline__ float quad(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, quad<0xB1>(v));      // 1, 0, 3, 2
  return fmaxf(v, quad<0x4E>(v));   // 2, 3, 0, 1
}

// Instructions stay on their side of this place.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }
// The value, computed anew from here on: what follows from it is not kept in
// registers from before.
__device__ __forceinline__ uint32_t fresh(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Changes in the registers that hold the value: written as an expression, the two
// ways through a (rare) branch around it get registers of their own, and the common
// way copies all of them every tile.  The matrix instructions' results are waited for
// first.
__device__ __forceinline__ void results_there() { asm volatile("s_nop 15\n\ts_nop 15"); }
__device__ __forceinline__ void scale_in_place(f32x16 &o, float k) {
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    float x = o[r];
    asm volatile("v_mul_f32 %0, %1, %0" : "+v"(x) : "v"(k));
    o[r] = x;
  }
}
// o = o k + z
__device__ __forceinline__ void add_in_place(f32x16 &o, float k, const f32x16 &z) {
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    float x = o[r];
    asm volatile("v_fma_f32 %0, %0, %1, %2" : "+v"(x) : "v"(k), "v"(z[r]));
    o[r] = x;
  }
}
// -infinity where token 16 b + j is not seen (16 b + j >= seen)
__device__ __forceinline__ void hide_in_place(f32x16 &x, int b, int32_t seen) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float y = x[8 * (b & 1) + j];
    asm volatile("v_cmp_lt_i32 vcc, %1, %2\n\ts_nop 1\n\tv_cndmask_b32 %0, %3, %0, vcc"
                 : "+v"(y) : "n"(16 * b + j), "v"(seen), "v"(-INFINITY) : "vcc");
    x[8 * (b & 1) + j] = y;
  }
}

__device__ __forceinline__ f32x16 mfma(f16v8 a, f16v8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

template <int D, int W>
struct Lds {
  static constexpr uint32_t kRow = D * 2 + 16;          // bytes of a key's row and
  static constexpr uint32_t vRow = kTile * 2 + 16;      // of a dimension's: rows begin four banks further
  static constexpr uint32_t kBytes = kTile * kRow, vBytes = D * vRow, bytes = 2 * (kBytes + vBytes);
};

// A tile as a lane sees it.
template <typename L>
struct Tile {
  const char *k, *v;   // the key that is its row of the first product, the dimension that is its row of the second
  int32_t base;        // first token
  float ks, vs, log;   // scales of block lane % 4, log2 of the value's
  float most, least;   // of the four logarithms
  __device__ f16v8 key(int half, int step) const {
    return *reinterpret_cast<const f16v8 *>(k + 32 * half * (int)L::kRow + 32 * step);
  }
  __device__ f16v8 value(int d, int block) const {
    return *reinterpret_cast<const f16v8 *>(v + 32 * d * (int)L::vRow + 16 * block);
  }
};

// Products of H halves of the tile's keys, from half `from` on, with the queries;
// between(i) goes between them.
template <int H, typename L, int KS, typename Between>
__device__ __forceinline__ void products(f32x16 *x, const Tile<L> &tile, int from, const f16v8 (&q)[KS], Between between) {
  constexpr int N = H * KS, kAhead = N < 6 ? N : 6;   // reads ahead of their products
  f16v8 w[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) w[i] = tile.key(from + i / KS, i % KS);
  in_order();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i % KS == 0)
#pragma unroll
      for (int r = 0; r < 16; ++r) x[i / KS][r] = 0.0f;
    x[i / KS] = mfma(w[i % kAhead], q[i % KS], x[i / KS]);
    if (i + kAhead < N) w[i % kAhead] = tile.key(from + (i + kAhead) / KS, (i + kAhead) % KS);
    between(i);
    in_order();
  }
}

// A tile whose scales and scores are ordinary ones: weights go into the product with
// their page's value scale, as 2^(t - m + log2(scale) - g), where g is held such that
// the largest are 2^10 to 2^(15.9) (f16 has 11 bits from 2^-14 on), and come out of
// its rounded weights for the sum.  m is raised only where it lags by more than kLag:
// that is one pass over the outputs.  False, and nothing done, for tiles that are not
// ordinary: values' scales more than a factor of 2^kSpread from one another or near the
// ends of the range, keys' not finite or close to 0 (a hidden score is -infinity times
// them), scores so far from 0 that a fused difference
// would have a rounding of the score left over, values so far from the unit that moving
// it could lose them.  (NaN fails.)
constexpr float kLag = 3.0f, kSpread = 2.75f, kRoom = 12.875f;
template <typename L, int DT>
__device__ __forceinline__ bool fast_tile(State &st, f32x16 (&o)[DT], const f32x16 (&x)[2], const Tile<L> &tile, float c) {
  float mx = -INFINITY;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    float most = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j) most = fmaxf(most, x[b >> 1][8 * (b & 1) + j]);
    mx = fmaxf(mx, most * (lane_of(tile.ks, b) * c));
  }
  mx = max32(mx);
  const bool move = !(tile.most - st.g <= kRoom + 0.025f && tile.least - st.g >= 10.0f);
  const float g = move ? tile.most - kRoom : st.g;
  const auto near = [](float y) { return (fabsf(y) < 32768.0f) | (y == -INFINITY); };
  const bool fine = (tile.ks < INFINITY) & (tile.ks >= 0x1p-60f) & (c >= 0x1p-60f) & (fabsf(tile.log) < 100.0f) & (tile.most - tile.least <= kSpread) & near(mx) & near(st.m) &
                    (!move | (st.top == -INFINITY) | (fabsf(g - st.g) <= 60.0f));
  if (!__all(fine)) return false;
  if (__any(move | (mx > st.m + kLag))) {
    const float m = fmaxf(st.m, mx), up = m == -INFINITY ? 0.0f : m - st.m, k = exp2_fast(-up);
    const float ko = st.top == -INFINITY ? 0.0f : k * exp2_fast(st.g - g);
    st.l *= k;
    st.top -= up;
    st.m = m;
    st.g = g;
    results_there();
#pragma unroll
    for (int d = 0; d < DT; ++d) scale_in_place(o[d], ko);
  }
  const float m = st.m == -INFINITY ? 0.0f : st.m, off = -st.g - m;
  st.top = fmaxf(st.top, mx - m + tile.least);
  const float unit = exp2_fast(st.g), rcp = __builtin_amdgcn_rcpf(tile.vs);
  // the weights of the next 16 tokens between the products of these
  u32x4 p[2];
  float part = 0.0f, sum = 0.0f;
  const auto pair = [&](int b, int j) {
    const float sc = lane_of(tile.ks, b) * c, by = lane_of(tile.log, b) + off;
    const float y0 = __builtin_fmaf(x[b >> 1][8 * (b & 1) + 2 * j], sc, by);
    const float y1 = __builtin_fmaf(x[b >> 1][8 * (b & 1) + 2 * j + 1], sc, by);
    p[b & 1][j] = Elem<ENTRO_F16>::pack2(exp2_fast(y0), exp2_fast(y1));
    part = Elem<ENTRO_F16>::add2(p[b & 1][j], j ? part : 0.0f);
    if (j == 3) sum = __builtin_fmaf(part, lane_of(rcp, b), sum);
  };
  f16v8 w[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) w[d] = tile.value(d, 0);
  in_order();
#pragma unroll
  for (int j = 0; j < 4; ++j) pair(0, j);
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      o[d] = mfma(w[d], __builtin_bit_cast(f16v8, p[b & 1]), o[d]);
      if (b < 3) {
        w[d] = tile.value(d, b + 1);
#pragma unroll
        for (int j = 4 * d / DT; j < 4 * (d + 1) / DT; ++j) pair(b + 1, j);
      }
      in_order();
    }
  st.l = __builtin_fmaf(sum, unit, st.l);
  return true;
}

// Any tile: 16 tokens at a time, the weights relative to their own largest and their
// product's part brought to the outputs' unit in 32 bits, the unit to the values'.  A
// block that a row does not see has no influence on it, whatever its scales are.
template <typename L, int DT, int KS>
__device__ __forceinline__ void slow_tile(State &st, f32x16 (&o)[DT], const f16v8 (&q)[KS], const Tile<L> &tile, float c,
                                          int32_t seen) {
#pragma unroll 1
  for (int hh = 0; hh < 2; ++hh) {
    f32x16 x;
    products<1>(&x, tile, hh, q, [](int) {});
#pragma unroll
    for (int cc = 0; cc < 2; ++cc) {
      const int blk = 2 * hh + cc;
      const float sc = lane_of(tile.ks, blk) * c;
      const Scale vs(lane_of(tile.vs, blk));
      float mx = -kFloatMax, y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = 16 * blk + j < seen ? rounded(x[8 * cc + j], sc) : -INFINITY;
        mx = fmaxf(mx, y[j]);
      }
      const bool any = max32(16 * blk < seen ? 1.0f : 0.0f) != 0.0f;   // (the row's other lane may see one)
      mx = max32(mx);
      float sum = 0.0f;
      u32x4 pw;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p0 = exp2_fast(y[2 * j] - mx), p1 = exp2_fast(y[2 * j + 1] - mx);
        sum += p0 + p1;
        pw[j] = Elem<ENTRO_F16>::pack2(p0 * 32768.0f, p1 * 32768.0f);
      }
      // the row's state with the block
      const float m = fmaxf(st.m, mx), up = m - st.m, down = mx - m;
      const float top = fmaxf(st.top - up, down + vs.log);
      float g = st.g;
      if (top > -kFloatMax && !(fabsf(top - kUnit - g) <= 30.0f)) g = top - kUnit;
      const float keep = any ? exp2_fast(st.g - g - up) : 1.0f;
      const float f = any && vs.part != 0.0f ? vs.part * exp2_fast(down + vs.whole - g - 15.0f) : 0.0f;
      if (any) {
        st.l = st.l * exp2_fast(-up) + sum * exp2_fast(down);
        st.m = m;
        st.g = g;
        st.top = top;
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        in_order();   // one part of the outputs after another: registers
        f32x16 z;
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = 0.0f;
        z = mfma(tile.value(d, blk), __builtin_bit_cast(f16v8, pw), z);
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = any ? z[i] * f : 0.0f;
        results_there();
        add_in_place(o[d], keep, z);
      }
      in_order();
    }
  }
}

// ---------------------------------------------------------------------------
// One workgroup takes pieces of blocks for one key/value head.  A block's rows are
// its tokens' queries of all heads that share the key/value head, 32 of them for each
// wavefront; the tiles of 64 tokens go by way of LDS, where their codes lie as f16
// (exactly), two buffers in turn.
//
// Scores are K Q^T and outputs V^T P^T on 32 x 32 x 16 matrix instructions with the
// rows as columns: a lane and its partner 32 further own one row's softmax.  The
// first product's rows are tokens in the order in which its results, in the lanes
// where they are, are the second product's operand: row 16 c + 8 i + 4 h + j is token
// 16 c + 8 h + 4 i + j.  A lane then has eight tokens of each 16, which are of one
// page: its scales are the same in the whole wavefront.
// ---------------------------------------------------------------------------
template <entro_dtype T, int D, int W>
__global__ __launch_bounds__(64 * W, 2) void attn_chunk_kernel(ChunkArg a) {
  typedef Lds<D, W> L;
  constexpr int KS = D / 16;                       // products over the dimensions
  constexpr int DT = D / 32;                       // 32-dimension parts of the output
  constexpr int PT = 8 / W;                        // 16-byte pieces of a tile's keys, and of its values, for a thread
  constexpr uint32_t kRows = 32 * W;
  char *lds = reinterpret_cast<char *>(dyn_lds);
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = rfl(tid >> 6);
  const uint32_t page = 1u << a.page_log2;
  Place at(a, lane);
  if (blockIdx.x == 0u && blockIdx.y == 0u && wave == 0u) {
    Spans spans(a.cu, a.total_q, a.n_seq, lane);
    for (uint32_t b0 = 0; b0 < a.n_seq; b0 += 64u) {
      bool ok;
      chunk_seq(a, spans, b0, &ok);
      if (b0 + lane < a.n_seq && !ok) atomicOr(a.status + b0 + lane, ENTRO_F_LENGTH);
    }
  }
  const Shares sh = shares_of(a, rfl64(at.count_all()));
  if (sh.tiles == 0u) return;
  for (uint32_t head_part = blockIdx.x; head_part < a.n_kv * a.parts; head_part += gridDim.x)
    for (uint32_t w = blockIdx.y; w < sh.n; w += gridDim.y) {
      const uint32_t kvh = head_part / a.parts, h0 = head_part % a.parts * a.heads;
      const uint32_t heads = min(a.heads, a.group - h0), head0 = kvh * a.group + h0;
      const uint32_t page_bytes = a.n_kv * page * D;   // from one page's codes to the next's, below 2^30
      const int8_t *const kb = a.k_codes + (uint64_t)kvh * page * D, *const vb = a.v_codes + (uint64_t)kvh * page * D;
      uint64_t now = sh.begin(w);
      const uint64_t end = sh.begin(w + 1u);
      at.find(now);
      for (; now < end; at.next()) {
        const Seq s = at.here();
        const Blocks blocks(a.block_log2, s);
        const uint32_t all_tiles = blocks.tiles(at.block);
        const uint32_t t0 = (uint32_t)(now - at.before), t1 = (uint32_t)min((uint64_t)all_tiles, end - at.before);
        now = at.before + t1;
        const int32_t *row = a.table + (uint64_t)at.seq * a.table_stride;
        const uint32_t token0 = at.block << a.block_log2;
        const uint32_t rows = min(1u << a.block_log2, s.count - token0) * heads;
        const bool active = wave * 32u < rows;
        // a lane's row; past the last, the last
        struct Row {
          uint32_t token, head;
        };
        const auto row_of = [&](uint32_t ln) {
          const uint32_t r = min(wave * 32u + (ln & 31u), rows - 1u);
          return (Row){token0 + r / heads, head0 + r % heads};
        };
        // tokens that the lane's row sees, less the first one of the lane's eight
        int32_t limit;
        int32_t least, most;   // tokens that the wavefront's rows see
        f16v8 qf[KS];          // the query as f16 times 2^-e, piece 2 i + lane / 32 of its dimensions as the keys lie in LDS
        float c = 0.0f;        // score = c * key scale * product
        {
          const uint32_t ln = fresh(lane), half = ln >> 5;
          const Row mine = row_of(ln);
          limit = (int32_t)max((int64_t)0, blocks.ahead + mine.token + 1);
          least = __builtin_amdgcn_readlane(limit, 0);
          most = __builtin_amdgcn_readlane(limit, 31);
          limit -= 8 * (int32_t)half;
          u32x4 raw[KS];
          const char *q = a.q + ((int64_t)s.begin + mine.token) * a.q_t + (int64_t)mine.head * a.q_h;
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            const uint32_t p = 2u * i + half;
            raw[i] = *reinterpret_cast<const u32x4 *>(q + (p < D / 16u ? 32u * p : 32u * (p - D / 16u) + 16u));
          }
          int e2 = 0;
          if (T == ENTRO_BF16) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < KS; ++i)
              for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(Elem<T>::lo(raw[i][e])), fabsf(Elem<T>::hi(raw[i][e]))));
            top = max32(top);
            e2 = top == 0.0f ? 0 : (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127;   // bf16 denormals: -127
          }
          c = ldexpf(a.scale, e2);
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            u32x4 x;
            for (int e = 0; e < 4; ++e) {
              const uint32_t y = T == ENTRO_F16 ? raw[i][e]
                                                : Elem<ENTRO_F16>::pack2(ldexpf(Elem<T>::lo(raw[i][e]), -e2),
                                                                         ldexpf(Elem<T>::hi(raw[i][e]), -e2));
              x[e] = y ^ a.q_xor;
            }
            qf[i] = __builtin_bit_cast(f16v8, x);
          }
        }

        f32x16 o[DT];
#pragma unroll
        for (int d = 0; d < DT; ++d)
          for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
        State st = {-INFINITY, 0.0f, 0.0f, -INFINITY};

        // A tile's way: page numbers three tiles ahead, codes and scales two, f16 in LDS
        // one.  (Past the piece's last tile the last is fetched again: no branches.)  A
        // block past the sequence's end, or of a page that does not exist, takes page 0.
        bool bad = false;
        const uint32_t last = t1 - 1u;
        const auto fetch_page = [&](uint32_t tile) {
          return (uint32_t)row[min(min(tile, last) * kTile + (fresh(lane) & 3u) * 16u, max(s.len, 1u) - 1u) >> a.page_log2];
        };
        const auto page_ok = [&](uint32_t p, uint32_t tile) {
          const bool there = min(tile, last) * kTile + (fresh(lane) & 3u) * 16u < s.len;
          bad |= there && p >= a.n_pages;
          return there && p < a.n_pages ? p : 0u;
        };
        // A thread's pieces: 16 dimensions of a key, eight threads a key (all of a
        // wavefront's eight keys on one page); 16 tokens of a dimension, four threads a
        // dimension where a tile lies in one page, or all of a wavefront's 64 dimensions of
        // one block, which lie side by side where pages are small.  In LDS a key's piece lies
        // in two halves, D / 2 apart; a dimension's in two halves, 32 tokens apart.
        const bool wide = page >= kTile;
        const uint32_t k_block = wave / 2u, v_block = wide ? 0u : wave & 3u;   // of a wavefront's page
        uint32_t k_from, k_to, v_from, v_to;
        bool k_mine, v_mine[PT];
        {
          const uint32_t ln = fresh(lane), key = wave * 8u + ln / 8u, piece = ln % 8u;
          k_mine = piece < D / 16u;
          k_from = (key & (page - 1u)) * D + min(piece, D / 16u - 1u) * 16u;
          k_to = key * L::kRow + piece * 16u;
          const uint32_t dim = wide ? wave * 16u + ln / 4u : (wave / 4u) * 64u + ln, block = wide ? ln & 3u : wave & 3u;
#pragma unroll
          for (int i = 0; i < PT; ++i) v_mine[i] = dim + 64u * i < D;
          v_from = (dim << a.page_log2) + (block * 16u & (page - 1u));
          v_to = L::kBytes + dim * L::vRow + block * 16u;
        }
        u32x4 kq[PT], vq[PT];
        const auto fetch_keys = [&](uint32_t tile, uint32_t pages, int i) {
          const uint32_t p = lane_of(pages, k_block + 2u * i), in = (min(tile, last) * kTile + 32u * i) & (page - 1u);
          kq[i] = *reinterpret_cast<const u32x4 *>(kb + ((uint64_t)p * page_bytes + in * D) + k_from);
        };
        const auto fetch_values = [&](uint32_t tile, uint32_t pages, int i) {
          const uint32_t p = lane_of(pages, v_block), in = (min(tile, last) * kTile) & (page - 1u);
          const uint32_t further = v_mine[i] ? v_from + (64u * i << a.page_log2) : 0u;
          vq[i] = *reinterpret_cast<const u32x4 *>(vb + ((uint64_t)p * page_bytes + in) + further);
        };
        const auto put = [&](uint32_t tile, int i, int which) {
          char *to = lds + (tile & 1u) * (L::kBytes + L::vBytes);
          if (which < 2 ? D < 128 && !k_mine : D < 64 * W / 4 * PT && !v_mine[i]) return;
          char *kp = to + k_to + 32 * i * (int)L::kRow, *vp = to + v_to + 64 * i * (int)L::vRow;
          if (which == 0) *reinterpret_cast<f16v8 *>(kp) = half8(kq[i].x, kq[i].y);
          if (which == 1) *reinterpret_cast<f16v8 *>(kp + D) = half8(kq[i].z, kq[i].w);
          if (which == 2) *reinterpret_cast<f16v8 *>(vp) = half8(vq[i].x, vq[i].y);
          if (which == 3) *reinterpret_cast<f16v8 *>(vp + kTile) = half8(vq[i].z, vq[i].w);
        };
        uint32_t pages = page_ok(fetch_page(t0), t0);
#pragma unroll
        for (int i = 0; i < PT; ++i) {
          fetch_keys(t0, pages, i);
          fetch_values(t0, pages, i);
        }
        float ks0 = a.k_scales[(uint64_t)pages * a.n_kv + kvh], vs0 = a.v_scales[(uint64_t)pages * a.n_kv + kvh];
        pages = page_ok(fetch_page(t0 + 1u), t0 + 1u);
        uint32_t pages_raw = fetch_page(t0 + 2u);
        float ks1 = a.k_scales[(uint64_t)pages * a.n_kv + kvh], vs1 = a.v_scales[(uint64_t)pages * a.n_kv + kvh];
#pragma unroll
        for (int i = 0; i < 4 * PT; ++i) put(t0, i / 4, i % 4);
#pragma unroll
        for (int i = 0; i < PT; ++i) {
          fetch_keys(t0 + 1u, pages, i);
          fetch_values(t0 + 1u, pages, i);
        }
        for (uint32_t t = t0; t < t1; ++t) {
          __syncthreads();   // tile t is there; the other buffer has been read
          // the next tiles' way, one step after another
          constexpr int kSteps = 6 * PT + 2;
          float ks2, vs2;
          const auto ahead = [&](int i) {
            if (i < 4 * PT) {
              put(t + 1u, i / 4, i % 4);
            } else if (i == 4 * PT) {
              pages = page_ok(pages_raw, t + 2u);
              pages_raw = fetch_page(t + 3u);
            } else if (i <= 5 * PT) {
              fetch_keys(t + 2u, pages, i - 4 * PT - 1);
            } else if (i <= 6 * PT) {
              fetch_values(t + 2u, pages, i - 5 * PT - 1);
            } else {
              const uint64_t mine = (uint64_t)pages * a.n_kv + kvh;
              ks2 = a.k_scales[mine];
              vs2 = a.v_scales[mine];
            }
          };
          if (!active || (int64_t)t * kTile >= most) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) ahead(i);
          } else {
            const uint32_t ln = fresh(lane), col = ln & 31u, half = ln >> 5;
            const char *kt = lds + (t & 1u) * (L::kBytes + L::vBytes), *vt = kt + L::kBytes;
            const uint32_t kr = (col & 0x13u) | ((col & 4u) << 1) | ((col & 8u) >> 1);   // the token of row `col`
            // (blocks past the end take the first one's scales)
            const bool past = t * kTile + (ln & 3u) * 16u >= s.len;
            const float k_first = quad<0x00>(ks0), v_first = quad<0x00>(vs0);
            const float v_scale = past ? v_first : vs0, log = __log2f(v_scale);
            const Tile<L> tile{kt + kr * L::kRow + half * 16u, vt + col * L::vRow + half * 64u, (int32_t)(t * kTile),
                               past ? k_first : ks0, v_scale, log, quad_max(log), -quad_max(-log)};
            f32x16 x[2];
            products<2>(x, tile, 0, qf, [&](int i) {   // kSteps steps among 2 KS products
#pragma unroll
              for (int j = kSteps * i / (2 * KS); j < kSteps * (i + 1) / (2 * KS); ++j) ahead(j);
            });
            const int32_t seen = limit - tile.base;
            if (tile.base + (int32_t)kTile > least) {
              results_there();
#pragma unroll
              for (int b = 0; b < 4; ++b) hide_in_place(x[b >> 1], b, seen);
            }
            if (!fast_tile(st, o, x, tile, c)) slow_tile(st, o, qf, tile, c, seen);
          }
          ks0 = ks1;
          vs0 = vs1;
          ks1 = ks2;
          vs1 = vs2;
        }
        if (bad) atomicOr(a.status + at.seq, ENTRO_F_PAGE);
        __syncthreads();   // the tiles' places are written again
        const uint32_t ln = fresh(lane), half = ln >> 5, r = wave * 32u + (ln & 31u);
        if (r >= rows) continue;
        const Row mine = row_of(ln);
        const float l = add32(st.l);
        if (t1 - t0 == all_tiles) {
          const float whole = floorf(fminf(fmaxf(st.g, -400.0f), 400.0f));
          const float k = l == 0.0f ? 0.0f : exp2_fast(st.g - whole) / l;
          char *to = a.out + ((int64_t)s.begin + mine.token) * a.o_t + (int64_t)mine.head * a.o_h;
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] = ldexpf(o[d][4 * i + j] * k, (int)whole);
              *reinterpret_cast<u32x2 *>(to + (32 * d + 8 * i + 4 * half) * 2) =
                  (u32x2){Elem<T>::pack2(v[0], v[1]), Elem<T>::pack2(v[2], v[3])};
            }
        } else {
          const uint64_t place = (((uint64_t)head_part * a.shares + w) * 2u + (t0 == 0u)) * kRows + r;
          if (half == 0u) a.part_s[place] = (f32x4){st.m, l, st.top == -INFINITY ? -INFINITY : st.g, 0.0f};
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<f32x4 *>(a.part_o + place * D + 32 * d + 8 * i + 4 * half) =
                  (f32x4){o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
        }
      }
    }
}

// Joins the pieces of a split block: one workgroup for the first share that begins
// inside the block and kJoinRows of its rows.  A thread has four dimensions of a row
// and takes the pieces in the tokens' order.
constexpr uint32_t kJoinRows = 8;
template <entro_dtype T, int D, int W>
__global__ __launch_bounds__(kJoinRows * D / 4) void attn_chunk_join_kernel(ChunkArg a) {
  constexpr uint32_t kRows = 32 * W, kGroups = kRows / kJoinRows;
  const uint32_t tid = threadIdx.x, lane = tid & 63u;
  Place at(a, lane);
  const Shares sh = shares_of(a, rfl64(at.count_all()));
  for (uint32_t w = 1u + blockIdx.y; w < sh.n; w += gridDim.y) {
    const uint64_t cut = sh.begin(w);
    at.find(cut);
    if (cut == at.before || sh.begin(w - 1u) > at.before) continue;
    const Seq s = at.here();
    const Blocks blocks(a.block_log2, s);
    const uint64_t end = at.before + blocks.tiles(at.block);
    const uint32_t token0 = at.block << a.block_log2, tokens = min(1u << a.block_log2, s.count - token0);
    for (uint64_t y = blockIdx.x; y < (uint64_t)a.n_kv * a.parts * kGroups; y += gridDim.x) {
      const uint32_t head_part = (uint32_t)(y / kGroups), r = (uint32_t)(y % kGroups) * kJoinRows + tid / (D / 4u);
      const uint32_t kvh = head_part / a.parts, h0 = head_part % a.parts * a.heads;
      const uint32_t heads = min(a.heads, a.group - h0), head0 = kvh * a.group + h0;
      if (r >= tokens * heads) continue;
      const uint32_t d = tid % (D / 4u) * 4u;
      float m = -INFINITY, l = 0.0f, g = -INFINITY;   // of the pieces so far: as in State
      f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
      for (uint32_t p = w - 1u; p < sh.n && (p < w || sh.begin(p) < end); ++p) {
        const uint64_t place = (((uint64_t)head_part * a.shares + p) * 2u + (p < w)) * kRows + r;
        const f32x4 q = a.part_s[place];
        const f32x4 x = *reinterpret_cast<const f32x4 *>(a.part_o + place * D + d);
        if (q.x == -INFINITY) continue;   // saw no token
        const float up = fmaxf(m, q.x), mine = g + (m - up), its = q.z + (q.x - up);
        l = (m == -INFINITY ? 0.0f : l * exp2_fast(m - up)) + q.y * exp2_fast(q.x - up);
        const float unit = fmaxf(g == -INFINITY ? -INFINITY : mine, its);
        if (unit != -INFINITY) {   // (NaN passes)
          const float k0 = g == -INFINITY ? 0.0f : exp2_fast(mine - unit), k1 = q.z == -INFINITY ? 0.0f : exp2_fast(its - unit);
          o = o * k0 + x * k1;
        }
        g = unit;
        m = up;
      }
      const float whole = floorf(fminf(fmaxf(g, -400.0f), 400.0f));
      const float k = l == 0.0f || g == -INFINITY ? l * 0.0f : exp2_fast(g - whole) / l;
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = ldexpf(o[j] * k, (int)whole);
      *reinterpret_cast<u32x2 *>(a.out + ((int64_t)s.begin + token0 + r / heads) * a.o_t + (int64_t)(head0 + r % heads) * a.o_h + d * 2u) =
          (u32x2){Elem<T>::pack2(v[0], v[1]), Elem<T>::pack2(v[2], v[3])};
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// How a call is laid out.
struct Plan {
  uint32_t waves, heads, parts, block_log2, shares;
  uint64_t rows() const { return 32u * waves; }
};
static Plan plan_of(uint32_t n_seq, uint32_t total_q, uint32_t n_heads, uint32_t n_kv) {
  Plan p{};
  const uint32_t group = n_heads / n_kv;
  p.waves = (uint64_t)total_q * group > 128ull * n_seq ? 8u : 4u;
  p.heads = std::min<uint32_t>(group, (uint32_t)p.rows());
  p.parts = (group + p.heads - 1u) / p.heads;
  while ((2u << p.block_log2) * p.heads <= p.rows()) ++p.block_log2;
  p.shares = std::max(1u, (p.waves == 8u ? 256u : 512u) / (n_kv * p.parts));
  return p;
}

template <entro_dtype T, int D, int W>
static entro_status launch_chunk(const ChunkArg &a, hipStream_t s) {
  const uint32_t lds = Lds<D, W>::bytes, heads = a.n_kv * a.parts;
  (void)hipGetLastError();
  hipLaunchKernelGGL((attn_chunk_kernel<T, D, W>), grid2(heads, a.shares), dim3(64 * W), lds, s, a);
  if (hipGetLastError() != hipSuccess) return ENTRO_E_HIP;
  if (a.shares > 1u) {
    hipLaunchKernelGGL((attn_chunk_join_kernel<T, D, W>), grid2((uint64_t)heads * (32u * W / kJoinRows), a.shares - 1u),
                       dim3(kJoinRows * D / 4), 0, s, a);
    if (hipGetLastError() != hipSuccess) return ENTRO_E_HIP;
  }
  return ENTRO_OK;
}

}  // namespace entro

using namespace entro;

extern "C" uint64_t entro_attn_chunk_work_bytes(uint32_t n_seq, uint32_t total_q, uint32_t n_heads, uint32_t n_kv_heads,
                                                uint32_t head_dim) {
  if (n_seq == 0 || total_q == 0 || total_q > 0x7FFFFFFFu || check_heads(n_heads, n_kv_heads, head_dim, ENTRO_BF16) != ENTRO_OK)
    return 0;
  const Plan p = plan_of(n_seq, total_q, n_heads, n_kv_heads);
  return (uint64_t)n_kv_heads * p.parts * p.shares * 2u * p.rows() * (head_dim + 4u) * 4u;
}

extern "C" entro_status entro_attn_chunk(const entro_kv_cache *c, const entro_kv_table *t, const entro_attn_chunk_args *a,
                                         uint32_t *d_status, hipStream_t stream) {
  if (!a) return ENTRO_E_INVAL;
  entro_status st = check_cache(c, t);
  if (st != ENTRO_OK) return st;
  st = check_heads(a->n_heads, c->n_kv_heads, c->head_dim, a->dtype);
  if (st != ENTRO_OK) return st;
  if (!std::isfinite(a->scale)) return ENTRO_E_INVAL;
  if (t->n_seq == 0) return ENTRO_OK;
  if (!a->d_cu_q || !a->d_lens || !d_status || a->total_q > 0x7FFFFFFFu) return ENTRO_E_INVAL;
  for (const entro_rows *r : {&a->q, &a->out}) {
    st = check_rows(*r, a->total_q);
    if (st != ENTRO_OK) return st;
  }
  const uint64_t need = entro_attn_chunk_work_bytes(t->n_seq, a->total_q, a->n_heads, c->n_kv_heads, c->head_dim);
  if (need && (!a->d_work || (reinterpret_cast<uintptr_t>(a->d_work) & 15u) || a->work_bytes < need)) return ENTRO_E_INVAL;
  const Plan p = plan_of(t->n_seq, a->total_q, a->n_heads, c->n_kv_heads);
  ChunkArg k{};
  k.k_codes = c->d_k_codes;
  k.v_codes = c->d_v_codes;
  k.k_scales = c->d_k_scales;
  k.v_scales = c->d_v_scales;
  k.table = t->d_table;
  k.table_stride = t->table_stride;
  k.table_pages = t->table_pages;
  k.n_seq = t->n_seq;
  k.n_pages = c->n_pages;
  k.n_kv = c->n_kv_heads;
  k.page_log2 = c->page_tokens == 16u ? 4u : c->page_tokens == 32u ? 5u : c->page_tokens == 64u ? 6u : 7u;
  k.q = static_cast<const char *>(a->q.d);
  k.out = static_cast<char *>(a->out.d);
  k.q_t = 2 * a->q.stride_t;
  k.q_h = 2 * a->q.stride_h;
  k.o_t = 2 * a->out.stride_t;
  k.o_h = 2 * a->out.stride_h;
  k.cu = a->d_cu_q;
  k.lens = a->d_lens;
  k.total_q = a->total_q;
  k.n_heads = a->n_heads;
  k.group = a->n_heads / c->n_kv_heads;
  k.heads = p.heads;
  k.parts = p.parts;
  k.block_log2 = p.block_log2;
  k.shares = p.shares;
  k.scale = std::fabs(a->scale) * kLog2e;
  k.q_xor = std::signbit(a->scale) ? 0x80008000u : 0u;
  k.part_s = static_cast<f32x4 *>(a->d_work);
  k.part_o = reinterpret_cast<float *>(k.part_s + (uint64_t)k.n_kv * k.parts * k.shares * 2u * p.rows());
  k.status = d_status;
  const auto waves = [&](auto type, auto dim) {
    return p.waves == 8u ? launch_chunk<decltype(type)::value, decltype(dim)::value, 8>(k, stream)
                         : launch_chunk<decltype(type)::value, decltype(dim)::value, 4>(k, stream);
  };
  const auto dims = [&](auto type) {
    return c->head_dim == 64u   ? waves(type, std::integral_constant<int, 64>{})
           : c->head_dim == 96u ? waves(type, std::integral_constant<int, 96>{})
                                : waves(type, std::integral_constant<int, 128>{});
  };
  return a->dtype == ENTRO_BF16 ? dims(std::integral_constant<entro_dtype, ENTRO_BF16>{})
                                : dims(std::integral_constant<entro_dtype, ENTRO_F16>{});
}

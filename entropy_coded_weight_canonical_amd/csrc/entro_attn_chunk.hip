// HIP kernels (gfx950) and entry points of the attention of chunks over the 8-bit
// cache: entro_attn_chunk.  Layout and definition are in entro_attn.h.
//
// One pass over a block's tiles with a running maximum and sum; the work of all blocks
// is cut into equal shares, one workgroup each, and a second kernel joins the pieces of
// blocks that were cut.  Two first kernels: attn_chunk_kernel for many rows, by way of
// LDS, and attn_few_kernel for few.
//
// Measured on an MI355X (copy 4.8 TB/s, 16384^3 f16 product 1300 TFLOP/s): 2048 tokens
// behind 30720, 32 / 8 heads of 128, bf16: 1.09 to 1.19 ms, 900 to 975 TFLOP/s as the card's
// clock goes; 61 tokens behind 40003, 64 / 8 heads of 128, f16: 115 us; 24 sequences of up to
// 7 tokens behind up to 12000, 32 / 8 heads of 128: 56 us; 5 tokens behind 85, 32 heads of 64:
// 9.2 us.
#include <algorithm>
#include <type_traits>

#include "entro_attn_device.h"
#include "entro_internal.h"

namespace entro {

constexpr uint32_t kTile = 64;          // tokens of a step
constexpr uint32_t kShareTiles = 6;     // least work of a workgroup's share, in tiles: less is a join that costs more
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
  uint32_t group;               // query heads per key/value head
  uint32_t heads, parts;        // query heads of a workgroup, workgroups per key/value head for all of them
  uint32_t block_log2;          // tokens of a workgroup
  uint32_t rows;                // rows (queries of a head) of a workgroup, at most
  uint32_t join_groups;         // workgroups that join a block's pieces
  uint32_t shares;              // that the tiles of a key/value head are split into at most
  float scale;                  // magnitude, times log2(e)
  uint32_t q_xor;               // on a pair of q: the scale's sign
  float *part_o;                // [n_kv parts][shares][2][rows][D]
  f32x4 *part_s;                // [n_kv parts][shares][2][rows]: a row's State
  u32x4 *cuts;                  // [shares]: see Cut
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
// has the tiles that its last token sees, and one at least; its work is counted in
// tiles, with kBegin for its queries' way in and its results' way out.  L is a whole
// number so that the work of a sequence's first blocks can be written down.
constexpr uint32_t kBegin = 2;
struct Blocks {
  uint32_t L, n, count;
  int64_t ahead;   // tokens in front of the first query; below 0 where the first ones see none
  __device__ Blocks(uint32_t log2, const Seq &s)
      : L(log2), n((uint32_t)(((uint64_t)s.count + (1ull << log2) - 1u) >> log2)), count(s.count),
        ahead((int64_t)s.len - (int64_t)s.count) {}
  // the work of the first x blocks, all of them full
  __device__ uint64_t full(uint32_t x) const { return (uint64_t)x * kBegin + full_tiles(x); }
  // their tiles: the sum over y = 1 .. x of max(1, ceil((ahead + 2^L y) / 64))
  __device__ uint64_t full_tiles(uint32_t blocks) const {
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
  __device__ uint32_t work(uint32_t b) const { return kBegin + tiles(b); }
  __device__ uint64_t all() const { return n ? full(n - 1u) + work(n - 1u) : 0u; }
  // the block of piece t of the work
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

// A place in the work of all sequences' blocks, one after another.
struct Place {
  const ChunkArg &a;
  uint32_t lane;
  Spans spans;
  uint32_t b0;          // own: of sequence b0 + lane
  Seq own;
  uint64_t mine, run;   // its work, and with that of the lanes before
  bool loaded;          // whether the first 64 sequences are there
  uint32_t seq;         // n_seq: past the last
  uint32_t block;
  uint64_t before;      // work before the block
  __device__ Place(const ChunkArg &arg, uint32_t lane_)
      : a(arg), lane(lane_), spans(arg.cu, arg.total_q, arg.n_seq, lane_), loaded(false) {}
  __device__ void load(uint32_t at) {
    b0 = at;
    own = chunk_seq(a, spans, b0);
    mine = Blocks(a.block_log2, own).all();
    run = wave_scan64(mine);
  }
  __device__ uint64_t count_all() {
    load(0u);
    uint64_t sum = lane_of(run, 63u);
    loaded = a.n_seq <= 64u;
    for (uint32_t at = 64u; at < a.n_seq; at += 64u) {
      load(at);
      sum += lane_of(run, 63u);
    }
    return rfl64(sum);
  }
  __device__ void find(uint64_t place) {
    uint64_t sum = 0;
    for (uint32_t at = 0; at < a.n_seq; at += 64u) {
      if (!loaded) load(at);   // (a chain of reads: 1 us)
      loaded = false;
      const uint64_t past = __ballot(sum + run > place);
      if (past) {
        const uint32_t l = (uint32_t)__builtin_ctzll(past);
        seq = rfl(at + l);
        sum += lane_of(run - mine, l);
        const Blocks b(a.block_log2, here());
        block = rfl(b.of(place - sum));
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
    before += b.work(block);
    if (++block < b.n) return;
    block = 0u;
    while (++seq < a.n_seq) {
      if (seq - b0 == 64u) own = chunk_seq(a, spans, b0 += 64u);
      if (here().count) return;
    }
  }
};

// The work of a key/value head in equal shares (to one tile), one workgroup each and as
// many as the GPU holds at once: share w is begin(w) .. begin(w + 1) - 1.  A share's
// tiles of one block are a piece; a block in one piece is finished by its workgroup, the
// others' pieces are joined by the second kernel.  A share has at most two pieces of
// blocks that it does not finish: one that lacks the block's first tile, always the
// share's first (place 0), and one that has it, always its last (place 1).
struct Shares {
  uint64_t work, each;   // of a share; the first `more` have one more
  uint32_t n, more;
  __device__ uint64_t begin(uint32_t w) const { return w * each + min(w, more); }
  // the share of place t
  __device__ uint32_t of(uint64_t t) const {
    const uint64_t longer = more * (each + 1u);
    const bool first = t < longer;
    const uint64_t x = first ? t : t - longer, y = first ? each + 1u : each;
    const uint32_t q = (x | y) >> 32 ? (uint32_t)(x / y) : (uint32_t)x / (uint32_t)y;
    return first ? q : more + q;
  }
};
__device__ __forceinline__ Shares shares_of(const ChunkArg &a, uint64_t work) {
  Shares s;
  s.work = work;
  s.n = (uint32_t)min((uint64_t)a.shares, max((uint64_t)1, work / kShareTiles));
  s.each = work >> 32 ? work / s.n : (uint32_t)work / s.n;
  s.more = (uint32_t)(work - s.each * s.n);
  return s;
}
// The tile of a block before which a share's begin or end cuts it; 0: before all.
__device__ __forceinline__ uint32_t cut_at(uint64_t place, uint64_t before) {
  return place > before + kBegin ? (uint32_t)(place - before - kBegin) : 0u;
}

// What the first kernel tells the second of each share's begin: where it is the first
// cut in a block, the block's first row of q, its tokens, and its last share; else
// (and for shares that there are not) no tokens.
typedef u32x4 Cut;   // row, tokens, share, 0

// Marks the sequences whose lengths do not fit (one wavefront of the call).
__device__ __forceinline__ void flag_lengths(const ChunkArg &a, uint32_t lane) {
  Spans spans(a.cu, a.total_q, a.n_seq, lane);
  for (uint32_t b0 = 0; b0 < a.n_seq; b0 += 64u) {
    bool ok;
    chunk_seq(a, spans, b0, &ok);
    if (b0 + lane < a.n_seq && !ok) atomicOr(a.status + b0 + lane, ENTRO_F_LENGTH);
  }
}
// The shares that there are; the others' cuts are none.
__device__ __forceinline__ uint32_t no_cuts(const ChunkArg &a, const Shares &sh, uint32_t tid) {
  const uint32_t units = sh.work ? sh.n : 0u;
  if (blockIdx.x == 0u && tid == 0u && a.total_q)   // (without rows there is no workspace)
    for (uint32_t w = blockIdx.y; w < a.shares; w += gridDim.y)
      if (w >= units) a.cuts[w] = (Cut){0u, 0u, 0u, 0u};
  return units;
}
__device__ __forceinline__ Cut cut_of(const ChunkArg &a, const Place &at, const Shares &sh, uint32_t w) {
  const Seq s = at.here();
  const Blocks blocks(a.block_log2, s);
  const uint32_t token0 = at.block << a.block_log2;
  Cut cut = {s.begin + token0, min(1u << a.block_log2, s.count - token0), 0u, 0u};
  if (!cut_at(sh.begin(w), at.before) || cut_at(sh.begin(w - 1u), at.before)) cut.y = 0u;   // none, or not the block's first
  if (cut.y) cut.z = sh.of(at.before + blocks.work(at.block) - 1u);
  return cut;
}

// What is known of a row (one query of one head) beside its outputs, in powers of
// two: the largest score m, the weights' sum l relative to 2^m, and the exponent g
// of the outputs' unit, relative to 2^m too.  top: the largest exponent, less m, with
// which values have been added (their scale's times their weight's; in an ordinary
// tile, to 2^kSpread); the unit stays within kApart of kUnit below it, so that outputs
// keep their bits whatever the pages' scales are, one after another.
struct State {
  float m, l, g, top;
  // of the weights: -g - m (m: 0 where nothing was seen), and 2^g
  float off, unit;
  __device__ void settle() {
    off = -g - (m == -INFINITY ? 0.0f : m);
    unit = exp2_fast(g);
  }
};
constexpr float kUnit = 11.5f;   // the unit lies by about as much below top
constexpr float kApart = 30.0f;  // (2^31 values then sum up to 2^83)
constexpr float kSpread = 2.75f; // and a tile's scales that are ordinary by as much from one another at most

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
template <typename V>
__device__ __forceinline__ void scale_in_place(V &o, float k) {
#pragma unroll
  for (int r = 0; r < (int)(sizeof(V) / 4); ++r) {
    float x = o[r];
    asm volatile("v_mul_f32 %0, %1, %0" : "+v"(x) : "v"(k));
    o[r] = x;
  }
}
// o = o k + z
template <typename V>
__device__ __forceinline__ void add_in_place(V &o, float k, const V &z) {
#pragma unroll
  for (int r = 0; r < (int)(sizeof(V) / 4); ++r) {
    float x = o[r];
    asm volatile("v_fma_f32 %0, %0, %1, %2" : "+v"(x) : "v"(k), "v"(z[r]));
    o[r] = x;
  }
}
// -infinity where token I is not seen (I >= seen)
template <int I>
__device__ __forceinline__ float hidden(float y, int32_t seen) {
  asm volatile("v_cmp_lt_i32 vcc, %1, %2\n\ts_nop 1\n\tv_cndmask_b32 %0, %3, %0, vcc"
               : "+v"(y) : "n"(I), "v"(seen), "v"(-INFINITY) : "vcc");
  return y;
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

template <int D>
struct Lds {
  static constexpr uint32_t kRow = D * 2 + 16;          // bytes of a key's row and
  static constexpr uint32_t vRow = kTile * 2 + 16;      // of a dimension's: rows begin four banks further
  static constexpr uint32_t kBytes = kTile * kRow, vBytes = D * vRow, bytes = 2 * (kBytes + vBytes);
};

// The scales of 16 blocks of 16 tokens, four tiles, in each 16 lanes.  Blocks past the
// sequence's end have those of their tile's first.
struct Scales {
  float k, v, log, rcp;   // log2 and reciprocal of v
  float most, least;      // of a tile's logarithms
  uint64_t fine;          // lanes whose tile can be an ordinary one, see fast_tile
  __device__ Scales(float ks, float vs, bool past) {
    const float k0 = quad<0x00>(ks), v0 = quad<0x00>(vs);
    k = past ? k0 : ks;
    v = past ? v0 : vs;
    log = __log2f(v);
    rcp = __builtin_amdgcn_rcpf(v);
    most = quad_max(log);
    least = -quad_max(-log);
    fine = __ballot(k < INFINITY && k >= 0x1p-60f && fabsf(log) < 100.0f && most - least <= kSpread);
  }
};

// A tile as a lane sees it.
template <typename L>
struct Tile {
  const char *k, *v;   // the key that is its row of the first product, the dimension that is its row of the second
  uint32_t at;         // the lane that has its first block's scales
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

constexpr float kLag = 3.0f, kRoom = 12.875f, kNear = 2048.0f, kUnder = 8.0f;   // see fast_tile
// How an ordinary tile changes a row's state: mx is its largest score (-infinity: the row
// sees nothing of it, and nothing changes), most and least the logarithms of its pages'
// value scales.
struct Rise {
  float m, g, up;
  bool rise, near;
  __device__ Rise(const State &st, float mx, float most, float least) {
    const bool seen = mx > -INFINITY;
    const bool move = seen && !(most - st.g <= kRoom + 0.025f && least - st.g >= 10.0f);
    rise = move || mx > st.m + kLag;
    g = move ? most - kRoom : st.g;
    m = fmaxf(st.m, mx);
    up = m == st.m ? 0.0f : m - st.m;
    const float over = fmaxf(st.top - up, mx - m + most) - kUnit - g;
    near = !seen || (fabsf(m) < kNear && over <= kApart && over >= -kUnder);
  }
  // returns the factor of the outputs
  __device__ float apply(State &st) const {
    const float k = st.top == -INFINITY ? 0.0f : exp2_fast(st.g - g - up);   // (no value added yet: any unit)
    st.l *= exp2_fast(-up);
    st.top -= up;
    st.m = m;
    st.g = g;
    st.settle();
    return k;
  }
};
// The top with an ordinary tile's values, once the state has risen where it does.
__device__ __forceinline__ float with_tile(const State &st, float mx, float most) { return fmaxf(st.top, mx - st.m + most); }

// A tile whose scales and scores are ordinary ones: weights go into the product with
// their page's value scale, as 2^(t - m + log2(scale) - g), where g is held such that
// the largest are 2^10 to 2^(15.9) (f16 has 11 bits from 2^-14 on), and come out of
// its rounded weights for the sum.  m is raised only where it lags by more than kLag:
// that is one pass over the outputs.  False, and nothing done, for tiles that are not
// ordinary: values' scales more than a factor of 2^kSpread from one another or near the
// ends of the range, keys' not finite or close to 0 (a hidden score is -infinity times
// them), scores so far from 0 (2^11: m + g is off by 2^-14) that a fused difference
// would have a rounding of the score left over (in a tile that does not raise m, too: m
// may have been raised by one that was not ordinary), a unit for the tile's values that
// lies far from the top's: kApart below it, moved tile after tile, the outputs would run
// out of their range; kUnder above it, large values' weights would be f16's smallest.
// (NaN fails.)
template <typename L, int DT>
__device__ __forceinline__ bool fast_tile(State &st, f32x16 (&o)[DT], const f32x16 (&x)[2], const Tile<L> &tile,
                                          const Scales &scales, float c) {
  float sc[4], mx = -INFINITY;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    sc[b] = lane_of(scales.k, tile.at + b) * c;
    float most = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j) most = fmaxf(most, x[b >> 1][8 * (b & 1) + j]);
    mx = fmaxf(mx, most * sc[b]);
  }
  // (all of it before the outputs are touched: with ways out in between they are copied)
  mx = max32(mx);
  const float most = lane_of(scales.most, tile.at);
  const Rise up(st, mx, most, lane_of(scales.least, tile.at));
  if ((scales.fine >> tile.at & 15u) != 15u || __any(!up.near)) return false;
  if (__any(up.rise)) {
    const float less = up.apply(st);
    results_there();
#pragma unroll
    for (int d = 0; d < DT; ++d) scale_in_place(o[d], less);
  }
  st.top = with_tile(st, mx, most);
  // the weights of the next 16 tokens between the products of these
  u32x4 p[2];
  float part = 0.0f, sum = 0.0f;
  const auto pair = [&](int b, int j) {
    const float by = lane_of(scales.log, tile.at + b) + st.off;
    const float y0 = __builtin_fmaf(x[b >> 1][8 * (b & 1) + 2 * j], sc[b], by);
    const float y1 = __builtin_fmaf(x[b >> 1][8 * (b & 1) + 2 * j + 1], sc[b], by);
    p[b & 1][j] = Elem<ENTRO_F16>::pack2(exp2_fast(y0), exp2_fast(y1));
    part = Elem<ENTRO_F16>::add2(p[b & 1][j], j ? part : 0.0f);
    if (j == 3) sum = __builtin_fmaf(part, lane_of(scales.rcp, tile.at + b), sum);
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
  st.l = __builtin_fmaf(sum, st.unit, st.l);
  return true;
}

// A row's state with 16 tokens more, whose largest score is mx and whose page's value
// scale v: the factors of its sum (less), of theirs (part), of its outputs (keep) and of
// their product (f: with weights times 2^15).
struct Block {
  float m, g, top, less, part, keep, f;
  __device__ Block(const State &st, float mx, const Scale &v, bool any) {
    m = fmaxf(st.m, mx);
    const float up = m - st.m, down = mx - m;
    top = fmaxf(st.top - up, down + v.log);
    g = st.g;
    if (top > -kFloatMax && !(fabsf(top - kUnit - g) <= kApart)) g = top - kUnit;
    less = exp2_fast(-up);
    part = exp2_fast(down);
    keep = any ? exp2_fast(st.g - g - up) : 1.0f;
    f = any && v.part != 0.0f ? v.part * exp2_fast(down + v.whole - g - 15.0f) : 0.0f;
  }
  __device__ void apply(State &st) const {
    st.m = m;
    st.g = g;
    st.top = top;
  }
};

// Any tile: 16 tokens at a time, the weights relative to their own largest and their
// product's part brought to the outputs' unit in 32 bits, the unit to the values'.  A
// block that a row does not see has no influence on it, whatever its scales are.
template <typename L, int DT, int KS>
__device__ __forceinline__ void slow_tile(State &st, f32x16 (&o)[DT], const f16v8 (&q)[KS], const Tile<L> &tile, float c,
                                          int32_t seen, const Scales &scales) {
#pragma unroll 1
  for (int hh = 0; hh < 2; ++hh) {
    f32x16 x;
    products<1>(&x, tile, hh, q, [](int) {});
#pragma unroll
    for (int cc = 0; cc < 2; ++cc) {
      const int blk = 2 * hh + cc;
      const float sc = lane_of(scales.k, tile.at + blk) * c;
      const Scale vs(lane_of(scales.v, tile.at + blk));
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
      const Block b(st, mx, vs, any);
      if (any) {
        st.l = st.l * b.less + sum * b.part;
        b.apply(st);
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        in_order();   // one part of the outputs after another: registers
        f32x16 z;
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = 0.0f;
        z = mfma(tile.value(d, blk), __builtin_bit_cast(f16v8, pw), z);
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = any ? z[i] * b.f : 0.0f;
        results_there();
        add_in_place(o[d], b.keep, z);
      }
      in_order();
    }
  }
  st.settle();
}

// Four dimensions of a row, of pieces of its tokens.
struct Joined {
  float m, l, g;   // of the pieces so far: as in State; g: -infinity where no value was added
  f32x4 o;
  // two of them, or one and a piece; factors from differences only
  __device__ void add(float m1, float l1, float g1, f32x4 o1) {
    if (m1 == -INFINITY && l1 == 0.0f) return;   // saw no token (a sum that is no number stays)
    const float up = fmaxf(m, m1), d0 = m - up, d1 = m1 - up;
    l = (m == -INFINITY ? 0.0f : l * exp2_fast(d0)) + l1 * exp2_fast(d1);
    const float u0 = g == -INFINITY ? -INFINITY : g + d0, u1 = g1 + d1, unit = fmaxf(u0, u1);
    if (unit != -INFINITY)   // (NaN passes)
      o = o * (u0 == -INFINITY ? 0.0f : exp2_fast(u0 - unit)) + o1 * (u1 == -INFINITY ? 0.0f : exp2_fast(u1 - unit));
    g = unit;
    m = up;
  }
  template <entro_dtype T>
  __device__ u32x2 result() const {
    const float whole = floorf(fminf(fmaxf(g, -400.0f), 400.0f));
    const float k = l == 0.0f || g == -INFINITY ? l * 0.0f : exp2_fast(g - whole) / l;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ldexpf(o[i] * k, (int)whole);
    return (u32x2){Elem<T>::pack2(v[0], v[1]), Elem<T>::pack2(v[2], v[3])};
  }
};

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
//
// Codes are exact in f16, and so are a bf16 query's elements down to 2^-17 of its largest
// (they go in times the power of two that makes that 1 to 2; smaller ones are off by 2^-25
// of it).  What is rounded to fewer than 32 bits is the weights: f16, half a step 2^-12, as
// the matrix instruction takes them; fast_tile's sum is of the rounded ones.
//
// Bound: the waits of a wavefront for its own steps (scores, softmax, outputs, one after
// another), of which two wavefronts a SIMD hide a part: with many rows matrix instructions
// are at work in 41% of the cycles and vector instructions in 49%, side by side where the
// wavefronts' steps differ (900 to 975 of 1300 TFLOP/s); with 64 dimensions 14% and 40%.
// With one block per sequence the way of a tile through registers and LDS, 0.65 us a tile
// and workgroup.  256 rows in a workgroup (W = 8) halve that way's cost per row, 128
// (W = 4) waste less where sequences have fewer: 2048 tokens behind 30720, 1141 us with
// W = 8 and 1245 with W = 4; plan_of has others.
// ---------------------------------------------------------------------------
template <entro_dtype T, int D, int W>
__global__ __launch_bounds__(64 * W, 2) void attn_chunk_kernel(ChunkArg a) {
  typedef Lds<D> L;
  constexpr int KS = D / 16;                       // products over the dimensions
  constexpr int DT = D / 32;                       // 32-dimension parts of the output
  constexpr int PT = 8 / W;                        // 16-byte pieces of a tile's keys, and of its values, for a thread
  constexpr uint32_t kRows = 32 * W;
  char *lds = reinterpret_cast<char *>(dyn_lds);
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = rfl(tid >> 6);
  const uint32_t page = 1u << a.page_log2;
  Place at(a, lane);
  if (blockIdx.x == 0u && blockIdx.y == 0u && wave == 0u) flag_lengths(a, lane);
  const Shares sh = shares_of(a, at.count_all());
  const uint32_t units = no_cuts(a, sh, tid);
  for (uint32_t head_part = blockIdx.x; head_part < a.n_kv * a.parts; head_part += gridDim.x)
    for (uint32_t w = blockIdx.y; w < units; w += gridDim.y) {
      const uint32_t kvh = head_part / a.parts, h0 = head_part % a.parts * a.heads;
      const uint32_t heads = min(a.heads, a.group - h0), head0 = kvh * a.group + h0;
      const uint32_t page_bytes = a.n_kv * page * D;   // from one page's codes to the next's, below 2^30
      const int8_t *const kb = a.k_codes + (uint64_t)kvh * page * D, *const vb = a.v_codes + (uint64_t)kvh * page * D;
      uint64_t now = sh.begin(w);
      const uint64_t end = sh.begin(w + 1u);
      at.find(now);
      if (head_part == 0u) {
        const Cut cut = cut_of(a, at, sh, w);
        if (tid == 0u) a.cuts[w] = cut;
      }
      for (; now < end; at.next()) {
        const Seq s = at.here();
        const Blocks blocks(a.block_log2, s);
        const uint32_t all_tiles = blocks.tiles(at.block);
        const uint32_t t0 = cut_at(now, at.before), t1 = min(all_tiles, cut_at(end, at.before));
        now = at.before + blocks.work(at.block);
        if (t0 == t1) continue;
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

        const bool plain = __all(c >= 0x1p-60f);   // see fast_tile

        f32x16 o[DT];
#pragma unroll
        for (int d = 0; d < DT; ++d)
          for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
        State st = {-INFINITY, 0.0f, 0.0f, -INFINITY, 0.0f, 1.0f};

        // A tile's way: page numbers eight tiles ahead and scales four (of four tiles at
        // once, 16 blocks in each 16 lanes), codes two, f16 in LDS one.  (Past the piece's
        // last tile the last is fetched again: no branches.)  A block past the sequence's
        // end, or of a page that does not exist, takes page 0.
        bool bad = false;
        const uint32_t last = t1 - 1u;
        const auto token_of = [&](uint32_t four) { return min(four, s.len / 256u) * 256u + (fresh(lane) & 15u) * 16u; };
        const auto fetch_page = [&](uint32_t four) {
          return (uint32_t)row[min(token_of(four), max(s.len, 1u) - 1u) >> a.page_log2];
        };
        const auto page_ok = [&](uint32_t p, uint32_t four) {
          const bool there = token_of(four) < s.len && four * 4u < t1;
          bad |= there && p >= a.n_pages;
          return there && p < a.n_pages ? p : 0u;
        };
        const auto scale_at = [&](const float *scales, uint32_t p) { return scales[(uint64_t)p * a.n_kv + kvh]; };
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
          const uint32_t p = lane_of(pages, min(tile, last) % 4u * 4u + k_block + 2u * i), in = (min(tile, last) * kTile + 32u * i) & (page - 1u);
          kq[i] = *reinterpret_cast<const u32x4 *>(kb + ((uint64_t)p * page_bytes + in * D) + k_from);
        };
        const auto fetch_values = [&](uint32_t tile, uint32_t pages, int i) {
          const uint32_t p = lane_of(pages, min(tile, last) % 4u * 4u + v_block), in = (min(tile, last) * kTile) & (page - 1u);
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
        uint32_t four = t0 / 4u, pages = page_ok(fetch_page(four), four);
        const auto fetch = [&](uint32_t tile, uint32_t p) {
#pragma unroll
          for (int i = 0; i < PT; ++i) {
            fetch_keys(tile, p, i);
            fetch_values(tile, p, i);
          }
        };
        fetch(t0, pages);
        float ks = scale_at(a.k_scales, pages), vs = scale_at(a.v_scales, pages);
        uint32_t pages_next = page_ok(fetch_page(four + 1u), four + 1u), pages_raw = fetch_page(four + 2u);
#pragma unroll
        for (int i = 0; i < 4 * PT; ++i) put(t0, i / 4, i % 4);
        fetch(t0 + 1u, min(t0 + 1u, last) / 4u == four ? pages : pages_next);
        for (uint32_t t = t0; t < t1; ++four) {
          const Scales scales(ks, vs, token_of(four) >= s.len);
          ks = scale_at(a.k_scales, pages_next);
          vs = scale_at(a.v_scales, pages_next);
          for (const uint32_t end4 = min(t1, 4u * four + 4u); t < end4; ++t) {
            __syncthreads();   // tile t is there; the other buffer has been read
            // the next tiles' way, one step after another
            constexpr int kSteps = 6 * PT;
            const uint32_t p2 = min(t + 2u, last) / 4u == four ? pages : pages_next;
            const auto ahead = [&](int i) {
              if (i < 4 * PT) put(t + 1u, i / 4, i % 4);
              else if (i < 5 * PT) fetch_keys(t + 2u, p2, i - 4 * PT);
              else fetch_values(t + 2u, p2, i - 5 * PT);
            };
            if (!active || (int64_t)t * kTile >= most) {
#pragma unroll
              for (int i = 0; i < kSteps; ++i) ahead(i);
              continue;
            }
            const uint32_t ln = fresh(lane), col = ln & 31u, half = ln >> 5;
            const char *kt = lds + (t & 1u) * (L::kBytes + L::vBytes), *vt = kt + L::kBytes;
            const uint32_t kr = (col & 0x13u) | ((col & 4u) << 1) | ((col & 8u) >> 1);   // the token of row `col`
            const Tile<L> tile{kt + kr * L::kRow + half * 16u, vt + col * L::vRow + half * 64u, t % 4u * 4u};
            f32x16 x[2];
            products<2>(x, tile, 0, qf, [&](int i) {   // kSteps steps among 2 KS products
#pragma unroll
              for (int j = kSteps * i / (2 * KS); j < kSteps * (i + 1) / (2 * KS); ++j) ahead(j);
            });
            const int32_t seen = limit - (int32_t)(t * kTile);
            if (least - (int32_t)(t * kTile) < (int32_t)kTile) {   // (t kTile + kTile may be 2^31)
              results_there();
#pragma unroll
              for (int b = 0; b < 4; ++b) hide_in_place(x[b >> 1], b, seen);
            }
            if (!plain || !fast_tile(st, o, x, tile, scales, c)) slow_tile(st, o, qf, tile, c, seen, scales);
          }
          pages = pages_next;
          pages_next = page_ok(pages_raw, four + 2u);
          pages_raw = fetch_page(four + 3u);
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

// ---------------------------------------------------------------------------
// Few rows: at most 64 in a block.  A wavefront has 16 of them, and where there are no more
// than 32 or 16, the wavefronts of the same rows take turns at the tiles and are joined over LDS at the end of a piece.
// Nothing of the cache passes through LDS: scores are K Q^T and outputs V^T P^T on
// 16 x 16 x 32 matrix instructions with the rows as columns.  The first product's row
// 4 g + r of its i-th part is token 16 g + 4 i + r of the tile: lane group g (16 lanes)
// then holds 16 consecutive tokens of a row, of one page, just the 16 bytes of codes that
// it reads of one dimension, and 64 bytes of a key or of a dimension are read side by side.
// (With 32 x 32 x 16 products a key gives 32 bytes a read: 24 sequences of up to 7 tokens,
// 61 us instead of 50.)
//
// Bound: the wait for a tile's codes; a wavefront has 16 KB on the way, and the queue of
// a CU's eight is 4 TB/s of the 6.4 that reads alone reach.
// ---------------------------------------------------------------------------
constexpr uint32_t kFewWaves = 4;

__device__ __forceinline__ f32x4 mfma16(f16v8 a, f16v8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float max_of_row(float v) { return max32(max16(v)); }

template <entro_dtype T, int D>
__global__ __launch_bounds__(64 * kFewWaves, 2) void attn_few_kernel(ChunkArg a) {
  constexpr int S64 = D / 64;            // 64-dimension parts of a key row read as 16 bytes a lane
  constexpr bool S32 = (D % 64) != 0;    // and one of 32 read as 8
  constexpr int KS = D / 32;             // matrix products over the dimensions
  constexpr int DT = D / 16;             // 16-dimension parts of the output
  constexpr uint32_t kRow = D + 4;       // of the results in LDS
  float *red_o = reinterpret_cast<float *>(dyn_lds);                         // [kFewWaves][16][kRow]
  f32x4 *red_s = reinterpret_cast<f32x4 *>(red_o + kFewWaves * 16u * kRow);  // [kFewWaves][16]
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = rfl(tid >> 6), n = lane & 15u, grp = lane >> 4;
  const uint32_t page = 1u << a.page_log2;
  Place at(a, lane);
  if (blockIdx.x == 0u && blockIdx.y == 0u && wave == 0u) flag_lengths(a, lane);
  const Shares sh = shares_of(a, at.count_all());
  const uint32_t units = no_cuts(a, sh, tid);
  for (uint32_t head_part = blockIdx.x; head_part < a.n_kv * a.parts; head_part += gridDim.x)
    for (uint32_t w = blockIdx.y; w < units; w += gridDim.y) {
      const uint32_t kvh = head_part / a.parts, h0 = head_part % a.parts * a.heads;
      const uint32_t heads = min(a.heads, a.group - h0), head0 = kvh * a.group + h0;
      const uint32_t page_bytes = a.n_kv * page * D;   // from one page's codes to the next's, below 2^30
      const int8_t *const kb = a.k_codes + (uint64_t)kvh * page * D, *const vb = a.v_codes + (uint64_t)kvh * page * D;
      uint64_t now = sh.begin(w);
      const uint64_t end = sh.begin(w + 1u);
      at.find(now);
      if (head_part == 0u) {
        const Cut cut = cut_of(a, at, sh, w);
        if (tid == 0u) a.cuts[w] = cut;
      }
      for (; now < end; at.next()) {
        const Seq s = at.here();
        const Blocks blocks(a.block_log2, s);
        const uint32_t all_tiles = blocks.tiles(at.block);
        const uint32_t t0 = cut_at(now, at.before), t1 = min(all_tiles, cut_at(end, at.before));
        now = at.before + blocks.work(at.block);
        if (t0 == t1) continue;
        const int32_t *row = a.table + (uint64_t)at.seq * a.table_stride;
        const uint32_t token0 = at.block << a.block_log2;
        const uint32_t rows = min(1u << a.block_log2, s.count - token0) * heads;
        const uint32_t sets = rows <= 16u ? 1u : rows <= 32u ? 2u : 4u, set = wave & (sets - 1u);   // of 16 rows
        const uint32_t phases = kFewWaves / sets;
        // the lane's row (past the last, the last): the tokens that it sees, less the first
        // of the lane's block, the query as f16 times 2^-e, the score's factor
        const uint32_t own_row = min(16u * set + n, rows - 1u), token = token0 + own_row / heads, head = head0 + own_row % heads;
        const int32_t sees = (int32_t)max((int64_t)0, blocks.ahead + token + 1);
        const int32_t least = (int32_t)rfl((uint32_t)sees), limit = sees - 16 * (int32_t)grp;
        f16v8 qf[KS];
        float c;
        {
          u32x4 raw[KS];
          const char *q = a.q + ((int64_t)s.begin + token) * a.q_t + (int64_t)head * a.q_h;
#pragma unroll
          for (int i = 0; i < S64; ++i) {
            raw[2 * i] = *reinterpret_cast<const u32x4 *>(q + (64 * i + 16 * grp) * 2);
            raw[2 * i + 1] = *reinterpret_cast<const u32x4 *>(q + (64 * i + 16 * grp + 8) * 2);
          }
          if (S32) raw[KS - 1] = *reinterpret_cast<const u32x4 *>(q + (64 * S64 + 8 * grp) * 2);
          int e2 = 0;
          if (T == ENTRO_BF16) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < KS; ++i)
              for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(Elem<T>::lo(raw[i][e])), fabsf(Elem<T>::hi(raw[i][e]))));
            top = max_of_row(top);
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
        const bool plain = __all(c >= 0x1p-60f);   // see fast_tile
        f32x4 o[DT];
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        State st = {-INFINITY, 0.0f, 0.0f, -INFINITY, 0.0f, 1.0f};

        // This wavefront's tiles are first + phases k, k = 0 .. count - 1.  Four tiles' page
        // numbers and scales at once, 16 blocks of 16 tokens in each 16 lanes, the page
        // numbers two groups ahead and the scales one; keys one tile ahead.  (Past its last
        // tile a wavefront fetches that one again: no branches.)  A block past the sequence's
        // end, or of a page that does not exist, takes page 0.
        bool bad = false;
        const uint32_t first = t0 + (wave - set) / sets, count = t1 > first ? (t1 - first + phases - 1u) / phases : 0u;
        const uint32_t last = count ? count - 1u : 0u;
        const auto tile_of = [&](uint32_t k) { return first + min(k, last) * phases; };
        const auto token_of = [&](uint32_t four) {
          return tile_of(4u * four + (fresh(lane) >> 2 & 3u)) * kTile + (fresh(lane) & 3u) * 16u;
        };
        const auto page_at = [&](uint32_t four) {
          return (uint32_t)row[min(token_of(four), max(s.len, 1u) - 1u) >> a.page_log2];
        };
        const auto page_ok = [&](uint32_t p, uint32_t four) {
          const bool there = token_of(four) < s.len;
          bad |= there && p >= a.n_pages;
          return there && p < a.n_pages ? p : 0u;
        };
        const auto scale_at = [&](const float *scales, uint32_t p) { return scales[(uint64_t)p * a.n_kv + kvh]; };
        u32x4 kq[4][S64], vq[DT];
        u32x2 kq2[4];
        const auto fetch_keys = [&](uint32_t k, uint32_t pages) {
          const uint32_t p = (uint32_t)__shfl((int)pages, (int)((min(k, last) & 3u) * 4u + (n >> 2)));
          const uint32_t in = ((tile_of(k) * kTile + (n >> 2) * 16u) & (page - 1u)) + (n & 3u);
          const int8_t *from = kb + (uint64_t)p * page_bytes + in * D;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int e = 0; e < S64; ++e) kq[i][e] = *reinterpret_cast<const u32x4 *>(from + 4 * i * D + 64 * e + 16 * grp);
            if (S32) kq2[i] = *reinterpret_cast<const u32x2 *>(from + 4 * i * D + 64 * S64 + 8 * grp);
          }
        };
        const auto value_of = [&](uint32_t k, uint32_t pages, uint32_t d) {
          const uint32_t p = (uint32_t)__shfl((int)pages, (int)((k & 3u) * 4u + grp));
          const uint32_t in = (tile_of(k) * kTile + grp * 16u) & (page - 1u);
          return reinterpret_cast<const u32x4 *>(vb + (uint64_t)p * page_bytes + (((16u * d + n) << a.page_log2) + in));
        };
        if (count) {
          uint32_t pages = page_ok(page_at(0u), 0u);
          fetch_keys(0u, pages);
          float ks = scale_at(a.k_scales, pages), vs = scale_at(a.v_scales, pages);
          uint32_t pages_next = page_ok(page_at(1u), 1u), pages_raw = page_at(2u);
          for (uint32_t four = 0, k = 0; k < count; ++four) {
            const Scales scales(ks, vs, token_of(four) >= s.len);
            ks = scale_at(a.k_scales, pages_next);
            vs = scale_at(a.v_scales, pages_next);
            for (const uint32_t stop = min(count, 4u * four + 4u); k < stop; ++k) {
#pragma unroll
              for (int d = 0; d < DT; ++d) vq[d] = *value_of(k, pages, (uint32_t)d);
              const uint32_t its = (k & 3u) * 4u;
              float sc = c * __shfl(scales.k, (int)(its + grp));
              float by = __shfl(scales.log, (int)(its + grp)), rcp = __shfl(scales.rcp, (int)(its + grp));
              f32x4 x[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                x[i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int e = 0; e < S64; ++e) {
                  x[i] = mfma16(half8(kq[i][e].x, kq[i][e].y), qf[2 * e], x[i]);
                  x[i] = mfma16(half8(kq[i][e].z, kq[i][e].w), qf[2 * e + 1], x[i]);
                }
                if (S32) x[i] = mfma16(half8(kq2[i].x, kq2[i].y), qf[KS - 1], x[i]);
              }
              fetch_keys(k + 1u, (k & 3u) == 3u ? pages_next : pages);
              const int32_t seen = limit - (int32_t)(tile_of(k) * kTile);
              if (least - (int32_t)(tile_of(k) * kTile) < (int32_t)kTile) {   // (the tile may end at 2^31)
                results_there();
#define ENTRO_HIDE(I)                                   \
  x[I][0] = hidden<4 * I>(x[I][0], seen);               \
  x[I][1] = hidden<4 * I + 1>(x[I][1], seen);           \
  x[I][2] = hidden<4 * I + 2>(x[I][2], seen);           \
  x[I][3] = hidden<4 * I + 3>(x[I][3], seen);
                ENTRO_HIDE(0) ENTRO_HIDE(1) ENTRO_HIDE(2) ENTRO_HIDE(3)
#undef ENTRO_HIDE
              }
              float mx = -INFINITY;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                for (int r = 0; r < 4; ++r) mx = fmaxf(mx, x[i][r]);
              mx = max_of_row(mx * sc);
              const float most = lane_of(scales.most, its);
              const Rise up(st, mx, most, lane_of(scales.least, its));
              if (!(plain && (scales.fine >> its & 15u) == 15u && !__any(!up.near))) {
                // as slow_tile, a block at a time: the others' lanes have weights of 0.  The
                // outputs pass through LDS: such tiles take time, but no registers.
                float *const own_o = red_o + (wave * 16u + n) * kRow + 4u * grp;
#pragma unroll
                for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4 *>(own_o + 16 * d) = o[d];
                float own = -kFloatMax, sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  for (int r = 0; r < 4; ++r) {
                    x[i][r] = 4 * i + r < seen ? rounded(x[i][r], sc) : -INFINITY;
                    own = fmaxf(own, x[i][r]);
                  }
                u32x4 pw[2];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  for (int r = 0; r < 4; r += 2) {
                    const float p0 = exp2_fast(x[i][r] - own), p1 = exp2_fast(x[i][r + 1] - own);
                    sum += p0 + p1;
                    pw[i >> 1][2 * (i & 1) + r / 2] = Elem<ENTRO_F16>::pack2(p0 * 32768.0f, p1 * 32768.0f);
                  }
#pragma unroll 1
                for (uint32_t e = 0; e < 4u; ++e) {
                  const Scale v(lane_of(scales.v, its + e));
                  const bool mine = grp == e, any = max_of_row(mine && 0 < seen ? 1.0f : 0.0f) != 0.0f;
                  const Block b(st, max_of_row(mine ? own : -kFloatMax), v, any);
                  if (any) {
                    st.l = st.l * b.less + (mine ? sum * b.part : 0.0f);
                    b.apply(st);
                  }
                  u32x4 q[2];
#pragma unroll
                  for (int h = 0; h < 2; ++h)
                    for (int i = 0; i < 4; ++i) q[h][i] = mine ? pw[h][i] : 0u;
#pragma unroll 1
                  for (uint32_t d = 0; d < (uint32_t)DT; ++d) {
                    const u32x4 code = *value_of(k, pages, d);
                    f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
                    z = mfma16(half8(code.x, code.y), __builtin_bit_cast(f16v8, q[0]), z);
                    z = mfma16(half8(code.z, code.w), __builtin_bit_cast(f16v8, q[1]), z);
                    f32x4 *const at_o = reinterpret_cast<f32x4 *>(own_o + 16u * d);
                    f32x4 y = *at_o;
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = y[i] * b.keep + (any ? z[i] * b.f : 0.0f);
                    *at_o = y;
                  }
                }
                st.settle();
#pragma unroll
                for (int d = 0; d < DT; ++d) o[d] = *reinterpret_cast<const f32x4 *>(own_o + 16 * d);
                // and nothing of the tile is left for below
                by = rcp = 0.0f;
                sc = 1.0f;
                for (int i = 0; i < 4; ++i) x[i] = (f32x4){-0x1p120f, -0x1p120f, -0x1p120f, -0x1p120f};
              } else {
                if (__any(up.rise)) {
                  const float less = up.apply(st);
                  results_there();
#pragma unroll
                  for (int d = 0; d < DT; ++d) scale_in_place(o[d], less);
                }
                st.top = with_tile(st, mx, most);
              }
              u32x4 p[2];
              float sum = 0.0f;
              const float off = by + st.off;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                for (int r = 0; r < 4; r += 2) {
                  const uint32_t y = Elem<ENTRO_F16>::pack2(exp2_fast(__builtin_fmaf(x[i][r], sc, off)),
                                                            exp2_fast(__builtin_fmaf(x[i][r + 1], sc, off)));
                  p[i >> 1][2 * (i & 1) + r / 2] = y;
                  sum = Elem<ENTRO_F16>::add2(y, sum);
                }
              st.l = __builtin_fmaf(sum * rcp, st.unit, st.l);
#pragma unroll
              for (int d = 0; d < DT; ++d) {
                o[d] = mfma16(half8(vq[d].x, vq[d].y), __builtin_bit_cast(f16v8, p[0]), o[d]);
                o[d] = mfma16(half8(vq[d].z, vq[d].w), __builtin_bit_cast(f16v8, p[1]), o[d]);
              }
            }
            pages = pages_next;
            pages_next = page_ok(pages_raw, four + 2u);
            pages_raw = page_at(four + 3u);
          }
        }
        if (bad) atomicOr(a.status + at.seq, ENTRO_F_PAGE);
        {
          const uint32_t place = wave * 16u + n;
          const float l = add32(add16(st.l));
          if (grp == 0u) red_s[place] = (f32x4){st.m, l, st.top == -INFINITY ? -INFINITY : st.g, 0.0f};
#pragma unroll
          for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4 *>(red_o + place * kRow + 16 * d + 4 * grp) = o[d];
        }
        __syncthreads();
        const uint64_t slot = (((uint64_t)head_part * a.shares + w) * 2u + (t0 == 0u)) * a.rows;
        for (uint32_t i = tid; i < rows * (D / 4u); i += 64u * kFewWaves) {
          const uint32_t r = i / (D / 4u), d = i % (D / 4u) * 4u;
          Joined j = {-INFINITY, 0.0f, -INFINITY, {0.0f, 0.0f, 0.0f, 0.0f}};
          for (uint32_t place = r; place < 16u * kFewWaves; place += 16u * sets) {
            const f32x4 q = red_s[place];
            j.add(q.x, q.y, q.z, *reinterpret_cast<const f32x4 *>(red_o + place * kRow + d));
          }
          if (t1 - t0 == all_tiles) {
            *reinterpret_cast<u32x2 *>(a.out + ((int64_t)s.begin + token0 + r / heads) * a.o_t + (int64_t)(head0 + r % heads) * a.o_h +
                                       d * 2u) = j.result<T>();
          } else {
            if (d == 0u) a.part_s[slot + r] = (f32x4){j.m, j.l, j.g, 0.0f};
            *reinterpret_cast<f32x4 *>(a.part_o + (slot + r) * D + d) = j.o;
          }
        }
        __syncthreads();   // red_o and red_s are written again
      }
    }
}

// Joins the pieces of the blocks that were cut: kJoinSlots slots of D / 4 threads, four
// dimensions each, for the first cut in a block.  A slot takes whole rows; where there
// are many pieces the slots take every kJoinSlots-th piece of one row and are joined
// over LDS.  Four pieces' reads at once; the order is the same in every call.  Its time
// is that of its waits: 2 to 15 us.
constexpr uint32_t kJoinSlots = 8;
template <entro_dtype T, int D>
__global__ __launch_bounds__(kJoinSlots * D / 4) void attn_chunk_join_kernel(ChunkArg a) {
  const uint32_t kRows = a.rows, kGroups = a.join_groups;
  __shared__ Joined red[kJoinSlots][D / 4];
  const uint32_t slot = threadIdx.x / (D / 4u), dq = threadIdx.x % (D / 4u);
  for (uint32_t w = 1u + blockIdx.y; w < a.shares; w += gridDim.y) {
    const Cut cut = a.cuts[w];
    if (cut.y == 0u) continue;
    const uint32_t pieces = rfl(cut.z) - w + 2u;
    for (uint64_t y = blockIdx.x; y < (uint64_t)a.n_kv * a.parts * kGroups; y += gridDim.x) {
      const uint32_t head_part = (uint32_t)(y / kGroups), group = (uint32_t)(y % kGroups);
      const uint32_t kvh = head_part / a.parts, h0 = head_part % a.parts * a.heads;
      const uint32_t heads = min(a.heads, a.group - h0), head0 = kvh * a.group + h0, rows = rfl(cut.y) * heads;
      const uint64_t base = ((uint64_t)head_part * a.shares + w) * 2u * kRows;
      // (steps of four pieces, one row after another in the first case)
      const bool many = (rows + kGroups - 1u) / kGroups * ((pieces + 4u * kJoinSlots - 1u) / (4u * kJoinSlots)) < (pieces + 3u) / 4u;
      for (uint32_t r0 = many ? group : group * kJoinSlots; r0 < rows; r0 += many ? kGroups : kRows) {
        const uint32_t r = many ? r0 : min(r0 + slot, rows - 1u), step = many ? kJoinSlots : 1u;
        Joined j = {-INFINITY, 0.0f, -INFINITY, {0.0f, 0.0f, 0.0f, 0.0f}};
        for (uint32_t p0 = many ? slot : 0u; p0 < pieces; p0 += 4u * step) {
          f32x4 q[4], x[4];
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i) {
            // the first piece is share w - 1's last, the others are first ones
            const uint32_t p = min(p0 + i * step, pieces - 1u);
            const uint64_t place = p ? base + (uint64_t)(p - 1u) * 2u * kRows + r : base - kRows + r;
            q[i] = a.part_s[place];
            x[i] = *reinterpret_cast<const f32x4 *>(a.part_o + place * D + 4u * dq);
          }
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i)
            if (p0 + i * step < pieces) j.add(q[i].x, q[i].y, q[i].z, x[i]);
        }
        if (many) {
          red[slot][dq] = j;
          __syncthreads();
          if (slot == 0u)
            for (uint32_t i = 1; i < kJoinSlots; ++i) j.add(red[i][dq].m, red[i][dq].l, red[i][dq].g, red[i][dq].o);
          __syncthreads();
          if (slot) continue;
        } else if (r0 + slot >= rows) {
          continue;
        }
        *reinterpret_cast<u32x2 *>(a.out + ((int64_t)cut.x + r / heads) * a.o_t + (int64_t)(head0 + r % heads) * a.o_h + dq * 8u) =
            j.result<T>();
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// How a call is laid out.
struct Plan {
  uint32_t waves;   // 0: few rows
  uint32_t rows, heads, parts, block_log2, shares;
};
static Plan plan_of(uint32_t n_seq, uint32_t total_q, uint32_t n_heads, uint32_t n_kv, uint32_t head_dim) {
  Plan p{};
  const uint32_t group = n_heads / n_kv;
  const uint64_t rows = (uint64_t)total_q * group;
  // By the rows of a sequence on average (the lengths are on the device).  Up to 48 the
  // kernel for few rows: 24 sequences of up to 16 tokens behind up to 6000, 32 / 8 heads
  // of 128 (34 rows on average), 38.6 us instead of 44.9; 4 tokens behind 40000 30.6
  // instead of 36.5.  Above that its blocks are too small: 16 tokens behind 40000 (64
  // rows), 66.6 us instead of 59.4.  (By heads of 64, 64 sequences of 40 rows behind 2000,
  // 32 heads, 248 us and 256 with blocks of 128 rows, of 64 rows 252 and 257; 96, 314 and
  // 316, then 334 and 325; of 128, 32 / 8 heads, the few rows' kernel is behind from some
  // 32 rows on: of 24 rows 61 and 72, of 40 107 and 88.)
  // Above 128 blocks of 256 rows.  The same sequences with 128 rows, blocks of 256 and of
  // 128: 428 and 319 us with heads of 64, 493 and 389 of 96, 137 and 105 of 128; with 160
  // rows 506 and 482, 575 and 629, 157 and 168; 16 with 1024 rows 632 and 638, 741 and 838,
  // 186 and 213.  Where lengths spread over a factor of 32 the average stands for few of
  // them, and blocks of 128 take less up to some 400 rows: 411 and 330 (182 rows on
  // average), 596 and 566 (210), 177 and 161 (223).
  p.waves = rows > 128ull * n_seq ? 8u : rows > 48ull * n_seq ? 4u : 0u;
  p.rows = p.waves ? 32u * p.waves : rows > 32ull * n_seq ? 64u : rows > 16ull * n_seq ? 32u : 16u;
  p.heads = std::min(group, p.rows);
  p.parts = (group + p.heads - 1u) / p.heads;
  while ((2u << p.block_log2) * p.heads <= p.rows) ++p.block_log2;
  // as many workgroups as the GPU holds at once: 1, 2 or (heads of 64) 3 a CU
  p.shares = std::max(1u, (p.waves == 8u ? 256u : p.waves == 4u && head_dim == 64u ? 768u : 512u) / (n_kv * p.parts));
  return p;
}

// Whether outputs lie where queries do, which workgroups that share a block still read:
// where both begin at the same place, or both are without gaps.  (Slices of one tensor
// may lie between one another.)
static bool same_place(const entro_rows &q, const entro_rows &out, uint32_t rows, uint32_t n_heads, uint32_t dim) {
  if (rows == 0) return false;
  const auto dense = [&](const entro_rows &x) { return x.stride_h == dim && x.stride_t == (int64_t)n_heads * dim; };
  const uintptr_t a = reinterpret_cast<uintptr_t>(q.d), b = reinterpret_cast<uintptr_t>(out.d);
  return a == b || (dense(q) && dense(out) && std::max(a, b) - std::min(a, b) < 2ull * rows * n_heads * dim);
}

template <entro_dtype T, int D>
static entro_status launch_chunk(const ChunkArg &a, uint32_t waves, hipStream_t s) {
  const uint32_t heads = a.n_kv * a.parts;
  const dim3 grid = grid2(heads, a.shares);
  (void)hipGetLastError();
  if (waves == 8u)
    hipLaunchKernelGGL((attn_chunk_kernel<T, D, 8>), grid, dim3(512), Lds<D>::bytes, s, a);
  else if (waves == 4u)
    hipLaunchKernelGGL((attn_chunk_kernel<T, D, 4>), grid, dim3(256), Lds<D>::bytes, s, a);
  else
    hipLaunchKernelGGL((attn_few_kernel<T, D>), grid, dim3(64 * kFewWaves), kFewWaves * 16u * (D + 8u) * 4u, s, a);
  if (hipGetLastError() != hipSuccess) return ENTRO_E_HIP;
  if (a.shares > 1u && a.total_q) {
    hipLaunchKernelGGL((attn_chunk_join_kernel<T, D>), grid2((uint64_t)heads * a.join_groups, a.shares - 1u),
                       dim3(kJoinSlots * D / 4), 0, s, a);
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
  const Plan p = plan_of(n_seq, total_q, n_heads, n_kv_heads, head_dim);
  if (p.shares == 1u) return 16u;   // (no block is cut)
  return (uint64_t)n_kv_heads * p.parts * p.shares * 2u * p.rows * (head_dim + 4u) * 4u + 16u * p.shares;
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
  if (same_place(a->q, a->out, a->total_q, a->n_heads, c->head_dim)) return ENTRO_E_INVAL;
  const uint64_t need = entro_attn_chunk_work_bytes(t->n_seq, a->total_q, a->n_heads, c->n_kv_heads, c->head_dim);
  if (need && (!a->d_work || (reinterpret_cast<uintptr_t>(a->d_work) & 15u) || a->work_bytes < need)) return ENTRO_E_INVAL;
  const Plan p = plan_of(t->n_seq, a->total_q, a->n_heads, c->n_kv_heads, c->head_dim);
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
  k.group = a->n_heads / c->n_kv_heads;
  k.heads = p.heads;
  k.parts = p.parts;
  k.block_log2 = p.block_log2;
  k.rows = p.rows;
  // (more for a sequence with many pieces: 4 tokens behind 40000, 30.6 us instead of 52.6;
  // where there are few, the workgroups without rows cost: 24 of up to 7 tokens, 11 us
  // instead of 6)
  k.join_groups = std::max(p.rows / kJoinSlots, p.shares >= 32u * t->n_seq ? 16u : 0u);
  k.shares = p.shares;
  k.scale = std::fabs(a->scale) * kLog2e;
  k.q_xor = std::signbit(a->scale) ? 0x80008000u : 0u;
  k.cuts = static_cast<u32x4 *>(a->d_work);
  k.part_s = reinterpret_cast<f32x4 *>(k.cuts + p.shares);
  k.part_o = reinterpret_cast<float *>(k.part_s + (uint64_t)k.n_kv * k.parts * k.shares * 2u * p.rows);
  k.status = d_status;
  const auto dims = [&](auto type) {
    return c->head_dim == 64u   ? launch_chunk<decltype(type)::value, 64>(k, p.waves, stream)
           : c->head_dim == 96u ? launch_chunk<decltype(type)::value, 96>(k, p.waves, stream)
                                : launch_chunk<decltype(type)::value, 128>(k, p.waves, stream);
  };
  return a->dtype == ENTRO_BF16 ? dims(std::integral_constant<entro_dtype, ENTRO_BF16>{})
                                : dims(std::integral_constant<entro_dtype, ENTRO_F16>{});
}

// HIP kernels (gfx950) and entry points of the attention over the 8-bit cache:
// entro_attn_cache.  Layout and definition are in entro_attn.h.
#include <algorithm>

#include "entro_attn_device.h"
#include "entro_internal.h"

namespace entro {

constexpr uint32_t kTile = 64;          // tokens a wavefront takes at a time
constexpr uint32_t kCacheWaves = 4;     // wavefronts per workgroup, interleaved over its tiles
constexpr uint32_t kHeadsPerWg = 16;    // query heads of one key/value head (columns of the matrix products)
constexpr uint32_t kShareTiles = 4;     // least tiles of a workgroup's share
constexpr float kFloatMax = 3.40282347e38f;

// Shares of a call, all heads together: the workgroups that 256 CUs hold at
// once by the kernel's registers, two on each at head dimension 128 and three
// below.  32 ragged sequences (32 heads, f16), two against three: up to 16384
// tokens at 64 119 and 117 us (four: 132), up to 8192 at 96 113 and 111.
constexpr uint32_t shares_at(uint32_t head_dim) { return head_dim == 128u ? 512u : 768u; }

struct CacheArg {
  const int8_t *k_codes, *v_codes;
  const float *k_scales, *v_scales;
  const int32_t *table;
  uint64_t table_stride;
  uint32_t table_pages, n_seq, n_pages, n_kv;
  uint32_t page_log2;
  const char *q;
  char *out;
  int64_t q_t, q_h, o_t, o_h;   // bytes
  const int32_t *lens;
  uint32_t n_heads, group;      // group: query heads per key/value head
  uint32_t parts;               // workgroups (of kHeadsPerWg query heads) per key/value head
  uint32_t shares;              // that the tokens of a key/value head are split into at most; 0: one sequence each
  float scale;                  // times log2(e)
  float *part_o;                // [n_seq + shares][n_heads][D]
  f32x2 *part_ml;               // [n_seq + shares][n_heads]: Piece's o and gap
  uint32_t *status;
};

__device__ __forceinline__ uint32_t cache_len(const CacheArg &a, uint32_t b, bool *ok = nullptr) {
  const int32_t n = a.lens[b];
  const bool fine = n >= 0 && (uint64_t)n <= ((uint64_t)a.table_pages << a.page_log2);
  if (ok) *ok = fine;
  return fine ? (uint32_t)n : 0u;
}

__device__ __forceinline__ uint32_t tiles_in(uint32_t len) { return (len + kTile - 1u) / kTile; }

// The sequences' lengths.  A wavefront's lanes keep the first 64, which are most
// calls' all: a workgroup's way to its first key is a chain of reads, and one
// less takes up to 0.6 us off a kernel (the join of 64 sequences 5.7 -> 5.1).
struct Lens {
  const CacheArg &a;
  uint32_t lane, first;
  __device__ explicit Lens(const CacheArg &arg, uint32_t lane_) : a(arg), lane(lane_) {
    first = lane < a.n_seq ? cache_len(a, lane) : 0u;
  }
  // of sequence b0 + lane (0 where there is none), b0 a multiple of 64
  __device__ uint32_t lanes(uint32_t b0) const {
    return b0 == 0u ? first : b0 + lane < a.n_seq ? cache_len(a, b0 + lane) : 0u;
  }
  // of sequence b, the same in all lanes
  __device__ uint32_t of(uint32_t b) const {
    return b < 64u ? (uint32_t)__builtin_amdgcn_readlane((int)first, (int)b) : rfl(cache_len(a, b));
  }
  // tiles of the sequences before b, one after another
  __device__ uint64_t tiles_before(uint32_t b) const {
    uint64_t sum = 0;
    for (uint32_t b0 = 0; b0 < b; b0 += 64u) {
      const uint32_t len = lanes(b0), t = b0 + lane < b ? tiles_in(len) : 0u;
      sum += (uint32_t)__builtin_amdgcn_readlane((int)wave_scan(t), 63);   // 64 terms of at most 2^25
    }
    return rfl64(sum);
  }
};

// The tiles of all sequences, one after another, in equal shares (to one tile)
// whatever the sequences' lengths, one workgroup each and as many as the GPU
// holds at once: share w has tiles begin(w) .. begin(w + 1) - 1.  A share's part
// of one sequence is a piece; a sequence in one piece is finished by its
// workgroup, the others' pieces are joined by the second kernel.  Piece (w, b)
// of share w and sequence b has the workspace's place w + b: going along the
// tiles, one of the two grows at each end of a piece.
struct Shares {
  uint64_t tiles;
  uint32_t n;
  __device__ uint64_t begin(uint32_t w) const { return w * tiles / n; }
  // the share of tile t: the last w with begin(w) <= t, i.e. w tiles < (t + 1) n
  __device__ uint32_t of(uint64_t t) const { return (uint32_t)(((t + 1u) * n + tiles - 1u) / tiles) - 1u; }
};
__device__ __forceinline__ Shares shares_of(const CacheArg &a, const Lens &lens) {
  Shares s;
  s.tiles = lens.tiles_before(a.n_seq);
  s.n = (uint32_t)min((uint64_t)a.shares, max((uint64_t)1, s.tiles / kShareTiles));
  return s;
}

// What is known of a piece of a head's tokens beside its outputs, in powers of
// two: `o`, the exponent of the outputs (times 2^15, see below), and `gap`, how far
// the logarithm of its softmax's sum lies below o.  o goes with the scores and may
// be large; the gap goes with the values' size, and is held by itself because it is
// what the result's size follows from.  Without tokens o is -inf and the gap inf; the
// gap is NaN where the result is.
typedef f32x2 Piece;
__device__ __forceinline__ float above(float o, float ref) { return o == ref ? 0.0f : o - ref; }

// Pieces joined: outputs relative to the largest o, their weights' sum relative
// to 2^(o + w).
struct Joined {
  float o, w;
  __device__ float of(Piece p) const { return above(p.x, o) - p.y; }   // logarithm of a piece's sum, less o
};
// What the joined outputs are multiplied by.
struct Factor {
  float r;
  int e;
  __device__ Factor(Joined j, float sum) {
    const float up = fminf(fmaxf(-j.w, -512.0f), 512.0f), whole = floorf(up);
    r = j.w == -INFINITY && sum == sum ? 0.0f : exp2_fast(up - whole) / sum;
    e = (int)whole - 15;
  }
  __device__ float of(float x) const { return ldexpf(x * r, e); }
};
// The gap of pieces whose weights sum to `sum` relative to 2^(o + w).
__device__ __forceinline__ float gap_of(float w, float sum) { return sum == 0.0f ? INFINITY : -(w + __log2f(sum)); }

__device__ __forceinline__ f32x4 mfma16(f16v8 a, f16v8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// One workgroup takes pieces of sequences for one key/value head and up to 16
// of its query heads; its four wavefronts take every fourth tile of 64 tokens
// and join their results in LDS.
//
// A tile's scores are K Q^T and its product V^T P^T, both on the matrix cores
// with the query heads as the 16 columns, so that softmax statistics are per
// column (a lane and the lanes 16, 32, 48 further hold one head) and the
// weights leave the first product in the lanes where the second wants them:
// the first product's row 4 g + r of its i-th part is made token
// 16 g + 4 i + r, and lane group g then holds 16 consecutive tokens, just the
// 16 bytes of value codes it reads for one dimension.  Nothing of the cache
// passes through LDS; each code is read once, 16 bytes a lane.  The next tile's
// keys are on their way from where this tile's scores are done, a tile's values
// from its start.
//
// Codes become f16 exactly; q is brought to f16 by a power of two (exact but
// for values below 2^-17 of the row's largest, which are rounded at 2^-25 of it).
// With t = s + log2(value scale) and M its running maximum, weights go into the
// product as 2^(t - M + 15): the scale of a page's values rides in the exponent,
// and f16 covers weights down to 2^-29 of the largest with 11 bits.
//
// A page's scale may be anything from 0 (values all zero; taken as 2^-200) to the
// type's largest, so the softmax's sum has a maximum of its own, of the scores
// alone, and one for each lane, whose 16 tokens of a tile are all of one page:
// weights are computed less the largest of the 16, added up in 32 bits, and brought
// to the product's by one factor of the lane.  Scores may be far from 0, where a
// scale's logarithm added to them is lost: M is held less an anchor, the score whose
// t was the largest when M last rose, and only differences of scores meet
// anything else (the scores are rounded first: a fused difference would have the
// rounding left over).
//
// Bound by the reading of the cache: 131072 tokens of one sequence (32 / 8 heads
// of 128) 43 us, 6.2 TB/s, where a kernel that only reads reaches 6.4; 64 ragged
// sequences of up to 16384 tokens 119 us, 5.3 TB/s; 8 of up to 4099 (32 heads of
// 96) 16 us, 3.7 TB/s, a third of it the way to the first key and the wavefronts'
// join.  90 tokens: 4.8 us.  At head dimension 128 registers for a
// third workgroup a CU would take spills: 120 -> 135 us.
// ---------------------------------------------------------------------------
template <entro_dtype T, int D>
__global__ __launch_bounds__(256, 2) void attn_cache_kernel(CacheArg a) {
  constexpr int S64 = D / 64;            // 64-dimension parts of a key row read as 16 bytes a lane
  constexpr bool S32 = (D % 64) != 0;    // and one of 32 read as 8
  constexpr int KS = D / 32;             // matrix products over the dimensions
  constexpr int DT = D / 16;             // 16-dimension parts of the output
  __shared__ float red_o[kCacheWaves][kHeadsPerWg][D + 4];
  __shared__ f32x2 red_ml[kCacheWaves][kHeadsPerWg];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
  const uint32_t n = lane & 15u, g = lane >> 4;
  const uint32_t page = 1u << a.page_log2;
  const Lens lens(a, lane);
  if (blockIdx.x == 0u && blockIdx.y == 0u)
    for (uint32_t b = tid; b < a.n_seq; b += 256u) {
      bool ok;
      cache_len(a, b, &ok);
      if (!ok) atomicOr(a.status + b, ENTRO_F_LENGTH);
    }
  Shares sh{};
  if (a.shares) sh = shares_of(a, lens);
  const uint32_t units = a.shares ? sh.n : a.n_seq;
  for (uint32_t part = blockIdx.y; part < a.n_kv * a.parts; part += gridDim.y)
    for (uint32_t w = blockIdx.x; w < units; w += gridDim.x) {
      const uint32_t kvh = part / a.parts, h0 = (part % a.parts) * kHeadsPerWg;
      const uint32_t heads = min(kHeadsPerWg, a.group - h0);
      const uint32_t head0 = kvh * a.group + h0;
      // empty sequences have no piece
      if (w == 0u)
        for (uint32_t b = wave; b < a.n_seq; b += kCacheWaves)
          if (lens.of(rfl(b)) == 0u)
            for (uint32_t i = lane; i < heads * (D / 2u); i += 64u)
              *reinterpret_cast<uint32_t *>(a.out + b * a.o_t + (int64_t)(head0 + i / (D / 2u)) * a.o_h + i % (D / 2u) * 4u) = 0u;
      // the tiles t0 .. t1 - 1 of sequence `seq` that come next, of the `left` that the share still has
      uint32_t seq, t0;
      uint64_t left;
      if (a.shares) {
        const uint64_t begin = sh.begin(w);
        left = sh.begin(w + 1u) - begin;
        uint64_t before = 0;
        seq = 0u;
        t0 = 0u;
        for (uint32_t b0 = 0; b0 < a.n_seq; b0 += 64u) {
          const uint32_t own = tiles_in(lens.lanes(b0));
          const uint32_t run = wave_scan(own);
          const uint64_t past = __ballot(before + run > begin);
          if (past) {
            const uint32_t at = (uint32_t)__builtin_ctzll(past);
            seq = rfl(b0 + at);
            t0 = rfl((uint32_t)(begin - before - __builtin_amdgcn_readlane(run - own, at)));
            break;
          }
          before += __builtin_amdgcn_readlane(run, 63);
        }
      } else {
        seq = w;
        t0 = 0u;
        left = tiles_in(lens.of(w));
      }
      for (; left; ++seq, t0 = 0u) {
        const uint32_t len = lens.of(seq), all_tiles = tiles_in(len);
        const uint32_t t1 = (uint32_t)min((uint64_t)all_tiles, t0 + left);
        if (t1 == t0) continue;   // an empty sequence
        left -= t1 - t0;
        const int32_t *row = a.table + (uint64_t)seq * a.table_stride;

        // the query head of this lane's column, as f16 times 2^-e
        f16v8 qf[KS];
        float c;                               // score = c * key scale * product
        {
          u32x4 raw[KS];
          const char *q = a.q + seq * a.q_t + (int64_t)(head0 + min(n, heads - 1u)) * a.q_h;
#pragma unroll
          for (int s = 0; s < S64; ++s) {
            raw[2 * s] = *reinterpret_cast<const u32x4 *>(q + (64 * s + 16 * g) * 2);
            raw[2 * s + 1] = *reinterpret_cast<const u32x4 *>(q + (64 * s + 16 * g + 8) * 2);
          }
          if (S32) raw[KS - 1] = *reinterpret_cast<const u32x4 *>(q + (64 * S64 + 8 * g) * 2);
          float top = 0.0f;
#pragma unroll
          for (int s = 0; s < KS; ++s)
            for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(Elem<T>::lo(raw[s][e])), fabsf(Elem<T>::hi(raw[s][e]))));
          top = max32(max16(top));
          int e2 = 0;
          if (T == ENTRO_BF16) e2 = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127;   // bf16 denormals: -127
          c = ldexpf(a.scale, e2);
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            if (T == ENTRO_F16) {
              qf[s] = __builtin_bit_cast(f16v8, raw[s]);
            } else {
              u32x4 w;
              for (int e = 0; e < 4; ++e)
                w[e] = Elem<ENTRO_F16>::pack2(ldexpf(Elem<T>::lo(raw[s][e]), -e2), ldexpf(Elem<T>::hi(raw[s][e]), -e2));
              qf[s] = __builtin_bit_cast(f16v8, w);
            }
          }
        }

        f32x4 o[DT];
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        float anchor = 0.0f, m = -INFINITY;   // M is their sum
        float top = -kFloatMax, l = 0.0f;     // of the scores, and the weights' sum: this lane's tokens only
        bool bad = false;

        // Pages of the 16-token blocks that this lane reads keys of (n / 4) and
        // values of (g).  A block past the end, or of a page that does not exist,
        // reads page 0 and counts as hidden.
        struct Pages {
          int32_t k, v;
        };
        auto pages = [&](uint32_t tile) {
          const uint32_t tk = tile * kTile + (n >> 2) * 16u, tv = tile * kTile + g * 16u;
          return (Pages){tk < len ? row[tk >> a.page_log2] : 0, tv < len ? row[tv >> a.page_log2] : 0};
        };
        u32x4 kq[4][S64], vq[DT];
        u32x2 kq2[4];
        auto keys = [&](uint32_t tile, int32_t p) {
          const uint32_t tk = tile * kTile + (n >> 2) * 16u;
          const uint64_t at = (uint64_t)((uint32_t)p < a.n_pages ? (uint32_t)p : 0u) * a.n_kv + kvh;
          const int8_t *kp = a.k_codes + ((at << a.page_log2) + (tk & (page - 1u)) + (n & 3u)) * D;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int s = 0; s < S64; ++s) kq[i][s] = *reinterpret_cast<const u32x4 *>(kp + 4 * i * D + 64 * s + 16 * g);
            if (S32) kq2[i] = *reinterpret_cast<const u32x2 *>(kp + 4 * i * D + 64 * S64 + 8 * g);
          }
        };
        const uint32_t first = t0 + wave;
        Pages now{}, next{};
        if (first < t1) {
          now = pages(first);
          keys(first, now.k);
        }
        for (uint32_t tile = first; tile < t1; tile += kCacheWaves) {
          const bool more = tile + kCacheWaves < t1;
          if (more) next = pages(tile + kCacheWaves);
          const uint32_t tv = tile * kTile + g * 16u;
          const bool v_bad = (uint32_t)now.v >= a.n_pages;
          bad |= v_bad;
          const uint64_t av = (uint64_t)(v_bad ? 0u : (uint32_t)now.v) * a.n_kv + kvh;
          const int8_t *vp = a.v_codes + ((av * D + n) << a.page_log2) + (tv & (page - 1u));
          const float ks = a.k_scales[av] * c;   // rows 4 g + r of the products are tokens of block g
          const float v_scale = a.v_scales[av];
#pragma unroll
          for (int d = 0; d < DT; ++d) vq[d] = *reinterpret_cast<const u32x4 *>(vp + ((uint64_t)(16 * d) << a.page_log2));

          f32x4 s4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s4[i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < S64; ++s) {
              s4[i] = mfma16(half8(kq[i][s].x, kq[i][s].y), qf[2 * s], s4[i]);
              s4[i] = mfma16(half8(kq[i][s].z, kq[i][s].w), qf[2 * s + 1], s4[i]);
            }
            if (S32) s4[i] = mfma16(half8(kq2[i].x, kq2[i].y), qf[KS - 1], s4[i]);
          }
          if (more) keys(tile + kCacheWaves, next.k);
          now = next;
          // scores in powers of two
          const uint32_t seen = v_bad || tv >= len ? 0u : min(16u, len - tv);
          const float vs = seen ? v_scale : 0.0f;
          const float lv = seen ? fmaxf(__log2f(vs), -200.0f) : -INFINITY;
          float mx = -kFloatMax;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            for (int r = 0; r < 4; ++r) {
              const float t = (uint32_t)(4 * i + r) < seen ? rounded(s4[i][r], ks) : -INFINITY;
              s4[i][r] = t;
              mx = fmaxf(mx, t);
            }
          const float t = mx - anchor + lv, mt = max32(max16(t));
          if (__any(mt > m)) {
            const bool rise = mt > m;
            const float next = rise ? max32(max16(t == mt ? mx : -INFINITY)) : anchor;
            const float mn = max32(max16(mx - next + lv)), k = rise ? exp2_fast(m - (next - anchor) - mn) : 1.0f;
            anchor = next;
            m = rise ? mn : m;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= k;
          }
          const float f = exp2_fast(fminf(mx - anchor + lv - m + 15.0f, 15.0f));   // (inf - inf counts as 15: all is 0)
          float sum = 0.0f;
          u32x4 pw[2];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float p[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              p[r] = exp2_fast(s4[i][r] - mx);
              sum += p[r];
            }
            pw[i >> 1][2 * (i & 1)] = Elem<ENTRO_F16>::pack2(p[0] * f, p[1] * f);
            pw[i >> 1][2 * (i & 1) + 1] = Elem<ENTRO_F16>::pack2(p[2] * f, p[3] * f);
          }
          const float up = fmaxf(top, mx);
          l = l * exp2_fast(top - up) + sum * exp2_fast(mx - up) + vs * 0.0f;   // NaN where the scale is no number
          top = up;
          const f16v8 p0 = __builtin_bit_cast(f16v8, pw[0]), p1 = __builtin_bit_cast(f16v8, pw[1]);
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            o[d] = mfma16(half8(vq[d].x, vq[d].y), p0, o[d]);
            o[d] = mfma16(half8(vq[d].z, vq[d].w), p1, o[d]);
          }
        }
        if (bad) atomicOr(a.status + seq, ENTRO_F_PAGE);
        // join the lanes, then the wavefronts
        const float wave_top = max32(max16(top));
        l = add32(add16(l * exp2_fast(top - wave_top)));
        if (g == 0u) red_ml[wave][n] = (Piece){anchor + m, gap_of(wave_top - anchor - m, l)};
#pragma unroll
        for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4 *>(&red_o[wave][n][16 * d + 4 * g]) = o[d];
        __syncthreads();
        const bool whole = t1 - t0 == all_tiles;
        for (uint32_t i = tid; i < heads * (D / 2u); i += 256u) {
          const uint32_t h = i / (D / 2u), d = i % (D / 2u) * 2u;
          Joined j{-INFINITY, -INFINITY};
#pragma unroll
          for (uint32_t v = 0; v < kCacheWaves; ++v) j.o = fmaxf(j.o, red_ml[v][h].x);
#pragma unroll
          for (uint32_t v = 0; v < kCacheWaves; ++v) j.w = fmaxf(j.w, j.of(red_ml[v][h]));
          float x = 0.0f, y = 0.0f, sum = 0.0f;
#pragma unroll
          for (uint32_t v = 0; v < kCacheWaves; ++v) {
            const float k = exp2_fast(above(red_ml[v][h].x, j.o));
            x += k * red_o[v][h][d];
            y += k * red_o[v][h][d + 1u];
            sum += join_factor(j.of(red_ml[v][h]), j.w);
          }
          if (whole) {
            const Factor f(j, sum);
            *reinterpret_cast<uint32_t *>(a.out + seq * a.o_t + (int64_t)(head0 + h) * a.o_h + d * 2u) =
                Elem<T>::pack2(f.of(x), f.of(y));
          } else {
            const uint64_t at = ((uint64_t)w + seq) * a.n_heads + head0 + h;
            *reinterpret_cast<f32x2 *>(a.part_o + at * D + d) = (f32x2){x, y};
            if (d == 0u) a.part_ml[at] = (Piece){j.o, gap_of(j.w, sum)};
          }
        }
        __syncthreads();
      }
    }
}

// Joins the pieces of a split sequence: one workgroup per sequence and query
// head.  G groups of 64 threads (two dimensions each) take every G-th piece,
// four at a time, then the groups are joined; the order is the same in every
// call.  The pieces' reads wait for one another only from batch to batch: with
// few workgroups (one long sequence: 64 pieces) 16 groups read them at once,
// with many (few pieces each) four leave room for more workgroups.  4 to 5.5 us,
// a chain of reads: what it moves would take less than one.
template <entro_dtype T, int D, int G>
__global__ __launch_bounds__(64 * G) void attn_join_kernel(CacheArg a) {
  __shared__ float red_o[G][D];
  __shared__ f32x2 red_ml[G];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, group = tid >> 6;
  const Lens lens(a, lane);
  const Shares sh = shares_of(a, lens);
  for (uint32_t head = blockIdx.y; head < a.n_heads; head += gridDim.y)
    for (uint32_t b = blockIdx.x; b < a.n_seq; b += gridDim.x) {
      const uint32_t tiles = tiles_in(lens.of(b));
      if (tiles == 0u) continue;
      const uint64_t begin = lens.tiles_before(b);
      const uint32_t w0 = sh.of(begin), n = sh.of(begin + tiles - 1u) - w0 + 1u;
      if (n == 1u) continue;
      const uint64_t at = ((uint64_t)w0 + b) * a.n_heads + head;
      const f32x2 *ml = a.part_ml + at;
      const float *po = a.part_o + at * D;
      const uint32_t d = min(lane * 2u, D - 2u);
      Joined j{-INFINITY, -INFINITY};
      float x = 0.0f, y = 0.0f, sum = 0.0f;
      for (uint32_t i0 = group; i0 < n; i0 += 4u * G) {
        f32x2 v[4], p[4];
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) {
          const uint64_t i = min(i0 + (uint32_t)G * c, n - 1u);
          v[c] = ml[i * a.n_heads];
          p[c] = *reinterpret_cast<const f32x2 *>(po + i * a.n_heads * D + d);
        }
        Joined up = j;
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) up.o = fmaxf(up.o, v[c].x);
        const float by = above(j.o, up.o), k = exp2_fast(by);
        j.w += by;
        up.w = j.w;
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) up.w = fmaxf(up.w, up.of(v[c]));
        x *= k;
        y *= k;
        sum *= join_factor(j.w, up.w);
        j = up;
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) {
          if (i0 + (uint32_t)G * c >= n) break;
          const float kc = exp2_fast(above(v[c].x, j.o));
          x += kc * p[c].x;
          y += kc * p[c].y;
          sum += join_factor(j.of(v[c]), j.w);
        }
      }
      if (lane * 2u < D) *reinterpret_cast<f32x2 *>(&red_o[group][d]) = (f32x2){x, y};
      if (lane == 0u) red_ml[group] = (Piece){j.o, gap_of(j.w, sum)};
      __syncthreads();
      if (group == 0u && lane * 2u < D) {
        j = Joined{-INFINITY, -INFINITY};
        x = y = sum = 0.0f;
        for (int g = 0; g < G; ++g) j.o = fmaxf(j.o, red_ml[g].x);
        for (int g = 0; g < G; ++g) j.w = fmaxf(j.w, j.of(red_ml[g]));
        for (int g = 0; g < G; ++g) {
          const float k = exp2_fast(above(red_ml[g].x, j.o));
          x += k * red_o[g][d];
          y += k * red_o[g][d + 1u];
          sum += join_factor(j.of(red_ml[g]), j.w);
        }
        const Factor f(j, sum);
        *reinterpret_cast<uint32_t *>(a.out + b * a.o_t + head * a.o_h + d * 2u) = Elem<T>::pack2(f.of(x), f.of(y));
      }
      __syncthreads();   // red_o and red_ml are written again
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Shares of one key/value head's tokens.
static uint32_t cache_shares(uint32_t n_kv, uint32_t parts, uint32_t head_dim) {
  return std::max(1u, shares_at(head_dim) / (n_kv * parts));
}

template <entro_dtype T, int D>
static entro_status launch_cache(CacheArg &a, hipStream_t s) {
  // Where no sequence can be long, a workgroup each and nothing to join: the
  // second kernel and its launch cost more than some rounds of the wavefronts
  // (32 / 8 heads of 128: 12 sequences of up to 393 tokens 16 us with and 7 us
  // without, 16 of up to 1000 15 and 11, one of 1000 11 and 10, one of 1536 11 and
  // 13).  With more workgroups than run at once the longest come on top: 64 of up
  // to 768 tokens, 32 heads of 96, 41 and 35; of up to 1000 35 and 46 in an earlier
  // state of the kernel.
  const uint64_t tiles = (((uint64_t)a.table_pages << a.page_log2) + kTile - 1u) / kTile;
  const bool split = tiles > ((uint64_t)a.n_seq * a.n_kv * a.parts <= shares_at(D) ? 24u : 12u);
  a.part_ml = reinterpret_cast<f32x2 *>(a.part_o + ((uint64_t)a.n_seq + a.shares) * a.n_heads * D);
  if (!split) a.shares = 0;
  (void)hipGetLastError();
  hipLaunchKernelGGL((attn_cache_kernel<T, D>), grid2(split ? a.shares : a.n_seq, a.n_kv * a.parts), dim3(256), 0, s, a);
  if (hipGetLastError() != hipSuccess) return ENTRO_E_HIP;
  if (split) {
    if ((uint64_t)a.n_seq * a.n_heads <= 256u)
      hipLaunchKernelGGL((attn_join_kernel<T, D, 16>), grid2(a.n_seq, a.n_heads), dim3(1024), 0, s, a);
    else
      hipLaunchKernelGGL((attn_join_kernel<T, D, 4>), grid2(a.n_seq, a.n_heads), dim3(256), 0, s, a);
    if (hipGetLastError() != hipSuccess) return ENTRO_E_HIP;
  }
  return ENTRO_OK;
}

}  // namespace entro

using namespace entro;

extern "C" uint64_t entro_attn_cache_work_bytes(uint32_t n_seq, uint32_t n_heads, uint32_t n_kv_heads, uint32_t head_dim) {
  if (n_seq == 0 || check_heads(n_heads, n_kv_heads, head_dim, ENTRO_BF16) != ENTRO_OK) return 0;
  const uint32_t parts = (n_heads / n_kv_heads + kHeadsPerWg - 1u) / kHeadsPerWg;
  return ((uint64_t)n_seq + cache_shares(n_kv_heads, parts, head_dim)) * n_heads * (head_dim + 2ull) * 4ull;
}

extern "C" entro_status entro_attn_cache(const entro_kv_cache *c, const entro_kv_table *t, const entro_attn_cache_args *a,
                                         uint32_t *d_status, hipStream_t stream) {
  if (!a) return ENTRO_E_INVAL;
  entro_status st = check_cache(c, t);
  if (st != ENTRO_OK) return st;
  st = check_heads(a->n_heads, c->n_kv_heads, c->head_dim, a->dtype);
  if (st != ENTRO_OK) return st;
  if (!std::isfinite(a->scale)) return ENTRO_E_INVAL;
  if (t->n_seq == 0) return ENTRO_OK;
  if (!a->d_lens || !d_status || !a->d_work || (reinterpret_cast<uintptr_t>(a->d_work) & 15u)) return ENTRO_E_INVAL;
  for (const entro_rows *r : {&a->q, &a->out}) {
    st = check_rows(*r, t->n_seq);
    if (st != ENTRO_OK) return st;
  }
  if (a->work_bytes < entro_attn_cache_work_bytes(t->n_seq, a->n_heads, c->n_kv_heads, c->head_dim)) return ENTRO_E_INVAL;
  CacheArg k{};
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
  k.lens = a->d_lens;
  k.n_heads = a->n_heads;
  k.group = a->n_heads / c->n_kv_heads;
  k.parts = (k.group + kHeadsPerWg - 1u) / kHeadsPerWg;
  k.shares = cache_shares(k.n_kv, k.parts, c->head_dim);
  k.scale = a->scale * kLog2e;
  k.part_o = static_cast<float *>(a->d_work);
  k.status = d_status;
  if (a->dtype == ENTRO_BF16)
    return c->head_dim == 64u   ? launch_cache<ENTRO_BF16, 64>(k, stream)
           : c->head_dim == 96u ? launch_cache<ENTRO_BF16, 96>(k, stream)
                                : launch_cache<ENTRO_BF16, 128>(k, stream);
  return c->head_dim == 64u   ? launch_cache<ENTRO_F16, 64>(k, stream)
         : c->head_dim == 96u ? launch_cache<ENTRO_F16, 96>(k, stream)
                              : launch_cache<ENTRO_F16, 128>(k, stream);
}

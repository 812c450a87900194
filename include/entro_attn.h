/*
 * entro_attn.h - attention and the 8-bit key/value cache beside the coded
 * weight products of entro.h (MI355X, gfx950).
 *
 * The fused products turn activations into queries, keys and values and take
 * the attention's output back; the four entry points here do what lies
 * between: causal attention of packed prompts (entro_attn_prompt), keys and
 * values into a paged 8-bit cache (entro_kv_store) and back to 16 bits
 * (entro_kv_load), and attention of one new token per sequence over the cache
 * (entro_attn_cache).
 *
 * Heads.  n_heads query heads, n_kv_heads key/value heads; n_kv_heads divides
 * n_heads and query head h reads key/value head h / (n_heads / n_kv_heads).
 * head_dim is 64, 96 or 128.
 *
 * 16-bit operands (q, k, v, out) are indexed [token][head][dim]: element
 * (t, h, d) at t * stride_t + h * stride_h + d, strides in elements, so that
 * slices of a joint projection need no copy.  Pointers are 16-byte aligned and
 * strides multiples of 8 (ENTRO_E_INVAL otherwise).  entro_attn_prompt takes
 * row strides of q, k and v up to 2^23 elements (ENTRO_E_UNSUPPORTED beyond).
 *
 * Packed sequences.  d_cu holds n_seq + 1 running sums: sequence b has rows
 * d_cu[b] .. d_cu[b + 1] - 1.  A sequence may be empty.
 *
 * Cache.  Pages of page_tokens tokens; sequence b's token p lies in page
 * d_table[b * table_stride + p / page_tokens], row p % page_tokens:
 *   key codes    int8 [page][kv head][row][dim]
 *   value codes  int8 [page][kv head][dim][row]
 *   scales       float [page][kv head], one array for keys, one for values
 * and the value of a code is code * scale; scales are 0 or more (entro_attn_cache
 * takes value scales below 2^-126 as 0).  Values are held with a row's
 * tokens side by side because the product with the attention weights runs
 * along the tokens.  A page belongs to one sequence while it is written;
 * pages that are only read may be shared.
 *
 * Conventions are those of entro.h: d_* are device pointers owned by the
 * caller, arguments are checked on the host before anything is enqueued, work
 * goes to the caller's stream, nothing is allocated or kept.  Problems in the
 * data are OR-ed into the caller-zeroed d_status[b] of sequence b, whose
 * outputs are then unspecified; kernels never leave the stated buffers.  Rows
 * that belong to no sequence are neither read nor written.  Codes that belong to
 * none are left as they are and influence nothing, but may be read: whole pages
 * of a sequence are, and page 0, with its scales, in the place of pages that a
 * sequence does not have.
 */
#ifndef ENTRO_ATTN_H
#define ENTRO_ATTN_H

#include "entro.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of q, k, v and out. */
typedef enum { ENTRO_BF16 = 0, ENTRO_F16 = 1 } entro_dtype;

/* Per-sequence faults OR-ed into d_status[b]. */
#define ENTRO_F_LENGTH 0x40u /* running sums not ascending within the stated rows (one
                                that begins before an earlier sequence's end among
                                them; keys of a prompt may be shared), a negative
                                position, or tokens past the table's row              */
#define ENTRO_F_PAGE 0x80u   /* a page index outside the cache where tokens lie; the
                                page is skipped                                       */

/* A 16-bit operand's place and strides (elements). */
typedef struct {
  void *d;
  int64_t stride_t, stride_h;
} entro_rows;

typedef struct {
  int8_t *d_k_codes;
  int8_t *d_v_codes;       /* both 16-byte aligned */
  float *d_k_scales;
  float *d_v_scales;
  uint32_t n_pages;
  uint32_t page_tokens;    /* 16, 32, 64 or 128 */
  uint32_t n_kv_heads;
  uint32_t head_dim;       /* 64, 96 or 128 */
} entro_kv_cache;

/* The pages of the sequences of a call. */
typedef struct {
  const int32_t *d_table;  /* [n_seq][table_stride], the first table_pages of a row used */
  uint32_t table_stride;
  uint32_t table_pages;
  uint32_t n_seq;
} entro_kv_table;

typedef struct {
  entro_rows q, k, v, out;
  const int32_t *d_cu_q;   /* [n_seq + 1] */
  const int32_t *d_cu_k;   /* [n_seq + 1]; may be d_cu_q */
  uint32_t n_seq;
  uint32_t total_q;        /* rows at q and out */
  uint32_t total_k;        /* rows at k and v   */
  uint32_t n_heads, n_kv_heads, head_dim;
  entro_dtype dtype;
  float scale;             /* factor of q . k, finite */
  void *d_work;            /* NULL, or entro_attn_prompt_work_bytes, 16-byte aligned; contents irrelevant */
  uint64_t work_bytes;
} entro_attn_prompt_args;

/* Bytes of workspace with which entro_attn_prompt splits the keys of a call
 * whose few queries have many keys each (a piece of a prompt behind a long
 * prefix) over more workgroups; 0 where it would not, or where an argument is
 * out of its range.  Without workspace the keys are not split. */
uint64_t entro_attn_prompt_work_bytes(uint32_t n_seq, uint32_t total_q, uint32_t total_k, uint32_t n_heads,
                                      uint32_t n_kv_heads, uint32_t head_dim);

/* Causal attention of packed prompts.  For sequence b with Lq queries and Lk
 * keys (the last Lq of them the queries' own), query i and head h:
 *   out = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale * q . k_j),
 *   j = 0 .. i + Lk - Lq;
 * a query with no key (Lk < Lq, or Lk = 0) gives 0.  Keys and values outside
 * a query's range have no influence on it, whatever they hold.  Products of
 * 16-bit values are exact and summed in 32 bits, as are the softmax's
 * statistics; the weights are rounded to the element type for the product
 * with v and for their sum, the result once at the end.  An infinite value
 * that a query sees gives it an infinity or, where its weight is no longer above
 * 0, NaN.  Finite values of any size give finite results; bf16 values below
 * 2^-118 * total_k count with fewer bits.  Sequences of any length up to 2^31 - 1
 * rows; out must not overlap the inputs. */
entro_status entro_attn_prompt(const entro_attn_prompt_args *a, uint32_t *d_status, hipStream_t stream);

typedef struct {
  entro_rows k, v;         /* the new tokens of all sequences, packed */
  const int32_t *d_held;   /* [n_seq] tokens that sequence b has in the cache before the call */
  const int32_t *d_cu_new; /* [n_seq + 1] */
  uint32_t total_new;      /* rows at k and v */
  entro_dtype dtype;
} entro_kv_store_args;

/* Write the new tokens of each sequence behind those it holds.  For every page
 * that gets tokens and every head, keys and values each on their own:
 *   s0 = the page's scale if it holds tokens of the sequence already, else 0
 *   s1 = max(s0, max |x| * float(1 / 127)) over the new finite x
 *   new codes = rint(x * (1 / s1)), limited to +-127 (infinities are
 *   limited, NaN becomes 0); codes held before = rint(code * (s0 / s1)),
 * in 32-bit arithmetic with rint to even, the scale s1 stored; where s1 is
 * below 2^-126 (all values zero, for one) the codes are 0.  No two sequences of
 * a call may write to the same page. */
entro_status entro_kv_store(const entro_kv_cache *c, const entro_kv_table *t, const entro_kv_store_args *a,
                            uint32_t *d_status, hipStream_t stream);

typedef struct {
  entro_rows k, v;         /* outputs, packed */
  const int32_t *d_first;  /* [n_seq] position of the first token to read */
  const int32_t *d_cu_out; /* [n_seq + 1] */
  uint32_t total_out;      /* rows at k and v */
  entro_dtype dtype;
} entro_kv_load_args;

/* Read tokens d_first[b] .. d_first[b] + (count of b) - 1 of each sequence
 * back as 16-bit values, code * scale rounded to nearest even (what
 * entro_attn_prompt takes as the keys and values in front of a prompt's next
 * piece).  The caller names only tokens that the cache holds. */
entro_status entro_kv_load(const entro_kv_cache *c, const entro_kv_table *t, const entro_kv_load_args *a,
                           uint32_t *d_status, hipStream_t stream);

typedef struct {
  entro_rows q, out;       /* [n_seq][n_heads][head_dim]; stride_t between sequences */
  const int32_t *d_lens;   /* [n_seq] tokens of sequence b, the new one among them */
  uint32_t n_heads;
  entro_dtype dtype;
  float scale;
  void *d_work;            /* entro_attn_cache_work_bytes, 16-byte aligned; contents irrelevant */
  uint64_t work_bytes;
} entro_attn_cache_args;

/* Bytes of workspace that entro_attn_cache needs (0 where an argument is out
 * of its range): the partial results of long sequences, whose tokens are split
 * over workgroups. */
uint64_t entro_attn_cache_work_bytes(uint32_t n_seq, uint32_t n_heads, uint32_t n_kv_heads, uint32_t head_dim);

/* Attention of one query per sequence over the cache: as entro_attn_prompt
 * with Lq = 1 and the cache's values.  A sequence without tokens gives 0.
 * The result does not depend on timing: partial results are joined in the
 * order of the tokens.  Where a table's row has room for more than 1536 tokens
 * (768 with more workgroups than run at once), tokens are split over workgroups
 * and joined by a second launch, however few d_lens names: a table_pages no larger
 * than the call's longest sequence needs takes half the time for short ones (12
 * of up to 393 tokens, 32 / 8 heads of 128, 7 us against 16 in a table of 2048
 * pages). */
entro_status entro_attn_cache(const entro_kv_cache *c, const entro_kv_table *t, const entro_attn_cache_args *a,
                              uint32_t *d_status, hipStream_t stream);

/* entro_set_max_workgroups for the launches of this header: at most n
 * workgroups each from now on (0, the default: no cap); returns the cap before. */
uint32_t entro_attn_set_max_workgroups(uint32_t n);

#ifdef __cplusplus
}
#endif

#endif /* ENTRO_ATTN_H */

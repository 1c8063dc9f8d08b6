/*
 * csbp_generate.h -- C ABI of libcsbp's generation operators: what a trained
 * block-diffusion model or drafter needs, next to csbp_attn_fwd, to produce
 * text block by block on one sm_103a GPU.
 *
 *   csbp_cache_write / csbp_cache_read   a paged K/V cache kept in E4M3 with
 *                     one power-of-two scale per 32 features, written from
 *                     bf16 and read back to bf16
 *   csbp_attn_prefix  attention of a batch of sequences that share one long
 *                     prefix: the prefix keys are read once for all of them
 *   csbp_draft_verify verification of drafted tokens against the target's
 *                     probabilities, from given random numbers
 *
 * A block of M tokens goes through them like this: the clean K/V of the block
 * before it are written to the cache, the sequences' own keys are read back
 * once, every denoising step runs csbp_attn_prefix with M queries per
 * sequence (its block reads itself bidirectionally, as a corrupted block
 * does in csbp_attn_fwd), and csbp_draft_verify keeps the drafts that the
 * target model accepts.  One token per sequence is the case queries = 1.
 * The method's pages describe training only (project page "Block Parallelism
 * for Efficient Distributed Long-Context Diffusion Language Model Training");
 * these operators have no counterpart there, except that they keep its
 * conventions: GQA heads h / (Hq / Hkv), natural-log LSE, exact merging of
 * partial attentions (blog section "在线 softmax 合并：为什么分两段算仍是同一个注意力").
 *
 * Conventions are those of csbp.h: caller-owned memory, asynchronous work on
 * `stream` of the current device, errors as csbp_status before anything is
 * enqueued, 16-byte aligned device pointers (4 bytes where stated).  Values
 * that only the device knows (lengths, pages, tokens) cannot be refused on
 * the host; each operator says below what an out-of-range one does, and none
 * makes a kernel read or write outside the given buffers.
 */
#ifndef CSBP_GENERATE_H_
#define CSBP_GENERATE_H_

#include <stddef.h>
#include <stdint.h>

#include "csbp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------- quantised cache
 * One layer's K and V, each as
 *   codes   uint8 [pages][page_size][Hkv][d]       E4M3 (csbp_e4m3_to_bf16)
 *   scales  uint8 [pages][page_size][Hkv][d / 32]  byte s stands for 2^(s-127),
 *           255 for NaN
 * d: a multiple of 32, 32 .. 1024.  A value is code x scale, so reading back
 * is exact in bf16 (wherever 2^(s-127) x code is a bf16 number; smaller ones
 * round to nearest even).                                                 */
typedef struct {
  int64_t pages;      /* >= 1, at most 2^31 - 1                             */
  int32_t page_size;  /* tokens per page, 1 .. 65536                        */
  int32_t Hkv, d;
  void *k, *v;              /* codes                                        */
  void *k_scale, *v_scale;  /* scale bytes (any alignment)                  */
} csbp_kv_cache;

/* Which tokens of the cache a call works on, and the strides of the bf16
 * tensors [batch][rows][Hkv][d] on the other side.  Row i of sequence b is
 * the token at position start[b] + i, which lives in page
 * table[b][position / page_size] at place position % page_size.
 *   table  device int32 [batch][table_pages], 4-byte aligned
 *   start  device int32 [batch];  count  device int32 [batch] or NULL: only
 *          rows i < count[b] take part (NULL: all rows)
 *   stride_tok[i], stride_batch[i]  element strides of K (i = 0) and V (1),
 *          as in csbp_inputs: 0 = contiguous, multiples of 8
 * batch = 0 or rows = 0 is a no-op.                                       */
typedef struct {
  int32_t batch, rows, table_pages;
  const int32_t *table, *start, *count;
  int64_t stride_tok[2], stride_batch[2];
} csbp_cache_rows;

/* Quantise and write.  Per token, head and group of 32 features x:
 *   A = max |x_c| over the finite x_c
 *   e = the smallest integer >= -127 with A <= 448 x 2^e   (A = 0: -127)
 *   code_c = E4M3 nearest-even of x_c x 2^-e (no overflow),  scale byte e+127
 * NaN and infinities are stored as NaN (E4M3 has no infinities).  A row whose
 * position is negative or past the table, or whose page is outside
 * [0, pages), is not written.  Rows that land on the same place of the same
 * page leave each byte of it as one of them writes it: codes and scales may
 * come from different rows.  Nothing else of the cache changes.            */
csbp_status csbp_cache_write(const csbp_kv_cache* cache, const csbp_cache_rows* rows,
                             const void* k, const void* v, void* stream);

/* Read back: bf16 [batch][rows][Hkv][d] (strides as given).  Rows i >=
 * count[b] of k and v are left as they were; a row whose position or page is
 * out of range (as above) reads as NaN.                                   */
csbp_status csbp_cache_read(const csbp_kv_cache* cache, const csbp_cache_rows* rows, void* k,
                            void* v, void* stream);

/* --------------------------------------------------- shared-prefix attention
 * `batch` sequences of `queries` tokens each.  Every query reads all
 * prefix_len prefix keys, which the sequences share, and keys of its own
 * sequence: with c = min(max(own_len[b], 0), own_max),
 *   causal = 0  own keys j < c (the block reads itself in both directions)
 *   causal = 1  own keys j <= c - queries + i for query i (the queries are
 *               the last tokens of the c)
 * O = softmax(scale Q K^T) V over those keys and LSE the natural log of the
 * softmax denominator.  A query that reads no key has O = 0, LSE = -inf.  A key
 * that a query does not read has no part in its result, whatever it holds (own
 * rows at and past c, later keys, other sequences' keys), NaN included.
 * O is summed in fp32 on the tensor cores, which drop what is below the last
 * place: a row reads about 262,144 keys (twice as many at most) into one sum,
 * which costs it 2^-10 (2^-9) of its value where all values share a sign.
 * causal = 1 is made for a few queries (drafted tokens, a block): all c own
 * keys pass by every query, so a chunk of thousands of queries does up to twice
 * the work that its own keys need.                                          */
typedef struct {
  int32_t batch, queries;       /* >= 1                                     */
  int32_t prefix_len, own_max;  /* >= 0, below 2^31 - 128                   */
  int32_t Hq, Hkv, d;           /* Hq % Hkv == 0; d 64 or 128               */
  int32_t causal;
  float scale;                  /* > 0, finite                              */
} csbp_prefix_problem;

/* bf16 device tensors: q [batch][queries][Hq][d], k_prefix and v_prefix
 * [prefix_len][Hkv][d] (NULL allowed when prefix_len is 0), k_own and v_own
 * [batch][own_max][Hkv][d] and own_len int32 [batch], 4-byte aligned (all
 * three NULL allowed when own_max is 0).  The work is cut up as if own_len were
 * five eighths of own_max: an own_max near the longest length in use (smaller than
 * the tensor's rows by its batch stride) is faster than a far larger one.
 * Strides as in csbp_inputs, in that
 * order; the batch strides of the prefix are not read.  batch x the batch
 * stride of q stays within 2^34 elements, batch x queries x Hq below 2^30.  */
typedef struct {
  const void *q, *k_prefix, *v_prefix, *k_own, *v_own;
  const int32_t* own_len;
  int64_t stride_tok[5];
  int64_t stride_batch[5];
} csbp_prefix_inputs;

/* Workspace bytes of csbp_attn_prefix on the current device: the status word
 * and the fp32 partial results (d + 1 numbers per query and head) of the key
 * ranges that a query's keys are cut into: as many as share its keys among the
 * SMs or, with many queries, one to two per 262,144 keys.  0 for an invalid
 * problem. */
size_t csbp_prefix_workspace_bytes(const csbp_prefix_problem* problem);

/*  o    bf16 [batch][queries][Hq][d];  lse  fp32 [batch][Hq][queries]
 *  workspace  as in csbp_attn_fwd (csbp_check_status reads its status word);
 *             calls that can overlap need workspaces of their own          */
csbp_status csbp_attn_prefix(const csbp_prefix_problem* problem, const csbp_prefix_inputs* in,
                             void* o, float* lse, void* workspace, size_t ws_bytes,
                             void* stream);

/* -------------------------------------------------------- draft verification
 * Sequence b drafted n = min(max(length[b], 0), drafts) tokens x_0 .. x_n-1
 * from the probabilities q_i; p_0 .. p_n are the target's.  Draft i is
 * accepted while u_i q_i(x_i) < p_i(x_i); a is the first i that is not, or n.
 * The next token comes from w_v = max(p_a(v) - q_a(v), 0) when a < n (from
 * p_a when that is 0 everywhere), from p_n when a = n: the smallest v with
 * w_0 + .. + w_v > r (w_0 + .. + w_V-1).
 * The products and comparisons are exact and the sums are kept to 2^-42 of
 * their value (2^-47 as a rule), for any vocabulary.  A negative weight or NaN counts as 0; without any positive
 * finite weight, or with sums that are not finite, the next token is -1.  A
 * draft outside [0, vocab) is not accepted.                               */
typedef struct {
  int32_t batch;   /* >= 0 (0: no-op)                                       */
  int32_t drafts;  /* 0 .. 4096                                             */
  int32_t vocab;   /* >= 1                                                  */
  int64_t p_row, p_batch;  /* element strides of p [batch][drafts + 1][vocab] */
  int64_t q_row, q_batch;  /* and q [batch][drafts][vocab]; 0 = contiguous,
                              else >= vocab, and >= rows x row stride       */
} csbp_verify_problem;

/*  p, q      device fp32, 4-byte aligned (16 is faster)
 *  token     device int32 [batch][drafts];  u  device fp32 [batch][drafts],
 *  r         device fp32 [batch], all in [0, 1)
 *  length    device int32 [batch] or NULL (all drafts)
 *  accepted  device int32 [batch] (out): a
 *  out       device int32 [batch][drafts + 1] (out): the accepted drafts, the
 *            next token, then -1
 * q, token and u may be NULL when drafts is 0 (plain sampling from p).     */
csbp_status csbp_draft_verify(const csbp_verify_problem* problem, const float* p,
                              const float* q, const int32_t* token, const float* u,
                              const float* r, const int32_t* length, int32_t* accepted,
                              int32_t* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CSBP_GENERATE_H_ */

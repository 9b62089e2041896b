/*
 * spec_decode.h — C ABI of libspecverify.so: the operators of a decode step around the verify step.
 *
 * One round of speculative decoding with a target model, per request b with ctx_len[b] tokens in the
 * cache and T_b new tokens (the last emitted token and the drafts behind it, or a tree of drafts):
 *   in every layer   spec_kv_append       rotates the new tokens' queries and keys to their positions
 *                                         and puts the keys and values into the paged cache;
 *                    spec_paged_attention the new tokens attend over the cache and one another;
 *   on the logits    spec_process_logits  penalties for repeated tokens, biases and grammar masks at
 *                                         every drafted position (then spec_verify / spec_verify_multi);
 *   after verifying  spec_kv_keep         moves the accepted branch's cache entries up behind the context.
 * Where the cache is to stay small, an E4M3 one may have a scale per page and head that follows what goes into it
 * (spec_kv_page_scales_t: the _ex forms below), and entries that attention does not look at may go:
 *   after verifying  spec_kv_weigh        adds up the weight that the accepted tokens gave every entry (before spec_kv_keep);
 *   now and then     spec_kv_select       picks the entries of each head that stay within a budget;
 *                    spec_kv_move         brings them together at the front.
 *
 * Conventions are those of spec_verify.h: caller-owned device memory, no allocation, no
 * synchronisation, work enqueued on `stream`, host-checkable errors as status codes.  Problems in
 * device data never trap and never reach outside the buffers; what each operator makes of them is
 * stated with it.  The structs are host memory, read before the call returns.
 *
 * Cache slots: token i of request b is in slot i, which is row i % page_size of page
 * pages[b, i / page_size].  The new tokens of a step take slots ctx_len[b] .. ctx_len[b] + T_b - 1.
 */
#ifndef SPEC_DECODE_H_
#define SPEC_DECODE_H_

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Flag bits that spec_kv_append ORs into out_flags (beside SPEC_FLAG_BAD_K for t_per_row). */
#define SPEC_FLAG_BAD_SLOT 64      /* a new token's slot or page lies outside the table or the pool,
                                      or ctx_len is negative                                        */
#define SPEC_FLAG_BAD_POSITION 128 /* a position outside [0, max_positions): clamped into range     */

/* Limits (SPEC_ERR_UNSUPPORTED beyond them). */
#define SPEC_MAX_BATCH 65535        /* B, but for spec_kv_append (B * T < 2^31)                      */
#define SPEC_MAX_NEW 64             /* T of spec_paged_attention (a tree mask has one bit per token)
                                       and of spec_process_logits                                    */
#define SPEC_MAX_GROUP 128          /* q heads per kv head of spec_paged_attention; its requests x kv
                                       heads x row groups (of at most 128 rows) x (page table's slots /
                                       128 + 4) stay under 2^31                                      */
#define SPEC_MAX_PAGE 4096          /* page_size: a power of two in [8, SPEC_MAX_PAGE]               */
#define SPEC_MAX_SLOTS (1 << 30)    /* max_pages * page_size of one request, and the length of its lists:
                                       max_keep, max_moves of spec_kv_move                           */
#define SPEC_MAX_HISTORY 1048448    /* history entries of spec_process_logits                        */
#define SPEC_MAX_BIAS 2046          /* bias entries per request of spec_process_logits               */

/*
 * Heads of a batch of tokens: element (b, t, h, d) is at data[b * row_stride + t * token_stride +
 * h * head_stride + d], bf16.  data is 16-byte aligned and the strides are multiples of 8 elements,
 * so the heads of q, k and v may be parts of one projection's output.
 */
typedef struct {
  void* data;
  int64_t row_stride, token_stride, head_stride;
} spec_heads_t;

/*
 * A paged cache of keys and values: element (l, page, row, h, d) of k is at k[l * layer_stride +
 * page * page_stride + row * slot_stride + h * head_stride + d], and v likewise.  The strides are in
 * elements and multiples of 16 bytes, k and v are 16-byte aligned: any order of the page, row and
 * head dimensions does, and head_dim is innermost.
 *   heads          kv heads; the q heads are a multiple of them (q head i reads kv head i / group);
 *   head_dim       64 or 128;
 *   dtype          SPEC_DTYPE_BF16 or SPEC_DTYPE_E4M3;
 *   k_scale, v_scale  [heads] float (device) or NULL = 1: an entry stands for its stored value times
 *                  its head's scale.  E4M3 only.
 */
typedef struct {
  void* k;
  void* v;
  int64_t layer_stride, page_stride, slot_stride, head_stride;
  int32_t layers, num_pages, page_size, heads, head_dim;
  spec_dtype_t dtype;
  const float* k_scale;
  const float* v_scale;
} spec_kv_cache_t;

/*
 * A scale per page and head of an E4M3 cache: an entry of layer l, page p and head h stands for its code times
 * k[l * layer_stride + p * heads + h] (v likewise).  A scale counts where it lies in [2^-24, 2^24]; spec_kv_append_ex,
 * spec_kv_keep_ex and spec_kv_move set it:
 *   need(a) = the smallest power of two s in that range with a <= 448 s, a the largest finite magnitude that goes in.
 * An E4M3 code has 4 significant bits whatever its scale, so a power of two loses none of them, and where a page's scale
 * grows the codes that stay are codes again, exactly but for those that become subnormal.  Pages of two requests that
 * share them must not be written to.
 */
typedef struct {
  float* k;
  float* v;
  int64_t layer_stride;
} spec_kv_page_scales_t;

/*
 * What is known about every entry of a cache: the attention weight that it has gathered and the position of its token,
 * element (l, page, h, row) at [l * layer_stride + (page * heads + h) * page_size + row].  Either may be NULL where an
 * operator says so.  The sizes are the cache's.
 */
typedef struct {
  float* weight;
  int32_t* position;
  int64_t layer_stride;
  int32_t layers, num_pages, page_size, heads;
} spec_kv_record_t;

/*
 * The batch of a step.
 *   pages      [B, max_pages] int32: the page of every page_size slots of a request.  Entries past
 *              those that hold its slots are not read;
 *   ctx_len    [B] int32: tokens in the cache before this step, >= 0 (a negative value counts as 0);
 *   t_per_row  [B] int32 or NULL (= T): the request's new tokens T_b in [0, T], clamped into it.
 */
typedef struct {
  const int32_t* pages;
  const int32_t* ctx_len;
  const int32_t* t_per_row;
  int32_t B, T, max_pages;
} spec_decode_batch_t;

/*
 * Position rotation.  The first rot_dim elements of a head are pairs: (i, i + rot_dim / 2), or
 * (2i, 2i + 1) where interleaved != 0; pair i of a token at position n becomes
 *   (x cos - y sin, y cos + x sin)   with cos = cos[n, i], sin = sin[n, i], [max_positions, rot_dim / 2] float.
 * rot_dim is 0 (no rotation; the tables may be NULL) or a multiple of 16 up to head_dim.  positions
 * [B, T] int32, or NULL: token t of request b is at position ctx_len[b] + t.  A tree's tokens are at
 * ctx_len[b] + their depth.
 */
typedef struct {
  const float* cos_table;
  const float* sin_table;
  const int32_t* positions;
  int32_t rot_dim, max_positions, interleaved;
} spec_rotary_t;

/*
 * Rotate the new tokens' queries and keys and put their keys and values into layer 0 of `cache`:
 *   q_out = rot(q),  K[slot] = rot(k) / k_scale,  V[slot] = v / v_scale,
 * in 32 bits and rounded once: to bf16, or to E4M3 with what is beyond +-448 cut to it (NaN stays NaN).
 *   q, q_out [B, T, q_heads, head_dim], k, v [B, T, heads, head_dim]; q_out may be q itself.
 *   q_out rows past a request's T_b tokens become 0; k and v rows past them are not read.
 *   out_flags [B] int32 or NULL: SPEC_FLAG_* bits are ORed into it (the caller clears it).  A token
 *   whose slot or page lies outside the table or the pool is not written to the cache.
 * q_heads == 0 (q and q_out NULL) appends keys and values alone.  T is not limited: prompts go the
 * same way as drafts.  Two requests must not share the page of a new token.
 */
spec_status_t spec_kv_append(const spec_heads_t* q, const spec_heads_t* k, const spec_heads_t* v,
                             const spec_heads_t* q_out, int32_t q_heads, const spec_kv_cache_t* cache,
                             const spec_decode_batch_t* batch, const spec_rotary_t* rotary,
                             int32_t* out_flags, void* stream);

/*
 * spec_kv_append into an E4M3 cache with page scales (layer 0 of `scales`; cache->k_scale and v_scale are NULL).  A page's
 * new scale is need(the new tokens' keys in it, rotated in 32 bits), values likewise; where the page also holds tokens from before
 * (slots < ctx_len[b]) and has a scale that counts, it is not less than that one, and if it is more, those tokens' codes
 * become round(code * old / new).  The new codes are round(x / scale), infinities cut to +-448.  scales == NULL is spec_kv_append.
 */
spec_status_t spec_kv_append_ex(const spec_heads_t* q, const spec_heads_t* k, const spec_heads_t* v,
                                const spec_heads_t* q_out, int32_t q_heads, const spec_kv_cache_t* cache,
                                const spec_kv_page_scales_t* scales, const spec_decode_batch_t* batch,
                                const spec_rotary_t* rotary, int32_t* out_flags, void* stream);

/* Bytes of device workspace spec_paged_attention needs for these sizes (0 for invalid ones). */
size_t spec_paged_attention_workspace_bytes(int32_t B, int32_t T, int32_t q_heads, int32_t heads,
                                            int32_t head_dim);

/*
 * Attention of the new tokens over layer 0 of the cache (their own entries included, so after
 * spec_kv_append):
 *   out[b, t, h] = sum_s w_s V_s / sum_s w_s,  w_s = exp(scale * q[b, t, h] . K_s - max),
 * over the request's context slots s < ctx_len[b] and the new tokens that t attends to: those up to
 * t, or, with `mask`, new token i where bit i of mask[b, t] is set ([B, T] int64, T <= 64).
 *   q, out [B, T, q_heads, head_dim] bf16.  Rows past T_b, and rows that attend to nothing, are 0.
 * Slots that a row does not attend to have no part in it, whatever they hold (NaN and infinities
 * among them).  A page outside the pool reads as zeros; slots past the page table are dropped.
 * Scores, weights and sums are fp32; the weights are rounded where they multiply V (bf16 for a bf16 cache, whose
 * row's sum is that of the rounded ones; fp16 for E4M3).  Over an E4M3 cache a query row enters the scores as an E4M3 and an E5M2
 * number an element: exactly where the element reaches 2^-13 of the row's largest, within 2^-21 of that largest elsewhere; a row
 * that holds an infinity gives NaN.
 * Each wait inside the kernel has a limit: should one run out, the rows that its block works on come
 * out as NaN, and the kernel ends.
 * The workspace (256-byte aligned) holds per-call scratch, needs no initialisation and must not be
 * used by two calls that may run at the same time.
 */
spec_status_t spec_paged_attention(const spec_heads_t* q, const spec_heads_t* out, int32_t q_heads,
                                   const spec_kv_cache_t* cache, const spec_decode_batch_t* batch,
                                   const int64_t* mask, float scale, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * spec_paged_attention with two things more, each of which may be NULL:
 *   scales   page scales of an E4M3 cache (layer 0; cache->k_scale and v_scale are NULL).  A row that attends to a slot
 *            whose page's scale does not count comes out as NaN.  A page outside the pool has scale 1;
 *   lse      [B, T, q_heads] float: log sum_s exp(scale * q . K_s) of every row, -inf for rows past T_b and rows that
 *            attend to nothing, NaN where a wait ran out before it was known.  The sum is in fp32, of weights before
 *            their rounding.
 */
spec_status_t spec_paged_attention_ex(const spec_heads_t* q, const spec_heads_t* out, int32_t q_heads,
                                      const spec_kv_cache_t* cache, const spec_kv_page_scales_t* scales,
                                      const spec_decode_batch_t* batch, const int64_t* mask, float scale, float* lse,
                                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * Move the accepted branch of a verified tree up behind the context, in every layer, K and V:
 *   slot ctx_len[b] + i  <-  slot ctx_len[b] + path[b, i]   for i < n_keep[b].
 *   path [B, max_keep] int32: the kept new tokens' indices, strictly increasing from >= 0;
 *   n_keep [B] int32 in [0, max_keep] (clamped).  batch->T and batch->t_per_row are not used.
 * Entries keep their positions' rotation (a tree's tokens were appended at theirs).  Moves whose
 * slots or pages lie outside the table or the pool are left out.
 */
spec_status_t spec_kv_keep(const spec_kv_cache_t* cache, const spec_decode_batch_t* batch,
                           const int32_t* path, const int32_t* n_keep, int32_t max_keep, void* stream);

/*
 * spec_kv_keep with two things more, each of which may be NULL:
 *   scales   page scales of an E4M3 cache.  A page that entries move into takes the scale max(its own, need(their
 *            values)); where it grows, the codes of its other slots < ctx_len[b] + n_keep[b] become round(code * old / new)
 *            (what lies behind them is left as it is).  max_keep <= SPEC_MAX_NEW;
 *   record   weights and positions that move with the entries.
 */
spec_status_t spec_kv_keep_ex(const spec_kv_cache_t* cache, const spec_kv_page_scales_t* scales,
                              const spec_kv_record_t* record, const spec_decode_batch_t* batch, const int32_t* path,
                              const int32_t* n_keep, int32_t max_keep, void* stream);

/*
 * Add up the attention weight that the new tokens of a step give every entry of layer 0 of the cache:
 *   weight[s, h] = (s < ctx_len[b] ? weight[s, h] : 0) + sum over the rows (t, i), i a q head of h's group, that attend to s
 *                  of exp(scale * q[b, t, i] . K_s - lse[b, t, i])
 * for the context's slots and the T_b new tokens', whose positions are recorded too (record->position may be NULL).  Who
 * attends to what, q, cache (v is not used), scales, batch and mask are as for spec_paged_attention_ex, and lse is what it
 * gave; a row whose lse is +inf or -inf has no part, NaN makes NaN of what the row attends to.  So that rejected drafts do not
 * count, a caller that has kept q and lse calls after the verdict, with the accepted tokens of a chain as t_per_row, or with the
 * lse of a tree's other rows set to +inf.
 * positions [B, T] int32 or NULL: ctx_len[b] + t.  Slots whose page lies outside the table or the pool are left out.
 * Two requests must not share a page.  Scores, weights and sums are fp32, queries over an E4M3 cache those that the attention takes
 * (within 2^-21 of a row's largest element).  Each wait inside the kernel has a limit, as for
 * spec_paged_attention: should one run out, weights that its block works on come out as NaN.
 */
spec_status_t spec_kv_weigh(const spec_heads_t* q, int32_t q_heads, const spec_kv_cache_t* cache,
                            const spec_kv_page_scales_t* scales, const spec_decode_batch_t* batch, const int64_t* mask,
                            float scale, const float* lse, const spec_kv_record_t* record, const int32_t* positions,
                            void* stream);

/*
 * Pick, for every layer, request and head, the m = min(ctx_len[b], budget[b]) entries of its context that stay:
 * those of the largest weight, where the lowest slot wins a tie.  Entries at a position < first, or, where recent > 0, at one
 * >= seen[b] - recent, count as of infinite weight, NaN as of -infinity, and those in pages outside the pool too.
 *   target [layers, B, heads, max_moves] int32: the slots < m that do not stay, in ascending order;
 *   source, likewise: the slots >= m that do, in ascending order.  There are as many of each: moves [layers, B, heads],
 *   at most half of the page table's slots, and max_moves is that half at least.  Elements past them are not written;
 *   new_len [B]: m;  budget [B] int32 (a negative one counts as 0);  seen [B] int32: tokens so far, NULL: ctx_len.
 *   new_len may be ctx_len, budget or seen itself, which it then replaces (SPEC_ERR_INVALID_ARG where it overlaps one otherwise).
 *   record->position may be NULL where first and recent are 0; weight and position are 16-byte aligned and layer_stride a
 *   multiple of 4.  batch->T and t_per_row are not used.
 */
spec_status_t spec_kv_select(const spec_kv_record_t* record, const spec_decode_batch_t* batch, const int32_t* budget,
                             const int32_t* seen, int32_t first, int32_t recent, int32_t* source, int32_t* target,
                             int32_t max_moves, int32_t* moves, int32_t* new_len, void* stream);

/*
 * Move entries of every layer and head within their request, keys, values and what `record` holds:
 *   slot target[l, b, h, i]  <-  slot source[l, b, h, i]   for i < moves[l, b, h] (clamped into [0, max_moves]).
 * The lists are spec_kv_select's, or others in ascending order with every target < batch->ctx_len[b] <= every source: ctx_len is
 * the context that the moves leave (new_len).  scales (or NULL): as for spec_kv_keep_ex; the codes that a growing scale
 * changes are those of the page's other slots < ctx_len[b].  Entries keep their positions' rotation, so the next tokens need their
 * positions given.  Moves whose slots or pages lie outside the table or the pool, or on the wrong side of ctx_len[b], are left out.
 * record may be NULL.  batch->T and t_per_row are not used.  Two requests must not share a page.
 */
spec_status_t spec_kv_move(const spec_kv_cache_t* cache, const spec_kv_page_scales_t* scales,
                           const spec_kv_record_t* record, const spec_decode_batch_t* batch, const int32_t* source,
                           const int32_t* target, const int32_t* moves, int32_t max_moves, void* stream);

/*
 * What shapes a batch's logits; every pointer is device memory and NULL leaves its part out.
 *   history [B, history_stride] int32, history_len [B]: the request's tokens so far; the first
 *       prompt_len[b] of them (NULL: none) are its prompt, the others its output.  Ids outside
 *       [0, V) are skipped, lengths are clamped into [0, history_stride];
 *   draft [B, T-1] int32: at position t the drafts before t count as output too;
 *   t_per_row [B] int32: rows past T_b are neither read nor written;
 *   repetition, presence, frequency [B] float (repetition in [2^-126, 2^126]);
 *   bias_ids [B, bias_n] int32, bias [B, bias_n] float: added to the logit of the id (an id
 *       outside [0, V) is skipped; of two entries with one id the later holds);
 *   mask [B, T, ceil(V / 32)] int32: token v is allowed where bit v % 32 of word v / 32 is set.
 */
typedef struct {
  const int32_t* history;
  const int32_t* history_len;
  const int32_t* prompt_len;
  const int32_t* draft;
  const int32_t* t_per_row;
  const float* repetition;
  const float* presence;
  const float* frequency;
  const int32_t* bias_ids;
  const float* bias;
  const int32_t* mask;
  int32_t history_stride, bias_n;
} spec_logit_rules_t;

/*
 * out[b, t, v] from logits[b, t, v] ([B, T, V] of dtype; out may be logits itself), each step in fp32 (a
 * logit or quotient outside 2^+-60 is divided to within 2 units in the last place); c = times v is among the output tokens and the drafts before t:
 *   z > 0 ? z / repetition : z * repetition   where v is in the prompt or c > 0;
 *   z - frequency * c - presence * (c > 0);
 *   z + bias;   -inf where the mask forbids v (whatever the logit was).
 * A row whose mask allows nothing comes out as -inf throughout.
 */
spec_status_t spec_process_logits(const void* logits, void* out, const spec_logit_rules_t* rules, int32_t B,
                                  int32_t T, int32_t V, spec_dtype_t dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_DECODE_H_ */

/*
 * tm_kvb.h -- C ABI of the paged 8-bit KV cache with one scale per block of
 * tokens and head (GB300, sm_103a): append (with position rotation), attention
 * (causal, or of a tree of drafts), accepted drafts, eviction.
 *
 * A page (block) holds T tokens of one sequence for every KV head:
 *   codes  k, v   [pages][Hkv][T][D], one byte each: int8 (-127..127) or e4m3
 *   scales ks, vs [pages][Hkv], fp32, 2^-30 or more, as the append and the
 *          eviction write them;  value = code * scale.  (A page of zero codes may
 *          have scale 0.  A smaller value scale is read as 2^-30; what a negative
 *          one gives is not defined.)
 * Token j of a sequence lives in slot j % T of page table[j / T].  The cache
 * of tm_w4a16.h (tm_kv_*) is dense, with a scale and a zero per token and head;
 * this one is for caches that grow, shrink and share pages.  Several sequences
 * may name a page that a call only reads; see the append and the eviction for
 * the pages that they write.
 *
 * Conventions are those of tm_w4a16.h: device pointers of the current device,
 * nothing throws, no call allocates or synchronises, every call is
 * asynchronous on `stream` (a cudaStream_t; NULL = the legacy default stream)
 * and can be captured into a CUDA graph.
 *
 * Table entries outside 0 .. pages-1 are holes: their tokens take no part in
 * attention, are not written by the append, and are the first to go in an
 * eviction.  No entry, length or row index makes a kernel leave the buffers
 * that the call names.
 */
#ifndef TM_KVB_H
#define TM_KVB_H

#include "tm_w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { TM_KVB_INT8 = 0, TM_KVB_E4M3 = 1 }; /* tm_kvb_cache.format */
enum { TM_KVB_F16 = 0, TM_KVB_BF16 = 1 };  /* the dtype arguments: Q, K, V and the output */

/* The pages of one layer. */
typedef struct {
  void* k;   /* codes, 16-byte aligned */
  void* v;
  float* ks; /* scales, 4-byte aligned */
  float* vs;
  int pages;  /* >= 0 */
  int Hkv;    /* 1 .. 65535 */
  int T;      /* tokens per page: 16, 32, 64 or 128 */
  int D;      /* head dimension: 64 or 128 */
  int format; /* TM_KVB_INT8 or TM_KVB_E4M3 */
} tm_kvb_cache;

/* The sequences of one step (the same for every layer). */
typedef struct {
  const int* table;   /* device int32 [B][table_stride]: page of each block of T tokens */
  const int* kv_len;  /* device int32 [B]: tokens of each sequence, this step's new ones included */
  const int* q_start; /* device int32 [B + 1]: sequence b's new tokens are rows q_start[b] .. q_start[b+1]-1
                         of Q, K and V, and the last of its kv_len[b] tokens.  NULL: one new token each */
  int B;              /* 0 .. 65535 */
  int table_stride;   /* entries per row of the table */
  int max_q;          /* host bound of the new tokens of a sequence: rows past it are not computed */
  int max_len;        /* host bound of kv_len, used for planning and the workspace; longer sequences are
                         read up to it.  0: table_stride * T.  The attention cuts all sequences into slices
                         of one size by it, so that a bound far above the lengths leaves SMs idle */
  long long rows;     /* rows of Q, K and V (q_start is clamped to 0 .. rows); B where q_start is NULL */
} tm_kvb_batch;

/*
 * Quantise the new tokens' keys and values into their pages.  For each page
 * that new tokens fall into, each head, K and V apart, in IEEE binary32 with
 * round-to-nearest-even at each step:
 *   a = max |x| over the new tokens in the page (NaN counts as 0, an infinity
 *       as the type's largest finite value)
 *   need = max(a * r, 2^-30),  r = 1 / 127 (int8) or 1 / 448 (e4m3), rounded once
 *   s = max(s_old, need) if the page holds earlier tokens of the sequence,
 *       else need
 *   new codes = Q(x / s); where s > s_old the page's earlier codes become
 *       Q((c * s_old) / s), so that a page keeps one scale as it fills
 * Q rounds to the nearest code, ties to even, and saturates.  Slots past the
 * sequence's length keep their bytes.
 *   Kn, Vn : device, dtype [rows][Hkv][D], token strides k_stride, v_stride in
 *            elements (multiples of 8, >= Hkv * D: slices of one fused projection are
 *            fine), 16-byte aligned
 *   w      : NULL, or the token weights fp32 [B][Hkv][w_stride]: the new
 *            tokens' entries are set to 0
 * A page written by a call belongs to one sequence of it.  One launch.
 */
tm_status tm_kvb_append(const tm_kvb_cache* cache, const tm_kvb_batch* batch, const void* Kn, long long k_stride,
                        const void* Vn, long long v_stride, int dtype, float* w, long long w_stride, void* stream);

/* Rotation by position. */
typedef struct {
  const float* table; /* device fp32 [positions][dims], 16-byte aligned: a position's dims / 2 cosines, then its sines */
  int positions;      /* >= 1 */
  int dims;           /* leading dimensions of a head that rotate: a multiple of 16, 16 .. D */
  int interleaved;    /* pairs (i, i + dims / 2), or, where not 0, neighbours (2 i, 2 i + 1); i: the pair's angle */
  const int* pos;     /* device int32 [rows]: each row's position; NULL: its slot.  Clamped to 0 .. positions - 1 */
} tm_kvb_rope;

/*
 * tm_kvb_append with the keys rotated on the way, and the queries beside them:
 *   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin
 * for every pair (x1, x2) of the rotating dimensions, in binary32 with each
 * product and each sum rounded.  Rotated keys are quantised as the append does
 * from binary32 (NaN that the rotation gives counts as 0, an infinity as the
 * largest finite binary32), values as they are; rotated queries
 * are rounded once to their type (no value is replaced).
 *   Q, q_out : device, dtype [rows][Hq][D], token strides q_stride, qo_stride in elements
 *           (multiples of 8, >= Hq * D), 16-byte aligned; Hkv divides Hq.  q_out may be Q
 *           (with its stride, and each row in one sequence at most), else it overlaps no input.  Rows of no
 *           sequence, and past max_q of one, are left as they are.  NULL, NULL: keys and values alone (Hq and the
 *           strides are then not read)
 * The rest as in tm_kvb_append.  One launch.
 */
tm_status tm_kvb_append_rope(const tm_kvb_cache* cache, const tm_kvb_batch* batch, const void* Kn, long long k_stride,
                             const void* Vn, long long v_stride, const void* Q, long long q_stride, int Hq,
                             void* q_out, long long qo_stride, const tm_kvb_rope* rope, int dtype, float* w,
                             long long w_stride, void* stream);

/* Bytes of device workspace that tm_kvb_attention needs for these shapes (only the
 * host fields of cache and batch are read); weights != 0: with w_out. */
tm_status tm_kvb_attention_workspace(const tm_kvb_cache* cache, const tm_kvb_batch* batch, int Hq, int weights,
                                     size_t* bytes);
/* The same for tm_kvb_attention_tree. */
tm_status tm_kvb_attention_tree_workspace(const tm_kvb_cache* cache, const tm_kvb_batch* batch, int Hq, int weights,
                                          size_t* bytes);

/*
 * Causal attention of the new tokens over the cache (their own keys and
 * values included: append first).  Row i of sequence b, query head h:
 *   s_j = scale * q . k~_j,  j = 0 .. kv_len[b] - n_b + i, holes left out
 *   p = softmax(s),  out = sum_j p_j v~_j,  lse = log sum_j exp(s_j)
 * with KV head h / (Hq / Hkv).  A row that sees nothing gives out = 0 and
 * lse = -inf.  Any Hq that Hkv divides.
 *   Q     : device, dtype [rows][Hq][D], token stride q_stride in elements (a
 *           multiple of 8, >= Hq * D), 16-byte aligned
 *   scale : of the scores, finite; 0 = 1 / sqrt(D)
 *   out   : device, dtype [rows][Hq][D], contiguous, 16-byte aligned
 *   lse   : NULL, or device fp32 [rows][Hq]
 *   w_out : NULL, or the weight that each token drew, device fp32
 *           [B][Hkv][w_stride]: w_out = w_in + the sum of p over the step's
 *           rows and the KV head's query heads.  w_in NULL counts as 0, and
 *           w_out may be w_in.  Summed in a fixed order.  w_stride >= max_len.
 *           Written where the step has no rows, too.
 *   workspace: device, at least tm_kvb_attention_workspace bytes, 16-byte
 *           aligned (may be NULL where that is 0); calls that can overlap on the GPU need
 *           one each
 * fp16 queries are exact in the products.  bf16 rows carry a power of two into
 * fp16: elements of at least 2^-31 of the row's largest are exact, smaller ones
 * are off by at most 2^-39 of it.  The scores, the softmax statistics and all
 * sums are fp32; p is rounded once to fp16 for its product with the codes (the
 * type that holds both formats' codes exactly), and the sum that divides takes
 * it unrounded.
 */
tm_status tm_kvb_attention(const tm_kvb_cache* cache, const tm_kvb_batch* batch, const void* Q, long long q_stride,
                           int Hq, int dtype, float scale, void* out, float* lse, const float* w_in, float* w_out,
                           long long w_stride, void* workspace, size_t workspace_bytes, void* stream);

/*
 * tm_kvb_attention for new tokens that are a tree (or any graph) of drafts: row
 * i of a sequence with n new tokens sees the kv_len - n tokens before them, and
 * of the new ones those that its mask names,
 *   j < kv_len - n, or bit (k % 32) of tree[row][k / 32] set, k = j - (kv_len - n)
 * -- a node's ancestors and itself, where the rows are a tree's nodes.  Any mask is
 * valid; a row that sees nothing gives out = 0 and lse = -inf.
 *   tree  : device, 32-bit words [rows][tree_stride], 4-byte aligned,
 *           tree_stride >= ceil(max_q / 32), which is how many words of a row are read: new
 *           tokens past them are not seen, and bits past the new tokens say nothing
 *   workspace: device, tm_kvb_attention_tree_workspace bytes, 16-byte aligned (may be NULL where that is 0).  With
 *           fewer the sequences are cut into fewer slices, which can be slower and sums in another order; what
 *           tm_kvb_attention_workspace says for the same step is always enough
 * The rest as in tm_kvb_attention.
 */
tm_status tm_kvb_attention_tree(const tm_kvb_cache* cache, const tm_kvb_batch* batch, const void* Q,
                                long long q_stride, int Hq, int dtype, float scale, const uint32_t* tree,
                                long long tree_stride, void* out, float* lse, const float* w_in, float* w_out,
                                long long w_stride, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Keep a path through the new tokens of each sequence: new token path[b][i], i <
 * count[b], moves to slot old + i, old = kv_len[b] - n.  A path is strictly ascending
 * (a tree's nodes come after their parents); it ends at its first entry that is
 * not above the one before it, or no new token (0 .. n - 1).
 * A token that stays in its page keeps its codes.  One that comes from another
 * page is a new value x = c * s_src of the page, by the rule of tm_kvb_append: the page's scale grows
 * to what these need, and becomes that where the page keeps no token (of before, or of the path).
 * Slots from old + count on keep what they hold.  A hole's tokens move as zeros,
 * and what falls into a hole is dropped.
 *   path   : device int32 [B][path_stride] (not read, and may be NULL, where path_stride is 0)
 *   count  : device int32 [B] (clamped to 0 .. path_stride)
 *   w      : NULL, or the token weights fp32 [B][Hkv][w_stride]: they move along, those of the
 *            new tokens that are not kept become 0
 *   new_len: device int32 [B]: old + count; kv_len where the sequence has no new token, or more of them than
 *            tokens (such a sequence is left as it is).  Not kv_len itself
 * A page of a sequence's new tokens belongs to that sequence alone.  Of the batch, max_q, max_len and (with q_start)
 * rows are not read.  One launch.
 */
tm_status tm_kvb_accept(const tm_kvb_cache* cache, const tm_kvb_batch* batch, const int* path, int path_stride,
                        const int* count, float* w, long long w_stride, int* new_len, void* stream);

/*
 * Cut every sequence to `budget` tokens per KV head: the first `first`, the
 * last `recent`, and of the rest those with the largest weight w (ties: the
 * lowest index; NaN and holes go first).  A sequence of at most `budget`
 * tokens keeps all of them.  Each head keeps its own tokens; they move, in
 * their order, to slots 0, 1, ... of the pages of dst_table:
 *   s = max(max |c * s_old| * r, 2^-30) over a new page's tokens, r as in the append,
 *   codes Q((c * s_old) / s); its slots past the last token become 0.
 *   A page whose tokens all keep their slots keeps its codes and its scale.
 *   dst_table: device int32 [B][dst_stride], dst_stride >= ceil(budget / T).
 *            May be the batch's own table (the eviction then runs in place): each page
 *            that it names then belongs to one sequence of the call.  A table with pages
 *            that sequences share goes into fresh ones; apart from a page that keeps its
 *            place, no destination page may be one that the call reads, or be named twice.
 *   w      : device fp32 [B][Hkv][w_stride], w_stride >= max_len
 *   w_out  : device fp32 [B][Hkv][w_out_stride], w_out_stride >= budget: the
 *            kept tokens' weights, 0 up to `budget` where fewer are kept.  May be w
 *            (with w_out_stride == w_stride)
 *   kept   : device int32 [B][Hkv][budget], the kept tokens' indices, then -1
 *   new_len: device int32 [B], min(kv_len, budget); not kv_len itself
 * Of the batch, table, kv_len, B, table_stride and max_len are read.
 * budget >= 1, first, recent >= 0, first + recent <= budget.  One launch.
 */
tm_status tm_kvb_evict(const tm_kvb_cache* cache, const tm_kvb_batch* batch, const int* dst_table, int dst_stride,
                       const float* w, long long w_stride, float* w_out, long long w_out_stride, int budget, int first,
                       int recent, int* kept, int* new_len, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TM_KVB_H */

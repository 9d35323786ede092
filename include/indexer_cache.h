/*
 * libindexer_bwd, third header -- the cache that a model with an indexer
 * answers from: keys and values (or an indexer's keys alone) in 8 bits, in
 * pages, written as tokens come, read back for the indexer's forward pass, and
 * the attention over all of a sequence's tokens or over those that the indexer
 * selected. Status codes and streams are those of indexer_bwd.h, the rules for
 * pointers and element types those of indexer_train.h.
 *
 * A cache is [pages, heads, page, dim] codes, contiguous and 16-byte aligned,
 * with fp32 scales [pages, heads]: a block (one head's tokens of one page) has
 * one scale, a code stands for code * scale. page is 16, 32, 64, 128 or 256
 * tokens, dim a multiple of 16 up to IBWD_MAX_HEAD_DIM.
 *
 * A sequence's position t is slot t % page of its page table[t / page].
 * Position numbers and lengths are int32. `lens` counts a sequence's tokens
 * with those that the call brings: of n packed tokens the i-th is position
 * lens - n + i.
 *
 * What the device memory holds cannot be refused by the host, and is never
 * followed out of bounds: a page number outside [0, pages) holds nothing (not
 * written, read as 0, not attended to), a length is cut to what the page table
 * has room for, negative positions and lengths are no tokens, offsets are cut to
 * [0, tokens]. Offsets that fall, and a page that two sequences are written to in one call,
 * leave those tokens' results undefined.
 */
#ifndef INDEXER_CACHE_H
#define INDEXER_CACHE_H

#include "indexer_train.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { IBWD_E4M3 = 0, IBWD_INT8 = 1 } ibwd_code;

typedef struct ibwd_cache {
  void* codes;  /* int8, or e4m3: 4 exponent and 3 mantissa bits, largest 448, NaN, no infinity */
  float* scale;
} ibwd_cache;

/* The sequences of a call, and the shape of its caches. */
typedef struct ibwd_sequences {
  const int32_t* table;  /* [batch, table_width], table_stride elements between sequences */
  int64_t table_stride;
  int table_width;
  int batch;             /* up to 2^20 */
  const int32_t* lens;   /* [batch] */
  const int32_t* cu;     /* [batch + 1] offsets of the sequences' packed tokens; NULL: one token each */
  int64_t tokens;        /* rows of the packed tokens, at most 2^27; those before cu[0] and from cu[batch] on are nobody's */
  int64_t pages;
  int heads, page, dim;
  int code;              /* ibwd_code */
} ibwd_sequences;

/*
 * Writes the packed tokens' keys and values. The scale of a block is the least
 * power of two 2^e, -126 <= e <= 120, with |x| <= M 2^e for the finite x that
 * the block was given (M = 448 or 127), and never falls while the page fills: a
 * token that raises it has the older tokens' codes rounded anew. A page whose
 * slot 0 the call writes begins anew. Codes are rounded to nearest even;
 * infinities become the largest code, as in int8 do finite values beyond
 * 127 * 2^120 (1.7e38), which no scale holds; NaN is e4m3's NaN, and in int8
 * makes the block's scale NaN until the page begins anew.
 *   k, v     type [tokens, heads, dim], unit stride along dim, `token` and `head` elements between
 *            tokens and heads; v, and v_cache with it, NULL for a cache of keys alone
 */
IBWD_API int ibwd_cache_write(const void* k, int64_t k_token, int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                              int type, const ibwd_cache* k_cache, const ibwd_cache* v_cache, const ibwd_sequences* seqs,
                              void* stream);

/* Reads positions [0, length) of every sequence: out, of any element type, is
 * [batch, length, heads, dim], contiguous and 16-byte aligned, and 0 from the
 * sequence's end on. cu and tokens are not looked at. */
IBWD_API int ibwd_cache_read(const ibwd_cache* cache, const ibwd_sequences* seqs, void* out, int type, int length,
                             void* stream);

/* Bytes of device workspace of ibwd_cache_attention; 0 for unsupported arguments. */
IBWD_API size_t ibwd_cache_attention_workspace_size(int dim);

/*
 * Attention of the packed tokens' queries over the cache. Query head h reads
 * KV head h / group. Token i of a sequence's n sees the positions up to its
 * own, lens - n + i, and with `select` those of them that its row lists (ids
 * outside are padding; one listed twice counts twice):
 *   s_t = scale * q . k_t,   p = softmax(s),   out = sum p_t v_t,   lse = log sum exp(s_t)
 * A token that sees nothing has out 0 and lse -inf. NaN and what is invisible
 * stay out of each other's way: an invisible position's NaN reaches nothing.
 * Statistics and sums are fp32; a query is taken in fp16 relative to its
 * largest entry, a probability in fp16 relative to the largest weight (of
 * its own or of the value it weighs), each with 11 bits.
 * Rows of tokens before the first sequence and behind the last are left as they were.
 *   q       type [tokens, heads * group, dim], IBWD_BF16 or IBWD_F16, unit stride along dim
 *   out     type [tokens, heads * group, dim], contiguous; 16-byte aligned
 *   lse     fp32 [tokens, heads * group], or NULL
 *   select  int32 [tokens, kept], or NULL; dim 64, 128 or 256; scale finite
 *           tokens * group up to 2^30, heads * group up to 2^31 - 1; calls that may have more than
 *           300 * (2^31 - 1) tiles of 16 rows and 64 positions (as the table is wide, or the list long)
 *           are unsupported
 *   workspace  at least ibwd_cache_attention_workspace_size bytes, 16-byte aligned
 */
IBWD_API int ibwd_cache_attention(const void* q, int64_t q_token, int64_t q_head, int type, int group,
                                  const ibwd_cache* k_cache, const ibwd_cache* v_cache, const ibwd_sequences* seqs,
                                  const int32_t* select, int kept, float scale, void* out, float* lse, void* workspace,
                                  size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* INDEXER_CACHE_H */

/*
 * csa_draft.h — C ABI of the operators of a serving step with drafted tokens over the latent
 * cache (csa_latent.h): norms of queries and keys with the position rotation, new latents
 * normed, rotated and stored in the paged cache, attention of drafted tokens (a tree, or a
 * chain; one drafted token is an ordinary decode row) over the cache, and the accepted
 * drafts' records moved to the front of the drafted ones. Same library, same conventions:
 * every pointer is device memory owned by the caller, nothing is allocated, freed or
 * synchronised, all work is enqueued on `stream`, which like the pointers belongs to the
 * calling thread's current device, calls are re-entrant and capturable as long as their
 * workspaces do not overlap while in flight, host-detectable errors launch nothing, and
 * data-dependent errors OR a CSA_DEV_* bit into *dev_status (when given) and leave the
 * offending record, row or request out.
 */
#ifndef CSA_DRAFT_H
#define CSA_DRAFT_H

#include "csa_latent.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CSA_DRAFT_ABI_VERSION 1

#define CSA_ROTATE_MAX_DIM 1024   /* values of a head                                    */
#define CSA_ROTATE_MAX_ROPE 256   /* rotated values of a head                            */
#define CSA_ROTATE_MAX_HEADS 65536 /* heads of a tensor                                   */
#define CSA_DRAFT_MAX_WORDS 16    /* 64-bit words of a draft's mask                      */
#define CSA_DRAFT_MAX_REQ 65536   /* requests of one csa_draft_attend call               */
#define CSA_COMMIT_MAX_REQ 16384  /* requests of one csa_draft_commit call               */

#define CSA_PAIRS_ADJACENT 0 /* pairs of values (2 j, 2 j + 1)             */
#define CSA_PAIRS_HALVES 1   /* pairs of values (j, j + rope_dim / 2)      */

int32_t csa_draft_abi_version(void);

/*
 * The position rotation: pair j of a row at position p becomes
 *   (a, b) -> scale * (a cos t - b sin t, b cos t + a sin t),  t = p * freq[j]
 * with the product taken exactly: the angle's turns are counted in 2^-63, so that far positions
 * lose nothing (p below 2^31, |freq| up to 2^10 radians a token).
 */
typedef struct csa_rotation {
  const float* freq;   /* [rope_dim / 2] radians a token, finite; may be NULL where rope_dim is 0 */
  int32_t rope_dim;
  int32_t pairing;     /* CSA_PAIRS_ADJACENT or CSA_PAIRS_HALVES */
  float scale;         /* of both outputs; finite, 1 where there is none */
  int32_t reserved0;   /* must be 0 */
} csa_rotation;

/*
 * Norm and rotation of every head's values, of queries and of keys in one pass:
 *   y_i = x_i / sqrt(mean(x^2) + eps) * weight_i   (where norm is 1, else y = x)
 *   out = y, its last rope_dim values (its first ones with rope_first) rotated to the row's position
 * computed in fp32 (the squares of a head in fp64 where they leave fp32's range), rounded once; where x_i / sqrt(..)
 * is below 2^-126 it is held to 2^-150, as fp32's subnormal numbers are, before its weight. NaN and infinities go
 * through the formula, within their own head. Rows whose position is -1 are left as they are.
 *
 * csa_heads: x [n, heads, dim] and out of the same shape; dim a multiple of 8, rope_dim .. CSA_ROTATE_MAX_DIM; up to
 * CSA_ROTATE_MAX_HEADS heads, 0: none (nothing of it is looked at). The strides are in elements, multiples of 16
 * bytes; the addresses are on 16 bytes. out may be x itself, with the same strides and type (the operation is then in
 * place), but must not overlap it, or the other tensor, in another way. weight [dim] fp32, on 16 bytes, or NULL (all 1).
 * rope_dim: 0, or a multiple of 16 up to CSA_ROTATE_MAX_ROPE.
 * pos [n] int32; NULL only where rope_dim is 0 (every row is there then). Device errors: a position below -1
 * CSA_DEV_LEN_OOB (the row is left as it is).
 */
typedef struct csa_heads {
  const void* x;
  void* out;
  const float* weight;
  int64_t x_row_stride, x_head_stride;
  int64_t out_row_stride, out_head_stride;
  int32_t heads;
  int32_t dim;
  int32_t norm;        /* 0 or 1 */
  int32_t reserved0;   /* must be 0 */
} csa_heads;

typedef struct csa_rotate_args {
  csa_heads q, k;
  int64_t n;
  const int32_t* pos;
  csa_rotation rotation;
  int32_t dtype;       /* of both x: CSA_KEYS_F32 or CSA_KEYS_BF16 */
  int32_t out_dtype;   /* of both out */
  int32_t rope_first;  /* 0 or 1 */
  float eps;           /* finite, at least 0 */
  int32_t* dev_status;
} csa_rotate_args;

csa_status csa_head_norm_rotate(const csa_rotate_args* args, void* stream);

/*
 * csa_latent_write with the norm and the rotation on the way: row i of x [n, 512 + rope_dim] becomes the
 * record at slot slots[i] (-1 skips the row), its 512 latent values normed as above (where norm is 1), its rope
 * values rotated to position pos[i], both rounded to the record's format from the result in fp32. In MXFP4 the
 * codes and scales are those of the exact norm: a value next to a border between two codes is decided in fp64.
 * Rows must target distinct records. Device errors (that row is not written): a slot outside the cache
 * CSA_DEV_PAGE_OOB; a position below 0 CSA_DEV_LEN_OOB; a result that is not finite CSA_DEV_RANGE.
 * rotation.rope_dim is the cache's; pos may be NULL where it is 0.
 */
typedef struct csa_append_args {
  csa_latent_cache cache;
  const void* x;             /* 16-byte aligned; x_stride bytes a multiple of 16 */
  int64_t x_stride;          /* elements between rows, >= 512 + rope_dim */
  int32_t dtype;             /* CSA_KEYS_F32 or CSA_KEYS_BF16 */
  int32_t norm;              /* 0 or 1 */
  int64_t n;
  const int64_t* slots;
  const int32_t* pos;
  csa_rotation rotation;
  const float* weight;       /* [512] fp32, 16-byte aligned, or NULL: all 1 */
  float eps;                 /* finite, at least 0 */
  int32_t reserved0;         /* must be 0 */
  int32_t* dev_status;
} csa_append_args;

csa_status csa_latent_append(const csa_append_args* args, void* stream);

/*
 * Latent attention (absorbed form, see csa_latent_attend) of drafted tokens. Request r has base_len[r] records of
 * history and the drafts row_start[r] .. row_start[r + 1]; draft j's query row is row_start[r] + j and its record
 * is at position base_len[r] + j of the same page table row (csa_build_tables with old_len = base_len and the drafts as new
 * records makes these tables). A draft's row sees the history and, of its request's drafts,
 *   with mask     those i whose bit i % 64 of word i / 64 of its mask is set (drafts past the words are not seen), or
 *   without       those i <= j (a chain).
 * (One draft a request may go to csa_latent_attend as well, the faster one up to 64 heads and for few requests.)
 * A mask may leave out the draft itself, and all drafts. A row that sees nothing gets out 0 and lse -infinity. What
 * records hold that a row does not see (NaN, infinities) does not matter to it; a record that it sees should be finite. (A draft's
 * whose score becomes -infinity is as one that is not seen.)
 *
 * q          [num_q, num_heads, 512 + rope_dim] bf16, 16-byte aligned, the strides in elements
 *            and multiples of 8; num_heads 1 .. CSA_LATENT_MAX_HEADS
 * page_table [num_req, pt_stride] int32; num_req up to CSA_DRAFT_MAX_REQ, 64 pt_stride up to 2^31 - 257
 * base_len   [num_req] int32
 * row_start  [num_req + 1] int32; rows of num_q that no request covers are left as they are
 * mask       [num_q, mask_words] 64-bit words, rows mask_stride words apart, or NULL (then mask_words is 0);
 *            mask_words up to CSA_DRAFT_MAX_WORDS
 * scale      above 0, below 2^127; q . c has to stay below 2^127 in magnitude, whatever the scale
 * out        [num_q, num_heads, 512] bf16, contiguous, 16-byte aligned. The softmax is fp32's; its weights are rounded to bf16 where
 *            they meet the values (the tensor cores' operand type), their sum is not.
 * lse        [num_q, num_heads] fp32, or NULL
 * ws         csa_draft_attend_workspace_bytes(args) bytes, 32-byte aligned
 * Device errors: CSA_DEV_LEN_OOB (base_len below 0 or beyond the table: cut to it; drafts beyond the table are not
 * seen; bounds of rows that descend or leave [0, num_q]: that request's rows are left as they are, and rows that two requests claim, as only such
 * bounds can, hold anything), CSA_DEV_PAGE_OOB (the page's
 * records are left out), CSA_DEV_TIMEOUT (an on-chip wait ran past its limit; output invalid).
 */
typedef struct csa_draft_attend_args {
  csa_latent_cache cache;
  const void* q;
  int64_t q_row_stride;
  int64_t q_head_stride;
  int32_t num_q;
  int32_t num_heads;
  const int32_t* page_table; /* [num_req, pt_stride] */
  int32_t num_req;
  int32_t pt_stride;
  const int32_t* base_len;
  const int32_t* row_start;
  const uint64_t* mask;
  int64_t mask_stride;
  int32_t mask_words;
  float scale;
  void* out;
  float* lse;
  int32_t* dev_status;
} csa_draft_attend_args;

/* Host arithmetic on the sizes only; 0 for sizes that the call refuses. */
size_t csa_draft_attend_workspace_bytes(const csa_draft_attend_args* args);

csa_status csa_draft_attend(const csa_draft_attend_args* args, void* ws, size_t ws_bytes, void* stream);

/*
 * The end of a step: of request r's drafts (draft_len[r] of them, behind base_len[r] records) those at
 * path[r][0] < path[r][1] < ... (path_len[r] of them) were accepted. In the caches of every layer (num_layers of
 * them, layer_stride_bytes apart, with one page table) record base_len + path[k] moves to base_len + k;
 *   new_len[r] = base_len[r] + path_len[r]
 * and the pages behind it, table entries ceil(new_len / 64) <= p < ceil((base_len + draft_len) / 64), are listed in
 * freed in the order of the requests: n_freed of them, of which the first `room` are written; the entries of freed
 * behind them become -1. The table itself stays as it is.
 *
 * path [num_req, path_stride] int32 (contiguous: path_stride is its width); base_len, draft_len, path_len, new_len
 * [num_req] int32; freed [room] int32; n_freed [1] int32; num_req 0 .. CSA_COMMIT_MAX_REQ. A page with drafts' records is one
 * entry of one request's table. What the call writes must not overlap what it reads: new_len is not base_len.
 * Device errors: CSA_DEV_LEN_OOB (a length below 0 or beyond the table; path_len above draft_len or the width of
 * path; a path that does not ascend within 0 .. draft_len - 1) and CSA_DEV_PAGE_OOB (a page that is moved from or to, or given
 * back, out of range): such a request is left as it is, new_len = base_len, and none of its pages are listed. CSA_DEV_ROWS:
 * more pages than room.
 */
typedef struct csa_commit_args {
  csa_latent_cache cache;    /* layer 0 */
  int64_t layer_stride_bytes; /* a multiple of 16, at least 64 records; the layers' pages must not overlap */
  int32_t num_layers;
  int32_t num_req;
  const int32_t* page_table; /* [num_req, pt_stride] */
  int32_t pt_stride;
  int32_t path_stride;
  const int32_t* base_len;
  const int32_t* draft_len;
  const int32_t* path;
  const int32_t* path_len;
  int32_t* new_len;
  int32_t* freed;
  int64_t room;
  int32_t* n_freed;
  int32_t* dev_status;
} csa_commit_args;

csa_status csa_draft_commit(const csa_commit_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CSA_DRAFT_H */

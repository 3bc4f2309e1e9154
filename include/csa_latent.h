/*
 * csa_latent.h — C ABI of the operators around the CSA indexer (csa_index.h): block tables
 * built on the GPU, the paged latent cache with its writer and reader, and latent attention
 * in its absorbed form (over the cache, at the indexer's positions or over the whole
 * history) and its expanded form (prompts). Same library, same conventions: every pointer
 * is device memory owned by the caller, nothing is allocated, freed or synchronised, all
 * work is enqueued on `stream`, which like the pointers belongs to the calling thread's current
 * device, calls are re-entrant and capturable as long as their
 * workspaces do not overlap while in flight, host-detectable errors launch nothing, and
 * data-dependent errors OR a CSA_DEV_* bit into *dev_status (when given) and leave the
 * offending record, row or request out.
 *
 * Latent cache: a record is what one token leaves behind for every head, 512 latent values
 * (key and value) and rope_dim (0 or 64) more key values. 64 records a page, pages
 * page_stride_bytes apart (at least 64 records, a multiple of 16; allocator padding is
 * allowed). Record formats:
 *   CSA_LATENT_BF16   512 + rope_dim bf16 values                        (1024 or 1152 bytes)
 *   CSA_LATENT_MXFP4  256 bytes of e2m1 codes of the latent values, element 2j in the low
 *                     nibble of byte j; 16 UE8M0 scale bytes of its 32-value blocks
 *                     (2^(byte - 127)); then the rope values in bf16      (272 or 400 bytes)
 * A slot is physical page * 64 + record.
 */
#ifndef CSA_LATENT_H
#define CSA_LATENT_H

#include "csa_index.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CSA_LATENT_ABI_VERSION 1

#define CSA_LATENT_DIM 512        /* latent values of a record                        */
#define CSA_LATENT_MAX_HEADS 128  /* query heads of csa_latent_attend                  */
#define CSA_TABLES_MAX_REQ 16384  /* requests of one csa_build_tables call             */
#define CSA_PREFILL_NOPE 128      /* expanded key values without rope                  */
#define CSA_PREFILL_ROPE 64       /* expanded key values with rope, shared by the heads */
#define CSA_PREFILL_V 128         /* expanded values                                   */

#define CSA_LATENT_BF16 0
#define CSA_LATENT_MXFP4 1

/* Further bits of *dev_status (csa_index.h lists the others). */
enum {
  CSA_DEV_POOL = 64,  /* the free pages ran out: the missing table entries and slots are -1  */
  CSA_DEV_ROWS = 128  /* more new records than n_rows: the rows past n_rows are left out      */
};

int32_t csa_latent_abi_version(void);

/* Bytes of one record; 0 for an unknown format or a rope_dim other than 0 or 64. */
int64_t csa_latent_record_bytes(int32_t record_format, int32_t rope_dim);

typedef struct csa_latent_cache {
  uint8_t* pages;            /* 16-byte aligned */
  int64_t num_pages;
  int64_t page_stride_bytes;
  int32_t rope_dim;          /* 0 or 64 */
  int32_t record_format;     /* CSA_LATENT_BF16 or CSA_LATENT_MXFP4 */
} csa_latent_cache;

/*
 * Block tables and slot maps of one step, from request lengths. Request r holds old_len[r]
 * records and gets new_len[r] more; the pages it starts are taken from free_pages in request
 * order. With a_r = ceil(old/64), b_r = ceil((old + new)/64), t_r the sum of b - a before r:
 *   page_table[r][p] = free_pages[t_r + p - a_r]     a_r <= p < b_r; other entries are kept
 *   row i = row_start[r] + j, 0 <= j < new_len[r]:
 *     row_req r, row_pos old_len[r] + j, row_len row_pos + 1 (the row's causal bound),
 *     row_slot page_table[r][row_pos / 64] * 64 + row_pos % 64
 * Rows past the last new record get row_req 0, row_pos -1, row_len 0, row_slot -1: an empty
 * query row and a row that csa_latent_write skips, so that a captured graph can keep n_rows.
 * A row stands for a new record. As the indexer's q_req and q_len, row_req and row_len are right
 * where each query token brings one record; where a record stands for several tokens, a query row
 * has to be made for each token by the caller (the slots and sums stay as they are).
 *
 * old_len, new_len  [num_req] int32; num_req 0 .. CSA_TABLES_MAX_REQ
 * page_table        [num_req, pt_stride] int32, in place
 * free_pages        [n_free] int32, the pool's free pages in the order they are handed out
 * row_req, row_pos, row_len [n_rows] int32; row_slot [n_rows] int64
 * row_start         [num_req + 1] int32, running sum of new_len
 * kv_start          [num_req + 1] int32, running sum of old_len + new_len
 * taken             [1] int32, free pages handed out (those that were missing are not counted)
 * Device errors: CSA_DEV_LEN_OOB (a length below 0 or beyond the table: cut to it; a running
 * sum past 2^31 - 1: held there), CSA_DEV_POOL, CSA_DEV_ROWS, CSA_DEV_PAGE_OOB (a row on a page
 * whose entry is negative: slot -1).
 */
typedef struct csa_tables_args {
  const int32_t* old_len;
  const int32_t* new_len;
  int32_t num_req;
  int32_t pt_stride;
  int32_t* page_table;
  const int32_t* free_pages;
  int64_t n_free;
  int64_t n_rows;
  int32_t* row_req;
  int32_t* row_pos;
  int32_t* row_len;
  int64_t* row_slot;
  int32_t* row_start;
  int32_t* kv_start;
  int32_t* taken;
  int32_t* dev_status;
} csa_tables_args;

csa_status csa_build_tables(const csa_tables_args* args, void* stream);

/*
 * Stores row i of x [n, 512 + rope_dim] (fp32 or bf16: CSA_KEYS_F32, CSA_KEYS_BF16; rows
 * x_stride elements apart) as the record at slot slots[i] (int64; -1 skips the row).
 *   bf16   each value rounded to nearest even
 *   MXFP4  per block of 32 latent values: e = max(floor(log2 amax) - 2, -127), scale byte
 *          e + 127 (amax 0: byte 0), code = the e2m1 value nearest to x 2^-e, ties to the even
 *          mantissa, saturating at 6, with x's sign; rope values as in bf16
 * Rows must target distinct records. Device errors (that row is not written): a slot outside
 * the cache CSA_DEV_PAGE_OOB; a non-finite value (after rounding to bf16, where bf16 is stored)
 * CSA_DEV_RANGE.
 */
typedef struct csa_latent_write_args {
  csa_latent_cache cache;
  const void* x;             /* 16-byte aligned; x_stride bytes a multiple of 16 */
  int64_t x_stride;          /* elements between rows, >= 512 + rope_dim */
  int32_t dtype;
  int32_t reserved0;         /* must be 0 */
  int64_t n;
  const int64_t* slots;
  int32_t* dev_status;
} csa_latent_write_args;

csa_status csa_latent_write(const csa_latent_write_args* args, void* stream);

/*
 * Reads histories back: out row kv_start[r] + j = the values of record j of request r, in bf16
 * (the 4-bit values are exact in it), for kv_start[r] + j < min(kv_start[r + 1], n_rows). Rows that
 * no request covers are left as they are. Device errors: a page out of range CSA_DEV_PAGE_OOB
 * (its rows become 0); kv_start descending, negative, or longer than the table CSA_DEV_LEN_OOB
 * (the rows beyond the table become 0).
 */
typedef struct csa_latent_read_args {
  csa_latent_cache cache;
  const int32_t* page_table; /* [num_req, pt_stride] */
  int32_t num_req;
  int32_t pt_stride;
  const int32_t* kv_start;   /* [num_req + 1] */
  int64_t n_rows;
  void* out;                 /* [n_rows, 512 + rope_dim] bf16, 16-byte aligned */
  int32_t* dev_status;
} csa_latent_read_args;

csa_status csa_latent_read(const csa_latent_read_args* args, void* stream);

/*
 * Latent attention, absorbed form: one record c_n is the key (all its values) and the value
 * (its 512 latent values) of every head. For query row b, head h:
 *   s_n = scale * q_bh . c_n,  p = softmax over the row's visible n,  out_bh = sum_n p_n c_n[0:512]
 *   lse_bh = log sum_n exp(s_n)
 * Visible records: positions n < row_len[b] of request row_req[b], or, with idx, the listed
 * ones among them (each as often as it is listed; -1 entries are skipped). A row with no visible
 * record gets out 0 and lse -infinity. What invisible records hold (NaN, infinities) does not
 * matter.
 *
 * q          [num_q, num_heads, 512 + rope_dim] bf16, 16-byte aligned, the strides in elements
 *            and multiples of 8; num_heads 1 .. CSA_LATENT_MAX_HEADS
 * row_req    [num_q] int32, or NULL for row b -> request b
 * row_len    [num_q] int32
 * idx        [num_q, top] int32 rows idx_stride apart, or NULL (then top is 0)
 * scale      above 0, below 2^127; s_n has to stay below 2^126 in magnitude, q . c below 2^127
 * out        [num_q, num_heads, 512] bf16, contiguous, 16-byte aligned
 * lse        [num_q, num_heads] fp32, or NULL
 * ws         csa_latent_attend_workspace_bytes(args) bytes, 16-byte aligned
 * Device errors: CSA_DEV_BAD_REQUEST (the row is empty), CSA_DEV_LEN_OOB (row_len below 0 or
 * beyond the table: cut to it; a position below -1 or not below row_len: left out),
 * CSA_DEV_PAGE_OOB (the page's records are left out), CSA_DEV_TIMEOUT (an on-chip wait ran past
 * its limit; output invalid).
 */
typedef struct csa_latent_attend_args {
  csa_latent_cache cache;
  const void* q;
  int64_t q_row_stride;
  int64_t q_head_stride;
  int32_t num_q;
  int32_t num_heads;
  const int32_t* page_table;
  int32_t num_req;
  int32_t pt_stride;
  const int32_t* row_req;
  const int32_t* row_len;
  const int32_t* idx;
  int64_t idx_stride;
  int32_t top;
  float scale;
  void* out;
  float* lse;
  int32_t* dev_status;
} csa_latent_attend_args;

/* Host arithmetic on the sizes only; 0 for sizes that the call refuses. */
size_t csa_latent_attend_workspace_bytes(const csa_latent_attend_args* args);

csa_status csa_latent_attend(const csa_latent_attend_args* args, void* ws, size_t ws_bytes, void* stream);

/*
 * Latent attention, expanded form: the latents expanded per head into keys k_nope and values v,
 * with one rope key a token for all heads. Request r has the query rows q_start[r] ..
 * q_start[r + 1] and the key rows kv_start[r] .. kv_start[r + 1]; with past = keys - queries,
 *   s_ij = scale * (q_ih[0:128] . k_nope_jh + q_ih[128:192] . k_rope_j)
 *   visible: j <= i + past (causal), or every j of the request
 *   out_ih = sum_j softmax_j(s_ij) v_jh,  lse_ih = log sum_j exp(s_ij)
 * A row that sees no key gets out 0 and lse -infinity. What keys and values of other requests
 * hold does not matter. Within a request a value v_jh that is not finite may reach rows that do
 * not see key j too (as 0 times it); rows that see no key stay 0. s_ij has to stay within 2^30 in magnitude (exponents
 * are differences of rounded products: beyond, a rounding is more than an exponent holds).
 *
 * q        [total_q, num_heads, 192] bf16; k_nope, v [total_k, num_heads, 128] bf16; k_rope
 *          [total_k, 64] bf16: 16-byte aligned, strides in elements and multiples of 8 (k_nope and
 *          v may be halves of one tensor, k_rope a slice of the latents)
 * q_start, kv_start [num_req + 1] int32
 * out      [total_q, num_heads, 128] bf16, contiguous, 16-byte aligned
 * lse      [total_q, num_heads] fp32, or NULL
 * Device errors: CSA_DEV_LEN_OOB (bounds that descend or leave [0, total]: that request's rows
 * are left as they are), CSA_DEV_TIMEOUT.
 */
typedef struct csa_latent_prefill_args {
  const void* q;
  const void* k_nope;
  const void* k_rope;
  const void* v;
  int64_t q_row_stride, q_head_stride;
  int64_t k_row_stride, k_head_stride;
  int64_t rope_row_stride;
  int64_t v_row_stride, v_head_stride;
  int64_t total_q;
  int64_t total_k;
  const int32_t* q_start;
  const int32_t* kv_start;
  int32_t num_req;
  int32_t num_heads;
  int32_t causal;            /* 0 or 1 */
  float scale;               /* above 0, below 2^127 */
  void* out;
  float* lse;
  int32_t* dev_status;
} csa_latent_prefill_args;

csa_status csa_latent_prefill(const csa_latent_prefill_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CSA_LATENT_H */

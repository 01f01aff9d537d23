/*
 * alhr_cache.h -- C ABI of the paged 8-bit key/value cache of libalhr.so.
 *
 * alhr.h reads one contiguous [batch][heads][n][d] block of keys and values: every sequence has
 * the same length and the values take 16 bits. Sequences that are served have lengths of their
 * own and grow token by token. The calls below keep their keys and values in fixed-size blocks of
 * tokens ("pages") at 8 bits a number, with one scale for each block and head, and read them
 * through a block table:
 *   alhr_plan_blocks            block table, slots and row offsets of a step, from the lengths
 *   alhr_store_cache            keys and values of new tokens into their slots
 *   alhr_load_cache             the numbers that given slots hold (the inverse)
 *   alhr_attend_cache           softmax attention over all visible keys of each request
 *   alhr_attend_cache_selected  the same over selected positions, e.g. those of alhr_route
 *
 * Cache layout (row-major, contiguous, device memory; codes 16-byte, scales 4-byte aligned):
 *   k, v             8-bit codes [blocks][heads][block_size][d]
 *   k_scale, v_scale float       [blocks][heads]
 *   A key or value is code * scale of its block and head; scales are finite and not negative.
 *   Codes are int8 in [-127, 127] or e4m3 (4 exponent bits, 3 mantissa bits, no infinities) that
 *   is not NaN, as alhr_store_cache writes them. A NaN in what some row of a request sees may
 *   reach the request's other rows too.
 * A slot is block * block_size + offset (64 bits). Position p of request r lies in block
 * block_table[r][p / block_size] at offset p % block_size.
 *
 * Everything alhr.h says about ownership, streams and errors holds here: the caller owns all
 * memory, nothing is allocated, no state is kept between calls, arguments are checked on the host
 * before anything is launched. Lengths, tables and slots live on the device and may change
 * between replays of a captured graph; what only the device can see is handled as listed, never
 * by an access outside the given arrays, and flagged in *dev_err when it is not NULL.
 */
#ifndef ALHR_CACHE_H
#define ALHR_CACHE_H

#include "alhr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits of *dev_err. */
#define ALHR_DEVERR_CAPACITY  0x10u /* alhr_plan_blocks: tokens were left without a slot       */
#define ALHR_DEVERR_BLOCK     0x20u /* a block number or slot outside the cache was skipped     */
#define ALHR_DEVERR_NONFINITE 0x40u /* alhr_store_cache: an infinity or NaN was stored          */

typedef enum { ALHR_CODE_INT8 = 0, ALHR_CODE_E4M3 = 1 } alhr_code;

/* Types of keys, values and queries. */
typedef enum {
  ALHR_TYPE_BF16 = 0,
  ALHR_TYPE_FP16 = 1,
  ALHR_TYPE_FP32 = 2,
  ALHR_TYPE_INT8 = 3
} alhr_type;

typedef struct {
  void* k;            /* codes, see above                                                     */
  void* v;
  float* k_scale;
  float* v_scale;
  int32_t blocks;     /* >= 1; blocks * heads * block_size < 2^31 (else ALHR_ERR_UNSUPPORTED) */
  int32_t heads;      /* key/value heads, 1 to 65535 (more: ALHR_ERR_UNSUPPORTED)             */
  int32_t block_size; /* 16, 32, 64 or 128 tokens                                             */
  int32_t d;          /* 64 or 128                                                            */
  int32_t code;       /* an alhr_code                                                         */
} alhr_cache;

/*
 * alhr_plan_blocks -- the block table and slots of one step, from the request lengths.
 *
 * Request r has ctx_len[r] tokens in the cache and adds new_len[r]. With bs = block_size, its row
 * of the table holds its blocks in order; ceil(ctx_len / bs) of them are there already. The step
 * needs ceil((ctx_len + new_len) / bs) in all; the missing ones are taken from free_blocks in
 * request order, beginning at entry *free_first:
 *   q_start[r]      sum of new_len before r (requests + 1 entries): the first of r's token rows
 *   block_table     the new entries are written; -1 where the free list has ended
 *   seq_len[r]      ctx_len + new_len, less what found no block
 *   positions[t]    position in its sequence of token row t; -1 for rows behind the last request
 *   slots[t]        its slot; -1 behind the last request, and where there is no block
 *   *free_next      the entry of free_blocks that the next step begins at
 * ALHR_DEVERR_CAPACITY is set, and the tokens go without a slot, where a sequence would pass
 * max_blocks * bs tokens, the free list ends, or there are more than `tokens` token rows (then
 * q_start stops at `tokens`). Negative lengths count as zero; a block number outside
 * [0, blocks) gives slot -1 and sets ALHR_DEVERR_BLOCK.
 *   requests     0 <= requests <= 8192; max_blocks * block_size <= 2^30 (else
 *                ALHR_ERR_UNSUPPORTED)
 *   tokens       length of slots and positions, >= 0
 *   free_count   length of free_blocks, >= 0
 *   block_table  device int32 [requests][max_blocks], updated in place
 *   free_next is not free_first, seq_len neither ctx_len nor new_len (ALHR_ERR_INVALID_ARG).
 */
ALHR_API alhr_status alhr_plan_blocks(int32_t requests, int32_t max_blocks, int32_t block_size,
                                      int32_t blocks, int32_t tokens, int32_t free_count,
                                      const int32_t* ctx_len, const int32_t* new_len,
                                      int32_t* block_table, const int32_t* free_blocks,
                                      const int32_t* free_first, int32_t* q_start,
                                      int32_t* seq_len, int64_t* slots, int32_t* positions,
                                      int32_t* free_next, uint32_t* dev_err, void* stream);

/*
 * alhr_store_cache -- keys and values of `tokens` token rows into their slots.
 *
 * Rows that follow one another into consecutive slots of one block form a run. For every run and
 * head, keys and values apart, with a = the largest |x| of the run's finite numbers and s0 the
 * block's scale (0 if the run begins at offset 0: the block is new):
 *   s    = max(s0, a / full, 2^-100)          full = 127 (int8), 256 (e4m3)
 *   codes of the block's rows before the run: round(code * (s0 / s)), if s > s0
 *   codes of the run:                         round(x / s)
 * all in fp32, to nearest, ties to even, saturated at 127 (int8) and 448 (e4m3). Rows behind the
 * run keep what they hold. 256 is a power of two, so that the scale of a new e4m3 block is exact;
 * 2^-100 keeps 1 / s finite. An infinity is stored saturated, a NaN as 0, both set
 * ALHR_DEVERR_NONFINITE. Rows with slot -1 are not read; another slot outside the cache is
 * skipped and sets ALHR_DEVERR_BLOCK.
 * The slots of one block must be one run, as alhr_plan_blocks writes them: a block that two runs
 * of one call name has unspecified codes and scale afterwards (the rest of the cache is not
 * touched).
 *   K, V      device, tokens x heads rows of d numbers of `type` (bf16, fp16 or fp32), strides
 *             in numbers; base pointers and strides 16-byte aligned, each row contiguous
 *   slots     device int64 [tokens]
 */
ALHR_API alhr_status alhr_store_cache(const alhr_cache* cache, const void* K, const void* V,
                                      int32_t type, int32_t tokens, int64_t k_token_stride,
                                      int64_t k_head_stride, int64_t v_token_stride,
                                      int64_t v_head_stride, const int64_t* slots,
                                      uint32_t* dev_err, void* stream);

/*
 * alhr_load_cache -- code * scale of the given slots, in fp32, rounded once to `type`.
 *   slots  device int64 [tokens]; -1 gives a row of zeros, another slot outside the cache too
 *          (and ALHR_DEVERR_BLOCK). A slot may be named more than once.
 *   K, V   device, [tokens][heads][d] of `type` (bf16, fp16 or fp32), overwritten
 */
ALHR_API alhr_status alhr_load_cache(const alhr_cache* cache, void* K, void* V, int32_t type,
                                     int32_t tokens, const int64_t* slots, uint32_t* dev_err,
                                     void* stream);

/* Queries of alhr_attend_cache. */
typedef struct {
  int32_t requests;       /* >= 0; at most 8192 (else ALHR_ERR_UNSUPPORTED)                    */
  int32_t tokens;         /* rows of Q and out, >= 0; tokens * q_heads < 2^31                  */
  int32_t q_heads;        /* a multiple of the cache's heads; query head h reads key head
                             h / (q_heads / heads); the quotient is at most 64                 */
  int32_t max_blocks;     /* columns of block_table, >= 1; max_blocks * block_size <= 2^30     */
  int32_t max_q;          /* no request has more rows than this: it chooses the kernels, and
                             is no bound on what they compute; 0 means `tokens`                */
  int32_t type;           /* of Q and out: ALHR_TYPE_BF16 or ALHR_TYPE_FP16                    */
  int64_t q_token_stride; /* strides of Q in numbers; multiples of 8                           */
  int64_t q_head_stride;
  float scale;            /* of the scores; finite                                             */
} alhr_cache_queries;

/* Bytes of workspace that alhr_attend_cache needs for these sizes on the current device (its
 * contents need no initialisation), or 0 for invalid arguments. */
ALHR_API size_t alhr_attend_cache_workspace(const alhr_cache* cache,
                                            const alhr_cache_queries* queries);

/*
 * alhr_attend_cache -- attention over all visible keys of each request.
 *
 * Rows [q_start[r], q_start[r + 1]) of Q belong to request r; row q_start[r] + t stands at
 * position ctx_len[r] + t and sees the keys [0, min(ctx_len[r] + t + 1, seq_len[r])):
 *   s_j = scale * (q . k_j),  out = sum_j exp(s_j) v_j / sum_j exp(s_j),  lse = ln sum_j exp(s_j)
 * A row that sees no key gets zeros and lse = -infinity. A NaN in another row of Q makes the
 * row's out and lse NaN and touches no other row. Rows outside every request keep what they hold.
 * seq_len is cut at max_blocks * block_size, q_start at [0, tokens]; keys in blocks outside
 * [0, blocks) are left out and set ALHR_DEVERR_BLOCK. Only table entries, scales and blocks that
 * hold visible keys are read, and codes behind seq_len have no effect. A value scale below 2^-100
 * (alhr_store_cache writes none) counts as 0.
 *   Q         device, type as given; base 16-byte aligned
 *   out       device [tokens][q_heads][d], type of Q, 16-byte aligned
 *   lse       device float [tokens][q_heads], or NULL
 *   workspace device, 16-byte aligned; used from launch to completion of this call, so calls that
 *             may run at the same time need one each
 * The sums are fp32; a key's weight times its value scale is held in 16 bits: to 2^-11 of itself
 * down to 2^-21 of the row's largest, below that to 2^-32 of the largest
 * (alhr_attend_cache_selected holds it to 2^-22 of itself). The result of a call depends on its
 * inputs and the device alone. Requests with more than 16 rows per key/value head are computed on the
 * tensor core, whose waits are bounded: should one run out (not expected), ALHR_DEVERR_TIMEOUT is
 * set and out and lse of the call are not to be used.
 */
ALHR_API alhr_status alhr_attend_cache(const alhr_cache* cache, const alhr_cache_queries* queries,
                                       const void* Q, const int32_t* block_table,
                                       const int32_t* ctx_len, const int32_t* seq_len,
                                       const int32_t* q_start, void* out, float* lse,
                                       void* workspace, size_t workspace_bytes,
                                       uint32_t* dev_err, void* stream);

/* Queries of alhr_attend_cache_selected. */
typedef struct {
  int32_t batch;      /* >= 1                                                                  */
  int32_t q_heads;    /* a multiple of the cache's heads, as above                             */
  int32_t nq;         /* query rows of each (b,h), >= 0; batch * q_heads * nq < 2^31           */
  int32_t max_keys;   /* columns of idx, 1 <= max_keys <= 96                                   */
  int32_t max_blocks; /* columns of block_table, >= 1; max_blocks * block_size <= 2^30         */
  int32_t type;       /* of Q: ALHR_TYPE_INT8, BF16 or FP16                                    */
  float scale;        /* of the scores; finite                                                 */
} alhr_cache_selection;

/*
 * alhr_attend_cache_selected -- alhr_attend over the cache: out = softmax(scale * q . k_j) . v_j
 * over the positions j = idx[0..count) of sequence b, in fp32.
 * Row t stands at position ctx_len[b] + t; entries of idx outside
 * [0, min(ctx_len[b] + t + 1, seq_len[b], max_blocks * block_size)) are skipped and set
 * ALHR_DEVERR_INDEX, entries in blocks outside [0, blocks) are skipped and set
 * ALHR_DEVERR_BLOCK. A position that is named twice counts twice. A row without keys gets zeros,
 * one with a NaN in Q gets NaN.
 *   Q            device, type as given, [batch][q_heads][nq][d], 16-byte aligned
 *   block_table  device int32 [batch][max_blocks]
 *   idx, count   device int32 [batch][q_heads][nq][max_keys], [batch][q_heads][nq]
 *   out          device float [batch][q_heads][nq][d], 16-byte aligned, overwritten
 */
ALHR_API alhr_status alhr_attend_cache_selected(const alhr_cache* cache,
                                                const alhr_cache_selection* queries,
                                                const void* Q, const int32_t* block_table,
                                                const int32_t* ctx_len, const int32_t* seq_len,
                                                const int32_t* idx, const int32_t* count,
                                                float* out, uint32_t* dev_err, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ALHR_CACHE_H */

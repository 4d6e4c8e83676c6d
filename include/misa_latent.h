/*
 * misa_latent.h -- C ABI of libmisa.so, second part: the latent key/value cache
 * held in 16, 8 or 4 bits, written and read back, and the attention that reads
 * it (the tokens the indexer lists, or a query's whole prefix).
 *
 * The conventions of misa.h hold: device pointers owned by the caller,
 * asynchronous on `stream`, nothing allocated, arguments checked on the host
 * before anything is launched, device-side findings as MISA_DEVERR_* bits in
 * the first word of the workspace.
 *
 * A latent row is MISA_MLA_DQK (576) numbers, one row a token, shared by every
 * query head: MISA_MLA_DV (512) latent entries, then 64 rotary ones.  Keys are
 * whole rows, values their first 512 entries.  A cache holds `nseq` sequences of
 * L rows; row s of sequence b starts at byte b * cache_seq_stride + s * R, with
 * R the row's bytes in the cache's form:
 *   MISA_KV_BF16 (1152 bytes)  the 576 bf16 numbers.
 *   MISA_KV_MX8  (656 bytes)   512 e4m3 numbers; 16 scale bytes; 64 bf16 rotary.
 *   MISA_KV_MX4  (400 bytes)   512 e2m1 numbers, two a byte, the even entry in
 *                              the low half; 16 scale bytes; 64 bf16 rotary.
 * Scale byte g is e + 127 for the 32 entries [32 g, 32 g + 32): entry c stands
 * for element[c] * 2^e.  e is the smallest integer for which no entry of the
 * group is above the largest number of the element type (448 or 6) times 2^e,
 * held within [-117, 119] (MX8) or [-117, 125] (MX4); entries are then rounded
 * to the nearest element, ties to even, and entries that the largest e still
 * leaves too large become the largest element.  A group with an infinity or a
 * NaN gets scale byte 255, and every entry of it reads back as NaN.  So each
 * entry is rounded once, when it is written: what an element and its scale stand
 * for is a bf16 number exactly, and reading back and attending use that number.
 */
#ifndef MISA_LATENT_H
#define MISA_LATENT_H

#include "misa.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MISA_KV_BF16 0
#define MISA_KV_MX8 1
#define MISA_KV_MX4 2

/* Operation ids for misa_workspace_bytes (arguments it uses):
 *   APPEND_KV: none;  READ_KV: none;  SPARSE_MLA_Q: T, H (= Hq), k;
 *   PREFIX_MLA: T, H (= Hq), L.
 * A workspace of that size also serves every call with fewer of any of them.  It
 * is 256 bytes and 2056 Hq bytes for each partial result: at most 128 a query, one
 * for each 64 rows, 296 in all.  Only the error word has to be cleared, once. */
#define MISA_OP_APPEND_KV 9
#define MISA_OP_READ_KV 10
#define MISA_OP_SPARSE_MLA_Q 11
#define MISA_OP_PREFIX_MLA 12

/* Bytes of one cache row in form `fmt` (host; 0 for an unknown form). */
MISA_API int64_t misa_kv_row_bytes(int fmt);

/*
 * misa_append_kv -- write new latent rows into a cache, quantising them.
 * rows: [nseq][n_new][576] bf16.  Rows i < counts[b] of sequence b (counts NULL:
 *   all n_new) go to cache rows [len[b], len[b] + counts[b]).  Nothing else of
 *   the cache is touched; len is not advanced.
 * A sequence with counts[b] outside [0, n_new], len[b] < 0 or len[b] + counts[b]
 *   > L_cap is skipped and sets MISA_DEVERR_BAD_LEN.
 * Limits: nseq, n_new, L_cap >= 1; rows and cache 16-byte aligned;
 *   cache_seq_stride a multiple of 16, and >= L_cap * R when nseq > 1;
 *   nseq * n_new < 2^31.
 * workspace: >= misa_workspace_bytes(MISA_OP_APPEND_KV, ...) (the error word).
 */
MISA_API misa_status misa_append_kv(const uint16_t* rows, int64_t nseq, int n_new, const int32_t* counts,
                                    const int32_t* len, int fmt, void* cache, int64_t cache_seq_stride, int64_t L_cap,
                                    void* workspace, size_t workspace_bytes, misa_stream_t stream);

/*
 * misa_read_kv -- cache rows back as bf16.  out: [T][n][576] bf16.
 *   idx != NULL: out[t][i] = row idx[t * idx_stride + i] of sequence seq_of[t];
 *     -1 gives a row of zeros; other values outside [0, L) too, and set
 *     MISA_DEVERR_BAD_INDEX.  first and prefix_len must be NULL.
 *   idx == NULL: out[t][i] = row first[t] + i (first NULL: i), zeros at and past
 *     min(prefix_len[t], L) (prefix_len NULL: L).  first[t] < 0 sets
 *     MISA_DEVERR_BAD_INDEX and gives zeros.
 * seq_of[t] outside [0, nseq) sets MISA_DEVERR_BAD_SEQ and gives zeros.
 * Limits: T, n, L, nseq >= 1; cache and out 16-byte aligned; cache_seq_stride a
 *   multiple of 16, and >= L * R when nseq > 1; L < 2^31, T * n < 2^31.
 * workspace: >= misa_workspace_bytes(MISA_OP_READ_KV, ...) (the error word).
 */
MISA_API misa_status misa_read_kv(const void* cache, int fmt, int64_t nseq, int64_t cache_seq_stride, int64_t L,
                                  const int32_t* seq_of, int T, const int32_t* idx, int64_t idx_stride,
                                  const int32_t* first, const int32_t* prefix_len, int64_t n, uint16_t* out,
                                  void* workspace, size_t workspace_bytes, misa_stream_t stream);

/*
 * misa_sparse_mla_q -- misa_sparse_mla over a quantised cache: attention of every
 * query head over its query's listed tokens (what the indexer selects).
 *   out[t][h] = sum_i p_i v_i / sum_i p_i, p_i = exp(scale * q[t][h] . k_i), i over
 *   the listed slots of query t; lse[t][h] = log sum_i p_i (natural logarithm).
 * q: [T][Hq][576] bf16.  idx: [T] rows of k int32 token ids (row stride
 *   idx_stride >= k) in cache seq_of[t]; -1 = empty slot, others outside [0, L)
 *   are treated as empty and set MISA_DEVERR_BAD_INDEX.  A token listed twice
 *   counts twice.  out: [T][Hq][512] bf16.  lse: [T][Hq] fp32, may be NULL.
 * A query with no valid slot, with scores of -inf only, or with seq_of[t] outside
 *   [0, nseq) (which sets MISA_DEVERR_BAD_SEQ), gets zeros and lse = -inf.  A NaN
 *   or +inf among the scores gives NaN.
 * Precision: products of bf16 numbers summed in fp32; weights summed in fp32 and
 *   rounded to bf16 for the value product; one rounding to bf16 at the end.
 * Limits: 1 <= Hq <= 128, 1 <= k <= MISA_MAX_TOPK, T, L, nseq >= 1, L < 2^31,
 *   T * Hq < 2^31, T < 2^29; scale finite and >= 0, and so scale * log2(e) in
 *   fp32; q, cache, out 16-byte aligned;
 *   cache_seq_stride as misa_read_kv; fmt MISA_KV_MX8 or MISA_KV_MX4
 *   (misa_sparse_mla reads bf16 rows).
 * workspace: >= misa_workspace_bytes(MISA_OP_SPARSE_MLA_Q, T, Hq, 0, 0, k, 0).
 */
MISA_API misa_status misa_sparse_mla_q(const uint16_t* q, const void* cache, int fmt, int64_t nseq,
                                       int64_t cache_seq_stride, int64_t L, const int32_t* seq_of, int T, int Hq,
                                       const int32_t* idx, int k, int64_t idx_stride, float scale, uint16_t* out,
                                       float* lse, void* workspace, size_t workspace_bytes, misa_stream_t stream);

/*
 * misa_prefix_mla -- attention of every query head over its query's whole prefix,
 * rows 0 <= s < min(prefix_len[t], L) of cache seq_of[t]: what a context no
 * longer than the selection needs, and what the selection is compared with.  The
 * formula, precision and outputs of misa_sparse_mla_q; prefix_len[t] <= 0 is a
 * query with no tokens (zeros, lse = -inf).  A prompt is T queries of one cache
 * with prefix_len[t] = the position + 1.
 * fmt: any of the three.  Limits as misa_sparse_mla_q without k.
 * workspace: >= misa_workspace_bytes(MISA_OP_PREFIX_MLA, T, Hq, L, 0, 0, 0).
 */
MISA_API misa_status misa_prefix_mla(const uint16_t* q, const void* cache, int fmt, int64_t nseq,
                                     int64_t cache_seq_stride, int64_t L, const int32_t* seq_of,
                                     const int32_t* prefix_len, int T, int Hq, float scale, uint16_t* out, float* lse,
                                     void* workspace, size_t workspace_bytes, misa_stream_t stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif /* MISA_LATENT_H */

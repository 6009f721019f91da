/* libfa's serving entry points: a paged K/V cache that is written as tokens
 * come, optionally quantised to FP8 E4M3, and attention of new tokens over it.
 * Part of libfa.so; status codes, streams, devices, workspaces and errors are
 * those of fa.h. (The pages describe decode as one query against many cached
 * keys and fix no cache: layouts and formats here are the library's own.)
 *
 * A ragged batch
 * --------------
 * B sequences; T token rows, the new tokens of all sequences packed in order:
 *  - cu_seqlens: int32 [B + 1], device: sequence b's new tokens are rows
 *    cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (its count n_b may be 0). Values are
 *    clamped to [0, T]; rows before cu_seqlens[0] and from cu_seqlens[B] on are
 *    padding: not read, and left as they were in every output. They must not
 *    decrease: where they do, nothing outside the tensors is reached, but rows that
 *    two sequences claim may hold either's result, and some may hold neither.
 *  - seqlens_k: int32 [B], device: sequence b's length L_b (0 when negative), its
 *    n_b new tokens included. New token t of sequence b (t = 0 .. n_b - 1) stands
 *    at position L_b - n_b + t. A position below 0 or past the block table
 *    (max_pages * 128 and on) is no place: a token there is not written, reads as
 *    zeros, and sees no key.
 * The lengths live on the device, so a call captured into a CUDA graph follows
 * whatever they hold at each replay.
 *
 * The cache
 * ---------
 *  - k_cache, v_cache: [num_pages][H_kv][128][d], 16-byte aligned; position j of
 *    sequence b is row j % 128 of page block_table[b][j / 128], block_table
 *    int32 [B][max_pages], device. A table entry outside [0, num_pages) is
 *    never followed: a write to it is dropped, a read of it gives zeros.
 *  - FA_CACHE_16BIT: elements of type dtype (BF16 or FP16). k_exp, v_exp NULL.
 *  - FA_CACHE_E4M3: one E4M3 code per element, and per row (one token of one KV
 *    head) one power of two: k_exp, v_exp are bytes [num_pages][H_kv][128], and
 *    an element stands for code * 2^(byte - 127), rounded to dtype (exact for
 *    every row fa_cache_append wrote from BF16 or FP16). Byte 255 with
 *    all codes 0x7F: a NaN row. In other rows the codes 0x7F and 0xFF are not
 *    allowed (their value is unspecified); fa_cache_append writes none.
 * d must be 64 or 128 (FA_ERR_UNSUPPORTED otherwise). */
#ifndef LIBFA_FA_SERVING_H
#define LIBFA_FA_SERVING_H

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a paged cache stores its elements. */
typedef enum { FA_CACHE_16BIT = 0, FA_CACHE_E4M3 = 1 } fa_cache_format;

/* Write the new tokens' K and V into the cache. k, v: dtype [T][H_kv][d], rows
 * of one token contiguous, tokens k_stride / v_stride elements apart (at least
 * H_kv * d, a multiple of 8: slices of a fused projection need no copy).
 * FA_CACHE_16BIT copies. FA_CACHE_E4M3 quantises each row: e = the smallest
 * integer >= -120 with max|x| <= 448 * 2^e, codes = x * 2^-e rounded to nearest
 * even, byte = e + 127 (a row of zeros: codes 0, byte 7). A row that holds a NaN
 * or an infinity becomes a NaN row (byte 255, codes 0x7F). A token whose position
 * is below 0 or past the table is dropped: a sequence that outgrows its table
 * loses what no longer fits, and keeps what it holds. The new tokens of a batch must lie in
 * distinct cache rows (two sequences sharing a page they both write race).
 * Returns FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED or FA_ERR_CUDA. */
int fa_cache_append(const void* k, const void* v, void* k_cache, void* v_cache, unsigned char* k_exp,
                    unsigned char* v_exp, const int* block_table, const int* cu_seqlens,
                    const int* seqlens_k, int B, int T, int H_kv, int num_pages, int max_pages, int d,
                    long long k_stride, long long v_stride, int dtype, int cache_format, void* stream);

/* Read rows back: k, v (dtype [T][H_kv][d], contiguous) receive what the cache
 * holds at the positions fa_cache_append would write (the last n_b of the first
 * L_b positions of each sequence; a whole sequence has n_b = L_b). E4M3 rows
 * come back as the values they stand for. A position below 0 or past the table gives
 * zeros.
 * Returns as fa_cache_append. */
int fa_cache_read(const void* k_cache, const void* v_cache, const unsigned char* k_exp,
                  const unsigned char* v_exp, const int* block_table, const int* cu_seqlens,
                  const int* seqlens_k, void* k, void* v, int B, int T, int H_kv, int num_pages,
                  int max_pages, int d, int dtype, int cache_format, void* stream);

/* Attention of the new tokens of a ragged batch over the paged cache, which holds
 * them already (fa_cache_append first): chunks of prompts, single tokens, or both
 * in one call. Token t of sequence b, at position pos = L_b - n_b + t, sees key j iff
 *     j <= pos  and  (window == 0  or  j > pos - window  or  j < sinks),
 * i.e. everything before it, or its last `window` keys (itself among them) and the
 * sequence's first `sinks` keys. O = softmax(scale * Q K^T) V over them, LSE as
 * fa_forward's; a token that sees no key (pos < 0 or past the table) gets O = 0 and
 * LSE = -inf.
 *  - q: dtype [T][H_q][d], rows of one token contiguous, tokens q_stride elements
 *    apart (at least H_q * d, a multiple of 8), 16-byte aligned; H_q % H_kv == 0.
 *  - o: dtype [T][H_q][d]; lse: FP32 [T][H_q] or NULL; contiguous.
 *  - max_q: the largest n_b. It sizes the launch; the tokens past max_q of a sequence
 *    that has more are left as they were.
 *  - k_exp, v_exp: 16-byte aligned.
 *  - Pages no token sees are not read, nor are a sequence's rows past its length used:
 *    they may hold anything. In a page that some token sees a key of, a sequence's own
 *    K and V must be finite: a NaN or infinity in V there reaches rows that do not see
 *    its key as 0 * NaN. Queries do not reach one another.
 *  - BF16: |V| up to 2^59 (the running maximum may lag behind a row's by 2^48), and |K| up
 *    to 2^105 in an E4M3 cache (queries are scaled up to 2^14 before their products).
 * FP32 accumulation, softmax statistics and LSE; P is rounded to 16 bits for P V; an
 * E4M3 cache is read as the values it stands for, exactly. Deterministic.
 * Rows that read one KV head ((H_q / H_kv) * max_q) of at most 16 take a kernel that
 * streams the cache once at HBM rate; more take tcgen05 tiles of 128 rows. Over E4M3
 * pages a few chunks beside many sequences of a token or two take both, each its own.
 * (One token a sequence over 16-bit pages, no window: fa_decode_paged is the leaner call.)
 * Returns FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED (d; H_q / H_kv > 128),
 * FA_ERR_NO_MEMORY or FA_ERR_CUDA. */
int fa_extend_paged(const void* q, const void* k_cache, const void* v_cache, const unsigned char* k_exp,
                    const unsigned char* v_exp, const int* block_table, const int* cu_seqlens,
                    const int* seqlens_k, void* o, float* lse, int B, int T, int max_q, int H_q, int H_kv,
                    int num_pages, int max_pages, int d, long long q_stride, int window, int sinks,
                    float scale, int dtype, int cache_format, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBFA_FA_SERVING_H */

/* libfa's attention under a sliding window with sinks, forward and backward: the
 * form long-context models are trained with. Part of libfa.so; layouts, GQA, status
 * codes, streams, devices, workspaces and errors are those of fa.h. (The pages have
 * no window; the mask is the causal one of fa_forward with keys taken out, and the
 * method is theirs: masked tiles are never loaded, "What interviewers probe next".)
 *
 * Query row i stands at position pos = i + (N_k - N_q) and sees key j iff
 *     j <= pos  and  (j > pos - window  or  j < sinks):
 * its last `window` keys, itself among them, and the first `sinks` keys. window >= 1,
 * sinks >= 0; a window of N_k or more is the causal mask. The same mask as
 * fa_extend_paged's. A row that sees no key gets O = 0 and LSE = -inf. */
#ifndef LIBFA_FA_WINDOW_H
#define LIBFA_FA_WINDOW_H

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* q: dtype [B][H_q][N_q][d]; k, v: [B][H_kv][N_k][d]; o as q; lse: FP32
 * [B][H_q][N_q] or NULL; dtype FA_DTYPE_BF16 or FA_DTYPE_FP16. Work and K/V traffic
 * follow the keys that are seen: tiles of 128 rows hold the query heads of one KV
 * head side by side. Deterministic. BF16: |V| up to 2^59 (the running maximum may lag
 * behind a row's by 2^48). Returns FA_OK, FA_ERR_INVALID_ARG,
 * FA_ERR_UNSUPPORTED (d not 64 or 128; H_q / H_kv > 128), FA_ERR_NO_MEMORY or
 * FA_ERR_CUDA. */
int fa_forward_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H_q,
                      int H_kv, int N_q, int N_k, int d, int window, int sinks, float scale, int dtype,
                      void* stream);

/* Gradients of fa_forward_window, given its o and lse and the upstream gradient
 * dout: everything else as fa_backward. Unlike there, o and lse must be those of exactly
 * the keys that this call shows each row: rowsum(dout * o) is put right by the row sums of
 * dS over them, which are 0 for no other lse. Keys held in pieces, each with the lse of
 * the whole, are fa_backward's case and not this one's. */
int fa_backward_window(const void* q, const void* k, const void* v, const void* o, const float* lse,
                       const void* dout, void* dq, void* dk, void* dv, int B, int H_q, int H_kv, int N_q,
                       int N_k, int d, int window, int sinks, float scale, int dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBFA_FA_WINDOW_H */

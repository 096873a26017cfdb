/*
 * qat_kv.h -- C ABI of a served decoder block's attention on gfx950: rotary
 * positions, a paged cache of keys and values in 8 bits, and the attention
 * that reads it.
 *
 * Conventions: those of qat.h (device pointers owned by the caller; checks of
 * the arguments before anything is enqueued; asynchronous on `stream`; a QAT_*
 * status returned; nothing allocated or kept), dtype QAT_BF16 or QAT_F16 of
 * qat_mx.h. Activations are [tokens][heads][head_dim], heads and head_dim
 * contiguous, ld* elements from one token to the next (a multiple of 8, at
 * least heads * head_dim), 16-byte aligned. head_dim is 64 or 128.
 *
 * A batch of `batch` sequences packs its new tokens one sequence after the
 * other: cu [batch + 1] int32, tokens cu[b] .. cu[b + 1] - 1 belong to
 * sequence b, cu[0] = 0. lens [batch] int32 is each sequence's length with
 * those tokens, so new token i of sequence b has position lens[b] - n_b + i,
 * n_b = cu[b + 1] - cu[b]. A sequence may have no new tokens, and no tokens at
 * all. max_new is a host-side bound on every n_b, max_len on every lens[b]; the
 * kernels and their grids are chosen by them, so they should be near the truth.
 *
 * The cache: pages of `page` tokens (16, 32, 64 or 128).
 *   k_cache [n_pages][heads][page][head_dim] e4m3 (OCP FP8 E4M3, uint8)
 *   v_cache [n_pages][heads][head_dim][page] e4m3: a value block is stored
 *           with its tokens innermost, the order in which the matrix cores
 *           contract over them
 *   k_scale, v_scale [n_pages][heads] fp32, not negative: a value is code * scale
 *   table [batch][table_cols] int32: position p of sequence b is in slot
 *           p % page of page table[b][p / page].
 * The lengths, cu and table are read on the device and never trusted for an
 * address: tokens of positions below 0 or at max_len, table_cols * page or
 * beyond, tokens outside [0, tokens), sequences' tokens beyond max_new and
 * entries of table outside [0, n_pages) are left out, as said at each call.
 */
#ifndef QAT_KV_H
#define QAT_KV_H

#include "qat_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { QAT_ROPE_PLAIN = 0, QAT_ROPE_LINEAR = 1, QAT_ROPE_PARTS = 2 };

/*
 * The angles per position of a rotary embedding, on the HOST (inv_freq: rot / 2
 * floats in host memory): f_i = base^(-2i / rot), and for a context stretched
 * by `factor` over the `original` one
 *   QAT_ROPE_LINEAR  f_i / factor (position interpolation);
 *   QAT_ROPE_PARTS   f_i (1 - w_i) / factor + f_i w_i: pairs that turn more
 *     than beta_fast times over the original context keep their angle, those
 *     below beta_slow are interpolated, with a linear ramp over the pair index
 *     between (YaRN, arXiv 2309.00071, section 3.2); *mscale = 0.1 ln(factor)
 *     + 1 (its section 3.4) for factor > 1.
 * *mscale is 1 otherwise. original, beta_fast and beta_slow are read by
 * QAT_ROPE_PARTS only, factor (>= 1) by both scalings.
 */
int32_t qat_rope_inv_freq(int32_t rot, double base, int32_t scaling, double factor, int64_t original,
                          double beta_fast, double beta_slow, float* inv_freq, float* mscale);

/*
 * Rotary positions. For token t, head h and pair i < rot / 2 with the angle
 * a = pos[t] * inv_freq[i] (the product and its reduction in 64 bits):
 *   (x_p, x_q) -> mscale (x_p cos a - x_q sin a, x_q cos a + x_p sin a),
 *   (p, q) = (i, i + rot / 2) with half = 1, (2i, 2i + 1) with half = 0;
 * elements rot .. head_dim - 1 are copied. inverse = 1 turns by -a: the
 * gradient of a loss to the input from the one to the output. rot is a
 * multiple of 16, 16 <= rot <= head_dim. q [tokens][heads_q][head_dim] and k
 * (with heads_k; heads_k = 0 and NULL pointers: none) are done in one launch;
 * an output may be its own input (same pointer and stride), and meets nothing
 * else.
 */
int32_t qat_rope(const void* q, const void* k, const int32_t* pos, const float* inv_freq, int64_t tokens,
                 int32_t heads_q, int32_t heads_k, int32_t head_dim, int32_t rot, int32_t half, int32_t inverse,
                 float mscale, int32_t dtype, int64_t ldq, int64_t ldk, void* q_out, int64_t ldq_out, void* k_out,
                 int64_t ldk_out, hipStream_t stream);

/*
 * Appends the new tokens' keys and values to the cache. Every (page, head)
 * block that new tokens reach gets the scale 2^e with e the larger of
 *   - the smallest e >= -126 with 448 2^e >= the largest finite magnitude of
 *     its new keys (values), and
 *   - if it held tokens of this sequence before, the e of its present scale;
 * its codes are e4m3(x 2^-e), to nearest, ties to even (earlier tokens' codes
 * are rounded again where e grew); infinities and NaN become the NaN code.
 * Slots of other positions keep their codes. Scales of blocks that hold
 * tokens are expected to be powers of two, as this call makes them. Left out
 * (not written): tokens that have no slot as said above. No page may be
 * appended to through two entries of the table in the same call (two sequences,
 * or one twice): its contents are undefined then.
 */
int32_t qat_kv_append(const void* k, const void* v, int32_t dtype, int64_t ldk, int64_t ldv, const int32_t* cu,
                      const int32_t* lens, const int32_t* table, int64_t table_cols, int64_t tokens, int64_t batch,
                      int32_t heads, int32_t head_dim, int32_t page, int64_t n_pages, int64_t max_new,
                      uint8_t* k_cache, uint8_t* v_cache, float* k_scale, float* v_scale, hipStream_t stream);

/* Workspace bytes of qat_kv_attn (partial results of sequences that are split);
 * 0 for invalid sizes. */
size_t qat_kv_attn_ws_bytes(int64_t tokens, int64_t batch, int32_t heads_q, int32_t heads_kv, int32_t head_dim,
                            int64_t max_new, int64_t max_len);

/*
 * out[t][h] = sum_j softmax_j(softmax_scale q[t][h] . K[j][h']) V[j][h'] with
 * h' = h heads_kv / heads_q, over the cached positions j of token t's sequence
 * (the new tokens' own keys and values are in the cache already): all of them
 * with causal = 0, those up to the token's own with causal = 1. Scores, the
 * softmax's maximum and sum and the output are held in fp32; probabilities are
 * rounded to fp16 for the second product. Keys in masked places and in pages
 * that are left out are never part of a result, whatever they hold. A token
 * that sees no key gets zeros. Rows of out at cu[batch] and beyond are left as
 * they were.
 */
int32_t qat_kv_attn(const void* q, int32_t dtype, int64_t ldq, const int32_t* cu, const int32_t* lens,
                    const int32_t* table, int64_t table_cols, int64_t tokens, int64_t batch, int32_t heads_q,
                    int32_t heads_kv, int32_t head_dim, int32_t page, int64_t n_pages, const uint8_t* k_cache,
                    const uint8_t* v_cache, const float* k_scale, const float* v_scale, float softmax_scale,
                    int32_t causal, int64_t max_new, int64_t max_len, void* out, int64_t ldo, void* ws,
                    size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QAT_KV_H */

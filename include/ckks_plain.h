/*
 * ckks_plain.h -- the plaintext side of an encrypted decoder on the same GPU.
 *
 * What the key holder computes in clear around the encrypted layers: a
 * decrypted hop is a few tokens' hidden states (the slots of a token's
 * ciphertexts), and next to it stand the values an encrypted layer is checked
 * against.  The operators, in the order of a token's way:
 *   embed:         rows of a table by token, scaled, before their encryption
 *                  (with the table's gradient);
 *   residual_norm: the residual stream takes a gated, optionally normalised
 *                  block output and is normalised for the next block (with its
 *                  gradient, and with an 8-bit output);
 *   head_norm_rotate: queries and keys normalised for each head and rotated by
 *                  position (with its gradient);
 *   matmul_i8:     rows quantised to 8 bits times 8-bit weights, with a scale
 *                  for each row (token) and each weight row (channel);
 *   sample:        the next token from logits by temperature, top-k, top-p and
 *                  min-p, from given random numbers;
 *   token_logprobs: log probabilities of given tokens, the entropy and the
 *                  largest alternatives (with the logits' gradient).
 *
 * Conventions shared by every call
 *  - Data pointers are DEVICE pointers on the calling thread's current HIP
 *    device; matrices are row-major with unit column stride and a row stride
 *    in elements, at least the number of columns.  Any row stride and element
 *    alignment is taken; rows that start at multiples of 16 bytes are faster.
 *  - `stream` is a hipStream_t (NULL = the default stream).  Calls only
 *    enqueue work: no synchronisation, no allocation, no state kept between
 *    calls.  Results are the same bits on every run.
 *  - Sums, means, deviations and softmax masses are held in 32 bits or more;
 *    a result is rounded once, where it is stored in a 16-bit type.  The squares
 *    of a normalised row have to add up to less than 2^128.
 *  - An output whose byte range overlaps an input's is rejected (CKKS_EINVAL)
 *    unless the call says otherwise.
 *  - Zero rows are valid; nothing is launched, except that gradients of
 *    weights and tables are written (as zeros).  There are fewer than 2^31.
 *  - Errors are the codes of ckks_gpu.h; arguments are validated before any
 *    launch.  CKKS_EALIGN: a pointer not aligned to its element type (8-bit
 *    rows: to 16 bytes).
 */
#ifndef CKKS_PLAIN_H
#define CKKS_PLAIN_H
#include <stddef.h>
#include <stdint.h>

#include "ckks_gpu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
#define CKKS_PLAIN_BF16 0
#define CKKS_PLAIN_F16 1
#define CKKS_PLAIN_F32 2

/* kinds of norm: v / sqrt(mean v^2 + eps), and (v - mean v) / sqrt(var v + eps) */
#define CKKS_PLAIN_RMS 0
#define CKKS_PLAIN_LAYER 1

/* most columns of a normalised or quantised row (a row is held in registers) */
#define CKKS_PLAIN_MAX_COLS 16384

/* Residual stream and norms around a block:
 *   n = y                                       (block_weight NULL), or
 *   n = block_weight norm(y) + block_bias       (the norm after the block);
 *   h = x + scale g n                           (g = 1 without a gate);
 *   u = next_weight norm(h) + next_bias         (the norm before the next block).
 * x, y: [rows][cols].  gate: [groups][cols], row r uses gate row
 * r / (rows / groups); groups = 0 means no gate, else it divides rows (1: a
 * gate for each channel; rows: one of its own for each token).  Weights,
 * biases [cols] and gate have the same type as x; biases may be NULL.  The
 * norm of h is taken before h is rounded. */
typedef struct {
    int type; /* CKKS_PLAIN_BF16, _F16 or _F32 */
    int kind; /* CKKS_PLAIN_RMS or _LAYER, for both norms */
    int64_t rows, cols, groups;
    const void *x, *y;
    int64_t x_stride, y_stride;
    const void *next_weight, *next_bias;
    const void *block_weight, *block_bias;
    const void *gate;
    float scale, eps;
} ckks_plain_norm;

/* h and u: [rows][cols] of the type of x.  h may be x itself (the same
 * pointer and stride). */
int ckks_plain_residual_norm(const ckks_plain_norm *p, void *h, int64_t h_stride, void *u, int64_t u_stride,
                             void *stream);
/* The same with u as 8-bit rows (ckks_plain_quantize_rows of the unrounded u). */
int ckks_plain_residual_norm_i8(const ckks_plain_norm *p, void *h, int64_t h_stride, int8_t *q, int64_t q_stride,
                                float *q_scale, void *stream);

/* Gradients, given those of h and u (dh, du: [rows][cols], the type of x):
 * dx, dy [rows][cols] of the type of x; of the weights, biases and gate in
 * 32 bits, each where the forward call has that operand (NULL otherwise).
 * Row values are recomputed from x and y.  ws: scratch of
 * ckks_plain_norm_grad_workspace_size bytes, aligned to 16. */
typedef struct {
    const void *dh, *du;
    int64_t dh_stride, du_stride;
    void *dx, *dy;
    int64_t dx_stride, dy_stride;
    float *next_weight, *next_bias, *block_weight, *block_bias; /* [cols] */
    float *gate;                                                /* [groups][cols] */
} ckks_plain_norm_grads;
int ckks_plain_norm_grad_workspace_size(const ckks_plain_norm *p, size_t *bytes);
int ckks_plain_residual_norm_grad(const ckks_plain_norm *p, const ckks_plain_norm_grads *g, void *ws, size_t ws_bytes,
                                  void *stream);

/* Queries and keys [tokens][heads][head_dim], normalised for each head and
 * rotated by position; y of a head x:
 *   n = x / sqrt(mean x^2 + eps) weight         (weight NULL: n = x)
 *   dimensions a and b of pair i < rotary / 2, at the angle
 *   f = positions[t] inv_freq[i]:
 *   y_a = n_a cos f - n_b sin f,  y_b = n_b cos f + n_a sin f,
 *   (a, b) = (i, i + rotary / 2), or (2 i, 2 i + 1) if interleaved; from
 *   rotary on, y = n.
 * Element (t, h, i) of a tensor is at t token_stride + h head_stride + i, both
 * strides at least head_dim where there is more than one token or head.
 * head_dim and rotary are even, rotary <= head_dim <= CKKS_PLAIN_MAX_HEAD.
 * positions [tokens] and inv_freq [rotary / 2] may be NULL where rotary is 0;
 * the angle's product and its turns are held in 64 bits, its sine and cosine
 * in 32.  k_heads = 0: queries alone (k and k_weight NULL).  Weights have the
 * type of q and k. */
#define CKKS_PLAIN_MAX_HEAD 512
typedef struct {
    int type; /* CKKS_PLAIN_BF16, _F16 or _F32 */
    int interleaved;
    int64_t tokens, q_heads, k_heads, head_dim, rotary;
    const void *q, *k;
    int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride;
    const void *q_weight, *k_weight; /* [head_dim] */
    const int64_t *positions;
    const float *inv_freq;
    float eps;
} ckks_plain_heads;

/* q_out and k_out may be q and k themselves (the same pointer and strides);
 * elements of an output do not share memory.  Tensors of one token stride whose
 * tokens lie beside each other (parts of a joint projection's rows) do not
 * overlap, here and in the gradient. */
int ckks_plain_head_norm_rotate(const ckks_plain_heads *p, void *q_out, int64_t q_out_token_stride,
                                int64_t q_out_head_stride, void *k_out, int64_t k_out_token_stride,
                                int64_t k_out_head_stride, void *stream);

/* Gradients, given those of the outputs (dq, dk): dq_in, dk_in of the type of
 * q; of the weights in 32 bits, each where the forward call has that operand
 * (NULL otherwise).  ws: scratch of ckks_plain_head_grad_workspace_size bytes,
 * aligned to 16 (may be NULL where that is 0). */
typedef struct {
    const void *dq, *dk;
    int64_t dq_token_stride, dq_head_stride, dk_token_stride, dk_head_stride;
    void *dq_in, *dk_in;
    int64_t dq_in_token_stride, dq_in_head_stride, dk_in_token_stride, dk_in_head_stride;
    float *q_weight, *k_weight; /* [head_dim] */
} ckks_plain_head_grads;
int ckks_plain_head_grad_workspace_size(const ckks_plain_heads *p, size_t *bytes);
int ckks_plain_head_norm_rotate_grad(const ckks_plain_heads *p, const ckks_plain_head_grads *g, void *ws,
                                     size_t ws_bytes, void *stream);

/* 8-bit rows: row t stands for scale[t] q[t][0..cols).  They start at
 * multiples of CKKS_PLAIN_I8_ROW bytes (q aligned to 16 bytes, q_stride a
 * multiple of CKKS_PLAIN_I8_ROW and at least cols rounded up to one) and hold
 * zeros from cols to the next such multiple.  Producers here write the zeros. */
#define CKKS_PLAIN_I8_ROW 128

/* q = rint(x / s) clamped to [-127, 127], s = max |x| of the row times 1/127
 * (that constant, the product and the quotient each rounded to 32 bits, ties
 * to even); a row of zeros has s = 0, and a row that holds an infinity or a
 * NaN has s = NaN and q = 0.  cols <=
 * CKKS_PLAIN_MAX_COLS. */
int ckks_plain_quantize_rows(int type, const void *x, int64_t x_stride, int64_t rows, int64_t cols, int8_t *q,
                             int64_t q_stride, float *q_scale, void *stream);

/* out[t][c] = a_scale[t] w_scale[c] sum_k a[t][k] w[c][k] + bias[c]: a is
 * [rows][cols], w [channels][cols] (both 8-bit rows as above), bias [channels]
 * in 32 bits or NULL, out [rows][channels] of out_type.  The sum is exact in
 * 32-bit integers: cols < 131072; a_stride and w_stride < 2^23; rows and
 * channels <= 2^31 - 256.  ws: ckks_plain_matmul_i8_workspace_size bytes,
 * aligned to 16 (may be NULL where that is 0). */
int ckks_plain_matmul_i8_workspace_size(int64_t rows, int64_t channels, int64_t cols, size_t *bytes);
int ckks_plain_matmul_i8(const int8_t *a, int64_t a_stride, const float *a_scale, const int8_t *w, int64_t w_stride,
                         const float *w_scale, const float *bias, int out_type, void *out, int64_t out_stride,
                         int64_t rows, int64_t channels, int64_t cols, void *ws, size_t ws_bytes, void *stream);

/* ckks_plain_quantize_rows of x and then the product, the 8-bit rows in ws:
 * ckks_plain_linear_i8_workspace_size bytes, aligned to 16.  cols <=
 * CKKS_PLAIN_MAX_COLS. */
int ckks_plain_linear_i8_workspace_size(int64_t rows, int64_t channels, int64_t cols, size_t *bytes);
int ckks_plain_linear_i8(int type, const void *x, int64_t x_stride, const int8_t *w, int64_t w_stride,
                         const float *w_scale, const float *bias, int out_type, void *out, int64_t out_stride,
                         int64_t rows, int64_t channels, int64_t cols, void *ws, size_t ws_bytes, void *stream);

/* One token for each row of logits z [rows][vocab] (type as above).
 * A token is possible if it is allowed (allowed [rows][vocab] bytes, 0 = no;
 * NULL = all) and its logit is neither NaN nor -infinity.  In the order of
 * falling logits (lower index first among equals), with e = exp((z - max z) /
 * temperature):
 *   top_k[r] > 0: the first top_k[r] stay;
 *   top_p[r] < 1: of those, each stays before which their mass is below
 *                 top_p[r] of their total;
 *   min_p[r] > 0: those stay with e >= min_p[r];
 * the first always stays.  token = the one that stays with the largest
 * (z - max z) / temperature + gumbel[r][token] (each step rounded to 32 bits;
 * lowest index among equals): with gumbel = -log(-log u), u uniform in (0, 1), token is
 * drawn with probability e / sum e of those that stay.  temperature[r] <= 0:
 * the first in order.  logprob = log(e / sum e over all possible tokens), at
 * temperature 1 where temperature[r] <= 0.  A row without a possible token:
 * token -1, logprob -infinity.  gumbel [rows][vocab] in 32 bits, no NaN;
 * top_k, top_p and min_p may be NULL (off); an infinite logit outweighs every
 * finite one.  Masses are held in 32 bits (or whole multiples of 2^-38 and
 * less): tokens whose difference is lost there, or is a subnormal number, weigh
 * the same.  vocab <= 2^24.  ws: ckks_plain_sample_workspace_size bytes,
 * aligned to 16. */
int ckks_plain_sample_workspace_size(int64_t rows, int64_t vocab, size_t *bytes);
int ckks_plain_sample(int type, const void *logits, int64_t logits_stride, const float *gumbel, int64_t gumbel_stride,
                      const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                      const uint8_t *allowed, int64_t allowed_stride, int64_t rows, int64_t vocab, int64_t *token,
                      float *logprob, void *ws, size_t ws_bytes, void *stream);

/* For each row of logits z [rows][vocab], with the possible tokens of
 * ckks_plain_sample, its temperature (temperature NULL, or temperature[r] <= 0:
 * 1) and x = (z - max z) / temperature of them (an infinite logit outweighs
 * every finite one, and x of the largest is 0):
 *   largest = max z, log_mass = log sum exp x;
 *   logprob = x[tokens[r]] - log_mass, -infinity if that token is not
 *             possible; 0 if tokens[r] is outside [0, vocab) (a padded row);
 *   entropy = -sum p log p, p = exp(x - log_mass);
 *   top_token, top_logprob [rows][top]: the `top` largest in the order of
 *             falling logits (lower index first among equals), behind the
 *             last possible one token -1, log probability -infinity.
 * A row without a possible token: largest and log_mass -infinity, entropy 0.
 * top <= CKKS_PLAIN_MAX_TOP (0: top_token and top_logprob NULL), vocab <= 2^24.
 * Temperatures below 2^-127 count as that.  ws:
 * ckks_plain_token_logprobs_workspace_size bytes, aligned to 16 (may be NULL
 * where that is 0). */
#define CKKS_PLAIN_MAX_TOP 64
int ckks_plain_token_logprobs_workspace_size(int64_t rows, int64_t vocab, int64_t top, size_t *bytes);
int ckks_plain_token_logprobs(int type, const void *logits, int64_t logits_stride, const int64_t *tokens,
                              const float *temperature, const uint8_t *allowed, int64_t allowed_stride, int64_t rows,
                              int64_t vocab, int64_t top, float *logprob, float *entropy, float *largest,
                              float *log_mass, int64_t *top_token, float *top_logprob, void *ws, size_t ws_bytes,
                              void *stream);

/* Gradient of the logits from those of logprob and entropy (either may be
 * NULL: zero), given the entropy, largest and log_mass of the call above:
 *   dz = (dlogprob (1 at the token - p) - dentropy p (log p + entropy)) / temperature
 * for possible tokens, 0 for others; a token that is not possible or outside
 * [0, vocab) takes no part.  dlogits [rows][vocab] has the type of the logits. */
int ckks_plain_token_logprobs_grad(int type, const void *logits, int64_t logits_stride, const int64_t *tokens,
                                   const float *temperature, const uint8_t *allowed, int64_t allowed_stride,
                                   int64_t rows, int64_t vocab, const float *entropy, const float *largest,
                                   const float *log_mass, const float *dlogprob, const float *dentropy, void *dlogits,
                                   int64_t dlogits_stride, void *stream);

/* out[t] = scale table[tokens[t]]: table [vocab][cols], out [rows][cols] of
 * out_type; the product is rounded to 32 bits, then to out_type.  A row whose
 * token is outside [0, vocab) (padding, or what ckks_plain_sample says where
 * nothing is possible) is zeros.  vocab <= 2^24, cols < 2^31. */
int ckks_plain_embed(int type, const void *table, int64_t table_stride, int64_t vocab, int64_t cols,
                     const int64_t *tokens, int64_t rows, float scale, int out_type, void *out, int64_t out_stride,
                     void *stream);
/* The same from 8-bit rows (their columns alone are read): out[t] = (scale
 * q_scale[v]) q[v], v = tokens[t]. */
int ckks_plain_embed_i8(const int8_t *q, int64_t q_stride, const float *q_scale, int64_t vocab, int64_t cols,
                        const int64_t *tokens, int64_t rows, float scale, int out_type, void *out, int64_t out_stride,
                        void *stream);

/* Gradient of the table from that of the rows, drows [rows][cols] of `type`:
 *   out[v] = scale sum of drows[t] over the rows of token v   [+ out[v] if add]
 * out: [vocab][cols] of out_type.  Sums are held in 32 bits, go in a fixed
 * order and are rounded once.  Without `add` every row of out is written;
 * with it, those of the tokens alone.  Sorting reads all rows' tokens at most
 * 256 times for a vocabulary of up to 131072 and once for each 512 tokens of a
 * larger one: about 2.5 ms for 131072 rows and 2^24 tokens.  ws: scratch of
 * ckks_plain_embed_grad_workspace_size bytes, aligned to 16. */
int ckks_plain_embed_grad_workspace_size(int64_t rows, int64_t vocab, int64_t cols, size_t *bytes);
int ckks_plain_embed_grad(int type, const void *drows, int64_t drows_stride, const int64_t *tokens, int64_t rows,
                          int64_t vocab, int64_t cols, float scale, int out_type, void *out, int64_t out_stride,
                          int add, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif

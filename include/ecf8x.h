/*
 * ecf8x.h -- C ABI of libecf8 for 4-bit weights and mixtures of experts.
 *
 * Beside the lossless FP8 form of a weight (ecf8.h) a user keeps lossy 4-bit
 * ones, and the mixture-of-experts layers that a decode dispatch fills need
 * their products.  On AMD Instinct MI355X (gfx950):
 *   - values brought to microscaled 4-bit floating point and back
 *     (ecf8x_quantize, ecf8x_dequantize);
 *   - the product with such a weight, of 16-bit activations or of activations
 *     in the same 4 bits (ecf8x_linear), and the gradient that a frozen one
 *     passes to its input (ecf8x_input_grad);
 *   - a mixture-of-experts layer for a few tokens: the choice of experts
 *     (ecf8x_route) and their gated products (ecf8x_moe), with E4M3 or 4-bit
 *     weights.
 *
 * ------------------------------------------------------------------------
 * The 4-bit format (MXFP4 of the OCP microscaling specification).  A row of K
 * values, K a multiple of 32, is cut into blocks of 32.  A block has a scale
 * byte s, which stands for 2^(s - 127) (255: NaN), and 32 codes c of 4 bits:
 * a sign (8) and the magnitudes 0 0.5 1 1.5 2 3 4 6.  value = e2m1(c) 2^(s - 127).
 * Stored: Kp = K rounded up to 128; codes Kp / 2 bytes a row, two to a byte,
 * the first in the low half; scales Kp / 32 bytes a row.  Rows follow each
 * other without a gap.  What lies past K is zero, codes and scales.
 *
 * Quantisation of a block with largest magnitude m (x as float32, E4M3 times
 * its scale as one float32 product):
 *   e    = max(floor(log2 m) - 2, -127), s = e + 127 (m = 0: s = 0)
 *   code = x 2^-e rounded to the nearest magnitude, ties to the even code,
 *          over 6 to 6; the sign of x, of zeros too
 *   a block that holds an infinity or NaN: s = 255, codes 0
 *
 *   linear:      y[t][n]  = sum_k x[t][k] * w[n][k] + bias[n]
 *   input_grad:  dx[t][k] = sum_n dy[t][n] * w[n][k]
 * Products are exact, sums are held in float32, and each result is rounded
 * once.  Widened weights are exact in bfloat16.  A block's power of two need not fit
 * float16: with float16 x the sums of one block at a time are scaled, in float32,
 * as they are added, and float16 dy enters as two bfloat16, exactly.  Magnitudes of
 * 2^128 and more, which quantisation never stores, are infinite in bfloat16: beside
 * bfloat16 x or dy, and in an expert layer, the results that they reach are infinite
 * or NaN.  (Beside float16 dy they count as they are.)
 *
 *   route: the `top` largest of a token's E logits, largest first, of equal
 *          ones the lowest expert (NaN counts as the largest); an expert with
 *          logit -inf is never chosen, and where fewer than `top` are left the
 *          ids are -1 and the weights 0.  With v the chosen logits:
 *            softmax:  p = exp(v - max)     sigmoid:  p = 1 / (1 + exp(-v))
 *          weight = scale * p / sum of the chosen p (normalise), else
 *          scale * p / sum of exp(v - max) over all experts, or scale * p.
 *   moe:   for each token t and choice j with expert e = ids[t][j] in [0, E)
 *            a = gate_scale[e] * (gate[e] x[t]),  b = up_scale[e] * (up[e] x[t])
 *            h = a / (1 + exp(-a)) * b
 *            y[t] = sum over j of weights[t][j] * down_scale[e] * (down[e] h)
 *          Other ids add nothing.  h is a float32 and enters its product with
 *          all of its 24 bits.  The same expert may be named twice.
 * The order of every sum is fixed: the same call gives the same bits.
 * ------------------------------------------------------------------------
 * Conventions as in ecf8a.h: ECF8_OK or a negative ECF8_ERR_*; the caller owns
 * every buffer, device pointers unless said otherwise; a hipStream_t is passed
 * as void* and every call is asynchronous on it; return codes cover argument
 * checks and launch errors; nothing is allocated, copied or kept between
 * calls, so every call can be captured into a graph.  Workspaces are scratch
 * of one call: calls that may overlap in time need one each (256-byte
 * aligned).  Results must not overlap what the call reads.  The kernels run on
 * the current device, which must be the buffers' and the stream's.
 */
#ifndef ECF8X_H
#define ECF8X_H

#include <stdint.h>

#include "ecf8a.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types: ECF8A_BF16, ECF8A_FP16, ECF8A_FP32, ECF8A_E4M3, and */
#define ECF8X_MX4 5

#define ECF8X_BLOCK 32                  /* values of one scale */
#define ECF8X_PITCH 128                 /* stored rows are whole multiples of this many values */
#define ECF8X_MAX_ROWS 1073741824ull    /* 2^30 */
#define ECF8X_MAX_EXPERTS 1024
#define ECF8X_MAX_TOP 32
#define ECF8X_MAX_PAIRS 512             /* tokens * top of ecf8x_moe */

/* A matrix in 4 bits, or a stack of `experts` E4M3 ones: */
typedef struct {
    const uint8_t* codes;    /* 4-bit codes, 16-byte aligned; ECF8A_E4M3: the bytes */
    const uint8_t* scales;   /* the blocks' scale bytes, 4-byte aligned; ECF8A_E4M3: NULL */
    const float* factors;    /* ecf8x_moe: one float32 an expert, or NULL for 1 */
} ecf8x_matrix;

/* ------------------------------ conversion ----------------------------- */

/* x (rows x cols, ld_x elements between rows, aligned to its elements) of type
 * ECF8A_BF16, ECF8A_FP16, ECF8A_FP32 or ECF8A_E4M3; x_scale: one float32 for
 * E4M3 (NULL: 1), else NULL.  codes 16-byte, scales 4-byte aligned.
 * Errors: ECF8_ERR_UNSUPPORTED (type), ECF8_ERR_SIZE (rows or cols past their
 * limits, cols not a multiple of 32, ld_x < cols), ECF8_ERR_ARG (NULL,
 * misaligned), ECF8_ERR_HIP. */
int ecf8x_quantize(const void* x, uint64_t ld_x, uint32_t type, const float* x_scale, uint64_t rows, uint64_t cols,
                   uint8_t* codes, uint8_t* scales, void* hip_stream);

/* The values (exact in float32, and in bfloat16 but for magnitudes that it
 * rounds to infinity; rounded in float16), rows ld_out elements apart, 16-byte
 * aligned with ld_out a multiple of 8.  Errors as ecf8x_quantize. */
int ecf8x_dequantize(const uint8_t* codes, const uint8_t* scales, uint64_t rows, uint64_t cols, uint32_t type, void* out,
                     uint64_t ld_out, void* hip_stream);

/* ------------------------------- products ------------------------------ */

/* Workspace bytes of ecf8x_linear (x_type: ECF8A_BF16, ECF8A_FP16 or
 * ECF8X_MX4); 0 where it needs none or refuses the sizes. */
uint64_t ecf8x_linear_bytes(uint64_t tokens, uint64_t out_features, uint64_t in_features, uint32_t x_type);

/* y = x w^T + bias.  x: ECF8A_BF16 or ECF8A_FP16, rows ld_x elements apart on
 * 16-byte borders, x_scales NULL, and y of the same type; or ECF8X_MX4 codes
 * with their x_scales (ld_x unused).  w: (out_features x in_features) in 4
 * bits.  bias: out_features values of y's type (y_type: ECF8A_BF16 or
 * ECF8A_FP16) or NULL.  y: rows ld_y elements apart, aligned to its elements.
 * in_features: a multiple of 32; any number of tokens and out_features within
 * ecf8a.h's limits; ld_x up to 2^22 (offsets inside a tile have 32 bits).
 * Errors: ECF8_ERR_UNSUPPORTED (types), ECF8_ERR_SIZE, ECF8_ERR_ARG,
 * ECF8_ERR_WORKSPACE, ECF8_ERR_HIP. */
int ecf8x_linear(const void* x, const uint8_t* x_scales, uint64_t ld_x, uint32_t x_type, uint64_t tokens, uint64_t out_features,
                 uint64_t in_features, const ecf8x_matrix* w, const void* bias, uint32_t y_type, void* y, uint64_t ld_y,
                 void* workspace, uint64_t workspace_bytes, void* hip_stream);

uint64_t ecf8x_input_grad_bytes(uint64_t tokens, uint64_t out_features, uint64_t in_features, uint32_t type);

/* dx = dy w, dy (tokens x out_features) and dx (tokens x in_features) of one
 * type (ECF8A_BF16 or ECF8A_FP16), rows on 16-byte borders, ld_dy up to 2^22.
 * Errors as ecf8x_linear. */
int ecf8x_input_grad(const void* dy, uint64_t ld_dy, uint32_t type, uint64_t tokens, uint64_t out_features, uint64_t in_features,
                     const ecf8x_matrix* w, void* dx, uint64_t ld_dx, void* workspace, uint64_t workspace_bytes,
                     void* hip_stream);

/* -------------------------- mixture of experts ------------------------- */

#define ECF8X_SOFTMAX 0
#define ECF8X_SIGMOID 1

/* logits (tokens x experts) of type ECF8A_FP32, ECF8A_BF16 or ECF8A_FP16, rows
 * ld elements apart; ids and weights: tokens x top.  1 <= top <= experts,
 * top <= ECF8X_MAX_TOP, experts <= ECF8X_MAX_EXPERTS.  Errors:
 * ECF8_ERR_UNSUPPORTED (type, score), ECF8_ERR_SIZE, ECF8_ERR_ARG,
 * ECF8_ERR_HIP. */
int ecf8x_route(const void* logits, uint64_t ld, uint32_t type, uint64_t tokens, uint32_t experts, uint32_t top, uint32_t score,
                uint32_t normalise, float scale, int32_t* ids, float* weights, void* hip_stream);

/* An expert layer: gate and up (experts x inner x features), down (experts x
 * features x inner), all of type ECF8A_E4M3 (features and inner multiples of
 * 16) or ECF8X_MX4 (multiples of 32, factors NULL). */
typedef struct {
    ecf8x_matrix gate, up, down;
    uint64_t features, inner;
    uint32_t experts, type;
} ecf8x_experts;

/* Workspace bytes of ecf8x_moe; 0 for sizes that it refuses, or no pairs. */
uint64_t ecf8x_moe_bytes(uint64_t tokens, uint32_t top, const ecf8x_experts* layer);

/* x (tokens x features) and y of one type (ECF8A_BF16 or ECF8A_FP16), rows of x
 * on 16-byte borders, y's aligned to its elements; ids and weights tokens x top,
 * contiguous; tokens * top <= ECF8X_MAX_PAIRS; features and inner up to 65536,
 * ld_x up to 2^21.  Two launches.  Errors as ecf8x_linear. */
int ecf8x_moe(const void* x, uint64_t ld_x, uint32_t type, uint64_t tokens, uint32_t top, const int32_t* ids, const float* weights,
              const ecf8x_experts* layer, void* y, uint64_t ld_y, void* workspace, uint64_t workspace_bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif

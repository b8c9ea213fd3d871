/*
 * ecf8a.h -- C ABI of libecf8 for what is adapted beside a compressed weight.
 *
 * A weight kept ECF8-compressed (ecf8.h) is frozen: it is decoded, multiplied
 * and never written.  What a user serves and trains next to it is a pair of
 * low-rank factors for each request or task, and this header holds the
 * operators that such a layer needs on AMD Instinct MI355X (gfx950):
 *   - the adapters of many requests added to the shared projection's output,
 *     from one token to long prompts (ecf8a_plan_prepare, ecf8a_add; ecf8a_add_few);
 *   - their gradients (ecf8a_grads);
 *   - the gradient the frozen E4M3 weight passes to its input
 *     (ecf8a_input_grad);
 *   - the global norm of many gradients, and the gradients scaled to a largest
 *     norm (ecf8a_clip_prepare, ecf8a_clip_run).
 *
 * ------------------------------------------------------------------------
 * Formulas.  T tokens, K inputs, N outputs, L adapters of up to R rows.  Token
 * t has adapter a = index[t]; an index outside [0, L) means none.  Row r of
 * adapter a takes part if r < ranks[a] (ranks NULL: every r < R; a value
 * outside [0, R] counts as the nearer of the two).
 *   h[t][r]      = scaling[a] * x_scale * sum_k x[t][k] * down[a][r][k]
 *   out[t][n]    = base[t][n] + sum_r h[t][r] * up[a][r][n]
 *   z[t][r]      = scaling[a] * sum_n dy[t][n] * up[a][r][n]
 *   dx[t][k]     = dx_base[t][k] + sum_r z[t][r] * down[a][r][k]
 *   d_down[a][r][k] = sum over a's tokens of z[t][r] * x[t][k]
 *   d_up[a][r][n]   = sum over a's tokens of h[t][r] * dy[t][n]
 *   input_grad:  dx[t][k] = w_scale * sum_n dy[t][n] * e4m3(w[n][k])
 *   clip:        norm = sqrt(sum of g^2 over every tensor)
 *                out  = g * min(1, max_norm / (norm + 1e-6))
 * Both factors are stored by rank row, down as (L, R, K) and up as (L, R, N),
 * so that the forward and the backward pass read either one the same way.
 * Products are exact and summed in float32 (the clip's squares in float64),
 * and each output is rounded once.  h and z, which are such sums, enter the
 * products that they are part of (out, dx, d_down, d_up) as two bfloat16, with
 * 16 significant bits: each term of those sums is off by up to 2^-16 of its
 * magnitude (float16 factors and rows: 2^-15, since of four partial products
 * the smallest is left out), far below the rounding of the result but for sums
 * whose terms cancel.  The order of every sum is fixed: the same call gives
 * the same bits.
 * ------------------------------------------------------------------------
 * Conventions as in ecf8.h: ECF8_OK or a negative ECF8_ERR_*; the caller owns
 * every buffer, device pointers unless said otherwise; a hipStream_t is passed
 * as void* and every call is asynchronous on it; return codes cover argument
 * checks and launch errors; nothing is allocated, copied or kept between
 * calls, so every call but ecf8a_clip_prepare can be captured into a graph
 * (that one is called before the capture).  Workspaces are scratch of one
 * call: calls that may overlap in time need one each.  The kernels run on the
 * current device, which must be the buffers' and the stream's.
 */
#ifndef ECF8A_H
#define ECF8A_H

#include <stdint.h>

#include "ecf8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations, factors and gradients. */
#define ECF8A_BF16 1
#define ECF8A_FP16 2
#define ECF8A_FP32 3    /* ecf8a_clip_* only */
#define ECF8A_E4M3 4    /* x of ecf8a_add only */

#define ECF8A_MAX_ADAPTERS 2048
#define ECF8A_MAX_RANK 256
#define ECF8A_MAX_TOKENS 16777216       /* 2^24 */
#define ECF8A_FEW_TOKENS 512            /* of ecf8a_add_few */
#define ECF8A_FEW_RANK 64               /* of ecf8a_add_few */
#define ECF8A_MAX_FEATURES 1048576      /* 2^20 */

/* ------------------------------ adapters ------------------------------- */

/* The grouping of a batch's tokens by adapter (a host struct, filled by
 * ecf8a_plan_prepare; the grouping itself is in the workspace). */
typedef struct {
    void* workspace;
    uint64_t workspace_bytes;
    uint64_t tokens;
    uint32_t adapters;
    uint32_t max_slots;      /* bounds that hold for every index of this length: slots (tokens */
    uint32_t max_chunks;     /* sorted by adapter, each group padded to 16), chunks of at most 64 */
    uint32_t max_units;      /* slots of one adapter, and units of at most unit_slots */
    uint32_t unit_slots;
} ecf8a_plan;

/* Workspace bytes a plan of `tokens` tokens and `adapters` adapters needs
 * (256-byte aligned device memory, owned by the caller and kept as long as the
 * plan is used).  0 for sizes that ecf8a_plan_prepare refuses. */
uint64_t ecf8a_plan_bytes(uint64_t tokens, uint32_t adapters);

/* Groups the tokens of a batch by adapter: one launch.  index: device, `tokens`
 * values of index_bytes bytes each (4: int32, 8: int64; aligned to their size),
 * read by the launch only.  A plan serves every projection that the batch
 * passes through, and any number of calls; calls on another stream must be
 * ordered after this one.
 * Errors: ECF8_ERR_ARG (NULL, misaligned, index_bytes), ECF8_ERR_SIZE (tokens
 * or adapters past their limits, adapters 0), ECF8_ERR_WORKSPACE,
 * ECF8_ERR_HIP. */
int ecf8a_plan_prepare(const void* index, uint32_t index_bytes, uint64_t tokens, uint32_t adapters,
                       void* workspace, uint64_t workspace_bytes, void* hip_stream, ecf8a_plan* plan);

/* A bank of adapters: contiguous factors of one type (ECF8A_BF16 or
 * ECF8A_FP16), aligned to their elements; scaling and ranks on the device. */
typedef struct {
    const void* down;        /* (adapters, rank, in_features) */
    const void* up;          /* (adapters, rank, out_features) */
    const float* scaling;    /* (adapters) */
    const int32_t* ranks;    /* (adapters) or NULL */
    uint64_t in_features;
    uint64_t out_features;
    uint32_t adapters;
    uint32_t rank;
    uint32_t type;
    uint32_t reserved;
} ecf8a_bank;

/* Bytes of the hidden buffer (the h of one ecf8a_add, in the plan's order,
 * 16-byte aligned) that carries h from a forward call to its gradients. */
uint64_t ecf8a_hidden_bytes(const ecf8a_plan* plan, uint32_t rank);

/* Workspace bytes of ecf8a_add (0: none is used), and of ecf8a_grads (256-byte
 * aligned). */
uint64_t ecf8a_add_bytes(const ecf8a_plan* plan, const ecf8a_bank* bank);
uint64_t ecf8a_grads_bytes(const ecf8a_plan* plan, const ecf8a_bank* bank);

/* out = base + the adapters' part (see the formulas).  x: tokens rows of
 * in_features values of x_type (the bank's type, or ECF8A_E4M3 with *x_scale;
 * x_scale NULL is 1), ldx elements apart; base and out: rows of out_features
 * values of the bank's type, ld_base and ld_out elements apart; base NULL is 0.
 * out may be base itself with the same spacing (rows without an adapter are
 * then not touched), and must not overlap any input otherwise.  Nothing but
 * the out_features values of each row is written.  hidden: NULL, or a buffer
 * of ecf8a_hidden_bytes that receives h for ecf8a_grads.
 * Errors: ECF8_ERR_ARG (NULL, misaligned, a plan of other adapters),
 * ECF8_ERR_SIZE (limits, a spacing below the row), ECF8_ERR_UNSUPPORTED
 * (types), ECF8_ERR_WORKSPACE, ECF8_ERR_HIP. */
int ecf8a_add(const ecf8a_plan* plan, const ecf8a_bank* bank, const void* x, uint64_t ldx, uint32_t x_type,
              const float* x_scale, const void* base, uint64_t ld_base, void* out, uint64_t ld_out,
              void* hidden, void* workspace, uint64_t workspace_bytes, void* hip_stream);

/* Whether ecf8a_add_few takes this many tokens and this bank (1: at most
 * ECF8A_FEW_TOKENS tokens and rank ECF8A_FEW_RANK) or a plan and ecf8a_add are
 * needed (0). */
int ecf8a_few(uint64_t tokens, const ecf8a_bank* bank);

/* Workspace bytes of ecf8a_add_few (256-byte aligned; 0: none is used). */
uint64_t ecf8a_add_few_bytes(uint64_t tokens, const ecf8a_bank* bank);

/* ecf8a_add for few tokens, from the index itself (as in ecf8a_plan_prepare)
 * without a plan: one or two launches.  Errors as ecf8a_plan_prepare and
 * ecf8a_add. */
int ecf8a_add_few(const void* index, uint32_t index_bytes, uint64_t tokens, const ecf8a_bank* bank, const void* x,
                  uint64_t ldx, uint32_t x_type, const float* x_scale, const void* base, uint64_t ld_base,
                  void* out, uint64_t ld_out, void* workspace, uint64_t workspace_bytes, void* hip_stream);

/* The gradients of ecf8a_add for dy, the gradient of out (which is base's own
 * gradient too).  dy, x, dx_base and dx: rows of the bank's type; hidden: what
 * ecf8a_add wrote for the same x, plan and bank, or NULL to compute it again.
 * dx (NULL: not wanted) = dx_base (NULL: 0) + the adapters' part, under
 * ecf8a_add's rules for base and out.  d_down and d_up (both NULL: not wanted):
 * contiguous, shaped and typed as the factors, wholly written: zero for
 * adapters without a token and rows that take no part.
 * Errors as ecf8a_add. */
int ecf8a_grads(const ecf8a_plan* plan, const ecf8a_bank* bank, const void* dy, uint64_t ld_dy,
                const void* x, uint64_t ldx, const void* hidden, const void* dx_base, uint64_t ld_dx_base,
                void* dx, uint64_t ld_dx, void* d_down, void* d_up, void* workspace,
                uint64_t workspace_bytes, void* hip_stream);

/* ------------------- the frozen weight's input gradient ----------------- */

/* Workspace bytes of ecf8a_input_grad for these sizes (256-byte aligned). */
uint64_t ecf8a_input_grad_bytes(uint64_t tokens, uint64_t out_features, uint64_t in_features);

/* dx = w_scale * dy w, the gradient that y = x (w * w_scale)^T passes to x.
 * dy: tokens rows of out_features values of `type` (ECF8A_BF16 or ECF8A_FP16),
 * ld_dy elements apart (at most 2^22); w: out_features x in_features E4M3 bytes, contiguous
 * and 16-byte aligned (a decoded weight); w_scale: device float; dx: tokens
 * rows of in_features values of the same type, ld_dx elements apart.  Both
 * feature counts are multiples of 16, as the FP8 product of the forward pass
 * asks; rows of dy and dx are 16-byte aligned.  tokens 0: nothing is done.
 * Errors: ECF8_ERR_ARG (NULL, misaligned), ECF8_ERR_SIZE, ECF8_ERR_UNSUPPORTED
 * (type), ECF8_ERR_WORKSPACE, ECF8_ERR_HIP. */
int ecf8a_input_grad(const void* dy, uint64_t ld_dy, uint64_t tokens, uint64_t out_features,
                     const uint8_t* w, uint64_t in_features, const float* w_scale, uint32_t type,
                     void* dx, uint64_t ld_dx, void* workspace, uint64_t workspace_bytes, void* hip_stream);

/* ----------------------- gradient norm and clipping --------------------- */

/* One gradient of a clip: n contiguous values at grad, and where the scaled
 * ones go (out = grad: in place). */
typedef struct {
    const void* grad;
    void* out;
    uint64_t n;
} ecf8a_grad;

/* A prepared clip (host struct, filled by ecf8a_clip_prepare). */
typedef struct {
    void* workspace;
    uint64_t workspace_bytes;
    uint64_t pieces;
    uint32_t count;
    uint32_t type;
    uint32_t grid;
    uint32_t in_place;       /* 1: every out is its grad */
} ecf8a_clip_plan;

/* Workspace bytes of a clip over these gradients (256-byte aligned device
 * memory, kept as long as the plan is used; grads on the host).  0 for what
 * ecf8a_clip_prepare refuses. */
uint64_t ecf8a_clip_bytes(const ecf8a_grad* grads, uint32_t count);

/* Checks the gradients (host array, read during the call only; each device
 * pointer aligned to its element; type ECF8A_BF16, ECF8A_FP16 or ECF8A_FP32
 * for all) and puts their list into the workspace with one host-to-device copy
 * on hip_stream.  No grad or out may overlap another tensor's, and a grad that
 * is not its own out must not overlap it.  The plan stays valid while the
 * workspace and the tensors do.  hip_stream must not be being captured: the
 * copy reads a list that is gone when this returns.
 * Errors: ECF8_ERR_ARG (NULL with n > 0, misaligned, overlapping, a stream
 * that is being captured), ECF8_ERR_UNSUPPORTED (type), ECF8_ERR_SIZE,
 * ECF8_ERR_WORKSPACE, ECF8_ERR_HIP. */
int ecf8a_clip_prepare(const ecf8a_grad* grads, uint32_t count, uint32_t type, void* workspace,
                       uint64_t workspace_bytes, void* hip_stream, ecf8a_clip_plan* plan);

/* norm = the norm of all gradients (device float, overwritten; inf or NaN if
 * the gradients hold one), and every out = grad * min(1, max_norm / (norm +
 * 1e-6)): two launches.  A NaN norm makes every output NaN, an infinite one
 * makes finite values 0.  Gradients in place are not written where the factor
 * is 1.  Runs of one plan must not overlap in time.
 * Errors: ECF8_ERR_ARG (NULL, max_norm negative or NaN), ECF8_ERR_HIP. */
int ecf8a_clip_run(const ecf8a_clip_plan* plan, float max_norm, float* norm, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* ECF8A_H */

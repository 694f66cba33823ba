/*
 * mok_ops.h -- operators around the expert layer of mok.h (included by it): the token sort
 * on its own, a linear layer for one matrix or one per expert, the optimizer step, a router with
 * scores, bias and groups, layer and RMS norms, and the loss over a vocabulary.
 *
 * The conventions of mok.h hold: device pointers owned by the caller and 16-byte aligned,
 * row-major; scratch from the caller's workspace; asynchronous on `stream`; arguments
 * validated on the host before anything is enqueued; problems the GPU finds recorded in the
 * device status word; bitwise identical results run to run; compute capability 10.3 only.
 * Unlike the layer's own arrays, rows here may be strided: a leading dimension (ld_*) is the
 * distance between consecutive rows in elements.
 */
#ifndef MOK_OPS_H
#define MOK_OPS_H

#include "mok.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mok_dtype { MOK_DTYPE_BF16 = 0, MOK_DTYPE_F32 = 1 } mok_dtype;

/* ---- tokens sorted by expert, and back ------------------------------------------------
 *
 * A row map gives each routed id f = t*K + k its row in an expert-sorted array: expert e owns
 * rows [starts[e], starts[e+1]), its kept[e] real rows first, in ascending f, and zero rows up
 * to the next multiple of 16 (so a group of rows fills whole tensor-core steps). An id whose
 * rank among its expert's rows is `capacity` or more is dropped: its map entry is -1, it
 * takes part in nothing and its gradients are zero. Any other map works as well: every entry
 * is -1 or a row of its own below n_rows; an entry at or past n_rows raises
 * MOK_ERR_DEVICE_INVARIANT and is treated as dropped.
 *
 * Shapes: T tokens (T >= 0), 1 <= K <= 32 experts per token, 1 <= E <= 1024 experts,
 * 1 <= H <= 2^24 columns, any number; H <= ld_tok, ld_row <= 2^30; T*K, n_rows < 2^31. Columns
 * past H of a row are neither read nor written. Rows are copied 16 bytes at a time where both ld are multiples of
 * 16 bytes, else element by element. */
typedef struct mok_rows_config {
    uint32_t abi_version; /* MOK_ABI_VERSION */
    int32_t T, K, E, H;
    int32_t dtype;    /* mok_dtype of tokens and rows */
    int32_t capacity; /* rows kept per expert; 0: all */
    int32_t reserved; /* 0 */
    int64_t n_rows;   /* rows of the sorted arrays; T*K + 15*min(E, T*K) always suffices */
    int64_t ld_tok;   /* row stride of token arrays (x, y, dy, dx, residual) */
    int64_t ld_row;   /* row stride of sorted arrays (xs, rows, drows, dxs) */
} mok_rows_config;

mok_status mok_check_rows_config(const mok_rows_config *cfg);

/* The row map of a schedule (mok_build_schedule; its counts, offsets and inv are read, the
 * other arrays may be NULL).
 *   topk_idx [T][K]; row_map [T*K] int32 out; starts [E+1] int32 out; kept [E] int32 out.
 * An expert id out of range, or a rank outside its expert's count (the schedule is of other ids),
 * maps to -1 and raises MOK_ERR_DEVICE_INVARIANT, as does starts[E] > n_rows. */
mok_status mok_build_row_map(const mok_rows_config *cfg, const int32_t *topk_idx,
                             const mok_schedule *sched, int32_t *row_map, int32_t *starts,
                             int32_t *kept, cudaStream_t stream);

/* xs[row_map[t*K + k]] = x[t], bit for bit. With starts and kept (both or neither), the rows
 * kept[e] .. of each expert up to the next multiple of 16 are set to zero; other rows are left
 * alone. */
mok_status mok_dispatch(const mok_rows_config *cfg, const void *x, const int32_t *row_map,
                        const int32_t *starts, const int32_t *kept, void *xs,
                        cudaStream_t stream);

/* The gradient of mok_dispatch: dx[t] = sum over k = 0..K-1, in that order, of
 * dxs[row_map[t*K + k]] in fp32, rounded once. */
mok_status mok_dispatch_backward(const mok_rows_config *cfg, const void *dxs,
                                 const int32_t *row_map, void *dx, cudaStream_t stream);

/* y[t] = residual[t] + sum over k, in order, of topk_w[t][k] * rows[row_map[t*K + k]], in fp32,
 * rounded once. topk_w fp32 [T][K], or NULL for weights of one; residual NULL or [T] rows
 * (may be y itself). rows must not overlap y. */
mok_status mok_combine(const mok_rows_config *cfg, const void *rows, const int32_t *row_map,
                       const float *topk_w, const void *residual, void *y,
                       cudaStream_t stream);

/* The gradients of mok_combine, with r = row_map[t*K + k]:
 *   drows[r] = topk_w[t][k] * dy[t], rounded once (zero rows as in mok_dispatch);
 *   d_topk_w[t][k] = <rows[r], dy[t]> in fp32, in a fixed order (0 where dropped, whatever dy
 *   holds).
 * The residual's gradient is dy. Either output may be NULL (then rows is not read where
 * d_topk_w is NULL and may be NULL too), not both. drows must not overlap rows. */
mok_status mok_combine_backward(const mok_rows_config *cfg, const void *dy, const void *rows,
                                const int32_t *row_map, const int32_t *starts,
                                const int32_t *kept, const float *topk_w, void *drows,
                                float *d_topk_w, cudaStream_t stream);

/* ---- linear layer, for one matrix or one per group of rows ----------------------------
 *
 *   z = x W^T + b        y = act(z) + residual
 *
 * x [rows][in], W [groups][out][in], b [groups][out]; products in bf16 operands with fp32
 * accumulation, everything after in fp32, rounded once. Two forms:
 *  - dense: groups == 1, starts and counts NULL: every row takes W[0];
 *  - grouped: group g owns rows [starts[g], starts[g] + counts[g]) (int32 device arrays; starts
 *    [groups+1] are multiples of 16, as mok_build_row_map makes them, starts[g+1] at or past
 *    starts[g] + counts[g], starts[groups] <= rows). The rows from there to the next multiple
 *    of 16 are padding: written as zeros in y, z and dx, and read (as zeros) in x and, without
 *    an activation, dy by the weight gradient, so they must hold zeros there, as mok_dispatch
 *    and mok_combine_backward write them. Rows past that are neither read nor written. A group
 *    that breaks these rules, or begins before the rows and padding of an earlier group end,
 *    raises MOK_ERR_DEVICE_INVARIANT and counts as empty.
 *
 * Activations: none; relu; silu z sigma(z); gelu_tanh 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715
 * z^3))); gelu 0.5 z (1 + erf(z / sqrt 2)). They and their slopes are computed to within
 * 2^-20 (1 + |z|); for finite z far from zero the slopes are 0 or 1.
 *
 * Limits: 1 <= groups <= 1024, 1 <= in_features, out_features <= 2^20 (any number, odd ones
 * among them), 0 <= rows < 2^31 - 512, fewer than 2^31 blocks of 16 rows x 256 columns in an
 * output (x, y or all of dW); strides ld_in >= in, ld_w >= in, ld_out >= out are
 * multiples of 8 elements, at most 2^30. Columns past a matrix's width are neither read nor written. */
typedef enum mok_activation {
    MOK_ACT_NONE = 0,
    MOK_ACT_RELU = 1,
    MOK_ACT_SILU = 2,
    MOK_ACT_GELU_TANH = 3,
    MOK_ACT_GELU = 4
} mok_activation;

typedef struct mok_linear_config {
    uint32_t abi_version; /* MOK_ABI_VERSION */
    int32_t groups;
    int32_t in_features, out_features;
    int64_t rows;       /* rows of x, y, z, dy, dx */
    int64_t ld_in;      /* row stride of x and dx */
    int64_t ld_w;       /* row stride of W and dW (a group is out_features rows) */
    int64_t ld_out;     /* row stride of y, z, residual and dy */
    int32_t act;        /* mok_activation */
    int32_t out_dtype;  /* mok_dtype of y and dy */
    int32_t grad_dtype; /* mok_dtype of dx and dW */
    int32_t reserved;   /* 0 */
} mok_linear_config;

typedef enum mok_linear_pass { MOK_LINEAR_FORWARD = 0, MOK_LINEAR_BACKWARD = 1 } mok_linear_pass;

mok_status mok_check_linear_config(const mok_linear_config *cfg);

/* Bytes of workspace of a pass (256-byte aligned, contents on entry do not matter); 0 for an
 * invalid configuration. */
size_t mok_linear_workspace_size(const mok_linear_config *cfg, int pass);

/* Forward. A sum over many inputs runs on the tensor cores 1024 of them at a time where y is
 * fp32, and the runs are added in fp32: y is then within about 1e-6 of its norm.
 * x, w bf16; bias NULL or fp32; residual NULL or [rows][out] bf16 (may be y where y
 * is bf16); y [rows][out]; z NULL or [rows][out] bf16 out: the value before the activation,
 * which the backward needs where there is one. */
mok_status mok_linear_forward(const mok_linear_config *cfg, const void *x, const void *w,
                              const float *bias, const void *residual, const int32_t *starts,
                              const int32_t *counts, void *y, void *z, void *ws,
                              size_t ws_bytes, cudaStream_t stream);

/* Backward, with dz = dy act'(z) (relu'(0) = 0):
 *   dx = dz W        dW[g] = sum over the group's rows of dz^T x        db[g] = sum of dz
 * How dz enters the products follows the gradients' type (it is exact where there is no activation
 * and dy is bf16):
 *   bf16 gradients: rounded to bf16, as the gradients are themselves. Their error is then 2.3e-3
 *     of their norm, where rounding the results alone gives 1.7e-3;
 *   fp32 gradients: as two bf16 values that add up to within 2^-17 of it, and sums run in
 *     segments of 1024 terms that are added in fp32: 2.6e-6 of the norm (1.0e-6 where dz is
 *     exact), for twice the matrix work.
 * db is the fp32 sum of the unrounded dz in a fixed order. The residual's gradient is dy.
 *   z    [rows][out] bf16 from the forward, or NULL without an activation
 *   dx   NULL or [rows][in] out; dw NULL or [groups][out][in] out (zero for an empty group);
 *   db   NULL or [groups][out] fp32 out. At least one of the three. */
mok_status mok_linear_backward(const mok_linear_config *cfg, const void *x, const void *w,
                               const void *z, const void *dy, const int32_t *starts,
                               const int32_t *counts, void *dx, void *dw, float *db, void *ws,
                               size_t ws_bytes, cudaStream_t stream);

/* ---- AdamW step over many tensors ---------------------------------------------------
 *
 * For every element, with g scaled by *grad_scale (NULL: one) and t = step:
 *   m = beta1 m + (1 - beta1) g          v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * in fp32; p, m and v are then stored in their own types, the update itself using the
 * unrounded m and v. `copy` (NULL, or bf16; only with fp32 parameters) receives p rounded to
 * nearest even: the weights the layer's kernels read.
 *
 * MOK_STATE_F32: m and v are fp32 arrays.
 * MOK_STATE_MXFP8: m and sqrt(v) are E4M3 codes with one E8M0 scale per 32 consecutive
 *   elements (m_scale, v_scale: [ceil(n/32)] bytes), 33/32 bytes per element and state. The
 *   scale is the least power of two (at least 2^-127) that brings the block's largest magnitude
 *   to 448 or less, so nothing saturates; a sqrt(v) above zero is never stored as zero (the
 *   least code instead), so m is never divided by eps alone. A block that holds an infinity
 *   or a NaN gets scale byte 255 and reads back as NaN. All-zero bytes are the zero state.
 *
 * Rounding: to nearest even; with MOK_ADAMW_STOCHASTIC the 8-bit states and bf16 parameters are
 * rounded up or down with probability proportional to the distance, so that changes smaller
 * than a step (sqrt(v) moves by 1/2000 of itself at beta2 = 0.999, E4M3 steps are 1/16 or more) are
 * kept on average. It is m and sqrt(v) whose mean is kept: their rounding spreads sqrt(v) by some
 * 15% from element to element, and v, its square, gains that variance: 2% (beta2 = 0.9) to 5%
 * (0.999) above the fp32 state's mean in a simulation of unit normal gradients. The random bits are a function of the seed and the element's number alone:
 * with the tensors numbered one after another, each beginning at the next multiple of 32,
 * element i gets h = mix(lo32(i) ^ mix(mix(hi32(i) ^ lo32(seed)) ^ hi32(seed))), mix being
 * h ^= h>>16, h *= 0x85EBCA6B, h ^= h>>13, h *= 0xC2B2AE35, h ^= h>>16 (the MurmurHash3
 * finaliser). m takes h's low 16 bits, sqrt(v) its high 16, a bf16 p the high 16 of
 * mix(h + 0x9E3779B9). Give every step its own seed. */
typedef enum mok_adamw_state { MOK_STATE_F32 = 0, MOK_STATE_MXFP8 = 1 } mok_adamw_state;
#define MOK_ADAMW_STOCHASTIC 1u

typedef struct mok_adamw_config {
    uint32_t abi_version;     /* MOK_ABI_VERSION */
    int32_t p_dtype, g_dtype; /* mok_dtype of parameters and gradients */
    int32_t state;            /* mok_adamw_state */
    uint32_t flags;           /* MOK_ADAMW_* */
    int32_t step;             /* t >= 1 */
    double lr, beta1, beta2, eps;
    uint64_t seed;
} mok_adamw_config;

typedef struct mok_adamw_tensor {
    void *p;       /* [n], in and out */
    void *copy;    /* NULL or [n] bf16 out */
    const void *g; /* [n] */
    void *m, *v;   /* [n] fp32, or E4M3 codes of m and sqrt(v), in and out */
    uint8_t *m_scale, *v_scale; /* [ceil(n/32)] E8M0, in and out (MXFP8 states; else NULL) */
    int64_t n;     /* elements, >= 0 */
    double weight_decay;
} mok_adamw_tensor;

/* lr, eps >= 0, 0 <= beta < 1, weight_decay finite. Host only. */
mok_status mok_check_adamw_config(const mok_adamw_config *cfg);

/* One step over `n_tensors` tensors (a host array, read before the call returns). The arrays
 * of one call must not overlap. grad_scale: NULL or a device float (a clipping coefficient
 * or an inverse loss scale, computed on the GPU without a host round trip). */
mok_status mok_adamw_step(const mok_adamw_config *cfg, const mok_adamw_tensor *tensors,
                          int32_t n_tensors, const float *grad_scale, cudaStream_t stream);

/* The step for programs that capture it in a CUDA graph and replay it. mok_adamw_step takes
 * step, lr and seed from the host, so a replayed graph would repeat one step's bias correction
 * and random bits; here they are in device memory, 16-byte aligned, and move with each replay.
 * Once per step mok_adamw_advance adds one to clock->step and fills in what follows from it
 * (cfg's betas); mok_adamw_step_at then updates a list of tensors (as often as there are lists)
 * with that step, clock->lr, and the seed cfg->seed + clock->step * clock->seed_stride. cfg's
 * step and lr have to be valid but are not used. A step below one, or an lr that is negative or
 * not finite, raises MOK_ERR_DEVICE_INVARIANT and leaves the parameters as they are. */
typedef struct mok_adamw_clock {
    int64_t step;         /* steps taken */
    uint64_t seed_stride; /* what the seed moves by from step to step */
    double lr;
    float step_lr, step_size, inv_root; /* lr, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t): of the
                                           step, written by mok_adamw_advance */
    float reserved;
} mok_adamw_clock;

mok_status mok_adamw_advance(const mok_adamw_config *cfg, mok_adamw_clock *clock,
                             cudaStream_t stream);
mok_status mok_adamw_step_at(const mok_adamw_config *cfg, const mok_adamw_tensor *tensors,
                             int32_t n_tensors, const mok_adamw_clock *clock,
                             const float *grad_scale, cudaStream_t stream);

/* ---- router ---------------------------------------------------------------------------
 *
 * mok_route_topk takes the largest logits and a softmax over them. Here the choice of experts and
 * their weights go by scores of all experts, a bias balances the experts' loads without a gradient,
 * and experts may come from a few groups only. For a token with logits l[0 .. E-1]:
 *   s = softmax(l) over all E, or sigmoid(l)              the scores
 *   c = s + bias                                          what the choice goes by
 *   groups > 1: group g holds experts g E/groups ..; its score is the sum of its group_top (1 or 2)
 *   largest c, and only the topk_groups groups of largest score are kept
 *   topk_idx  the K experts of largest c in the kept groups, c descending
 *   topk_w    scale * s of them, with `renormalize` divided by their sum
 * Ties, of experts and of groups, go to the lower id.
 *
 * The choice is that of exact arithmetic as far as 64 bits hold it: where two scores, or sums of
 * scores, are closer than 32 bits can tell, the token is done again in 64. Without a bias experts
 * are compared by their logits.
 *
 * A logit of -inf masks an expert out: its score is 0, it adds nothing to its group, and it is
 * chosen only where the kept groups have too few others (then the lowest ids, with weight 0); a
 * group of masked experts is kept only where there are too few others. A row of nothing else has
 * weights and gradients of 0. Logits of NaN or +inf give unspecified ids in range, each once, and
 * unspecified weights and gradients of that token. Bias values are finite.
 *
 * Limits: T >= 0, 1 <= E <= 1024, 1 <= K <= min(32, topk_groups E / groups), 1 <= topk_groups <=
 * groups <= 32, groups divides E, T K < 2^31; E <= ld <= 2^30, any number. Columns past E of a row are
 * neither read nor written. */
typedef enum mok_score { MOK_SCORE_SOFTMAX = 0, MOK_SCORE_SIGMOID = 1 } mok_score;

typedef struct mok_router_config {
    uint32_t abi_version; /* MOK_ABI_VERSION */
    int32_t T, E, K;
    int32_t dtype;       /* mok_dtype of logits and d_logits */
    int32_t score;       /* mok_score */
    int32_t groups;      /* 1: every expert may be chosen */
    int32_t topk_groups; /* groups kept */
    int32_t group_top;   /* experts whose c make a group's score: 1 or 2 */
    int32_t renormalize; /* 0 or 1 */
    float scale;         /* finite, above 0 */
    int32_t reserved;    /* 0 */
    int64_t ld;          /* row stride of logits and d_logits */
} mok_router_config;

mok_status mok_check_router_config(const mok_router_config *cfg);

/* Bytes of workspace of mok_router_forward where counts or score_sum are asked for (256-byte
 * aligned, contents on entry do not matter); 0 for an invalid configuration. */
size_t mok_router_workspace_size(const mok_router_config *cfg);

/* logits [T][E]; bias NULL or fp32 [E]; topk_idx [T][K] int32 out, topk_w [T][K] fp32 out.
 * counts NULL or [E] int32 out: tokens that chose each expert. score_sum NULL or [E] fp32 out: the
 * sum over all tokens of each expert's score, in a fixed order (times counts it makes a balance
 * loss). ws may be NULL where both are. */
mok_status mok_router_forward(const mok_router_config *cfg, const void *logits, const float *bias,
                              int32_t *topk_idx, float *topk_w, int32_t *counts, float *score_sum,
                              void *ws, size_t ws_bytes, cudaStream_t stream);

/* d_logits = the gradient of sum(d_topk_w topk_w) + sum(d_score_sum score_sum) for the chosen
 * topk_idx (the bias has none), rounded once; zero for masked experts. d_topk_w fp32 [T][K];
 * d_score_sum NULL or fp32 [E]. An id out of range raises MOK_ERR_DEVICE_INVARIANT and takes no part.
 * d_logits may be logits itself. */
mok_status mok_router_backward(const mok_router_config *cfg, const void *logits,
                               const int32_t *topk_idx, const float *d_topk_w,
                               const float *d_score_sum, void *d_logits, cudaStream_t stream);

/* new_bias[e] = bias[e] + rate * sign(T K / E - counts[e]): up for an expert that fewer than an
 * average number of tokens chose. rate finite; new_bias may be bias. */
mok_status mok_router_update_bias(const mok_router_config *cfg, const int32_t *counts, float rate,
                                  const float *bias, float *new_bias, cudaStream_t stream);

/* ---- layer norm and RMS norm ----------------------------------------------------------
 *
 *   h = x + residual (rounded to its type)
 *   MOK_NORM_LAYER: mean = mean(h), rstd = 1 / sqrt(mean((h - mean)^2) + eps)
 *   MOK_NORM_RMS:   mean = 0,       rstd = 1 / sqrt(mean(h^2) + eps)
 *   y = (h - mean) rstd weight + bias
 * over each row, statistics of the rounded h, everything in fp32, each output rounded once.
 *
 * Limits: 0 <= rows < 2^31 - 512, 1 <= H <= 2^20 (any number); strides ld_x, ld_y >= H are multiples
 * of 8 elements, at most 2^30. Columns past H are neither read nor written. */
typedef enum mok_norm_kind { MOK_NORM_LAYER = 0, MOK_NORM_RMS = 1 } mok_norm_kind;

typedef struct mok_norm_config {
    uint32_t abi_version; /* MOK_ABI_VERSION */
    int32_t H;
    int64_t rows;
    int64_t ld_x;     /* row stride of x, residual, h, dh, dx */
    int64_t ld_y;     /* row stride of y, dy */
    int32_t kind;     /* mok_norm_kind */
    int32_t x_dtype;  /* mok_dtype of x, residual, h, dh, dx */
    int32_t y_dtype;  /* mok_dtype of y, dy */
    float eps;        /* finite, above 0 */
} mok_norm_config;

mok_status mok_check_norm_config(const mok_norm_config *cfg);

/* Bytes of workspace of mok_norm_backward where dw or db are asked for (256-byte aligned, contents on
 * entry do not matter); 0 for an invalid configuration. */
size_t mok_norm_workspace_size(const mok_norm_config *cfg);

/* x [rows][H]; residual NULL or [rows][H]; weight, bias NULL (one, zero) or fp32 [H]; h NULL or
 * [rows][H] out (with a residual; may be x or residual); y [rows][H] out (may be x or residual where
 * the types and strides are the same and h is another); mean, rstd NULL or fp32 [rows] out, for the backward
 * (mean of MOK_NORM_LAYER only). */
mok_status mok_norm_forward(const mok_norm_config *cfg, const void *x, const void *residual,
                            const float *weight, const float *bias, void *h, void *y, float *mean,
                            float *rstd, cudaStream_t stream);

/* Backward, with n = (h - mean) rstd and g = dy weight:
 *   dx = dh + rstd (g - n mean(g n) - mean(g))   (the last mean of MOK_NORM_LAYER only)
 *   dw = sum over the rows of dy n               db = sum of dy
 * in fp32, the sums over rows in a fixed order. It is the gradient of x and of the residual.
 *   h     [rows][H]: h, or x where there was no residual; mean (MOK_NORM_LAYER), rstd of the forward
 *   dh    NULL or [rows][H]: the gradient that reaches h beside the norm (may be dx)
 *   dx    NULL or [rows][H] out (may be dy where the types and strides are the same); dw, db NULL or
 *         fp32 [H] out. At least one of the three; ws may be NULL without dw and db. */
mok_status mok_norm_backward(const mok_norm_config *cfg, const void *h, const float *mean,
                             const float *rstd, const float *weight, const void *dy, const void *dh,
                             void *dx, float *dw, float *db, void *ws, size_t ws_bytes,
                             cudaStream_t stream);

/* ---- loss over a vocabulary -----------------------------------------------------------
 *
 *   l = x W^T       lse = log sum_v exp(l_v)       loss = lse - l_target + z_loss lse^2
 * for rows of x [rows][H] and the vocabulary's W [V][H], bf16 with fp32 accumulation. The logits are
 * never in memory: the forward keeps running maxima and sums, the backward makes the gradient of the
 * logits for a piece of the vocabulary at a time. A target below 0 takes no part (loss and gradients
 * 0); one at or past V raises MOK_ERR_DEVICE_INVARIANT and counts as below 0.
 *
 * Limits: 0 <= rows < 2^31 - 512, 1 <= H <= 2^20, 1 <= V <= 2^24, any numbers, fewer than 2^31 blocks
 * of 16 rows x 256 columns in rows x V, rows x H and V x H; strides ld_x, ld_w >= H are multiples of 8
 * elements, at most 2^30. Columns past H are neither read nor written. */
typedef struct mok_vocab_loss_config {
    uint32_t abi_version; /* MOK_ABI_VERSION */
    int32_t H, V;
    int32_t grad_dtype;   /* mok_dtype of dx and dW */
    int64_t rows;
    int64_t ld_x;         /* row stride of x and dx */
    int64_t ld_w;         /* row stride of W and dW */
    float z_loss;         /* finite, >= 0 */
    int32_t piece;        /* vocabulary entries of a piece, a multiple of 256; 0: as many as keep the
                             gradient of a piece's logits within 1 GiB */
} mok_vocab_loss_config;

typedef enum mok_vocab_loss_pass {
    MOK_VOCAB_LOSS_FORWARD = 0,
    MOK_VOCAB_LOSS_BACKWARD = 1
} mok_vocab_loss_pass;

mok_status mok_check_vocab_loss_config(const mok_vocab_loss_config *cfg);

/* Bytes of workspace of a pass (256-byte aligned, contents on entry do not matter); 0 for an
 * invalid configuration. The forward's grows with rows V / 8 (a maximum and a sum for each row and 64
 * entries: 134 MB for 8192 rows and 131072 entries), up to 64 rows with rows alone (4864 bytes each); the backward's with
 * rows times piece (2 bytes of each value of dl) and rows times H. */
size_t mok_vocab_loss_workspace_size(const mok_vocab_loss_config *cfg, int pass);

/* targets int32 [rows]; loss NULL or fp32 [rows] out, lse fp32 [rows] out (of every row, whatever its
 * target). */
mok_status mok_vocab_loss_forward(const mok_vocab_loss_config *cfg, const void *x, const void *w,
                                  const int32_t *targets, float *loss, float *lse, void *ws,
                                  size_t ws_bytes, cudaStream_t stream);

/* With d_loss fp32 [rows] and lse from the forward:
 *   dl_v = d_loss ((1 + 2 z_loss lse) exp(l_v - lse) - [v == target])
 *   dx = dl W            dW = dl^T x
 * dl enters the products as three bf16 values that add up to it for fp32 gradients, as two for bf16
 * gradients of up to 512 rows, and rounded to one (as the linear layer's dz does) for bf16 gradients of more
 * rows, whether they take part or not. Each entry is then off by up to 2^-8 of itself, and since a row's gradient
 * is for the most part its target's entry, that may scale a row of dx, or of dW, by as much, whatever the other
 * rows are (2.3e-3 of the norm, with the outputs' own rounding, where that alone is 1.7e-3); fp32
 * gradients have 4e-7 to 1.2e-6. Logits are summed over up to 1024 elements of H at a time, for bf16
 * gradients 4096.
 * dx NULL or [rows][H] out, dw NULL or [V][H] out; one of them at least, and neither is x or W. */
mok_status mok_vocab_loss_backward(const mok_vocab_loss_config *cfg, const void *x, const void *w,
                                   const int32_t *targets, const float *lse, const float *d_loss,
                                   void *dx, void *dw, void *ws, size_t ws_bytes,
                                   cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOK_OPS_H */

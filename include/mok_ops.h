/*
 * mok_ops.h -- operators around the expert layer of mok.h (included by it): the token sort
 * on its own, a linear layer for one matrix or one per expert, and the optimizer step.
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

#ifdef __cplusplus
}
#endif
#endif /* MOK_OPS_H */

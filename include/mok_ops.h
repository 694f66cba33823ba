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
 * Shapes: T tokens (T >= 0), 1 <= K <= 32 experts per token, 1 <= E <= 1024 experts, H >= 1
 * columns of any number; ld_tok, ld_row >= H; T*K, n_rows < 2^31. Columns past H of a row are
 * neither read nor written. Rows are copied 16 bytes at a time where both ld are multiples of
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
 * An expert id out of range, or a rank outside its expert's count, maps to -1 and raises
 * MOK_ERR_DEVICE_INVARIANT, as does starts[E] > n_rows. */
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
 * (may be y itself). */
mok_status mok_combine(const mok_rows_config *cfg, const void *rows, const int32_t *row_map,
                       const float *topk_w, const void *residual, void *y,
                       cudaStream_t stream);

/* The gradients of mok_combine, with r = row_map[t*K + k]:
 *   drows[r] = topk_w[t][k] * dy[t], rounded once (zero rows as in mok_dispatch);
 *   d_topk_w[t][k] = <rows[r], dy[t]> in fp32, in a fixed order (0 where dropped).
 * The residual's gradient is dy. Either output may be NULL (then rows is not read where
 * d_topk_w is NULL and may be NULL too), not both. drows must not overlap rows. */
mok_status mok_combine_backward(const mok_rows_config *cfg, const void *dy, const void *rows,
                                const int32_t *row_map, const int32_t *starts,
                                const int32_t *kept, const float *topk_w, void *drows,
                                float *d_topk_w, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOK_OPS_H */

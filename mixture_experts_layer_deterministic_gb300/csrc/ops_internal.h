// ops_internal.h -- what the operators around the layer (mok_ops.h) share: profiling kinds,
// the launch macro of their entry points, pointer checks.
#pragma once

#include "mok_internal.h"

namespace mok {

// profiling kinds, numbered after the layer's KernelKind
enum OpKind {
    OP_ROW_MAP = KK_COUNT, OP_DISPATCH, OP_COMBINE, OP_COMBINE_BWD, OP_ADAMW, OP_LINEAR_TILES,
    OP_LINEAR_FWD, OP_LINEAR_DZ, OP_LINEAR_DX, OP_LINEAR_DW, OP_COUNT
};

inline bool op_aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// rounding up to a multiple
inline int64_t round_up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

}  // namespace mok

// a launch of `nk` kernels of one kind, bracketed by events while profiling is on
#define MOK_OP_LAUNCH(kind, nk, expr)                      \
    do {                                                   \
        prof_begin(kind, stream);                          \
        cudaError_t _e = (expr);                           \
        prof_end(kind, stream, nk);                        \
        if (_e != cudaSuccess) return MOK_ERR_CUDA;        \
    } while (0)

// ops_internal.h -- what the operators around the layer (mok_ops.h) share: profiling kinds,
// the launch macro of their entry points, launches that overlap, pointer checks.
#pragma once

#include "mok_internal.h"
#ifdef __CUDACC__
#include "common.cuh"
#endif

namespace mok {

// profiling kinds, numbered after the layer's KernelKind
enum OpKind {
    OP_ROW_MAP = KK_COUNT, OP_DISPATCH, OP_COMBINE, OP_COMBINE_BWD, OP_ADAMW, OP_LINEAR_TILES,
    OP_LINEAR_FWD, OP_LINEAR_DZ, OP_LINEAR_DX, OP_LINEAR_DW, OP_COUNT
};

inline bool op_aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// rounding up to a multiple
inline int64_t round_up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

#ifdef __CUDACC__
// The operators' launches overlap at their edges: a kernel may be started while the one before it
// in the stream drains, sets itself up, and waits here before it touches global memory.
MOK_DEV void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
MOK_DEV void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// So what a kernel reads may still be written while it exists: loads go the ordinary way, not the
// read-only one.
MOK_DEV uint4 ld_v4(const void *p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// a launch that may start while the kernel before it drains (its kernel waits for that one
// itself); cluster: CTAs per cluster
template <class... KA, class... A>
cudaError_t launch_edge(void (*kernel)(KA...), dim3 grid, int threads, int smem, int cluster,
                        cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}
#endif

}  // namespace mok

// a launch of `nk` kernels of one kind, bracketed by events while profiling is on
#define MOK_OP_LAUNCH(kind, nk, expr)                      \
    do {                                                   \
        prof_begin(kind, stream);                          \
        cudaError_t _e = (expr);                           \
        prof_end(kind, stream, nk);                        \
        if (_e != cudaSuccess) return MOK_ERR_CUDA;        \
    } while (0)

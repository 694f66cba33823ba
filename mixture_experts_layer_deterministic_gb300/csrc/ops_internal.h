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
    OP_LINEAR_FWD, OP_LINEAR_DZ, OP_LINEAR_DX, OP_LINEAR_DW, OP_ROUTER, OP_ROUTER_BWD, OP_NORM,
    OP_NORM_BWD, OP_VOCAB_FWD, OP_VOCAB_DL, OP_VOCAB_GRADS, OP_COUNT
};

inline bool op_aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// SMs of a GB300: what a result's bits depend on (the number of parts of a sum) goes by them, not by the device's
constexpr int64_t GB300_SMS = 152;

// rounding up to a multiple
inline int64_t round_up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

// How these run: parts of K, `per` 64-element blocks each, by the sizes alone (the bits depend on them);
// the pairs of SMs that dW gets of a launch of both (0: one after the other), and of both; the height
// of dx's tiles beside dW, and with all pairs to itself.
struct GradCut {
    int parts, per, height;
};
struct GradPlan {
    GradCut x, w;
    int64_t split, pairs;
    int height, alone;
};
GradPlan plan_dense_grads(int64_t rows, int N, int Kin, int halves, bool cut);

// The products of a dense layer's backward, dx = dz W and dW = dz^T x, with dz made elsewhere: bf16
// [rows][N] rows ld_dz apart, or for fp32 gradients `halves` such planes that add up to it.
struct DenseGrads {
    const uint16_t *x, *w, *dz;  // [rows][Kin], [N][Kin], [halves][rows][N]
    int64_t rows;
    int N, Kin, halves;
    int run;                     // K elements that fp32 gradients sum at a time, a multiple of 64
    int64_t ld_x, ld_dx, ld_w, ld_dz;  // of x, of dx, of w and dw, of dz
    void *dx, *dw;               // one of them may be nullptr
    bool f32;                    // their type
    // where not nullptr, dx goes to dx_sum in fp32 (rows round_up(Kin, 4) apart), if dx is not nullptr;
    // where N is a piece of the layer's, dx adds to it (or to an fp32 dx) from the second piece on
    float *dx_sum;
    bool add;
    GradPlan plan;
    void *ws;  // dense_grads_bytes, where the plan cuts K
};
size_t dense_grads_bytes(const GradPlan &p, int64_t rows, int N, int Kin);
// *launches: how many it took
cudaError_t launch_dense_grads(const DenseGrads &a, int *status, int *launches, cudaStream_t s);

#ifdef __CUDACC__
// two fp32 values to bf16 in one conversion, lo in the low half (two single conversions run on
// the slow pipe and held the epilogue: dW of 64 x 1024 x 4096 164 against 139 us)
MOK_DEV uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// 2^x in hardware, off by 2^-22 of itself; 0 below 2^-126
MOK_DEV float exp2_hw(float x) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
    return e;
}

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

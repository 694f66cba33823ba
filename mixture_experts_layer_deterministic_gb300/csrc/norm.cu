// norm.cu -- layer norm and RMS norm of a residual sum, and their gradients.
//
//   h = x + residual, n = (h - mean) rstd, y = n w + b
//   g = dy w, dx = dh + rstd (g - n mean(g n) - mean(g)), dw = sum dy n, db = sum dy
//
// All of it is HBM traffic. A row belongs to a power of two of threads, whose vectors of 8 elements
// stay in registers between the passes over it; rows longer than that are read again. The mean is
// taken in two steps (of h, then of h less the first), so that rows far from zero keep their
// digits; the variance is that of h less the mean.
#include "ops_internal.h"

namespace mok {
namespace {

constexpr int NORM_TPB = 256;
constexpr int NORM_VECS = 4;  // vectors of 8 a thread at most
// blocks whose column sums are added in order: not of the device, the sums' bits depend on it
constexpr int64_t NORM_PARTS = 2 * 152;

// 8 elements from column c on, zeros past H (F32: two vectors)
template <bool F32>
MOK_DEV void load8(const void *row, int c, int H, float (&v)[8]) {
    if (c + 8 <= H) {
        if (F32) {
            const uint4 a = ld_v4(static_cast<const float *>(row) + c);
            const uint4 b = ld_v4(static_cast<const float *>(row) + c + 4);
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
        } else {
            const uint4 a = ld_v4(static_cast<const uint16_t *>(row) + c);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = bf16_lo(w[j]);
                v[2 * j + 1] = bf16_hi(w[j]);
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = c + j >= H ? 0.0f
               : F32      ? static_cast<const float *>(row)[c + j]
                          : bf16_to_f32(static_cast<const uint16_t *>(row)[c + j]);
}
MOK_DEV uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <bool F32>
MOK_DEV void store8(void *row, int c, int H, const float (&v)[8]) {
    if (c + 8 <= H) {
        if (F32) {
            float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(row) + c);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(row) + c) = make_uint4(
                pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7]));
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (c + j >= H) continue;
        if (F32)
            static_cast<float *>(row)[c + j] = v[j];
        else
            static_cast<uint16_t *>(row)[c + j] = f32_to_bf16(v[j]);
    }
}
// as it will be read back
template <bool F32>
MOK_DEV float rounded(float v) {
    return F32 ? v : bf16_to_f32(f32_to_bf16(v));
}

struct NormShape {
    int64_t rows, ld_x, ld_y;
    int H;
    int tpr;  // threads of a row: a power of two
    bool layer;
    float eps;
};

template <bool F32>
MOK_DEV const void *row_of(const void *p, int64_t r, int64_t ld) {
    return static_cast<const char *>(p) + r * ld * (F32 ? 4 : 2);
}
template <bool F32>
MOK_DEV void *row_of(void *p, int64_t r, int64_t ld) {
    return static_cast<char *>(p) + r * ld * (F32 ? 4 : 2);
}

// sums of a and b over the tpr threads of a row, the same in all of them. More than a warp's: through
// sh, which the threads of every row of the block call together.
struct RowSum {
    float2 *sh;  // [warps of the block]
    int tpr;
    MOK_DEV void operator()(float &a, float &b) const {
        const int w = tpr < 32 ? tpr : 32;
        for (int o = 1; o < w; o <<= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        if (tpr <= 32) return;
        const int warp = threadIdx.x >> 5, n = tpr / 32, first = warp / n * n;
        __syncthreads();  // the last sums have been read
        if ((threadIdx.x & 31) == 0) sh[warp] = make_float2(a, b);
        __syncthreads();
        a = b = 0.0f;
        for (int k = 0; k < n; ++k) {
            const float2 v = sh[first + k];
            a += v.x;
            b += v.y;
        }
    }
};

struct NormFwd {
    NormShape s;
    const void *x, *res;
    const float *w, *b;
    void *h, *y;
    float *mean, *rstd;
};

// h of 8 columns, stored where asked for
template <bool X32>
MOK_DEV void load_h(const NormFwd &a, int64_t r, int c, float (&v)[8]) {
    load8<X32>(row_of<X32>(a.x, r, a.s.ld_x), c, a.s.H, v);
    if (a.res == nullptr) return;
    float q[8];
    load8<X32>(row_of<X32>(a.res, r, a.s.ld_x), c, a.s.H, q);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = rounded<X32>(v[j] + q[j]);
}

template <bool Y32>
MOK_DEV void store_y(const NormFwd &a, int64_t r, int c, float mean, float rest, float rstd,
                     float (&v)[8]) {
    float p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (v[j] - mean - rest) * rstd;
    if (a.w != nullptr) {
        load8<true>(a.w, c, a.s.H, p);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= p[j];
    }
    if (a.b != nullptr) {
        load8<true>(a.b, c, a.s.H, p);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += p[j];
    }
    store8<Y32>(row_of<Y32>(a.y, r, a.s.ld_y), c, a.s.H, v);
}

// columns past H of a vector are zeros: they add to no sum but that of (0 - mean)^2
MOK_DEV float square_from(const float (&v)[8], float mean, int n) {
    float q = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) q = fmaf(v[j] - mean, v[j] - mean, q);
    return q;
}

// NV vectors a thread: rows of at most 8 NV tpr elements
template <int NV, bool X32, bool Y32>
__global__ void __launch_bounds__(1024) norm_kernel(const NormFwd a) {
    __shared__ float2 sh[32];
    const NormShape &s = a.s;
    const RowSum row_sum{sh, s.tpr};
    let_next_start();
    wait_for_previous();
    const int i = threadIdx.x % s.tpr;
    const int64_t r = (int64_t)blockIdx.x * (blockDim.x / s.tpr) + threadIdx.x / s.tpr;
    const bool in = r < s.rows;
    float v[NV][8];
    float sum = 0.0f, rest = 0.0f, sq = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = 8 * (i + k * s.tpr);
        if (in && c < s.H) {
            load_h<X32>(a, r, c, v[k]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[k][j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += v[k][j];
    }
    float mean = 0.0f;
    if (s.layer) {
        row_sum(sum, rest);
        mean = sum / s.H;
    }
    rest = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = 8 * (i + k * s.tpr), n = in && c < s.H ? s.H - c : 0;
        sq += square_from(v[k], mean, n);
        if (s.layer)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) rest += v[k][j] - mean;
    }
    row_sum(sq, rest);
    rest /= s.H;  // what the mean's rounding left
    const float var = fmaxf(sq / s.H - rest * rest, 0.0f);
    const float rstd = 1.0f / sqrtf(var + s.eps);
    if (!in) return;
    if (i == 0) {
        if (a.mean != nullptr) a.mean[r] = mean + rest;
        if (a.rstd != nullptr) a.rstd[r] = rstd;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = 8 * (i + k * s.tpr);
        if (c >= s.H) continue;
        if (a.h != nullptr) store8<X32>(row_of<X32>(a.h, r, s.ld_x), c, s.H, v[k]);
        store_y<Y32>(a, r, c, mean, rest, rstd, v[k]);
    }
}

// longer rows: one a block, read three times (h is written last, so x or the residual may be h)
template <bool X32, bool Y32>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormFwd a) {
    __shared__ float2 sh[32];
    const NormShape &s = a.s;
    const RowSum row_sum{sh, 1024};
    let_next_start();
    wait_for_previous();
    const int64_t r = blockIdx.x;
    float v[8], sum = 0.0f, rest = 0.0f, sq = 0.0f, mean = 0.0f;
    if (s.layer) {
        for (int c = 8 * threadIdx.x; c < s.H; c += 8 * 1024) {
            load_h<X32>(a, r, c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += v[j];
        }
        row_sum(sum, rest);
        mean = sum / s.H;
        rest = 0.0f;
    }
    for (int c = 8 * threadIdx.x; c < s.H; c += 8 * 1024) {
        load_h<X32>(a, r, c, v);
        sq += square_from(v, mean, s.H - c);
        if (s.layer)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < s.H) rest += v[j] - mean;
    }
    row_sum(sq, rest);
    rest /= s.H;
    const float var = fmaxf(sq / s.H - rest * rest, 0.0f);
    const float rstd = 1.0f / sqrtf(var + s.eps);
    if (threadIdx.x == 0) {
        if (a.mean != nullptr) a.mean[r] = mean + rest;
        if (a.rstd != nullptr) a.rstd[r] = rstd;
    }
    for (int c = 8 * threadIdx.x; c < s.H; c += 8 * 1024) {
        load_h<X32>(a, r, c, v);
        if (a.h != nullptr) store8<X32>(row_of<X32>(a.h, r, s.ld_x), c, s.H, v);
        store_y<Y32>(a, r, c, mean, rest, rstd, v);
    }
}

// ---------------------------------------------------------------- backward
struct NormBwd {
    NormShape s;
    const void *h, *dy, *dh;
    const float *mean, *rstd, *w;
    void *dx;
    float *dw_part, *db_part;  // [NORM_PARTS][H], or nullptr
};

// n and g of 8 columns, and what they add to the row's sums
template <bool X32, bool Y32>
MOK_DEV void load_ng(const NormBwd &a, int64_t r, int c, float mean, float rstd, float (&n)[8],
                     float (&dy)[8], float &sg, float &sgn) {
    float w[8];
    load8<X32>(row_of<X32>(a.h, r, a.s.ld_x), c, a.s.H, n);
    load8<Y32>(row_of<Y32>(a.dy, r, a.s.ld_y), c, a.s.H, dy);
    if (a.w != nullptr) load8<true>(a.w, c, a.s.H, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        n[j] = c + j < a.s.H ? (n[j] - mean) * rstd : 0.0f;
        const float g = a.w != nullptr ? dy[j] * w[j] : dy[j];
        sg += g;
        sgn = fmaf(g, n[j], sgn);
    }
}
template <bool X32>
MOK_DEV void store_dx(const NormBwd &a, int64_t r, int c, float rstd, float mg, float mgn,
                      const float (&n)[8], const float (&dy)[8]) {
    float w[8], v[8];
    if (a.w != nullptr) load8<true>(a.w, c, a.s.H, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float g = a.w != nullptr ? dy[j] * w[j] : dy[j];
        v[j] = rstd * (g - n[j] * mgn - mg);
    }
    if (a.dh != nullptr) {
        load8<X32>(row_of<X32>(a.dh, r, a.s.ld_x), c, a.s.H, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += w[j];
    }
    store8<X32>(row_of<X32>(a.dx, r, a.s.ld_x), c, a.s.H, v);
}

// Block b takes rows b, b + blocks, .. (a row to each tpr of its threads at a time), keeps its
// columns' sums in registers and adds its rows' threads in order at the end.
template <int NV, bool X32, bool Y32>
__global__ void __launch_bounds__(1024) norm_backward_kernel(const NormBwd a) {
    extern __shared__ float norm_smem[];
    __shared__ float2 sh[32];
    const NormShape &s = a.s;
    const RowSum row_sum{sh, s.tpr};
    let_next_start();
    wait_for_previous();
    const int i = threadIdx.x % s.tpr, slot = threadIdx.x / s.tpr, slots = blockDim.x / s.tpr;
    float dw[NV][8], db[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[k][j] = db[k][j] = 0.0f;
    for (int64_t r0 = (int64_t)blockIdx.x * slots; r0 < s.rows; r0 += (int64_t)gridDim.x * slots) {
        const int64_t r = r0 + slot;
        const bool in = r < s.rows;
        const float mean = in && s.layer ? a.mean[r] : 0.0f, rstd = in ? a.rstd[r] : 0.0f;
        float n[NV][8], dy[NV][8], sg = 0.0f, sgn = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = 8 * (i + k * s.tpr);
            if (in && c < s.H) {
                load_ng<X32, Y32>(a, r, c, mean, rstd, n[k], dy[k], sg, sgn);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) n[k][j] = dy[k][j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[k][j] = fmaf(dy[k][j], n[k][j], dw[k][j]);
                db[k][j] += dy[k][j];
            }
        }
        if (a.dx == nullptr) continue;
        row_sum(sgn, sg);
        if (!in) continue;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = 8 * (i + k * s.tpr);
            if (c < s.H)
                store_dx<X32>(a, r, c, rstd, s.layer ? sg / s.H : 0.0f, sgn / s.H, n[k], dy[k]);
        }
    }
    for (int part = 0; part < 2; ++part) {
        float *out = part == 0 ? a.dw_part : a.db_part;
        if (out == nullptr) continue;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = 8 * (i + k * s.tpr);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < s.H) norm_smem[slot * s.H + c + j] = part == 0 ? dw[k][j] : db[k][j];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < s.H; c += blockDim.x) {
            float t = 0.0f;
            for (int k = 0; k < slots; ++k) t += norm_smem[k * s.H + c];
            out[(int64_t)blockIdx.x * s.H + c] = t;
        }
    }
}

// longer rows: dx by a block a row, read twice
template <bool X32, bool Y32>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(const NormBwd a) {
    __shared__ float2 sh[32];
    const NormShape &s = a.s;
    const RowSum row_sum{sh, 1024};
    let_next_start();
    wait_for_previous();
    const int64_t r = blockIdx.x;
    const float mean = s.layer ? a.mean[r] : 0.0f, rstd = a.rstd[r];
    float n[8], dy[8], sg = 0.0f, sgn = 0.0f, unused = 0.0f;
    for (int c = 8 * threadIdx.x; c < s.H; c += 8 * 1024)
        load_ng<X32, Y32>(a, r, c, mean, rstd, n, dy, sg, sgn);
    row_sum(sgn, sg);
    for (int c = 8 * threadIdx.x; c < s.H; c += 8 * 1024) {
        load_ng<X32, Y32>(a, r, c, mean, rstd, n, dy, unused, unused);
        store_dx<X32>(a, r, c, rstd, s.layer ? sg / s.H : 0.0f, sgn / s.H, n, dy);
    }
}
// ... and the column sums by a thread per 8 columns and part of the rows
template <bool X32, bool Y32>
__global__ void __launch_bounds__(NORM_TPB) norm_columns_kernel(const NormBwd a) {
    const NormShape &s = a.s;
    let_next_start();
    wait_for_previous();
    const int c = 8 * (blockIdx.x * NORM_TPB + threadIdx.x);
    if (c >= s.H) return;
    float dw[8], db[8], n[8], dy[8], unused = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = db[j] = 0.0f;
    for (int64_t r = blockIdx.y; r < s.rows; r += gridDim.y) {
        load_ng<X32, Y32>(a, r, c, s.layer ? a.mean[r] : 0.0f, a.rstd[r], n, dy, unused, unused);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[j] = fmaf(dy[j], n[j], dw[j]);
            db[j] += dy[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (c + j >= s.H) continue;
        const int64_t at = (int64_t)blockIdx.y * s.H + c + j;
        if (a.dw_part != nullptr) a.dw_part[at] = dw[j];
        if (a.db_part != nullptr) a.db_part[at] = db[j];
    }
}

// the parts of dw and db, added in order: 32 columns a block, each warp a slice of the parts
constexpr int NORM_SLICES = 16;
__global__ void __launch_bounds__(32 * NORM_SLICES)
    norm_join_kernel(const float *dw_part, const float *db_part, int parts, int H, float *dw,
                     float *db) {
    __shared__ float sh[2][NORM_SLICES][32];
    let_next_start();
    wait_for_previous();
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f, t = 0.0f;
    if (c < H) {
        if (dw != nullptr)
#pragma unroll 8
            for (int p = slice; p < parts; p += NORM_SLICES) s += dw_part[(int64_t)p * H + c];
        if (db != nullptr)
#pragma unroll 8
            for (int p = slice; p < parts; p += NORM_SLICES) t += db_part[(int64_t)p * H + c];
    }
    sh[0][slice][lane] = s;
    sh[1][slice][lane] = t;
    __syncthreads();
    if (slice != 0 || c >= H) return;
    s = t = 0.0f;
#pragma unroll
    for (int k = 0; k < NORM_SLICES; ++k) {
        s += sh[0][k][lane];
        t += sh[1][k][lane];
    }
    if (dw != nullptr) dw[c] = s;
    if (db != nullptr) db[c] = t;
}

// ---------------------------------------------------------------- host side
NormShape norm_shape(const mok_norm_config &c) {
    return NormShape{c.rows, c.ld_x, c.ld_y, c.H, 1024, c.kind == MOK_NORM_LAYER, c.eps};
}
int pow2_up(int n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

struct NormPlan {
    bool whole;      // rows fit the registers of 1024 threads
    int nv, tpr;     // vectors a thread, threads a row
    int64_t parts;   // of the backward's column sums
};
NormPlan norm_plan(const mok_norm_config &c) {
    const int vecs = (c.H + 7) / 8;
    NormPlan p = {};
    p.whole = vecs <= 1024 * NORM_VECS;
    p.nv = vecs <= 32 ? 1 : vecs <= 1024 ? 2 : NORM_VECS;
    p.tpr = pow2_up((vecs + p.nv - 1) / p.nv);
    if (p.tpr > 1024) p.tpr = 1024;
    const int slots = p.tpr < NORM_TPB ? NORM_TPB / p.tpr : 1;
    const int64_t groups = p.whole ? (c.rows + slots - 1) / slots : c.rows;
    p.parts = groups < NORM_PARTS ? groups : NORM_PARTS;
    if (!p.whole && p.parts > 32) p.parts = 32;
    return p;
}
size_t norm_part_bytes(const mok_norm_config &c) {
    return (size_t)round_up(norm_plan(c).parts * c.H * 4, 256);
}

#define MOK_NORM_TYPES(F)                                   \
    (x32 ? (y32 ? F(true, true) : F(true, false))           \
         : (y32 ? F(false, true) : F(false, false)))

cudaError_t launch_norm(NormFwd a, const NormPlan &p, bool x32, bool y32, cudaStream_t s) {
    a.s.tpr = p.tpr;
    const int tpb = p.tpr < NORM_TPB ? NORM_TPB : p.tpr;
    const unsigned grid = (unsigned)((a.s.rows + tpb / p.tpr - 1) / (tpb / p.tpr));
#define MOK_F(X, Y)                                                                 \
    (!p.whole    ? launch_edge(norm_long_kernel<X, Y>, (unsigned)a.s.rows, 1024, 0, 1, s, a) \
     : p.nv == 1 ? launch_edge(norm_kernel<1, X, Y>, grid, tpb, 0, 1, s, a)         \
     : p.nv == 2 ? launch_edge(norm_kernel<2, X, Y>, grid, tpb, 0, 1, s, a)         \
                 : launch_edge(norm_kernel<NORM_VECS, X, Y>, grid, tpb, 0, 1, s, a))
    return MOK_NORM_TYPES(MOK_F);
#undef MOK_F
}

cudaError_t launch_norm_backward(NormBwd a, const NormPlan &p, bool x32, bool y32, cudaStream_t s) {
    a.s.tpr = p.tpr;
    const bool sums = a.dw_part != nullptr || a.db_part != nullptr;
    if (!p.whole) {
        const dim3 cols((unsigned)((a.s.H + 8 * NORM_TPB - 1) / (8 * NORM_TPB)), (unsigned)p.parts);
        cudaError_t e = cudaSuccess;
#define MOK_F(X, Y) launch_edge(norm_columns_kernel<X, Y>, cols, NORM_TPB, 0, 1, s, a)
        if (sums) e = MOK_NORM_TYPES(MOK_F);
#undef MOK_F
        if (e != cudaSuccess || a.dx == nullptr) return e;
#define MOK_F(X, Y) \
    launch_edge(norm_backward_long_kernel<X, Y>, (unsigned)a.s.rows, 1024, 0, 1, s, a)
        return MOK_NORM_TYPES(MOK_F);
#undef MOK_F
    }
    const int tpb = p.tpr < NORM_TPB ? NORM_TPB : p.tpr;
    const int smem = sums ? tpb / p.tpr * a.s.H * 4 : 0;
    const unsigned grid = (unsigned)p.parts;
#define MOK_G(K)                                                                                    \
    (smem <= 48 * 1024 ||                                                                           \
             cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess \
         ? launch_edge(K, grid, tpb, smem, 1, s, a)                                                 \
         : cudaErrorInvalidValue)
#define MOK_F(X, Y)                                                      \
    (p.nv == 1   ? MOK_G((norm_backward_kernel<1, X, Y>))                \
     : p.nv == 2 ? MOK_G((norm_backward_kernel<2, X, Y>))                \
                 : MOK_G((norm_backward_kernel<NORM_VECS, X, Y>)))
    return MOK_NORM_TYPES(MOK_F);
#undef MOK_F
#undef MOK_G
}

}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

mok_status mok_check_norm_config(const mok_norm_config *c) {
    if (c == nullptr) return MOK_ERR_INVALID_ARG;
    if (c->abi_version != MOK_ABI_VERSION) return MOK_ERR_ABI;
    if (c->H < 1 || c->H > (1 << 20)) return MOK_ERR_INVALID_ARG;
    if (c->rows < 0 || c->rows >= ((int64_t)1 << 31) - 512) return MOK_ERR_INVALID_ARG;
    const int64_t lds[] = {c->ld_x, c->ld_y};
    for (int64_t ld : lds)
        if (ld < c->H || ld % 8 != 0 || ld > ((int64_t)1 << 30)) return MOK_ERR_INVALID_ARG;
    if (c->kind != MOK_NORM_LAYER && c->kind != MOK_NORM_RMS) return MOK_ERR_INVALID_ARG;
    const int32_t dts[] = {c->x_dtype, c->y_dtype};
    for (int32_t d : dts)
        if (d != MOK_DTYPE_BF16 && d != MOK_DTYPE_F32) return MOK_ERR_INVALID_ARG;
    if (!(c->eps > 0.0f && c->eps <= 3.402823466e38f)) return MOK_ERR_INVALID_ARG;
    return MOK_OK;
}

size_t mok_norm_workspace_size(const mok_norm_config *c) {
    if (mok_check_norm_config(c) != MOK_OK) return 0;
    const size_t n = 2 * norm_part_bytes(*c);
    return n > 0 ? n : 256;
}

mok_status mok_norm_forward(const mok_norm_config *c, const void *x, const void *residual,
                            const float *weight, const float *bias, void *h, void *y, float *mean,
                            float *rstd, cudaStream_t stream) {
    mok_status st = mok_check_norm_config(c);
    if (st != MOK_OK) return st;
    int *status;
    if ((st = current_device_status_word(&status)) != MOK_OK) return st;
    if (c->rows == 0) return MOK_OK;
    if (!x || !y || (h && !residual) || (mean && c->kind == MOK_NORM_RMS)) return MOK_ERR_INVALID_ARG;
    if (y == h || (y == x && (c->x_dtype != c->y_dtype || c->ld_x != c->ld_y)))
        return MOK_ERR_INVALID_ARG;
    const void *ps[] = {x, residual, weight, bias, h, y, mean, rstd};
    for (const void *p : ps)
        if (p && !op_aligned16(p)) return MOK_ERR_INVALID_ARG;
    const NormFwd a{norm_shape(*c), x, residual, weight, bias, h, y, mean, rstd};
    MOK_OP_LAUNCH(OP_NORM, 1,
                  launch_norm(a, norm_plan(*c), c->x_dtype == MOK_DTYPE_F32,
                              c->y_dtype == MOK_DTYPE_F32, stream));
    return MOK_OK;
}

mok_status mok_norm_backward(const mok_norm_config *c, const void *h, const float *mean,
                             const float *rstd, const float *weight, const void *dy, const void *dh,
                             void *dx, float *dw, float *db, void *ws, size_t ws_bytes,
                             cudaStream_t stream) {
    mok_status st = mok_check_norm_config(c);
    if (st != MOK_OK) return st;
    int *status;
    if ((st = current_device_status_word(&status)) != MOK_OK) return st;
    if (!dx && !dw && !db) return MOK_ERR_INVALID_ARG;
    const bool sums = dw || db;
    if (sums && (!ws || ((uintptr_t)ws & 255u) != 0 || ws_bytes < mok_norm_workspace_size(c)))
        return MOK_ERR_WORKSPACE;
    if (c->rows > 0 && (!h || !rstd || !dy || (c->kind == MOK_NORM_LAYER && !mean)))
        return MOK_ERR_INVALID_ARG;
    if (dx && (dx == h || (dx == dy && (c->x_dtype != c->y_dtype || c->ld_x != c->ld_y))))
        return MOK_ERR_INVALID_ARG;
    const void *ps[] = {h, mean, rstd, weight, dy, dh, dx, dw, db};
    for (const void *p : ps)
        if (p && !op_aligned16(p)) return MOK_ERR_INVALID_ARG;
    const NormPlan plan = norm_plan(*c);
    float *wp = dw ? (float *)ws : nullptr;
    float *bp = db ? (float *)((char *)ws + norm_part_bytes(*c)) : nullptr;
    if (c->rows > 0) {
        const NormBwd a{norm_shape(*c), h, dy, dh, mean, rstd, weight, dx, wp, bp};
        MOK_OP_LAUNCH(OP_NORM_BWD, 1,
                      launch_norm_backward(a, plan, c->x_dtype == MOK_DTYPE_F32,
                                           c->y_dtype == MOK_DTYPE_F32, stream));
    }
    if (sums)
        MOK_OP_LAUNCH(OP_NORM_BWD, 1,
                      launch_edge(norm_join_kernel, (unsigned)((c->H + 31) / 32), 32 * NORM_SLICES, 0,
                                  1, stream, (const float *)wp, (const float *)bp, (int)plan.parts,
                                  c->H, dw, db));
    return MOK_OK;
}

}  // extern "C"

// rows.cu -- the token sort as operators: row map, dispatch, combine and their gradients.
//
// With r(t,k) the row of routed id f = t*K + k (or none):
//   dispatch           xs[r(t,k)] = x[t]
//   combine            y[t] = res[t] + sum_k w[t,k] rows[r(t,k)]
//   combine backward   drows[r(t,k)] = w[t,k] dy[t],  dw[t,k] = <rows[r(t,k)], dy[t]>
//   dispatch backward  dx[t] = sum_k dxs[r(t,k)]       (combine with weights of one)
// All of it is HBM traffic of R = T*K rows; every token row is touched once. Work is cut by
// token and by column segment, so a row is read or written by whole warps, 16 bytes a lane.
// Sums over k run in ascending k in fp32; dot products over H in a fixed tree: no atomics.
#include <type_traits>

#include "common.cuh"
#include "ops_internal.h"

namespace mok {
namespace {

constexpr int TPB = 256;
constexpr int WARPS = TPB / 32;
constexpr int MAX_E = 1024;
// 16-byte pieces per lane and row of an item: a warp reads a row in runs of 1 KB (16384 tokens x
// 10 rows x 4096 bf16: combine 321 us at one piece, 232 us at two;
// and its gradient 273 us at one, 233 us at two for 8192 tokens)
constexpr int COMBINE_U = 2;
constexpr int COMBINE_BWD_U = 2;
// with at most 4 copies a round of one segment leaves few loads in flight: longer segments for
// combine, more blocks for its gradient (16384 tokens x 2 rows x 4096 bf16: 98 -> 76 us and
// 156 -> 126 us; 8192 x 4: 69 -> 63 us and 113 -> 98 us)
constexpr int FEW = 4;
constexpr int FEW_U = 4;
constexpr int FEW_BWD_BLOCKS = 3;
// blocks per SM, looping over the items: dispatch holds few registers and wants many stores in
// flight (16: 235 us, 4: 261 us); the other two hold 8 rows a lane in registers, two blocks an SM
// are resident, and longer-lived blocks read neighbouring rows together (2: 232 and 233 us,
// 4: 236 and 234 us, 16: 247 and 242 us, the gradient over 8192 tokens)
constexpr int DISPATCH_BLOCKS = 16;
constexpr int COMBINE_BLOCKS = 2;

// blocks for `items` work items, `per_block` of them a block: looping blocks, per_sm on each SM,
// where there are at least four rounds of them; below that one block per share of the items
// (1.7 rounds of looping blocks would run as two)
inline unsigned grid_for(int64_t items, int per_block, int per_sm) {
    const int64_t cap = (int64_t)device_sm_count() * per_sm;
    const int64_t b = (items + per_block - 1) / per_block;
    return (unsigned)(b < 1 ? 1 : b > 4 * cap ? cap : b);
}

// ---------------------------------------------------------------- row map
// Every block scans the experts' kept rows for itself (E <= 1024: ten steps in shared
// memory), then maps its share of the ids: one launch, no order between blocks.
__global__ void __launch_bounds__(MAX_E)
    row_map_kernel(const int32_t *idx, const int32_t *counts,
                   const int32_t *offsets, const int32_t *inv,
                   int64_t R, int E, int capacity, int64_t n_rows, int32_t *map,
                   int32_t *starts, int32_t *kept, int *status) {
    let_next_start();
    wait_for_previous();
    __shared__ int64_t warp_sum[MAX_E / 32];
    __shared__ int32_t s_start[MAX_E], s_count[MAX_E], s_kept[MAX_E], s_off[MAX_E];
    const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
    int32_t n = 0;
    if (e < E) {
        n = counts[e];
        if (n < 0 || n > R) {
            raise_status(status, MOK_ERR_DEVICE_INVARIANT);
            n = 0;
        }
        s_count[e] = n;
        if (capacity > 0 && n > capacity) n = capacity;
    }
    int64_t v = ((int64_t)n + 15) & ~(int64_t)15;
    const int64_t own = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    int64_t base = 0;
    for (int w = 0; w < warp; ++w) base += warp_sum[w];
    const int64_t end = base + v, begin = end - own;
    if (e < E) {
        // past 31 bits nothing fits n_rows; the ids of such experts are dropped below
        s_start[e] = begin < 0x7FFFFFFF ? (int32_t)begin : 0x7FFFFFFF;
        s_kept[e] = n;
        s_off[e] = offsets[e];
        if (blockIdx.x == 0) {
            starts[e] = s_start[e];
            kept[e] = n;
            if (e == E - 1) {
                starts[E] = end < 0x7FFFFFFF ? (int32_t)end : 0x7FFFFFFF;
                if (end > n_rows) raise_status(status, MOK_ERR_DEVICE_INVARIANT);
            }
        }
    }
    __syncthreads();
    const int64_t stride = (int64_t)gridDim.x * MAX_E;
    for (int64_t f = (int64_t)blockIdx.x * MAX_E + threadIdx.x; f < R; f += stride) {
        const int32_t x = idx[f];
        int32_t row = -1;
        if (x < 0 || x >= E) {
            raise_status(status, MOK_ERR_DEVICE_INVARIANT);
        } else {
            const int64_t rank = (int64_t)inv[f] - s_off[x];
            // past the count the schedule is of other ids; from the capacity on an id is dropped
            if (rank < 0 || rank >= s_count[x]) {
                raise_status(status, MOK_ERR_DEVICE_INVARIANT);
            } else if (rank < s_kept[x] && (int64_t)s_start[x] + rank < n_rows) {
                row = (int32_t)(s_start[x] + rank);
            }
        }
        map[f] = row;
    }
}

// ---------------------------------------------------------------- row access
// Elements of a row handled per lane and step: one 16-byte vector, or one element where the
// strides do not keep rows 16-byte aligned.
template <bool F32>
struct Elem {
    using Raw = typename std::conditional<F32, uint32_t, uint16_t>::type;
    static constexpr int BYTES = F32 ? 4 : 2;
    static constexpr int PER = 16 / BYTES;  // elements of a 16-byte vector
};

// the routed row of id f: a valid row index, or -1 (an index at or past n_rows is reported)
MOK_DEV int32_t checked_row(int32_t r, int64_t n_rows, int *status) {
    if (r >= n_rows) {
        raise_status(status, MOK_ERR_DEVICE_INVARIANT);
        r = -1;
    }
    return r;
}
MOK_DEV int32_t row_of(const int32_t *map, int64_t f, int64_t n_rows, int *status) {
    return checked_row(map[f], n_rows, status);
}

template <bool F32>
MOK_DEV float load_elem(const void *p, int64_t i) {
    return F32 ? static_cast<const float *>(p)[i]
               : bf16_to_f32(static_cast<const uint16_t *>(p)[i]);
}
template <bool F32>
MOK_DEV void store_elem(void *p, int64_t i, float v) {
    if (F32)
        static_cast<float *>(p)[i] = v;
    else
        static_cast<uint16_t *>(p)[i] = f32_to_bf16(v);
}
template <bool F32>
MOK_DEV void unpack(const uint4 &u, float (&v)[Elem<F32>::PER]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (F32) {
            v[q] = __uint_as_float(w[q]);
        } else {
            v[2 * q] = bf16_lo(w[q]);
            v[2 * q + 1] = bf16_hi(w[q]);
        }
    }
}
template <bool F32>
MOK_DEV uint4 pack(const float (&v)[Elem<F32>::PER]) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
        w[q] = F32 ? __float_as_uint(v[q]) : pack_bf16x2(v[2 * q], v[2 * q + 1]);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// zero rows of the sorted array after each expert's own: item (e, j), row kept[e] + j below
// the next multiple of 16; one warp per item
template <bool F32, bool VEC>
MOK_DEV void zero_pad_row(int64_t item, const int32_t *starts,
                          const int32_t *kept, int64_t n_rows, int H, int64_t ld,
                          void *out, int lane) {
    const int e = (int)(item >> 4), j = (int)(item & 15);
    const int64_t n = kept[e];
    if (n + j >= ((n + 15) & ~(int64_t)15)) return;
    const int64_t row = starts[e] + n + j;
    if (row < 0 || row >= n_rows) return;
    uint8_t *p = static_cast<uint8_t *>(out) + row * ld * Elem<F32>::BYTES;
    int c = 0;
    if (VEC) {
        c = H / Elem<F32>::PER * Elem<F32>::PER;
        for (int v = lane; v < H / Elem<F32>::PER; v += 32)
            reinterpret_cast<uint4 *>(p)[v] = make_uint4(0, 0, 0, 0);
    }
    for (c += lane; c < H; c += 32) store_elem<F32>(p, c, 0.f);
}

// ---------------------------------------------------------------- dispatch
// Work item: (token, segment of 32*U vectors), one warp each; a token's row is read once and
// written to the rows of its K copies. Items past the tokens' are the pad rows. Bound by the
// writes: 16384 tokens x 10 copies x 4096 bf16 224 us, 6.6 TB/s.
template <bool F32, bool VEC, int U>
__global__ void __launch_bounds__(TPB)
    dispatch_kernel(const void *x, const int32_t *map,
                    const int32_t *starts, const int32_t *kept,
                    int64_t T, int K, int E, int H, int64_t ld_tok, int64_t ld_row,
                    int64_t n_rows, void *xs, int *status) {
    let_next_start();
    wait_for_previous();
    constexpr int B = Elem<F32>::BYTES, PER = VEC ? Elem<F32>::PER : 1;
    const int lane = threadIdx.x & 31;
    const int nv = H / PER;                          // whole vectors of a row
    const int segs = (H + PER * 32 * U - 1) / (PER * 32 * U);
    const int64_t tok_items = T * segs;
    const int64_t items = tok_items + (starts != nullptr ? (int64_t)E * 16 : 0);
    const int64_t nw = (int64_t)gridDim.x * WARPS;
    for (int64_t it = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5); it < items; it += nw) {
        if (it >= tok_items) {
            zero_pad_row<F32, VEC>(it - tok_items, starts, kept, n_rows, H, ld_row, xs, lane);
            continue;
        }
        const int64_t t = it / segs;
        const int v0 = (int)(it % segs) * 32 * U + lane;
        const int32_t rk = lane < K ? row_of(map, t * K + lane, n_rows, status) : -1;
        const uint8_t *src = static_cast<const uint8_t *>(x) + t * ld_tok * B;
        using Raw = typename Elem<F32>::Raw;  // elements are copied bit for bit
        if (VEC) {
            uint4 b[U];
            Raw tail = 0;  // the columns past the last whole vector, at most PER - 1
            const int tc = nv * PER + lane;
            const bool has_tail = v0 - lane + 32 * U > nv && tc < H;
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (v0 + 32 * j < nv) b[j] = ld_v4(src + (int64_t)(v0 + 32 * j) * 16);
            if (has_tail) tail = reinterpret_cast<const Raw *>(src)[tc];
            for (int k = 0; k < K; ++k) {
                const int64_t r = __shfl_sync(0xFFFFFFFFu, rk, k);
                if (r < 0) continue;
                uint8_t *dst = static_cast<uint8_t *>(xs) + r * ld_row * B;
#pragma unroll
                for (int j = 0; j < U; ++j)
                    if (v0 + 32 * j < nv) reinterpret_cast<uint4 *>(dst)[v0 + 32 * j] = b[j];
                if (has_tail) reinterpret_cast<Raw *>(dst)[tc] = tail;
            }
        } else {
            Raw b[U];
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (v0 + 32 * j < nv) b[j] = reinterpret_cast<const Raw *>(src)[v0 + 32 * j];
            for (int k = 0; k < K; ++k) {
                const int64_t r = __shfl_sync(0xFFFFFFFFu, rk, k);
                if (r < 0) continue;
                Raw *dst = reinterpret_cast<Raw *>(static_cast<uint8_t *>(xs) + r * ld_row * B);
#pragma unroll
                for (int j = 0; j < U; ++j)
                    if (v0 + 32 * j < nv) dst[v0 + 32 * j] = b[j];
            }
        }
    }
}

// ---------------------------------------------------------------- combine
// PER elements of a row from column c, as fp32; elements past H are zero
template <bool F32, bool VEC>
struct Piece {
    static constexpr int PER = VEC ? Elem<F32>::PER : 1;
    uint4 q;
    float e;
    // raw load: whole vectors only (VEC), or one element
    MOK_DEV void load(const uint8_t *row, int c, bool in) {
        if (VEC) {
            q = make_uint4(0, 0, 0, 0);
            if (in) q = ld_v4(row + (int64_t)c * Elem<F32>::BYTES);
        } else {
            e = in ? load_elem<F32>(row, c) : 0.f;
        }
    }
    MOK_DEV void values(float (&v)[PER]) const {
        if constexpr (VEC) unpack<F32>(q, v);
        else v[0] = e;
    }
};

// Work item: (token, segment of 32*U pieces of 16 bytes), one warp each. Lane k holds row and
// weight of copy k. The K rows are read in rounds of equal size, at most J rows x U pieces a
// lane, all loads of a round before the first is used (16384 tokens x 10 rows x 4096 bf16 230 us,
// 6.4 TB/s): the rounds' memory latency is what
// bounds a warp here. A dropped copy has weight zero and reads as zero.
template <bool F32, bool VEC, int J, int U>
__global__ void __launch_bounds__(TPB, COMBINE_BLOCKS)
    combine_rows_kernel(const void *rows, const int32_t *map,
                        const float *w, const void *res, int64_t T, int K, int H,
                        int64_t ld_tok, int64_t ld_row, int64_t n_rows, void *y, int *status) {
    let_next_start();
    wait_for_previous();
    using P = Piece<F32, VEC>;
    constexpr int B = Elem<F32>::BYTES, PER = P::PER;
    const int lane = threadIdx.x & 31;
    const int segs = (H + PER * 32 * U - 1) / (PER * 32 * U);
    const int rounds = (K + J - 1) / J, per_round = (K + rounds - 1) / rounds;
    const int64_t nw = (int64_t)gridDim.x * WARPS;
    // row and weight of copy `lane` of token i; the next item's are fetched while this one's rows
    // are on their way
    const auto fetch = [&](int64_t i, int32_t &r, float &v) {
        r = -1;
        v = 0.f;
        if (i < T && lane < K) {
            r = map[i * K + lane];
            v = w != nullptr ? w[i * K + lane] : 1.0f;
        }
    };
    // this item's token and segment, and what a step of the grid adds to them: no division a turn
    const int64_t it = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
    int64_t next_t = it / segs;
    int next_seg = (int)(it - next_t * segs);
    const int64_t step_t = nw / segs;
    const int step_seg = (int)(nw - step_t * segs);
    int32_t next_r;
    float next_w;
    fetch(next_t, next_r, next_w);
    while (next_t < T) {
        const int32_t rk = checked_row(next_r, n_rows, status);
        const float wk = rk >= 0 ? next_w : 0.f;
        const int64_t t = next_t;
        const int seg = next_seg;
        next_t += step_t;
        next_seg += step_seg;
        if (next_seg >= segs) {
            next_seg -= segs;
            ++next_t;
        }
        fetch(next_t, next_r, next_w);
        const int c0 = (seg * 32 * U + lane) * PER;  // first column, step 32 PER
        float acc[U][PER];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int q = 0; q < PER; ++q) acc[u][q] = 0.f;
        for (int k0 = 0; k0 < K; k0 += per_round) {
            P b[J][U];
            float s[J];
            const int kn = K - k0 < per_round ? K - k0 : per_round;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (j >= kn) break;
                const int32_t r = __shfl_sync(0xFFFFFFFFu, rk, k0 + j);
                s[j] = __shfl_sync(0xFFFFFFFFu, wk, k0 + j);
                const uint8_t *p = static_cast<const uint8_t *>(rows) + r * ld_row * B;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    b[j][u].load(p, c0 + u * 32 * PER, r >= 0 && c0 + u * 32 * PER + PER <= H);
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (j >= kn) break;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float v[PER];
                    b[j][u].values(v);
#pragma unroll
                    for (int q = 0; q < PER; ++q) acc[u][q] = fmaf(s[j], v[q], acc[u][q]);
                }
            }
        }
        const uint8_t *resp =
            res != nullptr ? static_cast<const uint8_t *>(res) + t * ld_tok * B : nullptr;
        uint8_t *yp = static_cast<uint8_t *>(y) + t * ld_tok * B;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * 32 * PER;
            if (c + PER <= H) {
                if constexpr (VEC) {
                    if (resp != nullptr) {
                        float v[PER];
                        unpack<F32>(*reinterpret_cast<const uint4 *>(resp + (int64_t)c * B), v);
#pragma unroll
                        for (int q = 0; q < PER; ++q) acc[u][q] += v[q];
                    }
                    *reinterpret_cast<uint4 *>(yp + (int64_t)c * B) = pack<F32>(acc[u]);
                } else {
                    store_elem<F32>(yp, c,
                                    acc[u][0] + (resp != nullptr ? load_elem<F32>(resp, c) : 0.f));
                }
            }
        }
        // the columns past the last whole vector, at most PER - 1: one a lane
        if (VEC && H % PER != 0) {
            const int c = H / PER * PER + lane;
            const int seg_of_tail = (H / PER) / (32 * U);
            if (seg == seg_of_tail) {
                float a = 0.f;
                for (int k0 = 0; k0 < K; k0 += 8) {  // 8 loads in flight
                    float e[8], s[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int k = k0 + j < K ? k0 + j : K - 1;
                        const int32_t r = __shfl_sync(0xFFFFFFFFu, rk, k);
                        s[j] = __shfl_sync(0xFFFFFFFFu, wk, k);
                        e[j] = 0.f;
                        if (k0 + j < K && r >= 0 && c < H)
                            e[j] = load_elem<F32>(
                                static_cast<const uint8_t *>(rows) + r * ld_row * B, c);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (k0 + j < K) a = fmaf(s[j], e[j], a);
                }
                if (c < H)
                    store_elem<F32>(yp, c, a + (resp != nullptr ? load_elem<F32>(resp, c) : 0.f));
            }
        }
    }
}

// ---------------------------------------------------------------- combine backward
// 2^wsh warps per token, as many as the row has segments of 32*U pieces (at most 8, a block);
// warp i of a token takes the segments i, i + 2^wsh, ... The copies go in rounds of equal size, at
// most J: a round's rows are loaded before the first is used, and each lane keeps its part of
// the round's dot products over all its segments. A butterfly that halves the number of values
// at each step (9 shuffles for 8 sums, not 40) adds the lanes, and the warps' parts are added
// in warp order. Items past the tokens' are the pad rows. 8192 tokens x 10 rows x 4096 bf16 233 us,
// 6.1 TB/s; a block a token at any width took 415 us for 32768 x 8 x 264, this 83.
template <bool F32, bool VEC, int J, bool BLOCK>
__global__ void __launch_bounds__(TPB, J == FEW ? FEW_BWD_BLOCKS : COMBINE_BLOCKS)
    combine_bwd_kernel(const void *dy, const void *rows,
                       const int32_t *map, const int32_t *starts,
                       const int32_t *kept, const float *w, int64_t T,
                       int K, int E, int H, int wsh_, int64_t ld_tok, int64_t ld_row,
                       int64_t n_rows, void *drows, float *dw,
                       int *status) {
    let_next_start();
    wait_for_previous();
    using P = Piece<F32, VEC>;
    constexpr int B = Elem<F32>::BYTES, PER = P::PER, U = COMBINE_BWD_U;
    __shared__ float part[WARPS][32];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int wsh = BLOCK ? 3 : wsh_;  // a token per block: known when compiling
    const int wpt = 1 << wsh, warp = wid & (wpt - 1);  // warps of a token, this one among them
    const bool pads = starts != nullptr && drows != nullptr;
    const int rounds = (K + J - 1) / J, per_round = (K + rounds - 1) / rounds;
    const int tail = H / PER * PER;  // the columns from here are taken one a lane, by one warp
    // items: tokens, then the pad rows (one warp each)
    const int64_t items = T + (pads ? (((int64_t)E * 16 - 1) >> wsh) + 1 : 0);
    const int64_t step = (int64_t)gridDim.x * (WARPS >> wsh);
    // row and weight of copy `lane` of token i, the next token's ahead of time
    const auto fetch = [&](int64_t i, int32_t &r, float &v) {
        r = -1;
        v = 0.f;
        if (i < T && lane < K) {
            r = map[i * K + lane];
            v = w != nullptr ? w[i * K + lane] : 1.0f;
        }
    };
    int32_t next_r;
    float next_w;
    int64_t t = (int64_t)blockIdx.x * (WARPS >> wsh) + (wid >> wsh);
    fetch(t, next_r, next_w);
    // every warp of a block makes the same number of turns (they meet at barriers)
    for (int64_t t0 = (int64_t)blockIdx.x * (WARPS >> wsh); t0 < items; t0 += step, t += step) {
        const int32_t rk = checked_row(next_r, n_rows, status);
        const float wk = rk >= 0 ? next_w : 0.f;
        fetch(t + step, next_r, next_w);
        if (t >= T) {
            const int64_t pad = ((t - T) << wsh) + warp;
            if (pads && pad < (int64_t)E * 16)
                zero_pad_row<F32, VEC>(pad, starts, kept, n_rows, H, ld_row, drows, lane);
        } else {
            const uint8_t *dyp = static_cast<const uint8_t *>(dy) + t * ld_tok * B;
            for (int k0 = 0; k0 < K; k0 += per_round) {
                const int kn = K - k0 < per_round ? K - k0 : per_round;
                float acc[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] = 0.f;
                for (int c0 = warp * 32 * PER * U; c0 < H; c0 += wpt * 32 * PER * U) {
                    const int c = c0 + lane * PER;  // and U - 1 more pieces, 32 PER apart
                    P gp[U], b[J][U];
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        gp[u].load(dyp, c + u * 32 * PER, c + u * 32 * PER + PER <= H);
                    if (dw != nullptr) {
#pragma unroll
                        for (int j = 0; j < J; ++j) {
                            if (j >= kn) break;
                            const int32_t r = __shfl_sync(0xFFFFFFFFu, rk, k0 + j);
#pragma unroll
                            for (int u = 0; u < U; ++u)
                                b[j][u].load(static_cast<const uint8_t *>(rows) + r * ld_row * B,
                                             c + u * 32 * PER,
                                             r >= 0 && c + u * 32 * PER + PER <= H);
                        }
                    }
                    float g[U][PER];
#pragma unroll
                    for (int u = 0; u < U; ++u) gp[u].values(g[u]);
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        if (j >= kn) break;
                        if (drows != nullptr) {
                            const int32_t r = __shfl_sync(0xFFFFFFFFu, rk, k0 + j);
                            const float s = __shfl_sync(0xFFFFFFFFu, wk, k0 + j);
                            uint8_t *o = static_cast<uint8_t *>(drows) + r * ld_row * B;
#pragma unroll
                            for (int u = 0; u < U; ++u) {
                                const int cu = c + u * 32 * PER;
                                if (r < 0 || cu + PER > H) continue;
                                float d[PER];
#pragma unroll
                                for (int q = 0; q < PER; ++q) d[q] = s * g[u][q];
                                if constexpr (VEC)
                                    *reinterpret_cast<uint4 *>(o + (int64_t)cu * B) = pack<F32>(d);
                                else
                                    store_elem<F32>(o, cu, d[0]);
                            }
                        }
                        if (dw != nullptr) {
#pragma unroll
                            for (int u = 0; u < U; ++u) {
                                float v[PER];
                                b[j][u].values(v);
#pragma unroll
                                for (int q = 0; q < PER; ++q) acc[j] = fmaf(v[q], g[u][q], acc[j]);
                            }
                        }
                    }
                }
                if (VEC && warp == wpt - 1 && tail < H) {  // the warp with the least else to do
                    const int c = tail + lane;
                    const float g = c < H ? load_elem<F32>(dyp, c) : 0.f;
                    float e[J];
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        if (j >= kn) break;
                        const int32_t r = __shfl_sync(0xFFFFFFFFu, rk, k0 + j);
                        e[j] = 0.f;
                        if (dw != nullptr && r >= 0 && c < H)
                            e[j] = load_elem<F32>(static_cast<const uint8_t *>(rows) + r * ld_row * B,
                                                  c);
                    }
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        if (j >= kn) break;
                        const int32_t r = __shfl_sync(0xFFFFFFFFu, rk, k0 + j);
                        const float s = __shfl_sync(0xFFFFFFFFu, wk, k0 + j);
                        if (drows != nullptr && r >= 0 && c < H)
                            store_elem<F32>(static_cast<uint8_t *>(drows) + r * ld_row * B, c, s * g);
                        acc[j] = fmaf(e[j], g, acc[j]);
                    }
                }
                if (dw != nullptr) {
                    // after the step with lane distance 16, 8, 4 a lane keeps the half of the values
                    // that its lane bit names; the last two add what is left of one value
                    float h4[4], h2[2], h1;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool up = lane & 16;
                        const float give = up ? acc[j] : acc[j + 4], keep = up ? acc[j + 4] : acc[j];
                        h4[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 16);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const bool up = lane & 8;
                        const float give = up ? h4[j] : h4[j + 2], keep = up ? h4[j + 2] : h4[j];
                        h2[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 8);
                    }
                    {
                        const bool up = lane & 4;
                        const float give = up ? h2[0] : h2[1], keep = up ? h2[1] : h2[0];
                        h1 = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 4);
                    }
                    h1 += __shfl_xor_sync(0xFFFFFFFFu, h1, 2);
                    h1 += __shfl_xor_sync(0xFFFFFFFFu, h1, 1);
                    const int j = ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
                    if ((lane & 3) == 0 && j < kn) part[wid][k0 + j] = h1;
                }
            }
        }
        if (dw != nullptr) {
            if (wsh > 0) __syncthreads();
            else __syncwarp();
            if (warp == 0 && lane < K && t < T) {
                float a = 0.f;
                for (int i = 0; i < wpt; ++i) a += part[wid + i][lane];
                dw[t * K + lane] = rk >= 0 ? a : 0.f;  // dropped: zero, whatever dy holds
            }
            if (wsh > 0) __syncthreads();
            else __syncwarp();
        }
    }
}

// ---------------------------------------------------------------- narrow rows
// Rows of at most 16 pieces (a piece is 16 bytes, or one element where rows are not aligned): a
// warp a row would leave most of its lanes idle, so a row gets a group of 2^sh lanes, the least
// power of two that covers its pieces, and a warp holds 32 / 2^sh rows.
// Rows of 65536 tokens x 8 copies of 64 bf16: dispatch 22 us, combine 37, gradient 43; with a
// warp a row 35, 69 and 125. Rows of 32 pieces are faster as whole rows (256 bf16, 32768 tokens x
// 8: 29, 45 and 72 us, against 38, 55 and 78 in groups of 32 lanes), so groups end at 16 lanes.
constexpr int NARROW = 4;  // rows of a dispatch thread, their loads in flight together (2: 41 us
                           // against 37 for 65536 x 8 of 128 bf16); one row in the gradient,
                           // whose loads fill the registers by themselves

template <bool F32, bool VEC>
MOK_DEV void get_piece(const void *p, int64_t row, int64_t ld, int c, int H,
                       float (&v)[VEC ? Elem<F32>::PER : 1]) {
    constexpr int PER = VEC ? Elem<F32>::PER : 1;
    const uint8_t *r = static_cast<const uint8_t *>(p) + row * ld * Elem<F32>::BYTES;
    if constexpr (VEC) {
        if (c + PER <= H) {
            unpack<F32>(*reinterpret_cast<const uint4 *>(r + (int64_t)c * Elem<F32>::BYTES), v);
            return;
        }
    }
#pragma unroll
    for (int q = 0; q < PER; ++q) v[q] = c + q < H ? load_elem<F32>(r, c + q) : 0.f;
}
template <bool F32, bool VEC>
MOK_DEV void put_piece(void *p, int64_t row, int64_t ld, int c, int H,
                       const float (&v)[VEC ? Elem<F32>::PER : 1]) {
    constexpr int PER = VEC ? Elem<F32>::PER : 1;
    uint8_t *r = static_cast<uint8_t *>(p) + row * ld * Elem<F32>::BYTES;
    if constexpr (VEC) {
        if (c + PER <= H) {
            *reinterpret_cast<uint4 *>(r + (int64_t)c * Elem<F32>::BYTES) = pack<F32>(v);
            return;
        }
    }
#pragma unroll
    for (int q = 0; q < PER; ++q)
        if (c + q < H) store_elem<F32>(r, c + q, v[q]);
}

// a piece as it is, bit for bit
template <bool F32, bool VEC>
MOK_DEV void copy_piece(const void *src, int64_t from, int64_t ld_src, void *dst, int64_t to,
                        int64_t ld_dst, int c, int H) {
    constexpr int PER = VEC ? Elem<F32>::PER : 1, B = Elem<F32>::BYTES;
    const uint8_t *a = static_cast<const uint8_t *>(src) + (from * ld_src + c) * B;
    uint8_t *b = static_cast<uint8_t *>(dst) + (to * ld_dst + c) * B;
    if constexpr (VEC) {
        if (c + PER <= H) {
            *reinterpret_cast<uint4 *>(b) = *reinterpret_cast<const uint4 *>(a);
            return;
        }
    }
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        if (c + q >= H) continue;
        if (F32)
            reinterpret_cast<uint32_t *>(b)[q] = reinterpret_cast<const uint32_t *>(a)[q];
        else
            reinterpret_cast<uint16_t *>(b)[q] = reinterpret_cast<const uint16_t *>(a)[q];
    }
}

// the pad row of item i (see zero_pad_row), one piece
template <bool F32, bool VEC>
MOK_DEV void zero_pad_piece(int64_t item, const int32_t *starts, const int32_t *kept,
                            int64_t n_rows, int c, int H, int64_t ld, void *out) {
    const int e = (int)(item >> 4), j = (int)(item & 15);
    const int64_t n = kept[e], row = starts[e] + n + j;
    if (n + j >= ((n + 15) & ~(int64_t)15) || row < 0 || row >= n_rows) return;
    float z[VEC ? Elem<F32>::PER : 1] = {};
    put_piece<F32, VEC>(out, row, ld, c, H, z);
}

template <bool F32, bool VEC>
__global__ void __launch_bounds__(TPB)
    dispatch_narrow_kernel(const void *x, const int32_t *map,
                           const int32_t *starts, const int32_t *kept,
                           int64_t T, int K, int E, int H, int sh, int64_t ld_tok, int64_t ld_row,
                           int64_t n_rows, void *xs, int *status) {
    let_next_start();
    wait_for_previous();
    constexpr int PER = VEC ? Elem<F32>::PER : 1;
    const int64_t R = T * K, i0 = (int64_t)blockIdx.x * TPB * NARROW + threadIdx.x;
    const int c = (int)(i0 & ((1 << sh) - 1)) * PER;  // the same for all of the thread's rows
    if (c >= H) return;
    int32_t r[NARROW];
#pragma unroll
    for (int j = 0; j < NARROW; ++j) {  // the rows' lookups in flight together
        const int64_t f = (i0 + j * TPB) >> sh;
        r[j] = f < R ? map[f] : -1;
    }
#pragma unroll
    for (int j = 0; j < NARROW; ++j) {
        const int64_t f = (i0 + j * TPB) >> sh;
        const int32_t to = checked_row(r[j], n_rows, status);
        if (to >= 0)
            copy_piece<F32, VEC>(x, (uint32_t)f / (uint32_t)K, ld_tok, xs, to, ld_row, c, H);
        else if (f >= R && starts != nullptr && f - R < (int64_t)E * 16)
            zero_pad_piece<F32, VEC>(f - R, starts, kept, n_rows, c, H, ld_row, xs);
    }
}

template <bool F32, bool VEC>
__global__ void __launch_bounds__(TPB)
    combine_narrow_kernel(const void *rows, const int32_t *map,
                          const float *w, const void *res, int64_t T, int K, int H,
                          int sh, int64_t ld_tok, int64_t ld_row, int64_t n_rows, void *y,
                          int *status) {
    let_next_start();
    wait_for_previous();
    constexpr int PER = VEC ? Elem<F32>::PER : 1;
    const int64_t i = (int64_t)blockIdx.x * TPB + threadIdx.x, t = i >> sh;
    const int c = (int)(i & ((1 << sh) - 1)) * PER;
    if (t >= T || c >= H) return;
    float acc[PER] = {};
    for (int k0 = 0; k0 < K; k0 += 4) {  // 4 rows in flight
        float v[4][PER], s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int32_t r = k0 + j < K ? row_of(map, t * K + k0 + j, n_rows, status) : -1;
            s[j] = r >= 0 ? (w != nullptr ? w[t * K + k0 + j] : 1.0f) : 0.f;
            if (r >= 0) {
                get_piece<F32, VEC>(rows, r, ld_row, c, H, v[j]);
            } else {
#pragma unroll
                for (int q = 0; q < PER; ++q) v[j][q] = 0.f;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < PER; ++q) acc[q] = fmaf(s[j], v[j][q], acc[q]);
    }
    if (res != nullptr) {
        float v[PER];
        get_piece<F32, VEC>(res, t, ld_tok, c, H, v);
#pragma unroll
        for (int q = 0; q < PER; ++q) acc[q] += v[q];
    }
    put_piece<F32, VEC>(y, t, ld_tok, c, H, acc);
}

template <bool F32, bool VEC>
__global__ void __launch_bounds__(TPB)
    combine_bwd_narrow_kernel(const void *dy, const void *rows,
                              const int32_t *map,
                              const int32_t *starts,
                              const int32_t *kept, const float *w,
                              int64_t T, int K, int E, int H, int sh, int64_t ld_tok,
                              int64_t ld_row, int64_t n_rows, void *drows,
                              float *dw, int *status) {
    let_next_start();
    wait_for_previous();
    constexpr int PER = VEC ? Elem<F32>::PER : 1;
    const int64_t i = (int64_t)blockIdx.x * TPB + threadIdx.x, f = i >> sh;
    const int v0 = (int)(i & ((1 << sh) - 1)), c = v0 * PER;
    const int64_t R = T * K;
    float dot = 0.f;
    if (f < R && c < H) {
        const int32_t r = row_of(map, f, n_rows, status);
        if (r >= 0) {
            float g[PER];
            get_piece<F32, VEC>(dy, (uint32_t)f / (uint32_t)K, ld_tok, c, H, g);
            if (dw != nullptr) {
                float v[PER];
                get_piece<F32, VEC>(rows, r, ld_row, c, H, v);
#pragma unroll
                for (int q = 0; q < PER; ++q) dot = fmaf(v[q], g[q], dot);
            }
            if (drows != nullptr) {
                const float s = w != nullptr ? w[f] : 1.0f;
#pragma unroll
                for (int q = 0; q < PER; ++q) g[q] *= s;
                put_piece<F32, VEC>(drows, r, ld_row, c, H, g);
            }
        }
    } else if (f >= R && f - R < (int64_t)E * 16 && c < H && starts != nullptr &&
               drows != nullptr) {
        zero_pad_piece<F32, VEC>(f - R, starts, kept, n_rows, c, H, ld_row, drows);
    }
    if (dw != nullptr) {  // the group's lanes, all of the warp taking part
        for (int o = (1 << sh) >> 1; o > 0; o >>= 1)
            dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
        if (v0 == 0 && f < R) dw[f] = dot;
    }
}

// rows start on 16-byte boundaries: both strides are multiples of 16 bytes
bool vectors(const mok_rows_config &c) {
    const int per = c.dtype == MOK_DTYPE_F32 ? 4 : 8;
    return c.ld_tok % per == 0 && c.ld_row % per == 0;
}

// lanes of a narrow row's group, as a shift; -1 for rows of more than 16 pieces
int narrow_shift(const mok_rows_config &c) {
    const int per = vectors(c) ? (c.dtype == MOK_DTYPE_F32 ? 4 : 8) : 1;
    const int pieces = (c.H + per - 1) / per;
    int sh = 0;
    while ((1 << sh) < pieces && sh < 5) ++sh;
    return sh <= 4 ? sh : -1;
}
int64_t narrow_blocks(int64_t items, int sh, int per_thread) {
    return ((items << sh) + TPB * per_thread - 1) / (TPB * per_thread);
}

}  // namespace

// instantiate KERNEL<F32, VEC> for the configuration
#define MOK_ROWS_CASES(c, CALL)                          \
    do {                                                 \
        const bool _v = vectors(c);                      \
        if ((c).dtype == MOK_DTYPE_F32) {                \
            if (_v) { CALL(true, true); }                \
            else { CALL(true, false); }                  \
        } else {                                         \
            if (_v) { CALL(false, true); }               \
            else { CALL(false, false); }                 \
        }                                                \
    } while (0)

cudaError_t launch_build_row_map(const mok_rows_config &c, const int32_t *idx,
                                 const mok_schedule &sch, int32_t *map, int32_t *starts,
                                 int32_t *kept, int *status, cudaStream_t s) {
    const int64_t R = (int64_t)c.T * c.K;
    return launch_edge(row_map_kernel, grid_for(R, MAX_E, 1), MAX_E, 0, 1, s, idx, sch.counts,
                       sch.offsets, sch.inv, R, c.E, c.capacity, c.n_rows, map, starts, kept, status);
}

cudaError_t launch_dispatch_rows(const mok_rows_config &c, const void *x, const int32_t *map,
                                 const int32_t *starts, const int32_t *kept, void *xs,
                                 int *status, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    constexpr int U = 4;
    const int per = vectors(c) ? (c.dtype == MOK_DTYPE_F32 ? 4 : 8) : 1;
    const int64_t segs = (c.H + per * 32 * U - 1) / (per * 32 * U);
    const int64_t items = c.T * segs + (starts != nullptr ? (int64_t)c.E * 16 : 0);
    if (items == 0) return cudaSuccess;
    if (const int sh = narrow_shift(c); sh >= 0) {
        const int64_t rows = (int64_t)c.T * c.K + (starts != nullptr ? (int64_t)c.E * 16 : 0);
        const int64_t blocks = narrow_blocks(rows, sh, NARROW);
        if (blocks <= 0x7FFFFFFF) {
#define CALL(F, V)                                                                          \
    e = launch_edge(dispatch_narrow_kernel<F, V>, (unsigned)blocks, TPB, 0, 1, s, \
        x, map, starts, kept, c.T, c.K, c.E, c.H, sh, c.ld_tok, c.ld_row, c.n_rows, xs, status)
            MOK_ROWS_CASES(c, CALL);
#undef CALL
            return e;
        }
    }
#define CALL(F, V)                                                                        \
    e = launch_edge(dispatch_kernel<F, V, U>, grid_for(items, WARPS, DISPATCH_BLOCKS), TPB, 0, 1, \
                    s, x, map, starts, kept, c.T, c.K, c.E, c.H, c.ld_tok, c.ld_row, c.n_rows,    \
                    xs, status)
    MOK_ROWS_CASES(c, CALL);
#undef CALL
    return e;
}

cudaError_t launch_combine_rows(const mok_rows_config &c, const void *rows, const int32_t *map,
                                const float *w, const void *res, void *y, int *status,
                                cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (c.T == 0) return cudaSuccess;
    const int per = vectors(c) ? (c.dtype == MOK_DTYPE_F32 ? 4 : 8) : 1;
    if (const int sh = narrow_shift(c); sh >= 0) {
        const int64_t blocks = narrow_blocks(c.T, sh, 1);
        if (blocks <= 0x7FFFFFFF) {
#define CALL(F, V)                                                               \
    e = launch_edge(combine_narrow_kernel<F, V>, (unsigned)blocks, TPB, 0, 1, s, \
        rows, map, w, res, c.T, c.K, c.H, sh, c.ld_tok, c.ld_row, c.n_rows, y, status)
            MOK_ROWS_CASES(c, CALL);
#undef CALL
            return e;
        }
    }
    // rows that two pieces a lane cover gain nothing from longer segments (4 copies of 264 bf16:
    // 41 us against 35 us)
    const bool few = c.K <= FEW && c.H > per * 32 * COMBINE_U;
    const int U = few ? FEW_U : COMBINE_U;
    const int64_t items = (int64_t)c.T * ((c.H + per * 32 * U - 1) / (per * 32 * U));
    const unsigned grid = grid_for(items, WARPS, COMBINE_BLOCKS);
#define ROWS(F, V, J, U)                                                               \
    e = launch_edge(combine_rows_kernel<F, V, J, U>, grid, TPB, 0, 1, s, \
        rows, map, w, res, c.T, c.K, c.H, c.ld_tok, c.ld_row, c.n_rows, y, status)
#define CALL(F, V)                           \
    if (few) ROWS(F, V, FEW, FEW_U);         \
    else ROWS(F, V, 8, COMBINE_U)
    MOK_ROWS_CASES(c, CALL);
#undef ROWS
#undef CALL
    return e;
}

cudaError_t launch_combine_bwd(const mok_rows_config &c, const void *dy, const void *rows,
                               const int32_t *map, const int32_t *starts, const int32_t *kept,
                               const float *w, void *drows, float *dw, int *status,
                               cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    const bool has_pads = starts != nullptr && drows != nullptr;
    if (c.T == 0 && !has_pads) return cudaSuccess;
    if (const int sh = narrow_shift(c); sh >= 0) {
        const int64_t n = (int64_t)c.T * c.K + (has_pads ? (int64_t)c.E * 16 : 0);
        const int64_t blocks = narrow_blocks(n, sh, 1);
        if (blocks <= 0x7FFFFFFF) {
#define CALL(F, V)                                                                            \
    e = launch_edge(combine_bwd_narrow_kernel<F, V>, (unsigned)blocks, TPB, 0, 1, s, \
        dy, rows, map, starts, kept, w, c.T, c.K, c.E, c.H, sh, c.ld_tok, c.ld_row, c.n_rows, \
        drows, dw, status)
            MOK_ROWS_CASES(c, CALL);
#undef CALL
            return e;
        }
    }
    const int per = vectors(c) ? (c.dtype == MOK_DTYPE_F32 ? 4 : 8) : 1;
    const int segs = (c.H + per * 32 * COMBINE_BWD_U - 1) / (per * 32 * COMBINE_BWD_U);
    int wsh = 0;
    while ((1 << wsh) < segs && (1 << wsh) < WARPS) ++wsh;
    const int64_t items = c.T + (has_pads ? (((int64_t)c.E * 16 - 1) >> wsh) + 1 : 0);
    const bool few = c.K <= FEW;
    const unsigned grid = grid_for(items, WARPS >> wsh, few ? FEW_BWD_BLOCKS : COMBINE_BLOCKS);
#define BWD(F, V, J, BLOCK)                                                                    \
    e = launch_edge(combine_bwd_kernel<F, V, J, BLOCK>, grid, TPB, 0, 1, s, \
        dy, rows, map, starts, kept, w, c.T, c.K, c.E, c.H, wsh, c.ld_tok, c.ld_row, c.n_rows, \
        drows, dw, status)
#define CALL(F, V)                           \
    if (few) {                               \
        if (wsh == 3) BWD(F, V, FEW, true);  \
        else BWD(F, V, FEW, false);          \
    } else {                                 \
        if (wsh == 3) BWD(F, V, 8, true);    \
        else BWD(F, V, 8, false);            \
    }
    MOK_ROWS_CASES(c, CALL);
#undef BWD
#undef CALL
    return e;
}

}  // namespace mok

// ---------------------------------------------------------------- entry points
using namespace mok;

extern "C" {

mok_status mok_check_rows_config(const mok_rows_config *c) {
    if (c == nullptr) return MOK_ERR_INVALID_ARG;
    if (c->abi_version != MOK_ABI_VERSION) return MOK_ERR_ABI;
    if (c->T < 0 || c->K < 1 || c->K > 32 || c->E < 1 || c->E > MAX_E || c->H < 1)
        return MOK_ERR_INVALID_ARG;
    if (c->H > (1 << 24)) return MOK_ERR_INVALID_ARG;
    if ((int64_t)c->T * c->K > 0x7FFFFFFF) return MOK_ERR_INVALID_ARG;
    if (c->dtype != MOK_DTYPE_BF16 && c->dtype != MOK_DTYPE_F32) return MOK_ERR_INVALID_ARG;
    if (c->capacity < 0 || c->reserved != 0) return MOK_ERR_INVALID_ARG;
    if (c->n_rows < 0 || c->n_rows > 0x7FFFFFFF) return MOK_ERR_INVALID_ARG;
    const int64_t most = (int64_t)1 << 30;
    if (c->ld_tok < c->H || c->ld_row < c->H || c->ld_tok > most || c->ld_row > most)
        return MOK_ERR_INVALID_ARG;
    return MOK_OK;
}

mok_status mok_build_row_map(const mok_rows_config *c, const int32_t *topk_idx,
                             const mok_schedule *sch, int32_t *row_map, int32_t *starts,
                             int32_t *kept, cudaStream_t stream) {
    mok_status st = mok_check_rows_config(c);
    if (st != MOK_OK) return st;
    int *status;
    if ((st = current_device_status_word(&status)) != MOK_OK) return st;
    if (!sch || !sch->counts || !sch->offsets || !starts || !kept) return MOK_ERR_INVALID_ARG;
    if (c->T > 0 && (!topk_idx || !row_map || !sch->inv)) return MOK_ERR_INVALID_ARG;
    const void *ps[] = {topk_idx, row_map, starts, kept, sch->counts, sch->offsets, sch->inv};
    for (const void *p : ps)
        if (p && !op_aligned16(p)) return MOK_ERR_INVALID_ARG;
    MOK_OP_LAUNCH(OP_ROW_MAP, 1,
               launch_build_row_map(*c, topk_idx, *sch, row_map, starts, kept, status, stream));
    return MOK_OK;
}

mok_status mok_dispatch(const mok_rows_config *c, const void *x, const int32_t *row_map,
                        const int32_t *starts, const int32_t *kept, void *xs,
                        cudaStream_t stream) {
    mok_status st = mok_check_rows_config(c);
    if (st != MOK_OK) return st;
    int *status;
    if ((st = current_device_status_word(&status)) != MOK_OK) return st;
    if ((starts == nullptr) != (kept == nullptr)) return MOK_ERR_INVALID_ARG;
    if (c->T > 0 && (!x || !row_map)) return MOK_ERR_INVALID_ARG;
    if (!xs && c->n_rows > 0) return MOK_ERR_INVALID_ARG;
    const void *ps[] = {x, row_map, starts, kept, xs};
    for (const void *p : ps)
        if (p && !op_aligned16(p)) return MOK_ERR_INVALID_ARG;
    MOK_OP_LAUNCH(OP_DISPATCH, 1,
               launch_dispatch_rows(*c, x, row_map, starts, kept, xs, status, stream));
    return MOK_OK;
}

mok_status mok_combine(const mok_rows_config *c, const void *rows, const int32_t *row_map,
                       const float *topk_w, const void *residual, void *y,
                       cudaStream_t stream) {
    mok_status st = mok_check_rows_config(c);
    if (st != MOK_OK) return st;
    int *status;
    if ((st = current_device_status_word(&status)) != MOK_OK) return st;
    if (c->T > 0 && (!row_map || !y || (!rows && c->n_rows > 0))) return MOK_ERR_INVALID_ARG;
    const void *ps[] = {rows, row_map, topk_w, residual, y};
    for (const void *p : ps)
        if (p && !op_aligned16(p)) return MOK_ERR_INVALID_ARG;
    MOK_OP_LAUNCH(OP_COMBINE, 1,
               launch_combine_rows(*c, rows, row_map, topk_w, residual, y, status, stream));
    return MOK_OK;
}

mok_status mok_dispatch_backward(const mok_rows_config *c, const void *dxs,
                                 const int32_t *row_map, void *dx, cudaStream_t stream) {
    return mok_combine(c, dxs, row_map, nullptr, nullptr, dx, stream);
}

mok_status mok_combine_backward(const mok_rows_config *c, const void *dy, const void *rows,
                                const int32_t *row_map, const int32_t *starts,
                                const int32_t *kept, const float *topk_w, void *drows,
                                float *d_topk_w, cudaStream_t stream) {
    mok_status st = mok_check_rows_config(c);
    if (st != MOK_OK) return st;
    int *status;
    if ((st = current_device_status_word(&status)) != MOK_OK) return st;
    if (!drows && !d_topk_w) return MOK_ERR_INVALID_ARG;
    if ((starts == nullptr) != (kept == nullptr)) return MOK_ERR_INVALID_ARG;
    if (c->T > 0 && (!dy || !row_map)) return MOK_ERR_INVALID_ARG;
    if (c->T > 0 && d_topk_w && !rows && c->n_rows > 0) return MOK_ERR_INVALID_ARG;
    const void *ps[] = {dy, rows, row_map, starts, kept, topk_w, drows, d_topk_w};
    for (const void *p : ps)
        if (p && !op_aligned16(p)) return MOK_ERR_INVALID_ARG;
    MOK_OP_LAUNCH(OP_COMBINE_BWD, 1,
               launch_combine_bwd(*c, dy, rows, row_map, starts, kept, topk_w, drows, d_topk_w,
                                  status, stream));
    return MOK_OK;
}

}  // extern "C"

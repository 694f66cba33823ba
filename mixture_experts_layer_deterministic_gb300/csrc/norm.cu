// norm.cu -- layer norm and RMS norm of a residual sum, and their gradients.
//
//   h = x + residual, n = (h - mean) rstd, y = n w + b
//   g = dy w, dx = dh + rstd (g - n mean(g n) - mean(g)), dw = sum dy n, db = sum dy
//
// All of it is HBM traffic. A row belongs to a team, a power of two of threads up to a warp or some
// warps of a block, that hold NV vectors of 8 elements each; long rows are cut over the blocks of a
// cluster, which exchange their sums through each other's shared memory. Blocks walk over the rows, and
// a thread's pieces of the next rows are on their way to shared memory of its own (cp.async, which also
// fills in the zeros past a row's end), so that the loads never pause and hold no registers. Rows too
// long for a cluster are read again instead. The mean is taken in two steps (of h, then of h less the first), so
// that rows far from zero keep their digits; the variance is that of h less the mean.
#include <atomic>

#include "ops_internal.h"
#include "tc.cuh"

namespace mok {
namespace {

constexpr int NORM_TPB = 512;

// 8 elements as they lie in memory
template <bool F32>
struct Raw {
    uint4 v[F32 ? 2 : 1];
};
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
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = c + j >= H ? 0.0f
                   : F32      ? static_cast<const float *>(row)[c + j]
                              : bf16_to_f32(static_cast<const uint16_t *>(row)[c + j]);
    }
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
                pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (c + j >= H) continue;
            if (F32)
                static_cast<float *>(row)[c + j] = v[j];
            else
                static_cast<uint16_t *>(row)[c + j] = f32_to_bf16(v[j]);
        }
    }
}
// `left` of 8 elements at p
template <bool F32>
MOK_DEV void store_left(void *p, int left, const float (&v)[8]) {
    store8<F32>(p, 0, left, v);
}
// as it will be read back
template <bool F32>
MOK_DEV float rounded(float v) {
    return F32 ? v : bf16_to_f32(f32_to_bf16(v));
}

// two fp32 values in one register pair, and the pipe's instructions on both at once
typedef unsigned long long f32x2;
MOK_DEV f32x2 pair(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
MOK_DEV float2 both(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
MOK_DEV f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
MOK_DEV f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
MOK_DEV f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

struct NormShape {
    int64_t rows, ld_x, ld_y;
    int H;
    int tpr;      // threads of a team
    int cluster;  // blocks of a row
    bool layer;
    float eps;
    int *status;
};

template <bool F32>
MOK_DEV const void *row_of(const void *p, int64_t r, int64_t ld) {
    return static_cast<const char *>(p) + r * ld * (F32 ? 4 : 2);
}
template <bool F32>
MOK_DEV void *row_of(void *p, int64_t r, int64_t ld) {
    return static_cast<char *>(p) + r * ld * (F32 ? 4 : 2);
}

template <bool F32>
MOK_DEV void unpack(const Raw<F32> &q, f32x2 (&v)[4]) {
    const uint4 b = q.v[F32 ? 1 : 0];
    const uint32_t w[8] = {q.v[0].x, q.v[0].y, q.v[0].z, q.v[0].w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = F32 ? pair(__uint_as_float(w[F32 ? 2 * j : j]), __uint_as_float(w[F32 ? 2 * j + 1 : j]))
                   : pair(bf16_lo(w[j]), bf16_hi(w[j]));
}
// A thread's pieces of the rows ahead: `stages` rows of UNITS 16-byte units, each in a place of its own.
// Nobody else reads them, so there is no barrier; a place is filled again when its row is done with.
struct Ahead {
    uint32_t base, stage_bytes, unit_bytes;
    MOK_DEV Ahead(void *smem, int units) {
        unit_bytes = blockDim.x * 16;
        stage_bytes = unit_bytes * units;
        base = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
    }
    MOK_DEV uint32_t at(int stage, int unit) const { return base + stage * stage_bytes + unit * unit_bytes; }
    // `left` elements (up to 8) from p on into unit `u` (and the next), zeros for the rest; nothing is
    // read where there are none, p has to be an address all the same
    template <bool F32>
    MOK_DEV void fetch(int stage, int u, const void *p, int left) const {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) {
            const int bytes = F32 ? min(max(4 * left - 16 * i, 0), 16) : 2 * left;
            const char *q = static_cast<const char *>(p) + (bytes > 0 ? 16 * i : 0);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(stage, u + i)), "l"(q),
                         "r"(bytes)
                         : "memory");
        }
    }
    template <bool F32>
    MOK_DEV void take(int stage, int u, Raw<F32> &q) const {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(q.v[i].x), "=r"(q.v[i].y), "=r"(q.v[i].z), "=r"(q.v[i].w)
                         : "r"(at(stage, u + i))
                         : "memory");
    }
    MOK_DEV static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    template <int N>
    MOK_DEV static void wait() {
        asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
    }
};
template <bool F32>
constexpr int units_of() {
    return F32 ? 2 : 1;
}

// Where a thread's vectors lie: number k is column 8 (first + k tpr).
struct Place {
    int first, slot, slots;  // slot: the team's number in its block
    MOK_DEV Place(const NormShape &s, int nv, uint32_t rank) {
        slot = threadIdx.x / s.tpr;
        slots = blockDim.x / s.tpr;
        first = threadIdx.x - slot * s.tpr + (int)rank * nv * s.tpr;
    }
};

// Sums of a and b over a team, the same in all of its threads. Teams of more than a warp: through sh
// [2][warps of the block], its halves in turn, so that one barrier of the team is enough. CLUSTER: then
// over the blocks of the cluster, each sending its sums to all of them (across [2][blocks]), where they
// are counted in by a barrier in shared memory. (A barrier of the cluster would have to wait for the
// stores of the row before: 2000 rows of 16384 fp32 in four blocks 241 us with one.) A half is sent to
// again only by blocks that have this block's next sums, which it sends when all of it has read.
constexpr int MOST_BLOCKS = 8;  // of a cluster
struct NormShared {
    float2 warps[2][32];
    float2 across[2][MOST_BLOCKS];
    uint64_t arrived[2];
    int gave_up;
};
template <bool CLUSTER>
struct TeamSum {
    NormShared *sh;
    int tpr, blocks;
    uint32_t rank;
    int *status;
    uint32_t calls;
    MOK_DEV TeamSum(NormShared *shared, const NormShape &s, uint32_t r)
        : sh(shared), tpr(s.tpr), blocks(s.cluster), rank(r), status(s.status), calls(0) {
        if constexpr (CLUSTER) {
            if (threadIdx.x == 0) {
                tc::mbar_init(&sh->arrived[0], 1);
                tc::mbar_init(&sh->arrived[1], 1);
                sh->gave_up = 0;
                tc::fence_mbar_init();
            }
            together();  // all blocks are there to be sent to
        }
    }
    MOK_DEV void operator()(float &a) {
        float none = 0.0f;
        add<false>(a, none);
    }
    MOK_DEV void operator()(float &a, float &b) { add<true>(a, b); }
    template <bool TWO>
    MOK_DEV void add(float &a, float &b) {
        const auto warp_sum = [&](int o) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            if (TWO) b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        };
        if (tpr < 32) {
            for (int o = 1; o < tpr; o <<= 1) warp_sum(o);
            return;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) warp_sum(o);
        if (tpr == 32) return;
        const int warp = threadIdx.x >> 5, n = tpr / 32, team = warp / n;
        const uint32_t turn = calls & 1;
        float2 *s = sh->warps[turn];
        if ((threadIdx.x & 31) == 0) s[warp] = make_float2(a, b);
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(tpr) : "memory");
        a = b = 0.0f;
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float2 v = s[team * n + k];
            a += v.x;
            if (TWO) b += v.y;
        }
        if constexpr (CLUSTER) {
            uint64_t *bar = &sh->arrived[turn];
            if (threadIdx.x == 0) tc::mbar_arrive_expect_tx(bar, (uint32_t)blocks * 8u);
            if (threadIdx.x < blocks) {
                uint32_t to, at;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                             : "=r"(to)
                             : "r"(tc::smem_u32(&sh->across[turn][rank])), "r"(threadIdx.x));
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                             : "=r"(at)
                             : "r"(tc::smem_u32(bar)), "r"(threadIdx.x));
                asm volatile(
                    "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::
                        "r"(to), "f"(a), "f"(b), "r"(at)
                    : "memory");
            }
            wait(bar, (calls >> 1) & 1);
            a = b = 0.0f;
            for (int k = 0; k < blocks; ++k) {
                const float2 v = sh->across[turn][k];
                a += v.x;
                b += v.y;
            }
        }
        ++calls;
    }
    // until the blocks' sums are here: bounded, once for all
    MOK_DEV void wait(uint64_t *bar, uint32_t parity) {
        uint64_t t0 = 0;
        for (uint32_t n = 1;; ++n) {
            uint32_t ok;
            asm volatile(
                "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
                "selp.u32 %0, 1, 0, p;\n}\n"
                : "=r"(ok)
                : "r"(tc::smem_u32(bar)), "r"(parity)
                : "memory");
            if (ok) return;
            if ((n & 63u) != 0) continue;
            if (*(volatile int *)&sh->gave_up) return;
            const uint64_t t = tc::globaltimer();
            if (t0 == 0) t0 = t;
            if (t - t0 > tc::WAIT_LIMIT_NS) {
                raise_status(status, MOK_ERR_TIMEOUT);
                *(volatile int *)&sh->gave_up = 1;
                return;
            }
        }
    }
    // all blocks of the cluster
    MOK_DEV void together() const {
        if constexpr (CLUSTER)
            asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
    }
};
template <bool CLUSTER>
MOK_DEV uint32_t block_of_cluster() {
    uint32_t r = 0;
    if (CLUSTER) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

struct NormFwd {
    NormShape s;
    const void *x, *res;
    const float *w, *b;
    void *h, *y;
    float *mean, *rstd;
};

// Vectors a thread. A row's own work is some 100 instructions a warp, so long rows take as many vectors
// as registers and the rows ahead allow: four of bf16 with two sums a row (layer), two with one (RMS, fp32).
// Short rows take one, which leaves room for two blocks a SM. 16384 x 4096 bf16, layer and RMS: 139 and 90
// us with one, 117 and 86 with two (6.2 TB/s), 89 and 99 with four; 20000 x 1111: 52, 58, 62; 1000000 x
// 16: 24, 34, 43.
int fwd_vecs(const mok_norm_config &c) {
    if (c.H <= 2048) return 1;
    return c.x_dtype == MOK_DTYPE_F32 || c.kind == MOK_NORM_RMS ? 2 : 4;
}
constexpr int blocks_of_sm(int nv) { return nv == 1 ? 2 : 1; }
constexpr int FWD_STAGES = 2;  // three do not help: 92 us for the layer norm above, 89 with two

// columns past H of a vector are zeros: they add to no sum but that of (0 - mean)^2
MOK_DEV float square_from(const float (&v)[8], float mean, int n) {
    float q = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) q = fmaf(v[j] - mean, v[j] - mean, q);
    return q;
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

template <int NV, bool X32, bool Y32, bool CLUSTER>
__global__ void __launch_bounds__(NORM_TPB, NV == 1 ? 2 : 0) norm_kernel(const NormFwd a) {
    extern __shared__ __align__(16) uint8_t norm_smem[];
    __shared__ NormShared sh;
    constexpr int U = units_of<X32>(), XS = X32 ? 4 : 2, YS = Y32 ? 4 : 2;
    const NormShape &s = a.s;
    const uint32_t rank = block_of_cluster<CLUSTER>();
    TeamSum<CLUSTER> team_sum(&sh, s, rank);
    const Ahead ahead(norm_smem, 2 * NV * U);
    let_next_start();
    wait_for_previous();
    const Place at(s, NV, rank);
    const int64_t walkers = CLUSTER ? gridDim.x / s.cluster : gridDim.x;
    const int64_t walker = CLUSTER ? blockIdx.x / s.cluster : blockIdx.x, step = walkers * at.slots;
    const int64_t first = walker * at.slots + at.slot;
    // the thread's vectors, and what of them is in the row
    int col[NV], left[NV];
    float w[NV][8], b[NV][8];  // weight and bias stay: from memory they would be waited for in every row
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = 8 * (at.first + k * s.tpr);
        left[k] = min(max(s.H - c, 0), 8);
        col[k] = left[k] > 0 ? c : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[k][j] = a.w != nullptr && c + j < s.H ? a.w[c + j] : 1.0f;
            b[k][j] = a.b != nullptr && c + j < s.H ? a.b[c + j] : 0.0f;
        }
    }
    const char *px = static_cast<const char *>(row_of<X32>(a.x, first, s.ld_x));
    const char *pr = static_cast<const char *>(row_of<X32>(a.res, first, s.ld_x));
    const int64_t dx = step * s.ld_x * XS;
    const auto fetch = [&](int stage, int64_t r) {
        const bool in = r < s.rows;
        const char *qx = in ? px : static_cast<const char *>(a.x), *qr = in ? pr : static_cast<const char *>(a.res);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            ahead.fetch<X32>(stage, k * U, qx + col[k] * XS, in ? left[k] : 0);
            if (a.res != nullptr) ahead.fetch<X32>(stage, (NV + k) * U, qr + col[k] * XS, in ? left[k] : 0);
        }
        ahead.commit();
        px += dx;
        pr += dx;
    };
#pragma unroll
    for (int k = 0; k < FWD_STAGES; ++k) fetch(k, first + k * step);
    char *ph = static_cast<char *>(row_of<X32>(a.h, first, s.ld_x));
    char *py = static_cast<char *>(row_of<Y32>(a.y, first, s.ld_y));
    const int64_t dy = step * s.ld_y * YS;
    const float inv_n = 1.0f / s.H;
    int stage = 0;
    for (int64_t r = first, r0 = walker * at.slots; r0 < s.rows; r0 += step, r += step, ph += dx, py += dy) {
        const bool in = r < s.rows;
        ahead.wait<FWD_STAGES - 1>();
        f32x2 v[NV][4], sum2 = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            Raw<X32> q;
            ahead.take<X32>(stage, k * U, q);
            unpack<X32>(q, v[k]);
            if (a.res != nullptr) {
                Raw<X32> e;
                f32x2 f[4];
                ahead.take<X32>(stage, (NV + k) * U, e);
                unpack<X32>(e, f);
                float o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[k][j] = add2(v[k][j], f[j]);
                    if (!X32) {  // as it is stored, and read by the backward pass
                        const uint32_t p = pack2(both(v[k][j]).x, both(v[k][j]).y);
                        v[k][j] = pair(bf16_lo(p), bf16_hi(p));
                    }
                    o[2 * j] = both(v[k][j]).x;
                    o[2 * j + 1] = both(v[k][j]).y;
                }
                if (a.h != nullptr && in) store_left<X32>(ph + col[k] * XS, left[k], o);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) sum2 = add2(sum2, v[k][j]);
        }
        float mean = 0.0f, rest = 0.0f;
        if (s.layer) {
            mean = both(sum2).x + both(sum2).y;
            team_sum(mean);
            mean *= inv_n;
            const f32x2 minus = pair(-mean, -mean);
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[k][j] = add2(v[k][j], minus);
                    if (2 * j + 1 >= left[k]) {  // past the row
                        const float2 d = both(v[k][j]);
                        v[k][j] = pair(2 * j < left[k] ? d.x : 0.0f, 0.0f);
                    }
                }
        }
        f32x2 sq2 = 0, rest2 = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sq2 = fma2(v[k][j], v[k][j], sq2);
                rest2 = add2(rest2, v[k][j]);
            }
        float sq = both(sq2).x + both(sq2).y;
        if (s.layer) {
            rest = both(rest2).x + both(rest2).y;
            team_sum(sq, rest);
            rest *= inv_n;  // what the mean's rounding left
        } else {
            team_sum(sq);
        }
        fetch(stage, r + FWD_STAGES * step);
        stage = stage + 1 == FWD_STAGES ? 0 : stage + 1;
        const float var = fmaxf(sq * inv_n - rest * rest, 0.0f);
        const float rstd = 1.0f / sqrtf(var + s.eps);
        if (!in) continue;
        if (at.first == 0) {
            if (a.mean != nullptr) a.mean[r] = mean + rest;
            if (a.rstd != nullptr) a.rstd[r] = rstd;
        }
        const f32x2 scale = pair(rstd, rstd), shift = pair(-rest * rstd, -rest * rstd);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (left[k] == 0) continue;
            float o[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x2 n = fma2(v[k][j], scale, shift);
                const f32x2 y = fma2(n, pair(w[k][2 * j], w[k][2 * j + 1]), pair(b[k][2 * j], b[k][2 * j + 1]));
                o[2 * j] = both(y).x;
                o[2 * j + 1] = both(y).y;
            }
            store_left<Y32>(py + col[k] * YS, left[k], o);
        }
    }
    ahead.wait<0>();
    team_sum.together();  // nobody sends to a block that has left
}

// h of 8 columns
template <bool X32>
MOK_DEV void load_h(const NormFwd &a, int64_t r, int c, float (&v)[8]) {
    load8<X32>(row_of<X32>(a.x, r, a.s.ld_x), c, a.s.H, v);
    if (a.res == nullptr) return;
    float q[8];
    load8<X32>(row_of<X32>(a.res, r, a.s.ld_x), c, a.s.H, q);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = rounded<X32>(v[j] + q[j]);
}

// longer rows: one a block, read three times (h is written last, so x or the residual may be h)
template <bool X32, bool Y32>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormFwd a) {
    __shared__ NormShared sh;
    const NormShape &s = a.s;
    TeamSum<false> row_sum(&sh, s, 0);
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
    float *dw_part, *db_part;  // [NormPlan::parts][H], or nullptr
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

// vectors a thread: two, whose sums and products take 80 registers; one for rows of a few (1000000 x 16:
// 44 us with two, 36 with one; 200000 x 100: 43 and 56)
int bwd_vecs(const mok_norm_config &c) { return c.H <= 64 ? 1 : 2; }
// rows ahead: up to three of what 192 KB a SM hold
template <int NV, bool X32, bool Y32>
constexpr int bwd_units() {
    return NV * (2 * units_of<X32>() + units_of<Y32>());
}
template <int NV, bool X32, bool Y32>
constexpr int bwd_stages() {
    return bwd_units<NV, X32, Y32>() * blocks_of_sm(NV) <= 8 ? 3 : 2;
}

// The teams of block (or cluster) b take the b-th, (b + blocks)-th, .. rows, keep their columns' sums in
// registers and add them in order at the end.
template <int NV, bool X32, bool Y32, bool CLUSTER>
__global__ void __launch_bounds__(NORM_TPB, NV == 1 ? 2 : 0) norm_backward_kernel(const NormBwd a) {
    extern __shared__ __align__(16) uint8_t norm_smem[];
    __shared__ NormShared sh;
    constexpr int UX = units_of<X32>(), UY = units_of<Y32>();
    constexpr int STAGES = bwd_stages<NV, X32, Y32>(), XS = X32 ? 4 : 2, YS = Y32 ? 4 : 2;
    const NormShape &s = a.s;
    const uint32_t rank = block_of_cluster<CLUSTER>();
    TeamSum<CLUSTER> team_sum(&sh, s, rank);
    const Ahead ahead(norm_smem, bwd_units<NV, X32, Y32>());
    let_next_start();
    wait_for_previous();
    const Place at(s, NV, rank);
    const int64_t walkers = CLUSTER ? gridDim.x / s.cluster : gridDim.x;
    const int64_t walker = CLUSTER ? blockIdx.x / s.cluster : blockIdx.x, step = walkers * at.slots;
    const int64_t first = walker * at.slots + at.slot;
    f32x2 dw[NV][4], db[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[k][j] = db[k][j] = 0;
    // the thread's vectors, and what of them is in the row
    int col[NV], left[NV];
    f32x2 w[NV][4];  // the weights stay: from memory they would be waited for in every row
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = 8 * (at.first + k * s.tpr);
        left[k] = min(max(s.H - c, 0), 8);
        col[k] = left[k] > 0 ? c : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[k][j] = pair(a.w != nullptr && c + 2 * j < s.H ? a.w[c + 2 * j] : 1.0f,
                           a.w != nullptr && c + 2 * j + 1 < s.H ? a.w[c + 2 * j + 1] : 1.0f);
    }
    // h, dy, dh of a row
    const char *ph = static_cast<const char *>(row_of<X32>(a.h, first, s.ld_x));
    const char *pd = static_cast<const char *>(row_of<X32>(a.dh, first, s.ld_x));
    const char *py = static_cast<const char *>(row_of<Y32>(a.dy, first, s.ld_y));
    const int64_t dx = step * s.ld_x * XS, dy = step * s.ld_y * YS;
    const auto fetch = [&](int stage, int64_t r) {
        const bool in = r < s.rows;
        const char *qh = in ? ph : static_cast<const char *>(a.h);
        const char *qd = in ? pd : static_cast<const char *>(a.dh);
        const char *qy = in ? py : static_cast<const char *>(a.dy);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int n = in ? left[k] : 0;
            ahead.fetch<X32>(stage, k * UX, qh + col[k] * XS, n);
            ahead.fetch<Y32>(stage, NV * UX + k * UY, qy + col[k] * YS, n);
            if (a.dh != nullptr)
                ahead.fetch<X32>(stage, NV * (UX + UY) + k * UX, qd + col[k] * XS, n);
        }
        ahead.commit();
        ph += dx;
        pd += dx;
        py += dy;
    };
#pragma unroll
    for (int k = 0; k < STAGES; ++k) fetch(k, first + k * step);
    float next_mean = s.layer && first < s.rows ? a.mean[first] : 0.0f;
    float next_rstd = first < s.rows ? a.rstd[first] : 0.0f;
    char *out_row = static_cast<char *>(row_of<X32>(a.dx, first, s.ld_x));
    const float inv_n = 1.0f / s.H;
    int stage = 0;
    for (int64_t r = first, r0 = walker * at.slots; r0 < s.rows; r0 += step, r += step, out_row += dx) {
        // with t = h - mean: n = t rstd, so sum(g n) = rstd sum(g t). Past H dy is zero, so t does not
        // matter there
        const float row_rstd = next_rstd;
        const f32x2 mean = pair(-next_mean, -next_mean), rstd = pair(row_rstd, row_rstd);
        next_mean = s.layer && r + step < s.rows ? a.mean[r + step] : 0.0f;
        next_rstd = r + step < s.rows ? a.rstd[r + step] : 0.0f;
        f32x2 t[NV][4], g[NV][4], sg2 = 0, sgt2 = 0;
        ahead.wait<STAGES - 1>();
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            Raw<X32> q;
            Raw<Y32> y;
            ahead.take<X32>(stage, k * UX, q);
            ahead.take<Y32>(stage, NV * UX + k * UY, y);
            unpack<X32>(q, t[k]);
            unpack<Y32>(y, g[k]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                t[k][j] = add2(t[k][j], mean);
                dw[k][j] = fma2(mul2(g[k][j], rstd), t[k][j], dw[k][j]);
                db[k][j] = add2(db[k][j], g[k][j]);
                g[k][j] = mul2(g[k][j], w[k][j]);
                sg2 = add2(sg2, g[k][j]);
                sgt2 = fma2(g[k][j], t[k][j], sgt2);
            }
        }
        if (a.dx != nullptr) {
            float sg = both(sg2).x + both(sg2).y, sgt = both(sgt2).x + both(sgt2).y;
            team_sum(sgt, sg);
            // dx = dh - rstd mean(g) + g rstd - t rstd^2 mean(g n)
            const float c0 = s.layer ? -row_rstd * (sg * inv_n) : 0.0f;
            // (from the inside: rstd^2 alone passes fp32 for a row of zeros and an eps below 3e-39)
            const float c1 = -row_rstd * (row_rstd * (row_rstd * (sgt * inv_n)));
            const f32x2 a0 = pair(c0, c0), a1 = pair(c1, c1);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (r >= s.rows || left[k] == 0) continue;
                f32x2 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = 0;
                if (a.dh != nullptr) {
                    Raw<X32> q;
                    ahead.take<X32>(stage, NV * (UX + UY) + k * UX, q);
                    unpack<X32>(q, v);
                }
                float o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j] = fma2(t[k][j], a1, fma2(g[k][j], rstd, add2(v[j], a0)));
                    o[2 * j] = both(v[j]).x;
                    o[2 * j + 1] = both(v[j]).y;
                }
                store_left<X32>(out_row + col[k] * XS, left[k], o);
            }
        }
        fetch(stage, r + STAGES * step);
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    ahead.wait<0>();
    float *sums = reinterpret_cast<float *>(norm_smem);
    for (int part = 0; part < 2; ++part) {
        float *out = part == 0 ? a.dw_part : a.db_part;
        if (out == nullptr) continue;
        const int width = NV * 8 * s.tpr, c0 = (int)rank * width;  // the block's columns
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int at_smem = at.slot * width + 8 * (at.first + k * s.tpr) - c0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 v = both(part == 0 ? dw[k][j >> 1] : db[k][j >> 1]);
                sums[at_smem + j] = (j & 1) ? v.y : v.x;
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < width && c0 + c < s.H; c += blockDim.x) {
            float t = 0.0f;
            for (int k = 0; k < at.slots; ++k) t += sums[k * width + c];
            out[walker * s.H + c0 + c] = t;
        }
    }
    team_sum.together();  // nobody sends to a block that has left
}

// longer rows: dx by a block a row, read twice
template <bool X32, bool Y32>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(const NormBwd a) {
    __shared__ NormShared sh;
    const NormShape &s = a.s;
    TeamSum<false> row_sum(&sh, s, 0);
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
constexpr int COLUMNS_TPB = 256;
template <bool X32, bool Y32>
__global__ void __launch_bounds__(COLUMNS_TPB) norm_columns_kernel(const NormBwd a) {
    const NormShape &s = a.s;
    let_next_start();
    wait_for_previous();
    const int c = 8 * (blockIdx.x * COLUMNS_TPB + threadIdx.x);
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
    // a batch of loads at a time, the last one too
    for (int p0 = slice; p0 < parts; p0 += 10 * NORM_SLICES) {
        float v[10], u[10];
#pragma unroll
        for (int k = 0; k < 10; ++k) {
            const int p = p0 + k * NORM_SLICES;
            const bool in = p < parts && c < H;
            v[k] = in && dw != nullptr ? dw_part[(int64_t)p * H + c] : 0.0f;
            u[k] = in && db != nullptr ? db_part[(int64_t)p * H + c] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 10; ++k) {
            s += v[k];
            t += u[k];
        }
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
NormShape norm_shape(const mok_norm_config &c, int *status) {
    return NormShape{c.rows, c.ld_x, c.ld_y, c.H, 1024, 1, c.kind == MOK_NORM_LAYER, c.eps, status};
}

// How rows are held: up to 512 threads a block, up to 8 blocks.
struct NormPlan {
    int nv, tpr, tpb, cluster;  // threads of a team and of a block, blocks of a row; tpr 0: read again
    int64_t groups;             // of rows that a block or cluster takes at a time
    int64_t parts;              // of the backward's column sums
};
NormPlan norm_plan(const mok_norm_config &c, bool backward) {
    const int vecs = (c.H + 7) / 8;
    const int nv = backward ? bwd_vecs(c) : fwd_vecs(c);
    NormPlan p = {};
    p.nv = nv;
    p.cluster = (vecs + nv * NORM_TPB - 1) / (nv * NORM_TPB);
    if (p.cluster > MOST_BLOCKS) {
        p.groups = c.rows;
        p.parts = c.rows < 32 ? c.rows : 32;
        return p;
    }
    const int threads = (vecs + p.cluster * nv - 1) / (p.cluster * nv);
    p.tpr = 1;
    while (p.tpr < threads && p.tpr < 32) p.tpr *= 2;
    if (threads > 32) p.tpr = (int)round_up(threads, 32);
    // as many teams as a block holds; with few rows fewer, on more SMs
    int teams = NORM_TPB / p.tpr;
    const int64_t blocks = GB300_SMS * blocks_of_sm(nv);
    while (teams > 1 && p.tpr * teams > 128 && c.rows < blocks * teams) teams /= 2;
    p.tpb = teams * p.tpr;
    p.groups = (c.rows + teams - 1) / teams;
    const int64_t most = blocks / p.cluster;
    p.parts = p.groups < most ? p.groups : most;
    return p;
}
size_t norm_part_bytes(const mok_norm_config &c) {
    return (size_t)round_up(norm_plan(c, true).parts * c.H * 4, 256);
}

// f by the types of x and y
#define MOK_NORM_TYPES(f, ...)                                                              \
    (c->x_dtype == MOK_DTYPE_F32                                                            \
         ? (c->y_dtype == MOK_DTYPE_F32 ? f<true, true>(__VA_ARGS__) : f<true, false>(__VA_ARGS__)) \
         : (c->y_dtype == MOK_DTYPE_F32 ? f<false, true>(__VA_ARGS__)                       \
                                        : f<false, false>(__VA_ARGS__)))

// a launch with `smem` bytes of shared memory, whose opt-in is set once per device
template <class... KA, class... A>
cudaError_t launch_norm_kernel(void (*kernel)(KA...), std::atomic<uint64_t> &attr_set, unsigned grid,
                               int tpb, int smem, int most_smem, int cluster, cudaStream_t s,
                               const A &...args) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= MAX_DEV) return cudaErrorInvalidDevice;
    const uint64_t bit = 1ull << dev;
    if ((attr_set.load(std::memory_order_acquire) & bit) == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem);
        if (e != cudaSuccess) return e;
        attr_set.fetch_or(bit, std::memory_order_acq_rel);
    }
    return launch_edge(kernel, grid, tpb, smem, cluster, s, args...);
}

template <int NV, bool X32, bool Y32>
cudaError_t launch_norm_whole(NormFwd a, const NormPlan &p, cudaStream_t s) {
    static std::atomic<uint64_t> attr_set[2];
    constexpr int per = FWD_STAGES * 2 * NV * units_of<X32>() * 16;  // a thread
    static_assert(per * NORM_TPB * blocks_of_sm(NV) <= 196608, "shared memory of a SM");
    const int64_t all = (int64_t)device_sm_count() * blocks_of_sm(NV) * (NORM_TPB / p.tpb) / p.cluster;
    const int64_t most = all > 1 ? all : 1;
    const unsigned grid = (unsigned)((p.groups < most ? p.groups : most) * p.cluster);
    const bool one = p.cluster == 1;
    return launch_norm_kernel(one ? norm_kernel<NV, X32, Y32, false> : norm_kernel<NV, X32, Y32, true>,
                              attr_set[one], grid, p.tpb, per * p.tpb, per * NORM_TPB, p.cluster, s, a);
}
template <bool X32, bool Y32>
cudaError_t launch_norm(NormFwd a, const NormPlan &p, cudaStream_t s) {
    if (p.tpr == 0)
        return launch_edge(norm_long_kernel<X32, Y32>, (unsigned)a.s.rows, 1024, 0, 1, s, a);
    a.s.tpr = p.tpr;
    a.s.cluster = p.cluster;
    if (p.nv == 1) return launch_norm_whole<1, X32, Y32>(a, p, s);
    if constexpr (!X32)
        if (p.nv == 4) return launch_norm_whole<4, X32, Y32>(a, p, s);
    return launch_norm_whole<2, X32, Y32>(a, p, s);
}

template <int NV, bool X32, bool Y32>
cudaError_t launch_norm_backward_whole(const NormBwd &a, const NormPlan &p, cudaStream_t s) {
    static std::atomic<uint64_t> attr_set[2];
    constexpr int per = bwd_stages<NV, X32, Y32>() * bwd_units<NV, X32, Y32>() * 16;  // a thread
    static_assert(per >= NV * 8 * 4, "the teams' sums of a block go where its rows were");
    static_assert(per * NORM_TPB * blocks_of_sm(NV) <= 196608, "shared memory of a SM");
    const bool one = p.cluster == 1;
    return launch_norm_kernel(
        one ? norm_backward_kernel<NV, X32, Y32, false> : norm_backward_kernel<NV, X32, Y32, true>,
        attr_set[one], (unsigned)(p.parts * p.cluster), p.tpb, per * p.tpb, per * NORM_TPB, p.cluster, s, a);
}
template <bool X32, bool Y32>
cudaError_t launch_norm_backward(NormBwd a, const NormPlan &p, cudaStream_t s) {
    const bool sums = a.dw_part != nullptr || a.db_part != nullptr;
    if (p.tpr == 0) {
        const dim3 cols((unsigned)((a.s.H + 8 * COLUMNS_TPB - 1) / (8 * COLUMNS_TPB)),
                        (unsigned)p.parts);
        cudaError_t e = cudaSuccess;
        if (sums) e = launch_edge(norm_columns_kernel<X32, Y32>, cols, COLUMNS_TPB, 0, 1, s, a);
        if (e != cudaSuccess || a.dx == nullptr) return e;
        return launch_edge(norm_backward_long_kernel<X32, Y32>, (unsigned)a.s.rows, 1024, 0, 1, s, a);
    }
    a.s.tpr = p.tpr;
    a.s.cluster = p.cluster;
    return p.nv == 1 ? launch_norm_backward_whole<1, X32, Y32>(a, p, s)
                     : launch_norm_backward_whole<2, X32, Y32>(a, p, s);
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
    if (y == h || ((y == x || y == residual) && (c->x_dtype != c->y_dtype || c->ld_x != c->ld_y)))
        return MOK_ERR_INVALID_ARG;
    const void *ps[] = {x, residual, weight, bias, h, y, mean, rstd};
    for (const void *p : ps)
        if (p && !op_aligned16(p)) return MOK_ERR_INVALID_ARG;
    const NormFwd a{norm_shape(*c, status), x, residual, weight, bias, h, y, mean, rstd};
    MOK_OP_LAUNCH(OP_NORM, 1,
                  MOK_NORM_TYPES(launch_norm, a, norm_plan(*c, false), stream));
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
    const NormPlan plan = norm_plan(*c, true);
    float *wp = dw ? (float *)ws : nullptr;
    float *bp = db ? (float *)((char *)ws + norm_part_bytes(*c)) : nullptr;
    if (c->rows > 0) {
        const NormBwd a{norm_shape(*c, status), h, dy, dh, mean, rstd, weight, dx, wp, bp};
        MOK_OP_LAUNCH(OP_NORM_BWD, 1,
                      MOK_NORM_TYPES(launch_norm_backward, a, plan, stream));
    }
    if (sums)
        MOK_OP_LAUNCH(OP_NORM_BWD, 1,
                      launch_edge(norm_join_kernel, (unsigned)((c->H + 31) / 32), 32 * NORM_SLICES, 0,
                                  1, stream, (const float *)wp, (const float *)bp, (int)plan.parts,
                                  c->H, dw, db));
    return MOK_OK;
}

}  // extern "C"

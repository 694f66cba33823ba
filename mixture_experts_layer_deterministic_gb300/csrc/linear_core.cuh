// linear_core.cuh -- products on pairs of SMs: the engine of the linear layer (linear.cu, which
// describes it) and of the vocabulary loss (vocab_loss.cu). A policy P says what a unit loads,
// multiplies and stores:
//   E              epilogue warps and threads (Epi<SUMS>)
//   F32_OUT, SUMS  outputs leave from registers in fp32; sums of segments are kept there
//   A_MN, B_MN     operands that lie along M or N in memory (else along K)
//   n_units(), unit(u), segments(unit), geom(unit, segment, rank), tx(geom), load(...), epilogue(...)
//   long_steps(unit), side_work(...)
// and, where a warp keeps more than a unit's sums from unit to unit:
//   State, start(state), finish(state, cluster, rank, ...)
#pragma once

#include <type_traits>

#include "gemm_tc_core.cuh"
#include "ops_internal.h"

namespace mok {
namespace {

constexpr int BOX = 64 * 128;      // one 64 x 64 bf16 box (8 KB)
constexpr int LSTAGES = 6;
constexpr int LSTAGE_BYTES = 4 * BOX;
constexpr uint32_t SET_COLS = 256; // TMEM columns of one accumulator set
constexpr int LTILE = 256;         // most rows of a tile
constexpr int SEG_K = 1024;        // fp32 outputs and gradients: K elements per accumulation segment

// Epilogue warps: two per TMEM lane quadrant, or four where the warps keep a unit's sums in
// registers between its segments (SUMS: 64 a thread, where two would need 128).
template <bool SUMS>
struct Epi {
    static constexpr int WARPS = SUMS ? 16 : 8;
    static constexpr int THREADS = 64 + 32 * WARPS;
    static constexpr int STEP = 32 * (WARPS / 4);   // columns between a warp's chunks of 32
    static constexpr int CHUNKS = LTILE / STEP;     // its chunks of a full tile
};
template <bool SUMS>
struct Carry {};  // what a warp keeps between the segments of a unit
template <>
struct Carry<true> {
    float v[2 * Epi<true>::CHUNKS][16];  // by 16 columns
};

// ---------------------------------------------------------------- row tiles
// A tile is up to `height` consecutive rows of one group. Dense: tile t covers rows
// [t height, ..). Grouped: a list built on the device, int32 [cap][4] = (group, first row,
// end row, 1 if the group's last), its count at list[-4].
struct Tiles {
    const int32_t *list;  // nullptr: dense
    int64_t cap;
    int64_t rows;
    int height;
    MOK_DEV int64_t count() const {
        if (list == nullptr) return (rows + height - 1) / height;
        return list[-4];
    }
    // (group, first row, end row, whether padding up to a multiple of 16 follows)
    MOK_DEV int4 get(int64_t t) const {
        if (list != nullptr) {
            const uint4 v = ld_v4(list + 4 * t);
            return make_int4((int)v.x, (int)v.y, (int)v.z, (int)v.w);
        }
        const int64_t r0 = t * height, r1 = r0 + height < rows ? r0 + height : rows;
        return make_int4(0, (int)r0, (int)r1, 0);
    }
};

// ---------------------------------------------------------------- the engine
// Outputs in bf16 leave through shared memory. A warp takes 32 columns of its 32 lanes at a
// time in the 16x256b shape, in which a thread holds two neighbouring columns of a lane;
// packed to bf16 pairs, stmatrix.trans turns them around into rows of consecutive lanes. Two
// warps of neighbouring lane quadrants share a patch of 32 rows of 64 lanes, so every row leaves
// as one 128-byte line: an SM writes lines much faster than half lines (64 bytes a row, by
// TMA or by the lanes, held dW of 64 x 1024 x 4096 at 3 TB/s, whatever the number of warps).
constexpr int PATCH_BYTES = 32 * 128;  // 32 columns of 64 lanes in bf16
constexpr int PATCHES = 2;             // per pair of warps, filled in turn

struct LinSmem {
    uint64_t full[LSTAGES];   // rank 0: both CTAs' copies of the stage have landed
    uint64_t empty[LSTAGES];  // each CTA: the MMAs that read the stage are done
    uint64_t tmem_full[2];    // each CTA: accumulator set b holds a finished unit
    uint64_t tmem_empty[2];   // rank 0: both CTAs' epilogues have drained set b
    uint32_t tmem_base;
    int abort;
};
constexpr int LIN_PATCHES = Epi<false>::WARPS / 2 * PATCHES * PATCH_BYTES;
constexpr int LIN_SMEM =
    LSTAGES * LSTAGE_BYTES + LIN_PATCHES + 1024 + (int)sizeof(LinSmem);
static_assert(LIN_SMEM <= 232448, "shared memory of a CTA");

// One unit: a tile of rows (or, for dW, the rows of a group), and which block of the output's
// contiguous dimension (mb) and of dW's features (nb).
struct Unit {
    int g, r0, nr, pad, mb, nb;
    int part;  // of K, where it is cut
};

// one unit as one CTA of the pair loads and multiplies it
struct LinGeom {
    int32_t a0, a1, a2;  // A coordinates (per policy)
    int32_t b0, b1;      // B coordinates
    int nbox;            // boxes of B per CTA: 64 columns (MN-major), 32 rows (K-major)
    int n_mma;           // N of each MMA
    int k_steps;         // 16-element K steps
    int k_first;         // K element to begin at
    int half;            // of dz, where it comes as two bf16 values

    // cut to segment `seg` of a sum that is kept in registers: `run` of its K, by one of the
    // halves of dz
    MOK_DEV void segment(int seg, int halves, int run) {
        const int first = seg / halves * (run / 16);
        half = seg % halves;
        k_first += first * 16;
        k_steps = k_steps - first < run / 16 ? k_steps - first : run / 16;
    }
    MOK_DEV int segments(int halves, int run) const {
        return k_steps > run / 16 ? (k_steps + run / 16 - 1) / (run / 16) * halves : halves;
    }
};

// Dense products with few units and a long K (dW of a narrow layer over many rows) leave most
// SMs idle: K is then cut into equal parts, one unit each, which write their fp32 sums to the
// workspace, and a join kernel adds them in order and finishes the output. Gradients of 16384
// rows, 64 x 64, 60 us without and 30 us with it, of 4096 rows, 512 x 512, 24 and 14 us; forward
// of 512 rows, 4096 -> 512, 15 and 10 us.
struct KParts {
    int parts;   // 1: K is whole and `out` not used
    int per;     // 64-element K blocks a part
    float *out;  // [parts][rows][ld]; nullptr: sums go to the output itself
    int64_t ld, stride;
    bool add;    // to what `out` (or an fp32 output) holds: a product in pieces of K, a launch each

    // number u of `units` times parts: the part, u becomes the unit's number
    MOK_DEV int take(uint32_t &u, uint32_t units) const {
        if (parts == 1) return 0;
        const uint32_t p = u / units;
        u -= p * units;
        return (int)p;
    }
    MOK_DEV void cut(LinGeom &q, int part) const {
        q.k_first = part * per * BK;
        const int left = q.k_steps - part * per * (BK / 16);
        q.k_steps = parts > 1 && left > per * (BK / 16) ? per * (BK / 16) : left;
    }
};

// values of tcgen05.ld instructions that a tmem_ld_wait before this covers: keeps their uses
// behind the wait
template <int N>
MOK_DEV void loaded(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}

MOK_DEV void tma_load_3d_pair(void *smem_dst, const CUtensorMap *m, uint32_t bar_cluster,
                              int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(tc::smem_u32(smem_dst)),
        "l"((uint64_t)m), "r"(bar_cluster), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// 32 columns of this warp's 32 lanes as pairs: v[h][b][..] are lane 16 h + t / 4 (first two)
// and 8 lanes on (last two), columns 8 b + 2 (t % 4) and the next, t the thread
MOK_DEV void ld_pairs(uint32_t c, float (&v)[2][4][4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
            "%13,%14,%15}, [%16];"
            : "=f"(v[h][0][0]), "=f"(v[h][0][1]), "=f"(v[h][0][2]), "=f"(v[h][0][3]),
              "=f"(v[h][1][0]), "=f"(v[h][1][1]), "=f"(v[h][1][2]), "=f"(v[h][1][3]),
              "=f"(v[h][2][0]), "=f"(v[h][2][1]), "=f"(v[h][2][2]), "=f"(v[h][2][3]),
              "=f"(v[h][3][0]), "=f"(v[h][3][1]), "=f"(v[h][3][2]), "=f"(v[h][3][3])
            : "r"(c + ((uint32_t)(16 * h) << 16)));
    tc::tmem_ld_wait();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < 4; ++b) loaded(v[h][b]);
}

// 32 columns, one lane per thread
MOK_DEV void ld32(uint32_t c, float (&v)[32]) {
    float a[16], b[16];
    tc::tmem_ld16(c, a);
    tc::tmem_ld16(c + 16, b);
    tc::tmem_ld_wait();
    loaded(a);
    loaded(b);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        v[j] = a[j];
        v[16 + j] = b[j];
    }
}

// 8 columns of this warp's 32 lanes: v[h][..] as v[h][b][..] of ld_pairs
MOK_DEV void ld_pairs8(uint32_t c, float (&v)[2][4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(v[h][0]), "=f"(v[h][1]), "=f"(v[h][2]), "=f"(v[h][3])
                     : "r"(c + ((uint32_t)(16 * h) << 16)));
    tc::tmem_ld_wait();
    loaded(v[0]);
    loaded(v[1]);
}

// byte of row n (a column of the accumulator), 16-byte piece i of a patch: pieces are exchanged
// by row, so that neither the matrices nor the rows collide on banks
MOK_DEV uint32_t patch_at(int n, int i) { return (uint32_t)(n * 128 + ((i ^ (n & 7)) << 4)); }

// 8 columns (rows 8 b .. of the patch) of this warp's lanes, rounded to bf16; half: which 64
// bytes of a row are the warp's
MOK_DEV void patch_write8(uint32_t patch, int half, int b, const float (&v)[2][4], int lane) {
    const uint32_t at = patch + patch_at(8 * b + (lane & 7), 4 * half + (lane >> 3));
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at),
                 "r"(pack2(v[0][0], v[0][1])), "r"(pack2(v[0][2], v[0][3])),
                 "r"(pack2(v[1][0], v[1][1])), "r"(pack2(v[1][2], v[1][3]))
                 : "memory");
}
// the reverse, added to v
MOK_DEV void patch_add8(uint32_t patch, int half, int b, float (&v)[2][4], int lane) {
    const uint32_t at = patch + patch_at(8 * b + (lane & 7), 4 * half + (lane >> 3));
    uint32_t r[4];
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i >> 1][2 * (i & 1)] += bf16_lo(r[i]);
        v[i >> 1][2 * (i & 1) + 1] += bf16_hi(r[i]);
    }
}

// `n` rows from `row` on of a part's sums, one of the columns a lane
template <int STEP>
MOK_DEV void emit_part(const KParts &kp, int part, uint32_t c, int hw, int64_t row, int n, int col,
                       int cols) {
    float *o = kp.out + part * kp.stride + row * kp.ld + col;
    for (int n0 = 32 * hw; n0 < n; n0 += STEP) {
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
            float v[16];
            tc::tmem_ld16(c + n0 + h, v);
            tc::tmem_ld_wait();
            loaded(v);
            if (col >= cols) continue;
            if (kp.add) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (n0 + h + j < n) v[j] += o[(n0 + h + j) * kp.ld];
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (n0 + h + j < n) o[(n0 + h + j) * kp.ld] = v[j];
        }
    }
}

// 16 columns at a time below column n of this warp's lanes: a unit's segments so far added up in
// registers, and after the last out(first column, sums)
template <class F>
MOK_DEV void sum_segments(uint32_t c, int hw, int n, bool first, bool last, Carry<true> &s, F &&out) {
#pragma unroll
    for (int k = 0; k < 2 * Epi<true>::CHUNKS; ++k) {
        const int n0 = 32 * hw + Epi<true>::STEP * (k >> 1) + 16 * (k & 1);
        if (n0 >= n) continue;
        float v[16];
        tc::tmem_ld16(c + n0, v);
        tc::tmem_ld_wait();
        loaded(v);
#pragma unroll
        for (int j = 0; j < 16; ++j) s.v[k][j] = first ? v[j] : s.v[k][j] + v[j];
        if (last) out(n0, s.v[k]);
    }
}

// a bf16 output: matrices of `rows` x `cols`, rows ld apart
struct OutRef {
    uint16_t *p;
    int64_t rows, ld;
    int cols;
};

// An epilogue warp's place: its half of the shared patches, its pair's barrier, the patch to
// fill next. A patch is refilled two turns later; the barrier of the turn between says that the
// other warp has read it.
struct Patches {
    uint32_t base;
    int bar, half, lane;
    int turn;

    // both warps' flags and-ed: they go on, or give up, together (neither may leave the other
    // at a barrier)
    MOK_DEV bool agree(bool ok) const {
        uint32_t r;
        asm volatile(
            "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.and.pred q, %2, 64, p;\n"
            "selp.u32 %0, 1, 0, q;\n}\n"
            : "=r"(r)
            : "r"(ok ? 1u : 0u), "r"(bar)
            : "memory");
        return r != 0;
    }
    MOK_DEV uint32_t patch() const { return base + (uint32_t)turn * PATCH_BYTES; }
    // both halves of the current patch are filled: rows [y0, y0 + 32) and below `end` of matrix
    // g of o get columns x .. x + 63 (x of the pair), this warp storing 16 of the rows, eight
    // lanes a row; element by element where the matrix's edge cuts 16 bytes
    MOK_DEV void store(const OutRef &o, int x, int64_t y0, int64_t end, int g) {
        asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");
        const uint32_t p0 = patch();
        turn ^= 1;
        const int col = x + 8 * (lane & 7), n0 = 16 * half + (lane >> 3);
        uint16_t *p = o.p + ((int64_t)g * o.rows + y0 + n0) * o.ld + col;
        uint32_t w[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                         : "r"(p0 + patch_at(n0 + 4 * i, lane & 7))
                         : "memory");
        const int64_t step = 4 * o.ld;
        if (y0 + 32 <= end && x + 64 <= o.cols) {
#pragma unroll
            for (int i = 0; i < 4; ++i, p += step)
                *reinterpret_cast<uint4 *>(p) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i, p += step) {
            if (y0 + n0 + 4 * i >= end) continue;
            if (col + 8 <= o.cols) {
                *reinterpret_cast<uint4 *>(p) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j < o.cols) p[j] = (uint16_t)(w[i][j >> 1] >> (16 * (j & 1)));
            }
        }
    }
};

// A chunk of an output with no arithmetic: 32 columns of the accumulator, rows from nr on (and
// everything, with nr <= 0) as zeros
MOK_DEV void emit_plain(Patches &pt, uint32_t c, int nr, const OutRef &o, int x, int64_t y0,
                        int64_t end, int g) {
    float v[2][4][4];
    ld_pairs(c, v);
    if (nr < 32) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (8 * k + 2 * (pt.lane & 3) + (i & 1) >= nr) v[0][k][i] = v[1][k][i] = 0.f;
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const float w[2][4] = {{v[0][b][0], v[0][b][1], v[0][b][2], v[0][b][3]},
                               {v[1][b][0], v[1][b][1], v[1][b][2], v[1][b][3]}};
        patch_write8(pt.patch(), pt.half, b, w, pt.lane);
    }
    pt.store(o, x, y0, end, g);
}

// Arrive on a barrier of either CTA of the pair. CTA scope: what the barrier hands over lives in
// TMEM, ordered by the tcgen05 fences. Cluster scope made the arriving thread wait for its
// global stores to land, about 2 us a unit (dW of 64 x 1024 x 4096: 208 against 164 us).
MOK_DEV void lin_arrive(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster)
                 : "memory");
}
// A bounded wait that takes the time only after many polls: the clock read costs more than
// most waits here are long. steps(): K steps that may run during it, a microsecond each on top of
// the limit (a step takes about 0.05 us; dW of a group of 2^30 rows is one sum of some seconds).
template <class F>
MOK_DEV bool lin_wait(uint64_t *bar, uint32_t parity, int *status, volatile int *abort, F &&steps) {
    uint64_t t0 = 0;
    for (uint32_t n = 1; !tc::mbar_try_wait(bar, parity); ++n) {
        if ((n & 255u) != 0) continue;
        if (*abort) return false;
        const uint64_t t = tc::globaltimer();
        if (t0 == 0) t0 = t;
        if (t - t0 > tc::WAIT_LIMIT_NS && t - t0 > tc::WAIT_LIMIT_NS + 1000ull * (uint32_t)steps()) {
            raise_status(status, MOK_ERR_TIMEOUT);
            *abort = 1;
            return false;
        }
    }
    return true;
}
MOK_DEV bool lin_wait(uint64_t *bar, uint32_t parity, int *status, volatile int *abort) {
    return lin_wait(bar, parity, status, abort, [] { return 0; });
}
// bounded drain of a barrier phase on the way out
MOK_DEV void lin_drain(uint64_t *bar, uint32_t parity) {
    const uint64_t t0 = tc::globaltimer();
    while (!tc::mbar_try_wait(bar, parity) && tc::globaltimer() - t0 < 100000000ull) {
    }
}

// what an epilogue warp of P keeps
template <class P, class = void>
struct StateOf {
    using Type = Carry<P::SUMS>;
    static constexpr bool LASTS = false;
};
template <class P>
struct StateOf<P, std::void_t<typename P::State>> {
    using Type = typename P::State;
    static constexpr bool LASTS = true;
};

// the kernel's work on the units cid, cid + ncl, ... of p, as one CTA of a pair
template <class P>
MOK_DEV void linear_body(const CUtensorMap &tmA, const CUtensorMap &tmB, const P &p,
                         const uint32_t cid, const uint32_t ncl) {
    constexpr int NS = LSTAGES, SB = LSTAGE_BYTES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    LinSmem *sm = (LinSmem *)(base + NS * SB + LIN_PATCHES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            tc::mbar_init(&sm->full[s], 1);
            tc::mbar_init(&sm->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&sm->tmem_full[b], 1);
            tc::mbar_init(&sm->tmem_empty[b], 2 * P::E::WARPS);
        }
        sm->abort = 0;
        tc::fence_mbar_init();
        tc::prefetch_tmap(&tmA);
        tc::prefetch_tmap(&tmB);
    }
    if (warp == 1) {
        tc::tmem_alloc_pair(&sm->tmem_base, TMEM_COLS);
        tc::tmem_relinquish_pair();
    }
    // both CTAs' barriers exist and TMEM is allocated before either CTA touches the other
    tc::tc_fence_before();
    tc::cluster_sync();
    tc::tc_fence_after();
    const uint32_t tmem = sm->tmem_base;
    volatile int *abort = &sm->abort;
    let_next_start();
    wait_for_previous();
    const uint32_t n_units = (uint32_t)p.n_units();

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (tc::elect_one()) {
            const uint32_t full0 = tc::cluster_addr(&sm->full[0], 0);  // rank 0's full[0]
            int s = 0;
            uint32_t ph = 0;
            int64_t issued = 0;
            bool ok = true;
            for (uint32_t u = cid; u < n_units && ok; u += ncl) {
                const Unit cur = p.unit(u);
                const int segs = p.segments(cur);
                for (int seg = 0; seg < segs && ok; ++seg) {
                    const LinGeom g = p.geom(cur, seg, rank);
                    const uint32_t tx = p.tx(g);
                    const int kblocks = (g.k_steps + 3) / 4;
                    for (int kb = 0; kb < kblocks; ++kb) {
                        if (!lin_wait(&sm->empty[s], ph ^ 1u, p.status, abort)) {
                            ok = false;
                            break;
                        }
                        if (rank == 0) tc::mbar_arrive_expect_tx(&sm->full[s], 2 * tx);
                        p.load(base + s * SB, full0 + (uint32_t)s * 8u, g, g.k_first + kb * BK, &tmA,
                               &tmB);
                        ++issued;
                        if (++s == NS) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                }
            }
            // do not leave while copies may still be landing: the MMAs that read the last
            // stages have finished (bounded)
            for (int q = 0; q < NS && q < issued; ++q) {
                if (--s < 0) {
                    s = NS - 1;
                    ph ^= 1u;
                }
                lin_drain(&sm->empty[s], ph);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (rank 0)
        if (rank == 1) p.side_work(cid, ncl, lane);
        if (rank == 0 && tc::elect_one()) {
            // Descriptors of stage 0; a stage, and a K step of 16 elements, move only the address
            // (in 16-byte units). MN-major: 16 K rows are two groups of eight 128-byte rows,
            // blocks of 64 M or N elements BOX apart; K-major: 32 bytes along the row. The
            // issuing thread's own instructions count here: with the descriptors built per
            // step a K block took no less time at N = 160 than at 256.
            constexpr uint32_t A_STEP = (P::A_MN ? 2048 : 32) >> 4;
            constexpr uint32_t B_STEP = (P::B_MN ? 2048 : 32) >> 4;
            const uint32_t s0 = tc::smem_u32(base);
            const uint64_t da0 = tc::sdesc_sw128(s0, P::A_MN ? BOX : 16, 1024);
            const uint64_t db0 = tc::sdesc_sw128(s0 + 2 * BOX, P::B_MN ? BOX : 16, 1024);
            int s = 0;
            uint32_t ph = 0;
            int64_t a = 0;  // accumulations so far: number a uses set a % 2
            bool ok = true;
            for (uint32_t u = cid; u < n_units && ok; u += ncl) {
                const Unit cur = p.unit(u);
                const int segs = p.segments(cur);
                for (int seg = 0; seg < segs && ok; ++seg) {
                    const LinGeom g = p.geom(cur, seg, 0);
                    const uint32_t idesc = tc::idesc_bf16(256, g.n_mma, P::A_MN, P::B_MN);
                    const int ab = (int)(a & 1);
                    const uint32_t use = (uint32_t)((a >> 1) & 1);
                    if (!lin_wait(&sm->tmem_empty[ab], use ^ 1u, p.status, abort)) {
                        ok = false;
                        break;
                    }
                    tc::tc_fence_after();
                    const uint32_t d = tmem + (uint32_t)ab * SET_COLS;
                    const int kblocks = (g.k_steps + 3) / 4;
                    for (int kb = 0; kb < kblocks; ++kb) {
                        if (!lin_wait(&sm->full[s], ph, p.status, abort)) {
                            ok = false;
                            break;
                        }
                        tc::tc_fence_after();
                        const uint64_t da = da0 + (uint64_t)(s * (SB >> 4));
                        const uint64_t db = db0 + (uint64_t)(s * (SB >> 4));
                        if (g.k_steps - kb * 4 >= 4) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                tc::mma_f16_pair(d, da + kk * A_STEP, db + kk * B_STEP, idesc,
                                                 kk > 0 ? 1u : (kb > 0 ? 1u : 0u));
                        } else {
                            for (int kk = 0; kk < g.k_steps - kb * 4; ++kk)
                                tc::mma_f16_pair(d, da + kk * A_STEP, db + kk * B_STEP, idesc,
                                                 kb > 0 || kk > 0 ? 1u : 0u);
                        }
                        tc::mma_commit_pair(&sm->empty[s], 3);  // frees the stage in both CTAs
                        if (++s == NS) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                    if (!ok) break;
                    tc::mma_commit_pair(&sm->tmem_full[ab], 3);
                    ++a;
                }
            }
            // do not free TMEM under MMAs still in flight (bounded)
            if (a > 0) {
                const int lb = (int)((a - 1) & 1);
                lin_drain(&sm->tmem_full[lb], (uint32_t)(((a - 1) >> 1) & 1));
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;          // TMEM lane quadrant this warp may access
        const int hw = (warp - 2) >> 2;  // which of the quadrant's warps: it takes every so-manyth chunk
        const uint32_t lane_base = (uint32_t)(q * 32) << 16;
        const uint32_t empty0 = tc::cluster_addr(&sm->tmem_empty[0], 0);
        const int pair = 2 * hw + (q >> 1);
        Patches pt{tc::smem_u32(base + NS * SB) + (uint32_t)(pair * PATCHES * PATCH_BYTES),
                   1 + pair, q & 1, lane, 0};
        typename StateOf<P>::Type carry;
        if constexpr (StateOf<P>::LASTS) p.start(carry);
        int64_t a = 0;
        bool ok = true;
        for (uint32_t u = cid; u < n_units && ok; u += ncl) {
            const Unit cur = p.unit(u);
            const int segs = p.segments(cur);
            for (int seg = 0; seg < segs; ++seg, ++a) {
                const int ab = (int)(a & 1);
                ok = lin_wait(&sm->tmem_full[ab], (uint32_t)((a >> 1) & 1), p.status, abort,
                              [&] { return p.long_steps(cur); });
                if constexpr (!P::F32_OUT) ok = pt.agree(ok);
                if (!ok) break;
                tc::tc_fence_after();
                p.epilogue(cur, seg, seg == segs - 1, rank, tmem + lane_base + (uint32_t)ab * SET_COLS,
                           q, hw, lane, pt, carry);
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) lin_arrive(empty0 + (uint32_t)ab * 8u);
            }
        }
        if constexpr (StateOf<P>::LASTS)
            if (ok) p.finish(carry, cid, rank, q, hw, lane);
    }

    // no MMA, copy or arrival of either CTA targets the other past this point
    tc::tc_fence_before();
    tc::cluster_sync();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc_pair(tmem, TMEM_COLS);
    }
}

template <class P>
__global__ void __launch_bounds__(P::E::THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tmA,
                  const __grid_constant__ CUtensorMap tmB, const P p) {
    linear_body(tmA, tmB, p, tc::cluster_id_x(), tc::cluster_count_x());
}

// two products at once: the first `split` pairs take the units of p, the others those of q
template <class P, class Q>
__global__ void __launch_bounds__(P::E::THREADS, 1)
    linear_both_kernel(const __grid_constant__ CUtensorMap pA,
                       const __grid_constant__ CUtensorMap pB, const P p,
                       const __grid_constant__ CUtensorMap qA,
                       const __grid_constant__ CUtensorMap qB, const Q q, const uint32_t split) {
    static_assert(P::E::THREADS == Q::E::THREADS, "one launch shape");
    const uint32_t c = tc::cluster_id_x();
    if (c < split)
        linear_body(pA, pB, p, c, split);
    else
        linear_body(qA, qB, q, c - split, tc::cluster_count_x() - split);
}

// ---------------------------------------------------------------- host side
// bf16 matrix of `rows` rows of `cols` elements, `ld` apart; boxes of 64 columns x box_rows
cudaError_t map2d(CUtensorMap *m, const void *p, int64_t rows, int64_t cols, int64_t ld,
                  int box_rows) {
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    cuuint32_t box[2] = {(cuuint32_t)BK, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides,
                  box, es) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}
// W [G][N][Kin]: (inputs, features, groups), boxes of 64 inputs x box_rows features; or the planes
// of dz
cudaError_t map_w(CUtensorMap *m, const void *p, int64_t G, int64_t N, int64_t Kin, int64_t ld,
                  int box_rows) {
    cuuint64_t dims[3] = {(cuuint64_t)Kin, (cuuint64_t)N, (cuuint64_t)G};
    cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)((G > 1 ? N : 1) * ld * 2)};
    cuuint32_t box[3] = {(cuuint32_t)BK, (cuuint32_t)box_rows, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides,
                  box, es) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

int64_t sm_pairs() { return device_sm_count() / 2 > 0 ? device_sm_count() / 2 : 1; }

// a launch of `pairs` clusters of two CTAs; the shared-memory opt-in is set once per device
template <class... KA, class... A>
cudaError_t launch_pairs(void (*kernel)(KA...), std::atomic<uint64_t> &attr_set, int threads,
                         int64_t pairs, cudaStream_t s, const A &...args) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= MAX_DEV) return cudaErrorInvalidDevice;
    const uint64_t bit = 1ull << dev;
    if ((attr_set.load(std::memory_order_acquire) & bit) == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, LIN_SMEM);
        if (e != cudaSuccess) return e;
        attr_set.fetch_or(bit, std::memory_order_acq_rel);
    }
    return launch_edge(kernel, dim3((unsigned)(2 * pairs)), threads, LIN_SMEM, 2, s, args...);
}

// one cluster per unit, at most `most` (the pairs of SMs that run at once)
template <class P>
cudaError_t launch_linear(const CUtensorMap &ma, const CUtensorMap &mb, const P &p,
                          int64_t units_cap, cudaStream_t s, int64_t most = sm_pairs()) {
    if (units_cap < 1) return cudaSuccess;
    if (units_cap > 0x7FFFFFFF) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> attr_set{0};
    return launch_pairs(linear_kernel<P>, attr_set, P::E::THREADS,
                        units_cap < most ? units_cap : most, s, ma, mb, p);
}
template <class P, class Q>
cudaError_t launch_both(const CUtensorMap &pa, const CUtensorMap &pb, const P &p,
                        const CUtensorMap &qa, const CUtensorMap &qb, const Q &q, int64_t split,
                        int64_t pairs, cudaStream_t s) {
    static std::atomic<uint64_t> attr_set{0};
    return launch_pairs(linear_both_kernel<P, Q>, attr_set, P::E::THREADS, pairs, s, pa, pb, p, qa,
                        qb, q, (uint32_t)split);
}

// Plans that a result's rounding depends on count the GB300's pairs of SMs, not the device's.
constexpr int64_t PLAN_PAIRS = GB300_SMS / 2;

// clocks of a 64-element K block on tiles of h rows: the larger of the MMAs' (2 a row) and the
// loads' (64 bytes a clock and SM: 256 for the weights, 64 for each box of 32 rows)
int64_t block_clocks(int64_t h) {
    const int64_t mma = 2 * h, load = 256 + 64 * ((h / 2 + 31) / 32);
    return mma > load ? mma : load;
}
// clocks of a unit of `blocks` K blocks on h columns: its loads and MMAs, or its epilogue (about
// 4500 clocks for 256 columns), whichever keeps the pair longer
int64_t unit_clocks(int64_t blocks, int64_t h) {
    const int64_t main = blocks * block_clocks(h), epi = 4500 * h / LTILE;
    return main > epi ? main : epi;
}
// Dense tiles of equal height: the height, up to 256 rows, at which `n_mb` blocks a tile take the
// least time, as waves over the SM pairs times a K block's clocks (*clocks).
int dense_height(int64_t rows, int64_t n_mb, int64_t pairs, int64_t *clocks) {
    int64_t best_h = LTILE, best = INT64_MAX;
    for (int64_t h0 = LTILE; h0 >= 16; h0 -= 16) {
        const int64_t n = (rows + h0 - 1) / h0;
        const int64_t h = n > 0 ? round_up((rows + n - 1) / n, 16) : 16;
        const int64_t t = (n * n_mb + pairs - 1) / pairs * block_clocks(h);
        if (t < best) {
            best = t;
            best_h = h;
        }
    }
    *clocks = best;
    return (int)best_h;
}
Tiles dense_tiles(int64_t rows, int height) {
    return Tiles{nullptr, (rows + height - 1) / height, rows, height};
}

}  // namespace
}  // namespace mok

// linear.cu -- a linear layer for one matrix or one per group of rows: products with bias,
// activation and residual in the epilogue, and their gradients.
//
//   forward   z = x W^T + b, y = act(z) + residual
//   backward  dz = dy act'(z), dx = dz W, dW = dz^T x, db = sum of dz over the rows
//
// The three products run on pairs of SMs (tcgen05 cta_group::2, M = 256): the dimension that is
// contiguous in the output (features of y, inputs of dx and dW) lies on M, so a warp's 32 TMEM
// lanes store consecutive elements, and the rows of x (or the features of dW) lie on N, so a
// ragged group costs at most 15 padding rows.
//   Fwd  A = W    (K-major),  B = x   (K-major)   -> y (and z)   [features x rows]
//   Dx   A = W    (MN-major), B = dz  (K-major)   -> dx          [inputs x rows]
//   Dw   A = x    (MN-major), B = dz  (MN-major)  -> dW          [inputs x features]
// W is a 3D tensor map (inputs, features, groups), so a tile past a matrix's edge reads zeros,
// not the next group's matrix. Every output element is one fp32 sum in an order that depends on the
// call's sizes alone.
//
// A few rows go to kernels of their own, few tiles over a long K to parts of K that a join adds.
//
// Per CTA, 320 threads: warp 0 loads (TMA, both CTAs), warp 1 issues the MMAs (rank 0), warps
// 2-9 drain accumulators (16 warps where sums stay in registers), two sets of 256 TMEM columns
// alternating between units. Every wait is bounded (2 s), after which MOK_ERR_TIMEOUT is
// recorded and the launch ends.
#include <type_traits>

#include "gemm_tc_core.cuh"
#include "ops_internal.h"

namespace mok {
namespace {

// two fp32 values to bf16 in one conversion, lo in the low half (two single conversions run on
// the slow pipe and held the epilogue: dW of 64 x 1024 x 4096 164 against 139 us)
MOK_DEV uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

constexpr int BOX = 64 * 128;      // one 64 x 64 bf16 box (8 KB)
constexpr int LSTAGES = 6;
constexpr int LSTAGE_BYTES = 4 * BOX;
constexpr uint32_t SET_COLS = 256; // TMEM columns of one accumulator set
constexpr int LTILE = 256;         // most rows of a tile
constexpr int SEG_K = 1024;        // fp32 outputs and gradients: K elements per accumulation segment
constexpr int MAX_G = 1024;

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

// Each group's rows in tiles of equal height (a multiple of 16, at most `most`); valid[g] gets
// the group's row count, 0 where its layout breaks the rules; first[g] its first tile (first[G]:
// their number). One block, two scans over the groups: about 2 us, most of them under the kernel
// before and after. Groups that count lie apart inside `rows`, so their tiles number at most
// tiles_cap and fit 31 bits.
__global__ void __launch_bounds__(MAX_G)
    linear_tiles_kernel(const int32_t *starts, const int32_t *counts, int G, int64_t rows,
                        int most, int32_t *list, int32_t *valid, int32_t *first, int *status) {
    __shared__ int32_t wsum[32], wend[32];
    static_assert(MAX_G == 32 * 32, "a warp total a lane");
    let_next_start();
    wait_for_previous();
    const int g = threadIdx.x, lane = g & 31, warp = g >> 5;
    int64_t b = 0, n = 0, h = most;
    int32_t nt = 0, end = 0;  // end: of the group's rows and their padding
    bool ok = g < G;
    if (ok) {
        b = starts[g];
        n = counts[g];
        const int64_t e = starts[g + 1];
        // the padding after the rows is written too, so it has to lie inside the group
        ok = n >= 0 && b >= 0 && (b & 15) == 0 && b + ((n + 15) & ~(int64_t)15) <= e && e <= rows;
        if (ok) end = (int32_t)(b + ((n + 15) & ~(int64_t)15));
    }
    // the largest end of the groups before this one: a group that begins below it would write
    // rows that are another's already
    int32_t before = end;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o && u > before) before = u;
    }
    if (lane == 31) wend[warp] = before;
    before = __shfl_up_sync(0xFFFFFFFFu, before, 1);
    if (lane == 0) before = 0;
    __syncthreads();
    // the earlier warps', one a lane
    before = max(before, __reduce_max_sync(0xFFFFFFFFu, lane < warp ? wend[lane] : 0));
    if (g < G) {
        if (!ok || b < before) {
            raise_status(status, MOK_ERR_DEVICE_INVARIANT);
            n = 0;
        }
        valid[g] = (int32_t)n;
        if (n > 0) {
            const int64_t n0 = (n + most - 1) / most;
            h = ((n + n0 - 1) / n0 + 15) & ~(int64_t)15;
            nt = (int32_t)((n + h - 1) / h);
        }
    }
    int32_t v = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) wsum[warp] = v;
    __syncthreads();
    const int32_t at = v - nt + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? wsum[lane] : 0);
    if (g < G) first[g] = at;
    if (g == MAX_G - 1) list[-4] = first[G] = at + nt;
    for (int32_t i = 0; i < nt; ++i) {
        const int64_t r0 = b + i * h, r1 = r0 + h < b + n ? r0 + h : b + n;
        reinterpret_cast<int4 *>(list)[at + i] =
            make_int4(g, (int32_t)r0, (int32_t)r1, i == nt - 1 ? 1 : 0);
    }
}

int64_t tiles_cap(int64_t rows, int G, int most) { return G + rows / most + 1; }

// ---------------------------------------------------------------- activations
// 2^x and the quotient are the hardware's, within 2^-22 of their values; the exponent itself is
// rounded to fp32, which costs half an ulp of it, so the activations and their slopes are within
// 2^-20 (1 + |z|): far inside the bf16 rounding of y and z, and of the size of the products' own
// error in fp32
MOK_DEV float sigmoid2_f(float x) {  // sigma(-x log 2) = 1 / (1 + 2^x)
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}
constexpr float LOG2E = 1.4426950408889634f;
MOK_DEV float sigmoid_f(float x) { return sigmoid2_f(-LOG2E * x); }

constexpr float GELU_C2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float GELU_A = 0.044715f;

// sigma(2 sqrt(2/pi) (z + a z^3)), z2 = z z
MOK_DEV float gelu_sigmoid(float z, float z2) {
    return sigmoid2_f(z * fmaf(-LOG2E * GELU_C2 * GELU_A, z2, -LOG2E * GELU_C2));
}
// 0.5 (1 + tanh u) = sigma(2u): gelu_tanh is z sigma(2 sqrt(2/pi) (z + a z^3))
template <int ACT>
MOK_DEV float act_f(float z) {
    if (ACT == MOK_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
    if (ACT == MOK_ACT_SILU) return z * sigmoid_f(z);
    if (ACT == MOK_ACT_GELU_TANH) return z * gelu_sigmoid(z, z * z);
    if (ACT == MOK_ACT_GELU) return 0.5f * z * erfcf(-0.70710678118654752f * z);
    return z;
}
// the nearest value of [-16, 16]; NaN stays NaN
MOK_DEV float within16(float z) {
    float r;
    asm("{\n.reg .f32 t;\nmin.NaN.f32 t, %1, %2;\nmax.NaN.f32 %0, t, %3;\n}\n"
        : "=f"(r)
        : "f"(z), "f"(16.0f), "f"(-16.0f));
    return r;
}
template <int ACT>
MOK_DEV float act_grad_f(float z) {
    if (ACT == MOK_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if (ACT == MOK_ACT_SILU) {
        const float s = sigmoid_f(z);
        return s * fmaf(z, 1.0f - s, 1.0f);
    }
    if (ACT == MOK_ACT_GELU_TANH) {
        const float c = within16(z);  // s is 0 or 1 past it, and z^3 must not meet that 0
        const float z2 = c * c, s = gelu_sigmoid(c, z2);
        const float du = fmaf(3.0f * GELU_A * GELU_C2, z2, GELU_C2);
        return s * fmaf(c * (1.0f - s), du, 1.0f);
    }
    if (ACT == MOK_ACT_GELU)
        return fmaf(z, 0.3989422804014327f * __expf(-0.5f * z * z),
                    0.5f * erfcf(-0.70710678118654752f * z));
    return 1.f;
}
// the runtime activation as a template argument: f(std::integral_constant<int, ACT>)
template <class F>
MOK_DEV void with_act(int act, F &&f) {
    switch (act) {
        case MOK_ACT_RELU: f(std::integral_constant<int, MOK_ACT_RELU>{}); break;
        case MOK_ACT_SILU: f(std::integral_constant<int, MOK_ACT_SILU>{}); break;
        case MOK_ACT_GELU_TANH: f(std::integral_constant<int, MOK_ACT_GELU_TANH>{}); break;
        case MOK_ACT_GELU: f(std::integral_constant<int, MOK_ACT_GELU>{}); break;
        default: f(std::integral_constant<int, MOK_ACT_NONE>{}); break;
    }
}

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

    // cut to segment `seg` of a sum that is kept in registers: SEG_K of its K, by one of the
    // halves of dz
    MOK_DEV void segment(int seg, int halves) {
        const int first = seg / halves * (SEG_K / 16);
        half = seg % halves;
        k_first += first * 16;
        k_steps = k_steps - first < SEG_K / 16 ? k_steps - first : SEG_K / 16;
    }
    MOK_DEV int segments(int halves) const {
        return k_steps > SEG_K / 16 ? (k_steps + SEG_K / 16 - 1) / (SEG_K / 16) * halves : halves;
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
    float *out;  // [parts][rows][ld]
    int64_t ld, stride;

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

// The product. 8192 x 4096 x 4096 137 to 157 us by the card's power state, within 1% of the
// library's plain product on the same card; 64 groups of 320 rows, 4096 -> 1024 with GELU and z
// 138 us, 147 to 151 where the arrays change from call to call (5.3 TB/s and 1160 TFLOP/s: 6.7
// waves of tiles of 160 rows, whose operands come slower than their MMAs run).
// PLAIN: only a bias after the product (no activation, residual or z); CUT: K is cut into parts
// (a variant of its own: the code for parts cost the router's product 1.3 of 52 us)
template <bool F32, bool PLAIN, bool CUT = false>
struct Fwd {
    using E = Epi<F32 && PLAIN>;
    static constexpr bool F32_OUT = F32 || CUT, SUMS = F32 && PLAIN;
    static constexpr bool A_MN = false, B_MN = false;
    Tiles tiles;
    int n_mb;      // ceil(N / 256)
    int segs;      // accumulation segments per unit (fp32 outputs), else 1
    int Kin, N;
    int64_t ld;    // row stride of y, z and residual
    const float *bias;
    const uint16_t *res;
    void *y;
    uint16_t *z;
    int act;
    int *status;
    KParts kp;

    MOK_DEV int64_t n_units() const { return tiles.count() * n_mb * (CUT ? kp.parts : 1); }
    MOK_DEV void side_work(uint32_t, uint32_t, int) const {}
    MOK_DEV Unit unit(uint32_t u) const {
        const int part = CUT ? kp.take(u, (uint32_t)(tiles.cap * n_mb)) : 0;
        const int4 t = tiles.get(u / (uint32_t)n_mb);
        return Unit{t.x, t.y, t.z - t.y, t.w, (int)(u % (uint32_t)n_mb), 0, part};
    }
    MOK_DEV int segments(const Unit &) const { return segs; }
    MOK_DEV int long_steps(const Unit &) const { return 0; }  // K is at most 2^20
    MOK_DEV LinGeom geom(const Unit &u, int seg, uint32_t rank) const {
        LinGeom q;
        q.n_mma = (u.nr + 15) & ~15;
        q.a0 = seg * SEG_K;
        q.a1 = u.mb * 256 + (int)rank * 128;
        q.a2 = u.g;
        q.b0 = q.a0;
        q.b1 = u.r0 + (int)rank * (q.n_mma / 2);
        q.nbox = (q.n_mma / 2 + 31) / 32;
        const int k = segs > 1 && Kin - q.a0 > SEG_K ? SEG_K : Kin - q.a0;
        q.k_steps = (k + 15) / 16;
        q.k_first = 0;
        if constexpr (CUT) kp.cut(q, u.part);
        return q;
    }
    MOK_DEV uint32_t tx(const LinGeom &q) const { return 2 * BOX + q.nbox * (BOX / 2); }
    // A: 128 features x 64 inputs; B: the rows' 64 inputs in boxes of 32 rows
    MOK_DEV void load(uint8_t *st, uint32_t fb, const LinGeom &q, int k0, const CUtensorMap *tmA,
                      const CUtensorMap *tmB) const {
        tma_load_3d_pair(st, tmA, fb, q.a0 + k0, q.a1, q.a2);
        for (int j = 0; j < q.nbox; ++j)
            tc::tma_load_2d_pair(st + 2 * BOX + j * (BOX / 2), tmB, fb, q.b0 + k0, q.b1 + 32 * j);
    }
    MOK_DEV void epilogue(const Unit &u, int seg, bool, uint32_t rank, uint32_t c, int q, int hw,
                          int lane, Patches &pt, Carry<SUMS> &carry) const {
        const int nr = u.nr, pad = u.pad;
        const int64_t r0 = u.r0;
        const int n_mma = (nr + 15) & ~15;
        const int f0 = u.mb * 256 + (int)rank * 128 + q * 32;  // the warp's features
        const int n_out = pad ? n_mma : nr;
        if constexpr (CUT)
            emit_part<E::STEP>(kp, u.part, c, hw, r0, nr, f0 + lane, N);
        else if constexpr (SUMS)
            direct_sums(seg, c, hw, f0 + lane, u.g, r0, nr, n_out, carry.v);
        else if constexpr (F32)
            direct(seg, c, hw, f0 + lane, u.g, r0, nr, n_out);
        else
            staged(c, hw, f0, u.g, r0, nr, n_out, pt);
    }
    // bf16: 32 rows at a time through patches, 8 rows in registers at once
    MOK_DEV void staged(uint32_t c, int hw, int f0, int g, int64_t r0, int nr, int n_out,
                        Patches &pt) const {
        const int lane = pt.lane;
        float bs[2][2];  // this thread's four features
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int f = f0 + 8 * i + (lane >> 2);
            bs[i >> 1][i & 1] = bias != nullptr && f < N ? bias[(int64_t)g * N + f] : 0.f;
        }
        const int x = f0 & ~63;
        const auto z_of = [&](int n, float (&v)[2][4]) {  // rows n.. ; the padding's z is zero
            ld_pairs8(c + n, v);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[h][i] = n + 2 * (lane & 3) + (i & 1) < nr ? v[h][i] + bs[h][i >> 1] : 0.f;
        };
        for (int n0 = 32 * hw; n0 < n_out; n0 += E::STEP) {
            uint4 t[4];
            if (res != nullptr) {  // rows of 64 bytes, four lanes each
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = 8 * i + (lane >> 2), f = f0 + 8 * (lane & 3);
                    t[i] = make_uint4(0, 0, 0, 0);
                    if (n0 + n < nr && f < N) {
                        const uint16_t *p = res + (r0 + n0 + n) * ld + f;
                        if (f + 8 <= N) {
                            t[i] = *reinterpret_cast<const uint4 *>(p);
                        } else {
                            uint32_t e[4] = {0, 0, 0, 0};
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (f + j < N) e[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
                            t[i] = make_uint4(e[0], e[1], e[2], e[3]);
                        }
                    }
                }
            }
            if (z != nullptr) {
#pragma unroll 2
                for (int b = 0; b < 4; ++b) {
                    float v[2][4];
                    z_of(n0 + 8 * b, v);
                    patch_write8(pt.patch(), pt.half, b, v, lane);
                }
                pt.store(OutRef{z, tiles.rows, ld, N}, x, r0 + n0, r0 + n_out, 0);
            }
            if (res != nullptr) {  // through the patch that y will fill, into the pairs' order
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                                     pt.patch() +
                                     patch_at(8 * i + (lane >> 2), 4 * pt.half + (lane & 3))),
                                 "r"(t[i].x), "r"(t[i].y), "r"(t[i].z), "r"(t[i].w)
                                 : "memory");
                __syncwarp();
            }
            with_act(act, [&](auto a) {
#pragma unroll 2
                for (int b = 0; b < 4; ++b) {
                    float v[2][4];
                    z_of(n0 + 8 * b, v);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[h][i] = act_f<a.value>(v[h][i]);
                    // act(0) and the residual's padding are zero
                    if (res != nullptr) {
                        patch_add8(pt.patch(), pt.half, b, v, lane);
                        __syncwarp();
                    }
                    patch_write8(pt.patch(), pt.half, b, v, lane);
                }
            });
            pt.store(OutRef{static_cast<uint16_t *>(y), tiles.rows, ld, N}, x, r0 + n0, r0 + n_out,
                     0);
        }
    }
    // fp32: from the lanes, 128 bytes a warp and row. The tensor cores' accumulation error grows
    // with its length (router logits over 4096 inputs 3.9e-6 of their norm in one run, 8.9e-7 in
    // runs of 1024), so a long K is cut into segments that are added in fp32 here: in registers,
    // kept between the calls of a unit, where nothing but a bias follows ...
    MOK_DEV void direct_sums(int seg, uint32_t c, int hw, int f, int g, int64_t r0, int nr,
                             int n_out, float (&acc)[2 * E::CHUNKS][16]) const {
        const bool last = seg == segs - 1;
        const float b = last && bias != nullptr && f < N ? bias[(int64_t)g * N + f] : 0.f;
#pragma unroll
        for (int k = 0; k < 2 * E::CHUNKS; ++k) {
            const int n0 = 32 * hw + E::STEP * (k >> 1) + 16 * (k & 1);
            if (n0 >= n_out) continue;
            float v[16];
            tc::tmem_ld16(c + n0, v);
            tc::tmem_ld_wait();
            loaded(v);
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[k][j] = (seg > 0 ? acc[k][j] : b) + v[j];
            if (!last || f >= N) continue;
            float *yp = static_cast<float *>(y) + (r0 + n0) * ld + f;
            const float b1 = segs > 1 ? b : 0.f;  // a single segment began with it
#pragma unroll
            for (int j = 0; j < 16; ++j, yp += ld)
                if (n0 + j < n_out) *yp = n0 + j < nr ? acc[k][j] + b1 : 0.f;
        }
    }
    // ... or in y, each element by the thread that will finish it
    MOK_DEV void direct(int seg, uint32_t c, int hw, int f, int g, int64_t r0, int nr,
                        int n_out) const {
        const bool ok = f < N, last = seg == segs - 1;
        const float b = last && bias != nullptr && ok ? bias[(int64_t)g * N + f] : 0.f;
        for (int n0 = 16 * hw; n0 < n_out; n0 += E::STEP / 2) {
            float v[16];
            tc::tmem_ld16(c + n0, v);
            tc::tmem_ld_wait();
            loaded(v);
            if (!ok) continue;
            const int64_t o = (r0 + n0) * ld + f;
            const int left = nr - n0, out = n_out - n0;  // real rows, rows to write
            float *yp = static_cast<float *>(y) + o;
            if (seg > 0) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < left) v[j] += yp[(int64_t)j * ld];
            }
            if (!last) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < left) yp[(int64_t)j * ld] = v[j];
                continue;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = j < left ? v[j] + b : 0.f;
            if (z != nullptr) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < out) z[o + (int64_t)j * ld] = (uint16_t)pack2(v[j], 0.f);
            }
            with_act(act, [&](auto a) {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = act_f<a.value>(v[j]);
            });
            if (res != nullptr) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < left) v[j] += bf16_to_f32(res[o + (int64_t)j * ld]);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (j < out) yp[(int64_t)j * ld] = v[j];
        }
    }
};

// The input gradient; CUT: K may be cut into parts. 64 groups of 320 rows, 1024 -> 4096: 126 us,
// 5.9 TB/s (W is most of it); tiles of 160 rows take longer to load than to multiply.
// F32: dz comes as `halves` planes of bf16 that add up to it, and the sums of segments of K, for
// the accuracy of a long sum, are added in registers (see Fwd). 16384 rows, 4096 -> 512, fp32 dy,
// dx and dW: 283 us and 2.6e-6 of the norm; with dz as one bf16 value and K in one run 169 us and
// 1.7e-3. bf16 gradients of the same 91 us. (Register sums spill 40 to 230 bytes.)
template <bool F32, bool CUT>
struct Dx {
    using E = Epi<F32>;
    static constexpr bool F32_OUT = F32, SUMS = F32;
    static constexpr bool A_MN = true, B_MN = false;
    Tiles tiles;
    int n_mb;     // ceil(Kin / 256)
    int halves;   // planes of dz: 2 for fp32 gradients of a dz that bf16 does not hold
    int Kin, N;
    int64_t ld;   // row stride of dx
    void *dx;
    int *status;
    KParts kp;

    MOK_DEV int64_t n_units() const { return tiles.count() * n_mb * (CUT ? kp.parts : 1); }
    MOK_DEV void side_work(uint32_t, uint32_t, int) const {}
    MOK_DEV Unit unit(uint32_t u) const {
        const int part = CUT ? kp.take(u, (uint32_t)(tiles.cap * n_mb)) : 0;
        const int4 t = tiles.get(u / (uint32_t)n_mb);
        return Unit{t.x, t.y, t.z - t.y, t.w, (int)(u % (uint32_t)n_mb), 0, part};
    }
    MOK_DEV LinGeom k_range(const Unit &u) const {
        LinGeom q;
        q.k_steps = (N + 15) / 16;
        q.k_first = q.half = 0;
        if constexpr (CUT) kp.cut(q, u.part);
        return q;
    }
    MOK_DEV int segments(const Unit &u) const { return F32 ? k_range(u).segments(halves) : 1; }
    MOK_DEV int long_steps(const Unit &) const { return 0; }
    MOK_DEV LinGeom geom(const Unit &u, int seg, uint32_t rank) const {
        LinGeom q = k_range(u);
        if constexpr (F32) q.segment(seg, halves);
        q.n_mma = (u.nr + 15) & ~15;
        q.a0 = u.mb * 256 + (int)rank * 128;
        q.a1 = 0;
        q.a2 = u.g;
        q.b0 = 0;
        q.b1 = u.r0 + (int)rank * (q.n_mma / 2);
        q.nbox = (q.n_mma / 2 + 31) / 32;
        return q;
    }
    MOK_DEV uint32_t tx(const LinGeom &q) const { return 2 * BOX + q.nbox * (BOX / 2); }
    // A: two boxes of 64 inputs x 64 features; B: the rows' 64 features of dz in boxes of 32 rows
    MOK_DEV void load(uint8_t *st, uint32_t fb, const LinGeom &q, int k0, const CUtensorMap *tmA,
                      const CUtensorMap *tmB) const {
        tma_load_3d_pair(st, tmA, fb, q.a0, k0, q.a2);
        tma_load_3d_pair(st + BOX, tmA, fb, q.a0 + 64, k0, q.a2);
        for (int j = 0; j < q.nbox; ++j) {
            uint8_t *b = st + 2 * BOX + j * (BOX / 2);
            if constexpr (F32)
                tma_load_3d_pair(b, tmB, fb, k0, q.b1 + 32 * j, q.half);
            else
                tc::tma_load_2d_pair(b, tmB, fb, k0, q.b1 + 32 * j);
        }
    }
    MOK_DEV void epilogue(const Unit &u, int seg, bool last, uint32_t rank, uint32_t c, int q, int hw,
                          int lane, Patches &pt, Carry<SUMS> &carry) const {
        const int nr = u.nr, pad = u.pad;
        const int64_t r0 = u.r0;
        const int n_mma = (nr + 15) & ~15;
        const int i0 = u.mb * 256 + (int)rank * 128 + q * 32;
        const bool part = CUT && kp.parts > 1;
        if constexpr (F32) {
            float *o = part ? kp.out + u.part * kp.stride + r0 * kp.ld
                            : static_cast<float *>(dx) + r0 * ld;
            const int64_t ldo = part ? kp.ld : ld;
            const int n_out = pad && !part ? n_mma : nr;
            sum_segments(c, hw, n_mma, seg == 0, last, carry, [&](int n0, const float (&v)[16]) {
                if (i0 + lane >= Kin) return;
                float *p = o + n0 * ldo + i0 + lane;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (n0 + j < n_out) p[j * ldo] = n0 + j < nr ? v[j] : 0.f;
            });
        } else if (part) {
            emit_part<E::STEP>(kp, u.part, c, hw, r0, nr, i0 + lane, Kin);
        } else {
            for (int n0 = 32 * hw; n0 < n_mma; n0 += E::STEP)
                emit_plain(pt, c + n0, nr - n0, OutRef{static_cast<uint16_t *>(dx), tiles.rows, ld, Kin},
                           i0 & ~63, r0 + n0, r0 + (pad ? n_mma : nr), 0);
        }
    }
};

// The bias gradient from the parts of the dz kernel: db[g][n] is the sum of the group's parts, in
// a fixed order.
constexpr int DZ_ROWS = 128;
constexpr int DZ_PARTS = LTILE / DZ_ROWS;  // parts of a tile
constexpr int DB_SLICES = 8;               // sums that a feature's parts are added in
struct DbArgs {
    const float *part;     // [tiles][DZ_PARTS][N]
    const int32_t *first;  // grouped: first tile of each group
    int64_t tiles;         // dense: all tiles
    float *db;             // [G][N], or nullptr
    // the group's parts: the first, and their number
    MOK_DEV const float *parts(int g, int n, int N, int64_t *count) const {
        const int64_t t0 = first != nullptr ? first[g] : 0;
        const int64_t t1 = first != nullptr ? first[g + 1] : tiles;
        *count = (t1 - t0) * DZ_PARTS;
        return part + t0 * DZ_PARTS * N + n;
    }
    // every DB_SLICES-th part from `slice` on
    MOK_DEV float slice(int g, int n, int N, int slice) const {
        int64_t count;
        const float *p = parts(g, n, N, &count);
        float a = 0.f;
#pragma unroll 16
        for (int64_t k = slice; k < count; k += DB_SLICES) a += p[k * N];
        return a;
    }
    // all of them in one thread, to the same bits as its slices added in order
    MOK_DEV float sum(int g, int n, int N) const {
        int64_t count;
        const float *p = parts(g, n, N, &count);
        float a[DB_SLICES], all = 0.f;
#pragma unroll
        for (int j = 0; j < DB_SLICES; ++j) a[j] = 0.f;
        int64_t k = 0;
        for (; k + 2 * DB_SLICES <= count; k += 2 * DB_SLICES) {
            float b[2 * DB_SLICES];
#pragma unroll
            for (int j = 0; j < 2 * DB_SLICES; ++j) b[j] = p[(k + j) * N];
#pragma unroll
            for (int j = 0; j < 2 * DB_SLICES; ++j) a[j % DB_SLICES] += b[j];
        }
        for (; k < count; k += DB_SLICES) {
            float b[DB_SLICES];
#pragma unroll
            for (int j = 0; j < DB_SLICES; ++j) b[j] = k + j < count ? p[(k + j) * N] : 0.f;
#pragma unroll
            for (int j = 0; j < DB_SLICES; ++j) a[j] += b[j];
        }
#pragma unroll
        for (int j = 0; j < DB_SLICES; ++j) all += a[j];
        return all;
    }
};

// The weight gradient, K along the group's rows. 64 groups of 320 rows, 1024 x 4096: 139 us,
// bound by writing 537 MB (132 us at the write-only rate of a memset, 4.06 TB/s).
template <bool F32, bool CUT>
struct Dw {
    using E = Epi<F32>;
    static constexpr bool F32_OUT = F32, SUMS = F32;
    static constexpr bool A_MN = true, B_MN = true;
    const int32_t *starts, *valid;  // grouped: first row and row count of each group
    int64_t rows;                   // dense
    int G, n_mb, n_nb;              // ceil(Kin / 256), ceil(N / 256)
    int halves;                     // planes of dz (F32; see Dx)
    int Kin, N;
    int64_t ld;                     // row stride of dW
    void *dw;
    int *status;
    DbArgs db;
    KParts kp;

    MOK_DEV int64_t n_units() const { return (int64_t)G * n_mb * n_nb * (CUT ? kp.parts : 1); }
    // a share of db, by the one warp of a pair that has nothing else to do
    MOK_DEV void side_work(uint32_t cid, uint32_t ncl, int lane) const {
        if (db.db == nullptr) return;
        for (int64_t i = (int64_t)cid * 32 + lane; i < (int64_t)G * N; i += (int64_t)ncl * 32)
            db.db[i] = db.sum((int)(i / N), (int)(i % N), N);
    }
    MOK_DEV Unit unit(uint32_t u) const {
        const uint32_t per = (uint32_t)n_mb * (uint32_t)n_nb;
        const int part = CUT ? kp.take(u, (uint32_t)G * per) : 0, g = (int)(u / per);
        const uint32_t rest = u % per;
        return Unit{g, starts != nullptr ? starts[g] : 0,
                    valid != nullptr ? valid[g] : (int)rows, 0,
                    (int)(rest % (uint32_t)n_mb), (int)(rest / (uint32_t)n_mb), part};
    }
    MOK_DEV LinGeom k_range(const Unit &u) const {
        LinGeom q;
        q.k_steps = (u.nr + 15) / 16;
        q.k_first = q.half = 0;
        if constexpr (CUT) kp.cut(q, u.part);
        return q;
    }
    MOK_DEV int segments(const Unit &u) const { return F32 ? k_range(u).segments(halves) : 1; }
    MOK_DEV int long_steps(const Unit &u) const { return F32 ? 0 : (u.nr + 15) / 16; }
    MOK_DEV LinGeom geom(const Unit &u, int seg, uint32_t rank) const {
        const int mb = u.mb, nb = u.nb;
        LinGeom q = k_range(u);
        if constexpr (F32) q.segment(seg, halves);
        // MN-major B comes in boxes of 64 columns per CTA: N of the MMA is 128 or 256, columns
        // past the matrix being zeros
        q.n_mma = N - nb * 256 <= 128 ? 128 : 256;
        q.nbox = q.n_mma / 128;
        q.a0 = mb * 256 + (int)rank * 128;
        q.a1 = u.r0;
        q.a2 = 0;
        q.b0 = nb * 256 + (int)rank * (q.n_mma / 2);
        q.b1 = q.a1;
        return q;
    }
    MOK_DEV uint32_t tx(const LinGeom &q) const { return (2 + q.nbox) * BOX; }
    MOK_DEV void load(uint8_t *st, uint32_t fb, const LinGeom &q, int k0, const CUtensorMap *tmA,
                      const CUtensorMap *tmB) const {
        tc::tma_load_2d_pair(st, tmA, fb, q.a0, q.a1 + k0);
        tc::tma_load_2d_pair(st + BOX, tmA, fb, q.a0 + 64, q.a1 + k0);
        for (int j = 0; j < q.nbox; ++j) {
            uint8_t *b = st + (2 + j) * BOX;
            if constexpr (F32)
                tma_load_3d_pair(b, tmB, fb, q.b0 + 64 * j, q.b1 + k0, q.half);
            else
                tc::tma_load_2d_pair(b, tmB, fb, q.b0 + 64 * j, q.b1 + k0);
        }
    }
    MOK_DEV void epilogue(const Unit &u, int seg, bool last, uint32_t rank, uint32_t c, int q, int hw,
                          int lane, Patches &pt, Carry<SUMS> &carry) const {
        const int g = u.g, mb = u.mb, nb = u.nb;
        const int nn = N - nb * 256 < 256 ? N - nb * 256 : 256;
        const bool any = u.nr > 0;
        const int i0 = mb * 256 + (int)rank * 128 + q * 32;
        const bool part = CUT && kp.parts > 1;
        if constexpr (F32) {
            float *o = part ? kp.out + u.part * kp.stride + nb * 256 * kp.ld
                            : static_cast<float *>(dw) + ((int64_t)g * N + nb * 256) * ld;
            const int64_t ldo = part ? kp.ld : ld;
            sum_segments(c, hw, nn, seg == 0, last, carry, [&](int n0, const float (&v)[16]) {
                if (i0 + lane >= Kin) return;
                float *p = o + n0 * ldo + i0 + lane;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (n0 + j < nn) p[j * ldo] = any ? v[j] : 0.f;
            });
        } else if (part) {
            emit_part<E::STEP>(kp, u.part, c, hw, nb * 256, nn, i0 + lane, Kin);
        } else {
            for (int n0 = 32 * hw; n0 < nn; n0 += E::STEP)
                emit_plain(pt, c + n0, any ? 32 : 0, OutRef{static_cast<uint16_t *>(dw), N, ld, Kin},
                           i0 & ~63, nb * 256 + n0, N, g);
        }
    }
};

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
        Carry<P::SUMS> carry;
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

// ---------------------------------------------------------------- parts of K
// The sums of the parts in order, for up to two outputs; bias, activation, residual and z (row
// strides as the output's) belong to the first. A thread takes four columns, loading eight parts
// at a time; the parts are still in L2, so launch and latency are what it costs, about 3 us.
struct JoinOut {
    const float *part;
    int64_t stride, ldp;  // of parts, of rows (a multiple of 4)
    int parts, cols;
    int64_t rows;
    void *out;
    int64_t ld;
    uint32_t blocks;
};
struct JoinArgs {
    JoinOut o[2];
    const float *bias;
    const uint16_t *res;
    uint16_t *z;
    int act;
};
constexpr int JOIN_TPB = 128;

template <bool F32>
__global__ void __launch_bounds__(JOIN_TPB) linear_join_kernel(const JoinArgs a) {
    let_next_start();
    wait_for_previous();
    const bool second = blockIdx.x >= a.o[0].blocks;
    const JoinOut &o = a.o[second];
    const uint32_t i = (blockIdx.x - (second ? a.o[0].blocks : 0)) * JOIN_TPB + threadIdx.x;
    const uint32_t nv = (uint32_t)(o.cols + 3) / 4, row = i / nv;
    const int c = (int)(i - row * nv) * 4;
    if (row >= o.rows) return;
    const float *p = o.part + row * o.ldp + c;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < o.parts; k0 += 8) {
        float4 b[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + k < o.parts)
                b[k] = *reinterpret_cast<const float4 *>(p + (k0 + k) * o.stride);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + k < o.parts) {
                v[0] += b[k].x;
                v[1] += b[k].y;
                v[2] += b[k].z;
                v[3] += b[k].w;
            }
    }
    const int64_t at = row * o.ld + c;
    const int n = o.cols - c < 4 ? o.cols - c : 4;  // columns past the matrix hold anything
    if (!second) {
        if (a.bias != nullptr)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < n) v[j] += a.bias[c + j];
        if (a.z != nullptr)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < n) a.z[at + j] = f32_to_bf16(v[j]);
        with_act(a.act, [&](auto act) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = act_f<act.value>(v[j]);
        });
        if (a.res != nullptr)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < n) v[j] += bf16_to_f32(a.res[at + j]);
    }
    if (F32 && n == 4) {
        *reinterpret_cast<float4 *>(static_cast<float *>(o.out) + at) =
            make_float4(v[0], v[1], v[2], v[3]);
    } else if (n == 4) {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(o.out) + at) =
            make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < n) st_val(o.out, at + j, v[j], F32);
    }
}

// ---------------------------------------------------------------- few rows
// Up to 32 dense rows (a decoded token, a small batch): the weights' bytes are all the work, and
// the 256-row tiles above put them on too few SMs (16 of 76 pairs for 4096 features). Here a
// warp takes 16 features and one of `parts` parts of the inputs with mma.sync (m16n8k16; its rate
// does not matter at 8 rows a weight), straight from registers: over 32 inputs a thread of a
// quad loads 8 consecutive ones of two features and of a row, 16 bytes each, and the
// instruction's K slots are assigned to inputs in that order, the same for both operands, since
// a sum does not care. Parts are added in order through shared memory.
constexpr int SMALL_ROWS = 32;
constexpr int SMALL_F = 16;  // features of a warp

struct SmallArgs {
    const uint16_t *x, *w, *res;
    const float *bias;
    void *y;
    uint16_t *z;
    int Kin, N, rows, act, parts;
    int64_t ld_in, ld_w, ld_out;
};

MOK_DEV void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                       uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 inputs from column c of a row, zeros past Kin
MOK_DEV uint4 load_piece(const uint16_t *row, int c, int Kin) {
    if (c + 8 <= Kin) return ld_v4(row + c);
    uint32_t e[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (c + j < Kin) e[j >> 1] |= (uint32_t)row[c + j] << (16 * (j & 1));
    return make_uint4(e[0], e[1], e[2], e[3]);
}

// NT groups of 8 rows (rows past a.rows repeat the last and are not stored), UN steps of 32 inputs
// in flight
template <int NT, int UN, bool F32>
__global__ void __launch_bounds__(256)
    linear_small_kernel(const SmallArgs a) {
    __shared__ float sh[8][SMALL_F][8 * NT + 1];
    let_next_start();
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = warp % a.parts, slot = warp / a.parts;
    const int per_block = 8 / a.parts * SMALL_F;
    const int f0 = blockIdx.x * per_block + slot * SMALL_F;
    const int q = lane >> 2, t = lane & 3;
    const uint16_t *w0 = a.w + (int64_t)(f0 + q < a.N ? f0 + q : a.N - 1) * a.ld_w;
    const uint16_t *w1 = a.w + (int64_t)(f0 + q + 8 < a.N ? f0 + q + 8 : a.N - 1) * a.ld_w;
    const uint16_t *xp[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
        xp[i] = a.x + (int64_t)(8 * i + q < a.rows ? 8 * i + q : a.rows - 1) * a.ld_in;
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    for (int k0 = part * 32 * UN; k0 < a.Kin; k0 += a.parts * 32 * UN) {
        uint4 wa[UN], wb[UN], xv[UN][NT];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int c = k0 + 32 * u + 8 * t;
            wa[u] = load_piece(w0, c, a.Kin);
            wb[u] = load_piece(w1, c, a.Kin);
        }
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int i = 0; i < NT; ++i) xv[u][i] = load_piece(xp[i], k0 + 32 * u + 8 * t, a.Kin);
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                mma_16816(acc[i], wa[u].x, wb[u].x, wa[u].y, wb[u].y, xv[u][i].x, xv[u][i].y);
                mma_16816(acc[i], wa[u].z, wb[u].z, wa[u].w, wb[u].w, xv[u][i].z, xv[u][i].w);
            }
    }
    // acc[i]: features q and q + 8 (second pair), rows 8 i + 2 t and the next
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sh[warp][q + 8 * (j >> 1)][8 * i + 2 * t + (j & 1)] = acc[i][j];
    __syncthreads();
    for (int o = threadIdx.x; o < per_block * a.rows; o += 256) {  // features side by side
        const int r = o / per_block, fb = o % per_block;
        const int f = blockIdx.x * per_block + fb;
        if (f >= a.N) continue;
        float v = 0.f;
        for (int k = 0; k < a.parts; ++k) v += sh[fb / SMALL_F * a.parts + k][fb % SMALL_F][r];
        if (a.bias != nullptr) v += a.bias[f];
        const int64_t at = r * a.ld_out + f;
        if (a.z != nullptr) a.z[at] = f32_to_bf16(v);
        with_act(a.act, [&](auto act) { v = act_f<act.value>(v); });
        if (a.res != nullptr) v += bf16_to_f32(a.res[at]);
        st_val(a.y, at, v, F32);
    }
}

// One or two rows, and up to four of few features: whole rows of W side by side on the lanes,
// products on the fp32 units, few features a warp. More warps start on a narrow layer than with 16
// features a warp (4096 inputs, weights from HBM: one row 512 features 3.2 against 6.0 us, 4096
// features 7.7 against 9.2, 16384 24 against 29). Two rows read x as often as W with two features
// a warp, so wide layers take eight (2 rows, 4096 -> 8192: 14.8 against 20.5 us; 4096 -> 512: 4.1
// against 3.3).
// F features a warp, UN pieces a lane in flight
template <int R, int F, int UN, bool F32>
__global__ void __launch_bounds__(256)
    linear_vector_kernel(const SmallArgs a) {
    __shared__ float sh[8][F * R];
    let_next_start();
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = warp % a.parts, slot = warp / a.parts;
    const int per_block = 8 / a.parts * F;
    const int f0 = blockIdx.x * per_block + slot * F;
    const int nv = a.Kin / 8;
    const uint16_t *wp[F], *xp[R];
#pragma unroll
    for (int f = 0; f < F; ++f)
        wp[f] = a.w + (int64_t)(f0 + f < a.N ? f0 + f : a.N - 1) * a.ld_w;
#pragma unroll
    for (int r = 0; r < R; ++r) xp[r] = a.x + (int64_t)(r < a.rows ? r : a.rows - 1) * a.ld_in;
    float acc[F][R];
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[f][r] = 0.f;
    for (int v0 = part * 32 + lane; v0 < nv; v0 += a.parts * 32 * UN) {
        uint4 wv[UN][F];
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const int v = v0 + u * a.parts * 32;
                wv[u][f] = make_uint4(0, 0, 0, 0);
                if (v < nv) wv[u][f] = ld_v4(wp[f] + (int64_t)v * 8);
            }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int v = v0 + u * a.parts * 32;
            if (v >= nv) break;
            float xf[R][8];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint4 q = ld_v4(xp[r] + (int64_t)v * 8);
                const uint32_t e[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    xf[r][2 * j] = bf16_lo(e[j]);
                    xf[r][2 * j + 1] = bf16_hi(e[j]);
                }
            }
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const uint32_t e[4] = {wv[u][f].x, wv[u][f].y, wv[u][f].z, wv[u][f].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float lo = bf16_lo(e[j]), hi = bf16_hi(e[j]);
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        acc[f][r] = fmaf(hi, xf[r][2 * j + 1], fmaf(lo, xf[r][2 * j], acc[f][r]));
                }
            }
        }
    }
    if (part == 0) {  // the inputs past the last whole piece
        const int c = nv * 8 + lane;
        if (c < a.Kin) {
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
                for (int r = 0; r < R; ++r)
                    acc[f][r] = fmaf(bf16_to_f32(wp[f][c]), bf16_to_f32(xp[r][c]), acc[f][r]);
        }
    }
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float v = acc[f][r];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            if (lane == 0) sh[warp][f * R + r] = v;
        }
    __syncthreads();
    // one thread per output of the block; features side by side
    const int n = per_block * R;
    if (threadIdx.x >= n) return;
    const int r = threadIdx.x / per_block, fb = threadIdx.x % per_block;
    const int f = blockIdx.x * per_block + fb;
    if (f >= a.N || r >= a.rows) return;
    float v = 0.f;
    for (int k = 0; k < a.parts; ++k)
        v += sh[fb / F * a.parts + k][fb % F * R + r];
    if (a.bias != nullptr) v += a.bias[f];
    const int64_t o = r * a.ld_out + f;
    if (a.z != nullptr) a.z[o] = f32_to_bf16(v);
    with_act(a.act, [&](auto act) { v = act_f<act.value>(v); });
    if (a.res != nullptr) v += bf16_to_f32(a.res[o]);
    st_val(a.y, o, v, F32);
}

// ---------------------------------------------------------------- dz and the bias gradient
// dz = dy act'(z) in bf16 (the products' operand), and the column sums of the unrounded dz. One
// block per half tile (up to 128 rows) and 64 columns: 8 threads side by side on 8 columns each, 32
// row lanes of 4 rows each, whose loads are all issued before the first is used (one row at a
// time, 20480 x 1024 took 47 us, so 27; 126 MB are 19 at the copy rate); the sums of a column's 32
// row lanes are added in lane order.
// LO: what bf16 leaves of dz goes to a second plane, `plane` elements on, in bf16 again: the two
// are within 2^-17 of dz. Nothing where dz is not finite in bf16.
template <bool DY32, int ACT, bool LO>
__global__ void __launch_bounds__(256)
    linear_dz_kernel(const void *dy, const uint16_t *z, Tiles tiles, int N, int64_t ld, uint16_t *dz,
                     int64_t ld_dz, int64_t plane, float *part) {
    __shared__ float red[32][65];
    let_next_start();
    wait_for_previous();
    // column blocks first: neighbours in time read neighbouring parts of the same rows
    const uint32_t ncb = (uint32_t)(N + 63) / 64, part_id = blockIdx.x / ncb, cb = blockIdx.x % ncb;
    const int64_t t = part_id / DZ_PARTS;
    if (t >= tiles.count()) return;
    const int4 tile = tiles.get(t);
    // the tile in equal parts, multiples of 16 rows; the last takes the padding
    const int per = ((tile.z - tile.y + DZ_PARTS - 1) / DZ_PARTS + 15) & ~15;
    const int64_t r0 = tile.y + (int64_t)(part_id % DZ_PARTS) * per;
    const int64_t all = tile.w != 0 ? (tile.z + 15) & ~15 : tile.z;  // one past the rows to write
    const int64_t rend = r0 + per < all ? r0 + per : all, r1 = rend < tile.z ? rend : tile.z;
    const int cv = threadIdx.x & 7, rl = threadIdx.x >> 3;
    const int c = (int)cb * 64 + cv * 8;
    constexpr int NR = DZ_ROWS / 32;
    const bool whole = c + 8 <= N;
    uint4 a[NR], a2[NR], q[NR];  // dy (fp32: two vectors), z
    if (whole) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int64_t r = r0 + rl + 32 * i, o = r * ld + c;
            a[i] = a2[i] = q[i] = make_uint4(0, 0, 0, 0);
            if (r < r1) {
                if (DY32) {
                    a[i] = ld_v4(static_cast<const float *>(dy) + o);
                    a2[i] = ld_v4(static_cast<const float *>(dy) + o + 4);
                } else {
                    a[i] = ld_v4(static_cast<const uint16_t *>(dy) + o);
                }
                if (ACT != MOK_ACT_NONE) q[i] = ld_v4(z + o);
            }
        }
    }
    float sum[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = 0.f;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int64_t r = r0 + rl + 32 * i, o = r * ld + c;
        if (r >= rend || c >= N) continue;
        float v[8], zz[8];
        if (whole) {
            const uint32_t w[8] = {a[i].x, a[i].y, a[i].z, a[i].w,
                                   a2[i].x, a2[i].y, a2[i].z, a2[i].w};
            const uint32_t y[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = DY32 ? __uint_as_float(w[j])
                            : (j & 1) ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
                zz[j] = (j & 1) ? bf16_hi(y[j >> 1]) : bf16_lo(y[j >> 1]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = c + j < N && r < r1;
                v[j] = !in ? 0.f
                       : DY32 ? static_cast<const float *>(dy)[o + j]
                              : bf16_to_f32(static_cast<const uint16_t *>(dy)[o + j]);
                zz[j] = in && ACT != MOK_ACT_NONE ? bf16_to_f32(z[o + j]) : 0.f;
            }
        }
        if (ACT != MOK_ACT_NONE) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= act_grad_f<ACT>(zz[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += v[j];  // absent rows and columns are zero
        if (dz != nullptr) {  // ld_dz is a multiple of 8: whole vectors
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = pack2(v[2 * j], v[2 * j + 1]);
            *reinterpret_cast<uint4 *>(dz + r * ld_dz + c) = make_uint4(h[0], h[1], h[2], h[3]);
            if constexpr (LO) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a = bf16_lo(h[j]), b = bf16_hi(h[j]);
                    h[j] = pack2(isfinite(a) ? v[2 * j] - a : 0.f, isfinite(b) ? v[2 * j + 1] - b : 0.f);
                }
                *reinterpret_cast<uint4 *>(dz + plane + r * ld_dz + c) =
                    make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
    }
    if (part == nullptr) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) red[rl][cv * 8 + j] = sum[j];
    __syncthreads();
    if (threadIdx.x < 64) {
        const int col = (int)cb * 64 + threadIdx.x;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
        if (col < N) part[(int64_t)part_id * N + col] = s;
    }
}

// db where the dW kernel does not add the parts: a block takes 32 features, each warp a slice of
// their parts (narrow layers have many rows and few features: dx, dW and db of 16384 rows x 64 x 64
// 30 us with a thread a feature, 17 us so)
__global__ void __launch_bounds__(32 * DB_SLICES)
    linear_db_kernel(const DbArgs d, int G, int N) {
    __shared__ float sh[DB_SLICES][32];
    let_next_start();
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + lane;
    const bool in = i < (int64_t)G * N;
    sh[warp][lane] = in ? d.slice((int)(i / N), (int)(i % N), N, warp) : 0.f;
    __syncthreads();
    if (warp != 0 || !in) return;
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < DB_SLICES; ++k) a += sh[k][lane];
    d.db[i] = a;
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

// one cluster per unit, at most the pairs of SMs that run at once
template <class P>
cudaError_t launch_linear(const CUtensorMap &ma, const CUtensorMap &mb, const P &p,
                          int64_t units_cap, cudaStream_t s) {
    if (units_cap < 1) return cudaSuccess;
    if (units_cap > 0x7FFFFFFF) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> attr_set{0};
    return launch_pairs(linear_kernel<P>, attr_set, P::E::THREADS,
                        units_cap < sm_pairs() ? units_cap : sm_pairs(), s, ma, mb, p);
}
template <class P, class Q>
cudaError_t launch_both(const CUtensorMap &pa, const CUtensorMap &pb, const P &p,
                        const CUtensorMap &qa, const CUtensorMap &qb, const Q &q, int64_t split,
                        int64_t pairs, cudaStream_t s) {
    static std::atomic<uint64_t> attr_set{0};
    return launch_pairs(linear_both_kernel<P, Q>, attr_set, P::E::THREADS, pairs, s, pa, pb, p, qa,
                        qb, q, (uint32_t)split);
}

template <bool DY32, bool LO>
cudaError_t launch_dz(int act, dim3 grid, const void *dy, const uint16_t *z, const Tiles &t, int N,
                      int64_t ld, uint16_t *dz, int64_t ld_dz, float *part, cudaStream_t s) {
#define MOK_DZ_CASE(A)                                                                          \
    case A:                                                                                     \
        return launch_edge(linear_dz_kernel<DY32, A, LO>, grid, 256, 0, 1, s, dy, z, t, N, ld,  \
                           dz, ld_dz, t.rows * ld_dz, part)
    switch (act) {
        MOK_DZ_CASE(MOK_ACT_RELU);
        MOK_DZ_CASE(MOK_ACT_SILU);
        MOK_DZ_CASE(MOK_ACT_GELU_TANH);
        MOK_DZ_CASE(MOK_ACT_GELU);
        MOK_DZ_CASE(MOK_ACT_NONE);
    }
#undef MOK_DZ_CASE
    return cudaErrorInvalidValue;
}

// Plans that a result's rounding depends on count the GB300's pairs of SMs, not the device's.
constexpr int64_t PLAN_PAIRS = 76;

// Whether a dense call of this size goes to the kernels for few rows; us with weights from HBM,
// these against the tiles (their K cut):
//   one row always, two but for wide layers with few inputs (one row, 4096 -> 4096: 7.7 against
//   10.1; 14336 -> 512: 5.6 against 9.8), up to four of few features (4096 -> 512: 3.8 against
//   7.5), all on the fp32 units;
//   up to 16 rows, but for wide layers (4 rows, 4096 -> 16384: 30 against 26) and for few features
//   over a long K, where the tiles' parts use more SMs (4 rows, 8192 -> 512: 10.2 against 8.3);
//   up to 32 rows on small layers (1024 -> 1024: 5.3 against 6.5; 4096 -> 4096: 16 against 12).
// Two rows, 1024 -> 4096: 5.1 on the fp32 units, 3.9 with mma.sync.
bool vector_rows(int64_t rows, int64_t Kin, int64_t N) {
    return rows == 1 || (rows == 2 && (N <= 2048 || Kin >= 2048)) || (rows <= 4 && N <= 1024);
}
bool few_rows(int64_t rows, int64_t Kin, int64_t N) {
    if (vector_rows(rows, Kin, N)) return true;
    if (rows <= 16) return !(N >= 8192 && Kin >= 1024) && !(Kin >= 8192 && N <= 2048);
    return rows <= SMALL_ROWS && Kin <= 1024 && N <= 4096;
}

template <bool F32>
cudaError_t launch_small(SmallArgs a, cudaStream_t s) {
    const bool vec = vector_rows(a.rows, a.Kin, a.N), wide = vec && a.rows == 2 && a.N >= 2048;
    const int per_warp = vec ? (wide ? 8 : 2) : SMALL_F;
    // a warp's features in more parts until there are two blocks an SM; on the fp32 units each part
    // keeps a few steps. With mma.sync also where parts stay empty: a block with fewer features has
    // fewer outputs to write (32 rows, 64 -> 512: 2.6 us, 7.8 with one part)
    a.parts = 1;
    while (a.parts < 8 && (!vec || a.Kin / a.parts >= 256) &&
           (int64_t)a.N * a.parts < 2 * (2 * PLAN_PAIRS) * 8 * per_warp)
        a.parts *= 2;
    const int per_block = 8 / a.parts * per_warp;
    const unsigned grid = (unsigned)((a.N + per_block - 1) / per_block);
    if (vec && a.rows == 1)
        return launch_edge(linear_vector_kernel<1, 2, 4, F32>, grid, 256, 0, 1, s, a);
    if (wide) return launch_edge(linear_vector_kernel<2, 8, 1, F32>, grid, 256, 0, 1, s, a);
    if (vec && a.rows == 2)
        return launch_edge(linear_vector_kernel<2, 2, 4, F32>, grid, 256, 0, 1, s, a);
    if (vec) return launch_edge(linear_vector_kernel<4, 2, 4, F32>, grid, 256, 0, 1, s, a);
    if (a.rows <= 8) return launch_edge(linear_small_kernel<1, 4, F32>, grid, 256, 0, 1, s, a);
    if (a.rows <= 16) return launch_edge(linear_small_kernel<2, 4, F32>, grid, 256, 0, 1, s, a);
    return launch_edge(linear_small_kernel<4, 2, F32>, grid, 256, 0, 1, s, a);
}

cudaError_t launch_join(bool f32, const JoinArgs &j, cudaStream_t s) {
    const dim3 grid(j.o[0].blocks + j.o[1].blocks);
    return launch_edge(f32 ? linear_join_kernel<true> : linear_join_kernel<false>, grid, JOIN_TPB, 0,
                       1, s, j);
}

bool grouped(const int32_t *starts) { return starts != nullptr; }

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

// The most rows of a tile of a grouped product: fewer than 256 where the groups' tiles by n_mb
// blocks would leave pairs of SMs idle, by the waves of evenly filled groups (4 groups of 256 rows,
// 4096 -> 256: 24 us with tiles of up to 256 rows, 17 us of 32). The order of db's sum follows the
// tiles.
int group_height(int64_t rows, int G, int64_t n_mb) {
    const int64_t per = rows / G > 0 ? rows / G : 1;
    int64_t best = INT64_MAX;
    int best_h = LTILE;
    for (int h0 = LTILE; h0 >= 32; h0 /= 2) {
        const int64_t n = (per + h0 - 1) / h0, h = round_up((per + n - 1) / n, 16);
        const int64_t t = (G * n * n_mb + PLAN_PAIRS - 1) / PLAN_PAIRS * block_clocks(h);
        if (best == INT64_MAX || t < best * 9 / 10) {
            best = t;
            best_h = h0;
        }
    }
    return best_h;
}

// How a dense product is cut along K, by the sizes alone.
constexpr int64_t MAX_PART_BYTES = 32 << 20;  // of all parts: they stay in L2
struct Cut {
    int parts, per, height;  // height: of the tiles the parts run on
};
// `rows` rows in tiles (of any height, or of `fixed` rows) by n_mb blocks of the other dimension
// on `pairs` pairs of SMs, K blocks `blocks` long, parts at most max_per of them; `cols` columns
// of output.
Cut plan_parts(int64_t rows, int64_t n_mb, int64_t blocks, int64_t cols, int64_t pairs,
               int64_t max_per, int fixed) {
    Cut best{1, (int)(blocks < INT32_MAX ? blocks : INT32_MAX), 0};
    if (rows * n_mb > pairs * 2 * LTILE || blocks < 4) return best;  // enough units as it is
    int64_t whole;
    if (fixed > 0)
        whole = ((rows + fixed - 1) / fixed * n_mb + pairs - 1) / pairs * block_clocks(fixed);
    else
        dense_height(rows, n_mb, pairs, &whole);
    // a part has to save more than the join kernel costs: about 5000 clocks, and the parts' bytes
    // written and read at 2500 a clock
    const int64_t join = 5000, bytes = rows * round_up(cols, 4) * 4;
    int64_t least = whole * blocks - 1000;
    if (least <= join) return best;
    for (int64_t h0 = fixed > 0 ? fixed : LTILE; h0 >= 16; h0 -= 16) {
        const int64_t n = (rows + h0 - 1) / h0;
        const int64_t h = fixed > 0 ? fixed : round_up((rows + n - 1) / n, 16);
        const int64_t units = n * n_mb, most = pairs / units;
        // 2, 3, 5, 8, 12, .. parts and as many as there are pairs for
        for (int64_t want = 2, next = 0; want <= most; want = next) {
            next = want * 3 / 2 + want % 2;
            if (want < most && next > most) next = most;
            const int64_t per = (blocks + want - 1) / want, parts = (blocks + per - 1) / per;
            if (parts < 2 || per > max_per || parts * bytes > MAX_PART_BYTES) continue;
            const int64_t t = per * block_clocks(h) + join + parts * bytes * 2 / 2500;
            if (t < least) {
                least = t;
                best = Cut{(int)parts, (int)per, (int)h};
            }
        }
        if (fixed > 0) break;
    }
    return best;
}
Cut forward_cut(const mok_linear_config &c) {
    return plan_parts(c.rows, (c.out_features + 255) / 256, (c.in_features + BK - 1) / BK,
                      c.out_features, PLAN_PAIRS,
                      c.out_dtype == MOK_DTYPE_F32 ? SEG_K / BK : INT32_MAX, 0);
}
// dx and dW side by side, each with its share of the SMs by its work (whether or not a call asks
// for both: its bits do not depend on that)
void backward_cuts(const mok_linear_config &c, Cut *x, Cut *w) {
    const int64_t kb = (c.in_features + 255) / 256, nb = (c.out_features + 255) / 256;
    const int64_t x_blocks = (c.out_features + BK - 1) / BK, w_blocks = (c.rows + BK - 1) / BK;
    const int fixed = c.out_features <= 128 ? 128 : LTILE;
    int64_t per_block;
    dense_height(c.rows, kb, PLAN_PAIRS, &per_block);
    const int64_t cx = per_block * x_blocks;
    const int64_t cw = (kb * nb + PLAN_PAIRS - 1) / PLAN_PAIRS * block_clocks(fixed) * w_blocks;
    int64_t px = PLAN_PAIRS * cx / (cx + cw > 0 ? cx + cw : 1);
    px = px < 1 ? 1 : px > PLAN_PAIRS - 1 ? PLAN_PAIRS - 1 : px;
    *x = plan_parts(c.rows, kb, x_blocks, c.in_features, px, INT32_MAX, 0);
    *w = plan_parts(c.out_features, kb, w_blocks, c.in_features, PLAN_PAIRS - px, INT32_MAX, fixed);
}
size_t part_bytes(const Cut &c, int64_t rows, int64_t cols) {
    return c.parts > 1 ? (size_t)c.parts * rows * round_up(cols, 4) * 4 : 0;
}
KParts k_parts(const Cut &c, float *out, int64_t rows, int64_t cols) {
    return KParts{c.parts, c.per, out, round_up(cols, 4), rows * round_up(cols, 4)};
}
JoinOut join_out(const KParts &k, int64_t rows, int cols, void *out, int64_t ld) {
    const int64_t n = rows * ((cols + 3) / 4);
    return JoinOut{k.out, k.stride, k.ld, k.parts, cols, rows, out, ld,
                   (uint32_t)((n + JOIN_TPB - 1) / JOIN_TPB)};
}

// Whether two products of `a` and `b` equal units (ta, tb clocks each) run better side by side
// than one after the other: *split pairs of SMs for the first and the rest of *pairs for the
// second, or 0. Side by side there is one launch and one tail, but each has fewer pairs.
void plan_both(int64_t a, int64_t ta, int64_t b, int64_t tb, int64_t *split, int64_t *pairs) {
    const int64_t all = sm_pairs(), once = 12000;  // clocks of a launch, its fill and its drain
    const auto waves = [](int64_t n, int64_t p) { return (n + p - 1) / p; };
    int64_t best = waves(a, all) * ta + waves(b, all) * tb + once;
    *split = *pairs = 0;
    for (int64_t k = 1; k < all; ++k) {
        const int64_t x = waves(a, k) * ta, y = waves(b, all - k) * tb;
        if ((x > y ? x : y) < best) {
            best = x > y ? x : y;
            *split = k < a ? k : a;
            *pairs = *split + (all - k < b ? all - k : b);
        }
    }
}

struct LinWs {
    int32_t *list;    // past its 16-byte header
    int64_t cap;
    int height;       // most rows of a tile in it
    int32_t *valid;   // [G]
    int32_t *first;   // [G + 1]
    uint16_t *dz;     // [halves][rows][ld_dz]
    int64_t ld_dz;
    float *part;      // [tiles][DZ_PARTS][N]
    Cut cut[2];       // along K: y, or dx and dW (dense)
    float *kp[2];     // their parts
};

// without an activation a bf16 dy is dz
bool dz_is_dy(const mok_linear_config &c) {
    return c.act == MOK_ACT_NONE && c.out_dtype == MOK_DTYPE_BF16;
}
// bf16 values that dz enters a product as: fp32 gradients take what one leaves as a second (see Dx)
int dz_halves(const mok_linear_config &c) {
    return c.grad_dtype == MOK_DTYPE_F32 && !dz_is_dy(c) ? 2 : 1;
}

size_t carve_linear(const mok_linear_config &c, int pass, void *ws, LinWs *o) {
    size_t off = 0;
    const auto take = [&](size_t bytes) {
        off = (size_t)round_up((int64_t)off, 256);
        void *p = ws != nullptr ? (char *)ws + off : nullptr;
        off += bytes;
        return p;
    };
    LinWs w = {};
    const int across = pass == MOK_LINEAR_BACKWARD ? c.in_features : c.out_features;
    w.height = group_height(c.rows, c.groups, (across + 255) / 256);
    w.cap = tiles_cap(c.rows, c.groups, w.height);
    int32_t *l = (int32_t *)take(16 + (size_t)w.cap * 16);
    w.list = l != nullptr ? l + 4 : nullptr;
    w.valid = (int32_t *)take((size_t)c.groups * 4);
    w.first = (int32_t *)take((size_t)(c.groups + 1) * 4);
    if (pass == MOK_LINEAR_BACKWARD) {
        w.ld_dz = round_up(c.out_features, 8);
        w.dz = (uint16_t *)take((size_t)c.rows * w.ld_dz * 2 * dz_halves(c));
        w.part = (float *)take((size_t)w.cap * DZ_PARTS * c.out_features * 4);
    }
    const Cut whole{1, 0, 0};
    w.cut[0] = w.cut[1] = whole;
    if (c.groups == 1 && pass == MOK_LINEAR_BACKWARD)
        backward_cuts(c, &w.cut[0], &w.cut[1]);
    else if (c.groups == 1 && !few_rows(c.rows, c.in_features, c.out_features))
        w.cut[0] = forward_cut(c);
    w.kp[0] = (float *)take(part_bytes(w.cut[0], c.rows, across));
    w.kp[1] = (float *)take(part_bytes(w.cut[1], c.out_features, c.in_features));
    if (o != nullptr) *o = w;
    return off;
}

mok_status check_linear(const mok_linear_config *c, const int32_t *starts, const int32_t *counts,
                        void *ws, size_t ws_bytes, int pass, int **status, LinWs *wk) {
    mok_status st = mok_check_linear_config(c);
    if (st != MOK_OK) return st;
    if ((st = current_device_status_word(status)) != MOK_OK) return st;
    if ((starts == nullptr) != (counts == nullptr)) return MOK_ERR_INVALID_ARG;
    if (starts == nullptr && c->groups != 1) return MOK_ERR_INVALID_ARG;
    if (carve_linear(*c, pass, ws, wk) > ws_bytes || ws == nullptr || ((uintptr_t)ws & 255u) != 0)
        return MOK_ERR_WORKSPACE;
    return MOK_OK;
}

}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

mok_status mok_check_linear_config(const mok_linear_config *c) {
    if (c == nullptr) return MOK_ERR_INVALID_ARG;
    if (c->abi_version != MOK_ABI_VERSION) return MOK_ERR_ABI;
    if (c->groups < 1 || c->groups > MAX_G) return MOK_ERR_INVALID_ARG;
    const int32_t most = 1 << 20;
    if (c->in_features < 1 || c->in_features > most || c->out_features < 1 ||
        c->out_features > most)
        return MOK_ERR_INVALID_ARG;
    if (c->rows < 0 || c->rows >= ((int64_t)1 << 31) - 512) return MOK_ERR_INVALID_ARG;
    const int64_t far = (int64_t)1 << 30;
    const int64_t lds[] = {c->ld_in, c->ld_w, c->ld_out};
    const int32_t widths[] = {c->in_features, c->in_features, c->out_features};
    for (int i = 0; i < 3; ++i)
        if (lds[i] < widths[i] || lds[i] % 8 != 0 || lds[i] > far) return MOK_ERR_INVALID_ARG;
    // units of the products and blocks of the dz kernel are numbered in 31 bits
    const int64_t G = c->groups, kb = (c->in_features + 255) / 256, nb = (c->out_features + 255) / 256;
    const int64_t tiles = c->rows / 16 + G + 1, limit = 0x7FFFFFFF;
    if (tiles * (kb > nb ? kb : nb) > limit || G * kb * nb > limit ||
        (c->rows / DZ_ROWS + 2 * G + 4) * ((c->out_features + 63) / 64) > limit)
        return MOK_ERR_INVALID_ARG;
    if (c->act < MOK_ACT_NONE || c->act > MOK_ACT_GELU || c->reserved != 0)
        return MOK_ERR_INVALID_ARG;
    const int32_t dts[] = {c->out_dtype, c->grad_dtype};
    for (int32_t d : dts)
        if (d != MOK_DTYPE_BF16 && d != MOK_DTYPE_F32) return MOK_ERR_INVALID_ARG;
    return MOK_OK;
}

size_t mok_linear_workspace_size(const mok_linear_config *c, int pass) {
    if (mok_check_linear_config(c) != MOK_OK) return 0;
    if (pass != MOK_LINEAR_FORWARD && pass != MOK_LINEAR_BACKWARD) return 0;
    return carve_linear(*c, pass, nullptr, nullptr);
}

mok_status mok_linear_forward(const mok_linear_config *c, const void *x, const void *w,
                              const float *bias, const void *residual, const int32_t *starts,
                              const int32_t *counts, void *y, void *z, void *ws, size_t ws_bytes,
                              cudaStream_t stream) {
    int *status;
    LinWs wk;
    mok_status st =
        check_linear(c, starts, counts, ws, ws_bytes, MOK_LINEAR_FORWARD, &status, &wk);
    if (st != MOK_OK) return st;
    if (c->rows == 0) return MOK_OK;
    if (!x || !w || !y) return MOK_ERR_INVALID_ARG;
    const void *ps[] = {x, w, bias, residual, starts, counts, y, z};
    for (const void *p : ps)
        if (p && !op_aligned16(p)) return MOK_ERR_INVALID_ARG;
    if (!grouped(starts) && few_rows(c->rows, c->in_features, c->out_features)) {
        const SmallArgs a{(const uint16_t *)x, (const uint16_t *)w, (const uint16_t *)residual, bias,
                          y, (uint16_t *)z, c->in_features, c->out_features, (int)c->rows, c->act,
                          1, c->ld_in, c->ld_w, c->ld_out};
        MOK_OP_LAUNCH(OP_LINEAR_FWD, 1,
                      c->out_dtype == MOK_DTYPE_F32 ? launch_small<true>(a, stream)
                                                    : launch_small<false>(a, stream));
        return MOK_OK;
    }
    if (init_host() != cudaSuccess) return MOK_ERR_CUDA;
    const int n_mb = (c->out_features + 255) / 256;
    Tiles tiles;
    Cut cut{1, 0, 0};
    if (grouped(starts)) {
        tiles = Tiles{wk.list, wk.cap, c->rows, wk.height};
        MOK_OP_LAUNCH(OP_LINEAR_TILES, 1,
                      launch_edge(linear_tiles_kernel, 1, MAX_G, 0, 1, stream, starts, counts,
                                  c->groups, c->rows, wk.height, wk.list, wk.valid, wk.first,
                                  status));
    } else {
        cut = wk.cut[0];
        int64_t t;
        tiles = dense_tiles(c->rows, cut.parts > 1 ? cut.height
                                                   : dense_height(c->rows, n_mb, sm_pairs(), &t));
    }
    const KParts kp = k_parts(cut, wk.kp[0], c->rows, c->out_features);
    const bool f32 = c->out_dtype == MOK_DTYPE_F32;
    CUtensorMap ma, mb;
    if (map_w(&ma, w, c->groups, c->out_features, c->in_features, c->ld_w, 128) != cudaSuccess ||
        map2d(&mb, x, c->rows, c->in_features, c->ld_in, 32) != cudaSuccess)
        return MOK_ERR_CUDA;
    const int segs = f32 && cut.parts == 1 ? (c->in_features + SEG_K - 1) / SEG_K : 1;
    const int64_t units = tiles.cap * n_mb * cut.parts;
    const bool plain = c->act == MOK_ACT_NONE && !residual && !z;
#define MOK_FWD(...)                                                                            \
    do {                                                                                        \
        const Fwd<__VA_ARGS__> p{tiles, n_mb, segs, c->in_features, c->out_features, c->ld_out, bias, \
                           (const uint16_t *)residual, y, (uint16_t *)z, c->act, status, kp};   \
        MOK_OP_LAUNCH(OP_LINEAR_FWD, 1, launch_linear(ma, mb, p, units, stream));               \
    } while (0)
    if (cut.parts > 1) MOK_FWD(false, false, true);
    else if (!f32) MOK_FWD(false, false);
    else if (plain) MOK_FWD(true, true);
    else MOK_FWD(true, false);
#undef MOK_FWD
    if (cut.parts > 1) {
        JoinArgs j = {};
        j.o[0] = join_out(kp, c->rows, c->out_features, y, c->ld_out);
        j.bias = bias;
        j.res = (const uint16_t *)residual;
        j.z = (uint16_t *)z;
        j.act = c->act;
        MOK_OP_LAUNCH(OP_LINEAR_FWD, 1, launch_join(f32, j, stream));
    }
    return MOK_OK;
}

mok_status mok_linear_backward(const mok_linear_config *c, const void *x, const void *w,
                               const void *z, const void *dy, const int32_t *starts,
                               const int32_t *counts, void *dx, void *dw, float *db, void *ws,
                               size_t ws_bytes, cudaStream_t stream) {
    int *status;
    LinWs wk;
    mok_status st =
        check_linear(c, starts, counts, ws, ws_bytes, MOK_LINEAR_BACKWARD, &status, &wk);
    if (st != MOK_OK) return st;
    if (!dx && !dw && !db) return MOK_ERR_INVALID_ARG;
    const bool act = c->act != MOK_ACT_NONE, dy32 = c->out_dtype == MOK_DTYPE_F32;
    if (c->rows > 0 && (!dy || (act && !z) || (dx && !w) || (dw && !x)))
        return MOK_ERR_INVALID_ARG;
    const void *ps[] = {x, w, z, dy, starts, counts, dx, dw, db};
    for (const void *p : ps)
        if (p && !op_aligned16(p)) return MOK_ERR_INVALID_ARG;
    const int G = c->groups, N = c->out_features, Kin = c->in_features;
    const bool g32 = c->grad_dtype == MOK_DTYPE_F32;
    if (c->rows == 0) {  // sums over nothing
        const size_t es = g32 ? 4 : 2;
        if (dw && cudaMemset2DAsync(dw, (size_t)c->ld_w * es, 0, (size_t)Kin * es, (size_t)G * N,
                                    stream) != cudaSuccess)
            return MOK_ERR_CUDA;
        if (db && cudaMemsetAsync(db, 0, (size_t)G * N * 4, stream) != cudaSuccess)
            return MOK_ERR_CUDA;
        return MOK_OK;
    }
    if (init_host() != cudaSuccess) return MOK_ERR_CUDA;
    const int n_kb = (Kin + 255) / 256;
    Tiles tiles;
    Cut xc{1, 0, 0}, wc{1, 0, 0};
    if (grouped(starts)) {
        tiles = Tiles{wk.list, wk.cap, c->rows, wk.height};
        MOK_OP_LAUNCH(OP_LINEAR_TILES, 1,
                      launch_edge(linear_tiles_kernel, 1, MAX_G, 0, 1, stream, starts, counts,
                                  c->groups, c->rows, wk.height, wk.list, wk.valid, wk.first,
                                  status));
    } else {
        xc = wk.cut[0];
        wc = wk.cut[1];
        int64_t t;
        tiles = dense_tiles(c->rows, xc.parts > 1 ? xc.height
                                                  : dense_height(c->rows, n_kb, sm_pairs(), &t));
    }
    const KParts xk = k_parts(xc, wk.kp[0], c->rows, Kin), wkp = k_parts(wc, wk.kp[1], N, Kin);
    const bool direct = dz_is_dy(*c);
    const int halves = dz_halves(*c);
    const uint16_t *dz = direct ? (const uint16_t *)dy : wk.dz;
    const int64_t ld_dz = direct ? c->ld_out : wk.ld_dz;
    // The dW kernel adds the parts of db on the side, in the warps of the second SMs that issue no
    // MMAs, which saves a launch; with few inputs that kernel would end before its side work.
    const bool db_in_dw = dw && Kin >= 256;
    DbArgs dba{wk.part, grouped(starts) ? wk.first : nullptr, (c->rows + LTILE - 1) / LTILE, db};
    if (db || (!direct && (dx || dw))) {
        uint16_t *dzo = direct || (!dx && !dw) ? nullptr : wk.dz;
        float *part = db ? wk.part : nullptr;
        // dz has tiles of its own: full ones, whatever the products take
        const Tiles dzt = grouped(starts) ? tiles
                                          : Tiles{nullptr, (c->rows + LTILE - 1) / LTILE, c->rows, LTILE};
        const int64_t blocks = dzt.cap * DZ_PARTS * ((N + 63) / 64);
        const dim3 grid((unsigned)blocks);
        MOK_OP_LAUNCH(OP_LINEAR_DZ, 1,
                      (halves == 2 ? dy32 ? launch_dz<true, true> : launch_dz<false, true>
                       : dy32      ? launch_dz<true, false>
                                   : launch_dz<false, false>)(c->act, grid, dy, (const uint16_t *)z,
                                                              dzt, N, c->ld_out, dzo, ld_dz, part,
                                                              stream));
        if (db && !db_in_dw)
            MOK_OP_LAUNCH(OP_LINEAR_DZ, 1,
                          launch_edge(linear_db_kernel, (unsigned)(((int64_t)G * N + 31) / 32),
                                      32 * DB_SLICES, 0, 1, stream, dba, G, N));
    }
    // for fp32 gradients dz is a stack of planes
    const auto map_dz = [&](CUtensorMap *m, int box_rows) {
        return g32 ? map_w(m, dz, halves, c->rows, N, ld_dz, box_rows)
                   : map2d(m, dz, c->rows, N, ld_dz, box_rows);
    };
    CUtensorMap xa, xb, wa, wb;
    if (dx && (map_w(&xa, w, G, N, Kin, c->ld_w, 64) != cudaSuccess ||
               map_dz(&xb, 32) != cudaSuccess))
        return MOK_ERR_CUDA;
    if (dw && (map2d(&wa, x, c->rows, Kin, c->ld_in, 64) != cudaSuccess ||
               map_dz(&wb, 64) != cudaSuccess))
        return MOK_ERR_CUDA;
    const int n_nb = (N + 255) / 256;
    const int64_t x_units = dx ? tiles.cap * n_kb * xc.parts : 0;
    const int64_t w_units = dw ? (int64_t)G * n_kb * n_nb * wc.parts : 0;
    const int32_t *valid = grouped(starts) ? wk.valid : nullptr;
    int64_t split = 0, pairs = 0;  // pairs of SMs for dW, and in all, where both go in one launch
    if (dx && dw && !grouped(starts))
        plan_both(w_units, unit_clocks((wc.parts > 1 ? wc.per : (c->rows + 63) / 64) * halves, LTILE),
                  x_units, unit_clocks((xc.parts > 1 ? xc.per : (N + 63) / 64) * halves, tiles.height),
                  &split, &pairs);
    DbArgs dwb = dba;
    if (!db_in_dw) dwb.db = nullptr;
#define MOK_BWD(F, CUT)                                                                         \
    do {                                                                                        \
        const Dx<F, CUT> px{tiles, n_kb, halves, Kin, N, c->ld_in, dx, status, xk};                       \
        const Dw<F, CUT> pw{starts, valid, c->rows, G, n_kb, n_nb, halves, Kin, N, c->ld_w, dw, status, dwb, \
                        wkp};                                                                   \
        if (split > 0) {                                                                        \
            MOK_OP_LAUNCH(OP_LINEAR_DX, 1,                                                      \
                          launch_both(wa, wb, pw, xa, xb, px, split, pairs, stream));           \
        } else {                                                                                \
            if (dx) MOK_OP_LAUNCH(OP_LINEAR_DX, 1, launch_linear(xa, xb, px, x_units, stream)); \
            if (dw) MOK_OP_LAUNCH(OP_LINEAR_DW, 1, launch_linear(wa, wb, pw, w_units, stream)); \
        }                                                                                       \
    } while (0)
    const bool cut = xc.parts > 1 || wc.parts > 1;
    if (g32 && cut) MOK_BWD(true, true);
    else if (g32) MOK_BWD(true, false);
    else if (cut) MOK_BWD(false, true);
    else MOK_BWD(false, false);
#undef MOK_BWD
    JoinArgs j = {};
    int n = 0;
    if (dx && xc.parts > 1) j.o[n++] = join_out(xk, c->rows, Kin, dx, c->ld_in);
    if (dw && wc.parts > 1) j.o[n++] = join_out(wkp, N, Kin, dw, c->ld_w);
    if (n > 0) MOK_OP_LAUNCH(dx ? OP_LINEAR_DX : OP_LINEAR_DW, 1, launch_join(g32, j, stream));
    return MOK_OK;
}

}  // extern "C"

// vocab_loss.cu -- softmax cross entropy over the projection of rows on a vocabulary, and its
// gradients, without the logits in memory.
//
//   forward   l = x W^T, lse = log sum_v exp(l_v), loss = lse - l_target + z lse^2
//   backward  dl_v = d ((1 + 2 z lse) exp(l_v - lse) - [v == target]), dx = dl W, dW = dl^T x
//
// The products run on the linear layer's engine (linear_core.cuh): pairs of SMs, operands by TMA,
// accumulators in TMEM.
//   VocabFwd  A = x, B = W, so a TMEM lane is a row and a thread takes the maximum and the sum of
//             exponentials of its row's columns without talking to others; each tile of 256 vocabulary
//             entries leaves a (maximum, sum) per row and warp, and a second kernel joins them in
//             order.
//   VocabFew  a few rows: A = W, B = x, so no tile is mostly padding (with 4 rows of x on M an SM
//             writes as many zeros to shared memory as it loads of W). A lane is a vocabulary
//             entry and keeps each row's maximum and sum from tile to tile; lanes are joined at the end.
//   VocabDl   A = W, B = x, as the linear layer's forward, with dl for an epilogue: bf16 rows of a
//             piece of the vocabulary in the workspace.
//   dx, dW    the linear layer's gradient products, with dl for dz.
#include "linear_core.cuh"

namespace mok {
namespace {

constexpr float LOG2E_F = 1.4426950408889634f, LN2_F = 0.6931471805599453f;
constexpr float LOWEST = -3.0e38f;  // below any logit; differences with it stay finite or -inf

// Running maximum and sum of exponentials, in powers of two.
struct MaxSum {
    float m, s;
    MOK_DEV void join(const MaxSum &o) {
        const float t = fmaxf(m, o.m);
        s = s * exp2_hw((m - t) * LOG2E_F) + o.s * exp2_hw((o.m - t) * LOG2E_F);
        m = t;
    }
};

// ---------------------------------------------------------------- forward
// SEGS: H in segments that are added in registers; else the sums are in TMEM whole.
template <bool SEGS>
struct VocabFwd {
    using E = Epi<true>;
    static constexpr bool F32_OUT = true, SUMS = SEGS, A_MN = false, B_MN = false;
    static constexpr int BAND = 16;  // row blocks that take a tile of W one after another: 4096
                                     // rows of x stay in L2 while W passes by
    int64_t rows;
    int n_rb, n_vt;   // row blocks and vocabulary tiles of 256
    int segs;         // of H
    int H, V;
    const int32_t *targets;
    float2 *part;     // [4 n_vt][rows]: (maximum, sum) of a warp's columns of a tile
    float *hit;       // [rows]: the target's logit
    int *status;

    MOK_DEV int64_t n_units() const { return (int64_t)n_rb * n_vt; }
    MOK_DEV void side_work(uint32_t, uint32_t, int) const {}
    MOK_DEV Unit unit(uint32_t u) const {
        const uint32_t per = (uint32_t)BAND * (uint32_t)n_vt, band = u / per, rest = u - band * per;
        const uint32_t left = (uint32_t)n_rb - band * BAND, nb = left < BAND ? left : BAND;
        return Unit{0, 0, 0, 0, (int)(band * BAND + rest % nb), (int)(rest / nb), 0};
    }
    MOK_DEV int segments(const Unit &) const { return segs; }
    MOK_DEV int long_steps(const Unit &) const { return 0; }
    MOK_DEV int cols(const Unit &u) const {
        const int left = V - u.nb * 256;
        return left < 256 ? left : 256;
    }
    MOK_DEV LinGeom geom(const Unit &u, int seg, uint32_t rank) const {
        LinGeom q;
        q.n_mma = (cols(u) + 15) & ~15;
        q.a0 = seg * SEG_K;
        q.a1 = u.mb * 256 + (int)rank * 128;
        q.a2 = 0;
        q.b0 = q.a0;
        q.b1 = u.nb * 256 + (int)rank * (q.n_mma / 2);
        q.nbox = (q.n_mma / 2 + 31) / 32;
        const int k = H - q.a0 > SEG_K ? SEG_K : H - q.a0;
        q.k_steps = (k + 15) / 16;
        q.k_first = q.half = 0;
        return q;
    }
    MOK_DEV uint32_t tx(const LinGeom &q) const { return 2 * BOX + q.nbox * (BOX / 2); }
    MOK_DEV void load(uint8_t *st, uint32_t fb, const LinGeom &q, int k0, const CUtensorMap *tmA,
                      const CUtensorMap *tmB) const {
        tma_load_3d_pair(st, tmA, fb, q.a0 + k0, q.a1, q.a2);
        for (int j = 0; j < q.nbox; ++j)
            tc::tma_load_2d_pair(st + 2 * BOX + j * (BOX / 2), tmB, fb, q.b0 + k0, q.b1 + 32 * j);
    }
    // columns n0 .. n0 + N - 1 of a tile, those below `n` of the vocabulary
    template <int N>
    MOK_DEV void take(MaxSum &a, int n0, int n, const float (&v)[N], int target, int64_t row) const {
        const bool whole = N > 16 && n0 + N <= n;  // (registers are short among segments)
        float t = a.m;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (whole || n0 + j < n) t = fmaxf(t, v[j]);
        a.s *= exp2_hw((a.m - t) * LOG2E_F);
        a.m = t;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (whole || n0 + j < n) a.s += exp2_hw((v[j] - t) * LOG2E_F);
        if (target >= n0 && target < n0 + N) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (target == n0 + j && n0 + j < n) hit[row] = v[j];
        }
    }
    MOK_DEV void epilogue(const Unit &u, int seg, bool last, uint32_t rank, uint32_t c, int q, int hw,
                          int lane, Patches &, Carry<SEGS> &carry) const {
        const int64_t row = (int64_t)u.mb * 256 + rank * 128 + q * 32 + lane;
        const int n = cols(u);
        MaxSum a{LOWEST, 0.0f};
        int target = -1;  // in the tile, where it is not below it
        if (last && row < rows) target = targets[row];
        target = target >= u.nb * 256 ? target - u.nb * 256 : -1;
        if constexpr (SEGS) {
            sum_segments(c, hw, n, seg == 0, last, carry, [&](int n0, const float (&v)[16]) {
                take(a, n0, n, v, target, row);
            });
        } else {
            for (int n0 = 32 * hw; n0 < n; n0 += 128) {
                float v[32];
                ld32(c + n0, v);
                take(a, n0, n, v, target, row);
            }
        }
        if (last && row < rows) part[((int64_t)u.nb * 4 + hw) * rows + row] = make_float2(a.m, a.s);
    }
};

// up to 64 rows: a warp takes 16 of them, four warps a TMEM lane quadrant
constexpr int FEW_ROWS = 64;
struct VocabFew {
    using E = Epi<true>;
    static constexpr bool F32_OUT = true, A_MN = false, B_MN = false;
    struct State {
        float v[16];      // the segments of H so far
        MaxSum a[16];
    };
    int rows, n_vt;
    int segs;
    int H, V;
    const int32_t *targets;
    float2 *part;     // [8 clusters][rows]
    float *hit;
    int *status;

    MOK_DEV int64_t n_units() const { return n_vt; }
    MOK_DEV void side_work(uint32_t, uint32_t, int) const {}
    MOK_DEV Unit unit(uint32_t u) const { return Unit{0, 0, rows, 0, (int)u, 0, 0}; }
    MOK_DEV int segments(const Unit &) const { return segs; }
    MOK_DEV int long_steps(const Unit &) const { return 0; }
    MOK_DEV LinGeom geom(const Unit &u, int seg, uint32_t rank) const {
        LinGeom q;
        q.n_mma = (rows + 15) & ~15;
        q.a0 = seg * SEG_K;
        q.a1 = u.mb * 256 + (int)rank * 128;
        q.a2 = 0;
        q.b0 = q.a0;
        q.b1 = (int)rank * (q.n_mma / 2);
        q.nbox = (q.n_mma / 2 + 31) / 32;
        const int k = H - q.a0 > SEG_K ? SEG_K : H - q.a0;
        q.k_steps = (k + 15) / 16;
        q.k_first = q.half = 0;
        return q;
    }
    MOK_DEV uint32_t tx(const LinGeom &q) const { return 2 * BOX + q.nbox * (BOX / 2); }
    MOK_DEV void load(uint8_t *st, uint32_t fb, const LinGeom &q, int k0, const CUtensorMap *tmA,
                      const CUtensorMap *tmB) const {
        tma_load_3d_pair(st, tmA, fb, q.a0 + k0, q.a1, q.a2);
        for (int j = 0; j < q.nbox; ++j)
            tc::tma_load_2d_pair(st + 2 * BOX + j * (BOX / 2), tmB, fb, q.b0 + k0, q.b1 + 32 * j);
    }
    MOK_DEV void start(State &k) const {
#pragma unroll
        for (int j = 0; j < 16; ++j) k.a[j] = MaxSum{LOWEST, 0.0f};
    }
    MOK_DEV void epilogue(const Unit &u, int seg, bool last, uint32_t rank, uint32_t c, int q, int hw,
                          int lane, Patches &, State &k) const {
        const int r0 = 16 * hw;
        if (r0 >= rows) return;
        float v[16];
        tc::tmem_ld16(c + r0, v);
        tc::tmem_ld_wait();
        loaded(v);
#pragma unroll
        for (int j = 0; j < 16; ++j) k.v[j] = seg > 0 ? k.v[j] + v[j] : v[j];
        const int f = u.mb * 256 + (int)rank * 128 + q * 32 + lane;
        if (!last || f >= V) return;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            if (r0 + j >= rows) continue;
            MaxSum &a = k.a[j];
            const float t = fmaxf(a.m, k.v[j]);
            a.s = a.s * exp2_hw((a.m - t) * LOG2E_F) + exp2_hw((k.v[j] - t) * LOG2E_F);
            a.m = t;
            if (targets[r0 + j] == f) hit[r0 + j] = k.v[j];
        }
    }
    MOK_DEV void finish(State &k, uint32_t cluster, uint32_t rank, int q, int hw, int lane) const {
        const int r0 = 16 * hw;
        if (r0 >= rows) return;
        const int64_t p = (int64_t)(cluster * 2 + rank) * 4 + q;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            MaxSum a = k.a[j];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                a.join(MaxSum{__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o)});
            if (lane == 0 && r0 + j < rows) part[p * rows + r0 + j] = make_float2(a.m, a.s);
        }
    }
};

// A block joins the parts of up to 32 rows: `across` lanes (a power of two) on rows, the other lanes and
// the warps on slices of the parts (with one row a part a lane), then lanes and warps by halves.
constexpr int FINISH_WARPS = 32;
__global__ void __launch_bounds__(32 * FINISH_WARPS)
    vocab_finish_kernel(const float2 *part, const float *hit, int64_t rows, int across, int parts,
                        int V, const int32_t *targets, float z, float *loss, float *lse, int *status) {
    __shared__ float2 sh[FINISH_WARPS][32];
    let_next_start();
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row0 = (int64_t)blockIdx.x * across, row = row0 + lane % across;
    const int slices = FINISH_WARPS * (32 / across);
    MaxSum a{LOWEST, 0.0f};
    // a batch of loads at a time, the last one too
    for (int p0 = warp * (32 / across) + lane / across; p0 < parts; p0 += 8 * slices) {
        float2 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int p = p0 + k * slices;
            v[k] = make_float2(LOWEST, 0.0f);
            if (p < parts && row < rows) v[k] = part[(int64_t)p * rows + row];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) a.join(MaxSum{v[k].x, v[k].y});
    }
    for (int o = 16; o >= across; o >>= 1)
        a.join(MaxSum{__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o)});
    sh[warp][lane] = make_float2(a.m, a.s);
    __syncthreads();
    // warp w joins the warps' values of row w
    const int64_t r = row0 + warp;
    if (warp >= across || r >= rows) return;
    a = MaxSum{sh[lane][warp].x, sh[lane][warp].y};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        a.join(MaxSum{__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o)});
    if (lane != 0) return;
    const float l = a.m + log2f(a.s) * LN2_F;
    lse[r] = l;
    const int t = targets[r];
    if (t >= V) raise_status(status, MOK_ERR_DEVICE_INVARIANT);
    if (loss != nullptr) loss[r] = t >= 0 && t < V ? (l - hit[r]) + z * l * l : 0.0f;
}

// ---------------------------------------------------------------- backward
// what dl needs of a row
struct alignas(16) RowGrad {
    float lse, p;    // p: d (1 + 2 z lse), the factor of the probabilities
    float d;
    int32_t target;  // -1: the row takes no part
};

__global__ void vocab_rows_kernel(const float *lse, const float *d_loss, const int32_t *targets,
                                  int64_t rows, int V, float z, RowGrad *out, int *status) {
    let_next_start();
    wait_for_previous();
    const int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (r >= rows) return;
    const int t = targets[r];
    if (t >= V) raise_status(status, MOK_ERR_DEVICE_INVARIANT);
    const bool in = t >= 0 && t < V;
    const float l = lse[r], d = in ? d_loss[r] : 0.0f;
    out[r] = RowGrad{l, in ? d * fmaf(2.0f * z, l, 1.0f) : 0.0f, d, in ? t : -1};
}

// x for the product of dW, zeros in the rows that take no part: their dl is zero, but nothing says that x is
// finite there, and zero times infinity would reach all of dW. 8192 x 4096 20 us, beside 10 ms of products.
// `copies` of them, one below the other.
__global__ void __launch_bounds__(256)
    vocab_live_kernel(const uint16_t *x, int64_t ld, const int32_t *targets, int64_t rows, int copies,
                      int H, int V, uint16_t *out, int64_t ld_out) {
    let_next_start();
    wait_for_previous();
    const int64_t per = ld_out / 8, n = rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per;
        const int c = (int)(i - r * per) * 8, t = targets[r];
        uint4 v = make_uint4(0, 0, 0, 0);
        if (t >= 0 && t < V) {
            const uint16_t *p = x + r * ld + c;
            if (c + 8 <= H) {
                v = ld_v4(p);
            } else {
                uint32_t e[4] = {0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < H) e[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
                v = make_uint4(e[0], e[1], e[2], e[3]);
            }
        }
        for (int k = 0; k < copies; ++k) *reinterpret_cast<uint4 *>(out + (k * rows + r) * ld_out + c) = v;
    }
}

// EXACT: the exponent's own rounding, half a unit of some 17, is put right to first order
template <bool EXACT>
MOK_DEV float dl_of(const RowGrad &g, float l, int v) {
    const float x = l - g.lse, t = x * LOG2E_F;
    float e = exp2_hw(t);
    if (EXACT) {
        constexpr float LOG2E_REST = 1.925963033500749e-8f;  // log2 e - LOG2E_F
        const float rest = fmaf(x, LOG2E_F, -t) + x * LOG2E_REST;
        if (rest == rest) e = fmaf(e * LN2_F, rest, e);  // not where x is infinite
    }
    const float p = g.p * e;
    return g.target < 0 ? 0.0f : v == g.target ? p - g.d : p;
}

// bf16 planes that dl comes in for fp32 gradients: each takes what the ones before it leave. Two
// would do as for the linear layer's dz (rms 2.7e-6 of it), but dl has no rounding of its own that
// this would hide behind. Gradients of 1001 rows, 1000 x 5003, are 2.7e-6 of their norm off with two
// and 1.2e-6 with three; plain fp32 products 1.3e-6 (dx) and 5.4e-7 (dW).
constexpr int PLANES = 3;
// and what the tensor cores sum of them at a time: their error grows with a run's length (see Fwd in
// linear.cu). Runs of 512, with the exponent's rounding put right in dl, 7.0e-7 and 6.9e-7 (3% slower
// than runs of 1024)
constexpr int GRAD_RUN = 512;

// Rows up to which bf16 gradients take two planes too, as rows of their own: dl is then twice as many rows,
// with x twice for dW, and dx the sum of its two halves. A row's gradient is for the most part its target's
// entry, so rounding that one entry to bf16 scales all of it, by up to 2^-8, whatever the other rows are: with
// one plane any number of rows is 2.3e-3 of the norm off where rounding the outputs alone is 1.7e-3, and few rows may be
// 2.5e-3. The bound is one of cost: two planes are half again the products of many rows, and little beside W's bytes and
// the launches of few.
// One plane against two, us: 3 rows, 45 x 11962 15 / 18; 4, 4096 x 131072 601 / 605; 64, 4096 x 32000 170 /
// 165; 256 185 / 228; 512 255 / 421.
constexpr int TWICE_ROWS = 512;

// Elements of H that the logits of bf16 gradients are summed over at a time. A tensor-core sum loses up to
// 2^-23 of what it has so far with every 16 terms, so a run of n terms of one sign n / 32 of that: 2^-16 of
// a logit with runs of 4096, while one of 2^18 may lose 2^-10: 0.3 of a logit of 300, 30% of its dl. Gradients
// of 4096 rows, 8192 x 32768, 3803 us with runs of 4096, 3787 with one, 3980 with runs of 1024 (the sums leave
// TMEM more often); 600 rows, 8192 x 32000, 760, 737 and 793; 16 rows 327, 324 and 328.
constexpr int BF16_RUN = 4096;
// ... and of fp32 gradients: 512, as many as GRAD_RUN, or all of H up to SEG_K where dl has many entries. A logit's
// error reaches the probabilities alone, which are the less of a row's dl the more entries share them, and sums in
// segments leave TMEM through fp32 stores of their own: 1001 rows, 1000 x 5003, 108 us and 7.2e-7 in one run, 124 us
// and 6.8e-7 in two. 2000 rows, 1000 x 64: 53 us, 1.4e-6 and 60 us, 8.4e-7; 6251 rows, 1044 x 90, with runs of 1024
// 99 us, 1.5e-6, of 512 99 us, 9.3e-7; 4096 rows, 4096 x 4096 651 and 657 us.
constexpr int F32_RUN = 512, F32_FEW = 512;
int dl_run(const mok_vocab_loss_config &c) {
    if (c.grad_dtype != MOK_DTYPE_F32) return BF16_RUN;
    return c.H <= SEG_K && c.V > F32_FEW ? SEG_K : F32_RUN;
}

// The gradient of the logits for vocabulary entries [v0, v0 + N), in N_PLANES planes of bf16. SEGS: of
// logits whose segments of H were added in fp32. Row tiles come first:
// a band of 4096 rows of x stays in L2 while W passes by once (the other way round W passes by for
// every tile, 4096 rows, 4096 x 65536: 1450 against 1200 us under the profiler).
template <int N_PLANES, bool SEGS>
struct VocabDl {
    using E = Epi<SEGS>;
    static constexpr bool F32_OUT = SEGS, SUMS = SEGS, A_MN = false, B_MN = false;
    Tiles tiles;
    int band;        // tiles that take a block of W one after another
    int n_mb;        // ceil(N / 256)
    int segs, run;   // of H, and their elements
    int H, v0, N;
    const RowGrad *rows;
    uint16_t *dl;
    int64_t ld, plane;
    int *status;

    MOK_DEV int64_t n_units() const { return tiles.count() * n_mb; }
    MOK_DEV void side_work(uint32_t, uint32_t, int) const {}
    MOK_DEV Unit unit(uint32_t u) const {
        const uint32_t per = (uint32_t)band * (uint32_t)n_mb, b = u / per, rest = u - b * per;
        const uint32_t left = (uint32_t)tiles.cap - b * band, nt = left < (uint32_t)band ? left : band;
        const int4 t = tiles.get(b * band + rest % nt);
        return Unit{0, t.y, t.z - t.y, 0, (int)(rest / nt), 0, 0};
    }
    MOK_DEV int segments(const Unit &) const { return segs; }
    MOK_DEV int long_steps(const Unit &) const { return 0; }
    MOK_DEV LinGeom geom(const Unit &u, int seg, uint32_t rank) const {
        LinGeom q;
        q.n_mma = (u.nr + 15) & ~15;
        q.a0 = seg * run;
        q.a1 = v0 + u.mb * 256 + (int)rank * 128;
        q.a2 = 0;
        q.b0 = q.a0;
        q.b1 = u.r0 + (int)rank * (q.n_mma / 2);
        q.nbox = (q.n_mma / 2 + 31) / 32;
        const int k = H - q.a0 > run ? run : H - q.a0;
        q.k_steps = (k + 15) / 16;
        q.k_first = q.half = 0;
        return q;
    }
    MOK_DEV uint32_t tx(const LinGeom &q) const { return 2 * BOX + q.nbox * (BOX / 2); }
    MOK_DEV void load(uint8_t *st, uint32_t fb, const LinGeom &q, int k0, const CUtensorMap *tmA,
                      const CUtensorMap *tmB) const {
        tma_load_3d_pair(st, tmA, fb, q.a0 + k0, q.a1, q.a2);
        for (int j = 0; j < q.nbox; ++j)
            tc::tma_load_2d_pair(st + 2 * BOX + j * (BOX / 2), tmB, fb, q.b0 + k0, q.b1 + 32 * j);
    }
    MOK_DEV void epilogue(const Unit &u, int seg, bool last, uint32_t rank, uint32_t c, int q, int hw,
                          int lane, Patches &pt, Carry<SUMS> &carry) const {
        const int64_t r0 = u.r0;
        const int f0 = u.mb * 256 + (int)rank * 128 + q * 32;  // the warp's entries of the piece
        if constexpr (SEGS) {
            const int f = f0 + lane;
            sum_segments(c, hw, u.nr, seg == 0, last, carry, [&](int n0, const float (&v)[16]) {
                if (f >= N) return;
                uint16_t *p = dl + (r0 + n0) * ld + f;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    if (n0 + j >= u.nr) continue;
                    float g = dl_of<(N_PLANES > 1)>(rows[r0 + n0 + j], v[j], v0 + f);
#pragma unroll
                    for (int k = 0; k < N_PLANES; ++k) {
                        const uint16_t b = f32_to_bf16(g);
                        p[k * plane + j * ld] = b;
                        g = isfinite(bf16_to_f32(b)) ? g - bf16_to_f32(b) : 0.0f;
                    }
                }
            });
        } else {
            for (int n0 = 32 * hw; n0 < u.nr; n0 += E::STEP) {
                // 32 rows: what they need first, so that its latency and the columns' run together
                RowGrad g[4][2];
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int n = n0 + 8 * b + 2 * (lane & 3) + i;
                        g[b][i] = rows[r0 + (n < u.nr ? n : u.nr - 1)];
                    }
                float w[2][4][4], v[4][2][4];
                ld_pairs(c + n0, w);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[b][h][i] = dl_of<(N_PLANES > 1)>(g[b][i & 1], w[h][b][i],
                                               v0 + f0 + 16 * h + 8 * (i >> 1) + (lane >> 2));
                    patch_write8(pt.patch(), pt.half, b, v[b], lane);
                }
                pt.store(OutRef{dl, tiles.rows, ld, N}, f0 & ~63, r0 + n0, r0 + u.nr, 0);
#pragma unroll
                for (int k = 1; k < N_PLANES; ++k) {
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float &g = v[b][i >> 2][i & 3];
                            const float r = bf16_to_f32(f32_to_bf16(g));
                            g = isfinite(r) ? g - r : 0.0f;
                        }
                        patch_write8(pt.patch(), pt.half, b, v[b], lane);
                    }
                    pt.store(OutRef{dl + k * plane, tiles.rows, ld, N}, f0 & ~63, r0 + n0, r0 + u.nr, 0);
                }
            }
        }
    }
};

// dx of several pieces, or of dl's two planes (`copies` 2), from fp32 sums
__global__ void __launch_bounds__(256)
    vocab_round_kernel(const float *sum, int64_t ld_sum, int64_t rows, int copies, int H, uint16_t *dx,
                       int64_t ld) {
    let_next_start();
    wait_for_previous();
    const int64_t n = rows * (ld_sum / 4);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / (ld_sum / 4);
        const int c = (int)(i - r * (ld_sum / 4)) * 4;
        float4 v = *reinterpret_cast<const float4 *>(sum + r * ld_sum + c);
        if (copies == 2) {
            const float4 u = *reinterpret_cast<const float4 *>(sum + (rows + r) * ld_sum + c);
            v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
        }
        uint16_t *p = dx + r * ld + c;
        if (c + 4 <= H) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
        } else {
            const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < H) p[j] = f32_to_bf16(e[j]);
        }
    }
}

// ---------------------------------------------------------------- host side
constexpr int64_t DL_BYTES = (int64_t)1 << 30;  // of a piece's dl, where the caller does not say

struct VocabWs {
    float2 *part;
    float *hit;
    RowGrad *rows;
    uint16_t *dl;
    uint16_t *x;      // of the rows that take part
    int64_t ld_x;
    float *dx_sum;
    GradPlan plan;    // of the gradient products, where the vocabulary is one piece
    void *grads;      // their parts
    int planes, copies;  // of dl; of the rows, as the gradient products take them
    int clusters;     // of a few rows' forward
    int piece, pieces;
    int64_t ld_dl;
};

size_t carve_vocab(const mok_vocab_loss_config &c, int pass, void *ws, VocabWs *o) {
    size_t off = 0;
    const auto take = [&](size_t bytes) {
        off = (size_t)round_up((int64_t)off, 256);
        void *p = ws != nullptr ? (char *)ws + off : nullptr;
        off += bytes;
        return p;
    };
    VocabWs w = {};
    if (pass == MOK_VOCAB_LOSS_FORWARD) {
        const int n_vt = (c.V + 255) / 256;
        w.clusters = n_vt < PLAN_PAIRS ? n_vt : (int)PLAN_PAIRS;
        w.part = (float2 *)take((size_t)c.rows * (c.rows <= FEW_ROWS ? 8 * w.clusters : 4 * n_vt) * 8);
        w.hit = (float *)take((size_t)c.rows * 4);
    } else {
        const bool f32 = c.grad_dtype == MOK_DTYPE_F32;
        const int64_t copies = !f32 && c.rows <= TWICE_ROWS ? 2 : 1, planes = f32 ? PLANES : copies;
        w.planes = (int)planes;
        w.copies = (int)copies;
        const int64_t all = round_up(c.V, 256), row = 2 * planes * (c.rows > 0 ? c.rows : 1);
        int64_t piece = c.piece;
        if (piece == 0) {
            int64_t most = DL_BYTES / row / 256 * 256;
            if (most < 256) most = 256;
            const int64_t n = (all + most - 1) / most;
            piece = round_up((c.V + n - 1) / n, 256);
        }
        if (piece > all) piece = all;
        w.piece = (int)piece;
        w.pieces = (int)((c.V + piece - 1) / piece);
        w.ld_dl = w.pieces > 1 ? piece : round_up(c.V, 8);
        w.rows = (RowGrad *)take((size_t)c.rows * sizeof(RowGrad));
        w.dl = (uint16_t *)take((size_t)planes * c.rows * w.ld_dl * 2);
        w.ld_x = round_up(c.H, 8);
        w.x = (uint16_t *)take((size_t)copies * c.rows * w.ld_x * 2);
        if (!f32 && (w.pieces > 1 || copies > 1))
            w.dx_sum = (float *)take((size_t)copies * c.rows * round_up(c.H, 4) * 4);
        if (w.pieces == 1) {
            w.plan = plan_dense_grads(copies * c.rows, c.V, c.H, f32 ? PLANES : 1, true);
            w.grads = take(dense_grads_bytes(w.plan, copies * c.rows, c.V, c.H));
        }
    }
    if (o != nullptr) *o = w;
    return off > 0 ? off : 256;
}

// Rows of dl's tiles: as waves over the SM pairs, each as long as its loads and MMAs or its epilogue
// (about 6000 clocks for 256 rows, 15000 with planes), and a first load and a last epilogue alone.
int dl_height(int64_t rows, int64_t n_mb, int H, bool planes) {
    const int64_t blocks = (H + BK - 1) / BK, pairs = sm_pairs();
    int64_t best = INT64_MAX, best_h = LTILE;
    for (int64_t h0 = LTILE; h0 >= 32; h0 -= 16) {
        const int64_t n = (rows + h0 - 1) / h0, h = round_up((rows + n - 1) / n, 16);
        const int64_t main = blocks * block_clocks(h), epi = (planes ? 15000 : 6000) * h / LTILE;
        const int64_t waves = (n * n_mb + pairs - 1) / pairs;
        const int64_t t = (waves - 1) * (main > epi ? main : epi) + main + epi;
        if (t < best) {
            best = t;
            best_h = h;
        }
    }
    return (int)best_h;
}

mok_status check_vocab(const mok_vocab_loss_config *c, int pass, void *ws, size_t ws_bytes,
                       int **status, VocabWs *w) {
    mok_status st = mok_check_vocab_loss_config(c);
    if (st != MOK_OK) return st;
    if ((st = current_device_status_word(status)) != MOK_OK) return st;
    if (carve_vocab(*c, pass, ws, w) > ws_bytes || ws == nullptr || ((uintptr_t)ws & 255u) != 0)
        return MOK_ERR_WORKSPACE;
    return MOK_OK;
}

}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

mok_status mok_check_vocab_loss_config(const mok_vocab_loss_config *c) {
    if (c == nullptr) return MOK_ERR_INVALID_ARG;
    if (c->abi_version != MOK_ABI_VERSION) return MOK_ERR_ABI;
    if (c->H < 1 || c->H > (1 << 20) || c->V < 1 || c->V > (1 << 24)) return MOK_ERR_INVALID_ARG;
    if (c->rows < 0 || c->rows >= ((int64_t)1 << 31) - 512) return MOK_ERR_INVALID_ARG;
    const int64_t lds[] = {c->ld_x, c->ld_w};
    for (int64_t ld : lds)
        if (ld < c->H || ld % 8 != 0 || ld > ((int64_t)1 << 30)) return MOK_ERR_INVALID_ARG;
    // units of the products are numbered in 31 bits
    const int64_t tiles = c->rows / 16 + 1, vb = (c->V + 255) / 256, hb = (c->H + 255) / 256;
    if (tiles * vb > INT32_MAX || tiles * hb > INT32_MAX || vb * 16 * hb > INT32_MAX)
        return MOK_ERR_INVALID_ARG;
    if (c->grad_dtype != MOK_DTYPE_BF16 && c->grad_dtype != MOK_DTYPE_F32) return MOK_ERR_INVALID_ARG;
    if (!(c->z_loss >= 0.0f && c->z_loss <= 3.402823466e38f)) return MOK_ERR_INVALID_ARG;
    if (c->piece < 0 || c->piece % 256 != 0) return MOK_ERR_INVALID_ARG;
    return MOK_OK;
}

size_t mok_vocab_loss_workspace_size(const mok_vocab_loss_config *c, int pass) {
    if (mok_check_vocab_loss_config(c) != MOK_OK) return 0;
    if (pass != MOK_VOCAB_LOSS_FORWARD && pass != MOK_VOCAB_LOSS_BACKWARD) return 0;
    return carve_vocab(*c, pass, nullptr, nullptr);
}

mok_status mok_vocab_loss_forward(const mok_vocab_loss_config *c, const void *x, const void *w,
                                  const int32_t *targets, float *loss, float *lse, void *ws,
                                  size_t ws_bytes, cudaStream_t stream) {
    int *status;
    VocabWs wk;
    mok_status st = check_vocab(c, MOK_VOCAB_LOSS_FORWARD, ws, ws_bytes, &status, &wk);
    if (st != MOK_OK) return st;
    if (c->rows == 0) return MOK_OK;
    if (!x || !w || !targets || !lse) return MOK_ERR_INVALID_ARG;
    const void *ps[] = {x, w, targets, loss, lse};
    for (const void *p : ps)
        if (p && !op_aligned16(p)) return MOK_ERR_INVALID_ARG;
    if (init_host() != cudaSuccess) return MOK_ERR_CUDA;
    CUtensorMap ma, mb;
    const int n_rb = (int)((c->rows + 255) / 256), n_vt = (c->V + 255) / 256;
    const int segs = (c->H + SEG_K - 1) / SEG_K;
    int parts = 4 * n_vt;
    if (c->rows <= FEW_ROWS) {
        parts = 8 * wk.clusters;
        if (map_w(&ma, w, 1, c->V, c->H, c->ld_w, 128) != cudaSuccess ||
            map2d(&mb, x, c->rows, c->H, c->ld_x, 32) != cudaSuccess)
            return MOK_ERR_CUDA;
        const VocabFew p{(int)c->rows, n_vt, segs, c->H, c->V, targets, wk.part, wk.hit, status};
        MOK_OP_LAUNCH(OP_VOCAB_FWD, 1, launch_linear(ma, mb, p, n_vt, stream, PLAN_PAIRS));
    } else {
        if (map_w(&ma, x, 1, c->rows, c->H, c->ld_x, 128) != cudaSuccess ||
            map2d(&mb, w, c->V, c->H, c->ld_w, 32) != cudaSuccess)
            return MOK_ERR_CUDA;
        const int64_t units = (int64_t)n_rb * n_vt;
        if (segs > 1) {
            const VocabFwd<true> p{c->rows, n_rb, n_vt, segs, c->H, c->V, targets, wk.part, wk.hit, status};
            MOK_OP_LAUNCH(OP_VOCAB_FWD, 1, launch_linear(ma, mb, p, units, stream));
        } else {
            const VocabFwd<false> p{c->rows, n_rb, n_vt, segs, c->H, c->V, targets, wk.part, wk.hit, status};
            MOK_OP_LAUNCH(OP_VOCAB_FWD, 1, launch_linear(ma, mb, p, units, stream));
        }
    }
    int across = 1;
    while (across < 32 && across < c->rows) across *= 2;
    MOK_OP_LAUNCH(OP_VOCAB_FWD, 1,
                  launch_edge(vocab_finish_kernel, (unsigned)((c->rows + across - 1) / across),
                              32 * FINISH_WARPS, 0, 1, stream, (const float2 *)wk.part,
                              (const float *)wk.hit, c->rows, across, parts, c->V, targets, c->z_loss,
                              loss, lse, status));
    return MOK_OK;
}

mok_status mok_vocab_loss_backward(const mok_vocab_loss_config *c, const void *x, const void *w,
                                   const int32_t *targets, const float *lse, const float *d_loss,
                                   void *dx, void *dw, void *ws, size_t ws_bytes,
                                   cudaStream_t stream) {
    int *status;
    VocabWs wk;
    mok_status st = check_vocab(c, MOK_VOCAB_LOSS_BACKWARD, ws, ws_bytes, &status, &wk);
    if (st != MOK_OK) return st;
    if (!dx && !dw) return MOK_ERR_INVALID_ARG;
    if ((dx && (dx == x || dx == w)) || (dw && (dw == x || dw == w))) return MOK_ERR_INVALID_ARG;
    if (c->rows > 0 && (!x || !w || !targets || !lse || !d_loss)) return MOK_ERR_INVALID_ARG;
    const void *ps[] = {x, w, targets, lse, d_loss, dx, dw};
    for (const void *p : ps)
        if (p && !op_aligned16(p)) return MOK_ERR_INVALID_ARG;
    const bool f32 = c->grad_dtype == MOK_DTYPE_F32;
    const size_t es = f32 ? 4 : 2;
    if (c->rows == 0) {  // sums over nothing
        if (dw && cudaMemset2DAsync(dw, (size_t)c->ld_w * es, 0, (size_t)c->H * es, (size_t)c->V,
                                    stream) != cudaSuccess)
            return MOK_ERR_CUDA;
        return MOK_OK;
    }
    if (init_host() != cudaSuccess) return MOK_ERR_CUDA;
    CUtensorMap ma, mb;
    if (map_w(&ma, w, 1, c->V, c->H, c->ld_w, 128) != cudaSuccess ||
        map2d(&mb, x, c->rows, c->H, c->ld_x, 32) != cudaSuccess)
        return MOK_ERR_CUDA;
    MOK_OP_LAUNCH(OP_VOCAB_DL, 1,
                  launch_edge(vocab_rows_kernel, (unsigned)((c->rows + 255) / 256), 256, 0, 1, stream,
                              lse, d_loss, targets, c->rows, c->V, c->z_loss, wk.rows, status));
    if (dw) {
        const int64_t blocks = (c->rows * (wk.ld_x / 8) + 255) / 256, most = (int64_t)device_sm_count() * 16;
        MOK_OP_LAUNCH(OP_VOCAB_DL, 1,
                      launch_edge(vocab_live_kernel, (unsigned)(blocks < most ? blocks : most), 256, 0, 1,
                                  stream, (const uint16_t *)x, c->ld_x, targets, c->rows, wk.copies,
                                  c->H, c->V, wk.x, wk.ld_x));
    }
    for (int k = 0; k < wk.pieces; ++k) {
        const int v0 = k * wk.piece, n = c->V - v0 < wk.piece ? c->V - v0 : wk.piece;
        const int n_mb = (n + 255) / 256;
        const Tiles tiles = dense_tiles(c->rows, dl_height(c->rows, n_mb, c->H, wk.planes > 1));
        const int band = 4096 / tiles.height;
        const int64_t units = tiles.cap * n_mb, plane = c->rows * wk.ld_dl;
        const int run = dl_run(*c), segs = (c->H + run - 1) / run;
#define MOK_DL(...)                                                                              \
    do {                                                                                         \
        const VocabDl<__VA_ARGS__> p{tiles, band, n_mb, segs, run, c->H, v0, n, wk.rows, wk.dl, wk.ld_dl, \
                                     plane, status};                                             \
        MOK_OP_LAUNCH(OP_VOCAB_DL, 1, launch_linear(ma, mb, p, units, stream));                  \
    } while (0)
        if (segs == 1) {
            if (wk.planes == 1) MOK_DL(1, false);
            else if (wk.planes == 2) MOK_DL(2, false);
            else MOK_DL(PLANES, false);
        } else {
            if (wk.planes == 1) MOK_DL(1, true);
            else if (wk.planes == 2) MOK_DL(2, true);
            else MOK_DL(PLANES, true);
        }
#undef MOK_DL
        const int64_t rows = wk.copies * c->rows;
        const DenseGrads g{wk.x, (const uint16_t *)w + v0 * c->ld_w, wk.dl, rows, n, c->H,
                           f32 ? PLANES : 1, GRAD_RUN, wk.ld_x, c->ld_x, c->ld_w, wk.ld_dl, dx,
                           dw ? (char *)dw + v0 * c->ld_w * es : nullptr, f32,
                           dx ? wk.dx_sum : nullptr, dx && k > 0,
                           wk.pieces == 1 ? wk.plan
                                          : plan_dense_grads(rows, n, c->H, f32 ? PLANES : 1, false),
                           wk.grads};
        int launches = 0;
        MOK_OP_LAUNCH(OP_VOCAB_GRADS, launches, launch_dense_grads(g, status, &launches, stream));
    }
    if (dx && wk.dx_sum != nullptr) {
        const int64_t n = c->rows * (round_up(c->H, 4) / 4), blocks = (n + 255) / 256;
        const int64_t most = (int64_t)device_sm_count() * 32;
        MOK_OP_LAUNCH(OP_VOCAB_GRADS, 1,
                      launch_edge(vocab_round_kernel, (unsigned)(blocks < most ? blocks : most), 256,
                                  0, 1, stream, (const float *)wk.dx_sum, round_up(c->H, 4), c->rows,
                                  wk.copies, c->H, (uint16_t *)dx, c->ld_x));
    }
    return MOK_OK;
}

}  // extern "C"

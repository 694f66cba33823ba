// router.cu -- scores of router logits, choice of experts by score, bias and groups, routing
// weights, loads; the gradient of the logits; the update of the balance bias.
//
//   s = softmax(l) or sigmoid(l), c = s + bias; the K largest c of the kept groups; weights from s
//
// One warp per token, whose logits stay in registers. Each group of experts has a power of two of
// lanes (32 where there is one group), which hold its experts in turn, four at a time where rows
// allow 16-byte loads. The K-th largest of the lanes' largest keys (order-preserving images; K integer
// reductions) is a bound below which no expert is chosen; the few above it go side by side through
// shared memory, one a lane, and count how many are before them. Where ties leave more than a warp
// holds, K rounds take the warp's largest one after another.
// Few experts have a thread a token instead (below).
// What bounds it is the instructions of a warp a token, some 600 for 512 experts: 16384 x 512, top 10,
// 14.9 us (rounds alone: 23.4), floor 5.2; a thread a token would compare 10 values with each of 512.
//
// The choice has to be that of exact scores. fp32 scores are off by a few units in their last place
// (bounds at score_error), so a choice is settled unless two neighbours in the order of the chosen,
// or the last kept and the first other group, are closer than both errors allow. Then 64 bits decide,
// between the experts and groups in question alone, one a lane (64-bit arithmetic is slow here, and
// a launch waits for its slowest token); with a bias and spread logits that is about one token in
// 4000. Only runs of more than 32 close scores take all experts. Experts whose logits and biases are the
// same numbers are ties, not close calls.
#include <type_traits>

#include "ops_internal.h"

namespace mok {
namespace {

constexpr int ROUTER_WARPS = 8;
// Blocks of a SM by the experts a lane holds (the registers' share), and all of them: their loads are
// added in order, so their number is not the device's (with an earlier choice 16384 x 512: 23.4 us in one
// wave, 26.6 in 1.3; 100000 x 60: 50 us at 4 blocks a SM, 75 at 3)
constexpr int per_sm(int held) { return held <= 4 ? 6 : held <= 8 ? 4 : held <= 16 ? 3 : held <= 32 ? 2 : 1; }
constexpr int MAX_E = 1024, MAX_GROUPS = 32;

// order-preserving image of a float; -0 as +0. Everything, NaN of either sign too, maps above 0
MOK_DEV uint32_t order_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return max(u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u), 1u);
}
MOK_DEV float of_order(uint32_t o) {
    return __uint_as_float(o ^ (~(uint32_t)((int32_t)o >> 31) | 0x80000000u));
}
constexpr uint32_t ORDER_MASKED = 0x007FFFFFu;  // of -inf

MOK_DEV float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
MOK_DEV float warp_max(float v) {
    return of_order(__reduce_max_sync(0xFFFFFFFFu, order_of(v)));
}

struct RouterShape {
    int64_t T, ld;
    int E, K, G, keep, top;
    int per, lanes;  // experts and lanes of a group
    bool softmax, renorm;
    float scale;
};

// Which experts a lane holds, VEC consecutive ones at a time: number j is first + (j / VEC) step +
// j % VEC, for j < n (n is a multiple of VEC); and its group.
template <int VEC>
struct Held {
    int first, step, n, g;
    MOK_DEV Held(const RouterShape &c, int lane) {
        const int i = VEC * (lane % c.lanes);
        g = lane / c.lanes;
        first = g * c.per + i;
        step = VEC * c.lanes;
        n = g < c.G && i < c.per ? (c.per - i + step - 1) / step * VEC : 0;
    }
    MOK_DEV int id(int j) const { return first + j / VEC * step + j % VEC; }
};

template <bool BF16>
MOK_DEV float load_logit(const void *row, int e) {
    return BF16 ? bf16_to_f32(static_cast<const uint16_t *>(row)[e])
                : static_cast<const float *>(row)[e];
}
// a lane's logits, -inf past its last
template <int PER, int VEC, bool BF16>
MOK_DEV void load_logits(const void *row, const Held<VEC> &h, float (&v)[PER]) {
#pragma unroll
    for (int j = 0; j < PER; j += VEC) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j + i] = -INFINITY;
        if (j >= h.n) continue;
        const int e = h.id(j);
        if (VEC == 1) {
            v[j] = load_logit<BF16>(row, e);
        } else if (BF16) {
            const uint2 q = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(row) + e);
            v[j] = bf16_lo(q.x);
            v[j + VEC / 4] = bf16_hi(q.x);
            v[j + VEC / 2] = bf16_lo(q.y);
            v[j + VEC - 1] = bf16_hi(q.y);
        } else {
            const float4 q = *reinterpret_cast<const float4 *>(static_cast<const float *>(row) + e);
            v[j] = q.x;
            v[j + VEC / 4] = q.y;
            v[j + VEC / 2] = q.z;
            v[j + VEC - 1] = q.w;
        }
    }
}

// weights are exact to fp32; scores that only order experts or enter sums take the hardware's 2^x
// and reciprocal
MOK_DEV float sigmoid32(float l) { return 1.0f / (1.0f + expf(-l)); }
constexpr float LOG2E_R = 1.4426950408889634f;
MOK_DEV float sigmoid_hw(float l) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + exp2_hw(-LOG2E_R * l)));
    return r;
}
// e^x in softmaxes whose largest x is `top`; -inf gives 0
MOK_DEV float finite_top(float top) { return isinf(top) ? 0.0f : top; }

// The lane's scores of a softmax (v becomes them) and 1 / their sum's e^-top: 0 for a row of -inf
template <int PER>
MOK_DEV float softmax_scores(float (&v)[PER], float &top) {
    top = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) top = fmaxf(top, v[j]);
    top = warp_max(top);
    const float shift = finite_top(top);
    float den = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        v[j] = exp2_hw((v[j] - shift) * LOG2E_R);
        den += v[j];
    }
    den = warp_sum(den);
    const float inv = den > 0.0f ? 1.0f / den : den == 0.0f ? 0.0f : den;
#pragma unroll
    for (int j = 0; j < PER; ++j) v[j] *= inv;
    return inv;
}

// a score as the choice takes it; -inf for a masked expert
MOK_DEV float unbiased_score(const RouterShape &c, float l, float top, float inv) {
    if (l == -INFINITY) return l;
    return c.softmax ? exp2_hw((l - finite_top(top)) * LOG2E_R) * inv : sigmoid_hw(l);
}

// Bound of the error of a score of a row whose largest is `most`. u = 2^-24, x the exponent:
//   sigmoid: 2^x is off by 4u + 1.5 |x| u of itself, which moves s by s (1 - s) times that, at most
//     (1 + 0.34) u; the sum and the reciprocal add s (u + 2u): below 4.5 u. Where s is small that is
//     s (7 + 1.5 |x|) u: 32 u s down to s = u, and less than 32 u^2 below
//   softmax: 2^x by 4u + 1.5 |x| u of itself (|x| e^x <= 0.37), the sum over up to 64 values a lane
//     and 5 steps across lanes 69 u and its terms' own 15 u, the reciprocal and product 2u: below
//     96 u of the largest
MOK_DEV float score_error(const RouterShape &c, float most) {
    constexpr float u = 5.9604644775390625e-8f;
    return c.softmax ? 96.0f * u * most : fminf(4.5f * u, 32.0f * u * (most + u));
}

// order-preserving image of a double that is no NaN, as two words
struct Key64 {
    uint32_t hi, lo;
    MOK_DEV bool operator>(const Key64 &o) const { return hi > o.hi || (hi == o.hi && lo > o.lo); }
};
MOK_DEV Key64 key64(double v) {
    v += 0.0;  // -0 as 0
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint64_t k = (u >> 63) ? ~u : (u | 0x8000000000000000ull);
    return Key64{(uint32_t)(k >> 32), (uint32_t)k};
}
// the warp's largest, of lanes whose key is not 0
MOK_DEV Key64 warp_max(const Key64 &k) {
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, k.hi);
    return Key64{hi, __reduce_max_sync(0xFFFFFFFFu, k.hi == hi ? k.lo : 0u)};
}

// a score in 64 bits; top and den of a softmax
MOK_DEV double score64(const RouterShape &c, float l, double top, double den) {
    return c.softmax ? exp((double)l - top) / den : 1.0 / (1.0 + exp(-(double)l));
}
// the denominator of a softmax in 64 bits
template <int VEC, bool BF16>
MOK_DEV double denominator64(const RouterShape &c, const Held<VEC> &h, const void *row, float top) {
    double den = 0.0;
#pragma unroll 1
    for (int j = 0; j < h.n; ++j) {
        const float l = load_logit<BF16>(row, h.id(j));
        if (l > -INFINITY) den += exp((double)l - (double)top);
    }
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xFFFFFFFFu, den, o);
    return den;
}
// what experts are ordered by in 64 bits; a masked one, or one without a number (of a logit of
// +inf), has to be taken by someone, last
MOK_DEV double order64(float l, double s, const float *bias, int e) {
    const double v = bias != nullptr ? s + (double)bias[e] : (double)l;
    return l > -INFINITY && v == v ? v : -1e300;
}

// The choice between `many` experts, one a lane: lane k < K gets the id of the k-th.
template <int VEC, bool BF16>
__device__ __noinline__ int choose_among(const RouterShape &c, const void *row, const float *bias,
                                         float top, int id, int many, int lane) {
    const Held<VEC> h(c, lane);
    const double den = c.softmax ? denominator64<VEC, BF16>(c, h, row, top) : 1.0;
    const float l = load_logit<BF16>(row, id);
    Key64 k{0u, 0u};
    if (lane < many) k = key64(order64(l, score64(c, l, (double)top, den), bias, id));
    int rank = 0;
    for (int o = 0; o < many; ++o) {
        const Key64 other{__shfl_sync(0xFFFFFFFFu, k.hi, o), __shfl_sync(0xFFFFFFFFu, k.lo, o)};
        const int oid = __shfl_sync(0xFFFFFFFFu, id, o);
        if (other > k || (!(k > other) && oid < id)) ++rank;
    }
    int mine = 0;
    for (int o = 0; o < many; ++o) {
        const int r = __shfl_sync(0xFFFFFFFFu, rank, o), oid = __shfl_sync(0xFFFFFFFFu, id, o);
        if (r == lane) mine = oid;
    }
    return mine;
}

// The choice in 64 bits from all experts of the kept groups: lane k < K gets the k-th expert's id.
template <int PER, int VEC, bool BF16>
__device__ __noinline__ int choose_exact(const RouterShape &c, const void *row, const float *bias,
                                         float top, bool kept, int lane) {
    const Held<VEC> h(c, lane);
    const double den = c.softmax ? denominator64<VEC, BF16>(c, h, row, top) : 1.0;
    Key64 key[PER];
#pragma unroll 1
    for (int j = 0; j < h.n; ++j) {
        const int e = h.id(j);
        const float l = load_logit<BF16>(row, e);
        key[j] = key64(order64(l, score64(c, l, (double)top, den), bias, e));
    }
    int mine = 0;
    uint64_t taken = kept ? 0 : ~0ull;
    for (int k = 0; k < c.K; ++k) {
        Key64 best{0u, 0u};
        int at = 0;
#pragma unroll 1
        for (int j = 0; j < h.n; ++j)
            if (((taken >> j) & 1u) == 0 && key[j] > best) {
                best = key[j];
                at = j;
            }
        const Key64 most = warp_max(best);
        const bool has = best.hi == most.hi && best.lo == most.lo && (best.hi | best.lo) != 0u;
        const uint32_t cand = has ? (uint32_t)h.id(at) : 0xFFFFFFFFu;
        const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, cand);
        if (has && cand == e) taken |= 1ull << at;
        if (lane == k) mine = e < (uint32_t)c.E ? (int)e : 0;
    }
    return mine;
}

// Which groups are kept, in 64 bits, among those too close to the border to tell: `among` of them take
// what the others leave. cand: the experts of a lane that may be one of its group's two largest. True
// for the lanes of a group that is kept.
template <int VEC, bool BF16>
__device__ __noinline__ bool keep_exact(const RouterShape &c, const void *row, const float *bias,
                                        float top, bool among, uint64_t cand, int left, int lane) {
    const Held<VEC> h(c, lane);
    const double den = c.softmax ? denominator64<VEC, BF16>(c, h, row, top) : 1.0;
    double b1 = -INFINITY, b2 = -INFINITY;
    if (!among) cand = 0;
    while (__any_sync(0xFFFFFFFFu, cand != 0)) {  // one a lane at a time, most often one in all
        if (cand == 0) continue;
        const int e = h.id(__ffsll((long long)cand) - 1);
        cand &= cand - 1;
        const float l = load_logit<BF16>(row, e);
        if (!(l > -INFINITY)) continue;
        const double v = score64(c, l, (double)top, den) + (bias != nullptr ? (double)bias[e] : 0.0);
        if (v > b1) {
            b2 = b1;
            b1 = v;
        } else if (v > b2) {
            b2 = v;
        }
    }
    for (int o = 1; o < c.lanes; o <<= 1) {
        const double o1 = __shfl_xor_sync(0xFFFFFFFFu, b1, o);
        const double o2 = __shfl_xor_sync(0xFFFFFFFFu, b2, o);
        const double lo = b1 < o1 ? b1 : o1, hi = b2 > o2 ? b2 : o2;
        b1 = b1 > o1 ? b1 : o1;
        b2 = lo > hi ? lo : hi;
    }
    const Key64 mine = key64(c.top == 2 && b2 > -INFINITY ? b1 + b2 : b1);
    int rank = 0;
    for (int g = 0; g < c.G; ++g) {
        const int from = g * c.lanes;
        const Key64 other{__shfl_sync(0xFFFFFFFFu, mine.hi, from), __shfl_sync(0xFFFFFFFFu, mine.lo, from)};
        const bool in = __shfl_sync(0xFFFFFFFFu, (int)among, from) != 0;
        if (in && (other > mine || (!(mine > other) && g < h.g))) ++rank;
    }
    return among && rank < left;
}

// Unscaled weight of a chosen logit among the K chosen (lane k < K holds the k-th): its score, or
// its share of the chosen scores. The shares of scores that all round to nothing in fp32 are those of
// the scores times e^-t.
MOK_DEV float chosen_weight(const RouterShape &c, int lane, float l, float top, float inv) {
    const bool in = lane < c.K && l > -INFINITY;
    if (!c.renorm)
        return !in ? 0.0f : c.softmax ? expf(l - finite_top(top)) * inv : sigmoid32(l);
    const float most = warp_max(in ? l : -INFINITY);
    float a = 0.0f;
    if (in) {
        if (c.softmax) {
            a = expf(l - most);
        } else {
            const float t = fminf(most, 0.0f);
            a = l >= 0.0f ? sigmoid32(l) : expf(l - t) / (1.0f + expf(l));
        }
    }
    const float total = warp_sum(a);
    return total > 0.0f ? __fdividef(a, total) : total == 0.0f ? 0.0f : total;
}

struct RouterFwd {
    RouterShape c;
    const void *logits;
    const float *bias;
    int32_t *idx;
    float *w;
    int32_t *count_part;  // [blocks][E], or nullptr
    float *sum_part;      // [blocks][E], or nullptr
};

// key j, j not a constant
template <int PER>
MOK_DEV uint32_t key_of(const uint32_t (&key)[PER], int j) {
    uint32_t u = 0u;
#pragma unroll
    for (int k = 0; k < PER; ++k)
        if (k == j) u = key[k];
    return u;
}

// What a lane has left to offer: its two largest keys that are not taken, with their experts.
template <int PER, int VEC>
struct Offer {
    std::conditional_t<(PER > 32), uint64_t, uint32_t> taken;
    uint32_t k0, k1;
    int j0, j1;
    // the two largest of what is left (at first nothing is taken)
    MOK_DEV void look(const uint32_t (&key)[PER], bool first) {
        k0 = k1 = 0u;
        j0 = j1 = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const uint32_t u = !first && ((taken >> j) & 1u) != 0 ? 0u : key[j];
            const bool best = u > k0, second = u > k1;
            k1 = best ? k0 : second ? u : k1;
            j1 = best ? j0 : second ? j : j1;
            k0 = best ? u : k0;
            j0 = best ? j : j0;
        }
    }
    // the warp's next: its key (0: none left) and expert, taken where `take`
    MOK_DEV uint32_t next(const uint32_t (&key)[PER], const Held<VEC> &h, bool take, int &e) {
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, k0);
        const uint32_t holds = __ballot_sync(0xFFFFFFFFu, k0 == top);
        const int mine = h.id(j0);
        if ((holds & (holds - 1)) == 0)
            e = __shfl_sync(0xFFFFFFFFu, mine, __ffs(holds) - 1);
        else
            e = (int)__reduce_min_sync(0xFFFFFFFFu, k0 == top ? (uint32_t)mine : 0xFFFFFFFFu);
        if (take && k0 == top && e == mine) {  // k0 is not 0: as many are left as are taken
            taken |= (decltype(taken))1 << j0;
            k0 = k1;
            j0 = j1;
            k1 = 0u;
            if (k0 == 0u) look(key, false);
        }
        return top;
    }
};

// The `want` largest keys in order, lane k getting the k-th and its expert (more lanes may get the next
// ones), by counting. False, and nothing done, where more than 32 are not below the bound.
template <int PER, int VEC>
MOK_DEV bool side_by_side(const uint32_t (&key)[PER], const Held<VEC> &h, int want, int lane,
                          uint2 (&side)[64], uint32_t &sel, int &id) {
    if (want > 32) return false;
    uint32_t most = 0u;
#pragma unroll
    for (int j = 0; j < PER; ++j) most = max(most, key[j]);
    uint32_t bound = 0u;  // lanes of equal keys go at once: then it is lower than it might be
    for (int k = 0; k < want; ++k) {
        bound = __reduce_max_sync(0xFFFFFFFFu, most);
        if (most == bound) most = 0u;
    }
    bound = max(bound, 1u);
    int n = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) n += key[j] >= bound ? 1 : 0;
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += u;
    }
    const int all = __shfl_sync(0xFFFFFFFFu, upto, 31);
    if (all > 32) return false;
    int at = upto - n;
#pragma unroll
    for (int j = 0; j < PER; ++j)
        if (key[j] >= bound) side[at++] = make_uint2(~(uint32_t)h.id(j), key[j]);
    __syncwarp();
    // largest key first, lowest expert among equals: one 64-bit order
    const uint64_t *as64 = reinterpret_cast<const uint64_t *>(side);
    const uint64_t mine = lane < all ? as64[lane] : 0ull;
    int rank = 0;
    for (int k = 0; k < all; ++k) rank += as64[k] > mine ? 1 : 0;
    if (lane < all) side[32 + rank] = make_uint2((uint32_t)mine, (uint32_t)(mine >> 32));
    __syncwarp();
    const uint2 got = side[32 + lane];
    sel = lane < all ? got.y : 0u;
    id = lane < all ? (int)~got.x : 0;
    return true;
}

// PER experts a lane. Scores are needed for the choice (SCORED: with a bias, or groups by the sum of
// two), for the sums or for weights out of all of a softmax.
template <int PER, int VEC, bool BF16, bool SCORED>
__global__ void __launch_bounds__(32 * ROUTER_WARPS, per_sm(PER)) router_kernel(const RouterFwd a) {
    extern __shared__ uint32_t router_smem[];
    __shared__ alignas(8) uint2 side[ROUTER_WARPS][64];
    const RouterShape &c = a.c;
    int32_t *hist = reinterpret_cast<int32_t *>(router_smem);            // [E]
    float *sums = reinterpret_cast<float *>(router_smem + c.E);          // [warps][E]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    let_next_start();
    wait_for_previous();
    if (a.count_part != nullptr) {
        for (int e = threadIdx.x; e < c.E; e += blockDim.x) hist[e] = 0;
        __syncthreads();
    }
    const Held<VEC> h(c, lane);
    const bool biased = SCORED && a.bias != nullptr;
    const bool row_scores = SCORED || a.sum_part != nullptr || (c.softmax && !c.renorm);
    float largest_bias = 0.0f;
    if (biased) {
        for (int j = 0; j < h.n; ++j) largest_bias = fmaxf(largest_bias, fabsf(a.bias[h.id(j)]));
        largest_bias = warp_max(largest_bias);
    }
    float acc[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) acc[j] = 0.0f;
    const int64_t step = (int64_t)gridDim.x * ROUTER_WARPS;
    for (int64_t t = (int64_t)blockIdx.x * ROUTER_WARPS + warp; t < c.T; t += step) {
        const void *row = static_cast<const char *>(a.logits) + t * c.ld * (BF16 ? 2 : 4);
        float v[PER];
        load_logits<PER, VEC, BF16>(row, h, v);
        // scores, and what the choice goes by
        float top = -INFINITY, inv = 0.0f, most = 0.0f;
        float b1 = -INFINITY, b2 = -INFINITY;  // the lane's two largest: of s + bias, or logits
        if (row_scores) {
            float s[PER];
#pragma unroll
            for (int j = 0; j < PER; ++j) s[j] = v[j];
            if (c.softmax) {
                inv = softmax_scores(s, top);
            } else {
#pragma unroll
                for (int j = 0; j < PER; ++j) s[j] = sigmoid_hw(s[j]);
            }
#pragma unroll
            for (int j = 0; j < PER; ++j) acc[j] += s[j];
            if (SCORED) {
#pragma unroll
                for (int j = 0; j < PER; ++j) most = fmaxf(most, s[j]);
                most = warp_max(most);
                if (biased) {
                    float b[PER];
                    load_logits<PER, VEC, false>(a.bias, h, b);
#pragma unroll
                    for (int j = 0; j < PER; ++j) s[j] += b[j];
                }
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    if (v[j] == -INFINITY) s[j] = -INFINITY;
                    b2 = fmaxf(b2, fminf(b1, s[j]));
                    b1 = fmaxf(b1, s[j]);
                    if (biased) v[j] = s[j];
                }
            }
        }
        if (!SCORED && c.G > 1) {
#pragma unroll
            for (int j = 0; j < PER; ++j) b1 = fmaxf(b1, v[j]);
        }
        const float err = SCORED ? score_error(c, most) : 0.0f, size = most + largest_bias;
        bool kept = h.n > 0;
        if (c.G > 1) {
            for (int o = 1; o < c.lanes; o <<= 1) {
                const float o1 = __shfl_xor_sync(0xFFFFFFFFu, b1, o);
                const float o2 = __shfl_xor_sync(0xFFFFFFFFu, b2, o);
                b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
                b1 = fmaxf(b1, o1);
            }
            // (two biases near the lowest value are still above a group of masked experts)
            const float score = SCORED && c.top == 2 && b2 > -INFINITY ? fmaxf(b1 + b2, -3.402823466e38f) : b1;
            int rank = 0;
            for (int g = 0; g < c.G; ++g) {
                const float other = __shfl_sync(0xFFFFFFFFu, score, g * c.lanes);
                rank += other > score || (other == score && g < h.g) ? 1 : 0;
            }
            kept = kept && rank < c.keep;
            if (SCORED && c.keep < c.G) {
                // The least kept and the largest other score, each of at most two c, which are at most
                // `size`: off by 2 err, the rounding of both c and of their sum, 4 x 2^-24 size
                const float tol = 4.0f * err + 4.76837158203125e-7f * size;
                const uint32_t o = order_of(score);
                const float low = of_order(__reduce_min_sync(0xFFFFFFFFu, kept ? o : 0xFFFFFFFFu));
                const float high = of_order(__reduce_max_sync(
                    0xFFFFFFFFu, h.n > 0 && !kept ? o : ORDER_MASKED));
                if (high > -INFINITY && !(low - high > tol)) {
                    // groups that clearly lie on their side of the border stay there
                    const bool among = h.n > 0 && (kept ? !(score - high > tol) : !(low - score > tol));
                    const uint32_t sure = __ballot_sync(0xFFFFFFFFu, kept && !among && lane % c.lanes == 0);
                    uint64_t cand = 0;
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const float s = biased ? v[j] : unbiased_score(c, v[j], top, inv);
                        if (j < h.n && !((c.top == 2 ? b2 : b1) - s > tol)) cand |= 1ull << j;
                    }
                    const bool now = keep_exact<VEC, BF16>(c, row, a.bias, finite_top(top), among, cand,
                                                           c.keep - __popc(sure), lane);
                    kept = among ? now : kept;
                }
            }
        }
        uint32_t key[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) key[j] = j / VEC * VEC < (kept ? h.n : 0) ? order_of(v[j]) : 0u;
        uint32_t sel = 0u;  // lane k: the k-th key and expert
        int id = 0, e = 0;
        Offer<PER, VEC> left;
        const auto rounds = [&] {
            left.taken = 0;
            left.look(key, true);
            for (int k = 0; k < c.K; ++k) {
                const uint32_t top_key = left.next(key, h, true, e);
                if (lane == k) {
                    sel = top_key;
                    id = e;
                }
            }
        };
        // with a bias one more, for the distance between the last chosen and the first that is not
        const bool quick = side_by_side<PER, VEC>(key, h, biased ? c.K + 1 : c.K, lane, side[warp], sel, id);
        if (!quick) rounds();
        bool exact = false;
        if (biased) {
            // neighbours in the order, the first that was not chosen among them, that the scores' errors
            // and the rounding of their sums with the bias could exchange
            const float tol = 2.0f * err + 1.1920928955078125e-7f * size;
            uint32_t after = __shfl_down_sync(0xFFFFFFFFu, sel, 1);
            if (!quick) {
                const uint32_t rest = __reduce_max_sync(0xFFFFFFFFu, left.k0);
                if (lane == c.K - 1) after = rest;
            }
            const auto near = [&](uint32_t x, uint32_t y) {
                return y > ORDER_MASKED && !(of_order(x) - of_order(y) > tol);
            };
            const auto alike = [&](int x, int y) {  // a tie, not a close call
                return load_logit<BF16>(row, x) == load_logit<BF16>(row, y) && a.bias[x] == a.bias[y];
            };
            if (__any_sync(0xFFFFFFFFu, lane < c.K && near(sel, after))) {
                // go on as long as the next is too close to the last to tell them apart
                if (quick) rounds();
                int many = c.K;
                for (; many < 32; ++many) {
                    const uint32_t last = __shfl_sync(0xFFFFFFFFu, sel, many - 1);
                    const uint32_t rest_key = left.next(key, h, false, e);
                    if (rest_key == 0u || !near(last, rest_key)) break;
                    left.next(key, h, true, e);
                    if (lane == many) {
                        sel = rest_key;
                        id = e;
                    }
                }
                after = __shfl_down_sync(0xFFFFFFFFu, sel, 1);
                const int other = __shfl_down_sync(0xFFFFFFFFu, id, 1);
                const bool close = __any_sync(0xFFFFFFFFu, lane < many - 1 && near(sel, after) && !alike(id, other));
                // No lane left: is any of the rest close? Ties of the last may stay behind only where the
                // order of the run stands: they may all be better than others in it.
                if (many == 32) {
                    const uint32_t last = __shfl_sync(0xFFFFFFFFu, sel, 31);
                    const int of_last = __shfl_sync(0xFFFFFFFFu, id, 31);
                    for (int j = 0; j < h.n; ++j) {
                        const int i = h.id(j);
                        const uint32_t u = kept && ((left.taken >> j) & 1u) == 0 ? key_of(key, j) : 0u;
                        exact = exact || (near(last, u) && (close || !alike(of_last, i)));
                    }
                    exact = __any_sync(0xFFFFFFFFu, exact);
                }
                if (!exact && close)
                    id = choose_among<VEC, BF16>(c, row, a.bias, finite_top(top), id, many, lane);
            }
        }
        if (SCORED && __any_sync(0xFFFFFFFFu, exact))
            id = choose_exact<PER, VEC, BF16>(c, row, a.bias, finite_top(top), kept, lane);
        const float l = lane < c.K ? load_logit<BF16>(row, id) : 0.0f;
        const float wt = chosen_weight(c, lane, l, top, inv);
        if (lane < c.K) {
            a.idx[t * c.K + lane] = id;
            a.w[t * c.K + lane] = c.scale * wt;
            if (a.count_part != nullptr) atomicAdd(&hist[id], 1);
        }
    }
    if (a.sum_part != nullptr) {
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (j < h.n) sums[warp * c.E + h.id(j)] = acc[j];
    }
    if (a.sum_part == nullptr && a.count_part == nullptr) return;
    __syncthreads();
    for (int e = threadIdx.x; e < c.E; e += blockDim.x) {
        const int64_t at = (int64_t)blockIdx.x * c.E + e;
        if (a.count_part != nullptr) a.count_part[at] = hist[e];
        if (a.sum_part != nullptr) {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < ROUTER_WARPS; ++k) s += sums[k * c.E + e];
            a.sum_part[at] = s;
        }
    }
}

// ---- few experts: a thread a token ----
//
// Up to FEW_E experts and FEW_K choices by the logits themselves (no bias, one group), and gradients of
// as many. A warp a token would leave most lanes idle: a row fits a thread's registers, K rounds compare
// it, and nothing crosses lanes but a block's loads at its end. The rule looks at E and K alone, so that a
// token's weights do not depend on how many others there are.
// A warp against a thread a token, us: 131072 x 8, top 2 of a softmax 41 / 5.6, its gradient with the sums'
// 67 / 5.8, 2.4 million x 2 of a sigmoid 693 / 48; 64 tokens of 8 top 2 2.3 / 2.4, of 16 top 4 2.3 / 3.1. With
// 32 experts, top 8 and 4096 tokens it is 4.6 / 10.3: a thread's rounds are its own to wait for. What bounds
// it: scattered rows of 8 to 64 bytes, and with loads the atomics on a block's few counts.
constexpr int FEW_E = 16, FEW_K = 4, FEW_WARPS = 4;
bool few(const RouterShape &c) { return c.G == 1 && c.E <= FEW_E && c.K <= FEW_K; }
RouterShape few_shape(RouterShape c) {
    c.lanes = 1;
    return c;
}

template <int PER>
MOK_DEV float few_softmax(float (&v)[PER], float &top) {
    top = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) top = fmaxf(top, v[j]);
    const float shift = finite_top(top);
    float den = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        v[j] = exp2_hw((v[j] - shift) * LOG2E_R);
        den += v[j];
    }
    const float inv = den > 0.0f ? 1.0f / den : den == 0.0f ? 0.0f : den;
#pragma unroll
    for (int j = 0; j < PER; ++j) v[j] *= inv;
    return inv;
}

// chosen_weight of a token's K logits (-inf past them): l becomes the weights
MOK_DEV void few_weights(const RouterShape &c, float (&l)[FEW_K], float top, float inv) {
    if (!c.renorm) {
#pragma unroll
        for (int k = 0; k < FEW_K; ++k)
            l[k] = !(l[k] > -INFINITY) ? 0.0f : c.softmax ? expf(l[k] - finite_top(top)) * inv : sigmoid32(l[k]);
        return;
    }
    float most = -INFINITY, total = 0.0f;
#pragma unroll
    for (int k = 0; k < FEW_K; ++k) most = fmaxf(most, l[k]);
    const float t = fminf(most, 0.0f);
#pragma unroll
    for (int k = 0; k < FEW_K; ++k) {
        if (k >= c.K) continue;
        const bool in = l[k] > -INFINITY;
        l[k] = !in          ? 0.0f
               : c.softmax  ? expf(l[k] - most)
               : l[k] >= 0.0f ? sigmoid32(l[k])
                            : expf(l[k] - t) / (1.0f + expf(l[k]));
        total += l[k];
    }
#pragma unroll
    for (int k = 0; k < FEW_K; ++k)
        l[k] = total > 0.0f ? __fdividef(l[k], total) : total == 0.0f ? 0.0f : total;
}

template <int PER, int VEC, bool BF16>
__global__ void __launch_bounds__(32 * FEW_WARPS) router_few_kernel(const RouterFwd a) {
    extern __shared__ uint32_t router_smem[];
    const RouterShape &c = a.c;
    int32_t *hist = reinterpret_cast<int32_t *>(router_smem);    // [E]
    float *sums = reinterpret_cast<float *>(router_smem + c.E);  // [warps][E]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    let_next_start();
    wait_for_previous();
    if (a.count_part != nullptr) {
        if (threadIdx.x < c.E) hist[threadIdx.x] = 0;
        __syncthreads();
    }
    const Held<VEC> h(c, 0);
    const bool row_scores = a.sum_part != nullptr || (c.softmax && !c.renorm);
    float acc[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) acc[j] = 0.0f;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; t < c.T; t += step) {
        float v[PER];
        load_logits<PER, VEC, BF16>(static_cast<const char *>(a.logits) + t * c.ld * (BF16 ? 2 : 4), h, v);
        uint32_t key[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) key[j] = j < c.E ? order_of(v[j]) : 0u;
        float top = -INFINITY, inv = 0.0f;
        if (row_scores) {
            if (c.softmax) {
                inv = few_softmax(v, top);
            } else {
#pragma unroll
                for (int j = 0; j < PER; ++j) v[j] = sigmoid_hw(v[j]);
            }
#pragma unroll
            for (int j = 0; j < PER; ++j) acc[j] += v[j];
        }
        int id[FEW_K];
        float l[FEW_K];
#pragma unroll
        for (int k = 0; k < FEW_K; ++k) {
            l[k] = -INFINITY;
            if (k >= c.K) continue;
            uint32_t most = 0u;
            id[k] = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if (key[j] > most) id[k] = j;
                most = max(most, key[j]);
            }
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (j == id[k]) key[j] = 0u;
            l[k] = of_order(most);
            if (a.count_part != nullptr) atomicAdd(&hist[id[k]], 1);
        }
        few_weights(c, l, top, inv);
#pragma unroll
        for (int k = 0; k < FEW_K; ++k) {
            if (k >= c.K) continue;
            a.idx[t * c.K + k] = id[k];
            a.w[t * c.K + k] = c.scale * l[k];
        }
    }
    if (a.sum_part == nullptr && a.count_part == nullptr) return;
    if (a.sum_part != nullptr) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const float s = warp_sum(acc[j]);
            if (lane == 0 && j < c.E) sums[warp * c.E + j] = s;
        }
    }
    __syncthreads();
    const int e = threadIdx.x;
    if (e >= c.E) return;
    const int64_t at = (int64_t)blockIdx.x * c.E + e;
    if (a.count_part != nullptr) a.count_part[at] = hist[e];
    if (a.sum_part != nullptr) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < FEW_WARPS; ++k) s += sums[k * c.E + e];
        a.sum_part[at] = s;
    }
}

// The blocks' counts (y = 0) and sums (y = 1), added in order: 32 experts a block, each warp a slice
// of the parts.
constexpr int LOAD_SLICES = 32;
template <class V>
MOK_DEV void add_parts(const V *part, int parts, int E, V *out, V (*sh)[32]) {
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane;
    V s = 0;
    // a batch of loads at a time, the last one too (an unrolled loop's rest is one after another)
    for (int p0 = slice; p0 < parts; p0 += 20 * LOAD_SLICES) {
        V v[20];
#pragma unroll
        for (int k = 0; k < 20; ++k) {
            const int p = p0 + k * LOAD_SLICES;
            v[k] = p < parts && e < E ? part[(int64_t)p * E + e] : 0;
        }
#pragma unroll
        for (int k = 0; k < 20; ++k) s += v[k];
    }
    sh[slice][lane] = s;
    __syncthreads();
    if (slice != 0 || e >= E) return;
    s = 0;
#pragma unroll
    for (int k = 0; k < LOAD_SLICES; ++k) s += sh[k][lane];
    out[e] = s;
}
__global__ void __launch_bounds__(32 * LOAD_SLICES)
    router_load_kernel(const int32_t *count_part, const float *sum_part, int parts, int E,
                       int32_t *counts, float *score_sum) {
    __shared__ int32_t sh[LOAD_SLICES][32];
    let_next_start();
    wait_for_previous();
    if (blockIdx.y == 0) {
        if (counts != nullptr) add_parts(count_part, parts, E, counts, sh);
    } else if (score_sum != nullptr) {
        add_parts(sum_part, parts, E, score_sum, reinterpret_cast<float(*)[32]>(sh));
    }
}

struct RouterBwd {
    RouterShape c;  // of one group: lanes hold experts of the whole row
    const void *logits;
    const int32_t *idx;
    const float *dw, *dsum;
    void *dlogits;
    int *status;
};

template <bool BF16>
MOK_DEV void store_logit(void *row, int e, float v) {
    if (BF16)
        static_cast<uint16_t *>(row)[e] = f32_to_bf16(v);
    else
        static_cast<float *>(row)[e] = v;
}
template <int PER, int VEC, bool BF16>
MOK_DEV void store_logits(void *row, const Held<VEC> &h, const float (&v)[PER]) {
#pragma unroll
    for (int j = 0; j < PER; j += VEC) {
        if (j >= h.n) continue;
        const int e = h.id(j);
        if (VEC == 1) {
            store_logit<BF16>(row, e, v[j]);
        } else if (BF16) {
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(row) + e) = make_uint2(
                pack_bf16x2(v[j], v[j + VEC / 4]), pack_bf16x2(v[j + VEC / 2], v[j + VEC - 1]));
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(row) + e) =
                make_float4(v[j], v[j + VEC / 4], v[j + VEC / 2], v[j + VEC - 1]);
        }
    }
}

// One warp per token at a time, walking over the tokens with the gradient of the sums in registers.
// The row is written as if nothing were chosen, then the chosen entries again, each from all that it
// gets, by the lane that holds it. DENSE: every logit of a row gets something.
// 16384 x 512 with the sums' gradient: 17.0 us, 67 MB at 4.0 TB/s: a warp's chain of reductions a token at
// 32 warps a SM (18.5 us at the 24 that the compiler's own choice of registers allows).
template <int PER, int VEC, bool BF16, bool DENSE>
__global__ void __launch_bounds__(32 * ROUTER_WARPS, DENSE && PER == 16   ? 4
                                                     : DENSE && PER == 32 ? 2
                                                                          : 0)
    router_backward_kernel(const RouterBwd a) {
    const RouterShape &c = a.c;
    const int lane = threadIdx.x & 31;
    let_next_start();
    wait_for_previous();
    const Held<VEC> h(c, lane);
    float ds[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j)
        ds[j] = DENSE && a.dsum != nullptr && j < h.n ? a.dsum[h.id(j)] : 0.0f;
    const int64_t step = (int64_t)gridDim.x * ROUTER_WARPS;
    int64_t t = (int64_t)blockIdx.x * ROUTER_WARPS + (threadIdx.x >> 5);
    // a token's ids and weights come a token early: its chosen logits wait for them
    int next_id = -1;
    float next_dw = 0.0f;
    const auto fetch = [&](int64_t n) {
        if (lane < c.K && n < c.T) {
            next_id = a.idx[n * c.K + lane];
            next_dw = a.dw[n * c.K + lane];
        }
    };
    fetch(t);
    for (; t < c.T; t += step) {
        const int64_t at = t * c.ld * (BF16 ? 2 : 4);
        const void *row = static_cast<const char *>(a.logits) + at;
        void *out = static_cast<char *>(a.dlogits) + at;
        float s[PER];
        if (DENSE) load_logits<PER, VEC, BF16>(row, h, s);
        int id = next_id;
        const float dw = next_dw;
        float l = -INFINITY;
        if (lane < c.K) {
            if (id < 0 || id >= c.E) {
                raise_status(a.status, MOK_ERR_DEVICE_INVARIANT);
                id = -1;
            } else {
                l = load_logit<BF16>(row, id);
            }
        }
        fetch(t + step);
        float top = -INFINITY, inv = 0.0f, mean = 0.0f;  // mean: of dsum under the scores
        if (DENSE && c.softmax) {
            inv = softmax_scores(s, top);
            if (a.dsum != nullptr) {
#pragma unroll
                for (int j = 0; j < PER; ++j) mean = fmaf(s[j], ds[j], mean);
                mean = warp_sum(mean);
            }
        }
        const float wt = chosen_weight(c, lane, l, top, inv);
        // what a chosen logit gets through its weight; a masked one nothing, whatever dw holds
        const bool live = l > -INFINITY;
        const float m = warp_sum(live ? dw * wt : 0.0f);
        float add = 0.0f;
        if (live) {
            add = c.scale * wt * (c.renorm ? dw - m : dw);
            if (!c.softmax) add *= 1.0f / (1.0f + expf(l));  // 1 - s
        }
        // a softmax's chosen weights take from all
        const float all = c.softmax && !c.renorm ? c.scale * m + mean : mean;
        // the same id twice: the first of its lanes adds up
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, id < 0 ? -1 - lane : id);
        if (__any_sync(0xFFFFFFFFu, (peers & (peers - 1)) != 0)) {
            float sum = 0.0f;
            for (int k = 0; k < 32; ++k) {
                const float other = __shfl_sync(0xFFFFFFFFu, add, k);
                if ((peers >> k) & 1u) sum += other;
            }
            add = sum;
            if (lane != __ffs(peers) - 1) id = -1;
        }
        if (DENSE && id >= 0 && live) {
            const float d = a.dsum != nullptr ? a.dsum[id] : 0.0f;
            add += c.softmax ? expf(l - finite_top(top)) * inv * (d - all)
                             : d * sigmoid32(l) * (1.0f / (1.0f + expf(l)));
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (!DENSE) {
                s[j] = 0.0f;
            } else if (c.softmax) {
                s[j] *= ds[j] - all;
            } else {
                // s (1 - s) = e / (1 + e)^2, e = 2^-|x|; nothing for a masked expert
                const float e = exp2_hw(-LOG2E_R * fabsf(s[j]));
                s[j] = __fdividef(ds[j] * e, (1.0f + e) * (1.0f + e));
            }
        }
        __syncwarp();  // d_logits may be logits: all of the row has been read
        store_logits<PER, VEC, BF16>(out, h, s);
        __syncwarp();
        if (id >= 0) store_logit<BF16>(out, id, add);
    }
}

// The gradient with a thread a token: the row as if nothing were chosen, then the chosen entries.
template <int PER, int VEC, bool BF16, bool DENSE>
__global__ void __launch_bounds__(32 * FEW_WARPS) router_few_backward_kernel(const RouterBwd a) {
    const RouterShape &c = a.c;
    let_next_start();
    wait_for_previous();
    const Held<VEC> h(c, 0);
    float ds[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) ds[j] = DENSE && a.dsum != nullptr && j < c.E ? a.dsum[j] : 0.0f;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; t < c.T; t += step) {
        const int64_t at = t * c.ld * (BF16 ? 2 : 4);
        const void *row = static_cast<const char *>(a.logits) + at;
        void *out = static_cast<char *>(a.dlogits) + at;
        float s[PER];
        if (DENSE) load_logits<PER, VEC, BF16>(row, h, s);
        int id[FEW_K];
        float dw[FEW_K], l[FEW_K], wt[FEW_K];
#pragma unroll
        for (int k = 0; k < FEW_K; ++k) {
            id[k] = -1;
            dw[k] = 0.0f;
            if (k < c.K) {
                id[k] = a.idx[t * c.K + k];
                dw[k] = a.dw[t * c.K + k];
            }
        }
#pragma unroll
        for (int k = 0; k < FEW_K; ++k) {
            l[k] = -INFINITY;
            if (k >= c.K) continue;
            if (id[k] < 0 || id[k] >= c.E) {
                raise_status(a.status, MOK_ERR_DEVICE_INVARIANT);
                id[k] = -1;
            } else {
                l[k] = load_logit<BF16>(row, id[k]);
            }
        }
        float top = -INFINITY, inv = 0.0f, mean = 0.0f;
        if (DENSE && c.softmax) {
            inv = few_softmax(s, top);
            if (a.dsum != nullptr) {
#pragma unroll
                for (int j = 0; j < PER; ++j) mean = fmaf(s[j], ds[j], mean);
            }
        }
#pragma unroll
        for (int k = 0; k < FEW_K; ++k) wt[k] = l[k];
        few_weights(c, wt, top, inv);
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < FEW_K; ++k)
            if (l[k] > -INFINITY) m += dw[k] * wt[k];
        const float all = c.softmax && !c.renorm ? c.scale * m + mean : mean;
        float add[FEW_K];
#pragma unroll
        for (int k = 0; k < FEW_K; ++k) {
            add[k] = 0.0f;
            if (k < c.K && l[k] > -INFINITY) {
                add[k] = c.scale * wt[k] * (c.renorm ? dw[k] - m : dw[k]);
                if (!c.softmax) add[k] *= 1.0f / (1.0f + expf(l[k]));  // 1 - s
            }
            // the same id twice: the first adds up
#pragma unroll
            for (int i = 0; i < k; ++i)
                if (id[i] >= 0 && id[i] == id[k]) {
                    add[i] += add[k];
                    id[k] = -1;
                }
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (!DENSE) {
                s[j] = 0.0f;
            } else if (c.softmax) {
                s[j] *= ds[j] - all;
            } else {
                const float e = exp2_hw(-LOG2E_R * fabsf(s[j]));  // as in a warp's
                s[j] = __fdividef(ds[j] * e, (1.0f + e) * (1.0f + e));
            }
        }
        store_logits<PER, VEC, BF16>(out, h, s);
#pragma unroll
        for (int k = 0; k < FEW_K; ++k) {
            if (id[k] < 0) continue;
            if (DENSE && l[k] > -INFINITY) {
                const float d = a.dsum != nullptr ? a.dsum[id[k]] : 0.0f;
                add[k] += c.softmax ? expf(l[k] - finite_top(top)) * inv * (d - all)
                                    : d * sigmoid32(l[k]) * (1.0f / (1.0f + expf(l[k])));
            }
            store_logit<BF16>(out, id[k], add[k]);
        }
    }
}

__global__ void router_bias_kernel(const int32_t *counts, int64_t routed, int E, float rate,
                                   const float *bias, float *out) {
    let_next_start();
    wait_for_previous();
    const int e = blockIdx.x * blockDim.x + threadIdx.x;
    if (e >= E) return;
    const int64_t less = routed - (int64_t)counts[e] * E;
    out[e] = bias[e] + (less > 0 ? rate : less < 0 ? -rate : 0.0f);
}

RouterShape shape_of(const mok_router_config &c, int groups) {
    RouterShape s = {};
    s.T = c.T;
    s.ld = c.ld;
    s.E = c.E;
    s.K = c.K;
    s.G = groups;
    s.keep = c.topk_groups;
    s.top = c.group_top;
    s.per = c.E / groups;
    s.lanes = 32;
    while (s.lanes * groups > 32) s.lanes /= 2;
    s.softmax = c.score == MOK_SCORE_SOFTMAX;
    s.renorm = c.renormalize != 0;
    s.scale = c.scale;
    return s;
}

// experts a load (four where groups and rows allow it), experts a lane
bool loads_four(const RouterShape &s) { return s.per % 4 == 0 && s.ld % 4 == 0; }
int held_of(const RouterShape &s) {
    const int n = loads_four(s) ? (s.per / 4 + s.lanes - 1) / s.lanes * 4
                                : (s.per + s.lanes - 1) / s.lanes;
    const int sizes[] = {2, 4, 8, 16, 32};
    for (int k : sizes)
        if (n <= k && (k != 2 || !loads_four(s))) return k;
    return 64;  // only with many groups: 17 of 60 experts have one lane each
}
int64_t blocks_of(const RouterShape &s) {
    const int64_t n = (s.T + ROUTER_WARPS - 1) / ROUTER_WARPS, most = GB300_SMS * per_sm(held_of(s));
    return n < most ? n : most;
}

// f(experts a lane, experts a load) as constants
template <class F>
cudaError_t with_held(const RouterShape &s, F &&f) {
    using std::integral_constant;
    const int n = held_of(s);
    const integral_constant<int, 1> one;
    const integral_constant<int, 4> four;
#define MOK_HELD(N) \
    if (n == N) return loads_four(s) ? f(integral_constant<int, N>{}, four) : f(integral_constant<int, N>{}, one)
    if (n == 2) return f(integral_constant<int, 2>{}, one);
    MOK_HELD(4);
    MOK_HELD(8);
    MOK_HELD(16);
    MOK_HELD(32);
    return loads_four(s) ? f(integral_constant<int, 64>{}, four) : f(integral_constant<int, 64>{}, one);
#undef MOK_HELD
}

template <class F>
cudaError_t with_few(const RouterShape &s, F &&f) {
    using std::integral_constant;
    const integral_constant<int, 1> one;
    const integral_constant<int, 4> four;
    const integral_constant<int, 8> eight;
    const integral_constant<int, FEW_E> all;
    if (s.E <= 8) return loads_four(s) ? f(eight, four) : f(eight, one);
    return loads_four(s) ? f(all, four) : f(all, one);
}
int64_t few_blocks(const RouterShape &s, int64_t most) {
    const int64_t n = (s.T + 32 * FEW_WARPS - 1) / (32 * FEW_WARPS);
    return n < most ? n : most;
}

// blocks of a forward pass, and so parts of its loads (never more than there is room for)
int64_t parts_of(const RouterFwd &a) {
    const int64_t n = blocks_of(a.c);
    return few(a.c) && a.bias == nullptr ? few_blocks(a.c, n) : n;
}

cudaError_t launch_router(const RouterFwd &a, bool bf16, cudaStream_t s) {
    const unsigned grid = (unsigned)parts_of(a);
    if (few(a.c) && a.bias == nullptr) {
        RouterFwd b = a;
        b.c = few_shape(a.c);
        return with_few(a.c, [&](auto per, auto vec) {
            const auto go = [&](auto *kernel) {
                return launch_edge(kernel, grid, 32 * FEW_WARPS, (1 + FEW_WARPS) * a.c.E * 4, 1, s, b);
            };
            return bf16 ? go(router_few_kernel<per.value, vec.value, true>)
                        : go(router_few_kernel<per.value, vec.value, false>);
        });
    }
    const int smem = a.sum_part != nullptr     ? (1 + ROUTER_WARPS) * a.c.E * 4
                     : a.count_part != nullptr ? a.c.E * 4
                                               : 0;
    const bool scored = a.bias != nullptr || (a.c.G > 1 && a.c.top == 2);
    return with_held(a.c, [&](auto per, auto vec) {
        const auto go = [&](auto *kernel) {
            return launch_edge(kernel, grid, 32 * ROUTER_WARPS, smem, 1, s, a);
        };
        if (scored)
            return bf16 ? go(router_kernel<per.value, vec.value, true, true>)
                        : go(router_kernel<per.value, vec.value, false, true>);
        return bf16 ? go(router_kernel<per.value, vec.value, true, false>)
                    : go(router_kernel<per.value, vec.value, false, false>);
    });
}

cudaError_t launch_router_backward(const RouterBwd &a, bool bf16, cudaStream_t s) {
    const int64_t tokens = (a.c.T + ROUTER_WARPS - 1) / ROUTER_WARPS;
    const int64_t most = (int64_t)device_sm_count() * 8;
    const unsigned grid = (unsigned)(tokens < most ? tokens : most);
    const bool dense = a.dsum != nullptr || (a.c.softmax && !a.c.renorm);
    if (few(a.c)) {
        RouterBwd b = a;
        b.c = few_shape(a.c);
        const unsigned blocks = (unsigned)few_blocks(a.c, 2 * most);
        return with_few(a.c, [&](auto per, auto vec) {
            const auto go = [&](auto *kernel) {
                return launch_edge(kernel, blocks, 32 * FEW_WARPS, 0, 1, s, b);
            };
            if (dense)
                return bf16 ? go(router_few_backward_kernel<per.value, vec.value, true, true>)
                            : go(router_few_backward_kernel<per.value, vec.value, false, true>);
            return bf16 ? go(router_few_backward_kernel<per.value, vec.value, true, false>)
                        : go(router_few_backward_kernel<per.value, vec.value, false, false>);
        });
    }
    return with_held(a.c, [&](auto per, auto vec) {
        const auto go = [&](auto *kernel) {
            return launch_edge(kernel, grid, 32 * ROUTER_WARPS, 0, 1, s, a);
        };
        if constexpr (per.value > 32) {
            return cudaErrorInvalidValue;  // one group of 1024 experts has 32 a lane
        } else {
            if (dense)
                return bf16 ? go(router_backward_kernel<per.value, vec.value, true, true>)
                            : go(router_backward_kernel<per.value, vec.value, false, true>);
            return bf16 ? go(router_backward_kernel<per.value, vec.value, true, false>)
                        : go(router_backward_kernel<per.value, vec.value, false, false>);
        }
    });
}

size_t part_bytes(const mok_router_config &c) {
    return (size_t)round_up(blocks_of(shape_of(c, c.groups)) * c.E * 4, 256);
}

}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

mok_status mok_check_router_config(const mok_router_config *c) {
    if (c == nullptr) return MOK_ERR_INVALID_ARG;
    if (c->abi_version != MOK_ABI_VERSION) return MOK_ERR_ABI;
    if (c->T < 0 || c->E < 1 || c->E > MAX_E) return MOK_ERR_INVALID_ARG;
    if (c->groups < 1 || c->groups > MAX_GROUPS || c->E % c->groups != 0) return MOK_ERR_INVALID_ARG;
    if (c->topk_groups < 1 || c->topk_groups > c->groups) return MOK_ERR_INVALID_ARG;
    if (c->K < 1 || c->K > 32 || c->K > c->topk_groups * (c->E / c->groups))
        return MOK_ERR_INVALID_ARG;
    if ((int64_t)c->T * c->K > INT32_MAX) return MOK_ERR_INVALID_ARG;
    if (c->dtype != MOK_DTYPE_BF16 && c->dtype != MOK_DTYPE_F32) return MOK_ERR_INVALID_ARG;
    if (c->score != MOK_SCORE_SOFTMAX && c->score != MOK_SCORE_SIGMOID) return MOK_ERR_INVALID_ARG;
    if (c->group_top < 1 || c->group_top > 2) return MOK_ERR_INVALID_ARG;
    if (c->renormalize < 0 || c->renormalize > 1 || c->reserved != 0) return MOK_ERR_INVALID_ARG;
    if (!(c->scale > 0.0f && c->scale <= 3.402823466e38f)) return MOK_ERR_INVALID_ARG;
    if (c->ld < c->E || c->ld > ((int64_t)1 << 30)) return MOK_ERR_INVALID_ARG;
    return MOK_OK;
}

size_t mok_router_workspace_size(const mok_router_config *c) {
    if (mok_check_router_config(c) != MOK_OK) return 0;
    const size_t n = 2 * part_bytes(*c);
    return n > 0 ? n : 256;
}

mok_status mok_router_forward(const mok_router_config *c, const void *logits, const float *bias,
                              int32_t *topk_idx, float *topk_w, int32_t *counts, float *score_sum,
                              void *ws, size_t ws_bytes, cudaStream_t stream) {
    mok_status st = mok_check_router_config(c);
    if (st != MOK_OK) return st;
    int *status;
    if ((st = current_device_status_word(&status)) != MOK_OK) return st;
    const bool load = counts != nullptr || score_sum != nullptr;
    if (load && (ws == nullptr || ((uintptr_t)ws & 255u) != 0 || ws_bytes < mok_router_workspace_size(c)))
        return MOK_ERR_WORKSPACE;
    if (c->T > 0 && (!logits || !topk_idx || !topk_w)) return MOK_ERR_INVALID_ARG;
    const void *ps[] = {logits, bias, topk_idx, topk_w, counts, score_sum};
    for (const void *p : ps)
        if (p && !op_aligned16(p)) return MOK_ERR_INVALID_ARG;
    int32_t *cp = counts != nullptr ? (int32_t *)ws : nullptr;
    float *sp = score_sum != nullptr ? (float *)((char *)ws + part_bytes(*c)) : nullptr;
    const RouterFwd a{shape_of(*c, c->groups), logits, bias, topk_idx, topk_w, cp, sp};
    const int parts = (int)parts_of(a);
    if (c->T > 0) {
        MOK_OP_LAUNCH(OP_ROUTER, 1, launch_router(a, c->dtype == MOK_DTYPE_BF16, stream));
    }
    if (load)
        MOK_OP_LAUNCH(OP_ROUTER, 1,
                      launch_edge(router_load_kernel, dim3((unsigned)((c->E + 31) / 32), 2), 32 * LOAD_SLICES,
                                  0, 1, stream, (const int32_t *)cp, (const float *)sp, parts, c->E,
                                  counts, score_sum));
    return MOK_OK;
}

mok_status mok_router_backward(const mok_router_config *c, const void *logits,
                               const int32_t *topk_idx, const float *d_topk_w,
                               const float *d_score_sum, void *d_logits, cudaStream_t stream) {
    mok_status st = mok_check_router_config(c);
    if (st != MOK_OK) return st;
    int *status;
    if ((st = current_device_status_word(&status)) != MOK_OK) return st;
    if (c->T == 0) return MOK_OK;
    if (!logits || !topk_idx || !d_topk_w || !d_logits) return MOK_ERR_INVALID_ARG;
    const void *ps[] = {logits, topk_idx, d_topk_w, d_score_sum, d_logits};
    for (const void *p : ps)
        if (p && !op_aligned16(p)) return MOK_ERR_INVALID_ARG;
    const RouterBwd a{shape_of(*c, 1), logits, topk_idx, d_topk_w, d_score_sum, d_logits, status};
    MOK_OP_LAUNCH(OP_ROUTER_BWD, 1, launch_router_backward(a, c->dtype == MOK_DTYPE_BF16, stream));
    return MOK_OK;
}

mok_status mok_router_update_bias(const mok_router_config *c, const int32_t *counts, float rate,
                                  const float *bias, float *new_bias, cudaStream_t stream) {
    mok_status st = mok_check_router_config(c);
    if (st != MOK_OK) return st;
    int *status;
    if ((st = current_device_status_word(&status)) != MOK_OK) return st;
    if (!counts || !bias || !new_bias || !(rate >= -3.402823466e38f && rate <= 3.402823466e38f))
        return MOK_ERR_INVALID_ARG;
    if (!op_aligned16(counts) || !op_aligned16(bias) || !op_aligned16(new_bias))
        return MOK_ERR_INVALID_ARG;
    MOK_OP_LAUNCH(OP_ROUTER, 1,
                  launch_edge(router_bias_kernel, (unsigned)((c->E + 255) / 256), 256, 0, 1, stream,
                              counts, (int64_t)c->T * c->K, c->E, rate, bias, new_bias));
    return MOK_OK;
}

}  // extern "C"

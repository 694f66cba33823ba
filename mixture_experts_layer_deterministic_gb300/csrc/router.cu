// router.cu -- scores of router logits, choice of experts by score, bias and groups, routing
// weights, loads; the gradient of the logits; the update of the balance bias.
//
//   s = softmax(l) or sigmoid(l), c = s + bias; the K largest c of the kept groups; weights from s
//
// One warp per token. With one group, lane l holds experts l, l + 32, ..; with more, each group has
// L lanes of its own (a power of two) and lane i of group g holds experts g E/groups + i, + L, ..
// A choice takes K rounds: the warp's largest key by one integer reduction over order-preserving
// images, the lowest id that holds it by a second; the lane that held it looks for its next.
//
// The choice has to be that of exact scores. fp32 scores are off by at most a few units in their
// last place (bounds at score_error), so a choice is settled unless two neighbours in the order of
// the chosen, or the last kept and the first other group, are closer than both errors allow; such a
// token (about one in several hundred with a bias and spread logits) is done again in 64 bits.
// Experts whose logits and biases are the same numbers are ties, not close calls.
#include "ops_internal.h"

namespace mok {
namespace {

constexpr int ROUTER_WARPS = 8;
// blocks whose loads are added in order: not of the device, the sums' bits depend on it
constexpr int64_t ROUTER_BLOCKS = 4 * 152;
constexpr int MAX_E = 1024, MAX_GROUPS = 32;

// order-preserving image of a float; -0 as +0. Everything, NaN of either sign too, maps above 0
MOK_DEV uint32_t order_of(float v) {
    uint32_t u = __float_as_uint(v);
    if (u == 0x80000000u) u = 0u;
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return u > 0u ? u : 1u;
}
MOK_DEV float of_order(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
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

// which experts a lane holds: first, first + step, .. (n of them); its group, and place in it
struct Held {
    int first, step, n, g;
    MOK_DEV Held(const RouterShape &c, int lane) {
        if (c.G == 1) {
            first = lane;
            step = 32;
            n = lane < c.E ? (c.E - lane + 31) / 32 : 0;
            g = 0;
        } else {
            const int i = lane % c.lanes;
            g = lane / c.lanes;
            first = g * c.per + i;
            step = c.lanes;
            n = g < c.G && i < c.per ? (c.per - i + c.lanes - 1) / c.lanes : 0;
        }
    }
};

template <bool BF16>
MOK_DEV float load_logit(const void *row, int e) {
    return BF16 ? bf16_to_f32(static_cast<const uint16_t *>(row)[e])
                : static_cast<const float *>(row)[e];
}

MOK_DEV float sigmoid32(float l) { return 1.0f / (1.0f + expf(-l)); }
// e^x in softmaxes whose largest x is 0; -inf gives 0
MOK_DEV float exp_below(float l, float top) { return expf(l - (isinf(top) ? 0.0f : top)); }

// Bound of the error of an fp32 score, relative to the row's largest.
// sigmoid: expf 2 ulp (2^-22), the sum and the quotient half an ulp each: below 2^-21.
// softmax: expf 2^-22, its argument's rounding 2^-24 |x| e^x <= 0.37 2^-24, the sum over up to 64
// values a lane and 5 steps across lanes 69 x 2^-24 and its terms' own 2^-22 + 7 x 2^-24, the
// reciprocal and the product 2^-23: below 96 x 2^-24 < 2^-17.
MOK_DEV float score_error(const RouterShape &c) {
    return c.softmax ? 7.62939453125e-6f : 4.76837158203125e-7f;
}

// the better of two (key, id), the lower id among equals
MOK_DEV void better(double &k, int &id, double k2, int id2) {
    if (k2 > k || (k2 == k && id2 < id)) {
        k = k2;
        id = id2;
    }
}

// The choice in 64 bits: lane k < K gets the k-th expert's id.
template <int PER, bool BF16>
__device__ __noinline__ int choose_exact(const RouterShape &c, const void *row, const float *bias,
                                         int lane) {
    const Held h(c, lane);
    double key[PER];
    double b1 = -INFINITY, b2 = -INFINITY;  // the lane's two largest s + bias
    double inv = 1.0;
    float top = -INFINITY;
    if (c.softmax) {
        for (int j = 0; j < h.n; ++j) top = fmaxf(top, load_logit<BF16>(row, h.first + j * h.step));
        top = warp_max(top);
        double den = 0.0;
        for (int j = 0; j < h.n; ++j) {
            const float l = load_logit<BF16>(row, h.first + j * h.step);
            if (l > -INFINITY) den += exp((double)l - (double)top);
        }
        for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xFFFFFFFFu, den, o);
        inv = 1.0 / den;
    }
    for (int j = 0; j < h.n; ++j) {
        const int e = h.first + j * h.step;
        const float l = load_logit<BF16>(row, e);
        const bool off = !(l > -INFINITY);
        const double s = off         ? 0.0
                         : c.softmax ? exp((double)l - (double)top) * inv
                                     : 1.0 / (1.0 + exp(-(double)l));
        const double v = s + (bias != nullptr ? (double)bias[e] : 0.0);
        // a score that is no number (of a logit of +inf) has to be taken by someone, last
        key[j] = off || v != v ? -1e300 : bias != nullptr ? v : (double)l;
        if (!off) {
            if (v > b1) {
                b2 = b1;
                b1 = v;
            } else if (v > b2) {
                b2 = v;
            }
        }
    }
    bool kept = h.n > 0;
    if (c.G > 1) {
        for (int o = 1; o < c.lanes; o <<= 1) {
            const double o1 = __shfl_xor_sync(0xFFFFFFFFu, b1, o);
            const double o2 = __shfl_xor_sync(0xFFFFFFFFu, b2, o);
            const double lo = b1 < o1 ? b1 : o1, hi = b2 > o2 ? b2 : o2;
            b1 = b1 > o1 ? b1 : o1;
            b2 = lo > hi ? lo : hi;
        }
        const double score = c.top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
        int rank = 0;
        for (int g = 0; g < c.G; ++g) {
            const double other = __shfl_sync(0xFFFFFFFFu, score, g * c.lanes);
            if (other > score || (other == score && g < h.g)) ++rank;
        }
        kept = kept && rank < c.keep;
    }
    int mine = 0;
    uint64_t taken = 0;  // the lane's chosen
    for (int k = 0; k < c.K; ++k) {
        double best = -INFINITY;
        int id = INT32_MAX, at = 0;
        if (kept)
            for (int j = 0; j < h.n; ++j)
                if (((taken >> j) & 1u) == 0 && key[j] > best) {
                    best = key[j];
                    id = h.first + j * h.step;
                    at = j;
                }
        const int own = id;
        for (int o = 16; o > 0; o >>= 1)
            better(best, id, __shfl_xor_sync(0xFFFFFFFFu, best, o),
                   __shfl_xor_sync(0xFFFFFFFFu, id, o));
        if (own == id && id != INT32_MAX) taken |= 1ull << at;
        if (lane == k) mine = id == INT32_MAX ? 0 : id;
    }
    return mine;
}

// Unscaled weight of a chosen logit among the K chosen (lane k < K holds the k-th): its score, or
// its share of the chosen scores. The shares of scores that all round to nothing in fp32 are those of
// the scores times e^-t.
MOK_DEV float chosen_weight(const RouterShape &c, int lane, float l, float top, float inv) {
    const bool in = lane < c.K && l > -INFINITY;
    if (!c.renorm)
        return !in ? 0.0f : c.softmax ? exp_below(l, top) * inv : sigmoid32(l);
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
    return total > 0.0f ? a / total : total == 0.0f ? 0.0f : total;
}

struct RouterFwd {
    RouterShape c;
    const void *logits;
    const float *bias;
    int32_t *idx;
    float *w;
    int32_t *count_part;  // [blocks][E], or nullptr
    float *sum_part;      // [blocks][E], or nullptr
    int64_t chunk;        // tokens of a block
};

// PER experts a lane
template <int PER, bool BF16>
__global__ void __launch_bounds__(32 * ROUTER_WARPS) router_kernel(const RouterFwd a) {
    extern __shared__ uint32_t router_smem[];
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
    const Held h(c, lane);
    const bool scored = a.bias != nullptr || (c.G > 1 && c.top == 2);  // the choice goes by scores
    const bool row_scores = scored || a.sum_part != nullptr || (c.softmax && !c.renorm);
    float acc[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) acc[j] = 0.0f;
    const int64_t t1 = (blockIdx.x + 1) * a.chunk < c.T ? (blockIdx.x + 1) * a.chunk : c.T;
    for (int64_t t = blockIdx.x * a.chunk + warp; t < t1; t += ROUTER_WARPS) {
        const void *row = static_cast<const char *>(a.logits) + t * c.ld * (BF16 ? 2 : 4);
        float v[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j)
            v[j] = j < h.n ? load_logit<BF16>(row, h.first + j * h.step) : -INFINITY;
        // scores, and what the choice goes by
        float top = -INFINITY, inv = 0.0f, most = 0.0f;
        uint32_t key[PER];
        float b1 = -INFINITY, b2 = -INFINITY;
        if (row_scores) {
            float s[PER];
            if (c.softmax) {
#pragma unroll
                for (int j = 0; j < PER; ++j) top = fmaxf(top, v[j]);
                top = warp_max(top);
                float den = 0.0f;
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    s[j] = exp_below(v[j], top);
                    den += s[j];
                }
                den = warp_sum(den);
                inv = den > 0.0f ? 1.0f / den : den == 0.0f ? 0.0f : den;
#pragma unroll
                for (int j = 0; j < PER; ++j) s[j] *= inv;
            } else {
#pragma unroll
                for (int j = 0; j < PER; ++j) s[j] = sigmoid32(v[j]);
            }
#pragma unroll
            for (int j = 0; j < PER; ++j) acc[j] += s[j];
            if (scored) {
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    most = fmaxf(most, s[j]);
                    if (a.bias != nullptr && j < h.n) s[j] += a.bias[h.first + j * h.step];
                    if (v[j] == -INFINITY) s[j] = -INFINITY;
                    b2 = fmaxf(b2, fminf(b1, s[j]));
                    b1 = fmaxf(b1, s[j]);
                    if (a.bias != nullptr) v[j] = s[j];
                }
                most = warp_max(most);
            }
        }
        if (!scored) {
#pragma unroll
            for (int j = 0; j < PER; ++j) b1 = fmaxf(b1, v[j]);
        }
        bool close = false, kept = h.n > 0;
        const float err = scored ? score_error(c) * most : 0.0f;
        if (c.G > 1) {
            for (int o = 1; o < c.lanes; o <<= 1) {
                const float o1 = __shfl_xor_sync(0xFFFFFFFFu, b1, o);
                const float o2 = __shfl_xor_sync(0xFFFFFFFFu, b2, o);
                b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
                b1 = fmaxf(b1, o1);
            }
            const float score = c.top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
            int rank = 0;
            for (int g = 0; g < c.G; ++g) {
                const float other = __shfl_sync(0xFFFFFFFFu, score, g * c.lanes);
                if (other > score || (other == score && g < h.g)) ++rank;
            }
            kept = kept && rank < c.keep;
            if (scored && c.keep < c.G) {
                // the least kept and the largest other score
                const uint32_t o = order_of(score);
                const float low = of_order(__reduce_min_sync(0xFFFFFFFFu, kept ? o : 0xFFFFFFFFu));
                const float high = of_order(__reduce_max_sync(
                    0xFFFFFFFFu, h.n > 0 && !kept ? o : ORDER_MASKED));
                close = high > -INFINITY &&
                        !(low - high > 4.0f * err + 4.76837158203125e-7f * fmaxf(fabsf(low), fabsf(high)));
            }
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) key[j] = kept && j < h.n ? order_of(v[j]) : 0u;
        uint32_t best = 0u;
        int bj = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (key[j] > best) {
                best = key[j];
                bj = j;
            }
        uint32_t sel = 0u, next = 0u;  // lane k: the k-th key, and the one after it
        int id = 0, next_id = 0;
        // with a bias one round more, for the distance between the last chosen and the first left
        const int rounds = a.bias != nullptr ? c.K + 1 : c.K;
        for (int k = 0; k < rounds; ++k) {
            const uint32_t most_key = __reduce_max_sync(0xFFFFFFFFu, best);
            if (k > 0 && lane == k - 1) next = most_key;
            if (most_key == 0u) break;  // fewer experts than rounds
            const uint32_t cand =
                best == most_key ? (uint32_t)(h.first + bj * h.step) : 0xFFFFFFFFu;
            const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, cand);
            if (k > 0 && lane == k - 1) next_id = (int)e;
            if (lane == k && k < c.K) {
                sel = most_key;
                id = (int)e;
            }
            if (cand == e) {
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (j == bj) key[j] = 0u;
                best = 0u;
                bj = 0;
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (key[j] > best) {
                        best = key[j];
                        bj = j;
                    }
            }
        }
        if (a.bias != nullptr && lane < c.K && next > ORDER_MASKED) {
            const float x = of_order(sel), y = of_order(next);
            if (!(x - y > 2.0f * err + 2.384185791015625e-7f * fmaxf(fabsf(x), fabsf(y))))
                close = close || load_logit<BF16>(row, id) != load_logit<BF16>(row, next_id) ||
                        a.bias[id] != a.bias[next_id];
        }
        if (__any_sync(0xFFFFFFFFu, close)) id = choose_exact<PER, BF16>(c, row, a.bias, lane);
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
            if (j < h.n) sums[warp * c.E + h.first + j * h.step] = acc[j];
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

// The blocks' counts and sums, added in order: 32 experts a block, each warp a slice of the parts.
constexpr int LOAD_SLICES = 16;
__global__ void __launch_bounds__(32 * LOAD_SLICES)
    router_load_kernel(const int32_t *count_part, const float *sum_part, int parts, int E,
                       int32_t *counts, float *score_sum) {
    __shared__ float fs[LOAD_SLICES][32];
    __shared__ int32_t is[LOAD_SLICES][32];
    let_next_start();
    wait_for_previous();
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane;
    float s = 0.0f;
    int32_t n = 0;
    if (e < E) {
        if (counts != nullptr)
#pragma unroll 8
            for (int p = slice; p < parts; p += LOAD_SLICES) n += count_part[(int64_t)p * E + e];
        if (score_sum != nullptr)
#pragma unroll 8
            for (int p = slice; p < parts; p += LOAD_SLICES) s += sum_part[(int64_t)p * E + e];
    }
    fs[slice][lane] = s;
    is[slice][lane] = n;
    __syncthreads();
    if (slice != 0 || e >= E) return;
    s = 0.0f;
    n = 0;
#pragma unroll
    for (int k = 0; k < LOAD_SLICES; ++k) {
        s += fs[k][lane];
        n += is[k][lane];
    }
    if (counts != nullptr) counts[e] = n;
    if (score_sum != nullptr) score_sum[e] = s;
}

struct RouterBwd {
    RouterShape c;
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

// One warp per token, experts l, l + 32, .. of a lane. The row is written as if nothing were chosen,
// then the chosen entries again, each from all that it gets, by the lane that holds it.
template <int PER, bool BF16>
__global__ void __launch_bounds__(32 * ROUTER_WARPS) router_backward_kernel(const RouterBwd a) {
    const RouterShape &c = a.c;
    const int lane = threadIdx.x & 31;
    let_next_start();
    wait_for_previous();
    const int64_t t = (int64_t)blockIdx.x * ROUTER_WARPS + (threadIdx.x >> 5);
    if (t >= c.T) return;
    const int64_t at = t * c.ld * (BF16 ? 2 : 4);
    const void *row = static_cast<const char *>(a.logits) + at;
    void *out = static_cast<char *>(a.dlogits) + at;
    int id = -1;
    float dw = 0.0f, l = -INFINITY;
    if (lane < c.K) {
        id = a.idx[t * c.K + lane];
        dw = a.dw[t * c.K + lane];
        if (id < 0 || id >= c.E) {
            raise_status(a.status, MOK_ERR_DEVICE_INVARIANT);
            id = -1;
        } else {
            l = load_logit<BF16>(row, id);
        }
    }
    const bool dense = a.dsum != nullptr || (c.softmax && !c.renorm);
    float s[PER];
    float top = -INFINITY, inv = 0.0f, mean = 0.0f;  // mean: of dsum under the scores
    if (dense) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = lane + 32 * j;
            s[j] = e < c.E ? load_logit<BF16>(row, e) : -INFINITY;
        }
        if (c.softmax) {
#pragma unroll
            for (int j = 0; j < PER; ++j) top = fmaxf(top, s[j]);
            top = warp_max(top);
            float den = 0.0f;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                s[j] = exp_below(s[j], top);
                den += s[j];
            }
            den = warp_sum(den);
            inv = den > 0.0f ? 1.0f / den : den == 0.0f ? 0.0f : den;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                s[j] *= inv;
                const int e = lane + 32 * j;
                if (a.dsum != nullptr && e < c.E) mean = fmaf(s[j], a.dsum[e], mean);
            }
            mean = warp_sum(mean);
        }
    }
    const float wt = chosen_weight(c, lane, l, top, inv);
    // what a chosen logit gets through its weight; a masked one nothing, whatever dw holds
    float add = 0.0f;
    const bool live = l > -INFINITY;
    const float m = warp_sum(live ? dw * wt : 0.0f);
    if (live) {
        if (c.softmax) {
            add = c.scale * wt * (c.renorm ? dw - m : dw);
        } else {
            const float rest = 1.0f / (1.0f + expf(l));  // 1 - s
            add = c.scale * wt * rest * (c.renorm ? dw - m : dw);
        }
    }
    // a softmax's chosen weights take from all
    const float all = c.softmax && !c.renorm ? c.scale * m + mean : mean;
    const auto base = [&](float score, float logit, int e) {
        if (c.softmax) return score * ((a.dsum != nullptr ? a.dsum[e] : 0.0f) - all);
        return logit > -INFINITY ? a.dsum[e] * score * (1.0f / (1.0f + expf(logit))) : 0.0f;
    };
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = lane + 32 * j;
        if (e < c.E)
            s[j] = !dense ? 0.0f : c.softmax ? base(s[j], 0.0f, e) : base(sigmoid32(s[j]), s[j], e);
    }
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
    if (dense && id >= 0)
        add += c.softmax ? (live ? base(exp_below(l, top) * inv, l, id) : 0.0f)
                         : base(sigmoid32(l), l, id);
    __syncwarp();  // d_logits may be logits: all of the row has been read
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = lane + 32 * j;
        if (e < c.E) store_logit<BF16>(out, e, s[j]);
    }
    __syncwarp();
    if (id >= 0) store_logit<BF16>(out, id, add);
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

RouterShape shape_of(const mok_router_config &c) {
    RouterShape s = {};
    s.T = c.T;
    s.ld = c.ld;
    s.E = c.E;
    s.K = c.K;
    s.G = c.groups;
    s.keep = c.topk_groups;
    s.top = c.group_top;
    s.per = c.E / c.groups;
    s.lanes = 32;
    while (s.lanes * c.groups > 32) s.lanes /= 2;
    s.softmax = c.score == MOK_SCORE_SOFTMAX;
    s.renorm = c.renormalize != 0;
    s.scale = c.scale;
    return s;
}

// experts a lane
int held_of(const RouterShape &s) {
    return s.G == 1 ? (s.E + 31) / 32 : (s.per + s.lanes - 1) / s.lanes;
}

int64_t chunk_of(int64_t T) {
    const int64_t n = (T + ROUTER_BLOCKS - 1) / ROUTER_BLOCKS;
    return round_up(n > 1 ? n : 1, ROUTER_WARPS);
}
int64_t blocks_of(int64_t T) { return (T + chunk_of(T) - 1) / chunk_of(T); }

#define MOK_ROUTER_PER(per, F, MOST)            \
    (per <= 1    ? F(1)                         \
     : per <= 2  ? F(2)                         \
     : per <= 4  ? F(4)                         \
     : per <= 8  ? F(8)                         \
     : per <= 16 ? F(16)                        \
     : per <= 32 ? F(32)                        \
                 : F(MOST))

cudaError_t launch_router(const RouterFwd &a, bool bf16, cudaStream_t s) {
    const int per = held_of(a.c);
    const unsigned grid = (unsigned)blocks_of(a.c.T);
    const int smem = a.sum_part != nullptr     ? (1 + ROUTER_WARPS) * a.c.E * 4
                     : a.count_part != nullptr ? a.c.E * 4
                                               : 0;
#define MOK_F(P)                                                                             \
    (bf16 ? launch_edge(router_kernel<P, true>, grid, 32 * ROUTER_WARPS, smem, 1, s, a)      \
          : launch_edge(router_kernel<P, false>, grid, 32 * ROUTER_WARPS, smem, 1, s, a))
    return MOK_ROUTER_PER(per, MOK_F, 64);  // 17 groups of 60 experts: one lane a group
#undef MOK_F
}

cudaError_t launch_router_backward(const RouterBwd &a, bool bf16, cudaStream_t s) {
    const int per = (a.c.E + 31) / 32;
    const unsigned grid = (unsigned)((a.c.T + ROUTER_WARPS - 1) / ROUTER_WARPS);
#define MOK_F(P)                                                                                  \
    (bf16 ? launch_edge(router_backward_kernel<P, true>, grid, 32 * ROUTER_WARPS, 0, 1, s, a)     \
          : launch_edge(router_backward_kernel<P, false>, grid, 32 * ROUTER_WARPS, 0, 1, s, a))
    return MOK_ROUTER_PER(per, MOK_F, 32);
#undef MOK_F
}

size_t part_bytes(const mok_router_config &c) {
    return (size_t)round_up(blocks_of(c.T) * c.E * 4, 256);
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
    const int parts = (int)blocks_of(c->T);
    int32_t *cp = counts != nullptr ? (int32_t *)ws : nullptr;
    float *sp = score_sum != nullptr ? (float *)((char *)ws + part_bytes(*c)) : nullptr;
    if (c->T > 0) {
        const RouterFwd a{shape_of(*c), logits, bias, topk_idx, topk_w, cp, sp, chunk_of(c->T)};
        MOK_OP_LAUNCH(OP_ROUTER, 1, launch_router(a, c->dtype == MOK_DTYPE_BF16, stream));
    }
    if (load)
        MOK_OP_LAUNCH(OP_ROUTER, 1,
                      launch_edge(router_load_kernel, (unsigned)((c->E + 31) / 32), 32 * LOAD_SLICES,
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
    const RouterBwd a{shape_of(*c), logits, topk_idx, d_topk_w, d_score_sum, d_logits, status};
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

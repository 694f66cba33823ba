// adamw.cu -- an AdamW step over many tensors in one launch, states in fp32 or in MXFP8.
//
// Per element (fp32):  m = b1 m + (1-b1) g,  v = b2 v + (1-b2) g^2,
//                      p = p (1 - lr wd) - lr/(1-b1^t) m / (sqrt(v)/sqrt(1-b2^t) + eps).
// Every array is read once and written once, so HBM traffic is the floor: with fp32 master
// parameters, a bf16 copy and bf16 gradients, 28 bytes per element with fp32 states and
// 16.125 with MXFP8 states. Measured on 403 M elements: 1588 us with fp32 states (7.1 TB/s;
// a plain copy reaches 6.8), 993 us with MXFP8 states (6.5 TB/s; about 65 instructions an
// element keep the issue slots as busy as the memory).
//
// The tensor list travels in the kernel's parameters (no device-side table to allocate, copy
// or keep alive, and a captured graph holds its own). A block takes one chunk of 1024
// elements of a tensor, found by a binary search over the tensors' first chunks (blocks that
// loop over chunks drift apart and read DRAM less in order: 403 M elements with fp32 states 1875
// against 1588 us); each thread owns
// 8 consecutive elements, so four threads hold a 32-element MXFP8 block and its largest
// magnitude takes two shuffles.
#include <cmath>

#include "common.cuh"
#include "ops_internal.h"

namespace mok {
namespace {

constexpr int TPB = 128;  // (403 M elements, MXFP8 states: 1017 us with 256 threads, 993 with 128)
constexpr int PER = 8;             // elements per thread
constexpr int CHUNK = TPB * PER;   // elements per block and step

struct TensorDesc {
    void *p, *copy;
    const void *g;
    void *m, *v;
    uint8_t *ms, *vs;
    int64_t n;
    int64_t base;    // element number of the tensor's first element
    uint32_t first;  // its first chunk
    float decay;     // 1 - lr weight_decay (weight_decay where a clock has lr)
};

struct Scalars {
    float b1, a1, b2, a2;  // beta and 1 - beta
    float step;            // lr / (1 - beta1^t)
    float inv_root;        // 1 / sqrt(1 - beta2^t)
    float eps;
    uint32_t seed_lo, seed_hi;
    int n_tensors;
    uint32_t n_chunks;
    const float *gscale;
    const mok_adamw_clock *clock;  // nullptr, or where step, inv_root, lr and the seed's step are
};

template <int NT>
struct Params {
    Scalars s;
    TensorDesc t[NT];
};
// tensors of one launch: the parameters are copied at each launch, so short lists take less
constexpr int NT_SMALL = 8, NT_MID = 64, NT_LARGE = 400;
static_assert(sizeof(Params<NT_LARGE>) <= 32764, "kernel parameters");

// the MurmurHash3 finaliser
MOK_DEV uint32_t mix32(uint32_t h) {
    h ^= h >> 16;
    h *= 0x85EBCA6Bu;
    h ^= h >> 13;
    h *= 0xC2B2AE35u;
    return h ^ (h >> 16);
}

// FULL: the thread's 8 elements all exist
template <bool F32, bool FULL>
MOK_DEV void load8(const void *p, int64_t i, int64_t n, float (&v)[PER]) {
    if (FULL || i + PER <= n) {
        if (F32) {
            const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
            const float4 b =
                *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 a =
                *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[2 * q] = bf16_lo(w[q]);
                v[2 * q + 1] = bf16_hi(w[q]);
            }
        }
    } else {
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const bool ok = i + q < n;
            v[q] = !ok ? 0.f
                   : F32 ? static_cast<const float *>(p)[i + q]
                         : bf16_to_f32(static_cast<const uint16_t *>(p)[i + q]);
        }
    }
}

template <bool FULL>
MOK_DEV void store8_f32(void *p, int64_t i, int64_t n, const float (&v)[PER]) {
    float *o = static_cast<float *>(p) + i;
    if (FULL || i + PER <= n) {
        *reinterpret_cast<float4 *>(o) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int q = 0; q < PER; ++q)
            if (i + q < n) o[q] = v[q];
    }
}

template <bool FULL>
MOK_DEV void store8_u16(void *p, int64_t i, int64_t n, const uint32_t (&w)[PER / 2]) {
    uint16_t *o = static_cast<uint16_t *>(p) + i;
    if (FULL || i + PER <= n) {
        *reinterpret_cast<uint4 *>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int q = 0; q < PER; ++q)
            if (i + q < n) o[q] = (uint16_t)(w[q / 2] >> (16 * (q & 1)));
    }
}

// fp32 -> bf16, rounded up with probability r / 2^16 of what is cut off (r: 16 random bits);
// infinities and NaN as they are
MOK_DEV uint32_t bf16_stochastic(float f, uint32_t r) {
    const uint32_t b = __float_as_uint(f);
    if ((b & 0x7F800000u) == 0x7F800000u) return f32_to_bf16(f);
    return (b + r) >> 16;
}

// 8 E4M3 codes to fp32, without their scale
MOK_DEV void decode8(uint2 q, float (&v)[PER]) {
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int j = 0; j < PER; j += 2) {
        uint32_t h;
        const uint16_t two = (uint16_t)(w[j / 4] >> (8 * (j & 3)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}\n"
            : "=f"(v[j]), "=f"(v[j + 1])
            : "r"(h));
    }
}

// square root, and the larger of two that is NaN where either is
MOK_DEV float sqrt_approx(float x) {
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
MOK_DEV float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <bool FULL>
MOK_DEV uint2 load8_u8(const void *p, int64_t i, int64_t n) {
    const uint8_t *s = static_cast<const uint8_t *>(p) + i;
    if (FULL || i + PER <= n) return *reinterpret_cast<const uint2 *>(s);
    uint2 q = make_uint2(0, 0);
#pragma unroll
    for (int j = 0; j < PER; ++j)
        if (i + j < n) (j < 4 ? q.x : q.y) |= (uint32_t)s[j] << (8 * (j & 3));
    return q;
}
template <bool FULL>
MOK_DEV void store8_u8(void *p, int64_t i, int64_t n, uint2 q) {
    uint8_t *o = static_cast<uint8_t *>(p) + i;
    if (FULL || i + PER <= n) {
        *reinterpret_cast<uint2 *>(o) = q;
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (i + j < n) o[j] = (uint8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
    }
}

// The MXFP8 encoder. A magnitude y = |x| / scale <= 448 keeps 4 significant bits (E4M3
// normals, y >= 2^-6): adding 20 bits below the last kept one to its fp32 pattern and cutting
// there rounds it, the carry moving into the exponent. Subnormals have the step 2^-9, which
// is the step of the octave [2^-6, 2^-5): 2^-6 is added before the cut and taken off after it.
// The result is an E4M3 value in fp32, sign and all, which the hardware conversion packs as
// it is, two at a time. The random bits are (r + 1/2) / 2^16 of a step.
template <bool SR>
MOK_DEV uint32_t round_bits(uint32_t b, uint32_t r16) {
    return (b + (SR ? (r16 << 4) + 8u : 0x7FFFFu + ((b >> 20) & 1u))) & 0xFFF00000u;
}
template <bool SR, bool POSITIVE>
MOK_DEV float round_low(float y, uint32_t r16) {
    if (POSITIVE && y > 0.f) y = fmaxf(y, 0.001953125f);  // the least code, not zero
    const float off = __uint_as_float((__float_as_uint(y) & 0x80000000u) | 0x3C800000u);  // 2^-6
    const bool low = fabsf(y) < 0.015625f;
    y = __uint_as_float(round_bits<SR>(__float_as_uint(low ? y + off : y), r16));
    return low ? y - off : y;
}

// codes of this thread's 8 values; the 4 threads of a 32-element block share the scale, which
// every one of them returns. Few threads hold a subnormal (a value under 1/28672 of its block's
// largest), so the steps for those are behind a branch on the thread's least magnitude.
template <bool SR, bool POSITIVE>
MOK_DEV uint2 encode8(const float (&x)[PER], const uint32_t (&r16)[PER], uint32_t *scale) {
    float top = 0.f, least = __uint_as_float(0x7F800000u);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const float a = POSITIVE ? x[j] : fabsf(x[j]);
        top = max_nan(top, a);
        least = fminf(least, a);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const uint32_t tb = __float_as_uint(top) & 0x7FFFFFFFu;
    const int ef = (int)(tb >> 23);
    // the least power of two with top / scale <= 448 = 1.75 2^8
    int sb = ef - 8 + ((tb & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    sb = sb < 0 ? 0 : sb;
    const float inv = mx_inv_scale((uint32_t)sb);
    float y[PER];
    if (least * inv >= 0.015625f) {
#pragma unroll
        for (int j = 0; j < PER; ++j)
            y[j] = __uint_as_float(round_bits<SR>(__float_as_uint(x[j] * inv), r16[j]));
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) y[j] = round_low<SR, POSITIVE>(x[j] * inv, r16[j]);
    }
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < PER; j += 2) q[j / 2] = e4m3x2(y[j], y[j + 1]);
    const bool bad = ef == 255;  // an infinity or a NaN: the block is NaN
    *scale = bad ? 255u : (uint32_t)sb;
    return bad ? make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu)
               : make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}

// this thread's 8 elements from element i of tensor t
template <bool PF32, bool GF32, bool S8, bool SR, bool FULL>
MOK_DEV void update8(const Scalars &S, const TensorDesc &t, float decay, int64_t i, float gs) {
    const int64_t n = t.n;
    float p[PER], g[PER], m[PER], v[PER];
    load8<PF32, FULL>(t.p, i, n, p);
    load8<GF32, FULL>(t.g, i, n, g);
    // the old states times beta
    if (S8) {
        const bool in = FULL || i < n;
        const float sm = in ? mx_scale(t.ms[i >> 5]) * S.b1 : 0.f;
        const float sv = in ? mx_scale(t.vs[i >> 5]) : 0.f;
        decode8(load8_u8<FULL>(t.m, i, n), m);
        decode8(load8_u8<FULL>(t.v, i, n), v);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            m[j] *= sm;
            v[j] *= sv;
            v[j] *= S.b2 * v[j];
        }
    } else {
        load8<true, FULL>(t.m, i, n, m);
        load8<true, FULL>(t.v, i, n, v);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            m[j] *= S.b1;
            v[j] *= S.b2;
        }
    }
    uint32_t rp[PER], rm[PER], rv[PER];
    if (SR) {
        const int64_t e = t.base + i;  // 8 elements from a multiple of 8: one high word
        const uint32_t key = mix32(mix32((uint32_t)((uint64_t)e >> 32) ^ S.seed_lo) ^ S.seed_hi);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const uint32_t h = mix32(((uint32_t)e + j) ^ key);
            rm[j] = h & 0xFFFFu;
            rv[j] = h >> 16;
            rp[j] = PF32 ? 0u : mix32(h + 0x9E3779B9u) >> 16;
        }
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) rm[j] = rv[j] = rp[j] = 0;
    }
    // square root and reciprocal are the hardware's (2^-22 of a value): p moves by lr of
    // what they give, sqrt(v) is then rounded to 4 bits
    float s[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const float gj = g[j] * gs;
        // two roundings, as the formula reads: a code next to its rounding threshold then comes out
        // as in any fp32 evaluation (fused, some 200 of 403 M codes did not, and it was no faster)
        m[j] = __fadd_rn(m[j], __fmul_rn(S.a1, gj));
        v[j] = fmaf(S.a2, gj * gj, v[j]);
        s[j] = sqrt_approx(v[j]);
        p[j] = fmaf(p[j], decay, -S.step * __fdividef(m[j], fmaf(s[j], S.inv_root, S.eps)));
    }
    if (PF32) {
        store8_f32<FULL>(t.p, i, n, p);
        if (t.copy != nullptr) {
            const uint32_t w[4] = {pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]),
                                   pack_bf16x2(p[4], p[5]), pack_bf16x2(p[6], p[7])};
            store8_u16<FULL>(t.copy, i, n, w);
        }
    } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < PER; j += 2)
            w[j / 2] = SR ? bf16_stochastic(p[j], rp[j]) |
                                (bf16_stochastic(p[j + 1], rp[j + 1]) << 16)
                          : pack_bf16x2(p[j], p[j + 1]);
        store8_u16<FULL>(t.p, i, n, w);
    }
    if (S8) {
        if (!FULL && i + PER > n) {  // what lies past the tensor's end counts for nothing
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (i + j >= n) m[j] = s[j] = 0.f;
        }
        uint32_t sm, sv;
        const uint2 qm = encode8<SR, false>(m, rm, &sm);
        const uint2 qv = encode8<SR, true>(s, rv, &sv);
        store8_u8<FULL>(t.m, i, n, qm);
        store8_u8<FULL>(t.v, i, n, qv);
        if ((threadIdx.x & 3) == 0 && (FULL || i < n)) {
            t.ms[i >> 5] = (uint8_t)sm;
            t.vs[i >> 5] = (uint8_t)sv;
        }
    } else {
        store8_f32<FULL>(t.m, i, n, m);
        store8_f32<FULL>(t.v, i, n, v);
    }
}

// The step that follows: one thread, in 64 bits as the host has it.
__global__ void advance_kernel(mok_adamw_clock *c, double b1, double b2, int *status) {
    const int64_t t = c->step + 1;
    const double lr = c->lr;
    const bool ok = t >= 1 && lr >= 0 && isfinite(lr);
    if (!ok) raise_status(status, MOK_ERR_DEVICE_INVARIANT);
    c->step = t;
    c->step_lr = ok ? (float)lr : 0.f;  // a step of nothing
    c->step_size = ok ? (float)(lr / (1.0 - pow(b1, (double)t))) : 0.f;
    c->inv_root = ok ? (float)(1.0 / sqrt(1.0 - pow(b2, (double)t))) : 1.f;
}

template <int NT, bool PF32, bool GF32, bool S8, bool SR, bool CLOCK>
__global__ void __launch_bounds__(TPB)
    adamw_kernel(const __grid_constant__ Params<NT> P) {
    const float gs = P.s.gscale != nullptr ? *P.s.gscale : 1.0f;
    const uint32_t c = blockIdx.x;
    int lo = 0, hi = P.s.n_tensors - 1;  // the last tensor whose first chunk is <= c
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (P.t[mid].first <= c) lo = mid; else hi = mid - 1;
    }
    const TensorDesc &t = P.t[lo];
    const int64_t i0 = (int64_t)(c - t.first) * CHUNK, i = i0 + (int64_t)threadIdx.x * PER;
    const auto update = [&](const Scalars &S, float decay) {
        if (i0 + CHUNK <= t.n)
            update8<PF32, GF32, S8, SR, true>(S, t, decay, i, gs);
        else
            update8<PF32, GF32, S8, SR, false>(S, t, decay, i, gs);
    };
    if constexpr (CLOCK) {
        Scalars S = P.s;
        const mok_adamw_clock k = *S.clock;
        S.step = k.step_size;
        S.inv_root = k.inv_root;
        const uint64_t seed = ((uint64_t)S.seed_hi << 32 | S.seed_lo) + (uint64_t)k.step * k.seed_stride;
        S.seed_lo = (uint32_t)seed;
        S.seed_hi = (uint32_t)(seed >> 32);
        update(S, fmaf(-k.step_lr, t.decay, 1.0f));
    } else {
        update(P.s, t.decay);
    }
}

template <bool CLOCK, int NT>
cudaError_t launch_group(const mok_adamw_config &c, Params<NT> &P, cudaStream_t s) {
    const bool pf = c.p_dtype == MOK_DTYPE_F32, gf = c.g_dtype == MOK_DTYPE_F32;
    const bool s8 = c.state == MOK_STATE_MXFP8;
    const bool sr = (c.flags & MOK_ADAMW_STOCHASTIC) != 0 && (s8 || !pf);
#define MOK_ADAMW_CASE(p_, g_, s_, r_)                                                          \
    if (pf == p_ && gf == g_ && s8 == s_ && sr == r_) {                                         \
        adamw_kernel<NT, p_, g_, s_, r_, CLOCK><<<P.s.n_chunks, TPB, 0, s>>>(P);                \
        return cudaGetLastError();                                                              \
    }
    MOK_ADAMW_CASE(true, true, false, false);
    MOK_ADAMW_CASE(true, false, false, false);
    MOK_ADAMW_CASE(true, true, true, false);
    MOK_ADAMW_CASE(true, false, true, false);
    MOK_ADAMW_CASE(true, true, true, true);
    MOK_ADAMW_CASE(true, false, true, true);
    MOK_ADAMW_CASE(false, true, false, false);
    MOK_ADAMW_CASE(false, false, false, false);
    MOK_ADAMW_CASE(false, true, false, true);
    MOK_ADAMW_CASE(false, false, false, true);
    MOK_ADAMW_CASE(false, true, true, false);
    MOK_ADAMW_CASE(false, false, true, false);
    MOK_ADAMW_CASE(false, true, true, true);
    MOK_ADAMW_CASE(false, false, true, true);
#undef MOK_ADAMW_CASE
    return cudaErrorInvalidValue;
}

// tensors [t0, t1) as one launch; *base: element number of the first, advanced past the last
template <bool CLOCK, int NT>
cudaError_t step_group(const mok_adamw_config &c, const mok_adamw_tensor *ts, int t0, int t1,
                       const mok_adamw_clock *clock, const float *gscale, int64_t *base,
                       cudaStream_t s) {
    Params<NT> P;
    const double bc1 = 1.0 - pow(c.beta1, (double)c.step);
    const double bc2 = 1.0 - pow(c.beta2, (double)c.step);
    P.s.b1 = (float)c.beta1;
    P.s.a1 = (float)(1.0 - c.beta1);
    P.s.b2 = (float)c.beta2;
    P.s.a2 = (float)(1.0 - c.beta2);
    P.s.step = (float)(c.lr / bc1);
    P.s.inv_root = (float)(1.0 / sqrt(bc2));
    P.s.eps = (float)c.eps;
    P.s.seed_lo = (uint32_t)c.seed;
    P.s.seed_hi = (uint32_t)(c.seed >> 32);
    P.s.gscale = gscale;
    P.s.clock = clock;
    int n = 0;
    int64_t chunks = 0;
    for (int i = t0; i < t1; ++i) {
        const mok_adamw_tensor &t = ts[i];
        if (t.n == 0) continue;
        const float decay = (float)(CLOCK ? t.weight_decay : 1.0 - c.lr * t.weight_decay);
        P.t[n++] = TensorDesc{t.p, t.copy, t.g, t.m, t.v, t.m_scale, t.v_scale, t.n, *base,
                              (uint32_t)chunks, decay};
        chunks += (t.n + CHUNK - 1) / CHUNK;
        *base += (t.n + 31) & ~(int64_t)31;
    }
    if (n == 0) return cudaSuccess;
    if (chunks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    P.s.n_tensors = n;
    P.s.n_chunks = (uint32_t)chunks;
    return launch_group<CLOCK, NT>(c, P, s);
}

mok_status check_step(const mok_adamw_config *c, const mok_adamw_tensor *tensors,
                      int32_t n_tensors, int **status) {
    mok_status st = mok_check_adamw_config(c);
    if (st != MOK_OK) return st;
    if ((st = current_device_status_word(status)) != MOK_OK) return st;
    if (n_tensors < 0 || (n_tensors > 0 && tensors == nullptr)) return MOK_ERR_INVALID_ARG;
    const bool s8 = c->state == MOK_STATE_MXFP8;
    for (int32_t i = 0; i < n_tensors; ++i) {
        const mok_adamw_tensor &t = tensors[i];
        if (t.n < 0 || t.n > ((int64_t)1 << 40) || !std::isfinite(t.weight_decay))
            return MOK_ERR_INVALID_ARG;
        if (t.copy != nullptr && c->p_dtype != MOK_DTYPE_F32) return MOK_ERR_INVALID_ARG;
        if (t.n == 0) continue;
        if (!t.p || !t.g || !t.m || !t.v || (s8 && (!t.m_scale || !t.v_scale)))
            return MOK_ERR_INVALID_ARG;
        const void *ps[] = {t.p, t.copy, t.g, t.m, t.v};
        for (const void *p : ps)
            if (!op_aligned16(p)) return MOK_ERR_INVALID_ARG;
    }
    return MOK_OK;
}

}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

mok_status mok_check_adamw_config(const mok_adamw_config *c) {
    if (c == nullptr) return MOK_ERR_INVALID_ARG;
    if (c->abi_version != MOK_ABI_VERSION) return MOK_ERR_ABI;
    const auto dtype_ok = [](int32_t d) { return d == MOK_DTYPE_BF16 || d == MOK_DTYPE_F32; };
    if (!dtype_ok(c->p_dtype) || !dtype_ok(c->g_dtype)) return MOK_ERR_INVALID_ARG;
    if (c->state != MOK_STATE_F32 && c->state != MOK_STATE_MXFP8) return MOK_ERR_INVALID_ARG;
    if ((c->flags & ~MOK_ADAMW_STOCHASTIC) != 0 || c->step < 1) return MOK_ERR_INVALID_ARG;
    if (!(c->lr >= 0) || !std::isfinite(c->lr)) return MOK_ERR_INVALID_ARG;
    if (!(c->eps >= 0) || !std::isfinite(c->eps)) return MOK_ERR_INVALID_ARG;
    if (!(c->beta1 >= 0 && c->beta1 < 1) || !(c->beta2 >= 0 && c->beta2 < 1))
        return MOK_ERR_INVALID_ARG;
    return MOK_OK;
}

mok_status mok_adamw_step(const mok_adamw_config *c, const mok_adamw_tensor *tensors,
                          int32_t n_tensors, const float *grad_scale, cudaStream_t stream) {
    int *status;
    const mok_status st = check_step(c, tensors, n_tensors, &status);
    if (st != MOK_OK) return st;
    int64_t base = 0;
    for (int t0 = 0; t0 < n_tensors; t0 += NT_LARGE) {
        const int t1 = n_tensors - t0 < NT_LARGE ? n_tensors : t0 + NT_LARGE, n = t1 - t0;
        MOK_OP_LAUNCH(OP_ADAMW, 1,
                      (n <= NT_SMALL ? step_group<false, NT_SMALL>
                       : n <= NT_MID ? step_group<false, NT_MID>
                                     : step_group<false, NT_LARGE>)(*c, tensors, t0, t1, nullptr,
                                                                    grad_scale, &base, stream));
    }
    return MOK_OK;
}

mok_status mok_adamw_advance(const mok_adamw_config *c, mok_adamw_clock *clock,
                             cudaStream_t stream) {
    mok_status st = mok_check_adamw_config(c);
    if (st != MOK_OK) return st;
    int *status;
    if ((st = current_device_status_word(&status)) != MOK_OK) return st;
    if (clock == nullptr || !op_aligned16(clock)) return MOK_ERR_INVALID_ARG;
    MOK_OP_LAUNCH(OP_ADAMW, 1,
                  (advance_kernel<<<1, 1, 0, stream>>>(clock, c->beta1, c->beta2, status),
                   cudaGetLastError()));
    return MOK_OK;
}

mok_status mok_adamw_step_at(const mok_adamw_config *c, const mok_adamw_tensor *tensors,
                             int32_t n_tensors, const mok_adamw_clock *clock,
                             const float *grad_scale, cudaStream_t stream) {
    int *status;
    const mok_status st = check_step(c, tensors, n_tensors, &status);
    if (st != MOK_OK) return st;
    if (clock == nullptr || !op_aligned16(clock)) return MOK_ERR_INVALID_ARG;
    int64_t base = 0;
    for (int t0 = 0; t0 < n_tensors; t0 += NT_MID) {
        const int t1 = n_tensors - t0 < NT_MID ? n_tensors : t0 + NT_MID;
        MOK_OP_LAUNCH(OP_ADAMW, 1,
                      (step_group<true, NT_MID>)(*c, tensors, t0, t1, clock, grad_scale, &base, stream));
    }
    return MOK_OK;
}

}  // extern "C"

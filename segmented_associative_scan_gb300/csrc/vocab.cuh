// Losses over a vocabulary: log-probabilities, the clipped policy loss, the preference loss and
// the distillation from a teacher's top logits are all functions of a row's softmax, and all
// their gradients by the logits have one form. With x = z / tau, m = max z, u_j = (z_j - m) / tau:
//   S = sum e^u_j,  h = -sum e^u_j u_j,  log p_a = u_a - log S,  H = log S + h / S
//   dz_j = e^u_j (kappa - alpha u_j) + (what the taken token, or the teacher's, adds at j)
// where alpha belongs to the entropy and kappa to everything else. So a row is read once for
// (m, S, h), a few scalars are worked out, and where the loss is a sum over steps with known
// weights the gradient follows from the row that was just read.
//
// u is formed by subtracting first: exact or rounded once, and a row of the type's lowest value
// gives 0 where a product first would give inf - inf.
#pragma once

#include "../../include/rlca_policy.h"
#include "sequence.cuh"

namespace rlca {
namespace seq {

// What z - m is multiplied by in front of 2^v: hi + lo, hi below the scale, so lo > 0 and -inf
// stays -inf; `near` the nearest float.
struct ExpScale {
    float hi, lo, near;
    float depth;  // z - m at which the exponential is surely 0

    __device__ __forceinline__ float operator*(float w) const { return fmaf(w, hi, w * lo); }
};

struct VocabParams {
    int64_t N, T, V, M;  // M = N T steps
    rlca_steps logits, grad;
    const void *tokens;
    int64_t token_ld;
    const int32_t *lengths;
    int token_bytes;
    float inv_tau, inv_tau_lo;  // 1 / tau to twice the digits
    ExpScale scale;             // log2(e) / tau
    float near;  // logits this close are e^4 apart or less
    int even;    // all rows begin on 16 bytes and are whole packs
    // forward results, contiguous [N,T]; saved [N,T,2] = (m, S)
    float *loss, *logp, *entropy, *kl, *saved;
    // clipped policy loss
    rlca_line old_logp, advantage, ref_logp, weight;
    float ratio_lo, ratio_hi, kl_coef, entropy_coef;
    // distillation
    rlca_steps index, teacher;
    int K, index_bytes, teacher_fp32;
    // backward from `saved`: dlogp and dentropy by step, or by row and pair (slope, dloss)
    rlca_line dlogp, dentropy;
    const float *entropy_in, *slope, *dloss;
};

struct PairParams {
    int64_t N, T, V;
    const void *tokens;
    int64_t token_ld;
    const int32_t *lengths;
    int token_bytes;
    const float *logp, *saved;
    rlca_line ref_logp;
    float beta, smoothing;
    int by_length;
    float *loss, *scores, *slope;
};

// kSlope: gradients from what a forward call saved.
enum class VocabOp : int { kLogp, kPolicy, kDistill, kSlope };

// ------------------------------------------------------------------------- small math

__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The one-instruction 2^v is low by 5.0e-8 on average for v < -1 (measured, any v from -1 to -32; 2e-8
// to 5e-8 up to 0, where it is exact): put back into a row's sums, the largest logit's 1 apart. (For v
// above 0, logits above a parked row's reference, it is high by 3.3e-8: a mean error of up to 6e-8 stays
// there.)
constexpr float kExp2Bias = 5.0e-8f;

// 2^v below this is 0 in fp32; cutting exponents off there keeps 0 (-inf) out of the entropy's sums.
constexpr float kLowest = -250.f;

// e^((z - ref) / tau) = 2^v by one instruction for each, and what v is below 0. The scale enters v with
// twice its digits where sums of many steps are taken from the result (log S): its own rounding, 1e-8 of
// v, is the same in every step of every row, and a score adds up hundreds of them. fp32 keeps the digits
// that rounding v leaves out, too: 2^(v + d) = 2^v (1 + d ln 2). (Nine instructions to two elements;
// CUDA's expf takes sixteen and more: policy loss with entropy [4096, 512, 18] 84 / 78 us,
// [64, 128, 32768] 395 / 358.)
struct ExpOf {
    Pair e, below;
};

template <typename T, bool CUT>
__device__ __forceinline__ ExpOf exp_of(Pair z, float ref, ExpScale c)
{
    Pair w = add2(z, pair(-ref, -ref));
    if (CUT || sizeof(T) == 4) w = pair(max_nan(w.x, c.depth), max_nan(w.y, c.depth));
    const Pair hi = pair(c.hi, c.hi), lo = pair(c.lo, c.lo), minus = pair(-c.hi, -c.hi);
    ExpOf r;
    if constexpr (sizeof(T) == 4) {
        r.below = mul2(w, minus);
        r.e = pair(exp2_fast(-r.below.x), exp2_fast(-r.below.y));
        const Pair d = fma2(w, lo, fma2(w, hi, r.below));
        r.e = fma2(r.e, mul2(d, pair(kLn2, kLn2)), r.e);
    } else {
        r.below = fma2(w, minus, mul2(w, pair(-c.lo, -c.lo)));
        r.e = pair(exp2_fast(-r.below.x), exp2_fast(-r.below.y));
    }
    return r;
}

// What a row, or a part of it, comes to: the largest logit (of a parked row, one that is at most e^4
// below it), sum e^u, -sum e^u v (v = u log2(e)).
struct RowStats {
    float m, s, h;
};

__device__ __forceinline__ RowStats no_stats() { return {-INFINITY, 0.f, 0.f}; }

// The sums of `a` relative to another largest logit m >= a.m.
template <bool ENT>
__device__ __forceinline__ void rebase(RowStats &a, float m, ExpScale c)
{
    // Equal ones are not subtracted: -inf - -inf, and inf - inf.
    const float d = a.m == m ? 0.f : max_nan(c * (a.m - m), kLowest);
    const float f = expf(d * kLn2);
    if (ENT) a.h = f * fmaf(-a.s, d, a.h);
    a.s *= f;
    a.m = m;
}

__device__ __forceinline__ RowStats unbiased(const RowStats &a)
{
    return {a.m, fmaf(a.s - 1.f, kExp2Bias, a.s), fmaf(a.h, kExp2Bias, a.h)};
}

// a + b = hi + lo exactly.
struct Two {
    float hi, lo;
};

__device__ __forceinline__ Two two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b), t = __fadd_rn(s, -a);
    return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -t)), __fadd_rn(b, -t))};
}

// log p_a to a little more than fp32: what a ratio or a KL term subtracts from it is near it, and
// their difference should not see its rounding.
struct LogProb {
    float u, u_lo, log_s;

    // log p_a - other, rounded once or so.
    __device__ __forceinline__ float minus(float other) const
    {
        const Two a = two_sum(u, -other), b = two_sum(a.hi, -log_s);
        const float r = b.hi + ((a.lo + b.lo) + u_lo);
        // Infinities and NaN leave no remainder.
        return isfinite(b.hi) ? r : (u - other) - log_s;
    }
};

__device__ __forceinline__ LogProb log_prob(float z, float m, float log_s, float inv, float inv_lo)
{
    const Two w = two_sum(z, -m);
    LogProb r;
    r.u = w.hi * inv;
    r.u_lo = fmaf(w.hi, inv, -r.u) + fmaf(w.hi, inv_lo, w.lo * inv);
    r.log_s = log_s;
    return r;
}

// e^d - 1 - d, to its own digits where |d| is small: d^2 times a polynomial (Taylor's, to 1e-8).
__device__ __forceinline__ float exp_excess(float d)
{
    if (fabsf(d) > 1.f) {
        const float e = expm1f(d);
        return e == INFINITY ? e : e - d;
    }
    float s = 1.f / 39916800.f;
    s = fmaf(s, d, 1.f / 3628800.f);
    s = fmaf(s, d, 1.f / 362880.f);
    s = fmaf(s, d, 1.f / 40320.f);
    s = fmaf(s, d, 1.f / 5040.f);
    s = fmaf(s, d, 1.f / 720.f);
    s = fmaf(s, d, 1.f / 120.f);
    s = fmaf(s, d, 1.f / 24.f);
    s = fmaf(s, d, 1.f / 6.f);
    s = fmaf(s, d, 0.5f);
    return d * d * s;
}

// ------------------------------------------------------------------------- a row's scalars

template <typename P>
__device__ __forceinline__ int64_t vocab_token(const P &p, int64_t n, int64_t t)
{
    const int64_t i = n * p.token_ld + t;
    return p.token_bytes == 8 ? (int64_t)__ldg(static_cast<const long long *>(p.tokens) + i)
                              : (int64_t)__ldg(static_cast<const int *>(p.tokens) + i);
}

template <typename P>
__device__ __forceinline__ bool inside_row(const P &p, int64_t n, int64_t t)
{
    return !p.lengths || t < __ldg(p.lengths + n);
}

__device__ __forceinline__ float at(const rlca_line &l, int64_t n, int64_t t)
{
    return __ldg(l.ptr + n * l.ld + t);
}

template <typename T>
__device__ __forceinline__ const T *row_of(const rlca_steps &a, int64_t n, int64_t t)
{
    return static_cast<const T *>(a.ptr) + n * a.row + t * a.step;
}

template <typename T>
__device__ __forceinline__ T *out_row(const rlca_steps &a, int64_t n, int64_t t)
{
    return const_cast<T *>(row_of<T>(a, n, t));
}

// A step's inputs, read before its logits are.
struct RowInputs {
    float old, advantage, ref, weight;
};

template <VocabOp OP>
__device__ __forceinline__ RowInputs row_inputs(const VocabParams &p, int64_t n, int64_t t)
{
    RowInputs r = {0.f, 0.f, 0.f, 1.f};
    if (OP == VocabOp::kPolicy) {
        r.old = at(p.old_logp, n, t);
        r.advantage = at(p.advantage, n, t);
        if (p.ref_logp.ptr) r.ref = at(p.ref_logp, n, t);
    }
    if (OP != VocabOp::kLogp && p.weight.ptr) r.weight = at(p.weight, n, t);
    return r;
}

// dz_j = e_j (kappa - alpha v_j) + gamma [j = token]; `zero`: whatever the row holds, 0.
struct RowSlope {
    float alpha, kappa, gamma;
    bool zero;
};

// The gradient g of log p_a and c of H, as a row's slope.
__device__ __forceinline__ RowSlope row_slope(float g, float c, float log_s, float inv_s,
                                              float entropy, float inv_tau)
{
    RowSlope r;
    r.alpha = c * inv_tau * inv_s * kLn2;
    r.kappa = -(g + c * (entropy - log_s)) * inv_tau * inv_s;
    r.gamma = g * inv_tau;
    r.zero = false;
    return r;
}

// Scalars of a step that counts: `write` writes its results, which step i of [N,T] takes.
template <typename T, VocabOp OP, bool ENT>
__device__ __forceinline__ RowSlope finish_row(const VocabParams &p, int64_t i, float z_a,
                                               const RowStats &raw, const RowInputs &in, bool write)
{
    const RowStats st = unbiased(raw);
    const float log_s = logf(st.s), inv_s = 1.f / st.s;
    const float entropy = ENT ? log_s + st.h * kLn2 * inv_s : 0.f;
    const LogProb lp = log_prob(z_a, st.m, log_s, p.inv_tau, p.inv_tau_lo);
    const float logp = lp.minus(0.f);
    if (write) {
        if (p.logp) p.logp[i] = logp;
        if (ENT && p.entropy) p.entropy[i] = entropy;
        if (p.saved) *reinterpret_cast<float2 *>(p.saved + 2 * i) = make_float2(st.m, st.s);
    }
    if constexpr (OP == VocabOp::kPolicy) {
        const float ratio = expf(lp.minus(in.old));
        const float free = -in.advantage * ratio;
        const float clipped = -in.advantage * fminf(fmaxf(ratio, p.ratio_lo), p.ratio_hi);
        float loss = max_nan(free, clipped), g = free >= clipped ? free : 0.f;
        if (isnan(free)) g = free;
        float kl = 0.f;
        if (p.ref_logp.ptr) {
            const float d = -lp.minus(in.ref);
            kl = exp_excess(d);
            if (p.kl_coef > 0.f) {
                loss = fmaf(p.kl_coef, kl, loss);
                g = fmaf(-p.kl_coef, expm1f(d), g);
            }
        }
        if (ENT) loss = fmaf(-p.entropy_coef, entropy, loss);
        if (write) {
            p.loss[i] = loss;
            if (p.kl) p.kl[i] = kl;
        }
        RowSlope r = row_slope(in.weight * g, ENT ? -in.weight * p.entropy_coef : 0.f, log_s,
                                  inv_s, entropy, p.inv_tau);
        r.zero = in.weight == 0.f;
        return r;
    }
    return {0.f, 0.f, 0.f, true};
}

// Results of a step that does not count.
__device__ __forceinline__ void write_uncounted(const VocabParams &p, int64_t i)
{
    if (p.loss) p.loss[i] = 0.f;
    if (p.logp) p.logp[i] = 0.f;
    if (p.entropy) p.entropy[i] = 0.f;
    if (p.kl) p.kl[i] = 0.f;
    if (p.saved) *reinterpret_cast<float2 *>(p.saved + 2 * i) = make_float2(-INFINITY, 0.f);
}

// ------------------------------------------------------------------------- packs

template <typename T>
__device__ __forceinline__ Pair widen_pair(const Pack<T, 16 / (int)sizeof(T)> &v, int i)
{
    if constexpr (sizeof(T) == 4) {
        return pair(v.e[2 * i], v.e[2 * i + 1]);
    } else {
        const uint32_t w = reinterpret_cast<const uint32_t *>(&v)[i];
        if constexpr (std::is_same<T, __nv_bfloat16>::value)
            return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
        else
            return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
}

template <typename T>
__device__ __forceinline__ void narrow_pair(Pack<T, 16 / (int)sizeof(T)> &v, int i, Pair x)
{
    if constexpr (sizeof(T) == 4) {
        v.e[2 * i] = x.x;
        v.e[2 * i + 1] = x.y;
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        reinterpret_cast<__nv_bfloat162 *>(&v)[i] = __floats2bfloat162_rn(x.x, x.y);
    } else {
        reinterpret_cast<__half2 *>(&v)[i] = __floats2half2_rn(x.x, x.y);
    }
}

// The largest element, two at a time.
template <typename T>
struct MaxOf {
    T a[2];  // fp32: one after the other
    __device__ __forceinline__ MaxOf() { a[0] = a[1] = narrow<T>(-INFINITY); }
    __device__ __forceinline__ void add(const Pack<T, 16 / (int)sizeof(T)> &v)
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i & 1] = max_nan(a[i & 1], v.e[i]);
        } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            auto &m = reinterpret_cast<__nv_bfloat162 &>(a);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                m = __hmax2_nan(m, reinterpret_cast<const __nv_bfloat162 *>(&v)[i]);
        } else {
            auto &m = reinterpret_cast<__half2 &>(a);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                m = __hmax2_nan(m, reinterpret_cast<const __half2 *>(&v)[i]);
        }
    }
    __device__ __forceinline__ float get() const { return max_nan(widen(a[0]), widen(a[1])); }
};

// A logit below m at which exponentials relative to m are 0, for logits of 16 bits: cutting them off
// there keeps 0 (-inf) out of the entropy's sums, two at a time. -inf where there is no such number:
// below the type's lowest one (fp16 ends at -65504), or where 173 temperatures are lost in m's own
// rounding. Exponents are cut off in 32 bits then (cut_late).
template <typename T>
__device__ __forceinline__ T lowest_logit(float m, ExpScale c)
{
    const float z = m + c.depth;
    if constexpr (std::is_same<T, __half>::value)
        return __float2half_rd(z < m && z >= -65504.f ? z : -INFINITY);
    else if constexpr (std::is_same<T, __nv_bfloat16>::value)
        return __float2bfloat16_rd(z < m ? z : -INFINITY);
    else
        return z;  // not used
}

template <typename T>
__device__ __forceinline__ bool cut_late(T low)
{
    return sizeof(T) != 4 && widen(low) == -INFINITY;
}

template <typename T>
__device__ __forceinline__ Pack<T, 16 / (int)sizeof(T)> cut_off(Pack<T, 16 / (int)sizeof(T)> v, T low)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            auto &x = reinterpret_cast<__nv_bfloat162 *>(&v)[i];
            x = __hmax2_nan(x, __nv_bfloat162(low, low));
        } else if constexpr (std::is_same<T, __half>::value) {
            auto &x = reinterpret_cast<__half2 *>(&v)[i];
            x = __hmax2_nan(x, __half2(low, low));
        }
    }
    return v;
}

// Two running sums, each of every other element.
struct RowSums {
    Pair s, h;
};

// LATE: exponents are cut off in 32 bits.
template <typename T, bool ENT, bool LATE>
__device__ __forceinline__ void add_pack(RowSums &a, const Pack<T, 16 / (int)sizeof(T)> &v,
                                         float ref, T low, ExpScale c)
{
    Pack<T, 16 / (int)sizeof(T)> z = v;
    if (ENT && !LATE) z = cut_off<T>(z, low);
#pragma unroll
    for (int i = 0; i < 8 / (int)sizeof(T); ++i) {
        const ExpOf x = exp_of<T, ENT && LATE>(widen_pair<T>(z, i), ref, c);
        a.s = add2(a.s, x.e);
        if (ENT) a.h = fma2(x.e, x.below, a.h);
    }
}

template <typename T, bool ENT, bool LATE = false>
__device__ __forceinline__ Pack<T, 16 / (int)sizeof(T)> pack_slope(
    const Pack<T, 16 / (int)sizeof(T)> &v, const RowSlope &r, float m, T low, ExpScale c)
{
    const Pair off = pair(-m, -m), alpha = pair(r.alpha, r.alpha), kappa = pair(r.kappa, r.kappa);
    Pack<T, 16 / (int)sizeof(T)> z = v;
    if (ENT && !LATE) z = cut_off<T>(z, low);
    Pack<T, 16 / (int)sizeof(T)> o;
#pragma unroll
    for (int i = 0; i < 8 / (int)sizeof(T); ++i) {
        ExpOf x;
        if constexpr (sizeof(T) == 4) {
            x = exp_of<T, ENT>(widen_pair<T>(z, i), m, c);
        } else {
            // 16 bits hide what the nearest scale is off by.
            x.below = mul2(add2(widen_pair<T>(z, i), off), pair(-c.near, -c.near));
            if (ENT && LATE)
                x.below = pair(-max_nan(-x.below.x, kLowest), -max_nan(-x.below.y, kLowest));
            x.e = pair(exp2_fast(-x.below.x), exp2_fast(-x.below.y));
        }
        narrow_pair<T>(o, i, mul2(x.e, ENT ? fma2(alpha, x.below, kappa) : kappa));
    }
    return o;
}

// One element's gradient in 32 bits, as pack_slope forms it: which of them an element gets depends on
// where its row lies in memory, and its bits should not.
template <typename T, bool ENT>
__device__ __forceinline__ float slope_at(float z, const RowSlope &r, float m, ExpScale c)
{
    if constexpr (sizeof(T) == 4) {
        const ExpOf x = exp_of<T, ENT>(pair(z, z), m, c);
        return x.e.x * (ENT ? fmaf(r.alpha, x.below.x, r.kappa) : r.kappa);
    } else {
        float a = (z - m) * c.near;
        if (ENT) a = max_nan(a, kLowest);
        return exp2_fast(a) * (ENT ? fmaf(r.alpha, -a, r.kappa) : r.kappa);
    }
}

// Writes 0 to elements lo <= j < hi of a row, every `step`-th pack of it from the `first`.
template <typename T>
__device__ __forceinline__ void clear_row(T *g, int64_t lo, int64_t hi, int first, int step)
{
    constexpr int W = 16 / (int)sizeof(T);
    const int64_t head = (reinterpret_cast<uintptr_t>(g + lo) % 16) / sizeof(T);
    for (int64_t j = lo - head + (int64_t)first * W; j < hi; j += (int64_t)step * W) {
        if (j >= lo && j + W <= hi) {
            *reinterpret_cast<uint4 *>(g + j) = make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll 1
            for (int e = 0; e < W; ++e)
                if (j + e >= lo && j + e < hi) g[j + e] = narrow<T>(0.f);
        }
    }
}

template <Fmt F, VocabOp OP>
cudaError_t launch_vocab(const VocabParams &p, bool entropy, cudaStream_t stream);
cudaError_t launch_pairs(const PairParams &p, cudaStream_t stream);

}  // namespace seq
}  // namespace rlca

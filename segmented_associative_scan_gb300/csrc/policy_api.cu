// C ABI of the losses over a vocabulary (declared in include/rlca_policy.h): argument
// validation, then the operator's launches on the caller's stream. No allocation, no
// synchronisation, no change of the current device.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "buffers.cuh"
#include "vocab.cuh"

namespace {

using namespace rlca::seq;
using rlca::Fmt;

bool choices_shape_ok(const rlca_choices &p)
{
    return p.N >= 0 && p.T >= 0 && p.T <= RLCA_MAX_T && p.V >= 1 && p.V <= RLCA_MAX_V &&
           (p.token_bytes == 4 || p.token_bytes == 8) && product_fits(p.N, p.T, p.V, 16) &&
           p.N * p.T <= INT32_MAX;
}

bool positive(float v) { return std::isfinite(v) && v > 0.f; }

// A range in which logits / temperature neither overflow nor vanish for no reason.
bool temperature_ok(float v) { return v >= 1e-6f && v <= 1e6f; }

// logits and lengths, the tokens of the operators that take any, and what is common to all calls.
void choices_inputs(Buffers &b, const rlca_choices &p, bool tokens, size_t es,
                    const rlca_steps *dlogits)
{
    if (dlogits && dlogits->ptr) b.in_place(p.logits, *dlogits, p.V, es);
    else b.steps(p.logits, p.V, es, true, false);
    if (tokens) b.line(p.tokens, p.token_ld, (size_t)p.token_bytes, true);
    if (p.N > 0) b.in(p.lengths, p.N, 4, false);
}

VocabParams vocab_params(const rlca_choices &p)
{
    VocabParams q;
    std::memset(&q, 0, sizeof(q));
    q.N = p.N;
    q.T = p.T;
    q.V = p.V;
    q.M = p.N * p.T;
    q.logits = p.logits;
    q.tokens = p.tokens;
    q.token_ld = p.token_ld;
    q.token_bytes = p.token_bytes;
    q.lengths = p.lengths;
    const double inv = 1.0 / (double)p.temperature;
    q.inv_tau = (float)inv;
    q.inv_tau_lo = (float)(inv - (double)q.inv_tau);
    const double scale = inv * 1.4426950408889634;
    q.scale.near = q.scale.hi = (float)scale;
    if ((double)q.scale.hi >= scale) q.scale.hi = std::nextafterf(q.scale.hi, 0.f);
    q.scale.lo = (float)(scale - (double)q.scale.hi);
    q.scale.depth = (float)(kLowest / scale);
    q.near = 4.f * p.temperature;
    return q;
}

template <VocabOp OP>
int run(const VocabParams &q, bool entropy, Fmt f, void *stream)
{
    return status(in_format(f, [&](auto fmt) {
        return launch_vocab<decltype(fmt)::value, OP>(q, entropy, static_cast<cudaStream_t>(stream));
    }));
}

int token_logprobs(const rlca_choices *pp, float *logp, float *entropy, float *saved, void *stream,
                   Fmt f)
{
    if (!pp) return RLCA_ERR_NULL;
    const rlca_choices &p = *pp;
    if (!choices_shape_ok(p)) return RLCA_ERR_SHAPE;
    if (!temperature_ok(p.temperature)) return RLCA_ERR_PARAM;
    if (p.N == 0 || p.T == 0) return RLCA_OK;
    const int64_t M = p.N * p.T;
    Buffers b(p.N, p.T);
    choices_inputs(b, p, true, bytes_of(f), nullptr);
    b.out(logp, M, 4);
    b.out(entropy, M, 4, false);
    b.out(saved, 2 * M, 4, false);
    b.aligned(saved, 8);
    const int st = b.check(nullptr, 0, 0);
    if (st != RLCA_OK) return st;
    VocabParams q = vocab_params(p);
    q.logp = logp;
    q.entropy = entropy;
    q.saved = saved;
    return run<VocabOp::kLogp>(q, entropy != nullptr, f, stream);
}

int token_logprobs_backward(const rlca_choices *pp, rlca_line dlogp, rlca_line dentropy,
                            const float *entropy, const float *saved, rlca_steps dlogits,
                            void *stream, Fmt f)
{
    if (!pp) return RLCA_ERR_NULL;
    const rlca_choices &p = *pp;
    if (!choices_shape_ok(p)) return RLCA_ERR_SHAPE;
    if (!temperature_ok(p.temperature)) return RLCA_ERR_PARAM;
    if (p.N == 0 || p.T == 0) return RLCA_OK;
    if (!dlogits.ptr) return RLCA_ERR_NULL;
    const int64_t M = p.N * p.T;
    Buffers b(p.N, p.T);
    choices_inputs(b, p, true, bytes_of(f), &dlogits);
    b.line(dlogp.ptr, dlogp.ld, 4, false);
    b.line(dentropy.ptr, dentropy.ld, 4, false);
    if (dentropy.ptr) b.in(entropy, M, 4);
    b.in(saved, 2 * M, 4);
    b.aligned(saved, 8);
    const int st = b.check(nullptr, 0, 0);
    if (st != RLCA_OK) return st;
    VocabParams q = vocab_params(p);
    q.saved = const_cast<float *>(saved);
    q.entropy_in = entropy;
    q.dlogp = dlogp;
    q.dentropy = dentropy;
    q.grad = dlogits;
    return run<VocabOp::kSlope>(q, dentropy.ptr != nullptr, f, stream);
}

int policy_loss(const rlca_choices *pp, const rlca_policy *qq, void *stream, Fmt f)
{
    if (!pp || !qq) return RLCA_ERR_NULL;
    const rlca_choices &p = *pp;
    const rlca_policy &l = *qq;
    if (!choices_shape_ok(p)) return RLCA_ERR_SHAPE;
    if (!temperature_ok(p.temperature) || !(l.clip_low >= 0.f && l.clip_low <= 1.f) ||
        !(std::isfinite(l.clip_high) && l.clip_high >= 0.f) ||
        !(std::isfinite(l.kl_coef) && l.kl_coef >= 0.f) || !std::isfinite(l.entropy_coef))
        return RLCA_ERR_PARAM;
    if (p.N == 0 || p.T == 0) return RLCA_OK;
    if ((l.kl_coef > 0.f || l.kl) && !l.ref_logp.ptr) return RLCA_ERR_NULL;
    const int64_t M = p.N * p.T;
    Buffers b(p.N, p.T);
    choices_inputs(b, p, true, bytes_of(f), &l.dlogits);
    b.line(l.old_logp.ptr, l.old_logp.ld, 4, true);
    b.line(l.advantage.ptr, l.advantage.ld, 4, true);
    b.line(l.ref_logp.ptr, l.ref_logp.ld, 4, false);
    b.line(l.weight.ptr, l.weight.ld, 4, false);
    b.out(l.loss, M, 4);
    b.out(l.logp, M, 4, false);
    b.out(l.entropy, M, 4, false);
    b.out(l.kl, M, 4, false);
    const int st = b.check(nullptr, 0, 0);
    if (st != RLCA_OK) return st;
    VocabParams q = vocab_params(p);
    q.old_logp = l.old_logp;
    q.advantage = l.advantage;
    q.ref_logp = l.ref_logp;
    q.weight = l.weight;
    q.ratio_lo = (float)(1.0 - (double)l.clip_low);
    q.ratio_hi = (float)(1.0 + (double)l.clip_high);
    q.kl_coef = l.kl_coef;
    q.entropy_coef = l.entropy_coef;
    q.loss = l.loss;
    q.logp = l.logp;
    q.entropy = l.entropy;
    q.kl = l.kl;
    q.grad = l.dlogits;
    return run<VocabOp::kPolicy>(q, l.entropy || l.entropy_coef != 0.f, f, stream);
}

int preference_loss(const rlca_choices *pp, const rlca_preference *qq, void *stream, Fmt f)
{
    if (!pp || !qq) return RLCA_ERR_NULL;
    const rlca_choices &p = *pp;
    const rlca_preference &l = *qq;
    if (!choices_shape_ok(p) || p.N % 2 != 0) return RLCA_ERR_SHAPE;
    if (!temperature_ok(p.temperature) || !positive(l.beta) ||
        !(l.smoothing >= 0.f && l.smoothing <= 1.f))
        return RLCA_ERR_PARAM;
    if (p.N == 0) return RLCA_OK;
    const int64_t M = p.N * p.T;
    Buffers b(p.N, p.T);
    choices_inputs(b, p, true, bytes_of(f), nullptr);
    b.line(l.ref_logp.ptr, l.ref_logp.ld, 4, false);
    b.out(l.loss, p.N / 2, 4);
    b.out(l.scores, p.N, 4);
    b.out(l.logp, M, 4);
    b.out(l.saved, 2 * M, 4);
    b.aligned(l.saved, 8);
    b.out(l.slope, p.N, 4, false);
    const int st = b.check(nullptr, 0, 0);
    if (st != RLCA_OK) return st;
    if (p.T > 0) {
        VocabParams q = vocab_params(p);
        q.logp = l.logp;
        q.saved = l.saved;
        const int rows = run<VocabOp::kLogp>(q, false, f, stream);
        if (rows != RLCA_OK) return rows;
    }
    PairParams q;
    std::memset(&q, 0, sizeof(q));
    q.N = p.N;
    q.T = p.T;
    q.V = p.V;
    q.tokens = p.tokens;
    q.token_ld = p.token_ld;
    q.token_bytes = p.token_bytes;
    q.lengths = p.lengths;
    q.logp = l.logp;
    q.saved = l.saved;
    q.ref_logp = l.ref_logp;
    q.beta = l.beta;
    q.smoothing = l.smoothing;
    q.by_length = l.by_length != 0;
    q.loss = l.loss;
    q.scores = l.scores;
    q.slope = l.slope;
    return status(launch_pairs(q, static_cast<cudaStream_t>(stream)));
}

int preference_loss_backward(const rlca_choices *pp, const float *dloss, const float *slope,
                             const float *saved, rlca_steps dlogits, void *stream, Fmt f)
{
    if (!pp) return RLCA_ERR_NULL;
    const rlca_choices &p = *pp;
    if (!choices_shape_ok(p) || p.N % 2 != 0) return RLCA_ERR_SHAPE;
    if (!temperature_ok(p.temperature)) return RLCA_ERR_PARAM;
    if (p.N == 0 || p.T == 0) return RLCA_OK;
    if (!dlogits.ptr) return RLCA_ERR_NULL;
    Buffers b(p.N, p.T);
    choices_inputs(b, p, true, bytes_of(f), &dlogits);
    b.in(dloss, p.N / 2, 4, false);
    b.in(slope, p.N, 4);
    b.in(saved, 2 * p.N * p.T, 4);
    b.aligned(saved, 8);
    const int st = b.check(nullptr, 0, 0);
    if (st != RLCA_OK) return st;
    VocabParams q = vocab_params(p);
    q.saved = const_cast<float *>(saved);
    q.slope = slope;
    q.dloss = dloss;
    q.grad = dlogits;
    return run<VocabOp::kSlope>(q, false, f, stream);
}

int distill_topk(const rlca_choices *pp, const rlca_distill *qq, void *stream, Fmt f)
{
    if (!pp || !qq) return RLCA_ERR_NULL;
    rlca_choices p = *pp;
    const rlca_distill &l = *qq;
    p.token_bytes = 8;  // no tokens
    p.tokens = nullptr;
    if (!choices_shape_ok(p) || l.K < 0 || l.K > RLCA_DISTILL_MAX_K ||
        (l.index_bytes != 4 && l.index_bytes != 8))
        return RLCA_ERR_SHAPE;
    if (!temperature_ok(p.temperature)) return RLCA_ERR_PARAM;
    if (p.N == 0 || p.T == 0) return RLCA_OK;
    Buffers b(p.N, p.T);
    choices_inputs(b, p, false, bytes_of(f), &l.dlogits);
    b.steps(l.index, l.K, (size_t)l.index_bytes, true, false);
    b.steps(l.teacher, l.K, l.teacher_fp32 ? 4 : bytes_of(f), true, false);
    b.line(l.weight.ptr, l.weight.ld, 4, false);
    b.out(l.loss, p.N * p.T, 4);
    const int st = b.check(nullptr, 0, 0);
    if (st != RLCA_OK) return st;
    VocabParams q = vocab_params(p);
    q.index = l.index;
    q.teacher = l.teacher;
    q.K = (int)l.K;
    q.index_bytes = l.index_bytes;
    q.teacher_fp32 = l.teacher_fp32 != 0 || f == Fmt::kF32;
    q.weight = l.weight;
    q.loss = l.loss;
    q.grad = l.dlogits;
    return run<VocabOp::kDistill>(q, false, f, stream);
}

}  // namespace

extern "C" {

#define RLCA_POLICY_ENTRY_POINTS(SUFFIX, FMT)                                                    \
    int rlca_token_logprobs##SUFFIX(const rlca_choices *p, float *logp, float *entropy,          \
                                    float *saved, void *stream)                                  \
    {                                                                                            \
        return token_logprobs(p, logp, entropy, saved, stream, FMT);                             \
    }                                                                                            \
    int rlca_token_logprobs_backward##SUFFIX(                                                    \
        const rlca_choices *p, rlca_line dlogp, rlca_line dentropy, const float *entropy,        \
        const float *saved, rlca_steps dlogits, void *stream)                                    \
    {                                                                                            \
        return token_logprobs_backward(p, dlogp, dentropy, entropy, saved, dlogits, stream, FMT); \
    }                                                                                            \
    int rlca_policy_loss##SUFFIX(const rlca_choices *p, const rlca_policy *q, void *stream)      \
    {                                                                                            \
        return policy_loss(p, q, stream, FMT);                                                   \
    }                                                                                            \
    int rlca_preference_loss##SUFFIX(const rlca_choices *p, const rlca_preference *q,            \
                                     void *stream)                                               \
    {                                                                                            \
        return preference_loss(p, q, stream, FMT);                                               \
    }                                                                                            \
    int rlca_preference_loss_backward##SUFFIX(const rlca_choices *p, const float *dloss,         \
                                              const float *slope, const float *saved,            \
                                              rlca_steps dlogits, void *stream)                  \
    {                                                                                            \
        return preference_loss_backward(p, dloss, slope, saved, dlogits, stream, FMT);           \
    }                                                                                            \
    int rlca_distill_topk##SUFFIX(const rlca_choices *p, const rlca_distill *q, void *stream)    \
    {                                                                                            \
        return distill_topk(p, q, stream, FMT);                                                  \
    }

RLCA_POLICY_ENTRY_POINTS(, Fmt::kF32)
RLCA_POLICY_ENTRY_POINTS(_bf16, Fmt::kBF16)
RLCA_POLICY_ENTRY_POINTS(_fp16, Fmt::kF16)

#undef RLCA_POLICY_ENTRY_POINTS

}  // extern "C"

/*
 * rlca_policy.h - C ABI of librlca: losses over a vocabulary of tokens (or actions), what a
 * policy is trained with once its steps are credited, on one GB300 (sm_103a).
 *
 *   logits -> rlca_token_logprobs                       log pi(token): V-trace's log_rho, the
 *                                                       behaviour policy of a clipped update
 *   logits, advantages (rlca_gae) -> rlca_policy_loss   clipped surrogate + KL - entropy
 *   logits of pairs -> rlca_preference_loss             -log sigmoid of paired log ratios
 *   logits, a teacher's top K -> rlca_distill_topk      KL(teacher || student)
 *
 * Common conventions (all entry points of this header)
 *   Layout    Logits and their gradients are [N, T, V] as the activations of rlca_sequence.h:
 *             fp32, or bf16 / fp16 in the entry points with that suffix; unit stride over the
 *             vocabulary, any stride from step to step and from row to row. Values per step are
 *             fp32: inputs with a row stride of their own (rlca_line), outputs contiguous [N, T].
 *   Notation  x = logits / temperature, p = softmax(x), logp = log p[token],
 *             H = -sum p log p.
 *   Counting  A step counts if it lies inside its row (lengths [N] int32, nullable = T, clamped
 *             to [0, T]), its token inside [0, V) (padding and prompts: -1) and at least one
 *             logit is above -inf. Per-step outputs and gradients of steps that do not count
 *             are written as 0; their logits, per-step inputs and, past the row, tokens may hold
 *             anything.
 *   Masks     A logit of -inf is a token that is not allowed: p = 0, no part in H, gradient 0, at
 *             any temperature. If it is the step's own token (or a teacher's), log p is -inf and its
 *             gradient what the formula gives; where the loss is infinite, the row's gradient
 *             may hold infinities and NaN. A row holding a NaN or +inf gives NaN, in that row only.
 *   In place  dlogits may be exactly the logits (same address and strides), which it replaces.
 *   Memory, overlap, stream, ownership and errors as in rlca_sequence.h (`saved` aligned to 8
 *             bytes). No entry point takes a workspace. Sizes: 1 <= V <= RLCA_MAX_V, N T < 2^31;
 *             N == 0 or T == 0 enqueues nothing but the outputs per pair.
 *   Precision fp32 arithmetic; logits' gradients are rounded to their type once. Sums are taken
 *             in a fixed order: a call repeated on the same inputs gives the same bits.
 */
#ifndef RLCA_POLICY_H
#define RLCA_POLICY_H

#include "rlca_sequence.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest supported vocabulary. */
#define RLCA_MAX_V (1 << 30)

/* One fp32 value per step: element (n, t) is at ptr + n * ld + t; ld >= 0 (0 repeats a row). */
typedef struct rlca_line {
    const float *ptr;
    int64_t ld;
} rlca_line;

/* Distributions over a vocabulary, and the token taken from each. */
typedef struct rlca_choices {
    int64_t N, T, V;
    rlca_steps logits;      /* [N,T,V] */
    const void *tokens;     /* [N, token_ld]; not used by rlca_distill_topk */
    int64_t token_ld;       /* >= 0, as in rlca_line */
    const int32_t *lengths; /* [N], nullable */
    int32_t token_bytes;    /* 4 (int32) or 8 (int64) */
    float temperature;      /* 1e-6 to 1e6 */
} rlca_choices;

/* ------------------------------------------------------------ token log-probabilities
 *
 * logp [N,T]; entropy H [N,T] and saved [N,T,2] (for the backward pass) nullable.
 */
int rlca_token_logprobs(const rlca_choices *p, float *logp, float *entropy, float *saved,
                        void *stream);
int rlca_token_logprobs_bf16(const rlca_choices *p, float *logp, float *entropy, float *saved,
                             void *stream);
int rlca_token_logprobs_fp16(const rlca_choices *p, float *logp, float *entropy, float *saved,
                             void *stream);

/* Gradient of sum(logp * dlogp) + sum(entropy * dentropy). dlogp.ptr and dentropy.ptr nullable
 * (= 0); `saved` and, with dentropy, `entropy` are what the forward call wrote. */
int rlca_token_logprobs_backward(const rlca_choices *p, rlca_line dlogp, rlca_line dentropy,
                                 const float *entropy, const float *saved, rlca_steps dlogits,
                                 void *stream);
int rlca_token_logprobs_backward_bf16(const rlca_choices *p, rlca_line dlogp, rlca_line dentropy,
                                      const float *entropy, const float *saved,
                                      rlca_steps dlogits, void *stream);
int rlca_token_logprobs_backward_fp16(const rlca_choices *p, rlca_line dlogp, rlca_line dentropy,
                                      const float *entropy, const float *saved,
                                      rlca_steps dlogits, void *stream);

/* --------------------------------------------------------------- clipped policy loss
 *
 * With r = exp(logp - old_logp), d = ref_logp - logp:
 *   loss = max(-r A, -clip(r, 1 - clip_low, 1 + clip_high) A)
 *          + kl_coef (e^d - 1 - d) - entropy_coef H
 * dlogits: the gradient of sum(weight * loss), from the same read of the logits; where
 * weight is 0 it is 0 whatever the row holds. The gradient of the maximum is that of -r A
 * where the two are equal.
 */
typedef struct rlca_policy {
    rlca_line old_logp, advantage;
    rlca_line ref_logp;            /* nullable: no KL term */
    rlca_line weight;              /* nullable = 1 */
    float clip_low, clip_high;     /* 0 <= clip_low <= 1, 0 <= clip_high, finite */
    float kl_coef, entropy_coef;   /* finite, kl_coef >= 0; kl_coef > 0 needs ref_logp */
    float *loss;                   /* [N,T] */
    float *logp, *entropy, *kl;    /* [N,T], nullable; kl (e^d - 1 - d) needs ref_logp */
    rlca_steps dlogits;            /* [N,T,V], ptr nullable */
} rlca_policy;

int rlca_policy_loss(const rlca_choices *p, const rlca_policy *q, void *stream);
int rlca_policy_loss_bf16(const rlca_choices *p, const rlca_policy *q, void *stream);
int rlca_policy_loss_fp16(const rlca_choices *p, const rlca_policy *q, void *stream);

/* ------------------------------------------------------------------- preference loss
 *
 * Rows 0..N/2-1 are the preferred answers of the pairs, rows N/2..N-1 the others (N even):
 *   score_n = beta (sum over counted t of logp - ref_logp) [/ counted steps: by_length]
 *   x = score of the preferred answer - score of the other
 *   loss = -(1 - smoothing) log sigmoid(x) - smoothing log sigmoid(-x)
 * A row without counted steps has a score of 0. For the backward pass saved [N,T,2] (written
 * in any case) and slope [N], the derivative of the pair's loss by each logp of the row.
 */
typedef struct rlca_preference {
    rlca_line ref_logp;      /* nullable = 0 */
    float beta, smoothing;   /* beta > 0, finite; 0 <= smoothing <= 1 */
    int32_t by_length;
    float *loss;             /* [N/2] */
    float *scores;           /* [N] */
    float *logp, *saved;     /* [N,T], [N,T,2] */
    float *slope;            /* [N], nullable */
} rlca_preference;

int rlca_preference_loss(const rlca_choices *p, const rlca_preference *q, void *stream);
int rlca_preference_loss_bf16(const rlca_choices *p, const rlca_preference *q, void *stream);
int rlca_preference_loss_fp16(const rlca_choices *p, const rlca_preference *q, void *stream);

/* Gradient of sum(loss * dloss); dloss [N/2] nullable = 1. */
int rlca_preference_loss_backward(const rlca_choices *p, const float *dloss, const float *slope,
                                  const float *saved, rlca_steps dlogits, void *stream);
int rlca_preference_loss_backward_bf16(const rlca_choices *p, const float *dloss,
                                       const float *slope, const float *saved,
                                       rlca_steps dlogits, void *stream);
int rlca_preference_loss_backward_fp16(const rlca_choices *p, const float *dloss,
                                       const float *slope, const float *saved,
                                       rlca_steps dlogits, void *stream);

/* ----------------------------------------------------------------------- distillation
 *
 * The teacher's K largest logits and their tokens for each step: q = softmax of its logits /
 * temperature over those K (an entry whose token is outside [0, V) or whose logit is -inf is
 * left out; a token given twice has the sum of both):
 *   loss = sum_k q_k (log q_k - log p[token_k])
 * A step counts if it lies inside its row, some entry is left and some logit is above -inf.
 * dlogits: the gradient of sum(weight * loss), from the same read of the logits; 0 where
 * weight is 0. 0 <= K <= RLCA_DISTILL_MAX_K.
 */
#define RLCA_DISTILL_MAX_K 256

typedef struct rlca_distill {
    int64_t K;
    rlca_steps index, teacher;  /* [N,T,K], K contiguous */
    int32_t index_bytes;        /* 4 (int32) or 8 (int64) */
    int32_t teacher_fp32;       /* the teacher's logits are fp32 (0: of the logits' type) */
    rlca_line weight;           /* nullable = 1 */
    float *loss;                /* [N,T] */
    rlca_steps dlogits;         /* [N,T,V], ptr nullable */
} rlca_distill;

int rlca_distill_topk(const rlca_choices *p, const rlca_distill *q, void *stream);
int rlca_distill_topk_bf16(const rlca_choices *p, const rlca_distill *q, void *stream);
int rlca_distill_topk_fp16(const rlca_choices *p, const rlca_distill *q, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* RLCA_POLICY_H */

/*
 * rlca_sequence.h - C ABI of librlca: the operators of a recurrent sequence model in front
 * of the credit-assignment estimators, on one GB300 (sm_103a).
 *
 *   tokens -> rlca_embed_tokens -> rlca_causal_conv -> rlca_selective_scan -> values
 *
 * The selective scan is the forward affine recurrence of rlca_eligibility_trace with a
 * decay and an input of its own for every channel and state, computed from the data; the
 * convolution mixes a few steps in front of it; the embedding's gradient is a segmented
 * sum over sorted tokens. All of them restart at episode ends, so a window of rollouts
 * trains as it was acted.
 *
 * Common conventions (all entry points of this header)
 *   Layout    Activations are [N, T, channels]: row n (an environment, a prompt), step t,
 *             unit stride over the channels, any stride from step to step and from row to
 *             row (rlca_steps; a slice of a wider projection qualifies, and so does a
 *             time-major buffer). Their type is fp32, or bf16 / fp16 in the entry points
 *             with that suffix. Parameters, the scan's states and all gradients of
 *             parameters are fp32 and contiguous.
 *   Episodes  terminated / truncated [N, flag_ld] (each nullable) are uint8, nonzero = the
 *             episode ended at that step. A step whose previous step ended an episode is
 *             its episode's first: it sees neither the state nor the inputs before it.
 *             What a state held before, an Inf or a NaN too, does not reach it.
 *   Lengths   lengths [N] int32 (nullable = T): row n has lengths[n] steps, clamped to
 *             [0, T]. Later steps are not read (they may hold anything); outputs and
 *             gradients there are written as 0.
 *   States    A final state is what the next window or step starts from: that after the
 *             row's last step, 0 if that step ended an episode, the initial state if the
 *             row has no steps. A NULL initial state is 0.
 *   Memory    Device or managed memory of the current device, aligned to its elements
 *             (RLCA_ERR_MEMORY otherwise).
 *             The library allocates nothing; a workspace is caller-owned device memory,
 *             256-byte aligned, of at least the bytes its query gives, with any contents.
 *             Calls that share a workspace must be ordered on the GPU.
 *   Overlap   Outputs must not overlap inputs or each other (RLCA_ERR_ALIAS), except where
 *             a step's new state may be its state. Two slices of one buffer whose channels
 *             lie side by side at the same strides do not overlap.
 *   Empty     N == 0 or no channels: RLCA_OK, nothing enqueued. T == 0 is valid: states are
 *             carried through, sums over steps are 0.
 *   Precision fp32 arithmetic and states; results of the data type are rounded once. Sums
 *             over steps, rows and channels are taken in a fixed order, so a call repeated
 *             on the same inputs gives the same bits. A step moves a scan's state on by the
 *             bits that a window does; only where the window is cut into spans (its forward
 *             pass asks for a workspace) do the last bits differ.
 *   Stream, ownership and errors as in rlca.h.
 */
#ifndef RLCA_SEQUENCE_H
#define RLCA_SEQUENCE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* An activation: element (n, t, c) is at ptr + n * row + t * step + c (in elements).
 * Inputs: row, step >= 0 (0 repeats a row or a step). Outputs: no two elements may share
 * an address. */
typedef struct rlca_steps {
    const void *ptr;
    int64_t row, step;
} rlca_steps;

/* Flags and lengths of the rows of one call. */
typedef struct rlca_rows {
    const uint8_t *terminated, *truncated; /* [N, flag_ld], nullable */
    int64_t flag_ld;                       /* >= T where a flag is given */
    const int32_t *lengths;                /* [N], nullable */
} rlca_rows;

/* ------------------------------------------------------------------ selective scan
 *
 * For channel e of group g (E / G channels to a group) and state s:
 *   d_t = softplus(dt_t + dt_bias)      (dt_softplus; else dt_t + dt_bias)
 *   h_t = exp(d_t A[e,s]) h_{t-1} + d_t x_t B_t[g,s],      h_{-1} = init_state
 *   y_t = sum_s C_t[g,s] h_t[s] + D[e] x_t,   out_t = y_t silu(z_t)   (z; else y_t)
 * with h_{t-1} = 0 at an episode's first step. 1 <= S <= RLCA_SCAN_MAX_S; G divides E.
 */
#define RLCA_SCAN_MAX_S 64
/* The forward pass saves h before every RLCA_SCAN_CHUNK-th step for the backward pass. */
#define RLCA_SCAN_CHUNK 8

typedef struct rlca_scan {
    int64_t N, T, E, S, G;
    rlca_steps x, dt, z;            /* [N,T,E]; z.ptr nullable (no gate) */
    rlca_steps B, C;                /* [N,T,G,S], groups contiguous */
    const float *A, *D, *dt_bias;   /* [E,S]; [E] nullable; [E] nullable */
    rlca_rows rows;
    const float *init_state;        /* [N,E,S], nullable */
    int32_t dt_softplus;
} rlca_scan;

/* Bytes of workspace for either direction, and for the forward pass alone (0: none needed;
 * both 0 for invalid shapes), and of `saved`: fp32 [N, ceil(T / RLCA_SCAN_CHUNK), E, S]. The
 * forward pass cuts rows into spans that run side by side where the rows alone leave SMs
 * idle; its workspace holds their states. */
size_t rlca_selective_scan_workspace_bytes(int64_t N, int64_t T, int64_t E, int64_t S, int64_t G);
size_t rlca_selective_scan_forward_workspace_bytes(int64_t N, int64_t T, int64_t E, int64_t S,
                                                   int64_t G);
size_t rlca_selective_scan_saved_bytes(int64_t N, int64_t T, int64_t E, int64_t S);

/* out [N,T,E]; final_state [N,E,S] and saved nullable. */
int rlca_selective_scan(const rlca_scan *p, rlca_steps out, float *final_state, float *saved,
                        void *workspace, size_t workspace_bytes, void *stream);
int rlca_selective_scan_bf16(const rlca_scan *p, rlca_steps out, float *final_state,
                             float *saved, void *workspace, size_t workspace_bytes,
                             void *stream);
int rlca_selective_scan_fp16(const rlca_scan *p, rlca_steps out, float *final_state,
                             float *saved, void *workspace, size_t workspace_bytes,
                             void *stream);

/* Gradients of sum(out * dout) + sum(final_state * d_final_state). `saved` is what the
 * forward call wrote for the same problem (init_state itself is not read). dz is given with
 * z, dD with D, ddt_bias with dt_bias; each of dD, ddt_bias, d_init_state nullable. */
typedef struct rlca_scan_grads {
    rlca_steps dout;                          /* [N,T,E] */
    const float *d_final_state;               /* [N,E,S], nullable = 0 */
    const float *saved;
    rlca_steps dx, ddt, dz;                   /* [N,T,E] */
    rlca_steps dB, dC;                        /* [N,T,G,S] */
    float *dA, *dD, *ddt_bias, *d_init_state; /* [E,S], [E], [E], [N,E,S] */
} rlca_scan_grads;

int rlca_selective_scan_backward(const rlca_scan *p, const rlca_scan_grads *g, void *workspace,
                                 size_t workspace_bytes, void *stream);
int rlca_selective_scan_backward_bf16(const rlca_scan *p, const rlca_scan_grads *g,
                                      void *workspace, size_t workspace_bytes, void *stream);
int rlca_selective_scan_backward_fp16(const rlca_scan *p, const rlca_scan_grads *g,
                                      void *workspace, size_t workspace_bytes, void *stream);

/* One step of N rows: p->T is 1 (the `step` strides are not used), p->init_state is the
 * state, p->rows is not used, out.row the output's row stride. Rows with reset[n] != 0
 * (nullable) start from 0. new_state [N,E,S] may be the state itself (updated in place). */
int rlca_selective_scan_step(const rlca_scan *p, const uint8_t *reset, rlca_steps out,
                             float *new_state, void *stream);
int rlca_selective_scan_step_bf16(const rlca_scan *p, const uint8_t *reset, rlca_steps out,
                                  float *new_state, void *stream);
int rlca_selective_scan_step_fp16(const rlca_scan *p, const uint8_t *reset, rlca_steps out,
                                  float *new_state, void *stream);

/* -------------------------------------------------------------- causal convolution
 *
 * One short filter per channel:
 *   p_t = bias[e] + sum_{k<K} weight[e,k] x_{t-K+1+k},   out_t = silu(p_t)   (silu; else p_t)
 * A tap before the episode's first step counts as 0; a tap before the window is
 * init_state's row (init_state [N, K-1, E], oldest first, of the data type). The final
 * state is the window's last K-1 inputs in that layout. 1 <= K <= RLCA_CONV_MAX_K.
 */
#define RLCA_CONV_MAX_K 8

typedef struct rlca_conv {
    int64_t N, T, E, K;
    rlca_steps x;                 /* [N,T,E] */
    const float *weight, *bias;   /* [E,K]; [E] nullable */
    rlca_rows rows;
    const void *init_state;       /* [N,K-1,E] contiguous, nullable */
    int32_t silu;
} rlca_conv;

int rlca_causal_conv(const rlca_conv *p, rlca_steps out, void *final_state, void *stream);
int rlca_causal_conv_bf16(const rlca_conv *p, rlca_steps out, void *final_state, void *stream);
int rlca_causal_conv_fp16(const rlca_conv *p, rlca_steps out, void *final_state, void *stream);

/* Gradients of sum(out * dout): dx [N,T,E], dweight [E,K], dbias [E] (nullable). The window
 * carried in is data: no gradient is taken with respect to it. */
size_t rlca_causal_conv_workspace_bytes(int64_t N, int64_t T, int64_t E, int64_t K);
int rlca_causal_conv_backward(const rlca_conv *p, rlca_steps dout, rlca_steps dx,
                              float *dweight, float *dbias, void *workspace,
                              size_t workspace_bytes, void *stream);
int rlca_causal_conv_backward_bf16(const rlca_conv *p, rlca_steps dout, rlca_steps dx,
                                   float *dweight, float *dbias, void *workspace,
                                   size_t workspace_bytes, void *stream);
int rlca_causal_conv_backward_fp16(const rlca_conv *p, rlca_steps dout, rlca_steps dx,
                                   float *dweight, float *dbias, void *workspace,
                                   size_t workspace_bytes, void *stream);

/* One step of N rows: p->T is 1, p->init_state the state (required when K > 1), p->rows not
 * used. Rows with reset[n] != 0 (nullable) start from a window of zeros. new_state
 * [N,K-1,E] may be the state itself. */
int rlca_causal_conv_step(const rlca_conv *p, const uint8_t *reset, rlca_steps out,
                          void *new_state, void *stream);
int rlca_causal_conv_step_bf16(const rlca_conv *p, const uint8_t *reset, rlca_steps out,
                               void *new_state, void *stream);
int rlca_causal_conv_step_fp16(const rlca_conv *p, const uint8_t *reset, rlca_steps out,
                               void *new_state, void *stream);

/* ----------------------------------------------------------------- token embedding
 *
 * out_i = scale * table[token_i], i < M; a token outside [0, V) (padding) gives a row of 0
 * and takes no gradient. tokens: int32 or int64 (token_bytes 4 or 8), contiguous [M]. table
 * [V, table_ld] and out [M, out_ld] of the data type, table_ld, out_ld >= D.
 * M < 2^31 and V < 2^31.
 */
int rlca_embed_tokens(const void *tokens, int32_t token_bytes, const void *table,
                      int64_t table_ld, float scale, int64_t M, int64_t V, int64_t D,
                      void *out, int64_t out_ld, void *stream);
int rlca_embed_tokens_bf16(const void *tokens, int32_t token_bytes, const void *table,
                           int64_t table_ld, float scale, int64_t M, int64_t V, int64_t D,
                           void *out, int64_t out_ld, void *stream);
int rlca_embed_tokens_fp16(const void *tokens, int32_t token_bytes, const void *table,
                           int64_t table_ld, float scale, int64_t M, int64_t V, int64_t D,
                           void *out, int64_t out_ld, void *stream);

/* dtable[v] = scale * sum of dout_i over the i with token_i = v, fp32 [V, D] contiguous,
 * every row written. The rows of a token are added in the order of i, in runs of fixed
 * length that are then added in order. */
size_t rlca_embed_tokens_workspace_bytes(int64_t M, int64_t V, int64_t D);
int rlca_embed_tokens_backward(const void *dout, int64_t dout_ld, const void *tokens,
                               int32_t token_bytes, float scale, int64_t M, int64_t V,
                               int64_t D, float *dtable, void *workspace,
                               size_t workspace_bytes, void *stream);
int rlca_embed_tokens_backward_bf16(const void *dout, int64_t dout_ld, const void *tokens,
                                    int32_t token_bytes, float scale, int64_t M, int64_t V,
                                    int64_t D, float *dtable, void *workspace,
                                    size_t workspace_bytes, void *stream);
int rlca_embed_tokens_backward_fp16(const void *dout, int64_t dout_ld, const void *tokens,
                                    int32_t token_bytes, float scale, int64_t M, int64_t V,
                                    int64_t D, float *dtable, void *workspace,
                                    size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* RLCA_SEQUENCE_H */

// C ABI of the sequence-model operators (declared in include/rlca_sequence.h): argument
// validation, then the operator's launches on the caller's stream. No allocation, no
// synchronisation, no change of the current device.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/rlca.h"
#include "buffers.cuh"
#include "conv.cuh"
#include "embed.cuh"
#include "scan.cuh"

namespace {

using namespace rlca::seq;
using rlca::Fmt;

// The activation as the scan's kernels address it. They form the addresses of whole tiles, of steps
// past the row's last too (a copy reads nothing there, but a 16-byte copy wants an aligned address all
// the same), so a stride that no element uses, which nothing has checked, becomes 0.
rlca_steps used_strides(const rlca_steps &a, int64_t N, int64_t T)
{
    return {a.ptr, N > 1 ? a.row : 0, T > 1 ? a.step : 0};
}

// ------------------------------------------------------------------ selective scan

bool scan_shape_ok(int64_t N, int64_t T, int64_t E, int64_t S, int64_t G)
{
    return N >= 0 && T >= 0 && T <= RLCA_MAX_T && E >= 0 && S >= 1 && S <= RLCA_SCAN_MAX_S &&
           G >= 1 && E % G == 0 && E <= INT32_MAX && product_fits(N, T + 16, E, 64) &&
           product_fits(N, T + 1, G, 512);
}

struct ScanWorkspace {
    size_t span_state, span_sum;  // both directions
    size_t forward;               // bytes the forward pass needs
    size_t bc, shares, bytes;     // backward
};

ScanWorkspace scan_workspace(int64_t N, int64_t T, int64_t E, int64_t S, int64_t G)
{
    const int64_t ch = scan_backward_channels(S), blocks = (E / G + ch - 1) / ch;
    const int64_t sp = 4 * scan_backward_lanes(S);
    ScanWorkspace w;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t r = at;
        at += align256(n);
        return r;
    };
    const int64_t forward = scan_forward_spans(N, T, E, S, G).spans;
    const int64_t backward = scan_backward_spans(N, T, E, S, G).spans;
    const int64_t spans = forward > backward ? forward : backward;
    w.span_state = take(spans > 1 ? (size_t)(N * spans * E * S) * 4 : 0);
    w.span_sum = take(spans > 1 ? (size_t)(N * spans * E) * 4 : 0);
    w.forward = forward > 1 ? at : 0;
    w.bc = take((size_t)(N * T * G * blocks * 2 * sp) * 4);
    w.shares = take((size_t)(N * backward * E * (S + 2)) * 4);
    w.bytes = at;
    return w;
}

ScanParams scan_params(const rlca_scan &p)
{
    ScanParams q;
    std::memset(&q, 0, sizeof(q));
    q.N = p.N;
    q.E = p.E;
    q.T = (int)p.T;
    q.S = (int)p.S;
    q.G = (int)p.G;
    q.Eg = (int)(p.E / p.G);
    q.x = used_strides(p.x, p.N, p.T);
    q.dt = used_strides(p.dt, p.N, p.T);
    q.z = used_strides(p.z, p.N, p.T);
    q.B = used_strides(p.B, p.N, p.T);
    q.C = used_strides(p.C, p.N, p.T);
    q.A = p.A;
    q.D = p.D;
    q.dt_bias = p.dt_bias;
    q.init = p.init_state;
    q.rows = RowFlags{p.rows.terminated, p.rows.truncated, p.rows.flag_ld, p.rows.lengths};
    q.softplus = p.dt_softplus != 0;
    q.spans = 1;
    return q;
}

void scan_inputs(Buffers &b, const rlca_scan &p, size_t es)
{
    b.steps(p.x, p.E, es, true, false);
    b.steps(p.dt, p.E, es, true, false);
    b.steps(p.z, p.E, es, false, false);
    b.steps(p.B, p.G * p.S, es, true, false);
    b.steps(p.C, p.G * p.S, es, true, false);
    b.in(p.A, p.E * p.S, 4);
    b.in(p.D, p.E, 4, false);
    b.in(p.dt_bias, p.E, 4, false);
}

bool scan_vectors(const rlca_scan &p, int V)
{
    return (p.E / p.G) % V == 0 && vectors(p.x, p.N, p.T, V) && vectors(p.dt, p.N, p.T, V) &&
           vectors(p.z, p.N, p.T, V);
}

int scan_forward(const rlca_scan *pp, rlca_steps out, float *final_state, float *saved, void *ws,
                 size_t ws_bytes, void *stream, Fmt f)
{
    if (!pp) return RLCA_ERR_NULL;
    const rlca_scan &p = *pp;
    if (!scan_shape_ok(p.N, p.T, p.E, p.S, p.G)) return RLCA_ERR_SHAPE;
    if (p.N == 0 || p.E == 0) return RLCA_OK;
    const size_t es = bytes_of(f);
    Buffers b(p.N, p.T);
    scan_inputs(b, p, es);
    b.rows(p.rows);
    b.in(p.init_state, p.N * p.E * p.S, 4, false);
    b.steps(out, p.E, es, true, true);
    b.out(final_state, p.N * p.E * p.S, 4, false);
    b.out(saved, (int64_t)(rlca_selective_scan_saved_bytes(p.N, p.T, p.E, p.S) / 4), 4, false);
    const ScanWorkspace w = scan_workspace(p.N, p.T, p.E, p.S, p.G);
    const int st = b.check(ws, ws_bytes, w.forward);
    if (st != RLCA_OK) return st;
    ScanParams q = scan_params(p);
    const int ch = scan_forward_channels(p.S);
    q.blocks_g = (q.Eg + ch - 1) / ch;
    const ScanSpans spans = scan_forward_spans(p.N, p.T, p.E, p.S, p.G);
    q.spans = spans.spans;
    q.span_steps = spans.steps;
    q.out = used_strides(out, p.N, p.T);
    q.final_state = final_state;
    q.saved = saved;
    q.span_state = reinterpret_cast<float *>(static_cast<char *>(ws) + w.span_state);
    q.span_sum = reinterpret_cast<float *>(static_cast<char *>(ws) + w.span_sum);
    const int V = 16 / (int)es;
    const bool vec = scan_vectors(p, V) && vectors(out, p.N, p.T, V);
    return status(in_format(f, [&](auto fmt) {
        return launch_scan_forward<decltype(fmt)::value>(q, vec, static_cast<cudaStream_t>(stream));
    }));
}

int scan_backward(const rlca_scan *pp, const rlca_scan_grads *gg, void *ws, size_t ws_bytes,
                  void *stream_, Fmt f)
{
    if (!pp || !gg) return RLCA_ERR_NULL;
    const rlca_scan &p = *pp;
    const rlca_scan_grads &g = *gg;
    if (!scan_shape_ok(p.N, p.T, p.E, p.S, p.G)) return RLCA_ERR_SHAPE;
    if (p.E == 0) return RLCA_OK;
    const size_t es = bytes_of(f);
    const int64_t states = p.N * p.E * p.S;
    Buffers b(p.N, p.T);
    scan_inputs(b, p, es);
    b.rows(p.rows);
    b.steps(g.dout, p.E, es, true, false);
    b.in(g.d_final_state, states, 4, false);
    b.in(g.saved, (int64_t)(rlca_selective_scan_saved_bytes(p.N, p.T, p.E, p.S) / 4), 4);
    b.steps(g.dx, p.E, es, true, true);
    b.steps(g.ddt, p.E, es, true, true);
    if (p.z.ptr) b.steps(g.dz, p.E, es, true, true);
    b.steps(g.dB, p.G * p.S, es, true, true);
    b.steps(g.dC, p.G * p.S, es, true, true);
    b.out(g.dA, p.E * p.S, 4);
    b.out(g.dD, p.E, 4, false);
    b.out(g.ddt_bias, p.E, 4, false);
    b.out(g.d_init_state, states, 4, false);
    const ScanWorkspace w = scan_workspace(p.N, p.T, p.E, p.S, p.G);
    const int st = b.check(ws, ws_bytes, w.bytes);
    if (st != RLCA_OK) return st;
    ScanParams q = scan_params(p);
    const int ch = scan_backward_channels(p.S);
    q.blocks_g = (q.Eg + ch - 1) / ch;
    const ScanSpans spans = scan_backward_spans(p.N, p.T, p.E, p.S, p.G);
    q.spans = spans.spans;
    q.span_steps = spans.steps;
    q.dout = used_strides(g.dout, p.N, p.T);
    q.d_final = g.d_final_state;
    q.saved = const_cast<float *>(g.saved);
    q.dx = used_strides(g.dx, p.N, p.T);
    q.ddt = used_strides(g.ddt, p.N, p.T);
    q.dz = used_strides(g.dz, p.N, p.T);
    q.dB = used_strides(g.dB, p.N, p.T);
    q.dC = used_strides(g.dC, p.N, p.T);
    q.d_init = g.d_init_state;
    char *base = static_cast<char *>(ws);
    q.span_state = reinterpret_cast<float *>(base + w.span_state);
    q.span_sum = reinterpret_cast<float *>(base + w.span_sum);
    q.part_bc = reinterpret_cast<float *>(base + w.bc);
    q.part_p = reinterpret_cast<float *>(base + w.shares);
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    const int V = 16 / (int)es;
    const bool vec = scan_vectors(p, V) && vectors(g.dout, p.N, p.T, V) &&
                     vectors(g.dx, p.N, p.T, V) && vectors(g.ddt, p.N, p.T, V) &&
                     (!p.z.ptr || vectors(g.dz, p.N, p.T, V));
    cudaError_t e = cudaSuccess;
    if (p.N > 0)
        e = in_format(f, [&](auto fmt) {
            return launch_scan_backward<decltype(fmt)::value>(q, vec, stream);
        });
    if (e == cudaSuccess)
        e = launch_sum_rows(SumRows{q.part_p, p.N * q.spans, p.E * (p.S + 2),
                                    {p.E * p.S, p.E, p.E}, {g.dA, g.dD, g.ddt_bias}, 0},
                            stream);
    return status(e);
}

int scan_step(const rlca_scan *pp, const uint8_t *reset, rlca_steps out, float *new_state,
              void *stream, Fmt f)
{
    if (!pp) return RLCA_ERR_NULL;
    const rlca_scan &p = *pp;
    if (p.T != 1 || !scan_shape_ok(p.N, p.T, p.E, p.S, p.G)) return RLCA_ERR_SHAPE;
    if (p.N == 0 || p.E == 0) return RLCA_OK;
    const size_t es = bytes_of(f);
    Buffers b(p.N, 1);
    scan_inputs(b, p, es);
    b.in(reset, p.N, 1, false);
    b.steps(out, p.E, es, true, true);
    b.state(p.init_state, new_state, p.N * p.E * p.S, 4, false);
    const int st = b.check(nullptr, 0, 0);
    if (st != RLCA_OK) return st;
    ScanParams q = scan_params(p);
    q.out = used_strides(out, p.N, p.T);
    q.reset = reset;
    q.final_state = new_state;
    const int V = 16 / (int)es;
    const bool vec = p.S % 8 == 0 && vectors(p.B, p.N, 1, V) && vectors(p.C, p.N, 1, V);
    return status(in_format(f, [&](auto fmt) {
        return launch_scan_step<decltype(fmt)::value>(q, vec, static_cast<cudaStream_t>(stream));
    }));
}

// ------------------------------------------------------------------ convolution

bool conv_shape_ok(int64_t N, int64_t T, int64_t E, int64_t K)
{
    return N >= 0 && T >= 0 && T <= RLCA_MAX_T && E >= 0 && E <= INT32_MAX && K >= 1 &&
           K <= RLCA_CONV_MAX_K && product_fits(N, T + 128, E, 64);
}

ConvParams conv_params(const rlca_conv &p)
{
    ConvParams q;
    std::memset(&q, 0, sizeof(q));
    q.N = p.N;
    q.E = p.E;
    q.T = (int)p.T;
    q.K = (int)p.K;
    q.x = p.x;
    q.weight = p.weight;
    q.bias = p.bias;
    q.rows = RowFlags{p.rows.terminated, p.rows.truncated, p.rows.flag_ld, p.rows.lengths};
    q.init = p.init_state;
    q.silu = p.silu != 0;
    return q;
}

void conv_inputs(Buffers &b, const rlca_conv &p, size_t es)
{
    b.steps(p.x, p.E, es, true, false);
    b.in(p.weight, p.E * p.K, 4);
    b.in(p.bias, p.E, 4, false);
}

int conv_forward(const rlca_conv *pp, rlca_steps out, void *final_state, void *stream, Fmt f)
{
    if (!pp) return RLCA_ERR_NULL;
    const rlca_conv &p = *pp;
    if (!conv_shape_ok(p.N, p.T, p.E, p.K)) return RLCA_ERR_SHAPE;
    if (p.N == 0 || p.E == 0) return RLCA_OK;
    const size_t es = bytes_of(f);
    const int64_t states = p.N * (p.K - 1) * p.E;
    Buffers b(p.N, p.T);
    conv_inputs(b, p, es);
    b.rows(p.rows);
    b.in(p.init_state, states, es, false);
    b.steps(out, p.E, es, true, true);
    b.out(final_state, states, es, false);
    const int st = b.check(nullptr, 0, 0);
    if (st != RLCA_OK) return st;
    if (p.T == 0 && (!final_state || p.K == 1)) return RLCA_OK;
    ConvParams q = conv_params(p);
    q.out = out;
    q.final_state = p.K > 1 ? final_state : nullptr;
    const int V = 16 / (int)es;
    const bool vec = p.E % V == 0 && vectors(p.x, p.N, p.T, V) && vectors(out, p.N, p.T, V) &&
                     aligned16(p.init_state) && aligned16(final_state);
    return status(in_format(f, [&](auto fmt) {
        return launch_conv_forward<decltype(fmt)::value>(q, vec, static_cast<cudaStream_t>(stream));
    }));
}

int conv_backward(const rlca_conv *pp, rlca_steps dout, rlca_steps dx, float *dweight,
                  float *dbias, void *ws, size_t ws_bytes, void *stream_, Fmt f)
{
    if (!pp) return RLCA_ERR_NULL;
    const rlca_conv &p = *pp;
    if (!conv_shape_ok(p.N, p.T, p.E, p.K)) return RLCA_ERR_SHAPE;
    if (p.E == 0) return RLCA_OK;
    const size_t es = bytes_of(f);
    Buffers b(p.N, p.T);
    conv_inputs(b, p, es);
    b.rows(p.rows);
    b.in(p.init_state, p.N * (p.K - 1) * p.E, es, false);
    b.steps(dout, p.E, es, true, false);
    b.steps(dx, p.E, es, true, true);
    b.out(dweight, p.E * p.K, 4);
    b.out(dbias, p.E, 4, false);
    const int st = b.check(ws, ws_bytes, rlca_causal_conv_workspace_bytes(p.N, p.T, p.E, p.K));
    if (st != RLCA_OK) return st;
    ConvParams q = conv_params(p);
    q.dout = dout;
    q.dx = dx;
    q.part_w = static_cast<float *>(ws);
    const int V = 16 / (int)es;
    const bool vec = p.E % V == 0 && vectors(p.x, p.N, p.T, V) && vectors(dout, p.N, p.T, V) &&
                     vectors(dx, p.N, p.T, V) && aligned16(p.init_state);
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    cudaError_t e = cudaSuccess;
    if (p.N > 0 && p.T > 0)
        e = in_format(f, [&](auto fmt) {
            return launch_conv_backward<decltype(fmt)::value>(q, vec, stream);
        });
    if (e == cudaSuccess)
        e = launch_sum_rows(SumRows{q.part_w, p.N * conv_span_blocks(p.T), p.E * (p.K + 1),
                                    {p.E * p.K, p.E, 0}, {dweight, dbias, nullptr}, (int)p.K},
                            stream);
    return status(e);
}

int conv_step(const rlca_conv *pp, const uint8_t *reset, rlca_steps out, void *new_state,
              void *stream, Fmt f)
{
    if (!pp) return RLCA_ERR_NULL;
    const rlca_conv &p = *pp;
    if (p.T != 1 || !conv_shape_ok(p.N, p.T, p.E, p.K)) return RLCA_ERR_SHAPE;
    if (p.N == 0 || p.E == 0) return RLCA_OK;
    const size_t es = bytes_of(f);
    const int64_t states = p.N * (p.K - 1) * p.E;
    Buffers b(p.N, 1);
    conv_inputs(b, p, es);
    b.in(reset, p.N, 1, false);
    b.steps(out, p.E, es, true, true);
    b.state(p.init_state, new_state, states, es, true);
    const int st = b.check(nullptr, 0, 0);
    if (st != RLCA_OK) return st;
    ConvParams q = conv_params(p);
    q.out = out;
    q.reset = reset;
    q.final_state = new_state;
    const int V = 16 / (int)es;
    const bool vec = p.E % V == 0 && vectors(p.x, p.N, 1, V) && vectors(out, p.N, 1, V) &&
                     aligned16(p.init_state) && aligned16(new_state);
    return status(in_format(f, [&](auto fmt) {
        return launch_conv_step<decltype(fmt)::value>(q, vec, static_cast<cudaStream_t>(stream));
    }));
}

// ------------------------------------------------------------------ embedding

bool embed_shape_ok(int32_t token_bytes, int64_t M, int64_t V, int64_t D, int64_t ld)
{
    return M >= 0 && M <= INT32_MAX && V >= 0 && V <= INT32_MAX && D >= 0 && D <= INT32_MAX &&
           ld >= D && (M == 0 || ld < kMaxExtent / 8 / M) && (V == 0 || ld < kMaxExtent / 8 / V) &&
           (token_bytes == 4 || token_bytes == 8);
}

int embed_forward(const void *tokens, int32_t token_bytes, const void *table, int64_t table_ld,
                  float scale, int64_t M, int64_t V, int64_t D, void *out, int64_t out_ld,
                  void *stream, Fmt f)
{
    if (!embed_shape_ok(token_bytes, M, V, D, table_ld) ||
        !embed_shape_ok(token_bytes, M, V, D, out_ld))
        return RLCA_ERR_SHAPE;
    if (M == 0 || D == 0) return RLCA_OK;
    const size_t es = bytes_of(f);
    Buffers b(1, 1);
    b.in(tokens, M, (size_t)token_bytes);
    b.in(table, V ? (V - 1) * table_ld + D : 0, es);
    b.out(out, (M - 1) * out_ld + D, es);
    const int st = b.check(nullptr, 0, 0);
    if (st != RLCA_OK) return st;
    EmbedParams q;
    std::memset(&q, 0, sizeof(q));
    q.tokens = tokens;
    q.token_bytes = token_bytes;
    q.table = table;
    q.ld = table_ld;
    q.out = out;
    q.out_ld = out_ld;
    q.scale = scale;
    q.M = M;
    q.V = V;
    q.D = D;
    const int w = 16 / (int)es;
    const bool vec = D % w == 0 && table_ld % w == 0 && out_ld % w == 0 && aligned16(table) &&
                     aligned16(out);
    return status(in_format(f, [&](auto fmt) {
        return launch_embed<decltype(fmt)::value>(q, vec, static_cast<cudaStream_t>(stream));
    }));
}

int embed_backward(const void *dout, int64_t dout_ld, const void *tokens, int32_t token_bytes,
                   float scale, int64_t M, int64_t V, int64_t D, float *dtable, void *ws,
                   size_t ws_bytes, void *stream_, Fmt f)
{
    if (!embed_shape_ok(token_bytes, M, V, D, dout_ld)) return RLCA_ERR_SHAPE;
    if (V == 0 || D == 0) return RLCA_OK;
    const size_t es = bytes_of(f);
    Buffers b(1, 1);
    b.in(tokens, M, (size_t)token_bytes);
    b.in(dout, M ? (M - 1) * dout_ld + D : 0, es);
    b.out(dtable, V * D, 4);
    const EmbedWorkspace w = embed_workspace(M, V, D);
    const int st = b.check(ws, ws_bytes, w.bytes);
    if (st != RLCA_OK) return st;
    EmbedParams q;
    std::memset(&q, 0, sizeof(q));
    q.tokens = tokens;
    q.token_bytes = token_bytes;
    q.dout = dout;
    q.ld = dout_ld;
    q.dtable = dtable;
    q.scale = scale;
    q.M = M;
    q.V = V;
    q.D = D;
    char *base = static_cast<char *>(ws);
    for (int i = 0; i < 2; ++i) q.pairs[i] = reinterpret_cast<uint2 *>(base + w.pairs[i]);
    q.present = reinterpret_cast<uint8_t *>(base + w.present);
    q.partial = reinterpret_cast<float *>(base + w.partial);
    const int v = 16 / (int)es;
    const bool vec = D % v == 0 && dout_ld % v == 0 && aligned16(dout) && aligned16(dtable);
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    cudaError_t e = M > 0 ? launch_embed_sort(q, stream) : cudaSuccess;
    if (e == cudaSuccess)
        e = in_format(f, [&](auto fmt) {
            return launch_embed_sum<decltype(fmt)::value>(q, vec, stream);
        });
    if (e == cudaSuccess && M > 0) e = launch_embed_join(q, stream);
    return status(e);
}

}  // namespace

extern "C" {

size_t rlca_selective_scan_workspace_bytes(int64_t N, int64_t T, int64_t E, int64_t S, int64_t G)
{
    return scan_shape_ok(N, T, E, S, G) ? scan_workspace(N, T, E, S, G).bytes : 0;
}

size_t rlca_selective_scan_forward_workspace_bytes(int64_t N, int64_t T, int64_t E, int64_t S,
                                                   int64_t G)
{
    return scan_shape_ok(N, T, E, S, G) ? scan_workspace(N, T, E, S, G).forward : 0;
}

size_t rlca_selective_scan_saved_bytes(int64_t N, int64_t T, int64_t E, int64_t S)
{
    if (!scan_shape_ok(N, T, E, S, 1)) return 0;
    return (size_t)(N * ((T + RLCA_SCAN_CHUNK - 1) / RLCA_SCAN_CHUNK) * E * S) * 4;
}

size_t rlca_causal_conv_workspace_bytes(int64_t N, int64_t T, int64_t E, int64_t K)
{
    if (!conv_shape_ok(N, T, E, K)) return 0;
    return align256((size_t)(N * conv_span_blocks(T) * (K + 1) * E) * 4);
}

size_t rlca_embed_tokens_workspace_bytes(int64_t M, int64_t V, int64_t D)
{
    return embed_shape_ok(4, M, V, D, D) ? embed_workspace(M, V, D).bytes : 0;
}

#define RLCA_SEQUENCE_ENTRY_POINTS(SUFFIX, FMT)                                                  \
    int rlca_selective_scan##SUFFIX(const rlca_scan *p, rlca_steps out, float *final_state,      \
                                    float *saved, void *workspace, size_t workspace_bytes,       \
                                    void *stream)                                                \
    {                                                                                            \
        return scan_forward(p, out, final_state, saved, workspace, workspace_bytes, stream,      \
                            FMT);                                                                \
    }                                                                                            \
    int rlca_selective_scan_backward##SUFFIX(const rlca_scan *p, const rlca_scan_grads *g,       \
                                             void *workspace, size_t workspace_bytes,            \
                                             void *stream)                                       \
    {                                                                                            \
        return scan_backward(p, g, workspace, workspace_bytes, stream, FMT);                     \
    }                                                                                            \
    int rlca_selective_scan_step##SUFFIX(const rlca_scan *p, const uint8_t *reset,               \
                                         rlca_steps out, float *new_state, void *stream)         \
    {                                                                                            \
        return scan_step(p, reset, out, new_state, stream, FMT);                                 \
    }                                                                                            \
    int rlca_causal_conv##SUFFIX(const rlca_conv *p, rlca_steps out, void *final_state,          \
                                 void *stream)                                                   \
    {                                                                                            \
        return conv_forward(p, out, final_state, stream, FMT);                                   \
    }                                                                                            \
    int rlca_causal_conv_backward##SUFFIX(const rlca_conv *p, rlca_steps dout, rlca_steps dx,    \
                                          float *dweight, float *dbias, void *workspace,         \
                                          size_t workspace_bytes, void *stream)                  \
    {                                                                                            \
        return conv_backward(p, dout, dx, dweight, dbias, workspace, workspace_bytes, stream,    \
                             FMT);                                                               \
    }                                                                                            \
    int rlca_causal_conv_step##SUFFIX(const rlca_conv *p, const uint8_t *reset, rlca_steps out,  \
                                      void *new_state, void *stream)                             \
    {                                                                                            \
        return conv_step(p, reset, out, new_state, stream, FMT);                                 \
    }                                                                                            \
    int rlca_embed_tokens##SUFFIX(const void *tokens, int32_t token_bytes, const void *table,    \
                                  int64_t table_ld, float scale, int64_t M, int64_t V,           \
                                  int64_t D, void *out, int64_t out_ld, void *stream)            \
    {                                                                                            \
        return embed_forward(tokens, token_bytes, table, table_ld, scale, M, V, D, out, out_ld,  \
                             stream, FMT);                                                       \
    }                                                                                            \
    int rlca_embed_tokens_backward##SUFFIX(                                                      \
        const void *dout, int64_t dout_ld, const void *tokens, int32_t token_bytes, float scale, \
        int64_t M, int64_t V, int64_t D, float *dtable, void *workspace, size_t workspace_bytes, \
        void *stream)                                                                            \
    {                                                                                            \
        return embed_backward(dout, dout_ld, tokens, token_bytes, scale, M, V, D, dtable,        \
                              workspace, workspace_bytes, stream, FMT);                          \
    }

RLCA_SEQUENCE_ENTRY_POINTS(, Fmt::kF32)
RLCA_SEQUENCE_ENTRY_POINTS(_bf16, Fmt::kBF16)
RLCA_SEQUENCE_ENTRY_POINTS(_fp16, Fmt::kF16)

#undef RLCA_SEQUENCE_ENTRY_POINTS

}  // extern "C"

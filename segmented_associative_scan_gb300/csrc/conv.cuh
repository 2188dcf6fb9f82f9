// Short causal convolution, one filter per channel, that does not look past the start of
// an episode: p_t = bias + sum_k w_k x_{t-K+1+k}, out = silu(p).
//
// Memory-bound: a thread owns a vector of channels and walks a span of steps with the
// last K - 1 inputs in registers, so each input is read once (plus K - 1 rows in front of
// every span) and each output written once.
#pragma once

#include "sequence.cuh"

namespace rlca {
namespace seq {

constexpr int kConvThreads = 128;
constexpr int kConvSpan = 32;       // steps a thread owns
constexpr int kConvLanes = 32;      // backward: channel vectors side by side in a CTA,
constexpr int kConvSpans = 4;       // and spans of steps

struct ConvParams {
    int64_t N, E;
    int T, K;
    rlca_steps x, out, dout, dx;
    const float *weight, *bias;
    RowFlags rows;
    const void *init;
    void *final_state;
    int silu;
    const uint8_t *reset;
    float *part_w;  // [N * span blocks, K + 1, E] shares of dweight and dbias
    float *dweight, *dbias;
};

inline int64_t conv_span_blocks(int64_t T)
{
    return (T + kConvSpan * kConvSpans - 1) / (kConvSpan * kConvSpans);
}

// The filter's taps in the last K of KM places.
template <int V, int KM>
struct Taps {
    float w[KM][V];
    float bias[V];
};

template <int V, int KM>
__device__ __forceinline__ void load_taps(const ConvParams &p, int64_t e, Taps<V, KM> &f)
{
#pragma unroll
    for (int i = 0; i < V; ++i) {
        f.bias[i] = p.bias ? __ldg(p.bias + e + i) : 0.f;
#pragma unroll
        for (int k = 0; k < KM; ++k)
            f.w[k][i] = k >= KM - p.K ? __ldg(p.weight + (e + i) * p.K + k - (KM - p.K)) : 0.f;
    }
}

template <int V, int KM>
__device__ __forceinline__ void clear_window(float (&win)[KM][V])
{
#pragma unroll
    for (int k = 0; k < KM; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) win[k][i] = 0.f;
}

// Takes the input of the next step into the window's last place.
template <typename T, int V, int KM>
__device__ __forceinline__ void push_window(float (&win)[KM][V], const Pack<T, V> &x)
{
#pragma unroll
    for (int k = 0; k + 1 < KM; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) win[k][i] = win[k + 1][i];
#pragma unroll
    for (int i = 0; i < V; ++i) win[KM - 1][i] = widen(x.e[i]);
}

// The row (t < 0: of the window carried in) that step t takes into the window.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> conv_input(const ConvParams &p, int64_t n, int t, int64_t e)
{
    if (t >= 0)
        return load_pack<T, V>(static_cast<const T *>(p.x.ptr) + n * p.x.row +
                               (int64_t)t * p.x.step + e);
    if (!p.init) return zero_pack<T, V>();
    return load_pack<T, V>(static_cast<const T *>(p.init) +
                           (n * (p.K - 1) + p.K - 1 + t) * p.E + e);
}

// The K - 1 inputs before step t0, those of earlier episodes left out.
template <typename T, int V, int KM>
__device__ __forceinline__ void open_window(const ConvParams &p, int64_t n, int t0, int64_t e,
                                            float (&win)[KM][V])
{
    clear_window<V, KM>(win);
    for (int t = t0 - (p.K - 1); t < t0; ++t) {
        if (t > 0 && step_ended(p.rows, n, t - 1)) clear_window<V, KM>(win);
        push_window<T, V, KM>(win, conv_input<T, V>(p, n, t, e));
    }
}

// p_t for the window that ends with x_t. Places that hold no tap are not multiplied: an Inf
// there must not turn into a NaN.
template <int V, int KM>
__device__ __forceinline__ void apply_taps(const Taps<V, KM> &f, const float (&win)[KM][V], int K,
                                           float (&acc)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = f.bias[i];
#pragma unroll
    for (int k = 0; k < KM; ++k)
        if (k >= KM - K)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(f.w[k][i], win[k][i], acc[i]);
}

template <typename T, int V, int KM>
__global__ void __launch_bounds__(kConvThreads) conv_forward_kernel(const ConvParams p)
{
    grid_dependency_sync();
    const int64_t vecs = p.E / V;
    const int64_t spans = p.T ? (p.T + kConvSpan - 1) / kConvSpan : 1;
    const int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
    const int64_t e = (i % vecs) * V, ns = i / vecs;
    const int64_t n = ns / spans;
    if (n >= p.N) return;
    const int t0 = (int)(ns % spans) * kConvSpan;
    const int t1 = p.T - t0 < kConvSpan ? p.T : t0 + kConvSpan;
    const int len = row_length(p.rows, n, p.T);
    const int end = len < t1 ? len : t1;
    T *out = static_cast<T *>(const_cast<void *>(p.out.ptr)) + n * p.out.row + e;

    Taps<V, KM> f;
    load_taps<V, KM>(p, e, f);
    float win[KM][V];
    const bool owns_final =
        p.final_state && (len > 0 ? t0 < len && len <= t1 : ns % spans == 0);
    if (t0 < end || owns_final) open_window<T, V, KM>(p, n, t0, e, win);
#pragma unroll 4
    for (int t = t0; t < end; ++t) {
        if (t > 0 && step_ended(p.rows, n, t - 1)) clear_window<V, KM>(win);
        push_window<T, V, KM>(win, conv_input<T, V>(p, n, t, e));
        float acc[V];
        apply_taps<V, KM>(f, win, p.K, acc);
        Pack<T, V> o;
#pragma unroll
        for (int k = 0; k < V; ++k) o.e[k] = narrow<T>(p.silu ? silu(acc[k]) : acc[k]);
        store_pack<T, V>(out + (int64_t)t * p.out.step, o);
    }
    for (int t = t0 > end ? t0 : end; t < t1; ++t)
        store_pack<T, V>(out + (int64_t)t * p.out.step, zero_pack<T, V>());
    if (owns_final) {
        if (len > 0 && step_ended(p.rows, n, len - 1)) clear_window<V, KM>(win);
        T *dst = static_cast<T *>(p.final_state) + n * (p.K - 1) * p.E + e;
#pragma unroll
        for (int k = 1; k < KM; ++k) {
            if (k < KM - p.K + 1) continue;
            Pack<T, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) o.e[j] = narrow<T>(win[k][j]);
            store_pack<T, V>(dst + (int64_t)(k - (KM - p.K + 1)) * p.E, o);
        }
    }
}

// dp_t = dout_t silu'(p_t); dx_t = sum_j w_{K-1-j} dp_{t+j} over the steps of the same
// episode; dw_k = sum_t dp_t x_{t-K+1+k}; db = sum_t dp_t. A thread owns the dx of its span
// and the shares of dw and db of its steps; it runs K - 1 steps past the span's end for dx.
template <typename T, int V, int KM>
__global__ void __launch_bounds__(kConvLanes *kConvSpans) conv_backward_kernel(const ConvParams p)
{
    __shared__ float sh[kConvSpans][KM + 1][kConvLanes * V];
    grid_dependency_sync();
    const int lane = threadIdx.x % kConvLanes, ty = threadIdx.x / kConvLanes;
    const int64_t vecs = p.E / V;
    const int64_t lane_blocks = (vecs + kConvLanes - 1) / kConvLanes;
    const int64_t span_blocks = (p.T + kConvSpan * kConvSpans - 1) / (kConvSpan * kConvSpans);
    const int64_t nb = blockIdx.x / lane_blocks;  // (n, span block)
    const int64_t n = nb / span_blocks;
    const int64_t e0 = (blockIdx.x % lane_blocks) * kConvLanes * V;
    const int64_t e = e0 + lane * V;
    const int t0 = ((int)(nb % span_blocks) * kConvSpans + ty) * kConvSpan;
    const int t1 = t0 >= p.T ? t0 : (p.T - t0 < kConvSpan ? p.T : t0 + kConvSpan);
    const int len = row_length(p.rows, n, p.T);

    float dw[KM][V], db[V];
    clear_window<V, KM>(dw);
#pragma unroll
    for (int i = 0; i < V; ++i) db[i] = 0.f;
    if (e < p.E && t0 < t1) {
        const T *dout = static_cast<const T *>(p.dout.ptr) + n * p.dout.row + e;
        T *dx = static_cast<T *>(const_cast<void *>(p.dx.ptr)) + n * p.dx.row + e;
        Taps<V, KM> f;
        load_taps<V, KM>(p, e, f);
        if (t0 < len) {
            const int stop = t1 + p.K - 1 < len ? t1 + p.K - 1 : len;  // steps that are run
            float win[KM][V], acc[KM][V];  // acc[j]: dx of step t - j so far
            open_window<T, V, KM>(p, n, t0, e, win);
            clear_window<V, KM>(acc);
            int reach = p.K - 1;  // earlier steps of the episode that x_t's filter sees
            auto emit = [&](int t, const float (&v)[V]) {
                if (t < t0 || t >= t1) return;
                Pack<T, V> o;
#pragma unroll
                for (int i = 0; i < V; ++i) o.e[i] = narrow<T>(v[i]);
                store_pack<T, V>(dx + (int64_t)t * p.dx.step, o);
            };
#pragma unroll 2
            for (int t = t0; t < stop; ++t) {
                reach = reach + 1 < p.K ? reach + 1 : p.K - 1;
                if (t > 0 && step_ended(p.rows, n, t - 1)) {
                    clear_window<V, KM>(win);
                    reach = 0;
                }
                push_window<T, V, KM>(win, conv_input<T, V>(p, n, t, e));
                const Pack<T, V> go = load_pack<T, V>(dout + (int64_t)t * p.dout.step);
                float dp[V];
                apply_taps<V, KM>(f, win, p.K, dp);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float sg = sigmoid(dp[i]);
                    dp[i] = widen(go.e[i]) * (p.silu ? sg * fmaf(dp[i], 1.f - sg, 1.f) : 1.f);
                }
                // One step on: acc[j] moves to acc[j + 1].
#pragma unroll
                for (int j = KM - 1; j >= 0; --j) {
                    if (j >= p.K) continue;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float before = j > 0 ? acc[j - 1][i] : 0.f;
                        acc[j][i] =
                            j <= reach ? fmaf(f.w[KM - 1 - j][i], dp[i], before) : before;
                    }
                }
                if (t < t1) {
#pragma unroll
                    for (int k = 0; k < KM; ++k)
                        if (k >= KM - p.K)
#pragma unroll
                            for (int i = 0; i < V; ++i)
                                dw[k][i] = fmaf(dp[i], win[k][i], dw[k][i]);
#pragma unroll
                    for (int i = 0; i < V; ++i) db[i] += dp[i];
                }
#pragma unroll
                for (int j = 0; j < KM; ++j)
                    if (j == p.K - 1) emit(t - j, acc[j]);
            }
#pragma unroll
            for (int j = 0; j + 1 < KM; ++j)
                if (j < p.K - 1) emit(stop - 1 - j, acc[j]);
        }
        for (int t = t0 > len ? t0 : len; t < t1; ++t)
            store_pack<T, V>(dx + (int64_t)t * p.dx.step, zero_pack<T, V>());
    }
    // The spans of the CTA add up in order.
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < KM; ++k) sh[ty][k][lane * V + i] = dw[k][i];
        sh[ty][KM][lane * V + i] = db[i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < (p.K + 1) * kConvLanes * V; c += kConvLanes * kConvSpans) {
        const int k = c / (kConvLanes * V), l = c % (kConvLanes * V);
        if (e0 + l >= p.E) continue;
        float sum = 0.f;
#pragma unroll
        for (int y = 0; y < kConvSpans; ++y) sum += sh[y][k + KM - p.K][l];
        p.part_w[(nb * (p.K + 1) + k) * p.E + e0 + l] = sum;
    }
}

// dweight [E, K] and dbias [E] from the shares [shares, K + 1, E], added in order.
cudaError_t launch_conv_weight(const ConvParams &p, cudaStream_t stream);

// One step of N rows. A thread owns one channel of one row.
template <typename T>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(const ConvParams p)
{
    grid_dependency_sync();
    const int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
    const int64_t n = i / p.E, e = i % p.E;
    if (n >= p.N) return;
    const bool keep = p.init && !(p.reset && __ldg(p.reset + n));
    const T *in = static_cast<const T *>(p.init) + n * (p.K - 1) * p.E + e;
    T *next = static_cast<T *>(p.final_state) + n * (p.K - 1) * p.E + e;
    const T x = static_cast<const T *>(p.x.ptr)[n * p.x.row + e];
    float acc = p.bias ? __ldg(p.bias + e) : 0.f;
    for (int k = 0; k + 1 < p.K; ++k) {
        const T v = keep ? in[(int64_t)k * p.E] : narrow<T>(0.f);
        acc = fmaf(__ldg(p.weight + e * p.K + k), widen(v), acc);
        if (k > 0) next[(int64_t)(k - 1) * p.E] = v;
    }
    if (p.K > 1) next[(int64_t)(p.K - 2) * p.E] = x;
    acc = fmaf(__ldg(p.weight + e * p.K + p.K - 1), widen(x), acc);
    static_cast<T *>(const_cast<void *>(p.out.ptr))[n * p.out.row + e] =
        narrow<T>(p.silu ? silu(acc) : acc);
}

}  // namespace seq
}  // namespace rlca

// Short causal convolution, one filter per channel, that does not look past the start of
// an episode: p_t = bias + sum_k w_k x_{t-K+1+k}, out = silu(p).
//
// Memory-bound: a lane owns a vector of channels and its warp a span of steps, with the last
// K - 1 inputs in registers, so each input is read once (plus K - 1 rows in front of every
// span) and each output written once. Where episodes start is one word of bits per span, so
// nothing that is read decides on the next read: several steps' loads are in flight at once.
//
// [16, 1024, 2048] x 4 taps, bf16: forward 43 us for 134 MB, backward 88 us for 201 MB (HBM needs
// 20 and 30); in fp32 [4, 4096, 2048] 49 us for 268 MB, 5.5 TB/s, and 86 for 403 MB. In 16 bits it is
// latency that bounds it: 24 instructions forward and 49 backward to an element keep the issue
// slots 46 % busy, at 17 and 14 warps to an SM that wait for their loads most of the time. dweight and
// dbias are sums of 32 steps, 4 spans and then of CTAs: 1.4e-7 off, 1.1e-7 for a sum in pairs; sums of
// 8 steps in front gave 1.2e-7 and took 124 us.
#pragma once

#include "sequence.cuh"

namespace rlca {
namespace seq {

constexpr int kConvWarps = 4;
constexpr int kConvThreads = 32 * kConvWarps;
constexpr int kConvSpan = 32;       // steps of a warp: one word of flags
// Steps of a batch: a batch's loads are in flight while the batch before it is computed.
constexpr int kConvBatch = 4;
constexpr int kConvBackBatch = 4;

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
};

// A CTA's warps take consecutive spans of the same channels (backward, they add up their
// shares of dweight and dbias).
inline int64_t conv_span_blocks(int64_t T)
{
    return (T + kConvSpan * kConvWarps - 1) / (kConvSpan * kConvWarps);
}

template <int V, int K>
struct Taps {
    float w[K][V];
    float bias[V];
};

// The filters of a CTA's 32 V channels, [tap][channel], read in one sweep (a lane reading its own
// [channel][tap] rows would touch a line of memory per lane and load) and padded so that
// neighbouring taps of a channel fall into different banks.
template <int V>
struct TapRows {
    float w[RLCA_CONV_MAX_K][32 * V + 8];
};

template <int V>
__device__ __forceinline__ void stage_taps(const ConvParams &p, int64_t e0, TapRows<V> &sh)
{
    for (int i = threadIdx.x; i < 32 * V * p.K; i += kConvThreads) {
        const int c = i / p.K, k = i - c * p.K;
        if (e0 + c < p.E) sh.w[k][c] = __ldg(p.weight + e0 * p.K + i);
    }
}

template <int V, int K>
__device__ __forceinline__ void load_taps(const ConvParams &p, int64_t e, const TapRows<V> &sh,
                                          Taps<V, K> &f)
{
    const int c = (threadIdx.x & 31) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        f.bias[i] = p.bias ? __ldg(p.bias + e + i) : 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) f.w[k][i] = sh.w[k][c + i];
    }
}

template <int V, int K>
__device__ __forceinline__ void clear_window(float (&win)[K][V])
{
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) win[k][i] = 0.f;
}

// Takes the input of the next step into the window's last place.
template <typename T, int V, int K>
__device__ __forceinline__ void push_window(float (&win)[K][V], const Pack<T, V> &x)
{
#pragma unroll
    for (int k = 0; k + 1 < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) win[k][i] = win[k + 1][i];
#pragma unroll
    for (int i = 0; i < V; ++i) win[K - 1][i] = widen(x.e[i]);
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

// The K - 1 inputs before step t0, those of earlier episodes left out. `starts`: bit i for step
// t0 - (K - 1) + i.
template <typename T, int V, int K>
__device__ __forceinline__ void open_window(const ConvParams &p, int64_t n, int t0, int64_t e,
                                            unsigned starts, float (&win)[K][V])
{
    Pack<T, V> r[K];
#pragma unroll
    for (int i = 0; i + 1 < K; ++i) r[i] = conv_input<T, V>(p, n, t0 - (K - 1) + i, e);
    clear_window<V, K>(win);
#pragma unroll
    for (int i = 0; i + 1 < K; ++i) {
        if ((starts >> i) & 1u) clear_window<V, K>(win);
        push_window<T, V, K>(win, r[i]);
    }
}

// p_t for the window that ends with x_t.
template <int V, int K>
__device__ __forceinline__ void apply_taps(const Taps<V, K> &f, const float (&win)[K][V],
                                           float (&acc)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = f.bias[i];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(f.w[k][i], win[k][i], acc[i]);
}

template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads, K > 4 ? 3 : 5) conv_forward_kernel(const ConvParams p)
{
    constexpr int U = kConvBatch;
    __shared__ TapRows<V> taps;
    grid_dependency_sync();
    const int64_t lane_blocks = (p.E / V + 31) / 32;
    const int64_t span_blocks =
        p.T ? (p.T + kConvSpan * kConvWarps - 1) / (kConvSpan * kConvWarps) : 1;
    const int64_t nb = blockIdx.x / lane_blocks;  // (n, span block)
    const int64_t n = nb / span_blocks;
    const int64_t e0 = (blockIdx.x % lane_blocks) * 32 * V;
    const int64_t e = e0 + (threadIdx.x & 31) * V;
    stage_taps<V>(p, e0, taps);
    const int span = (int)(nb % span_blocks) * kConvWarps + (threadIdx.x >> 5);
    const int t0 = span * kConvSpan;
    const int t1 = t0 >= p.T ? t0 : (p.T - t0 < kConvSpan ? p.T : t0 + kConvSpan);
    const int len = row_length(p.rows, n, p.T);
    const int end = len < t1 ? len : t1;
    const unsigned starts = start_bits(p.rows, n, t0, end);
    const unsigned before = start_bits(p.rows, n, t0 - (K - 1), t0 < len ? t0 : len);
    __syncthreads();
    if (e >= p.E) return;
    const T *x = static_cast<const T *>(p.x.ptr) + n * p.x.row + t0 * p.x.step + e;
    T *out = static_cast<T *>(const_cast<void *>(p.out.ptr)) + n * p.out.row + t0 * p.out.step + e;

    const bool owns_final =
        p.final_state && (len > 0 ? t0 < len && len <= t1 : span == 0);
    float win[K][V];
    if (t0 < end || owns_final) {
        Taps<V, K> f;
        load_taps<V, K>(p, e, taps, f);
        Pack<T, V> next[U];
        auto fetch = [&](int j) {  // x is at step t0 + j
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t0 + j + u < end) next[u] = load_pack<T, V>(x + u * p.x.step);
        };
        fetch(0);
        open_window<T, V, K>(p, n, t0, e, before, win);
#pragma unroll 1
        for (int j0 = 0; t0 + j0 < end; j0 += U) {
            Pack<T, V> r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = next[u];
            x += U * p.x.step;
            fetch(j0 + U);
            // WHOLE: a batch of U steps of one episode, with nothing to decide step by step.
            auto run = [&](auto whole) {
                constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (!WHOLE && t0 + j0 + u >= end) break;
                    if (!WHOLE && ((starts >> (j0 + u)) & 1u)) clear_window<V, K>(win);
                    push_window<T, V, K>(win, r[u]);
                    float acc[V];
                    apply_taps<V, K>(f, win, acc);
                    Pack<T, V> o;
#pragma unroll
                    for (int k = 0; k < V; ++k) o.e[k] = narrow<T>(p.silu ? silu<T>(acc[k]) : acc[k]);
                    store_pack<T, V>(out + u * p.out.step, o);
                }
            };
            if (t0 + j0 + U <= end && ((starts >> j0) & ((1u << U) - 1u)) == 0)
                run(std::true_type{});
            else
                run(std::false_type{});
            out += U * p.out.step;
        }
    }
    out = static_cast<T *>(const_cast<void *>(p.out.ptr)) + n * p.out.row + t0 * p.out.step + e;
    for (int t = t0 > end ? t0 : end; t < t1; ++t)
        store_pack<T, V>(out + (t - t0) * p.out.step, zero_pack<T, V>());
    if (owns_final) {
        if (len > 0 && step_ended(p.rows, n, len - 1)) clear_window<V, K>(win);
        T *dst = static_cast<T *>(p.final_state) + n * (K - 1) * p.E + e;
#pragma unroll
        for (int k = 1; k < K; ++k) {
            Pack<T, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) o.e[j] = narrow<T>(win[k][j]);
            store_pack<T, V>(dst + (int64_t)(k - 1) * p.E, o);
        }
    }
}

// dp_t = dout_t silu'(p_t); dx_t = sum_j w_{K-1-j} dp_{t+j} over the steps of the same
// episode; dw_k = sum_t dp_t x_{t-K+1+k}; db = sum_t dp_t. A warp owns the dx of its span and
// the shares of dw and db of its steps; it runs K - 1 steps past the span's end for dx.
// 4 channels to a lane: at 4 taps the window, the filter, dx on its way and dw take 16
// registers each.
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads, K > 4 ? 2 : (sizeof(T) == 4 ? 3 : 4))
    conv_backward_kernel(const ConvParams p)
{
    constexpr int U = kConvBackBatch;
    __shared__ float sh[kConvWarps][K + 1][32 * V];
    __shared__ TapRows<V> taps;
    grid_dependency_sync();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t lane_blocks = (p.E / V + 31) / 32;
    const int64_t span_blocks = (p.T + kConvSpan * kConvWarps - 1) / (kConvSpan * kConvWarps);
    const int64_t nb = blockIdx.x / lane_blocks;  // (n, span block)
    const int64_t n = nb / span_blocks;
    const int64_t e0 = (blockIdx.x % lane_blocks) * 32 * V;
    const int64_t e = e0 + lane * V;
    const int t0 = ((int)(nb % span_blocks) * kConvWarps + warp) * kConvSpan;
    const int t1 = t0 >= p.T ? t0 : (p.T - t0 < kConvSpan ? p.T : t0 + kConvSpan);
    const int len = row_length(p.rows, n, p.T);
    const int stop = t1 + K - 1 < len ? t1 + K - 1 : len;  // steps that are run
    stage_taps<V>(p, e0, taps);
    __syncthreads();
    const unsigned starts = start_bits(p.rows, n, t0, stop);
    const unsigned before = start_bits(p.rows, n, t0 - (K - 1), t0 < len ? t0 : len);
    const unsigned later = start_bits(p.rows, n, t0 + kConvSpan, stop);  // past the span

    float dw[K][V], db[V];
    clear_window<V, K>(dw);
#pragma unroll
    for (int i = 0; i < V; ++i) db[i] = 0.f;
    if (e < p.E && t0 < t1) {
        const T *x = static_cast<const T *>(p.x.ptr) + n * p.x.row + t0 * p.x.step + e;
        const T *dout = static_cast<const T *>(p.dout.ptr) + n * p.dout.row + t0 * p.dout.step + e;
        T *dx = static_cast<T *>(const_cast<void *>(p.dx.ptr)) + n * p.dx.row + t0 * p.dx.step + e;
        if (t0 < len) {
            Taps<V, K> f;
            load_taps<V, K>(p, e, taps, f);
            float win[K][V], acc[K][V];  // acc[j]: dx of step t - j so far
            Pack<T, V> nx[U], ng[U];
            auto fetch = [&](int j) {  // x and dout are at step t0 + j
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (t0 + j + u < stop) {
                        nx[u] = load_pack<T, V>(x + u * p.x.step);
                        ng[u] = load_pack<T, V>(dout + u * p.dout.step);
                    }
            };
            fetch(0);
            open_window<T, V, K>(p, n, t0, e, before, win);
            clear_window<V, K>(acc);
            int reach = K - 1;  // earlier steps of the episode that x_t's filter sees
            auto put = [&](int j, const float (&v)[V]) {
                Pack<T, V> o;
#pragma unroll
                for (int i = 0; i < V; ++i) o.e[i] = narrow<T>(v[i]);
                store_pack<T, V>(dx + j * p.dx.step, o);
            };
            auto emit = [&](int j, const float (&v)[V]) {
                if (j >= 0 && t0 + j < t1) put(j, v);
            };
#pragma unroll 1
            for (int j0 = 0; t0 + j0 < stop; j0 += U) {
                Pack<T, V> rx[U], rg[U];
#pragma unroll
                for (int u = 0; u < U; ++u) rx[u] = nx[u], rg[u] = ng[u];
                x += U * p.x.step, dout += U * p.dout.step;
                fetch(j0 + U);
                // WHOLE: a batch inside the span and one episode, K - 1 steps and more after
                // its start and the span's: nothing to decide step by step.
                auto run = [&](auto whole) {
                    constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int j = j0 + u;
                        if (!WHOLE) {
                            if (t0 + j >= stop) break;
                            reach = reach + 1 < K ? reach + 1 : K - 1;
                            if (((j < kConvSpan ? starts : later) >> (j % kConvSpan)) & 1u) {
                                clear_window<V, K>(win);
                                reach = 0;
                            }
                        }
                        push_window<T, V, K>(win, rx[u]);
                        float dp[V];
                        apply_taps<V, K>(f, win, dp);
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float sg = sigmoid<T>(dp[i]);
                            dp[i] = widen(rg[u].e[i]) *
                                    (p.silu ? sg * fmaf(dp[i], 1.f - sg, 1.f) : 1.f);
                        }
                        // One step on: acc[m] moves to acc[m + 1].
#pragma unroll
                        for (int m = K - 1; m >= 0; --m) {
#pragma unroll
                            for (int i = 0; i < V; ++i) {
                                const float before = m > 0 ? acc[m - 1][i] : 0.f;
                                acc[m][i] = WHOLE || m <= reach
                                                ? fmaf(f.w[K - 1 - m][i], dp[i], before)
                                                : before;
                            }
                        }
                        if (WHOLE || t0 + j < t1) {
#pragma unroll
                            for (int k = 0; k < K; ++k)
#pragma unroll
                                for (int i = 0; i < V; ++i)
                                    dw[k][i] = fmaf(dp[i], win[k][i], dw[k][i]);
#pragma unroll
                            for (int i = 0; i < V; ++i) db[i] += dp[i];
                        }
                        if (WHOLE)
                            put(j - (K - 1), acc[K - 1]);
                        else
                            emit(j - (K - 1), acc[K - 1]);
                    }
                };
                const bool plain = j0 + U <= kConvSpan && ((starts >> j0) & ((1u << U) - 1u)) == 0;
                const int whole = t1 < stop ? t1 : stop;
                if (plain && reach == K - 1 && j0 >= K - 1 && t0 + j0 + U <= whole)
                    run(std::true_type{});
                else
                    run(std::false_type{});
            }
#pragma unroll
            for (int m = 0; m + 1 < K; ++m) emit(stop - t0 - 1 - m, acc[m]);
        }
        for (int t = t0 > len ? t0 : len; t < t1; ++t)
            store_pack<T, V>(dx + (t - t0) * p.dx.step, zero_pack<T, V>());
    }
    // The spans of the CTA add up in order.
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < K; ++k) sh[warp][k][lane * V + i] = dw[k][i];
        sh[warp][K][lane * V + i] = db[i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < (K + 1) * 32 * V; c += kConvThreads) {
        const int k = c / (32 * V), l = c % (32 * V);
        if (e0 + l >= p.E) continue;
        float sum = 0.f;
#pragma unroll
        for (int y = 0; y < kConvWarps; ++y) sum += sh[y][k][l];
        p.part_w[(nb * (K + 1) + k) * p.E + e0 + l] = sum;
    }
}

// One step of N rows: a lane owns V channels, a warp one row. The state is read before the
// barrier behind the filters, so both are on their way together. It is read and written by
// the same thread only: the new state may be the state.
template <typename T, int V>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(const ConvParams p)
{
    __shared__ TapRows<V> taps;
    grid_dependency_sync();
    const int64_t lane_blocks = (p.E / V + 31) / 32;
    const int64_t n = blockIdx.x / lane_blocks * kConvWarps + (threadIdx.x >> 5);
    const int64_t e0 = blockIdx.x % lane_blocks * 32 * V;
    const int c = (threadIdx.x & 31) * V;
    const int64_t e = e0 + c;
    const bool in = n < p.N && e < p.E;
    const bool keep = in && p.init && !(p.reset && __ldg(p.reset + n));
    const T *state = static_cast<const T *>(p.init) + n * (p.K - 1) * p.E + e;
    Pack<T, V> x = zero_pack<T, V>(), w[RLCA_CONV_MAX_K];
    if (in)
        x = load_pack<T, V>(static_cast<const T *>(p.x.ptr) + n * p.x.row + e);
#pragma unroll
    for (int k = 0; k + 1 < RLCA_CONV_MAX_K; ++k)
        if (k + 1 < p.K)
            w[k] = keep ? *reinterpret_cast<const Pack<T, V> *>(state + (int64_t)k * p.E)
                        : zero_pack<T, V>();
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = in && p.bias ? __ldg(p.bias + e + v) : 0.f;
    stage_taps<V>(p, e0, taps);
    __syncthreads();
    if (!in) return;
    T *next = static_cast<T *>(p.final_state) + n * (p.K - 1) * p.E + e;
#pragma unroll
    for (int k = 0; k + 1 < RLCA_CONV_MAX_K; ++k)
        if (k + 1 < p.K) {
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = fmaf(taps.w[k][c + v], widen(w[k].e[v]), acc[v]);
            if (k > 0) *reinterpret_cast<Pack<T, V> *>(next + (int64_t)(k - 1) * p.E) = w[k];
        }
    if (p.K > 1) *reinterpret_cast<Pack<T, V> *>(next + (int64_t)(p.K - 2) * p.E) = x;
    Pack<T, V> o;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float a = fmaf(taps.w[p.K - 1][c + v], widen(x.e[v]), acc[v]);
        o.e[v] = narrow<T>(p.silu ? silu<T>(a) : a);
    }
    store_pack<T, V>(static_cast<T *>(const_cast<void *>(p.out.ptr)) + n * p.out.row + e, o);
}

}  // namespace seq
}  // namespace rlca

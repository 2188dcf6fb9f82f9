// Shared parts of the sequence-model kernels (selective scan, causal convolution, token
// embedding): data types, vector access, episode flags, small math.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "../../include/rlca_sequence.h"
#include "launch.cuh"

namespace rlca {
namespace seq {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The data type of one format.
template <Fmt F>
struct DataType;
template <>
struct DataType<Fmt::kF32> {
    using type = float;
};
template <>
struct DataType<Fmt::kBF16> {
    using type = __nv_bfloat16;
};
template <>
struct DataType<Fmt::kF16> {
    using type = __half;
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v)
{
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half narrow<__half>(float v)
{
    return __float2half_rn(v);
}

// V consecutive elements, read and written in one access (V = 1, or 16 bytes of them).
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
    T e[V];
};

template <typename T>
__host__ __device__ constexpr int vec_of()
{
    return 16 / (int)sizeof(T);
}

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> zero_pack()
{
    Pack<T, V> p;
#pragma unroll
    for (int i = 0; i < V; ++i) p.e[i] = narrow<T>(0.f);
    return p;
}

// Streaming data are read once: no need to keep them in L1.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T *p)
{
    Pack<T, V> r;
    if constexpr (sizeof(Pack<T, V>) == 16) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(p));
        r = *reinterpret_cast<const Pack<T, V> *>(&w);
    } else if constexpr (sizeof(Pack<T, V>) == 8) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p));
        r = *reinterpret_cast<const Pack<T, V> *>(&w);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) r.e[i] = p[i];
    }
    return r;
}

template <typename T, int V>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, V> &v)
{
    if constexpr (sizeof(Pack<T, V>) == 16) {
        *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(&v);
    } else if constexpr (sizeof(Pack<T, V>) == 8) {
        *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(&v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = v.e[i];
    }
}

// Two fp32 lanes in one register pair. The fma unit takes 128 lanes a clock and SM either way
// (measured: 116 scalar, 2 x 52 paired), but a pair needs one issue slot, and the recurrences
// here are bound by slots.
using Pair = float2;

__device__ __forceinline__ Pair pair(float lo, float hi) { return make_float2(lo, hi); }
__device__ __forceinline__ float2 split(Pair p) { return p; }
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ Pair add2(Pair a, Pair b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ Pair mul2(Pair a, Pair b) { return __fmul2_rn(a, b); }

// 2^x, one instruction (at most 2 ulp off; results below 2^-126 are 0).
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ Pair exp2_fast(Pair x)
{
    const float2 f = split(x);
    return pair(exp2_fast(f.x), exp2_fast(f.y));
}

// 1 / x, one instruction (1 ulp; 0 for |x| > 2^126, inf for subnormals).
__device__ __forceinline__ float rcp_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// sigmoid(x) = 1 / (1 + e^-x), 0 where e^-x overflows (x < -88). fp32 takes CUDA's expf: the fast
// exponential's error is that of its argument's rounding, up to |x| 7e-8. For 16-bit types that
// is far inside the rounding of what it scales. Measured, largest error of the fp32 form and of
// the 16-bit one: x in -5..-2 2e-7 / 3e-7, -20..-10 2e-7 / 1e-6, at -87 2e-7 / 4e-6. The reciprocal
// is within 1 ulp; the rounded one gains nothing that shows and costs: fp32 training pass of
// [4, 4096, 2048] x 4 taps 159 us in place of 135 (133 with the fast exponential), of the scan
// [16, 1024, 2048] 2756 in place of 2379 (2387).
template <typename T>
__device__ __forceinline__ float sigmoid(float x)
{
    return rcp_fast(1.f + (sizeof(T) == 4 ? expf(-x) : exp2_fast(-kLog2e * x)));
}

template <typename T>
__device__ __forceinline__ float silu(float x)
{
    return x * sigmoid<T>(x);
}

// min(|x|, top), a NaN if x is one.
__device__ __forceinline__ float abs_up_to(float x, float top)
{
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(fabsf(x)), "f"(top));
    return y;
}

// softplus(x) = max(x, 0) + log(1 + e), e = exp(-|x|) in (0, 1]. An error of the step size is one
// of the whole state: fp32 takes CUDA's expf and log1pf. For 16-bit types, whose states are fp32
// too, log(1 + e) = 2 atanh(u), u = e / (2 + e) <= 1/3, so small step sizes keep their relative
// accuracy, which log(1 + e) from a rounded 1 + e would lose; atanh(u) / u as a polynomial in
// u^2 <= 1/9, fitted to the least largest error (8e-9). e is 2^t, t = -|x| log2(e) rounded, times
// e^(-|x| - t ln 2), which puts back what the rounding left out (largest error, measured
// in -87..-10: 5e-7; without it 1e-6 to 4e-6, CUDA's functions 2e-7). |x| is cut off at 90, where e
// is 0, so that an Inf leaves no Inf - Inf; a NaN comes through the second term. The fast
// exponential is low by 5e-8 on average: 1.9999999 for 2 puts that back into u (mean error in -20..2
// 1e-8 to 7e-8, with 2 up to -5e-8). 1.5 % of a forward scan's time.
template <typename T>
__device__ __forceinline__ float softplus(float x)
{
    if constexpr (sizeof(T) == 4) return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
    const float m = abs_up_to(x, 90.f);
    const float t = -kLog2e * m;
    float e = exp2_fast(t);
    e = fmaf(e, fmaf(t, -kLn2, -m), e);
    const float u = e * rcp_fast(1.9999999f + e);
    const float q = u * u;
    float s = 0.14095773f;
    s = fmaf(s, q, 0.13978833f);
    s = fmaf(s, q, 0.20012557f);
    s = fmaf(s, q, 0.33333155f);
    s = fmaf(s, q, 1.f);
    return fmaf(2.f * u, s, fmaxf(x, 0.f));
}

// The decay exp(d A) of a state, or of two, from the prepared A (decay_base): fp32 takes CUDA's
// expf, 16-bit types 2^(d A2) with A2 = A log2(e), one instruction to a state. That instruction is
// low on average, and a decay's error comes back in every later state: measured, for exponents in
// -0.005..0 by 0.5e-8 to 1e-8, in -0.05..-0.005 by 2.2e-8 to 2.6e-8, in -0.5..-0.05 by 1e-8 to
// 1.5e-8. 2.9e-8 on the exponent, in the multiply-add that forms it, leaves at most 1.5e-8 on either
// side there, which is what CUDA's expf is off by on average. Below -0.5 it is lost in the
// exponent's rounding (5e-8 too low below -1, where a state remembers a step or two). 2^2.9e-8 is
// 1: a step size of 0 keeps the state.
template <typename T>
__device__ __forceinline__ float decay_base(float A)
{
    return sizeof(T) == 4 ? A : kLog2e * A;
}

// The same for kernels that run steps past a row's end with a step size of 0: A = -inf, a decay of 0,
// becomes the lowest finite rate, which decays to 0 as well and by nothing in 0 steps (-inf: NaN). A
// NaN stays one.
template <typename T>
__device__ __forceinline__ float finite_decay_base(float A)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(decay_base<T>(A)), "f"(-FLT_MAX));
    return y;
}

template <typename T>
__device__ __forceinline__ float decay(float d, float A)
{
    return sizeof(T) == 4 ? expf(d * A) : exp2_fast(fmaf(d, A, 2.9e-8f));
}

template <typename T>
__device__ __forceinline__ Pair decay(Pair d, Pair A)
{
    if constexpr (sizeof(T) == 4) {
        const Pair t = mul2(d, A);
        return pair(expf(t.x), expf(t.y));
    }
    return exp2_fast(fma2(d, A, pair(2.9e-8f, 2.9e-8f)));
}

// What turns a sum over prepared A back into one over A.
template <typename T>
__device__ __forceinline__ float decay_unit()
{
    return sizeof(T) == 4 ? 1.f : kLn2;
}

// Sums each of V values over the G lanes whose lane numbers differ by multiples of STRIDE.
// The lane of index i in its group ends with the sums of the values i V / G .. (or, when
// V < G, of value i / (G / V)) in v[0..]. G - 1 exchanges of halves and no more: every
// lane keeps only what it will hold.
template <int V, int G, int STRIDE>
__device__ __forceinline__ void reduce_scatter(float (&v)[V])
{
    const int lane = threadIdx.x & 31;
    int m = V;
#pragma unroll
    for (int w = G / 2; w >= 1; w /= 2) {
        if (m > 1) {
            const bool upper = (lane & (w * STRIDE)) != 0;
            m /= 2;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                if (i >= m) break;
                const float send = upper ? v[i] : v[i + m];
                const float keep = upper ? v[i + m] : v[i];
                v[i] = keep + __shfl_xor_sync(kFullMask, send, w * STRIDE);
            }
        } else {
            v[0] += __shfl_xor_sync(kFullMask, v[0], w * STRIDE);
        }
    }
}

// Row lengths and episode flags, as the kernels see them.
struct RowFlags {
    const uint8_t *term, *trunc;
    int64_t ld;
    const int32_t *lengths;
};

__device__ __forceinline__ int row_length(const RowFlags &r, int64_t n, int T)
{
    if (!r.lengths) return T;
    const int v = __ldg(r.lengths + n);
    return v < 0 ? 0 : (v > T ? T : v);
}

// Whether step t (0 <= t < T) of row n ended an episode.
__device__ __forceinline__ bool step_ended(const RowFlags &r, int64_t n, int t)
{
    bool e = false;
    if (r.term) e = __ldg(r.term + n * r.ld + t) != 0;
    if (r.trunc) e |= __ldg(r.trunc + n * r.ld + t) != 0;
    return e;
}

// Bit i: step t0 + i (i < 32) is the first of its episode (t > 0 and step t - 1 ended one).
// Every lane of the warp calls this.
__device__ __forceinline__ unsigned start_bits(const RowFlags &r, int64_t n, int t0, int len)
{
    if (!r.term && !r.trunc) return 0u;
    const int t = t0 + (threadIdx.x & 31);
    const bool s = t > 0 && t < len && step_ended(r, n, t - 1);
    return __ballot_sync(kFullMask, s);
}

// The last step of sums that are taken in shares: sum over r < rows of src[r * stride + i] for
// i < count[0] + count[1] + count[2], written to dst[0], dst[1] and dst[2] in turn (nullptr: not
// wanted). Always in the same order: eight interleaved sums over r, then those. `tap` > 0: the
// first part is [tap, count[0] / tap] and is written transposed.
struct SumRows {
    const float *src;
    int64_t rows, stride;
    int64_t count[3];
    float *dst[3];
    int tap;
};
cudaError_t launch_sum_rows(const SumRows &p, cudaStream_t stream);

// Workspace pieces start on 256-byte boundaries.
inline size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Launches of a 1-D grid counted in 64 bits: one that is too large for the device fails.
template <typename Kernel, typename... Args>
cudaError_t launch_grid(Kernel kernel, int64_t grid, unsigned block, cudaStream_t stream,
                        const Args &...args)
{
    if (grid <= 0 || grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_pdl(kernel, (unsigned)grid, block, 0, stream, args...);
}

// ------------------------------------------------------------------ launches, per format

struct ScanParams;
struct ConvParams;
struct EmbedParams;
// vec: every array allows accesses of 16 bytes.
template <Fmt F>
cudaError_t launch_scan_forward(const ScanParams &p, bool vec, cudaStream_t stream);
template <Fmt F>
cudaError_t launch_scan_backward(const ScanParams &p, bool vec, cudaStream_t stream);
template <Fmt F>
cudaError_t launch_scan_step(const ScanParams &p, bool vec, cudaStream_t stream);
template <Fmt F>
cudaError_t launch_conv_forward(const ConvParams &p, bool vec, cudaStream_t stream);
template <Fmt F>
cudaError_t launch_conv_backward(const ConvParams &p, bool vec, cudaStream_t stream);
template <Fmt F>
cudaError_t launch_conv_step(const ConvParams &p, bool vec, cudaStream_t stream);
template <Fmt F>
cudaError_t launch_embed(const EmbedParams &p, bool vec, cudaStream_t stream);
template <Fmt F>
cudaError_t launch_embed_sum(const EmbedParams &p, bool vec, cudaStream_t stream);

}  // namespace seq
}  // namespace rlca

// Selective state space scan: parameters and tile geometry shared by its kernels.
//
//   h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,   y_t = C_t . h_t + D x_t,   out = y silu(z)
//
// States stay in registers: a lane holds a few states of one or two channels, neighbouring lanes
// the other states of the same channels. A CTA walks the steps of one row in tiles; the raw
// activations of the next tile arrive in shared memory by asynchronous copies meanwhile.
#pragma once

#include "sequence.cuh"

namespace rlca {
namespace seq {

constexpr int kForwardWarps = 2;
constexpr int kForwardThreads = 32 * kForwardWarps;
constexpr int kBackwardWarps = 2;
constexpr int kBackwardThreads = 32 * kBackwardWarps;

struct ScanParams {
    int64_t N, E;
    int T, S, G, Eg;  // Eg = E / G channels in a group
    int blocks_g;     // channel blocks in a group
    rlca_steps x, dt, z, B, C;
    const float *A, *D, *dt_bias, *init;
    RowFlags rows;
    int softplus;
    rlca_steps out;
    float *final_state, *saved;
    // backward
    rlca_steps dout, dx, ddt, dz, dB, dC;
    const float *d_final;
    float *d_init;
    float *part_bc;      // [N, T, G, blocks_g, 2, 4 SL] shares of dB and dC
    float *part_p;       // [N, spans, E S + 2 E] shares of dA, dD and ddt_bias
    const uint8_t *reset;
    // A row cut into `spans` of `span_steps` (a multiple of the tile) walked side by side.
    int spans, span_steps;
    float *span_state;  // [N, spans, E, S]: what a span leaves from 0, then what it starts from
    float *span_sum;    // [N, spans, E]: sum of d over the span; NaN where an episode starts
};

// Lanes that share a channel's states, `per` states each: a power of two, at least `least`.
inline int scan_state_lanes(int64_t S, int per, int least = 1)
{
    int sl = least;
    while (per * sl < S) sl *= 2;
    return sl;
}

// Channels of a CTA: forward, a lane holds 8 states of one channel; backward, 4 states of 2
// channels, at least 2 lanes to a channel.
inline int scan_forward_channels(int64_t S) { return kForwardThreads / scan_state_lanes(S, 8); }
inline int scan_backward_lanes(int64_t S) { return scan_state_lanes(S, 4, 2); }
inline int scan_backward_channels(int64_t S)
{
    return 2 * kBackwardThreads / scan_backward_lanes(S);
}

// Spans of a row, and their steps. Spans fill the GPU where the rows' CTAs leave SMs idle;
// they cost a second pass over the arithmetic.
struct ScanSpans {
    int spans, steps;
};

// `per_sm` CTAs to an SM in all, `units` CTAs to a span; spans of 32 steps and more. The callers'
// waves are those of 16 states in bf16, where 8 CTAs to an SM run forward and 6 backward; other types
// and state sizes hold 4 to 8 (their spans are measured as they are, not whole waves).
inline ScanSpans scan_cut(int64_t units, int64_t per_sm, int64_t T, int64_t least)
{
    constexpr int64_t kTile = 32;
    int64_t spans = units > 0 ? per_sm * sm_count() / units : 1;
    if (spans > T / kTile) spans = T / kTile;
    if (spans < least) return {1, (int)((T + kTile - 1) / kTile * kTile)};
    int64_t steps = (T + spans - 1) / spans;
    steps = (steps + kTile - 1) / kTile * kTile;
    return {(int)((T + steps - 1) / steps), (int)steps};
}

// Forward, spans double the arithmetic: only where the rows' CTAs fill a quarter of a wave of 8
// to an SM. Measured, [N, 1024, 2048] x 16 states, bf16, us, one span / cut: N = 1 130 / 42,
// 2 130 / 70, 3 131 / 94, 4 134 / 124; from N = 6 on (163) spans no longer pay.
inline ScanSpans scan_forward_spans(int64_t N, int64_t T, int64_t E, int64_t S, int64_t G)
{
    const int64_t ch = scan_forward_channels(S), units = N * G * ((E / G + ch - 1) / ch);
    return scan_cut(units, 4 * units <= 8 * sm_count() ? 8 : 0, T, 4);
}

// Backward they add a fifth: up to half a wave of 6 to an SM, then three waves, so that SMs that
// are done early take more. Measured there, us, one span / one wave / two / three: N = 3
// - / 278 / 232 / 224, 6 503 / - / 443 / 412, 8 471 / - / 584 / 538; N = 12 646 / - / 850 / 827.
inline ScanSpans scan_backward_spans(int64_t N, int64_t T, int64_t E, int64_t S, int64_t G)
{
    const int64_t ch = scan_backward_channels(S), units = N * G * ((E / G + ch - 1) / ch);
    return scan_cut(units, 2 * units <= 6 * sm_count() ? 18 : 0, T, 2);
}

template <typename T>
__device__ __forceinline__ T *row_ptr(const rlca_steps &a, int64_t n, int64_t t, int64_t c)
{
    return const_cast<T *>(static_cast<const T *>(a.ptr)) + n * a.row + t * a.step + c;
}

// What every span starts from, out of what the spans before it leave (first pass).
// `reverse`: the adjoint, from the last span to the first (it starts at d_final).
cudaError_t launch_scan_join(const ScanParams &p, bool reverse, cudaStream_t stream);

// A CTA's place in the work.
template <int CH>
struct ScanPlace {
    int64_t n, c0;        // row; first channel
    int span, g, blk;     // span of steps; group; channel block within the group
    int nch;              // channels in use

    __device__ explicit ScanPlace(const ScanParams &p)
    {
        const unsigned blocks = (unsigned)p.G * p.blocks_g;
        const unsigned ns = blockIdx.x / blocks, gb = blockIdx.x % blocks;
        n = ns / p.spans;
        span = (int)(ns % p.spans);
        g = (int)(gb / p.blocks_g);
        blk = (int)(gb % p.blocks_g);
        const int cb = blk * CH;
        nch = p.Eg - cb < CH ? p.Eg - cb : CH;
        c0 = (int64_t)g * p.Eg + cb;
    }
};

// The 4 states of channel c at base + c * S + 4 sl, zeros where there are none.
__device__ __forceinline__ void load_states(const float *base, int64_t c, int sl, int S, bool in,
                                            float (&v)[4])
{
    const float *p = base + c * S + sl * 4;
    if (in && S % 4 == 0 && sl * 4 < S) {
        if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
            const float4 q = *reinterpret_cast<const float4 *>(p);
            v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
            return;
        }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = in && sl * 4 + s < S ? p[s] : 0.f;
}

__device__ __forceinline__ void store_states(float *base, int64_t c, int sl, int S, bool in,
                                             const float (&v)[4])
{
    float *p = base + c * S + sl * 4;
    if (in && S % 4 == 0 && sl * 4 < S) {
        if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
            *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
            return;
        }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
        if (in && sl * 4 + s < S) p[s] = v[s];
}

// B or C of a tile of TS steps on its way to shared memory. Thread i holds the elements i,
// i + NT, ... of the tile.
template <typename T, int SP, int TS, int NT>
struct TileBC {
    static constexpr int kAll = TS * SP;
    static constexpr int kPer = (kAll + NT - 1) / NT;
    // A thread's elements: one state of every kSkip-th step, or kAcross states of every step.
    static constexpr int kAcross = SP > NT ? SP / NT : 1;
    static constexpr int kSkip = SP > NT ? 1 : NT / SP;
    static_assert(SP > NT ? SP % NT == 0 : NT % SP == 0, "a thread keeps its states");
    const T *src;  // the thread's first element of step 0
    int64_t step;
    int have;  // states from the thread's first on
    int tid;
    T e[kPer];

    __device__ TileBC(const rlca_steps &a, const ScanParams &p, int64_t n, int g, int tid)
        : step(a.step), have(tid < kAll ? p.S - tid % SP : 0), tid(tid)
    {
        src = row_ptr<T>(a, n, tid / SP, (int64_t)g * p.S + tid % SP);
    }
    __device__ void load(int t0, int limit)
    {
        const int t = t0 + tid / SP;
        const T *s = src + t0 * step;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int off = k % kAcross * NT, down = k / kAcross * kSkip;
            e[k] = narrow<T>(0.f);
            if (off < have && t + down < limit) e[k] = s[down * step + off];
        }
    }
    __device__ void store(float (&dst)[TS][SP]) const
    {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = tid + k * NT;
            if (kAll % NT == 0 || i < kAll) dst[i / SP][i % SP] = widen(e[k]);
        }
    }
};

__device__ __forceinline__ void copies_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Copies a [TS, CH] tile of one activation into shared memory at pitch P, asynchronously where
// the elements allow it: 16 bytes at a time when the rows are aligned (VEC), 4 bytes for fp32,
// else element by element through registers: start() reads, land() writes what was read. Steps
// from `limit` on and channels from `nch` on become zeros.
template <typename T, bool VEC, int CH, int TS, int P, int NT>
struct TileCopy {
    static constexpr bool kAsync = VEC || sizeof(T) == 4;
    static constexpr int kPiece = VEC ? 16 / (int)sizeof(T) : 1;  // elements
    static constexpr int kCols = CH / kPiece;
    static constexpr int kAll = TS * kCols;
    static constexpr int kPer = (kAll + NT - 1) / NT;
    // A thread's pieces: the same column every kSkip steps, or kAcross columns of every step.
    static constexpr int kAcross = kCols > NT ? kCols / NT : 1;
    static constexpr int kSkip = kCols > NT ? 1 : NT / kCols;
    static_assert(kCols > NT ? kCols % NT == 0 : NT % kCols == 0, "a thread keeps its channels");
    const T *src;  // the thread's first piece of step 0
    int64_t step;
    int have;  // channels from the thread's first on
    int tid;
    T v[kAsync ? 1 : kPer];

    __device__ TileCopy(const rlca_steps &a, int64_t n, int64_t c0, int nch, int tid)
        : step(a.step), tid(tid)
    {
        const int c = tid % kCols * kPiece;
        have = nch - c;
        src = row_ptr<T>(a, n, tid / kCols, c0 + c);
    }
    __device__ static int across(int k) { return k % kAcross * NT * kPiece; }
    __device__ static int down(int k) { return k / kAcross * kSkip; }

    __device__ void start(T (*dst)[P], int t0, int limit)
    {
        const int j0 = tid / kCols, c = tid % kCols * kPiece;
        const T *s = src + t0 * step;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int j = j0 + down(k);
            if (kAll % NT != 0 && j >= TS) break;
            const bool in = across(k) < have && t0 + j < limit;
            const T *from = s + down(k) * step + across(k);  // not read unless `in`
            if constexpr (kAsync) {
                constexpr int kBytes = kPiece * (int)sizeof(T);
                const unsigned to = (unsigned)__cvta_generic_to_shared(&dst[j][c + across(k)]);
                const int bytes = in ? kBytes : 0;
                if constexpr (kBytes == 16)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                                 "l"(from), "r"(bytes)
                                 : "memory");
                else
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to),
                                 "l"(from), "r"(bytes)
                                 : "memory");
            } else {
                v[k] = narrow<T>(0.f);
                if (in) v[k] = *from;
            }
        }
    }
    __device__ void land(T (*dst)[P]) const
    {
        if constexpr (!kAsync) {
            const int j0 = tid / kCols, c = tid % kCols * kPiece;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int j = j0 + down(k);
                if (kAll % NT == 0 || j < TS) dst[j][c + across(k)] = v[k];
            }
        }
    }
};

// Eight consecutive floats of shared memory as pairs.
__device__ __forceinline__ void load_pairs(const float *src, Pair (&v)[4])
{
    const float4 a = *reinterpret_cast<const float4 *>(src);
    const float4 b = *reinterpret_cast<const float4 *>(src + 4);
    v[0] = pair(a.x, a.y), v[1] = pair(a.z, a.w), v[2] = pair(b.x, b.y), v[3] = pair(b.z, b.w);
}

// Eight consecutive elements, 16-byte aligned.
template <typename T>
__device__ __forceinline__ Pack<T, 8> load_eight(const T *src)
{
    constexpr int V = vec_of<T>();
    Pack<T, 8> r;
#pragma unroll
    for (int i = 0; i < 8; i += V) {
        const Pack<T, V> v = load_pack<T, V>(src + i);
#pragma unroll
        for (int k = 0; k < V; ++k) r.e[i + k] = v.e[k];
    }
    return r;
}

template <typename T>
__device__ __forceinline__ Pack<T, 2> get2(const T *src)
{
    return *reinterpret_cast<const Pack<T, 2> *>(src);
}

}  // namespace seq
}  // namespace rlca

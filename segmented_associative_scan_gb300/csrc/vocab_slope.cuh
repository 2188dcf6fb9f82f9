// Gradients by the logits from what a forward call saved of each row, (m, S): every warp a share of
// one row, read into registers, and its gradient written: a copy with an exponential to an element.
// [16, 256, 32768] in bf16: 79 us, 6.8 TB/s, what a copy of its bytes takes; rows that lie at another
// offset to 16 bytes than their gradients take exchanges between lanes.
#pragma once

#include "vocab_rows.cuh"

namespace rlca {
namespace seq {

constexpr int kSlopeWarps = 8;
// Packs of a lane, and the CTAs to an SM that the registers are cut for: loads in flight are bought by
// warps as well as by packs, and spilled registers (220 and, with entropies, 272 bytes a thread in fp32,
// 12 and 54 in bf16) cost less than the warps that they make room for.
// Measured, packs x CTAs, us: fp32 [64, 128, 32768] with entropies 4 x 4 404, 4 x 5 387, 4 x 6 354,
// 4 x 7 386, 6 x 4 353 (but [512, 256, 1000] 185 / 226), 2 x 8 429; bf16 [16, 256, 32768] 8 x 3 84.6,
// 8 x 4 79.1, 8 x 5 84.9, 4 x 5 88.8, 10 x 4 80.0.
template <typename T>
constexpr int kSlopePacks = sizeof(T) == 4 ? 4 : 8;
template <typename T>
constexpr int kSlopeCtas = sizeof(T) == 4 ? 6 : 4;

// The slope of step i, which counts, and the logit that its saved sum is relative to.
template <typename T, bool ENT>
__device__ __forceinline__ RowSlope saved_slope(const VocabParams &p, int i, const StepAt &s, float &m)
{
    const float2 ms = __ldg(reinterpret_cast<const float2 *>(p.saved) + i);
    float dl = 0.f, dh = 0.f;
    if (p.slope) {
        const int half = (int)(p.N / 2);
        dl = __ldg(p.slope + s.n);
        if (p.dloss) dl *= __ldg(p.dloss + (s.n < half ? s.n : s.n - half));
    } else if (p.dlogp.ptr) {
        dl = at(p.dlogp, s.n, s.t);
    }
    if (ENT) dh = at(p.dentropy, s.n, s.t);
    m = ms.x;
    RowSlope r = row_slope(dl, dh, logf(ms.y), 1.f / ms.y, ENT ? __ldg(p.entropy_in + i) : 0.f,
                              p.inv_tau);
    r.zero = m == -INFINITY || (dl == 0.f && dh == 0.f);
    return r;
}

template <typename T, bool ENT>
__global__ void __launch_bounds__(32 * kSlopeWarps, kSlopeCtas<T>)
    vocab_slope_kernel(const VocabParams p, int warps)
{
    constexpr int W = 16 / (int)sizeof(T), U = kSlopePacks<T>;
    grid_dependency_sync();
    // The last rows first: a forward pass over the same logits left those in the L2.
    const int64_t at_warp = (int64_t)blockIdx.x * kSlopeWarps + (threadIdx.x >> 5);
    const int64_t from_end = at_warp / warps;
    if (from_end >= p.M) return;
    const int i = (int)(p.M - 1 - from_end), lane = threadIdx.x & 31;
    const StepAt s = step_at(p, i);
    const Share<T, U> a(row_of<T>(p.logits, s.n, s.t), (int)p.V, (int)(at_warp % warps));
    T *g = out_row<T>(p.grad, s.n, s.t);

    RowSlope r = {0.f, 0.f, 0.f, true};
    float m = 0.f;
    int token = -1;
    if (inside_row(p, s.n, s.t)) {
        const int64_t j = vocab_token(p, s.n, s.t);
        if (j >= 0 && j < p.V) {
            token = (int)j;
            r = saved_slope<T, ENT>(p, i, s, m);
        }
    }
    if (r.zero) {
        const int64_t lo = (int64_t)a.k0 * W, hi = lo + 32 * U * W;
        const int64_t last = a.k0 / (32 * U) == warps - 1 ? p.V : hi;
        clear_row(g, min(lo, p.V), min(last, p.V), lane, 32);
        return;
    }
    Held<T, U> held;
    held.load(a);
    float z_a = 0.f;
    const int pack = (token + a.head) / W;
    const bool mine = pack >= a.k0 && pack < a.k0 + 32 * U;
    if (mine) z_a = widen(a.z[token]);
    __syncwarp();  // the gradient may take the logits' place
    held.template store<ENT>(a, g, r, m, p.scale);
    if (mine && lane == 0) g[token] = narrow<T>(slope_at<T, ENT>(z_a, r, m, p.scale) + r.gamma);
}

}  // namespace seq
}  // namespace rlca

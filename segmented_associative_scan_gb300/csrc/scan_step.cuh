// Selective scan, one step of N rows: the state is read, moved on by one step and written.
// A lane holds 4 states of one channel (one 16-byte access when S % 4 == 0), SL lanes side
// by side the states of a channel; their sum over states is a few shuffles.
#pragma once

#include "scan.cuh"

namespace rlca {
namespace seq {

template <typename T, int SL>
__global__ void __launch_bounds__(128) scan_step_kernel(const ScanParams p)
{
    grid_dependency_sync();
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
    const int sl = threadIdx.x % SL;
    const int64_t ne = i / SL;
    const bool live = ne < p.N * p.E;
    const int64_t n = live ? ne / p.E : 0, e = live ? ne % p.E : 0;
    const int g = (int)(e / p.Eg);
    const int64_t bc = (int64_t)g * p.S;
    const bool keep = p.init && !(p.reset && __ldg(p.reset + n));

    const float x = widen(*row_ptr<T>(p.x, n, 0, e));
    const float raw = widen(*row_ptr<T>(p.dt, n, 0, e)) + (p.dt_bias ? __ldg(p.dt_bias + e) : 0.f);
    const float d = p.softplus ? softplus<T>(raw) : raw;
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int s = sl * 4 + k;
        if (!live || s >= p.S) continue;
        const int64_t at = (n * p.E + e) * p.S + s;
        const float h0 = keep ? p.init[at] : 0.f;
        const float a = exp2_fast(d * (kLog2e * __ldg(p.A + e * p.S + s)));
        const float h = fmaf(a, h0, d * x * widen(*row_ptr<T>(p.B, n, 0, bc + s)));
        p.final_state[at] = h;
        y = fmaf(widen(*row_ptr<T>(p.C, n, 0, bc + s)), h, y);
    }
#pragma unroll
    for (int w = 1; w < SL; w *= 2) y += __shfl_xor_sync(kFullMask, y, w);
    if (live && sl == 0) {
        float v = p.D ? fmaf(__ldg(p.D + e), x, y) : y;
        if (p.z.ptr) v *= silu(widen(*row_ptr<T>(p.z, n, 0, e)));
        *row_ptr<T>(p.out, n, 0, e) = narrow<T>(v);
    }
}

}  // namespace seq
}  // namespace rlca

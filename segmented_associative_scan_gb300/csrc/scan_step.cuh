// Selective scan, one step of N rows: the state is read, moved on by one step and written.
// A lane holds 8 states of one channel (two 16-byte accesses when S % 4 == 0), SL lanes side by
// side the states of a channel; their sum over states is a few shuffles. The states are all of
// the traffic that counts: a thread takes the same states of ROWS rows, reads everything that
// it needs of them before it computes, and reads A once for them.
// 4096 rows x 1024 channels x 16 states: bf16 112 us for 571 MB, 5.1 TB/s of the 6.7 that a copy
// reaches (216 us with 4 states to a lane and one row at a time), fp16 100, fp32 136 for 604 MB
// (CUDA's expf and wider rows; 95 registers, 5 CTAs to an SM); 16 rows 2.5 us, the launch. States
// that are no multiple of 4 are read one by one: [4096, 1021] x 13 150 us.
#pragma once

#include "scan.cuh"

namespace rlca {
namespace seq {

// VEC: 8 values of B and C lie in one aligned access.
//
// Whether a channel's parameters are read before the rows or after them decides how many registers
// hold them and how many loads are in flight: before, where B and C are read wide and several lanes
// share a channel, else after. Measured, us, before / after: [4096, 1024] x 16 bf16 112 / 119, fp16
// 100 / 119; x 8 bf16 57.7 / 57.4, fp16 58 / 54; [4096, 1021] x 13 (B and C element by element) bf16
// 182 / 150, fp32 199 / 149.
template <typename T, int SL, int ROWS, bool VEC>
__global__ void __launch_bounds__(128) scan_step_kernel(const ScanParams p)
{
    grid_dependency_sync();
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
    const int sl = threadIdx.x % SL;
    const int64_t block = i / SL / p.E, e = i / SL % p.E, n0 = block * ROWS;
    const int64_t bc = e / p.Eg * p.S + sl * 8;  // the group's row of B and C, the lane's states
    float h[ROWS][8], A[8], x[ROWS], d[ROWS];
    T z[ROWS];
    Pack<T, 8> B[ROWS], C[ROWS];
    auto states = [&](const float *base, bool in, float (&v)[8]) {
        float a[4], b[4];
        load_states(base, e, 2 * sl, p.S, in, a);
        load_states(base, e, 2 * sl + 1, p.S, in, b);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = a[k], v[4 + k] = b[k];
    };
    constexpr bool kFirst = VEC && SL > 1;
    float bias, skip;
    auto parameters = [&]() {
        states(p.A, true, A);
        bias = p.dt_bias ? __ldg(p.dt_bias + e) : 0.f;
        skip = p.D ? __ldg(p.D + e) : 0.f;
    };
    if constexpr (kFirst) parameters();
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t n = n0 + r;
        const bool keep = n < p.N && p.init && !(p.reset && __ldg(p.reset + n));
        states(p.init + n * p.E * p.S, keep, h[r]);
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t n = n0 + r < p.N ? n0 + r : 0;
        x[r] = widen(*row_ptr<T>(p.x, n, 0, e));
        d[r] = widen(*row_ptr<T>(p.dt, n, 0, e));
        if (p.z.ptr) z[r] = *row_ptr<T>(p.z, n, 0, e);
        const T *b = row_ptr<T>(p.B, n, 0, bc), *c = row_ptr<T>(p.C, n, 0, bc);
        B[r] = C[r] = zero_pack<T, 8>();
        if constexpr (VEC) {
            if (sl * 8 < p.S) B[r] = load_eight(b), C[r] = load_eight(c);
        } else {
#pragma unroll
            for (int s = 0; s < 8; ++s)
                if (sl * 8 + s < p.S) B[r].e[s] = b[s], C[r].e[s] = c[s];
        }
    }
    if constexpr (!kFirst) parameters();
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t n = n0 + r;
        const bool live = n < p.N;
        const float raw = d[r] + bias, step = p.softplus ? softplus<T>(raw) : raw;
        const float w = step * x[r];
        float y = 0.f;
        // The window's operations one by one: a token moves the state on by the same bits either
        // way.
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            h[r][s] = fmaf(decay<T>(step, decay_base<T>(A[s])), h[r][s], w * widen(B[r].e[s]));
            y = fmaf(widen(C[r].e[s]), h[r][s], y);
        }
        float *next = p.final_state + n * p.E * p.S;
        const float a[4] = {h[r][0], h[r][1], h[r][2], h[r][3]};
        const float b[4] = {h[r][4], h[r][5], h[r][6], h[r][7]};
        store_states(next, e, 2 * sl, p.S, live, a);
        store_states(next, e, 2 * sl + 1, p.S, live, b);
#pragma unroll
        for (int m = 1; m < SL; m *= 2) y += __shfl_xor_sync(kFullMask, y, m);
        if (live && sl == 0) {
            float v = fmaf(skip, x[r], y);
            if (p.z.ptr) v *= silu<T>(widen(z[r]));
            *row_ptr<T>(p.out, n, 0, e) = narrow<T>(v);
        }
    }
}

}  // namespace seq
}  // namespace rlca

// Selective scan, forward.
#pragma once

#include "scan.cuh"

namespace rlca {
namespace seq {

template <typename T, int V, int SL, int CPT>
__global__ void __launch_bounds__(kScanThreads) scan_forward_kernel(const ScanParams p)
{
    using Geo = ScanGeom<SL, CPT>;
    using IO = TileIO<T, V, Geo::CH>;
    constexpr int CH = Geo::CH, SP = Geo::SP, TS = kTileSteps;
    __shared__ __align__(16) float sd[TS][CH];  // d
    __shared__ __align__(16) float sw[TS][CH];  // d x
    __shared__ __align__(16) float sy[TS][CH];  // C . h
    __shared__ __align__(16) float sB[TS][SP];
    __shared__ __align__(16) float sC[TS][SP];
    grid_dependency_sync();

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sl = lane % SL, cg = lane / SL;
    const int blocks = p.G * p.blocks_g;
    const int64_t n = blockIdx.x / blocks;
    const int g = (blockIdx.x % blocks) / p.blocks_g;
    const int cb = (blockIdx.x % p.blocks_g) * CH;  // first channel within the group
    const int nch = p.Eg - cb < CH ? p.Eg - cb : CH;
    const int64_t c0 = (int64_t)g * p.Eg + cb;
    const int len = row_length(p.rows, n, p.T);

    // The lane's channels and states.
    const int lch = warp * Geo::WCH + cg * CPT;
    float A2[CPT][4], h[CPT][4];
#pragma unroll
    for (int c = 0; c < CPT; ++c)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const bool in = lch + c < nch && sl * 4 + s < p.S;
            const int64_t i = (c0 + lch + c) * p.S + sl * 4 + s;
            A2[c][s] = in ? kLog2e * __ldg(p.A + i) : 0.f;
            h[c][s] = in && p.init ? __ldg(p.init + n * p.E * p.S + i) : 0.f;
        }

    // The thread's share of a tile's elements.
    const int col = IO::col();
    const bool active = col < nch;
    const int64_t ec = c0 + col;
    float bias[V], Dv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bias[i] = active && p.dt_bias ? __ldg(p.dt_bias + ec + i) : 0.f;
        Dv[i] = active && p.D ? __ldg(p.D + ec + i) : 0.f;
    }

    for (int t0 = 0; t0 < p.T; t0 += TS) {
        Pack<T, V> rx[IO::kPer], rd[IO::kPer], rz[IO::kPer];
        IO::load(p.x, n, ec, active, t0, len, rx);
        IO::load(p.dt, n, ec, active, t0, len, rd);
        if (p.z.ptr) IO::load(p.z, n, ec, active, t0, len, rz);
        // h before the chunk, for the backward pass.
        if (p.saved && t0 < len) {
            const int64_t chunks = (p.T + TS - 1) / TS;
            float *dst = p.saved + (n * chunks + t0 / TS) * p.E * p.S;
#pragma unroll
            for (int c = 0; c < CPT; ++c)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    if (lch + c < nch && sl * 4 + s < p.S)
                        dst[(c0 + lch + c) * p.S + sl * 4 + s] = h[c][s];
        }
#pragma unroll
        for (int k = 0; k < IO::kPer; ++k) {
            if (!IO::has(k)) continue;
            const int j = IO::step(k);
            const bool inside = t0 + j < len;  // later steps keep the state: d = 0
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float raw = widen(rd[k].e[i]) + bias[i];
                const float d = !inside ? 0.f : (p.softplus ? softplus(raw) : raw);
                sd[j][col + i] = d;
                sw[j][col + i] = d * widen(rx[k].e[i]);
            }
        }
        stage_bc<T, SP>(p, n, g, t0, len, sB, sC);
        const unsigned starts = start_bits(p.rows, n, t0, len);
        __syncthreads();

        const int steps = len - t0 < TS ? len - t0 : TS;
        for (int j = 0; j < steps; ++j) {
            if ((starts >> j) & 1u) {
#pragma unroll
                for (int c = 0; c < CPT; ++c)
#pragma unroll
                    for (int s = 0; s < 4; ++s) h[c][s] = 0.f;
            }
            float B[4], C[4], y[CPT];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                B[s] = sB[j][sl * 4 + s];
                C[s] = sC[j][sl * 4 + s];
            }
#pragma unroll
            for (int c = 0; c < CPT; ++c) {
                const float d = sd[j][lch + c], w = sw[j][lch + c];
                y[c] = 0.f;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    h[c][s] = fmaf(exp2_fast(d * A2[c][s]), h[c][s], w * B[s]);
                    y[c] = fmaf(C[s], h[c][s], y[c]);
                }
            }
            reduce_scatter<CPT, SL, 1>(y);
            constexpr int kOut = CPT >= SL ? CPT / SL : 1;
            constexpr int kRep = SL > CPT ? SL / CPT : 1;
#pragma unroll
            for (int i = 0; i < kOut; ++i)
                if (sl % kRep == 0) sy[j][lch + (sl / kRep) * kOut + i] = y[i];
        }
        __syncthreads();

#pragma unroll
        for (int k = 0; k < IO::kPer; ++k) {
            const int j = IO::step(k), t = t0 + j;
            if (!active || !IO::has(k) || t >= p.T) continue;
            Pack<T, V> o = zero_pack<T, V>();
            if (t < len) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float v = fmaf(Dv[i], widen(rx[k].e[i]), sy[j][col + i]);
                    if (p.z.ptr) v *= silu(widen(rz[k].e[i]));
                    o.e[i] = narrow<T>(v);
                }
            }
            store_pack<T, V>(row_ptr<T>(p.out, n, t, ec), o);
        }
    }
    if (p.final_state) {
        const bool ended = len > 0 && step_ended(p.rows, n, len - 1);
#pragma unroll
        for (int c = 0; c < CPT; ++c)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (lch + c < nch && sl * 4 + s < p.S)
                    p.final_state[(n * p.E + c0 + lch + c) * p.S + sl * 4 + s] =
                        ended ? 0.f : h[c][s];
    }
}

}  // namespace seq
}  // namespace rlca

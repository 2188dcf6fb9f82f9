// Selective scan, backward.
//
// With q_t = dout_t silu(z_t) and the state's adjoint run from the last step to the first,
//   g_t = (a_{t+1} g_{t+1} unless t + 1 starts an episode) + q_t C_t,   a_t = exp(d_t A):
//   dB_t = sum_e g_t d_t x_t          dC_t = sum_e q_t h_t
//   dA   = sum_t g_t d_t a_t h_{t-1}  dx_t = D q_t + d_t (g_t . B_t)
//   dd_t = g_t . (A a_t h_{t-1}) + x_t (g_t . B_t),   ddt_t = dd_t sigmoid(dt_t + bias).
//
// The chunks of 16 steps are walked from the last to the first. Within a chunk h is run
// forward again from the state the forward pass saved, 8 steps at a time, h_{t-1} of the 8
// steps held in registers for the reverse run over them.
#pragma once

#include "scan.cuh"

namespace rlca {
namespace seq {

constexpr int kBackSteps = 8;  // steps whose h is held in registers

template <typename T, int V, int SL, int CPT>
__global__ void __launch_bounds__(kScanThreads) scan_backward_kernel(const ScanParams p)
{
    using Geo = ScanGeom<SL, CPT>;
    using IO = TileIO<T, V, Geo::CH>;
    constexpr int CH = Geo::CH, SP = Geo::SP, TS = kTileSteps, CG = Geo::CG, HB = kBackSteps;
    __shared__ __align__(16) float sd[TS][CH];  // d, then the scan's share of dd
    __shared__ __align__(16) float sx[TS][CH];  // x, then the scan's share of dx
    __shared__ __align__(16) float sq[TS][CH];  // q
    __shared__ __align__(16) float sy[TS][CH];  // C . h
    __shared__ __align__(16) float sB[TS][SP];
    __shared__ __align__(16) float sC[TS][SP];
    __shared__ float red[kScanWarps][TS][2 * SP];
    grid_dependency_sync();

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sl = lane % SL, cg = lane / SL;
    const int blocks = p.G * p.blocks_g;
    const int64_t n = blockIdx.x / blocks;
    const int g = (blockIdx.x % blocks) / p.blocks_g;
    const int blk = blockIdx.x % p.blocks_g;
    const int cb = blk * CH;
    const int nch = p.Eg - cb < CH ? p.Eg - cb : CH;
    const int64_t c0 = (int64_t)g * p.Eg + cb;
    const int len = row_length(p.rows, n, p.T);
    const int64_t chunks = (p.T + TS - 1) / TS;

    const int lch = warp * Geo::WCH + cg * CPT;
    float A2[CPT][4], adj[CPT][4], dA[CPT][4];
    const bool ended = len > 0 && step_ended(p.rows, n, len - 1);
#pragma unroll
    for (int c = 0; c < CPT; ++c)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const bool in = lch + c < nch && sl * 4 + s < p.S;
            const int64_t i = (c0 + lch + c) * p.S + sl * 4 + s;
            A2[c][s] = in ? kLog2e * __ldg(p.A + i) : 0.f;
            adj[c][s] =
                in && p.d_final && !ended ? __ldg(p.d_final + n * p.E * p.S + i) : 0.f;
            dA[c][s] = 0.f;
        }

    const int col = IO::col();
    const bool active = col < nch;
    const int64_t ec = c0 + col;
    float bias[V], Dv[V], accD[V], accb[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bias[i] = active && p.dt_bias ? __ldg(p.dt_bias + ec + i) : 0.f;
        Dv[i] = active && p.D ? __ldg(p.D + ec + i) : 0.f;
        accD[i] = accb[i] = 0.f;
    }

    for (int t0 = (int)(chunks - 1) * TS; t0 >= 0; t0 -= TS) {
        Pack<T, V> rx[IO::kPer], rd[IO::kPer], rz[IO::kPer], rg[IO::kPer];
        IO::load(p.x, n, ec, active, t0, len, rx);
        IO::load(p.dt, n, ec, active, t0, len, rd);
        IO::load(p.dout, n, ec, active, t0, len, rg);
        if (p.z.ptr) IO::load(p.z, n, ec, active, t0, len, rz);
        const int steps = len - t0 < TS ? len - t0 : TS;
        unsigned starts = 0;
        if (steps > 0) {
#pragma unroll
            for (int k = 0; k < IO::kPer; ++k) {
                if (!IO::has(k)) continue;
                const int j = IO::step(k);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float raw = widen(rd[k].e[i]) + bias[i];
                    float q = widen(rg[k].e[i]);
                    if (p.z.ptr) q *= silu(widen(rz[k].e[i]));
                    sd[j][col + i] = p.softplus ? softplus(raw) : raw;
                    sx[j][col + i] = widen(rx[k].e[i]);
                    sq[j][col + i] = q;
                }
            }
            stage_bc<T, SP>(p, n, g, t0, len, sB, sC);
            starts = start_bits(p.rows, n, t0, len);
            __syncthreads();

            const float *saved = p.saved + (n * chunks + t0 / TS) * p.E * p.S;
            auto run = [&](int j, float (&h)[CPT][4]) {
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
                    const float d = sd[j][lch + c], w = d * sx[j][lch + c];
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        h[c][s] = fmaf(exp2_fast(d * A2[c][s]), h[c][s], w * sB[j][sl * 4 + s]);
                }
            };
#pragma unroll 1
            for (int j0 = TS - HB; j0 >= 0; j0 -= HB) {
                if (j0 >= steps) continue;
                float h[CPT][4], hp[HB][CPT][4];
#pragma unroll
                for (int c = 0; c < CPT; ++c)
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        h[c][s] = lch + c < nch && sl * 4 + s < p.S
                                      ? saved[(c0 + lch + c) * p.S + sl * 4 + s]
                                      : 0.f;
#pragma unroll 1
                for (int j = 0; j < j0; ++j) {
                    if ((starts >> j) & 1u)
#pragma unroll
                        for (int c = 0; c < CPT; ++c)
#pragma unroll
                            for (int s = 0; s < 4; ++s) h[c][s] = 0.f;
                    run(j, h);
                }
#pragma unroll
                for (int i = 0; i < HB; ++i) {
                    const int j = j0 + i;
                    if (j >= steps) break;
                    float y[CPT];
#pragma unroll
                    for (int c = 0; c < CPT; ++c)
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            if ((starts >> j) & 1u) h[c][s] = 0.f;
                            hp[i][c][s] = h[c][s];
                        }
                    run(j, h);
#pragma unroll
                    for (int c = 0; c < CPT; ++c) {
                        y[c] = 0.f;
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            y[c] = fmaf(sC[j][sl * 4 + s], h[c][s], y[c]);
                    }
                    reduce_scatter<CPT, SL, 1>(y);
                    constexpr int kOut = CPT >= SL ? CPT / SL : 1;
                    constexpr int kRep = SL > CPT ? SL / CPT : 1;
#pragma unroll
                    for (int o = 0; o < kOut; ++o)
                        if (sl % kRep == 0) sy[j][lch + (sl / kRep) * kOut + o] = y[o];
                }
#pragma unroll
                for (int i = HB - 1; i >= 0; --i) {
                    const int j = j0 + i;
                    if (j >= steps) continue;
                    float dbc[8], dd[CPT], gB[CPT];
#pragma unroll
                    for (int s = 0; s < 8; ++s) dbc[s] = 0.f;
#pragma unroll
                    for (int c = 0; c < CPT; ++c) {
                        const float d = sd[j][lch + c], x = sx[j][lch + c], q = sq[j][lch + c];
                        const float w = d * x;
                        dd[c] = gB[c] = 0.f;
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            const float B = sB[j][sl * 4 + s], C = sC[j][sl * 4 + s];
                            const float a = exp2_fast(d * A2[c][s]);
                            const float ah = a * hp[i][c][s];
                            const float gs = fmaf(q, C, adj[c][s]);
                            const float gah = gs * ah;
                            dbc[s] = fmaf(gs, w, dbc[s]);
                            dbc[4 + s] = fmaf(q, fmaf(w, B, ah), dbc[4 + s]);
                            dA[c][s] = fmaf(gah, d, dA[c][s]);
                            dd[c] = fmaf(gah, A2[c][s], dd[c]);
                            gB[c] = fmaf(gs, B, gB[c]);
                            adj[c][s] = (starts >> j) & 1u ? 0.f : a * gs;
                        }
                    }
                    reduce_scatter<CPT, SL, 1>(dd);
                    reduce_scatter<CPT, SL, 1>(gB);
                    reduce_scatter<8, CG, SL>(dbc);
                    constexpr int kOut = CPT >= SL ? CPT / SL : 1;
                    constexpr int kRep = SL > CPT ? SL / CPT : 1;
                    __syncwarp();  // the step's d and x have been read
#pragma unroll
                    for (int o = 0; o < kOut; ++o)
                        if (sl % kRep == 0) {
                            const int ch = lch + (sl / kRep) * kOut + o;
                            const float d = sd[j][ch], x = sx[j][ch];
                            sd[j][ch] = fmaf(gB[o], x, kLn2 * dd[o]);
                            sx[j][ch] = gB[o] * d;
                        }
                    constexpr int kBc = CG <= 8 ? 8 / CG : 1;
                    constexpr int kBcRep = CG > 8 ? CG / 8 : 1;
#pragma unroll
                    for (int o = 0; o < kBc; ++o)
                        if (cg % kBcRep == 0) {
                            const int v = (cg / kBcRep) * kBc + o;
                            red[warp][j][(v >> 2) * SP + sl * 4 + (v & 3)] = dbc[o];
                        }
                }
            }
            __syncthreads();

            for (int i = threadIdx.x; i < steps * 2 * SP; i += kScanThreads) {
                const int j = i / (2 * SP), v = i % (2 * SP);
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < kScanWarps; ++w) sum += red[w][j][v];
                p.part_bc[(((n * p.T + t0 + j) * p.G + g) * p.blocks_g + blk) * (2 * SP) + v] =
                    sum;
            }
        }
#pragma unroll
        for (int k = 0; k < IO::kPer; ++k) {
            const int j = IO::step(k), t = t0 + j;
            if (!active || !IO::has(k) || t >= p.T) continue;
            Pack<T, V> ox = zero_pack<T, V>(), od = ox, oz = ox;
            if (t < len) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float x = widen(rx[k].e[i]), go = widen(rg[k].e[i]);
                    float q = go;
                    if (p.z.ptr) {
                        const float z = widen(rz[k].e[i]), sg = sigmoid(z);
                        const float y = fmaf(Dv[i], x, sy[j][col + i]);
                        oz.e[i] = narrow<T>(go * y * sg * fmaf(z, 1.f - sg, 1.f));
                        q *= z * sg;
                    }
                    float dr = sd[j][col + i];
                    if (p.softplus) dr *= sigmoid(widen(rd[k].e[i]) + bias[i]);
                    od.e[i] = narrow<T>(dr);
                    ox.e[i] = narrow<T>(fmaf(Dv[i], q, sx[j][col + i]));
                    accD[i] = fmaf(q, x, accD[i]);
                    accb[i] += dr;
                }
            }
            store_pack<T, V>(row_ptr<T>(p.dx, n, t, ec), ox);
            store_pack<T, V>(row_ptr<T>(p.ddt, n, t, ec), od);
            if (p.z.ptr) store_pack<T, V>(row_ptr<T>(p.dz, n, t, ec), oz);
        }
        __syncthreads();
    }

#pragma unroll
    for (int c = 0; c < CPT; ++c)
#pragma unroll
        for (int s = 0; s < 4; ++s)
            if (lch + c < nch && sl * 4 + s < p.S) {
                const int64_t i = (n * p.E + c0 + lch + c) * p.S + sl * 4 + s;
                p.part_A[i] = dA[c][s];
                if (p.d_init) p.d_init[i] = adj[c][s];
            }
    // dD and ddt_bias: the threads that share a column add up in order.
    constexpr int kRows = IO::kVecs < kScanThreads ? IO::kVecs / IO::kCols
                                                   : kScanThreads / IO::kCols;
    static_assert(kRows <= TS, "one row of the tile per thread row");
    const int r = threadIdx.x / IO::kCols;
    if (IO::has(0)) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sd[r][col + i] = accD[i];
            sx[r][col + i] = accb[i];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < nch; c += kScanThreads) {
        float a = 0.f, b = 0.f;
        for (int k = 0; k < kRows; ++k) {
            a += sd[k][c];
            b += sx[k][c];
        }
        p.part_D[(n * 2 + 0) * p.E + c0 + c] = a;
        p.part_D[(n * 2 + 1) * p.E + c0 + c] = b;
    }
}

// dB and dC from the channel blocks' shares. One thread per (n, t, g, dB or dC, state).
template <typename T, int SP>
__global__ void __launch_bounds__(256) scan_bc_kernel(const ScanParams p)
{
    grid_dependency_sync();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int v = (int)(i % (2 * SP)), s = v % SP;
    const int64_t row = i / (2 * SP);  // (n, t, g)
    const int g = (int)(row % p.G);
    const int64_t nt = row / p.G;
    const int64_t n = nt / p.T;
    const int t = (int)(nt % p.T);
    if (n >= p.N || s >= p.S) return;
    float sum = 0.f;
    if (t < row_length(p.rows, n, p.T)) {
        const float *src = p.part_bc + row * p.blocks_g * (2 * SP) + v;
        for (int b = 0; b < p.blocks_g; ++b) sum += __ldcg(src + (int64_t)b * (2 * SP));
    }
    *row_ptr<T>(v < SP ? p.dB : p.dC, n, t, (int64_t)g * p.S + s) = narrow<T>(sum);
}

}  // namespace seq
}  // namespace rlca

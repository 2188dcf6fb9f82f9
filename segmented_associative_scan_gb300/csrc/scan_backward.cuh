// Selective scan, backward.
//
// With q_t = dout_t silu(z_t) and the state's adjoint run from the last step to the first,
//   g_t = adj_{t+1} + q_t C_t,   adj_t = a_t g_t (0 where t starts an episode),
//   dB_t = sum_e g_t d_t x_t          dC_t = sum_e q_t h_t
//   dA   = sum_t d_t adj_t h_{t-1}    dx_t = D q_t + d_t (g_t . B_t)
//   dd_t = A . (adj_t h_{t-1}) + x_t (g_t . B_t),   ddt_t = dd_t sigmoid(dt_t + bias),
// a_t = exp(d_t A). adj_t h_{t-1} is g_t a_t h_{t-1}, so the reverse step needs nine
// multiply-adds per state, and running h forward again four.
//
// A lane holds 4 states of 2 channels. The chunks of 8 steps are walked from the last to the
// first: h runs forward from the state the forward pass saved before the chunk and all 8
// states stay in registers for the reverse run over them. That is what chooses the chunk:
// 64 registers at 8 steps; saving every 16th step instead halves what is saved (8 bytes per
// element of x at 16 states) but repeats half of the forward run.
//
// Sums over states (C . h, A . adj h, g . B) leave the recurrence as one share per lane in
// shared memory, added where they are used. The shares of dB and dC are laid down there too
// and added up by lanes that take four of them in one read, a few steps at a time: exchanges
// of halves by shuffles took 29 instructions a step in place of 8. The warps of a CTA then add
// their shares, and the CTAs' shares are added in order by scan_bc_kernel. What a thread
// computes once per element (softplus, gate and their derivatives) runs in a phase of its own
// over a tile of steps, before and after the recurrence.
//
// [16, 1024, 2048] x 16 states, bf16: 884 us with its sums, 0.6 T states/s (fp32, where decays are
// CUDA's expf: 1302 us). The thirteen multiply-adds and two exponentials of a state and step need
// 190 and 116 us, HBM 85 (with the saved states 120). The load/store unit is what is fullest (70 %:
// broadcast reads of B, C, d, d x, q and the shares laid down and read again, 60 wavefronts to a
// warp's step of 256 states), then issue (228 instructions, 1.9 to a clock and SM at 12.7 warps).
#pragma once

#include "scan.cuh"

namespace rlca {
namespace seq {

template <int SL>
struct BackwardGeom {
    static constexpr int SP = 4 * SL;                 // states, padded
    static constexpr int CG = 32 / SL;                // lanes side by side in channels
    static constexpr int WC = 2 * CG;                 // channels of a warp
    static constexpr int CH = kBackwardWarps * WC;    // of a CTA
    static constexpr int L = RLCA_SCAN_CHUNK;         // steps of a tile: one chunk
    static constexpr int GS = 16 / SL < 1 ? 1 : (16 / SL > L ? L : 16 / SL);
    // steps whose dB and dC are added up together: every lane adds four sums of one step
};

// Bytes of shared memory that the kernel below declares (it checks them), and the CTAs to an SM that
// they let in: of 228 KB, 1 KB of it held back for each.
template <typename T, int SL, bool GATE>
__host__ __device__ constexpr int backward_shared()
{
    using Geo = BackwardGeom<SL>;
    constexpr int L = Geo::L, W = kBackwardWarps;
    constexpr int stage = 2 * (int)sizeof(T) * Geo::CH * (3 * L + (GATE ? L : 1));
    constexpr int steps = 2 * 4 * L * Geo::SP + 3 * 4 * L * Geo::CH;
    constexpr int shares = 8 * W * (GATE ? L : 1) * 32 + 16 * W * L * 32 + 16 * W * Geo::GS * 32 * 2 +
                           4 * W * L * 2 * Geo::SP;
    return stage + steps + shares;
}

template <typename T, int SL, bool GATE>
__host__ __device__ constexpr int backward_fit()
{
    return 228 * 1024 / (backward_shared<T, SL, GATE>() + 1024);
}

// CTAS: CTAs to an SM that the registers are cut for.
template <typename T, bool VEC, int SL, bool GATE, int CTAS>
__global__ void __launch_bounds__(kBackwardThreads, CTAS) scan_backward_kernel(const ScanParams p)
{
    using Geo = BackwardGeom<SL>;
    constexpr int CH = Geo::CH, SP = Geo::SP, CG = Geo::CG, L = Geo::L, GS = Geo::GS;
    constexpr int NT = kBackwardThreads, W = kBackwardWarps;
    static_assert(L % GS == 0 && CH <= NT, "whole groups; a thread for each channel");
    struct Stage {
        alignas(16) T x[L][CH];
        alignas(16) T d[L][CH];
        alignas(16) T g[L][CH];
        alignas(16) T z[GATE ? L : 1][CH];
    };
    __shared__ Stage stage[2];
    __shared__ __align__(16) float sB[L][SP];
    __shared__ __align__(16) float sC[L][SP];
    __shared__ __align__(16) float sd[L][CH];              // d
    __shared__ __align__(16) float sw[L][CH];              // d x
    __shared__ __align__(16) float sq[L][CH];              // q
    __shared__ float2 sy[W][GATE ? L : 1][32];             // lanes' shares of C . h, both channels
    __shared__ float4 sg[W][L][32];                        // of A2 . (adj h) and g . B, both
    __shared__ float4 sbc[W][GS][32][2];                   // of dB and dC
    __shared__ __align__(16) float red[W][L][2 * SP];      // warps' shares of dB and dC
    static_assert(sizeof(stage) + sizeof(sB) + sizeof(sC) + sizeof(sd) + sizeof(sw) + sizeof(sq) +
                          sizeof(sy) + sizeof(sg) + sizeof(sbc) + sizeof(red) ==
                      backward_shared<T, SL, GATE>(),
                  "the launch counts with what is declared here");
    grid_dependency_sync();

    const ScanPlace<CH> at(p);
    const int64_t n = at.n;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sl = lane % SL, cg = lane / SL;
    const int len = row_length(p.rows, n, p.T);
    const int tb = at.span * p.span_steps;
    const int te = p.T - tb < p.span_steps ? p.T : tb + p.span_steps;
    const int end = te < len ? te : len;  // steps tb .. end - 1 are run
    const int64_t chunks = (p.T + L - 1) / L;
    const int64_t slot = n * p.spans + at.span;

    // The lane's channels and states.
    const int lch = warp * Geo::WC + cg * 2;
    const int64_t ch = at.c0 + lch;
    const bool in[2] = {lch < at.nch, lch + 1 < at.nch};
    Pair A2[2][2], adj[2][2], dA[2][2];
    {
        const bool ended = len > 0 && step_ended(p.rows, n, len - 1);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float a[4], v[4];
            load_states(p.A, ch + c, sl, p.S, in[c], a);
            if (p.spans > 1)
                load_states(p.span_state + slot * p.E * p.S, ch + c, sl, p.S, in[c], v);
            else
                load_states(p.d_final + n * p.E * p.S, ch + c, sl, p.S,
                            in[c] && p.d_final && !ended, v);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                A2[c][i] = pair(finite_decay_base<T>(a[2 * i]), finite_decay_base<T>(a[2 * i + 1]));
                adj[c][i] = pair(v[2 * i], v[2 * i + 1]);
                dA[c][i] = pair(0.f, 0.f);
            }
        }
    }

    // The thread's elements of a tile: two channels, every kSkip-th step.
    constexpr int kSkip = NT / (CH / 2), kPairs = L > kSkip ? L / kSkip : 1;
    static_assert(NT % (CH / 2) == 0, "a thread keeps its channels");
    const int ec = threadIdx.x % (CH / 2) * 2, ej = threadIdx.x / (CH / 2);
    const int have = at.nch - ec < 0 ? 0 : (at.nch - ec < 2 ? at.nch - ec : 2);
    float bias[2], skip[2];
    // dD and ddt_bias: sums of 16 tiles, and of those (one running sum over a thousand steps
    // loses digits).
    float accD[2] = {0.f, 0.f}, accb[2] = {0.f, 0.f}, sumD[2] = {0.f, 0.f}, sumb[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        bias[c] = c < have && p.dt_bias ? __ldg(p.dt_bias + at.c0 + ec + c) : 0.f;
        skip[c] = c < have && p.D ? __ldg(p.D + at.c0 + ec + c) : 0.f;
    }
    auto write = [&](T *dst, float a, float b) {
        if constexpr (VEC) {
            Pack<T, 2> v;
            v.e[0] = narrow<T>(a), v.e[1] = narrow<T>(b);
            if (have) *reinterpret_cast<Pack<T, 2> *>(dst) = v;
        } else {
            if (have > 0) dst[0] = narrow<T>(a);
            if (have > 1) dst[1] = narrow<T>(b);
        }
    };

    // One warp fetches x, dt and B, the other dout, z and C: half the addresses in each.
    static_assert(W == 2, "two warps share the loads");
    TileCopy<T, VEC, CH, L, CH, 32> c1(warp ? p.dout : p.x, n, at.c0, at.nch, lane),
        c2(warp ? p.z : p.dt, n, at.c0, at.nch, lane);
    TileBC<T, SP, L, 32> nBC(warp ? p.C : p.B, p, n, at.g, lane);
    auto copy = [&](int b, int t0) {
        c1.start(warp ? stage[b].g : stage[b].x, t0, end);
        if (GATE || warp == 0) c2.start(warp ? stage[b].z : stage[b].d, t0, end);
        copies_commit();
    };
    auto land = [&](int b) {
        c1.land(warp ? stage[b].g : stage[b].x);
        if (GATE || warp == 0) c2.land(warp ? stage[b].z : stage[b].d);
    };
    // The states saved before the chunk of step t (zeros before the span), t going down from
    // the span's last chunk.
    const bool wide = p.S % 4 == 0 && reinterpret_cast<uintptr_t>(p.saved) % 16 == 0;
    auto load_saved = [&](int t, Pair (&h)[2][2]) {
        const float *base = p.saved + (n * chunks + t / L) * p.E * p.S + ch * p.S + sl * 4;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            const float *q = base + c * p.S;
            if (in[c] && t >= tb && sl * 4 < p.S) {
                if (wide) {
                    v = *reinterpret_cast<const float4 *>(q);
                } else {
                    v.x = q[0];
                    if (sl * 4 + 1 < p.S) v.y = q[1];
                    if (sl * 4 + 2 < p.S) v.z = q[2];
                    if (sl * 4 + 3 < p.S) v.w = q[3];
                }
            }
            h[c][0] = pair(v.x, v.y);
            h[c][1] = pair(v.z, v.w);
        }
    };

    // Steps past the row.
    for (int t = (end > tb ? end : tb) + ej; t < te; t += kSkip) {
        write(row_ptr<T>(p.dx, n, t, at.c0 + ec), 0.f, 0.f);
        write(row_ptr<T>(p.ddt, n, t, at.c0 + ec), 0.f, 0.f);
        if (GATE) write(row_ptr<T>(p.dz, n, t, at.c0 + ec), 0.f, 0.f);
    }

    const int tiles = end > tb ? (end - tb + L - 1) / L : 0;
    // The thread's first element of a tile, from the last tile on.
    T *dx = row_ptr<T>(p.dx, n, tb + (tiles - 1) * L + ej, at.c0 + ec);
    T *ddt = row_ptr<T>(p.ddt, n, tb + (tiles - 1) * L + ej, at.c0 + ec);
    T *dz = row_ptr<T>(p.dz, n, tb + (tiles - 1) * L + ej, at.c0 + ec);
    // The thread's first share of dB and dC of a tile.
    constexpr int kRows = NT / (2 * SP) > 0 ? NT / (2 * SP) : 1;  // steps of one sweep
    const int64_t share_step = (int64_t)p.G * p.blocks_g * (2 * SP);
    float *share = p.part_bc +
                   ((n * p.T + tb + (tiles - 1) * L) * p.G + at.g) * p.blocks_g * (2 * SP) +
                   at.blk * (2 * SP);
    unsigned word = 0;  // where episodes start, 32 steps at a time
    Pair h[2][2];
    if (tiles > 0) {
        copy((tiles - 1) & 1, tb + (tiles - 1) * L);
        land((tiles - 1) & 1);
        nBC.load(tb + (tiles - 1) * L, end);
        load_saved(tb + (tiles - 1) * L, h);
    }
#pragma unroll 1
    for (int k = tiles - 1; k >= 0; --k) {
        const int t0 = tb + k * L;
        const Stage &st = stage[k & 1];
        const int steps = end - t0 < L ? end - t0 : L;
        copies_wait();
        __syncthreads();  // the tile is there; the last tile's results have been read
        nBC.store(warp ? sC : sB);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const int j = ej + i * kSkip;
            if (kSkip > L && j >= L) break;
            const Pack<T, 2> rx = get2(&st.x[j][ec]), rd = get2(&st.d[j][ec]),
                             rg = get2(&st.g[j][ec]);
            float2 d, q;
            d.x = widen(rd.e[0]) + bias[0], d.y = widen(rd.e[1]) + bias[1];
            if (p.softplus) d.x = softplus<T>(d.x), d.y = softplus<T>(d.y);
            if (j >= steps) d.x = d.y = 0.f;  // steps past the row keep state and adjoint
            q.x = widen(rg.e[0]), q.y = widen(rg.e[1]);
            if (GATE) {
                const Pack<T, 2> rz = get2(&st.z[j][ec]);
                q.x *= silu<T>(widen(rz.e[0])), q.y *= silu<T>(widen(rz.e[1]));
            }
            *reinterpret_cast<float2 *>(&sd[j][ec]) = d;
            *reinterpret_cast<float2 *>(&sw[j][ec]) =
                make_float2(d.x * widen(rx.e[0]), d.y * widen(rx.e[1]));
            *reinterpret_cast<float2 *>(&sq[j][ec]) = q;
        }
        if (k == tiles - 1 || t0 % 32 == 32 - L)
            word = start_bits(p.rows, n, t0 / 32 * 32, end);
        const unsigned starts = word >> (t0 % 32);
        __syncthreads();
        if (k > 0) copy((k - 1) & 1, t0 - L);

        // Forward over the chunk.
        Pair hs[L][2][2];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if ((starts >> i) & 1u)
#pragma unroll
                for (int c = 0; c < 2; ++c) h[c][0] = h[c][1] = pair(0.f, 0.f);
            asm volatile("" ::: "memory");  // no reads ahead: registers are short
            const float2 d = *reinterpret_cast<const float2 *>(&sd[i][lch]);
            const float2 w = *reinterpret_cast<const float2 *>(&sw[i][lch]);
            const float4 Bv = *reinterpret_cast<const float4 *>(&sB[i][sl * 4]);
            const Pair B[2] = {pair(Bv.x, Bv.y), pair(Bv.z, Bv.w)};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const Pair d2 = c ? pair(d.y, d.y) : pair(d.x, d.x);
                const Pair w2 = c ? pair(w.y, w.y) : pair(w.x, w.x);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    h[c][s] = fma2(decay<T>(d2, A2[c][s]), h[c][s], mul2(w2, B[s]));
                    hs[i][c][s] = h[c][s];
                }
            }
            if (GATE) {
                const float4 Cv = *reinterpret_cast<const float4 *>(&sC[i][sl * 4]);
                const Pair C[2] = {pair(Cv.x, Cv.y), pair(Cv.z, Cv.w)};
                const float2 a = split(fma2(C[1], h[0][1], mul2(C[0], h[0][0])));
                const float2 b = split(fma2(C[1], h[1][1], mul2(C[0], h[1][0])));
                sy[warp][i][lane] = make_float2(a.x + a.y, b.x + b.y);
            }
        }
        // And back. The chunk's share of dA is added up by itself: over a thousand steps one
        // running sum loses more than all else.
        Pair local[2][2];
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            asm volatile("" ::: "memory");
            if (i == L / 2 - 1) load_saved(t0, h);  // again: the registers are free by now
            const float2 d = *reinterpret_cast<const float2 *>(&sd[i][lch]);
            const float2 w = *reinterpret_cast<const float2 *>(&sw[i][lch]);
            const float2 q = *reinterpret_cast<const float2 *>(&sq[i][lch]);
            const float4 Bv = *reinterpret_cast<const float4 *>(&sB[i][sl * 4]);
            const float4 Cv = *reinterpret_cast<const float4 *>(&sC[i][sl * 4]);
            const Pair B[2] = {pair(Bv.x, Bv.y), pair(Bv.z, Bv.w)};
            const Pair C[2] = {pair(Cv.x, Cv.y), pair(Cv.z, Cv.w)};
            const bool reset = (starts >> i) & 1u;
            Pair dB[2], dC[2];
            float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const Pair d2 = c ? pair(d.y, d.y) : pair(d.x, d.x);
                const Pair w2 = c ? pair(w.y, w.y) : pair(w.x, w.x);
                const Pair q2 = c ? pair(q.y, q.y) : pair(q.x, q.x);
                Pair g[2], gB;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    g[s] = fma2(q2, C[s], adj[c][s]);
                    dB[s] = c ? fma2(g[s], w2, dB[s]) : mul2(g[s], w2);
                    dC[s] = c ? fma2(q2, hs[i][c][s], dC[s]) : mul2(q2, hs[i][c][s]);
                    gB = s ? fma2(g[s], B[s], gB) : mul2(g[s], B[s]);
                }
                sums[2 + c] = gB.x + gB.y;
                if (i == L - 1) local[c][0] = local[c][1] = pair(0.f, 0.f);
                if (reset) {
                    adj[c][0] = adj[c][1] = pair(0.f, 0.f);
                } else {
                    Pair gA;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        adj[c][s] = mul2(decay<T>(d2, A2[c][s]), g[s]);
                        const Pair ah = mul2(adj[c][s], i ? hs[i ? i - 1 : 0][c][s] : h[c][s]);
                        local[c][s] = fma2(ah, d2, local[c][s]);
                        gA = s ? fma2(ah, A2[c][s], gA) : mul2(ah, A2[c][s]);
                    }
                    sums[c] = gA.x + gA.y;
                }
            }
            sg[warp][i][lane] = make_float4(sums[0], sums[1], sums[2], sums[3]);
            // Neighbouring lanes' halves change places, so that no banks collide.
            const int half = (lane >> 2) & 1;
            sbc[warp][i % GS][lane][half] = make_float4(dB[0].x, dB[0].y, dB[1].x, dB[1].y);
            sbc[warp][i % GS][lane][half ^ 1] = make_float4(dC[0].x, dC[0].y, dC[1].x, dC[1].y);
            if (i % GS == 0) {
                __syncwarp();
                // Lane (step, dB or dC, state quarter) adds over the lanes of the channels.
#pragma unroll
                for (int o = lane; o < GS * 2 * SL; o += 32) {
                    const int step = o / (2 * SL), v = o / SL % 2, s = o % SL;
                    Pair a = pair(0.f, 0.f), b = a;
#pragma unroll
                    for (int m = 0; m < CG; ++m) {
                        const int from = m * SL + s;
                        const float4 f = sbc[warp][step][from][v ^ ((from >> 2) & 1)];
                        a = m ? add2(a, pair(f.x, f.y)) : pair(f.x, f.y);
                        b = m ? add2(b, pair(f.z, f.w)) : pair(f.z, f.w);
                    }
                    *reinterpret_cast<float4 *>(&red[warp][i + step][v * SP + s * 4]) =
                        make_float4(a.x, a.y, b.x, b.y);
                }
                __syncwarp();
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int s = 0; s < 2; ++s) dA[c][s] = add2(dA[c][s], local[c][s]);
        load_saved(t0 - L, h);  // for the next tile
        if (k > 0) land((k - 1) & 1);
        __syncthreads();

        if (k > 0) nBC.load(t0 - L, end);  // arrives while the results are finished
        {
            constexpr int kWide = 2 * SP < NT ? 2 * SP : NT;
            const int j0 = threadIdx.x / kWide;
            float *dst = share + j0 * share_step;
#pragma unroll
            for (int j = j0; j < L; j += kRows, dst += kRows * share_step) {
                if (j < steps)
#pragma unroll
                    for (int v = threadIdx.x % kWide; v < 2 * SP; v += kWide) {
                        float sum = red[0][j][v];
#pragma unroll
                        for (int w = 1; w < W; ++w) sum += red[w][j][v];
                        dst[v] = sum;
                    }
            }
            share -= L * share_step;
        }
        T *px = dx, *pd = ddt, *pz = dz;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const int j = ej + i * kSkip;
            if (j < steps) {
                const int sw_ = ec / Geo::WC, from = ec % Geo::WC / 2 * SL;  // warp, first lane
                const float2 q = *reinterpret_cast<const float2 *>(&sq[j][ec]);
                const float2 d = *reinterpret_cast<const float2 *>(&sd[j][ec]);
                const Pack<T, 2> rx = get2(&st.x[j][ec]);
                const float x[2] = {widen(rx.e[0]), widen(rx.e[1])};
                Pair gA = pair(0.f, 0.f), gB = gA;
#pragma unroll
                for (int m = 0; m < SL; ++m) {
                    const float4 f = sg[sw_][j][from + m];
                    gA = m ? add2(gA, pair(f.x, f.y)) : pair(f.x, f.y);
                    gB = m ? add2(gB, pair(f.z, f.w)) : pair(f.z, f.w);
                }
                if (GATE) {
                    Pair y = sy[sw_][j][from];
#pragma unroll
                    for (int m = 1; m < SL; ++m) y = add2(y, sy[sw_][j][from + m]);
                    const Pack<T, 2> rg = get2(&st.g[j][ec]), rz = get2(&st.z[j][ec]);
                    float v[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float z = widen(rz.e[c]), s = sigmoid<T>(z);
                        const float yc = fmaf(skip[c], x[c], c ? y.y : y.x);
                        v[c] = widen(rg.e[c]) * yc * (s * fmaf(z, 1.f - s, 1.f));
                    }
                    write(pz, v[0], v[1]);
                }
                float2 dr = make_float2(fmaf(gB.x, x[0], decay_unit<T>() * gA.x),
                                        fmaf(gB.y, x[1], decay_unit<T>() * gA.y));
                if (p.softplus) {
                    const Pack<T, 2> rd = get2(&st.d[j][ec]);
                    dr.x *= sigmoid<T>(widen(rd.e[0]) + bias[0]);
                    dr.y *= sigmoid<T>(widen(rd.e[1]) + bias[1]);
                }
                write(pd, dr.x, dr.y);
                write(px, fmaf(skip[0], q.x, gB.x * d.x), fmaf(skip[1], q.y, gB.y * d.y));
                accD[0] = fmaf(q.x, x[0], accD[0]), accD[1] = fmaf(q.y, x[1], accD[1]);
                accb[0] += dr.x, accb[1] += dr.y;
            }
            px += kSkip * p.dx.step, pd += kSkip * p.ddt.step, pz += kSkip * p.dz.step;
        }
        dx -= L * p.dx.step, ddt -= L * p.ddt.step, dz -= L * p.dz.step;
        if (k % 16 == 0) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                sumD[c] += accD[c], sumb[c] += accb[c];
                accD[c] = accb[c] = 0.f;
            }
        }
    }

#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const float v[4] = {dA[c][0].x, dA[c][0].y, dA[c][1].x, dA[c][1].y};
        store_states(p.part_p + slot * p.E * (p.S + 2), ch + c, sl, p.S, in[c], v);
        if (p.d_init && at.span == 0) {
            const float w[4] = {adj[c][0].x, adj[c][0].y, adj[c][1].x, adj[c][1].y};
            store_states(p.d_init + n * p.E * p.S, ch + c, sl, p.S, in[c], w);
        }
    }
    // dD and ddt_bias: the threads that share a channel add up in order.
    __syncthreads();
    float *shared = &sg[0][0][0].x;
    static_assert(sizeof(sg) >= 4 * NT * sizeof(float), "a place for each thread's sums");
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        shared[ej * CH + ec + c] = sumD[c];
        shared[2 * NT + ej * CH + ec + c] = sumb[c];
    }
    __syncthreads();
    if (threadIdx.x < at.nch) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int k = 0; k < kSkip; ++k) {
            a += shared[k * CH + threadIdx.x];
            b += shared[2 * NT + k * CH + threadIdx.x];
        }
        float *dst = p.part_p + slot * p.E * (p.S + 2) + p.E * p.S + at.c0 + threadIdx.x;
        dst[0] = a;
        dst[p.E] = b;
    }
}

// First pass over spans, run backwards: what a span adds to the adjoint before it, from an
// adjoint of zero behind it, and the sum of its step sizes. A lane holds 8 states of one
// channel; a block of steps is shared by the SL lanes of a channel, as in the forward pass.
template <typename T, int SL, bool GATE>
__global__ void __launch_bounds__(kForwardThreads) scan_adjoint_kernel(const ScanParams p)
{
    constexpr int SP = 8 * SL, CH = kForwardThreads / SL, TS = 16, U = SL < 4 ? 4 : SL, K = U / SL;
    __shared__ __align__(16) float sC[2][TS][SP];
    grid_dependency_sync();
    const ScanPlace<CH> at(p);
    if (at.span == 0) return;  // nothing comes before it
    const int64_t n = at.n;
    const int lane = threadIdx.x & 31;
    const int sl = lane % SL, lch = threadIdx.x / SL;
    const bool active = lch < at.nch;
    const int64_t ch = at.c0 + lch;
    const int len = row_length(p.rows, n, p.T);
    const int tb = at.span * p.span_steps;
    const int te = p.T - tb < p.span_steps ? p.T : tb + p.span_steps;
    const int end = te < len ? te : len;
    Pair A2[4], adj[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float a[4];
        load_states(p.A, ch, 2 * sl + k, p.S, active, a);
        A2[2 * k] = pair(finite_decay_base<T>(a[0]), finite_decay_base<T>(a[1]));
        A2[2 * k + 1] = pair(finite_decay_base<T>(a[2]), finite_decay_base<T>(a[3]));
        adj[2 * k] = adj[2 * k + 1] = pair(0.f, 0.f);
    }
    float sum = 0.f;
    const float bias = active && p.dt_bias ? __ldg(p.dt_bias + ch) : 0.f;
    TileBC<T, SP, TS, kForwardThreads> nC(p.C, p, n, at.g, threadIdx.x);
    T rd[K], rg[K], rz[K];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int t = t0 + k * SL + sl;
            const bool in = active && t >= tb && t < end;
            rd[k] = in ? *row_ptr<T>(p.dt, n, t, ch) : narrow<T>(0.f);
            rg[k] = in ? *row_ptr<T>(p.dout, n, t, ch) : narrow<T>(0.f);
            if (GATE) rz[k] = in ? *row_ptr<T>(p.z, n, t, ch) : narrow<T>(0.f);
        }
    };
    const int tiles = end > tb ? (end - tb + TS - 1) / TS : 0;
    if (tiles > 0) {
        nC.load(tb + (tiles - 1) * TS, end);
        fetch(tb + (tiles - 1) * TS + TS - U);
    }
    for (int k0 = tiles - 1; k0 >= 0; --k0) {
        const int t0 = tb + k0 * TS;
        nC.store(sC[k0 & 1]);
        __syncthreads();
        if (k0 > 0) nC.load(t0 - TS, end);
        const unsigned starts = start_bits(p.rows, n, t0, end);
#pragma unroll 1
        for (int j0 = TS - U; j0 >= 0; j0 -= U) {
            float d[K], q[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float raw = widen(rd[k]) + bias;
                d[k] = p.softplus ? softplus<T>(raw) : raw;
                if (t0 + j0 + k * SL + sl >= end) d[k] = 0.f;
                q[k] = widen(rg[k]);
                if (GATE) q[k] *= silu<T>(widen(rz[k]));
            }
            fetch(t0 + j0 - U);
#pragma unroll
            for (int u = U - 1; u >= 0; --u) {
                float du = d[u / SL], qu = q[u / SL];
                if (SL > 1) {
                    const int from = (lane & ~(SL - 1)) | (u % SL);
                    du = __shfl_sync(kFullMask, du, from);
                    qu = __shfl_sync(kFullMask, qu, from);
                }
                const Pair d2 = pair(du, du), q2 = pair(qu, qu);
                Pair C[4];
                load_pairs(&sC[k0 & 1][j0 + u][sl * 8], C);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    adj[i] = mul2(decay<T>(d2, A2[i]), fma2(q2, C[i], adj[i]));
                sum += du;
                if ((starts >> (j0 + u)) & 1u) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) adj[i] = pair(0.f, 0.f);
                    sum = __int_as_float(0x7fc00000);
                }
            }
        }
    }
    const int64_t slot = n * p.spans + at.span;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float v[4] = {adj[2 * k].x, adj[2 * k].y, adj[2 * k + 1].x, adj[2 * k + 1].y};
        store_states(p.span_state + slot * p.E * p.S, ch, 2 * sl + k, p.S, active, v);
    }
    if (sl == 0 && active) p.span_sum[slot * p.E + ch] = sum;
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
#pragma unroll 8
        for (int b = 0; b < p.blocks_g; ++b) sum += __ldcg(src + (int64_t)b * (2 * SP));
    }
    *row_ptr<T>(v < SP ? p.dB : p.dC, n, t, (int64_t)g * p.S + s) = narrow<T>(sum);
}

}  // namespace seq
}  // namespace rlca

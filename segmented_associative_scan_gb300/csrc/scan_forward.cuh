// Selective scan, forward.
//
// A lane holds 8 states of one channel, SL lanes side by side all of its states. In a block of
// U steps each of the SL lanes turns x, dt and z of its U / SL steps into d and d x (so the
// softplus and the gate are computed once per element), hands them to the others by shuffles
// and, after the sums over states are exchanged, ends with C . h of the same steps, which it
// finishes and writes. The raw x, dt, z of the next tile of steps arrive in shared memory by
// asynchronous copies while a tile is computed; B and C, which all channels of the group need,
// are staged there in fp32. One barrier to a tile.
//
// States go in pairs through two-lane instructions: B and C then need no copies in registers.
// Per step and state one exponential (32 lanes a clock and SM) and four fp32 operations (128)
// are needed, and B and C cost the load/store unit 4 bytes each per lane: 8 states of one
// channel to a lane keep twice the warps of 4 channels x 4 states, and at [16, 1024, 2048]
// warps are what is short (measured 490 us there with 4 x 4, 1.7 warps to a scheduler).
//
// [16, 1024, 2048] x 16 states, bf16: 217 us, 2.5 T states/s and 1.25 TB/s (236 us with the states
// saved for the backward pass). The exponentials alone need 58 us, the fp32 operations as long
// beside them, HBM 40. What takes the time is issue and latency: 77 instructions to a warp's step of
// 256 states, 2.35 to a clock of the 4 that an SM can, with 3 warps to a scheduler; half of them
// are the recurrence, a fifth the work per element. No unit is full.
//
// Where the rows and channels alone leave SMs idle, a row is cut into spans. A first pass
// runs each span from a zero state (no C, no outputs), a small kernel joins the spans in
// order (a span multiplies what comes in by exp(A sum d)), and the second pass runs all
// spans from their true states, at twice the arithmetic.
#pragma once

#include <cstddef>

#include "scan.cuh"

namespace rlca {
namespace seq {

template <typename T, int SL>
struct ForwardGeom {
    static constexpr int SP = 8 * SL;                      // states, padded
    static constexpr int WC = 32 / SL;                     // channels of a warp
    static constexpr int CH = kForwardWarps * WC;             // of a CTA
    static constexpr int U = SL < 4 ? 4 : SL;              // steps of a block
    static constexpr int K = U / SL;                       // of which a lane reads
    static constexpr int kRow = CH * (int)sizeof(T);
    static constexpr int TS = kRow >= 512 ? 8 : (kRow >= 256 ? 16 : 32);  // steps of a tile
    // The SL steps that a warp reads at once fall into different banks.
    static constexpr int kPad = WC * (int)sizeof(T) < 16 ? 16 / (int)sizeof(T) : WC;
    static constexpr int P = CH + kPad;                    // pitch of a staged row
};

// CTAs to an SM that the registers are cut for (0: the compiler's choice). Measured, 1024 steps of
// 2048 channels (64 states: 1024), us, 0 / 4 / 5 / 6 / 8:
//    8 states  bf16 N = 16  175 / 151 / 175 / 175 / 178   fp32 N = 16  289 / 239 / 284 / 284 / 291
//   16 states  bf16 N = 16  217 / 290 / 280 / 268 / 217   fp32 N = 4   214 / 189 / 202 / 194 / 213
//                                                         fp32 N = 16  433 / 456 / 480 / 443 / 413
//                                                         fp32 N = 32  723 / 842 / 761 / 723 / 719
//   32 states  bf16 N = 8   227 / 292 / 294 / 304 / 226   fp32 N = 8   412 / 423 / 406 / 399 / 410
//   64 states  bf16 N = 8   416 / 442 / 413 / 397 / 389   fp32 N = 8   457 / 504 / 447 / 449 / 526
// (bf16 [1, 8192, 2048] x 16 in spans 211 / 220 / - / - / 173.) 16 bits: 8 above 8 states, also at 64,
// where shared memory lets in 5 and 72 bytes spill. fp32: 4, the fastest of few CTAs and of up to 8
// states, although many CTAs would run up to a seventh faster at 8: one cut for all grids. 16-bit rows
// of odd alignment pass through registers ([33, 517, 1027] ragged: 105 at 0, 164 at 8).
template <typename T, bool VEC, int SL>
__host__ __device__ constexpr int forward_ctas()
{
    if (sizeof(T) == 4 || SL == 1) return 4;
    return VEC ? 8 : 0;
}

// LOCAL: the first pass over spans: leaves span_state and span_sum. GATE: z is given.
template <typename T, bool VEC, int SL, bool LOCAL, bool GATE>
__global__ void __launch_bounds__(kForwardThreads, forward_ctas<T, VEC, SL>())
    scan_forward_kernel(const ScanParams p)
{
    using Geo = ForwardGeom<T, SL>;
    constexpr int SP = Geo::SP, TS = Geo::TS, U = Geo::U, K = Geo::K, CH = Geo::CH, P = Geo::P;
    static_assert(TS % U == 0 && RLCA_SCAN_CHUNK % U == 0, "blocks fit tiles and chunks");
    // One struct, so that a lane's place in all its arrays moves on with one addition.
    struct Stage {
        alignas(16) T x[TS][P];
        T d[TS][P];
        T z[GATE ? TS : 1][P];
        float B[TS][SP];
        float C[LOCAL ? 1 : TS][SP];
    };
    __shared__ Stage stage[2];
    constexpr int kD = (int)(offsetof(Stage, d) - offsetof(Stage, x)) / (int)sizeof(T);
    constexpr int kZ = (int)(offsetof(Stage, z) - offsetof(Stage, x)) / (int)sizeof(T);
    constexpr int kC = (int)(offsetof(Stage, C) - offsetof(Stage, B)) / 4;
    grid_dependency_sync();

    const ScanPlace<CH> at(p);
    if (LOCAL && at.span == p.spans - 1) return;  // nothing comes after it
    const int64_t n = at.n;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sl = lane % SL, lch = warp * Geo::WC + lane / SL;
    const bool active = lch < at.nch;
    const int64_t ch = at.c0 + lch;
    const int len = row_length(p.rows, n, p.T);
    const int tb = at.span * p.span_steps;
    const int te = p.T - tb < p.span_steps ? p.T : tb + p.span_steps;
    const int end = te < len ? te : len;  // steps tb .. end - 1 are run

    Pair A2[4], h[4];
    float sum = 0.f;
    {
        float a[2][4], v[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            load_states(p.A, ch, 2 * sl + k, p.S, active, a[k]);
            if (!LOCAL && p.spans > 1)
                load_states(p.span_state + (n * p.spans + at.span) * p.E * p.S, ch, 2 * sl + k,
                            p.S, active, v[k]);
            else
                load_states(p.init + n * p.E * p.S, ch, 2 * sl + k, p.S,
                            !LOCAL && p.init && active, v[k]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            A2[i] = pair(finite_decay_base<T>(a[i / 2][i % 2 * 2]),
                         finite_decay_base<T>(a[i / 2][i % 2 * 2 + 1]));
            h[i] = pair(v[i / 2][i % 2 * 2], v[i / 2][i % 2 * 2 + 1]);
        }
    }
    auto store_h = [&](float *base) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 a = split(h[2 * k]), b = split(h[2 * k + 1]);
            const float v[4] = {a.x, a.y, b.x, b.y};
            store_states(base, ch, 2 * sl + k, p.S, active, v);
        }
    };
    auto clear_h = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = pair(0.f, 0.f);
    };
    const float bias = active && p.dt_bias ? __ldg(p.dt_bias + ch) : 0.f;
    const float skip = active && p.D && !LOCAL ? __ldg(p.D + ch) : 0.f;

    TileCopy<T, VEC, CH, TS, P, kForwardThreads> cx(p.x, n, at.c0, at.nch, threadIdx.x),
        cd(p.dt, n, at.c0, at.nch, threadIdx.x), cz(p.z, n, at.c0, at.nch, threadIdx.x);
    TileBC<T, SP, TS, kForwardThreads> nB(p.B, p, n, at.g, threadIdx.x),
        nC(p.C, p, n, at.g, threadIdx.x);
    auto copy = [&](int b, int t0) {
        cx.start(stage[b].x, t0, end);
        cd.start(stage[b].d, t0, end);
        if (GATE) cz.start(stage[b].z, t0, end);
        copies_commit();
    };
    auto land = [&](int b) {
        cx.land(stage[b].x);
        cd.land(stage[b].d);
        if (GATE) cz.land(stage[b].z);
    };
    auto load_bc = [&](int t0) {
        nB.load(t0, end);
        if (!LOCAL) nC.load(t0, end);
    };
    if (tb < end) {
        copy(0, tb);
        load_bc(tb);
        land(0);
    }
    unsigned starts = start_bits(p.rows, n, tb, end);
    T *out = row_ptr<T>(p.out, n, tb + sl, ch);  // the lane's first step of a block
    const int64_t out_next = SL * p.out.step, out_block = U * p.out.step;

    int buf = 0;
    for (int t0 = tb; t0 < end; t0 += TS, buf ^= 1) {
        nB.store(stage[buf].B);
        if constexpr (!LOCAL) nC.store(stage[buf].C);
        const unsigned now = starts;
        copies_wait();
        __syncthreads();  // the tile is there, and the other buffers have been read
        if (t0 + TS < end) {
            copy(buf ^ 1, t0 + TS);
            load_bc(t0 + TS);
            starts = start_bits(p.rows, n, t0 + TS, end);
        }
        const int stop = end - t0 < TS ? end - t0 : TS;
        const T *px = &stage[buf].x[sl][lch];
        const float *pB = &stage[buf].B[0][sl * 8];
#pragma unroll 1
        for (int j0 = 0; j0 < stop; j0 += U, px += U * P, pB += U * SP, out += out_block) {
            // h before the chunk, for the backward pass.
            if (!LOCAL && p.saved && (t0 + j0) % RLCA_SCAN_CHUNK == 0) {
                const int64_t chunks = (p.T + RLCA_SCAN_CHUNK - 1) / RLCA_SCAN_CHUNK;
                store_h(p.saved + (n * chunks + (t0 + j0) / RLCA_SCAN_CHUNK) * p.E * p.S);
            }
            float d[K], w[K], x[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float raw = widen(px[k * SL * P + kD]) + bias;
                x[k] = widen(px[k * SL * P]);
                d[k] = p.softplus ? softplus<T>(raw) : raw;
                if (j0 + k * SL + sl >= stop) d[k] = 0.f;  // steps past the row keep the state
                w[k] = d[k] * x[k];
            }
            const unsigned first = (now >> j0) & ((1u << U) - 1u);
            float y[U];
            auto run = [&](auto resets) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (decltype(resets)::value && ((first >> u) & 1u)) {
                        clear_h();
                        sum = __int_as_float(0x7fc00000);
                    }
                    float du = d[u / SL], wu = w[u / SL];
                    if (SL > 1) {
                        const int from = (lane & ~(SL - 1)) | (u % SL);
                        du = __shfl_sync(kFullMask, du, from);
                        wu = __shfl_sync(kFullMask, wu, from);
                    }
                    const Pair d2 = pair(du, du), w2 = pair(wu, wu);
                    Pair B[4];
                    load_pairs(pB + u * SP, B);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        h[i] = fma2(decay<T>(d2, A2[i]), h[i], mul2(w2, B[i]));
                    if constexpr (LOCAL) {
                        sum += du;
                    } else {
                        Pair C[4];
                        load_pairs(pB + u * SP + kC, C);
                        const Pair a = fma2(C[1], h[1], mul2(C[0], h[0]));
                        const Pair b = fma2(C[3], h[3], mul2(C[2], h[2]));
                        const float2 f = split(add2(a, b));
                        // Lane i of the SL keeps the steps k SL + i.
                        y[(u % SL) * K + u / SL] = f.x + f.y;
                    }
                }
            };
            if (first)
                run(std::true_type{});
            else
                run(std::false_type{});
            if constexpr (!LOCAL) {
                reduce_scatter<U, SL, 1>(y);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int j = j0 + k * SL + sl;
                    float v = fmaf(skip, x[k], y[k]);
                    if (GATE) v *= silu<T>(widen(px[k * SL * P + kZ]));
                    if (active && j < stop) out[k * out_next] = narrow<T>(v);
                }
            }
        }
        if (t0 + TS < end) land(buf ^ 1);
    }
    if constexpr (LOCAL) {
        store_h(p.span_state + (n * p.spans + at.span) * p.E * p.S);
        if (sl == 0 && active) p.span_sum[(n * p.spans + at.span) * p.E + ch] = sum;
    } else {
        // Steps past the row.
        for (int t = (end > tb ? end : tb) + sl; t < te && active; t += SL)
            *row_ptr<T>(p.out, n, t, ch) = narrow<T>(0.f);
        if (p.final_state && at.span == p.spans - 1) {
            if (len > 0 && step_ended(p.rows, n, len - 1)) clear_h();
            store_h(p.final_state + n * p.E * p.S);
        }
    }
}

}  // namespace seq
}  // namespace rlca

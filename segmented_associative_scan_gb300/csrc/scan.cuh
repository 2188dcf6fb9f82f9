// Selective state space scan: parameters and tile geometry shared by its kernels.
//
//   h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,   y_t = C_t . h_t + D x_t,   out = y silu(z)
//
// A warp owns a block of channels with all their states: a lane holds CPT channels x 4
// states in registers, SL lanes side by side hold the SL * 4 states of the same channels.
// A CTA of 4 warps walks the steps of one row in tiles of kTileSteps. Per tile the raw
// x, dt (z, dout) are read once with wide loads, a thread turning each element into what
// the recurrence needs (the softplus once per element, not once per state), and passed on
// through shared memory; B and C, common to all channels of the group, are staged there
// too. The outputs go back through shared memory to the threads that hold the raw x and z
// and are finished and written with wide stores.
#pragma once

#include "sequence.cuh"

namespace rlca {
namespace seq {

constexpr int kScanWarps = 4;
constexpr int kScanThreads = 32 * kScanWarps;
constexpr int kTileSteps = RLCA_SCAN_CHUNK;

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
    float *part_A;       // [N, E, S] shares of dA
    float *part_D;       // [N, 2, E] shares of dD and ddt_bias
    const uint8_t *reset;
};

// Geometry for SL lanes of states (S <= 4 SL) and CPT channels per lane.
template <int SL_, int CPT_>
struct ScanGeom {
    static constexpr int SL = SL_, CPT = CPT_;
    static constexpr int SP = 4 * SL;          // states, padded
    static constexpr int CG = 32 / SL;         // channel groups of a warp
    static constexpr int WCH = CG * CPT;       // channels per warp
    static constexpr int CH = kScanWarps * WCH;
};

// Lanes that share a channel's states (4 states each, a power of two).
inline int scan_state_lanes(int64_t S)
{
    int sl = 1;
    while (4 * sl < S) sl *= 2;
    return sl;
}

// Channels per lane: 4, fewer where a CTA would pass 128 channels.
constexpr int scan_lane_channels(int sl) { return sl < 4 ? sl : 4; }

// Channels of a CTA.
inline int scan_block_channels(int64_t S)
{
    const int sl = scan_state_lanes(S);
    return kScanWarps * (32 / sl) * scan_lane_channels(sl);
}

// Rows of a [steps, CH] tile of one activation: which elements a thread reads and writes.
// Thread i takes vectors i, i + 128, ...; its channels are the same in each.
template <typename T, int V, int CH>
struct TileIO {
    static constexpr int kVecs = kTileSteps * CH / V;
    static constexpr int kPer = (kVecs + kScanThreads - 1) / kScanThreads;
    static constexpr int kCols = CH / V;
    static_assert(kScanThreads % kCols == 0, "a thread keeps its channels");

    __device__ static int col() { return (threadIdx.x % kCols) * V; }
    __device__ static int step(int k) { return (threadIdx.x + k * kScanThreads) / kCols; }
    __device__ static bool has(int k)
    {
        return kVecs % kScanThreads == 0 || threadIdx.x + k * kScanThreads < kVecs;
    }

    // Elements of steps t0 + step(k) < limit; zeros elsewhere and for inactive columns.
    __device__ static void load(const rlca_steps &a, int64_t n, int64_t c, bool active, int t0,
                                int limit, Pack<T, V> (&r)[kPer])
    {
        const T *base = static_cast<const T *>(a.ptr) + n * a.row + c;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int t = t0 + step(k);
            if (active && has(k) && t < limit)
                r[k] = load_pack<T, V>(base + (int64_t)t * a.step);
            else
                r[k] = zero_pack<T, V>();
        }
    }
};

template <typename T>
__device__ __forceinline__ T *row_ptr(const rlca_steps &a, int64_t n, int64_t t, int64_t c)
{
    return const_cast<T *>(static_cast<const T *>(a.ptr)) + n * a.row + t * a.step + c;
}

// B and C of a tile, fp32, into shared memory (zeros past `limit` and past S).
template <typename T, int SP>
__device__ __forceinline__ void stage_bc(const ScanParams &p, int64_t n, int g, int t0, int limit,
                                         float (&sB)[kTileSteps][SP], float (&sC)[kTileSteps][SP])
{
#pragma unroll 4
    for (int i = threadIdx.x; i < kTileSteps * SP; i += kScanThreads) {
        const int j = i / SP, s = i % SP, t = t0 + j;
        float b = 0.f, c = 0.f;
        if (s < p.S && t < limit) {
            b = widen(*row_ptr<T>(p.B, n, t, (int64_t)g * p.S + s));
            c = widen(*row_ptr<T>(p.C, n, t, (int64_t)g * p.S + s));
        }
        sB[j][s] = b;
        sC[j][s] = c;
    }
}

}  // namespace seq
}  // namespace rlca

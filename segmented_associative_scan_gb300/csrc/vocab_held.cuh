// A few rows of logits, held in registers: by the CTAs of a cluster, each warp a contiguous share of
// the row, so that one row is many SMs' work. A warp's largest logit and sums go to all CTAs of the cluster, which
// join them in one order, and the gradient is formed from the registers, so HBM moves the row
// in and its gradient out and no more. The clusters stay and walk the rows; while one row is
// worked on, every thread's part of the next is on its way to shared memory.
#pragma once

#include <cooperative_groups.h>

#include "vocab_rows.cuh"

namespace rlca {
namespace seq {

constexpr int kHeldMaxWarps = 128;  // of a row
constexpr int kHeldMaxThreads = 1024;

// On its way to shared memory: whole packs by asynchronous copies, which the thread that asked
// for them reads back; the elements of the row's first and last pack, where they are cut, in a
// register each.
template <typename T, int U>
struct Coming {
    static constexpr int W = 16 / (int)sizeof(T);
    T cut;

    // `slots`: this lane's of the warp's [U][32].
    __device__ __forceinline__ void ask(const Share<T, U> &a, uint4 *slots)
    {
        const int lane = threadIdx.x & 31;
        const T *from = a.z + a.first(lane);
        if (a.full) {
#pragma unroll
            for (int u = 0; u < U; ++u) copy_async(slots + u * 32, from + u * 32 * W);
        } else {
            const int w0 = a.w0(), w1 = a.w1();
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (u * 32 + lane >= w0 && u * 32 + lane < w1)
                    copy_async(slots + u * 32, from + u * 32 * W);
            // Lanes 0..15: an element of the share's first pack; 16..31 of its last.
            const int n = a.n(), k = lane < 16 ? 0 : n - 1, j = a.first(k) + (lane & 15);
            cut = narrow<T>(-INFINITY);
            if (n > 0 && (lane & 15) < W && !a.whole(k) && j >= 0 && j < a.V) cut = a.z[j];
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // What was asked for, as this lane's packs; -inf where there is nothing. `edge`: an element of
    // the share's first or last pack, by lane as above.
    __device__ __forceinline__ void get(const Share<T, U> &a, uint4 *slots, Pack<T, W> (&v)[U], T &edge)
    {
        const int lane = threadIdx.x & 31;
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        T *ends = reinterpret_cast<T *>(slots - lane) + (lane & (W - 1));
        if (a.full) {
            edge = lane < 16 ? ends[0] : ends[(32 * U - 1) * W];
#pragma unroll
            for (int u = 0; u < U; ++u) *reinterpret_cast<uint4 *>(&v[u]) = slots[u * 32];
        } else {
            const int n = a.n(), k = lane < 16 || n == 0 ? 0 : n - 1;
            if (n > 0 && (lane & 15) < W && !a.whole(k)) ends[k * W] = cut;
            __syncwarp();
            edge = ends[k * W];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                uint4 x = slots[u * 32];
                if (u * 32 + lane >= n) {
                    const T none[2] = {narrow<T>(-INFINITY), narrow<T>(-INFINITY)};
                    x.x = x.y = x.z = x.w = *reinterpret_cast<const uint32_t *>(none);
                }
                *reinterpret_cast<uint4 *>(&v[u]) = x;
            }
        }
        __syncwarp();
    }
};

struct HeldShared {
    RowStats parts[2][kHeldMaxWarps];
    RowsAhead ahead[2];
    RowSlope slope;
    float m, sum;
};

// 64 registers: 32 warps to an SM, in CTAs of as many as a row fills (clusters where those are more).
template <typename T, VocabOp OP, bool ENT, bool GRAD, int U>
__global__ void __launch_bounds__(kHeldMaxThreads, 1) vocab_held_kernel(const VocabParams p, int ctas)
{
    constexpr bool TEACH = OP == VocabOp::kDistill;
    namespace cg = cooperative_groups;
    extern __shared__ uint4 stage[];  // [warp][U][32]
    __shared__ HeldShared sh;
    __shared__ typename std::conditional<TEACH, TeacherParts, int>::type teach;
    grid_dependency_sync();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = ctas > 1 ? (int)(blockIdx.x % ctas) : 0, warps = ctas * (blockDim.x / 32);
    const int row_warp = rank * (blockDim.x / 32) + warp;
    const int step = (int)gridDim.x / ctas, first = (int)blockIdx.x / ctas, rows = (int)p.M;
    const int wide = rank * blockDim.x + tid;  // of the cluster's threads
    const int V = (int)p.V;
    uint4 *slots = stage + warp * (32 * U) + lane;

    // All CTAs of the cluster run before one writes to another.
    if (ctas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    if (warp == 0) look_ahead<T, OP, true>(p, sh.ahead[0], first, step);
    if (ctas > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    __syncthreads();

    Coming<T, U> coming;
    Entry next = {-1, -INFINITY};
    auto ask = [&](const RowsAhead &from, int k, unsigned i) {
        coming.ask(Share<T, U>(static_cast<const T *>(from.row[k]), V, row_warp), slots);
        if constexpr (TEACH) next = teacher_entry<T>(p, step_at(p, i), tid);
    };
    if (first < rows && sh.ahead[0].token[0] >= 0) ask(sh.ahead[0], 0, first);
    int par = 0;
    unsigned k = 0;  // rows walked, modulo 2 kAhead
    for (unsigned i = first; i < (unsigned)rows; i += step, k = (k + 1) % (2 * kAhead)) {
        const unsigned at_k = k % kAhead, k1 = (k + 1) % (2 * kAhead);
        const RowsAhead &now = sh.ahead[k / kAhead];
        if (at_k == kAhead * 3 / 4) {
            __syncthreads();  // nobody reads the rows before these any more
            if (warp == 0)
                look_ahead<T, OP, true>(p, sh.ahead[k / kAhead ^ 1],
                                  i + (int64_t)(kAhead - at_k) * step, step);
        }
        if (at_k == kAhead - 1) __syncthreads();
        T *g = GRAD ? static_cast<T *>(now.grad[at_k]) : nullptr;
        const RowsAhead &then = sh.ahead[k1 / kAhead];
        const bool more = (int64_t)i + step < rows && then.token[k1 % kAhead] >= 0;
        const int32_t token = now.token[at_k];
        if (token < 0) {
            if (wide == 0) write_uncounted(p, i);
            if (GRAD) clear_row(g, 0, p.V, wide, ctas * blockDim.x);
            if (more) ask(then, k1 % kAhead, i + step);
            continue;
        }
        const Share<T, U> a(static_cast<const T *>(now.row[at_k]), V, row_warp);
        Held<T, U> held;
        T edge;
        coming.get(a, slots, held.v, edge);
        const float top = held.largest();
        const Entry entry = next;
        float z_entry = 0.f;
        if constexpr (TEACH) {
            if (entry.token >= 0) z_entry = widen(a.z[entry.token]);
        }
        // The slots are read (their largest value is known): the next row may come.
        if (more) ask(then, k1 % kAhead, i + step);
        const RowStats own = held.template stats<ENT>(top, a.full, a.full ? 32 * U : a.n(), p.scale);
        if constexpr (TEACH) teacher_send(p, teach, par, entry);
        RowStats *parts = sh.parts[par];
        if (ctas > 1) {
            if (lane < (GRAD || TEACH ? ctas : 1))
                cg::this_cluster().map_shared_rank(parts, lane)[row_warp] = own;
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        } else {
            if (lane == 0) parts[warp] = own;
            __syncthreads();
        }
        const int tpar = par;
        par ^= 1;
        if (!GRAD && !TEACH && rank) continue;

        const RowInputs &in = now.in[at_k];
        if (warp == 0) {
            const RowStats st = join_parts<T, ENT>(parts, warps, p.scale);
            RowSlope r = {0.f, 0.f, 0.f, true};
            if constexpr (TEACH) {
                const float sum = unbiased<T>(st).s;
                r = teacher_slope(p, teach, tpar, st.m, sum, in.weight);
                if (lane == 0) sh.sum = sum;
            } else if (st.m != -INFINITY) {
                r = finish_row<T, OP, ENT>(p, i, now.z[at_k], st, in, rank == 0 && lane == 0);
            } else if (wide == 0) {
                write_uncounted(p, i);
            }
            if ((GRAD || TEACH) && lane == 0) {
                sh.slope = r;
                sh.m = st.m;
            }
        }
        if (!GRAD && !TEACH) continue;
        __syncthreads();
        const RowSlope r = sh.slope;
        const float m = sh.m;
        if (GRAD) {
            if (r.zero) clear_row(g, 0, p.V, wide, ctas * blockDim.x);
            else held.template store<ENT>(a, g, r, m, edge, p.scale);
        }
        if constexpr (TEACH) {
            teacher_share(p, teach, tpar, entry, z_entry, m, sh.sum);
            __syncthreads();
            if (wide == 0) p.loss[i] = teacher_loss(p, teach, tpar);
            if (GRAD && !r.zero && entry.token >= 0) {
                const int pack = (entry.token + a.head) / (16 / (int)sizeof(T)), mine = blockDim.x * U;
                if (pack >= rank * mine && pack < (rank + 1) * mine)
                    g[entry.token] =
                        teacher_gradient<T>(p, teach, tpar, entry, z_entry, r, m, in.weight);
            }
        } else if (GRAD && !r.zero) {
            const int pack = (token + a.head) / (16 / (int)sizeof(T));
            if (pack >= a.k0 && pack < a.k0 + 32 * U && lane == 0)
                g[token] = narrow<T>(slope_at<T, ENT>(now.z[at_k], r, m, p.scale) + r.gamma);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace seq
}  // namespace rlca

// A few rows of logits, held in registers by the CTAs of a cluster, each warp a contiguous share of its
// row, so that one row is the work of many SMs. A warp's largest logit and sums go to all CTAs of the
// cluster, which join them in one order, and the gradient is formed from the registers. What bounds
// such calls is how long the parts wait for one another: 16 rows of 32768 in bf16 take 2.9 us, with the
// policy loss and its gradient 4.4 (an empty kernel 2.3).
#pragma once

#include <cooperative_groups.h>

#include "vocab_rows.cuh"

namespace rlca {
namespace seq {

constexpr int kHeldMaxWarps = 128;  // of a row

struct HeldShared {
    RowStats parts[kHeldMaxWarps];
    RowSlope slope;
    float m, sum;
};

// Cluster i has row i, every warp 32 U packs of it.
template <typename T, VocabOp OP, bool ENT, bool GRAD, int U>
__global__ void __launch_bounds__(512) vocab_held_kernel(const VocabParams p, int ctas)
{
    constexpr bool TEACH = OP == VocabOp::kDistill;
    constexpr int W = 16 / (int)sizeof(T);
    namespace cg = cooperative_groups;
    __shared__ HeldShared sh;
    __shared__ typename std::conditional<TEACH, TeacherParts, int>::type teach;
    grid_dependency_sync();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = ctas * (blockDim.x / 32);
    const int i = (int)blockIdx.x / ctas, rank = (int)blockIdx.x % ctas;
    const int row_warp = rank * (blockDim.x / 32) + warp;
    const int wide = rank * blockDim.x + tid;  // of the cluster's threads
    const StepAt s = step_at(p, i);
    const Share<T, U> a(row_of<T>(p.logits, s.n, s.t), (int)p.V, row_warp);
    T *g = GRAD ? out_row<T>(p.grad, s.n, s.t) : nullptr;

    // Every thread looks up the row for itself, and before it, if it has to be read.
    bool counted = inside_row(p, s.n, s.t);
    int token = -1;
    if (!TEACH && counted) {
        const int64_t j = vocab_token(p, s.n, s.t);
        counted = j >= 0 && j < p.V;
        token = (int)j;
    }
    if (!counted) {  // all CTAs of the cluster alike
        if (wide == 0) write_uncounted(p, i);
        if (GRAD) clear_row(g, 0, p.V, wide, ctas * blockDim.x);
        return;
    }
    // All CTAs of the cluster run before one writes to another.
    if (ctas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    Held<T, U> held;
    held.load(a);
    Entry entry = {-1, -INFINITY};
    if constexpr (TEACH) {
        entry = teacher_entry<T>(p, s, tid);
        token = entry.token;
    }
    const float z_a = token >= 0 ? widen(a.z[token]) : 0.f;
    const RowInputs in = row_inputs<OP>(p, s.n, s.t);
    const RowStats own = held.template stats<ENT>(held.largest(), p.scale);
    if constexpr (TEACH) teacher_send(p, teach, 0, entry);
    if (ctas > 1) {
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        if (lane < (GRAD || TEACH ? ctas : 1))
            cg::this_cluster().map_shared_rank(sh.parts, lane)[row_warp] = own;
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
        if (lane == 0) sh.parts[warp] = own;
        __syncthreads();
    }
    if (!GRAD && !TEACH && rank) return;

    if (warp == 0) {
        const RowStats st = join_parts<ENT>(sh.parts, warps, p.scale);
        RowSlope r = {0.f, 0.f, 0.f, true};
        if constexpr (TEACH) {
            const float sum = unbiased(st).s;
            r = teacher_slope(p, teach, 0, st.m, sum, in.weight);
            if (lane == 0) sh.sum = sum;
        } else if (st.m != -INFINITY) {
            r = finish_row<T, OP, ENT>(p, i, z_a, st, in, wide == 0);
        } else if (wide == 0) {
            write_uncounted(p, i);
        }
        if ((GRAD || TEACH) && lane == 0) {
            sh.slope = r;
            sh.m = st.m;
        }
    }
    if (!GRAD && !TEACH) return;
    __syncthreads();
    const RowSlope r = sh.slope;
    const float m = sh.m;
    if (GRAD) {
        if (r.zero) clear_row(g, 0, p.V, wide, ctas * blockDim.x);
        else held.template store<ENT>(a, g, r, m, p.scale);
    }
    const int pack = (token + a.head) / W;
    if constexpr (TEACH) {
        teacher_share(p, teach, 0, entry, z_a, m, sh.sum);
        __syncthreads();
        if (wide == 0) p.loss[i] = teacher_loss(p, teach, 0);
        // Of this CTA's elements.
        const int mine = blockDim.x * U;
        if (GRAD && !r.zero && token >= 0 && pack >= rank * mine && pack < (rank + 1) * mine)
            g[token] = teacher_gradient<T>(p, teach, 0, entry, z_a, r, m, in.weight);
    } else if (GRAD && !r.zero && lane == 0 && pack >= a.k0 && pack < a.k0 + 32 * U) {
        g[token] = narrow<T>(slope_at<T, ENT>(z_a, r, m, p.scale) + r.gamma);
    }
}

}  // namespace seq
}  // namespace rlca

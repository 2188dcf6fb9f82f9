// Rows of logits that are read once and held in registers: by the CTAs of a cluster, each warp a
// contiguous share of the row. A warp's largest logit and sums go to all CTAs of the cluster, which
// join them in one order, and the gradient is formed from the registers, so HBM moves the row
// in and its gradient out and no more. The clusters stay and walk the rows; while one row is
// worked on, every thread's part of the next is on its way to shared memory.
#pragma once

#include <cooperative_groups.h>

#include "vocab.cuh"

namespace rlca {
namespace seq {

constexpr int kHeldMaxWarps = 128;  // of a row
constexpr int kHeldMaxThreads = 1024;

// ------------------------------------------------------------------------- cut packs

template <typename T>
__device__ __forceinline__ T shift_out(uint4 &r)
{
    T x;
    if constexpr (sizeof(T) == 4) {
        x = __uint_as_float(r.x);
        r = make_uint4(r.y, r.z, r.w, 0);
    } else {
        const uint16_t b = (uint16_t)r.x;
        x = *reinterpret_cast<const T *>(&b);
        r = make_uint4(__funnelshift_r(r.x, r.y, 16), __funnelshift_r(r.y, r.z, 16),
                       __funnelshift_r(r.z, r.w, 16), r.w >> 16);
    }
    return x;
}

// Elements lo <= e < hi of a pack whose first is j, those inside the row. (A loop that is not
// unrolled: a row has few such packs.)
template <typename T>
__device__ __noinline__ void store_cut(T *g, int64_t j, int64_t V, uint4 r, int lo, int hi)
{
#pragma unroll 1
    for (int e = 0; e < hi; ++e) {
        const T x = shift_out<T>(r);
        if (e >= lo && j + e >= 0 && j + e < V) g[j + e] = x;
    }
}

__device__ __forceinline__ void copy_async(void *to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 :
                 : "r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from)
                 : "memory");
}
// 16 bytes from byte `off` of a and b, one after the other (off < 16, a multiple of 2; the same
// in all lanes).
__device__ __forceinline__ uint4 bytes_from(uint4 a, uint4 b, int off)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (off & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (off & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const int bits = (off & 2) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// ------------------------------------------------------------------------- a warp's share

// A warp's packs of a row: k0 .. k0 + n - 1, 32 U of them but at the row's end; lane l has packs
// k0 + l, k0 + l + 32, ... Of those w0 .. w1 - 1 are whole; the others, the row's first and last
// where they are cut, are read and written element by element. `full`: 32 U, all of them whole.
template <typename T, int U>
struct Share {
    static constexpr int W = 16 / (int)sizeof(T);
    const T *z;
    int V, head, k0;
    bool full;

    __device__ __forceinline__ Share(const T *z_, int V_, int warp)
        : z(z_), V(V_), head((int)((reinterpret_cast<uintptr_t>(z_) % 16) / sizeof(T))),
          k0(warp * (32 * U))
    {
        full = first(32 * U) <= V && (k0 > 0 || head == 0);
    }
    __device__ __forceinline__ int n() const
    {
        return max(0, min(32 * U, (V + head + W - 1) / W - k0));
    }
    __device__ __forceinline__ int w0() const { return k0 == 0 && head != 0 ? 1 : 0; }
    __device__ __forceinline__ int w1() const { return min(32 * U, (V + head) / W - k0); }
    __device__ __forceinline__ int first(int i) const { return (k0 + i) * W - head; }
    __device__ __forceinline__ bool whole(int i) const { return i >= w0() && i < w1(); }
    __device__ __forceinline__ bool cut() const { return n() > 0 && (w0() != 0 || w1() != n()); }
};

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

template <typename T, int U>
struct Held {
    static constexpr int W = 16 / (int)sizeof(T);
    Pack<T, W> v[U];

    __device__ __forceinline__ float largest() const
    {
        MaxOf<T> top;
#pragma unroll
        for (int u = 0; u < U; ++u) top.add(v[u]);
        float m = top.get();
#pragma unroll
        for (int w = 16; w >= 1; w /= 2) m = max_nan(m, __shfl_xor_sync(kFullMask, m, w));
        return m;
    }

    // (m, S, h) of the share with the largest element m, in all lanes.
    template <bool ENT>
    __device__ __forceinline__ RowStats stats(float m, bool full, int n, ExpScale c) const
    {
        const float ref = m == -INFINITY ? 0.f : m;
        const T low = lowest_logit<T>(ref, c);
        RowSums a[2] = {{pair(0.f, 0.f), pair(0.f, 0.f)}, {pair(0.f, 0.f), pair(0.f, 0.f)}};
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (full || u * 32 < n) add_pack<T, ENT>(a[u & 1], v[u], ref, low, c);
        const Pair s2 = add2(a[0].s, a[1].s), h2 = add2(a[0].h, a[1].h);
        float s = s2.x + s2.y, h = flat_row(low) ? 0.f : h2.x + h2.y;
#pragma unroll
        for (int w = 16; w >= 1; w /= 2) {
            s += __shfl_xor_sync(kFullMask, s, w);
            if (ENT) h += __shfl_xor_sync(kFullMask, h, w);
        }
        return {m, s, h};
    }

    // The gradient of the share's elements.
    template <bool ENT>
    __device__ __forceinline__ void store(const Share<T, U> &a, T *g, const RowSlope &r, float m, T edge,
                                          ExpScale c) const
    {
        const T low = lowest_logit<T>(m, c);
        const int head = (int)((reinterpret_cast<uintptr_t>(g) % 16) / sizeof(T));
        const int s = (a.head - head + W) % W;
        if (ENT && flat_row(low)) {
            careful<false>(a, g, s, r, m, low, c);
        } else if (s == 0) {
            aligned<ENT>(a, g, r, m, low, c);
            if (!a.full) {
                const int lane = threadIdx.x & 31, n = a.n(), k = lane < 16 ? 0 : n - 1;
                if (n > 0 && !a.whole(k)) edges<ENT>(a, g, k, 0, W, r, m, edge, c);
            }
        } else if (!a.full) {
            careful<ENT>(a, g, s, r, m, low, c);
        } else {
            shifted<ENT>(a, g, s, r, m, low, c);
            const bool first = (threadIdx.x & 31) < 16;
            edges<ENT>(a, g, first ? 0 : 32 * U - 1, first ? 0 : s, first ? s : W, r, m, edge, c);
        }
        __syncwarp();
    }

private:
    // Elements lo <= e < hi of pack k: the share's first for lanes 0..15, its last for 16..31.
    template <bool ENT>
    __device__ __forceinline__ void edges(const Share<T, U> &a, T *g, int k, int lo, int hi,
                                          const RowSlope &r, float m, T edge, ExpScale c) const
    {
        const int e = threadIdx.x & 15, j = a.first(k) + e;
        if (e >= lo && e < hi && j >= 0 && j < a.V)
            g[j] = narrow<T>(slope_at<T, ENT>(widen(edge), r, m, c));
    }
    template <bool ENT>
    __device__ __forceinline__ void aligned(const Share<T, U> &a, T *g, const RowSlope &r, float m,
                                            T low, ExpScale c) const
    {
        const int lane = threadIdx.x & 31;
        T *to = g + a.first(lane);
        const int w0 = a.full ? 0 : a.w0() - lane, w1 = a.full ? 32 * U : a.w1() - lane;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Pack<T, W> o = pack_slope<T, ENT>(v[u], r, m, low, c);
            if (u * 32 >= w0 && u * 32 < w1)
                *reinterpret_cast<uint4 *>(to + u * 32 * W) = *reinterpret_cast<const uint4 *>(&o);
        }
    }
    // The gradient's row lies at another offset to 16 bytes than the logits': its packs, which
    // begin s elements later, are put together from a lane's own and the next lane's. (A full
    // share.)
    template <bool ENT>
    __device__ __forceinline__ void shifted(const Share<T, U> &a, T *g, int s, const RowSlope &r, float m,
                                            T low, ExpScale c) const
    {
        const int lane = threadIdx.x & 31;
        T *to = g + a.first(lane) + s;
        Pack<T, W> cur = pack_slope<T, ENT>(v[0], r, m, low, c);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Pack<T, W> next =
                u + 1 < U ? pack_slope<T, ENT>(v[u + 1 < U ? u + 1 : u], r, m, low, c) : cur;
            const uint4 o = joined(cur, next, s);
            if (u + 1 < U || lane < 31) *reinterpret_cast<uint4 *>(to + u * 32 * W) = o;
            cur = next;
        }
    }
    // Elements s.. of this lane's pack of `cur` and ..s of the next lane's (of lane 0's of `next`).
    static __device__ __forceinline__ uint4 joined(const Pack<T, W> &cur, const Pack<T, W> &next, int s)
    {
        const int lane = threadIdx.x & 31;
        const uint4 x = *reinterpret_cast<const uint4 *>(lane == 0 ? &next : &cur);
        uint4 y;
        y.x = __shfl_sync(kFullMask, x.x, lane + 1);
        y.y = __shfl_sync(kFullMask, x.y, lane + 1);
        y.z = __shfl_sync(kFullMask, x.z, lane + 1);
        y.w = __shfl_sync(kFullMask, x.w, lane + 1);
        return bytes_from(*reinterpret_cast<const uint4 *>(&cur), y, s * (int)sizeof(T));
    }
    // The same with cut packs and shares that are not full, and for s = 0.
    template <bool ENT>
    __device__ __forceinline__ void careful(const Share<T, U> &a, T *g, int s, const RowSlope &r, float m,
                                            T low, ExpScale c) const
    {
        const int lane = threadIdx.x & 31, n = a.n();
        Pack<T, W> cur = pack_slope<T, ENT>(v[0], r, m, low, c);
        if (lane == 0 && n > 0)
            store_cut<T>(g, a.first(0), a.V, *reinterpret_cast<const uint4 *>(&cur), 0, s);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u * 32 >= n) break;
            Pack<T, W> next = cur;
            if (u + 1 < U && (u + 1) * 32 < n)
                next = pack_slope<T, ENT>(v[u + 1 < U ? u + 1 : u], r, m, low, c);
            const uint4 o = joined(cur, next, s);
            const int i = u * 32 + lane, j = a.first(i) + s;
            if (i + 1 < n && j >= 0 && j <= a.V - W)
                *reinterpret_cast<uint4 *>(g + j) = o;
            else if (i < n)
                store_cut<T>(g, j, a.V, o, 0, i + 1 < n ? W : W - s);
            cur = next;
        }
    }
};

// ------------------------------------------------------------------------- rows in clusters

// What is known of the rows that a cluster walks next, looked up 32 at a time.
constexpr int kAhead = 32;
struct RowsAhead {
    const void *row[kAhead];
    void *grad[kAhead];
    int32_t token[kAhead];  // -1: does not count
    float z[kAhead];        // its logit, if asked for
    RowInputs in[kAhead];
};

struct HeldShared {
    RowStats parts[2][kHeldMaxWarps];
    RowsAhead ahead[2];
    RowSlope slope;
    float m, sum;
};

// A teacher's entries are the first warps' own, one to a thread.
constexpr int kTeachWarps = RLCA_DISTILL_MAX_K / 32;

__host__ __device__ __forceinline__ int teach_warps(int K) { return K > 32 ? (K + 31) / 32 : 1; }

// Of this row and the one before.
struct TeacherParts {
    int32_t index[2][RLCA_DISTILL_MAX_K];  // -1: left out
    float q[2][RLCA_DISTILL_MAX_K];
    float2 parts[2][kTeachWarps];  // largest logit, sum of a warp's entries
    float loss[2][kTeachWarps];
};

struct StepAt {
    int n, t;

    __device__ __forceinline__ StepAt after(const StepAt &by, int T) const
    {
        StepAt r = {n + by.n, t + by.t};
        if (r.t >= T) {
            r.t -= T;
            ++r.n;
        }
        return r;
    }
};

__device__ __forceinline__ StepAt step_at(const VocabParams &p, int i)
{
    const unsigned n = (unsigned)i / (unsigned)p.T;
    return {(int)n, (int)((unsigned)i - n * (unsigned)p.T)};
}

// Lane l looks up row i0 + l step.
template <typename T, VocabOp OP, bool LOGIT>
__device__ __forceinline__ void look_ahead(const VocabParams &p, RowsAhead &a, int64_t i0, int step)
{
    const int lane = threadIdx.x & 31;
    const int64_t i = i0 + (int64_t)lane * step;
    int32_t token = -1;
    if (i < p.M) {
        const StepAt s = step_at(p, (int)i);
        a.row[lane] = row_of<T>(p.logits, s.n, s.t);
        if (p.grad.ptr) a.grad[lane] = out_row<T>(p.grad, s.n, s.t);
        if (inside_row(p, s.n, s.t)) {
            int64_t j = 0;
            if (OP != VocabOp::kDistill) j = vocab_token(p, s.n, s.t);
            if (j >= 0 && j < p.V) {
                token = (int32_t)j;
                if (LOGIT && OP != VocabOp::kDistill) a.z[lane] = widen(row_of<T>(p.logits, s.n, s.t)[j]);
                a.in[lane] = row_inputs<OP>(p, s.n, s.t);
            }
        }
    }
    a.token[lane] = token;
}

// A thread's entry of a teacher's row: its token (-1: left out) and logit.
struct Entry {
    int32_t token;
    float logit;
};

template <typename T>
__device__ __forceinline__ Entry teacher_entry(const VocabParams &p, const StepAt &s, int k)
{
    Entry e = {-1, -INFINITY};
    if (k >= p.K) return e;
    const int64_t at_k = s.n * p.index.row + s.t * p.index.step + k;
    const int64_t j = p.index_bytes == 8
                          ? (int64_t)__ldg(static_cast<const long long *>(p.index.ptr) + at_k)
                          : (int64_t)__ldg(static_cast<const int *>(p.index.ptr) + at_k);
    const float x = p.teacher_fp32 ? __ldg(row_of<float>(p.teacher, s.n, s.t) + k)
                                   : widen(row_of<T>(p.teacher, s.n, s.t)[k]);
    if (j < 0 || j >= p.V || x == -INFINITY) return e;
    return {(int32_t)j, x};
}

// What a distilled row takes between its passes, in the order of the CTA's barriers: the entries'
// softmax by warps; after the first barrier its slope (one warp); after the gradient every entry's q
// and share of the loss, off the way; after the last barrier the loss, and the gradient where the
// entries are.
__device__ __forceinline__ void teacher_send(const VocabParams &p, TeacherParts &t, int par,
                                             const Entry &entry)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp >= teach_warps(p.K)) return;
    float m = entry.logit;
#pragma unroll
    for (int w = 16; w >= 1; w /= 2) m = max_nan(m, __shfl_xor_sync(kFullMask, m, w));
    float x = entry.token >= 0 ? expf((entry.logit - m) * p.inv_tau) : 0.f;
#pragma unroll
    for (int w = 16; w >= 1; w /= 2) x += __shfl_xor_sync(kFullMask, x, w);
    if (lane == 0) t.parts[par][warp] = make_float2(m, x);
    t.index[par][threadIdx.x] = entry.token;
}

__device__ __forceinline__ float teacher_top(const VocabParams &p, const TeacherParts &t, int par)
{
    float top = -INFINITY;
    for (int w = 0; w < teach_warps(p.K); ++w) top = max_nan(top, t.parts[par][w].x);
    return top;
}

__device__ __forceinline__ RowSlope teacher_slope(const VocabParams &p, const TeacherParts &t, int par,
                                                  float m, float sum, float weight)
{
    const bool counted = teacher_top(p, t, par) != -INFINITY && m != -INFINITY;
    return {0.f, weight * p.inv_tau / sum, 0.f, weight == 0.f || !counted};
}

__device__ __forceinline__ void teacher_share(const VocabParams &p, TeacherParts &t, int par,
                                              const Entry &entry, float z, float m, float sum)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp >= teach_warps(p.K)) return;
    const float top = teacher_top(p, t, par);
    float total = 0.f;
    for (int w = 0; w < teach_warps(p.K); ++w) {
        const float2 x = t.parts[par][w];
        if (x.x != -INFINITY) total += x.y * expf((x.x - top) * p.inv_tau);
    }
    const float v = (entry.logit - top) * p.inv_tau;
    const float q = entry.token >= 0 ? expf(v) / total : 0.f;
    float part = 0.f;
    if (m != -INFINITY && (q > 0.f || isnan(q)))
        part = -q * log_prob(z, m, logf(sum), p.inv_tau, p.inv_tau_lo).minus(v - logf(total));
#pragma unroll
    for (int w = 16; w >= 1; w /= 2) part += __shfl_xor_sync(kFullMask, part, w);
    if (lane == 0) t.loss[par][warp] = part;
    t.q[par][threadIdx.x] = q;
}

__device__ __forceinline__ float teacher_loss(const VocabParams &p, const TeacherParts &t, int par)
{
    float loss = 0.f;
    for (int w = 0; w < teach_warps(p.K); ++w) loss += t.loss[par][w];
    return loss;
}

// The gradient at an entry's token, where more entries may have the same.
template <typename T>
__device__ __forceinline__ T teacher_gradient(const VocabParams &p, const TeacherParts &t, int par,
                                              const Entry &entry, float z, const RowSlope &r, float m,
                                              float weight)
{
    float both = 0.f;
    for (int j = 0; j < p.K; ++j)
        if (t.index[par][j] == entry.token) both += t.q[par][j];
    return narrow<T>(fmaf(-both, weight * p.inv_tau, slope_at<T, false>(z, r, m, p.scale)));
}

// Joins parts[0 .. n) in a warp, in one order, in all lanes.
template <typename T, bool ENT>
__device__ __forceinline__ RowStats join_parts(const RowStats *parts, int n, ExpScale c)
{
    const int lane = threadIdx.x & 31;
    float m = -INFINITY;
    for (int w = lane; w < n; w += 32) m = max_nan(m, parts[w].m);
#pragma unroll
    for (int w = 16; w >= 1; w /= 2) m = max_nan(m, __shfl_xor_sync(kFullMask, m, w));
    float s = 0.f, h = 0.f;
    for (int w = lane; w < n; w += 32) {
        RowStats a = parts[w];
        rebase<T, ENT>(a, m, c);
        s += a.s;
        h += a.h;
    }
#pragma unroll
    for (int w = 16; w >= 1; w /= 2) {
        s += __shfl_xor_sync(kFullMask, s, w);
        if (ENT) h += __shfl_xor_sync(kFullMask, h, w);
    }
    return {m, s, h};
}

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
            if (GRAD) clear_row(RowPacks<T>(g, p.V), g, wide, ctas * blockDim.x);
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
            if (r.zero) clear_row(RowPacks<T>(g, p.V), g, wide, ctas * blockDim.x);
            else held.template store<ENT>(a, g, r, m, edge, p.scale);
        }
        if constexpr (TEACH) {
            teacher_share(p, teach, tpar, entry, z_entry, m, sh.sum);
            __syncthreads();
            if (wide == 0) p.loss[i] = teacher_loss(p, teach, tpar);
            if (GRAD && !r.zero && entry.token >= 0) {
                const int pack = (entry.token + a.head) / RowPacks<T>::W, mine = blockDim.x * U;
                if (pack >= rank * mine && pack < (rank + 1) * mine)
                    g[entry.token] =
                        teacher_gradient<T>(p, teach, tpar, entry, z_entry, r, m, in.weight);
            }
        } else if (GRAD && !r.zero) {
            const int pack = (token + a.head) / RowPacks<T>::W;
            if (pack >= a.k0 && pack < a.k0 + 32 * U && lane == 0)
                g[token] = narrow<T>(slope_at<T, ENT>(now.z[at_k], r, m, p.scale) + r.gamma);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace seq
}  // namespace rlca

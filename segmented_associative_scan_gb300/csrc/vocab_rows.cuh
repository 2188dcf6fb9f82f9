// What the kernels over whole rows of logits share: packs that are cut at a row's ends, a warp's
// share of a row and its gradient, the rows that a CTA walks next, and a teacher's entries.
#pragma once

#include "vocab.cuh"

namespace rlca {
namespace seq {

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

// 16 bytes from byte `off` of a and b, one after the other (off < 16, a multiple of 2).
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
};

// Packs of a share in registers.
template <typename T, int U>
struct Held {
    static constexpr int W = 16 / (int)sizeof(T);
    Pack<T, W> v[U];
    T edge;  // an element of the share's first pack (lanes 0..15) or last (16..31)

    // -inf where there is nothing.
    __device__ __forceinline__ void load(const Share<T, U> &a)
    {
        const int lane = threadIdx.x & 31;
        const T *from = a.z + a.first(lane);
        edge = narrow<T>(-INFINITY);
        if (a.full) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                *reinterpret_cast<uint4 *>(&v[u]) =
                    *reinterpret_cast<const uint4 *>(from + u * 32 * W);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = a.first(u * 32 + lane);
#pragma unroll
                for (int e = 0; e < W; ++e) v[u].e[e] = narrow<T>(-INFINITY);
                if (a.whole(u * 32 + lane)) {
                    *reinterpret_cast<uint4 *>(&v[u]) =
                        *reinterpret_cast<const uint4 *>(from + u * 32 * W);
                } else if (u * 32 + lane < a.n()) {
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (j + e >= 0 && j + e < a.V) v[u].e[e] = a.z[j + e];
                }
            }
        }
        const int n = a.n(), j = a.first(lane < 16 ? 0 : n - 1) + (lane & 15);
        if (n > 0 && (lane & 15) < W && j >= 0 && j < a.V) edge = a.z[j];
    }

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
    __device__ __forceinline__ RowStats stats(float m, ExpScale c) const
    {
        const float ref = m == -INFINITY ? 0.f : m;
        const T low = lowest_logit<T>(ref, c);
        RowSums a[2] = {{pair(0.f, 0.f), pair(0.f, 0.f)}, {pair(0.f, 0.f), pair(0.f, 0.f)}};
        if (ENT && cut_late(low)) {
#pragma unroll
            for (int u = 0; u < U; ++u) add_pack<T, ENT, true>(a[u & 1], v[u], ref, low, c);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) add_pack<T, ENT, false>(a[u & 1], v[u], ref, low, c);
        }
        const Pair s2 = add2(a[0].s, a[1].s), h2 = add2(a[0].h, a[1].h);
        float s = s2.x + s2.y, h = h2.x + h2.y;
#pragma unroll
        for (int w = 16; w >= 1; w /= 2) {
            s += __shfl_xor_sync(kFullMask, s, w);
            if (ENT) h += __shfl_xor_sync(kFullMask, h, w);
        }
        return {m, s, h};
    }

    // The gradient of the share's elements.
    template <bool ENT>
    __device__ __forceinline__ void store(const Share<T, U> &a, T *g, const RowSlope &r, float m,
                                          ExpScale c) const
    {
        const T low = lowest_logit<T>(m, c);
        const int head = (int)((reinterpret_cast<uintptr_t>(g) % 16) / sizeof(T));
        const int s = (a.head - head + W) % W;
        if (ENT && cut_late(low)) {
            careful<ENT, true>(a, g, s, r, m, low, c);
        } else if (s == 0) {
            aligned<ENT>(a, g, r, m, low, c);
            if (!a.full) {
                const int lane = threadIdx.x & 31, n = a.n(), k = lane < 16 ? 0 : n - 1;
                if (n > 0 && !a.whole(k)) edges<ENT>(a, g, k, 0, W, r, m, c);
            }
        } else if (!a.full) {
            careful<ENT, false>(a, g, s, r, m, low, c);
        } else {
            shifted<ENT>(a, g, s, r, m, low, c);
            const bool first = (threadIdx.x & 31) < 16;
            edges<ENT>(a, g, first ? 0 : 32 * U - 1, first ? 0 : s, first ? s : W, r, m, c);
        }
        __syncwarp();
    }

private:
    // Elements lo <= e < hi of pack k: the share's first for lanes 0..15, its last for 16..31.
    template <bool ENT>
    __device__ __forceinline__ void edges(const Share<T, U> &a, T *g, int k, int lo, int hi,
                                          const RowSlope &r, float m, ExpScale c) const
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
    template <bool ENT, bool LATE>
    __device__ __forceinline__ void careful(const Share<T, U> &a, T *g, int s, const RowSlope &r, float m,
                                            T low, ExpScale c) const
    {
        const int lane = threadIdx.x & 31, n = a.n();
        Pack<T, W> cur = pack_slope<T, ENT, LATE>(v[0], r, m, low, c);
        if (lane == 0 && n > 0)
            store_cut<T>(g, a.first(0), a.V, *reinterpret_cast<const uint4 *>(&cur), 0, s);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u * 32 >= n) break;
            Pack<T, W> next = cur;
            if (u + 1 < U && (u + 1) * 32 < n)
                next = pack_slope<T, ENT, LATE>(v[u + 1 < U ? u + 1 : u], r, m, low, c);
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

// ------------------------------------------------------------------------- rows to walk

// What is known of the rows that a CTA walks next, looked up 32 at a time.
constexpr int kAhead = 32;
struct RowsAhead {
    const void *row[kAhead];
    void *grad[kAhead];
    int32_t token[kAhead];  // -1: does not count
    float z[kAhead];        // its logit, if asked for
    RowInputs in[kAhead];
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
template <bool ENT>
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
        rebase<ENT>(a, m, c);
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

}  // namespace seq
}  // namespace rlca

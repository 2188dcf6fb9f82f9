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

constexpr int kHeldWarps = 8;
constexpr int kHeldThreads = 32 * kHeldWarps;
constexpr int kHeldMaxCtas = 16;

// Packs of one of a row's `warps` warps; whole lines where the row begins on one.
__host__ __device__ __forceinline__ int held_share(int packs, int warps)
{
    return ((packs + warps - 1) / warps + 7) / 8 * 8;
}

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

// A warp's packs of a row: k0 .. k0 + n - 1, n <= 32 U; lane l has packs k0 + l, k0 + l + 32, ...
// Of those w0 .. w1 - 1 are whole; the others, the row's first and last where they are cut, are read
// and written element by element.
template <typename T>
struct Share {
    static constexpr int W = 16 / (int)sizeof(T);
    const T *z;
    int V, head, k0, n, w0, w1;

    __device__ __forceinline__ Share(const T *z_, int V_, int warp, int size)
        : z(z_), V(V_), head((int)((reinterpret_cast<uintptr_t>(z_) % 16) / sizeof(T)))
    {
        const int packs = (V + head + W - 1) / W, whole = (V + head) / W;
        k0 = warp * size;
        n = max(0, min(size, packs - k0));
        w0 = k0 == 0 && head != 0 ? 1 : 0;
        w1 = min(n, whole - k0);
    }
    __device__ __forceinline__ int first(int i) const { return (k0 + i) * W - head; }
    // This lane's first pack.
    __device__ __forceinline__ const T *pack0() const
    {
        return z + first((int)(threadIdx.x & 31));
    }
    __device__ __forceinline__ bool whole(int i) const
    {
        return (unsigned)(i - w0) < (unsigned)max(0, w1 - w0);
    }
    __device__ __forceinline__ bool cut() const { return n > 0 && (w0 != 0 || w1 != n); }
};

// On its way to shared memory: whole packs by asynchronous copies, which the thread that asked
// for them reads back; the elements of the row's first and last pack, where they are cut, in a
// register each.
template <typename T, int U>
struct Coming {
    static constexpr int W = 16 / (int)sizeof(T);
    T cut;

    __device__ __forceinline__ void ask(const Share<T> &a, uint4 *slots)
    {
        const int lane = threadIdx.x & 31;
        const T *from = a.pack0();
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (a.whole(u * 32 + lane)) copy_async(slots + u * kHeldThreads, from + u * 32 * W);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (a.cut()) {
            // Lanes 0..15: an element of the share's first pack; 16..31 of its last.
            const int i = lane < 16 ? 0 : a.n - 1, j = a.first(i) + (lane & 15);
            cut = narrow<T>(-INFINITY);
            if ((lane & 15) < W && !a.whole(i) && j >= 0 && j < a.V) cut = a.z[j];
        }
    }
    // What was asked for, as this lane's packs; -inf where there is nothing.
    __device__ __forceinline__ void get(const Share<T> &a, uint4 *slots, Pack<T, W> (&v)[U])
    {
        const int lane = threadIdx.x & 31;
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (a.cut()) {
            const int i = lane < 16 ? 0 : a.n - 1;
            if ((lane & 15) < W && !a.whole(i))
                reinterpret_cast<T *>(slots - lane + i / 32 * kHeldThreads + i % 32)[lane & 15] = cut;
            __syncwarp();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u * 32 + 32 > a.n) {
#pragma unroll
                for (int e = 0; e < W; ++e) v[u].e[e] = narrow<T>(-INFINITY);
                if (u * 32 + lane >= a.n) continue;
            }
            *reinterpret_cast<uint4 *>(&v[u]) = slots[u * kHeldThreads];
        }
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

    // (m, S, h) of the share of n packs with the largest element m, in all lanes.
    template <bool ENT>
    __device__ __forceinline__ RowStats stats(float m, int n, ExpScale c) const
    {
        const float ref = m == -INFINITY ? 0.f : m;
        const T low = lowest_logit<T>(ref, c);
        RowSums a[2] = {{pair(0.f, 0.f), pair(0.f, 0.f)}, {pair(0.f, 0.f), pair(0.f, 0.f)}};
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u * 32 < n) add_pack<T, ENT>(a[u & 1], v[u], ref, low, c);
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
    __device__ __forceinline__ void store(const Share<T> &a, T *g, const RowSlope &r, float m,
                                          ExpScale c) const
    {
        const T low = lowest_logit<T>(m, c);
        const int head = (int)((reinterpret_cast<uintptr_t>(g) % 16) / sizeof(T));
        const int s = (a.head - head + W) % W;
        if (ENT && flat_row(low)) shifted<false>(a, g, s, r, m, low, c);
        else if (s == 0) aligned<ENT>(a, g, r, m, low, c);
        else shifted<ENT>(a, g, s, r, m, low, c);
        __syncwarp();
    }

private:
    template <bool ENT>
    __device__ __forceinline__ void aligned(const Share<T> &a, T *g, const RowSlope &r, float m,
                                            T low, ExpScale c) const
    {
        const int lane = threadIdx.x & 31;
        T *to = g + a.first(lane);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u * 32 >= a.n) break;
            const Pack<T, W> o = pack_slope<T, ENT>(v[u], r, m, low, c);
            const int i = u * 32 + lane;
            if (a.whole(i))
                *reinterpret_cast<uint4 *>(to + u * 32 * W) = *reinterpret_cast<const uint4 *>(&o);
            else if (i < a.n)
                store_cut<T>(g, a.first(i), a.V, *reinterpret_cast<const uint4 *>(&o), 0, W);
        }
    }
    // The gradient's row lies at another offset to 16 bytes than the logits': its packs, which
    // begin s elements later, are put together from a lane's own and the next lane's.
    template <bool ENT>
    __device__ __forceinline__ void shifted(const Share<T> &a, T *g, int s, const RowSlope &r, float m,
                                            T low, ExpScale c) const
    {
        const int lane = threadIdx.x & 31;
        T *to = g + a.first(lane) + s;
        Pack<T, W> cur = pack_slope<T, ENT>(v[0], r, m, low, c);
        if (lane == 0 && a.n > 0)
            store_cut<T>(g, a.first(0), a.V, *reinterpret_cast<const uint4 *>(&cur), 0, s);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u * 32 >= a.n) break;
            Pack<T, W> next = cur;
            if (u + 1 < U && (u + 1) * 32 < a.n)
                next = pack_slope<T, ENT>(v[u + 1 < U ? u + 1 : u], r, m, low, c);
            const uint4 x = *reinterpret_cast<const uint4 *>(lane == 0 ? &next : &cur);
            uint4 y;
            y.x = __shfl_sync(kFullMask, x.x, lane + 1);
            y.y = __shfl_sync(kFullMask, x.y, lane + 1);
            y.z = __shfl_sync(kFullMask, x.z, lane + 1);
            y.w = __shfl_sync(kFullMask, x.w, lane + 1);
            const uint4 o = bytes_from(*reinterpret_cast<const uint4 *>(&cur), y, s * (int)sizeof(T));
            const int i = u * 32 + lane, j = a.first(i) + s;
            if (i + 1 < a.n && j >= 0 && j <= a.V - W)
                *reinterpret_cast<uint4 *>(to + u * 32 * W) = o;
            else if (i < a.n)
                store_cut<T>(g, j, a.V, o, 0, i + 1 < a.n ? W : W - s);
            cur = next;
        }
    }
};

// ------------------------------------------------------------------------- rows in clusters

// What is known of the rows that a cluster walks next, looked up 32 at a time.
constexpr int kAhead = 32;
struct RowsAhead {
    int32_t token[kAhead];  // -1: does not count
    float z[kAhead];        // its logit
    RowInputs in[kAhead];
};

struct HeldShared {
    RowStats parts[2][kHeldMaxCtas * kHeldWarps];
    RowsAhead ahead[2];
    RowSlope slope;
    float m;
};

struct TeacherParts {
    TeacherShared row;
    float2 parts[2][kHeldWarps];  // largest logit, sum of a warp's entries
    float loss[kHeldWarps];
};

struct StepAt {
    int64_t n, t;

    __device__ __forceinline__ StepAt after(const StepAt &by, int64_t T) const
    {
        StepAt r = {n + by.n, t + by.t};
        if (r.t >= T) {
            r.t -= T;
            ++r.n;
        }
        return r;
    }
};

__device__ __forceinline__ StepAt step_at(const VocabParams &p, int64_t i)
{
    if (p.M <= INT32_MAX) {
        const uint32_t n = (uint32_t)i / (uint32_t)p.T;
        return {(int64_t)n, (int64_t)((uint32_t)i - n * (uint32_t)p.T)};
    }
    return {i / p.T, i % p.T};
}

// Lane l looks up row i0 + l step.
template <typename T, VocabOp OP>
__device__ __forceinline__ void look_ahead(const VocabParams &p, RowsAhead &a, int64_t i0, int64_t step)
{
    const int lane = threadIdx.x & 31;
    const int64_t i = i0 + lane * step;
    int32_t token = -1;
    if (i < p.M) {
        const StepAt s = step_at(p, i);
        if (inside_row(p, s.n, s.t)) {
            int64_t j = 0;
            if (OP != VocabOp::kDistill) j = vocab_token(p, s.n, s.t);
            if (j >= 0 && j < p.V) {
                token = (int32_t)j;
                if (OP != VocabOp::kDistill) a.z[lane] = widen(row_of<T>(p.logits, s.n, s.t)[j]);
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

// MIN: CTAs that the registers are cut for.
template <typename T, VocabOp OP, bool ENT, bool GRAD, int U, int MIN>
__global__ void __launch_bounds__(kHeldThreads, MIN) vocab_held_kernel(const VocabParams p, int ctas)
{
    constexpr bool TEACH = OP == VocabOp::kDistill;
    constexpr int WARPS = kHeldWarps;
    namespace cg = cooperative_groups;
    __shared__ uint4 stage[U * kHeldThreads];
    __shared__ HeldShared sh;
    __shared__ typename std::conditional<TEACH, TeacherParts, int>::type teach;
    grid_dependency_sync();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)(blockIdx.x % ctas), warps = ctas * WARPS;
    const int64_t step = gridDim.x / ctas, first = blockIdx.x / ctas;
    const int wide = rank * kHeldThreads + tid;  // of the cluster's threads
    uint4 *slots = stage + tid;

    // All CTAs of the cluster run before one writes to another.
    if (ctas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    if (warp == 0) look_ahead<T, OP>(p, sh.ahead[0], first, step);
    if (ctas > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    __syncthreads();

    const StepAt by = step_at(p, step);
    StepAt s = step_at(p, first);
    const int V = (int)p.V;
    Coming<T, U> coming;
    Entry next = {-1, -INFINITY};
    auto ask = [&](const StepAt &at_row) {
        coming.ask(Share<T>(row_of<T>(p.logits, at_row.n, at_row.t), V, rank * WARPS + warp, p.share),
                   slots);
        if constexpr (TEACH) next = teacher_entry<T>(p, at_row, tid);
    };
    if (first < p.M && sh.ahead[0].token[0] >= 0) ask(s);
    int par = 0;
    unsigned k = 0;  // rows walked, modulo 2 kAhead
    StepAt s1;
    for (int64_t i = first; i < p.M; i += step, s = s1, k = (k + 1) % (2 * kAhead)) {
        const unsigned at_k = k % kAhead, k1 = (k + 1) % (2 * kAhead);
        const RowsAhead &now = sh.ahead[k / kAhead];
        if (at_k == kAhead * 3 / 4) {
            __syncthreads();  // nobody reads the rows before these any more
            if (warp == 0)
                look_ahead<T, OP>(p, sh.ahead[k / kAhead ^ 1], i + (kAhead - at_k) * step, step);
        }
        if (at_k == kAhead - 1) __syncthreads();
        s1 = s.after(by, p.T);
        T *g = GRAD ? out_row<T>(p.grad, s.n, s.t) : nullptr;
        const bool more = i + step < p.M && sh.ahead[k1 / kAhead].token[k1 % kAhead] >= 0;
        const int32_t token = now.token[at_k];
        if (token < 0) {
            if (wide == 0) write_uncounted(p, i);
            if (GRAD) clear_row(RowPacks<T>(g, p.V), g, wide, ctas * kHeldThreads);
            if (more) ask(s1);
            continue;
        }
        const Share<T> a(row_of<T>(p.logits, s.n, s.t), V, rank * WARPS + warp, p.share);
        Held<T, U> held;
        coming.get(a, slots, held.v);
        const float top = held.largest();
        const Entry entry = next;
        float z_entry = 0.f;
        if constexpr (TEACH) {
            if (entry.token >= 0) z_entry = widen(a.z[entry.token]);
        }
        // The slots are read (their largest value is known): the next row may come.
        if (more) ask(s1);
        const RowStats own = held.template stats<ENT>(top, a.n, p.scale);
        if constexpr (TEACH) {
            float m = entry.logit;
#pragma unroll
            for (int w = 16; w >= 1; w /= 2) m = max_nan(m, __shfl_xor_sync(kFullMask, m, w));
            float x = entry.token >= 0 ? expf((entry.logit - m) * p.inv_tau) : 0.f;
#pragma unroll
            for (int w = 16; w >= 1; w /= 2) x += __shfl_xor_sync(kFullMask, x, w);
            if (lane == 0) teach.parts[par][warp] = make_float2(m, x);
            teach.row.index[tid] = entry.token;
        }
        RowStats *parts = sh.parts[par];
        if (ctas > 1) {
            if (lane < (GRAD || TEACH ? ctas : 1))
                cg::this_cluster().map_shared_rank(parts, lane)[rank * WARPS + warp] = own;
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        } else {
            if (lane == 0) parts[warp] = own;
            __syncthreads();
        }
        par ^= 1;
        if (!GRAD && !TEACH && rank) continue;

        if constexpr (TEACH) {
            const RowStats st = join_parts<T, false>(parts, warps, p.scale);
            float t_top = -INFINITY, total = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) t_top = max_nan(t_top, teach.parts[par ^ 1][w].x);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float2 q = teach.parts[par ^ 1][w];
                if (q.x != -INFINITY) total += q.y * expf((q.x - t_top) * p.inv_tau);
            }
            const bool counted = t_top != -INFINITY && st.m != -INFINITY;
            const float weight = now.in[at_k].weight;
            const float v = entry.token >= 0 ? (entry.logit - t_top) * p.inv_tau : -INFINITY;
            const float q = entry.token >= 0 ? expf(v) / total : 0.f;
            const float sum = unbiased<T>(st).s;
            float part = 0.f;
            if (counted && (q > 0.f || isnan(q))) {
                const LogProb lp =
                    log_prob(z_entry, st.m, logf(sum), p.inv_tau, p.inv_tau_lo);
                part = -q * lp.minus(v - logf(total));
            }
#pragma unroll
            for (int w = 16; w >= 1; w /= 2) part += __shfl_xor_sync(kFullMask, part, w);
            if (lane == 0) teach.loss[warp] = part;
            teach.row.q[tid] = q;
            RowSlope r = {0.f, weight * p.inv_tau / sum, 0.f, weight == 0.f || !counted};
            if (GRAD) {
                if (r.zero) clear_row(RowPacks<T>(g, p.V), g, wide, ctas * kHeldThreads);
                else held.template store<false>(a, g, r, st.m, p.scale);
            }
            __syncthreads();  // entries of the row are overwritten by what they come to
            if (wide == 0) {
                float loss = 0.f;
                for (int w = 0; w < WARPS; ++w) loss += teach.loss[w];
                p.loss[i] = loss;
            }
            if (GRAD && !r.zero && entry.token >= 0) {
                const int pack = (entry.token + a.head) / RowPacks<T>::W;
                const int mine = WARPS * p.share;
                if (pack >= rank * mine && pack < (rank + 1) * mine) {
                    float both = 0.f;
                    for (int j = 0; j < p.K; ++j)
                        if (teach.row.index[j] == entry.token) both += teach.row.q[j];
                    g[entry.token] = narrow<T>(fmaf(-both, weight * p.inv_tau,
                                                    slope_at<T, false>(z_entry, r, st.m, p.scale)));
                }
            }
            __syncthreads();  // before the next row's entries take these places
        } else {
            if (warp == 0) {
                const RowStats st = join_parts<T, ENT>(parts, warps, p.scale);
                RowSlope r = {0.f, 0.f, 0.f, true};
                if (st.m != -INFINITY)
                    r = finish_row<T, OP, ENT>(p, i, now.z[at_k], st, now.in[at_k],
                                               rank == 0 && lane == 0);
                else if (wide == 0)
                    write_uncounted(p, i);
                if (GRAD && lane == 0) {
                    sh.slope = r;
                    sh.m = st.m;
                }
            }
            if (!GRAD) continue;
            __syncthreads();
            const RowSlope r = sh.slope;
            const float m = sh.m;
            if (r.zero) {
                clear_row(RowPacks<T>(g, p.V), g, wide, ctas * kHeldThreads);
                continue;
            }
            held.template store<ENT>(a, g, r, m, p.scale);
            const int pack = (token + a.head) / RowPacks<T>::W;
            if (pack >= a.k0 && pack < a.k0 + a.n && lane == 0)
                g[token] = narrow<T>(slope_at<T, ENT>(now.z[at_k], r, m, p.scale) + r.gamma);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace seq
}  // namespace rlca

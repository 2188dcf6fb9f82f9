// Rows of logits parked in shared memory, a CTA to a row: one pass over the parked row gives its
// largest logit and sums, a second the gradient, so HBM moves the row in and its gradient out and
// no more. The CTAs stay and walk the rows, two or more to an SM: while one waits for its row, or for
// the scalars between the passes, the others compute. Where logits and gradient lie alike, every
// thread asks for its part of the next row as it reads the last of this one. Of a row that is longer
// than an SM's share of shared memory the rest is read in both passes, the second time from the L2.
//
// Policy loss with KL and entropy and its gradient, [16, 1024, 32768] in bf16: 372 us, 5.8 TB/s or 0.85
// of the measured copy rate (0.93 without the entropy). One exponential and some four to five
// instructions to an element and pass, issue at 57 %; the rest are the waits at the two barriers of a
// row, which 22 warps to an SM do not hide. Held in registers instead, with a second row on its way
// (422 us): registers for one row of 100 KB and no second CTA. A gradient from a second read of HBM: 648.
#pragma once

#include "vocab_rows.cuh"

namespace rlca {
namespace seq {

constexpr int kParkedWarps = 16;
constexpr int kParkedPacks = 4;  // of a lane, read together: a warp's chunk is 128 packs
constexpr int kParkedChunk = 32 * kParkedPacks;

// Sums of rows of any length: what a lane adds up in 64 additions goes to a sum that keeps what its
// rounding leaves out. (2^30 logits alike would be off by 1 % otherwise: every addition rounds the same
// way. A whole parked row is at most 96 additions.)
struct LongSums {
    Two s, h;

    template <bool ENT>
    __device__ __forceinline__ void take(RowSums &a)
    {
        add(s, a.s.x + a.s.y);
        if (ENT) add(h, a.h.x + a.h.y);
        a = {pair(0.f, 0.f), pair(0.f, 0.f)};
    }

private:
    static __device__ __forceinline__ void add(Two &sum, float x)
    {
        const Two t = two_sum(sum.hi, x);
        sum = {t.hi, sum.lo + t.lo};
    }
};

struct ParkedShared {
    RowStats parts[2][kParkedWarps];
    RowsAhead ahead[2];
    RowSlope slope;
    float m, sum;
};

// A row's image in shared memory is that of its aligned packs: element j at head + j. LONG: it may
// end before the row does.
template <typename T, bool LONG>
struct Parked {
    static constexpr int W = 16 / (int)sizeof(T);
    const T *z;
    int V, head, packs, whole;  // pack 0 is whole where head is 0
    int room;                   // packs that the image holds, whole chunks

    __device__ __forceinline__ Parked(const T *z_, int V_, int room_)
        : z(z_), V(V_), head((int)((reinterpret_cast<uintptr_t>(z_) % 16) / sizeof(T))), room(room_)
    {
        packs = (V + head + W - 1) / W;
        whole = (V + head) / W;
    }
    __device__ __forceinline__ T value(const T *image, int j) const
    {
        return !LONG || j + head < room * W ? image[j + head] : z[j];
    }
    // Whether all packs of the chunk that begins with pack k are whole.
    __device__ __forceinline__ bool full(int k) const
    {
        return k + kParkedChunk <= whole && (k > 0 || head == 0);
    }
    // Asks for this lane's packs of the chunk that begins with pack k, if it is parked.
    __device__ __forceinline__ void ask(uint4 *image, int k) const
    {
        if (LONG && k >= room) return;
        const int lane = threadIdx.x & 31;
        const T *from = z + (k + lane) * W - head;
        uint4 *to = image + k + lane;
        if (full(k)) {
#pragma unroll
            for (int u = 0; u < kParkedPacks; ++u) copy_async(to + 32 * u, from + 32 * u * W);
        } else {
#pragma unroll
            for (int u = 0; u < kParkedPacks; ++u) {
                const int j = k + lane + 32 * u;
                if (j < whole && (j > 0 || head == 0)) copy_async(to + 32 * u, from + 32 * u * W);
            }
        }
    }
    // This lane's packs of a chunk; -inf where there are none.
    __device__ __forceinline__ void get(const uint4 *image, int k, Pack<T, W> (&v)[kParkedPacks]) const
    {
        const uint4 *from = image + k + (threadIdx.x & 31);
        if (LONG && k >= room) {
            read(k, v);
        } else if (k + kParkedChunk <= packs) {
#pragma unroll
            for (int u = 0; u < kParkedPacks; ++u) *reinterpret_cast<uint4 *>(&v[u]) = from[32 * u];
        } else {
#pragma unroll
            for (int u = 0; u < kParkedPacks; ++u) {
                const T none[2] = {narrow<T>(-INFINITY), narrow<T>(-INFINITY)};
                const uint32_t x = *reinterpret_cast<const uint32_t *>(none);
                uint4 q = make_uint4(x, x, x, x);
                if (k + (int)(threadIdx.x & 31) + 32 * u < packs) q = from[32 * u];
                *reinterpret_cast<uint4 *>(&v[u]) = q;
            }
        }
    }
    // The same of a chunk that is not parked.
    __device__ __forceinline__ void read(int k, Pack<T, W> (&v)[kParkedPacks]) const
    {
        const int j = k + (threadIdx.x & 31);
        const T *from = z + j * W - head;
        if (k + kParkedChunk <= whole) {
#pragma unroll
            for (int u = 0; u < kParkedPacks; ++u)
                *reinterpret_cast<uint4 *>(&v[u]) = *reinterpret_cast<const uint4 *>(from + 32 * u * W);
        } else {
#pragma unroll
            for (int u = 0; u < kParkedPacks; ++u) {
#pragma unroll
                for (int e = 0; e < W; ++e) v[u].e[e] = narrow<T>(-INFINITY);
                if (j + 32 * u < whole) {
                    *reinterpret_cast<uint4 *>(&v[u]) =
                        *reinterpret_cast<const uint4 *>(from + 32 * u * W);
                } else if (j + 32 * u < packs) {
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if ((j + 32 * u) * W - head + e < V) v[u].e[e] = from[32 * u * W + e];
                }
            }
        }
    }
    // The element of a cut pack that a thread is to put in: the first pack's by the threads of warp 0,
    // the last's by those of the warp that has it, in lanes 16 and on. -1: none.
    __device__ __forceinline__ int cut() const
    {
        const int lane = threadIdx.x & 31, e = lane & 15;
        if (e >= W) return -1;
        if (lane < 16) return threadIdx.x < 16 && (head != 0 || whole == 0) ? e : -1;
        return whole < packs && (!LONG || whole < room) && whole / kParkedChunk % (int)(blockDim.x / 32) == (int)(threadIdx.x / 32)
                   ? whole * W + e
                   : -1;
    }
    __device__ __forceinline__ T cut_value(int i) const
    {
        return i >= head && i < V + head ? z[i - head] : narrow<T>(-INFINITY);
    }
};

template <typename T, VocabOp OP, bool ENT, bool GRAD, bool LONG>
__global__ void __launch_bounds__(32 * kParkedWarps, 2)
    vocab_parked_kernel(const VocabParams p, int room)
{
    constexpr bool TEACH = OP == VocabOp::kDistill;
    constexpr int W = 16 / (int)sizeof(T), U = kParkedPacks;
    extern __shared__ uint4 image[];
    __shared__ ParkedShared sh;
    __shared__ typename std::conditional<TEACH, TeacherParts, int>::type teach;
    grid_dependency_sync();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
    const int warps = threads / 32, tile = warps * kParkedChunk;
    const unsigned step = gridDim.x, rows = (unsigned)p.M;
    const int V = (int)p.V;
    const ExpScale scale = p.scale;

    if (warp == 0) look_ahead<T, OP, !GRAD>(p, sh.ahead[0], blockIdx.x, step);
    __syncthreads();

    T cut = narrow<T>(0.f);
    Entry next = {-1, -INFINITY};
    // All of a row, or, where its packs are asked for one by one, the rest.
    auto ask = [&](const RowsAhead &from, int k, unsigned i, bool packs) {
        const Parked<T, LONG> a(static_cast<const T *>(from.row[k]), V, room);
        if (packs) {
            for (int c = warp * kParkedChunk; c < (LONG ? min(room, a.packs) : a.packs); c += tile)
                a.ask(image, c);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        if (!p.even) {
            const int c = a.cut();
            if (c >= 0) cut = a.cut_value(c);
        }
        if constexpr (TEACH) next = teacher_entry<T>(p, step_at(p, i), tid);
    };
    if (sh.ahead[0].token[0] >= 0) ask(sh.ahead[0], 0, blockIdx.x, true);
    int par = 0;
    unsigned k = 0;  // rows walked, modulo 2 kAhead
    for (unsigned i = blockIdx.x; i < rows; i += step, k = (k + 1) % (2 * kAhead)) {
        const unsigned at_k = k % kAhead, k1 = (k + 1) % (2 * kAhead);
        const RowsAhead &now = sh.ahead[k / kAhead];
        if (at_k == kAhead * 3 / 4) {
            __syncthreads();  // nobody reads the rows before these any more
            if (warp == 0)
                look_ahead<T, OP, !GRAD>(p, sh.ahead[k / kAhead ^ 1],
                                  i + (int64_t)(kAhead - at_k) * step, step);
        }
        if (at_k == kAhead - 1) __syncthreads();
        T *g = GRAD ? static_cast<T *>(now.grad[at_k]) : nullptr;
        const RowsAhead &then = sh.ahead[k1 / kAhead];
        const bool more = (int64_t)i + step < rows && then.token[k1 % kAhead] >= 0;
        const int32_t token = now.token[at_k];
        if (token < 0) {
            if (tid == 0) write_uncounted(p, i);
            if (GRAD) clear_row(g, 0, V, tid, threads);
            if (more) ask(then, k1 % kAhead, i + step, true);
            continue;
        }
        const Parked<T, LONG> a(static_cast<const T *>(now.row[at_k]), V, room);
        const Parked<T, LONG> b(more ? static_cast<const T *>(then.row[k1 % kAhead]) : a.z, V, room);
        const int reach = max(a.packs, b.packs);  // a row's packs are one more where it begins amid one
        const Entry entry = next;

        // First pass. Sums relative to the largest logit of the warp's first chunk, which is changed only where a
        // later chunk's is more than e^4 above it (or a NaN): the largest logits of a row are near
        // one another, and a change costs every lane an exponential.
        float ref = -INFINITY;
        T low = lowest_logit<T>(0.f, scale);
        RowSums sums = {pair(0.f, 0.f), pair(0.f, 0.f)};
        LongSums all = {{0.f, 0.f}, {0.f, 0.f}};
        int added = 0;
        // The sums so far, of this lane.
        auto stats = [&]() {
            RowStats st = {ref, sums.s.x + sums.s.y, sums.h.x + sums.h.y};
            if (LONG) {
                st.s = all.s.hi + (all.s.lo + st.s);
                st.h = all.h.hi + (all.h.lo + st.h);
            }
            return st;
        };
        auto add = [&](const Pack<T, W> (&v)[U]) {
            MaxOf<T> most;
#pragma unroll
            for (int u = 0; u < U; ++u) most.add(v[u]);
            float top = most.get();
            if (__any_sync(kFullMask, !(top <= ref + p.near))) {
#pragma unroll
                for (int w = 16; w >= 1; w /= 2)
                    top = max_nan(top, __shfl_xor_sync(kFullMask, top, w));
                top = max_nan(top, ref);
                RowStats st = stats();
                rebase<ENT>(st, top, scale);
                sums = {pair(st.s, 0.f), pair(st.h, 0.f)};
                all = {{0.f, 0.f}, {0.f, 0.f}};
                ref = top;
                low = lowest_logit<T>(ref, scale);
            }
            const float from = ref == -INFINITY ? 0.f : ref;
            if (ENT && cut_late(low)) {
#pragma unroll
                for (int u = 0; u < U; ++u) add_pack<T, ENT, true>(sums, v[u], from, low, scale);
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) add_pack<T, ENT, false>(sums, v[u], from, low, scale);
            }
            if (LONG && (added += U * W / 2) == 64) {
                all.template take<ENT>(sums);
                added = 0;
            }
        };
        // What is not parked first: the rest may still be on its way.
        for (int c = room + warp * kParkedChunk; LONG && c < a.packs; c += tile) {
            Pack<T, W> v[U];
            a.read(c, v);
            add(v);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (!p.even) {
            const int c = a.cut();
            if (c >= 0) reinterpret_cast<T *>(image)[c] = cut;
            __syncwarp();
        }
        const int end = GRAD || TEACH ? a.packs : reach;
        for (int c = warp * kParkedChunk; c < (LONG ? min(room, end) : end); c += tile) {
            Pack<T, W> v[U];
            a.get(image, c, v);
            add(v);
            if (!GRAD && !TEACH && more) b.ask(image, c);
        }
        {
            RowStats own = stats();
#pragma unroll
            for (int w = 16; w >= 1; w /= 2) {
                own.s += __shfl_xor_sync(kFullMask, own.s, w);
                if (ENT) own.h += __shfl_xor_sync(kFullMask, own.h, w);
            }
            if (lane == 0) sh.parts[par][warp] = own;
        }
        if constexpr (TEACH) teacher_send(p, teach, par, entry);
        float z_a = 0.f;
        if (!GRAD && !TEACH) z_a = now.z[at_k];
        __syncthreads();
        const RowStats *parts = sh.parts[par];
        const int tpar = par;
        par ^= 1;
        if (TEACH ? entry.token >= 0 : GRAD && warp == 0)
            z_a = widen(a.value(reinterpret_cast<const T *>(image), TEACH ? entry.token : token));

        const RowInputs &in = now.in[at_k];
        if (warp == 0) {
            const RowStats st = join_parts<ENT>(parts, warps, scale);
            RowSlope r = {0.f, 0.f, 0.f, true};
            if constexpr (TEACH) {
                const float sum = unbiased(st).s;
                r = teacher_slope(p, teach, tpar, st.m, sum, in.weight);
                if (lane == 0) sh.sum = sum;
            } else if (st.m != -INFINITY) {
                r = finish_row<T, OP, ENT>(p, i, z_a, st, in, lane == 0);
            } else if (lane == 0) {
                write_uncounted(p, i);
            }
            if ((GRAD || TEACH) && lane == 0) {
                sh.slope = r;
                sh.m = st.m;
            }
        }
        if (!GRAD && !TEACH) {
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (more) ask(then, k1 % kAhead, i + step, false);
            continue;
        }
        __syncthreads();
        const RowSlope r = sh.slope;
        const float m = sh.m;
        // Second pass.
        bool asked = false;
        if (GRAD && r.zero) {
            clear_row(g, 0, V, tid, threads);
        } else if (GRAD) {
            const T low = lowest_logit<T>(m, scale);
            const int head = (int)((reinterpret_cast<uintptr_t>(g) % 16) / sizeof(T));
            const bool late = ENT && cut_late(low);
            if (head == a.head && !late) {
                asked = true;
                for (int c = warp * kParkedChunk; c < reach; c += tile) {
                    Pack<T, W> v[U];
                    a.get(image, c, v);
                    T *to = g + (c + lane) * W - head;
                    if (a.full(c)) {
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const Pack<T, W> o = pack_slope<T, ENT>(v[u], r, m, low, scale);
                            *reinterpret_cast<uint4 *>(to + 32 * u * W) =
                                *reinterpret_cast<const uint4 *>(&o);
                        }
                    } else {
#pragma unroll 1
                        for (int u = 0; u < U; ++u) {
                            const int j = c + lane + 32 * u;
                            const Pack<T, W> o = pack_slope<T, ENT>(v[0], r, m, low, scale);
                            if (j < a.whole && (j > 0 || head == 0))
                                *reinterpret_cast<uint4 *>(to + 32 * u * W) =
                                    *reinterpret_cast<const uint4 *>(&o);
                            else if (j < a.packs)
                                store_cut<T>(g, j * W - head, V, *reinterpret_cast<const uint4 *>(&o),
                                             0, W);
#pragma unroll
                            for (int x = 0; x + 1 < U; ++x) v[x] = v[x + 1];
                        }
                    }
                    if (more) b.ask(image, c);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            } else {
                // The gradient's packs lie across the image's: each is put together from two.
                const int packs = (V + head + W - 1) / W, off = (a.head - head) * (int)sizeof(T);
                const int whole = (V + head) / W;
                for (int c = warp * kParkedChunk; c < packs; c += tile) {
                    T *to = g + (c + lane) * W - head;
                    // Between the ends: the image's pack in which the gradient's begins, and the next.
                    const uint4 *from = image + c + lane + (off >> 4);
                    // (From what is parked, or, where the next is a whole pack too, from memory.)
                    const bool inside = c + kParkedChunk <= whole && c > 0 && !late;
                    const bool apart = LONG && c >= room && c + kParkedChunk < a.whole;
                    if (apart)
                        from = reinterpret_cast<const uint4 *>(a.z + (c + lane) * W - a.head) + (off >> 4);
                    if (inside && (!LONG || c + kParkedChunk < room || apart)) {
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const uint4 x = bytes_from(from[32 * u], from[32 * u + 1], off & 15);
                            const Pack<T, W> o = pack_slope<T, ENT>(
                                *reinterpret_cast<const Pack<T, W> *>(&x), r, m, low, scale);
                            *reinterpret_cast<uint4 *>(to + 32 * u * W) =
                                *reinterpret_cast<const uint4 *>(&o);
                        }
                    } else {
#pragma unroll 1
                        for (int u = 0; u < U; ++u) {
                            const int j = c + lane + 32 * u, first = j * W - head;
                            if (j >= packs) break;
                            Pack<T, W> v;
#pragma unroll
                            for (int e = 0; e < W; ++e) {
                                const int x = min(max(first + e, 0), V - 1);
                                v.e[e] = a.value(reinterpret_cast<const T *>(image), x);
                            }
                            const Pack<T, W> o = late ? pack_slope<T, ENT, true>(v, r, m, low, scale)
                                                      : pack_slope<T, ENT>(v, r, m, low, scale);
                            if (first >= 0 && first + W <= V)
                                *reinterpret_cast<uint4 *>(to + 32 * u * W) =
                                    *reinterpret_cast<const uint4 *>(&o);
                            else
                                store_cut<T>(g, first, V, *reinterpret_cast<const uint4 *>(&o), 0, W);
                        }
                    }
                }
            }
        }
        if constexpr (TEACH) teacher_share(p, teach, tpar, entry, z_a, m, sh.sum);
        __syncthreads();  // the row's gradient is written, and its image free
        if (more) ask(then, k1 % kAhead, i + step, !asked);
        if constexpr (TEACH) {
            if (tid == 0) p.loss[i] = teacher_loss(p, teach, tpar);
            if (GRAD && !r.zero && entry.token >= 0)
                g[entry.token] = teacher_gradient<T>(p, teach, tpar, entry, z_a, r, m, in.weight);
        } else if (GRAD && !r.zero && tid == 0) {
            g[token] = narrow<T>(slope_at<T, ENT>(z_a, r, m, scale) + r.gamma);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace seq
}  // namespace rlca

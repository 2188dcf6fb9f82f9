// Short rows of logits (a few actions to a thousand): a warp takes a tile of up to 32 rows through
// shared memory, so that memory moves in whole lines whatever the rows' length is. Groups of G lanes
// take the rows' sums; then every lane works out the scalars of one row, which cost a few hundred
// instructions and would be most of the work if a warp did them row by row; then the groups form
// the gradients in place. Rows of a few elements that are no whole packs are a lane's own.
//
// Policy loss with entropy and its gradient, [4096, 512, 18] in fp32: 78 us, 4.7 TB/s, 0.70 of the
// measured copy rate: issue slots 69 % busy with some 1000 instructions to a tile of 576 elements, a third
// of them the scalars of its rows; the rest is a warp's wait for its only tile, which no other work of its
// own covers. A CTA to a row took 12.7 ms, groups of four lanes to each of these rows 160 us. Rows of 512
// in bf16, policy loss with KL and entropy: 132 us, 4.1 TB/s; of 511, whose packs begin anywhere, 198 us,
// 2.7 TB/s.
#pragma once

#include "vocab_slope.cuh"

namespace rlca {
namespace seq {

constexpr int kTileWarps = 8;  // at the most; a CTA's tiles stay below 48 KB
constexpr int kTileBytes = 8192;       // of logits to a warp
constexpr int kTileMostBytes = 16384;  // the same, where fewer rows would not do
constexpr int kTilePacks = 4;          // of a lane, at the most
constexpr int kTileOwn = 40;           // elements of a row that may be a lane's own

struct TileShape {
    int group;    // lanes to a row, a power of two
    int rows;     // of a tile, a multiple of 32 / group
    int from, to; // how the rows of logits and gradients lie (tile_layout)
    int bytes;    // of a warp's shared memory
    int step;     // bytes that every row's beginning is a multiple of: 2, 4, 8 or 16
};

// Copies a tile to shared memory (IN) or from it, in pieces as wide as its rows allow. `mine`: this
// lane's row in memory, of `rows`, which are one behind the other (near) or not.
template <typename T, bool IN>
__device__ __forceinline__ void tile_copy(T *mine, T *image, int rows, int V, bool near, bool even)
{
    constexpr int W = 16 / (int)sizeof(T);
    const int lane = threadIdx.x & 31, all = rows * V;
    auto row = [&](int r) {
        return reinterpret_cast<T *>(
            __shfl_sync(kFullMask, (unsigned long long)mine, min(r, rows - 1)));
    };
    auto piece = [&](auto zero, T *at_image, T *at_memory) {
        using P = decltype(zero);
        if constexpr (IN && sizeof(P) == 16) {
            copy_async(at_image, at_memory);
        } else if constexpr (IN) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;"
                         :
                         : "r"((uint32_t)__cvta_generic_to_shared(at_image)), "l"(at_memory),
                           "n"(sizeof(P))
                         : "memory");
        } else {
            *reinterpret_cast<P *>(at_memory) = *reinterpret_cast<const P *>(at_image);
        }
    };
    auto pieces = [&](auto zero, T *memory) {
        constexpr int n = (int)(sizeof(zero) / sizeof(T));
        int k = lane * n;
        for (; k + n <= all; k += 32 * n) piece(zero, image + k, memory + k);
        for (k = all / n * n + lane; k < all; k += 32) {
            if (IN) image[k] = memory[k];
            else memory[k] = image[k];
        }
    };
    if (near) {
        T *memory = row(0);
        const uintptr_t at = reinterpret_cast<uintptr_t>(memory);
        if (at % 16 == 0) {
            pieces(uint4{}, memory);
        } else if (at % 8 == 0) {
            pieces(uint2{}, memory);
        } else if (at % 4 == 0) {
            pieces(uint32_t{}, memory);
        } else {
#pragma unroll 4
            for (int k = lane; k < all; k += 32) {
                if (IN) image[k] = memory[k];
                else memory[k] = image[k];
            }
        }
        return;
    }
    // Row by row: pack, or element, k of the tile is number e of row r.
    const int size = even ? V / W : V, dr = 32 / size, de = 32 % size;
    int r = lane / size, e = lane % size;
    for (int k = lane; k - lane < rows * size; k += 32) {
        T *memory = row(r);
        if (k < rows * size) {
            if (even) piece(uint4{}, image + k * W, memory + e * W);
            else if (IN) image[k] = memory[e];
            else memory[e] = image[k];
        }
        r += dr;
        e += de;
        if (e >= size) {
            e -= size;
            ++r;
        }
    }
}

// Applies f(two elements, how many of them there are) to a lane's own row; WRITE: what it gives takes
// their place. Rows of an even length are pairs of words, or whole words.
template <bool WRITE, typename T, typename F>
__device__ __forceinline__ void own_elements(T *x, int V, F f)
{
    if (V % 2 == 0) {
#pragma unroll 4
        for (int j = 0; j < V; j += 2) {
            Pack<T, 2> &at = *reinterpret_cast<Pack<T, 2> *>(x + j);
            const Pack<T, 2> z = at;
            const Pair y = f(pair(widen(z.e[0]), widen(z.e[1])), 2);
            if (WRITE) at = Pack<T, 2>{{narrow<T>(y.x), narrow<T>(y.y)}};
        }
    } else {
#pragma unroll 2
        for (int j = 0; j + 1 < V; j += 2) {
            const Pair y = f(pair(widen(x[j]), widen(x[j + 1])), 2);
            if (WRITE) {
                x[j] = narrow<T>(y.x);
                x[j + 1] = narrow<T>(y.y);
            }
        }
        const float last = widen(x[V - 1]);
        const Pair y = f(pair(last, last), 1);
        if (WRITE) x[V - 1] = narrow<T>(y.x);
    }
}

// A row is a lane's own, of whole packs, or neither.
enum class TileRows : int { kOwn, kWhole, kAny };

// CTAs of 8 warps that the registers are cut for. Rows of any length take 110 registers without (policy
// loss, 268 MB of rows of 129 in bf16: 316 us, 241 with); a lane's own rows run best with few
// (rows of 18 in fp32: 148 us at 40 registers, 165 at up to 64).
constexpr int tile_ctas(TileRows rows) { return rows == TileRows::kOwn ? 6 : 4; }

template <typename T, VocabOp OP, bool ENT, bool GRAD, TileRows ROWS>
__global__ void __launch_bounds__(32 * kTileWarps, tile_ctas(ROWS))
    vocab_tile_kernel(const VocabParams p, const TileShape sh)
{
    constexpr bool SLOPE = OP == VocabOp::kSlope, EVEN = ROWS == TileRows::kWhole;
    constexpr bool lonely = ROWS == TileRows::kOwn;
    // The exponentials of a lane's own row of fp32 stay in its place for the second pass, where that does
    // not need their exponents too.
    constexpr bool kept = lonely && !SLOPE && GRAD && !ENT && sizeof(T) == 4;
    constexpr int W = 16 / (int)sizeof(T), E = kTilePacks;
    extern __shared__ uint4 tiles[];
    grid_dependency_sync();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, V = (int)p.V;
    const int64_t i0 = ((int64_t)blockIdx.x * (blockDim.x / 32) + warp) * sh.rows;
    if (i0 >= p.M) return;
    const int rows = (int)(p.M - i0 < sh.rows ? p.M - i0 : sh.rows);
    float4 *scalars = reinterpret_cast<float4 *>(reinterpret_cast<char *>(tiles) + warp * sh.bytes);
    uint4 *image4 = reinterpret_cast<uint4 *>(scalars + 32);
    T *image = reinterpret_cast<T *>(image4);
    const ExpScale c = p.scale;

    // The tile, and what is known of its rows: a row to a lane.
    StepAt s = {0, 0};
    if (lane < rows) s = step_at(p, (int)i0 + lane);
    const int first_t = __shfl_sync(kFullMask, s.t, 0);
    const auto near = [&](int layout) {
        return (layout & 3) == 3 || ((layout & 3) == 1 && first_t + rows <= p.T);
    };
    tile_copy<T, true>(out_row<T>(p.logits, s.n, s.t), image, rows, V, near(sh.from),
                       EVEN && (sh.from & 4));
    asm volatile("cp.async.commit_group;" ::: "memory");
    bool counted = lane < rows && inside_row(p, s.n, s.t);
    int token = -1;
    RowInputs in = {0.f, 0.f, 0.f, 1.f};
    if (counted) {
        const int64_t j = vocab_token(p, s.n, s.t);
        counted = j >= 0 && j < V;
        if (counted) {
            token = (int)j;
            if (!SLOPE) in = row_inputs<OP>(p, s.n, s.t);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();

    const int G = lonely ? 1 : sh.group, own = lane & (G - 1), turns = (rows * G + 31) / 32;
    const int held = (V + W - 1) / W;  // packs of a row
    // This lane's packs of row r; -inf where there is nothing.
    auto get = [&](int r, Pack<T, W> (&v)[E]) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (e * G >= held) break;
            const int k = own + e * G;
            if (k < held && r < rows) {
                uint4 x;
                if constexpr (EVEN) {
                    x = image4[r * held + k];
                } else {
                    const int byte = (r * V + k * W) * (int)sizeof(T);
                    if (sh.step == 8) {
                        const uint2 *at8 = reinterpret_cast<const uint2 *>(image4) + (byte >> 3);
                        const uint2 lo = at8[0], hi = at8[1];
                        x = make_uint4(lo.x, lo.y, hi.x, hi.y);
                    } else {
                        const uint32_t *w = reinterpret_cast<const uint32_t *>(image4) + (byte >> 2);
                        x = make_uint4(w[0], w[1], w[2], w[3]);
                        if (sizeof(T) == 2 && sh.step == 2) {
                            const int bits = (byte & 2) * 8;
                            x.x = __funnelshift_r(x.x, x.y, bits);
                            x.y = __funnelshift_r(x.y, x.z, bits);
                            x.z = __funnelshift_r(x.z, x.w, bits);
                            x.w = __funnelshift_r(x.w, w[4], bits);
                        }
                    }
                }
                *reinterpret_cast<uint4 *>(&v[e]) = x;
                if (!EVEN && k == held - 1) {
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        if (k * W + i >= V) v[e].e[i] = narrow<T>(-INFINITY);
                }
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i) v[e].e[i] = narrow<T>(-INFINITY);
            }
        }
    };
    const float z_a = counted ? widen(image[lane * V + token]) : 0.f;
    RowStats st = no_stats();
    if constexpr (SLOPE) {
    } else if constexpr (lonely) {
        T *x = image + lane * V;
        if (lane < rows) {
            own_elements<false>(x, V, [&](Pair z, int) {
                st.m = max_nan(max_nan(st.m, z.x), z.y);
                return z;
            });
            const float ref = st.m == -INFINITY ? 0.f : st.m;
            Pair sum = pair(0.f, 0.f), h = sum;
            own_elements<kept>(x, V, [&](Pair z, int n) {
                ExpOf y = exp_of<T, ENT>(z, ref, c);
                if (n == 1) y.e.y = 0.f;
                sum = add2(sum, y.e);
                if (ENT) h = fma2(y.e, y.below, h);
                return kept ? y.e : z;
            });
            st.s = sum.x + sum.y;
            st.h = h.x + h.y;
        }
    } else {
        for (int turn = 0; turn < turns; ++turn) {
            const int r = (turn * 32 + lane) / G;
            Pack<T, W> v[E];
            get(r, v);
            MaxOf<T> top;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (e * G >= held) break;
                top.add(v[e]);
            }
            float m = top.get();
            for (int w = G / 2; w >= 1; w /= 2) m = max_nan(m, __shfl_xor_sync(kFullMask, m, w));
            const float ref = m == -INFINITY ? 0.f : m;
            const T low = lowest_logit<T>(ref, c);
            // (The rows of a turn alike: either way gives the same bits.)
            const bool late = ENT && sizeof(T) == 2 && __any_sync(kFullMask, cut_late(low));
            RowSums a = {pair(0.f, 0.f), pair(0.f, 0.f)};
            if (late) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (e * G >= held) break;
                    add_pack<T, ENT, true>(a, v[e], ref, low, c);
                }
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (e * G >= held) break;
                    add_pack<T, ENT, false>(a, v[e], ref, low, c);
                }
            }
            float sum = a.s.x + a.s.y, h = ENT ? a.h.x + a.h.y : 0.f;
            for (int w = G / 2; w >= 1; w /= 2) {
                sum += __shfl_xor_sync(kFullMask, sum, w);
                if (ENT) h += __shfl_xor_sync(kFullMask, h, w);
            }
            if (own == 0 && r < rows) scalars[r] = make_float4(m, sum, h, 0.f);
        }
        __syncwarp();
        if (lane < rows) {
            const float4 q = scalars[lane];
            st = {q.x, q.y, q.z};
        }
    }

    RowSlope r = {0.f, 0.f, 0.f, true};
    float m = 0.f;
    if constexpr (SLOPE) {
        if (counted) {
            r = saved_slope<T, ENT>(p, (int)i0 + lane, s, m);
        }
    } else if (lane < rows) {
        m = st.m;
        if (counted && m != -INFINITY)
            r = finish_row<T, OP, ENT>(p, i0 + lane, z_a, st, in, true);
        else
            write_uncounted(p, i0 + lane);
    }
    if (!GRAD) return;
    if constexpr (lonely) {
        if (lane < rows) {
            const Pair alpha = pair(r.alpha, r.alpha), kappa = pair(r.kappa, r.kappa);
            own_elements<true>(image + lane * V, V, [&](Pair z, int) {
                ExpOf y = {z, z};
                if (!kept) y = exp_of<T, ENT>(z, m, c);
                y.e = mul2(y.e, ENT ? fma2(alpha, y.below, kappa) : kappa);
                return r.zero ? pair(0.f, 0.f) : y.e;
            });
        }
    } else {
        __syncwarp();
        scalars[lane] = make_float4(r.alpha, r.kappa, m, r.zero ? 1.f : 0.f);
        __syncwarp();
    }
    for (int turn = 0; !lonely && turn < turns; ++turn) {
        const int row = (turn * 32 + lane) / G;
        const float4 q = scalars[row & 31];
        const RowSlope slope = {q.x, q.y, 0.f, q.w != 0.f};
        Pack<T, W> v[E];
        get(row, v);
        const T low = lowest_logit<T>(q.z, c);
        const bool late = ENT && sizeof(T) == 2 && __any_sync(kFullMask, cut_late(low));
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (e * G >= held) break;
            const int k = own + e * G;
            Pack<T, W> o;
            if (late) o = pack_slope<T, ENT, true>(v[e], slope, q.z, low, c);
            else o = pack_slope<T, ENT>(v[e], slope, q.z, low, c);
            if (slope.zero) o = zero_pack<T, W>();
            if (k >= held || row >= rows) continue;
            if constexpr (EVEN) {
                image4[row * held + k] = *reinterpret_cast<const uint4 *>(&o);
            } else {
                T *to = image + row * V + k * W;
                const uint4 x = *reinterpret_cast<const uint4 *>(&o);
                if (k * W + W > V) {
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        if (k * W + i < V) to[i] = o.e[i];
                } else if (sh.step == 8) {
                    reinterpret_cast<uint2 *>(to)[0] = make_uint2(x.x, x.y);
                    reinterpret_cast<uint2 *>(to)[1] = make_uint2(x.z, x.w);
                } else if (sizeof(T) == 4 || reinterpret_cast<uintptr_t>(to) % 4 == 0) {
                    uint32_t *words = reinterpret_cast<uint32_t *>(to);
                    words[0] = x.x;
                    words[1] = x.y;
                    words[2] = x.z;
                    words[3] = x.w;
                } else {
                    // From the second element on, whole words.
                    uint32_t *words = reinterpret_cast<uint32_t *>(to + 1);
                    to[0] = o.e[0];
                    words[0] = __funnelshift_r(x.x, x.y, 16);
                    words[1] = __funnelshift_r(x.y, x.z, 16);
                    words[2] = __funnelshift_r(x.z, x.w, 16);
                    to[W - 1] = o.e[W - 1];
                }
            }
        }
        __syncwarp();
    }
    __syncwarp();
    if (!r.zero) image[lane * V + token] = narrow<T>(slope_at<T, ENT>(z_a, r, m, c) + r.gamma);
    __syncwarp();
    tile_copy<T, false>(out_row<T>(p.grad, s.n, s.t), image, rows, V, near(sh.to),
                        EVEN && (sh.to & 4));
}

}  // namespace seq
}  // namespace rlca

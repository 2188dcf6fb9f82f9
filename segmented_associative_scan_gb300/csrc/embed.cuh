// Token embedding: rows of a table, scaled; and the table's gradient, a segmented sum over
// the positions sorted by token.
//
// Gradient: the (token, position) pairs are sorted by token, stably, so the positions of a
// token stay in order. The sorted pairs are cut into runs of kRun; a CTA adds up the rows
// of one run segment by segment. A segment inside a run is written at once; what crosses
// a run's border goes to a partial row and is added up, run after run, by a last kernel. So
// the sums are taken in one fixed order whatever the GPU does, frequent tokens are spread
// over many CTAs, and no atomics are needed. The sort leaves a byte per row of the table that
// says whether its token occurs; rows that do not are written as 0 by CTAs of the same launch
// as the runs, so every row is written once (clearing all of the table beside the sort kept
// the sort waiting for memory: 113 us for both at 65536 tokens and 205 MB).
//
// 65536 rows of 1024 in bf16 into [50000, 1024]: 90 us for 339 MB: the sort 21 us (two passes,
// barriers and scattered stores of 16 SMs), the runs with the absent rows 53 us (6.4 TB/s), the join
// 18 us (dependent reads at 15 warps to an SM). A lookup of 16384 such rows
// takes 8 us (its table and rows stay in the L2 between repetitions).
#pragma once

#include "sequence.cuh"

namespace rlca {
namespace seq {

constexpr int kEmbedThreads = 128;
constexpr int kRun = 32;               // sorted pairs of one run
constexpr int kSortCtas = 16;          // one cluster
constexpr int kSortThreads = 512;
constexpr int kSortItems = 8;          // pairs of a thread per sweep

struct EmbedParams {
    const void *tokens;
    int token_bytes;
    const void *table, *dout;
    int64_t ld;      // of table or dout
    void *out;
    int64_t out_ld;
    float *dtable;
    float scale;
    int64_t M, V, D;
    // gradient workspace
    uint2 *pairs[2];             // (token or V, position): the sort ends in [0]
    uint8_t *present;            // [V] (and up to 15 more): the token occurs
    float *partial;              // [runs, 2, D]: what a run holds of the segment that came
                                 // in, and of the one that goes on
};

struct EmbedWorkspace {
    size_t pairs[2], present, partial, bytes;
};

inline EmbedWorkspace embed_workspace(int64_t M, int64_t V, int64_t D)
{
    EmbedWorkspace w;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t r = at;
        at += align256(n);
        return r;
    };
    for (int i = 0; i < 2; ++i) w.pairs[i] = take((size_t)M * 8);
    w.present = take((size_t)V + 16);
    w.partial = take((size_t)((M + kRun - 1) / kRun) * 2 * (size_t)D * 4);
    w.bytes = at;
    return w;
}

// Passes of 8 bits that sort keys 0..V (V: outside the table).
inline int sort_passes(int64_t V)
{
    int bits = 1;
    while (bits < 32 && (V >> bits) != 0) ++bits;
    return (bits + 7) / 8;
}

cudaError_t launch_embed_sort(const EmbedParams &p, cudaStream_t stream);
cudaError_t launch_embed_join(const EmbedParams &p, cudaStream_t stream);

__device__ __forceinline__ int64_t token_at(const EmbedParams &p, int64_t i)
{
    return p.token_bytes == 8 ? (int64_t)__ldg(static_cast<const long long *>(p.tokens) + i)
                              : (int64_t)__ldg(static_cast<const int *>(p.tokens) + i);
}

// A thread takes one vector of columns of kEmbedRows rows: their tokens are read together, then
// their table rows.
constexpr int kEmbedRows = 4;

template <typename T, int V>
__global__ void __launch_bounds__(kEmbedThreads) embed_kernel(const EmbedParams p)
{
    grid_dependency_sync();
    const int64_t vecs = p.D / V;
    const int64_t i = (int64_t)blockIdx.x * kEmbedThreads + threadIdx.x;
    const int64_t m0 = i / vecs * kEmbedRows, c = (i % vecs) * V;
    int64_t tok[kEmbedRows];
#pragma unroll
    for (int k = 0; k < kEmbedRows; ++k) {
        tok[k] = m0 + k < p.M ? token_at(p, m0 + k) : -1;
        if (tok[k] >= p.V) tok[k] = -1;
    }
    Pack<T, V> o[kEmbedRows];
#pragma unroll
    for (int k = 0; k < kEmbedRows; ++k)
        o[k] = tok[k] >= 0 ? load_pack<T, V>(static_cast<const T *>(p.table) + tok[k] * p.ld + c)
                           : zero_pack<T, V>();
#pragma unroll
    for (int k = 0; k < kEmbedRows; ++k) {
        if (m0 + k >= p.M) break;
        // A row of padding is 0 whatever the scale is.
        if (tok[k] >= 0)
#pragma unroll
            for (int v = 0; v < V; ++v) o[k].e[v] = narrow<T>(widen(o[k].e[v]) * p.scale);
        store_pack<T, V>(static_cast<T *>(p.out) + (m0 + k) * p.out_ld + c, o[k]);
    }
}

template <int V>
__device__ __forceinline__ void write_sums(float *dst, const float (&acc)[V], float scale)
{
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int k = 0; k < V; k += 4)
            *reinterpret_cast<float4 *>(dst + k) = make_float4(
                acc[k] * scale, acc[k + 1] * scale, acc[k + 2] * scale, acc[k + 3] * scale);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) dst[k] = acc[k] * scale;
    }
}

// Rows of the table that a CTA looks through for absent tokens: 64 KB of them, or kClearRows.
constexpr int kClearRows = 128;
__host__ __device__ __forceinline__ int64_t clear_rows(int64_t D)
{
    const int64_t r = 16384 / (D > 0 ? D : 1);
    return r < 1 ? 1 : (r > kClearRows ? kClearRows : r);
}

// Threads that take one run's columns: a power of two that holds them, 8 to kEmbedThreads.
constexpr int kRunGroups = kEmbedThreads / 8;
__host__ __device__ __forceinline__ int run_threads(int64_t vecs)
{
    int w = 8;
    while (w < vecs && w < kEmbedThreads) w *= 2;
    return w;
}

// The first `run_ctas` CTAs: one run of sorted pairs and kEmbedThreads vectors of columns each.
// Which rows to add and where the segments end is in shared memory before the first row is
// read, so a batch of rows is in flight at a time. The other CTAs write the absent rows.
template <typename T, int V>
__global__ void __launch_bounds__(kEmbedThreads) embed_runs_kernel(const EmbedParams p,
                                                                   int64_t run_ctas)
{
    constexpr int U = 8;
    __shared__ uint32_t all_keys[kRunGroups][kRun + 2], all_pos[kRunGroups][kRun];
    grid_dependency_sync();
    if (blockIdx.x >= run_ctas) {
        const int64_t rows = clear_rows(p.D), v0 = (blockIdx.x - run_ctas) * rows;
        constexpr int W = V % 4 == 0 ? 4 : 1;
        __shared__ uint8_t there[kClearRows];
        for (int i = threadIdx.x; i < rows; i += kEmbedThreads)
            there[i] = v0 + i < p.V ? (p.M > 0 ? __ldcg(p.present + v0 + i) : 0) : 1;
        __syncthreads();
        // Each warp takes every fourth row.
        for (int i = threadIdx.x >> 5; i < rows; i += kEmbedThreads / 32) {
            if (there[i]) continue;
            const int64_t v = v0 + i;
            for (int64_t c = (threadIdx.x & 31) * W; c < p.D; c += 32 * W) {
                if constexpr (W == 4)
                    *reinterpret_cast<float4 *>(p.dtable + v * p.D + c) =
                        make_float4(0.f, 0.f, 0.f, 0.f);
                else
                    p.dtable[v * p.D + c] = 0.f;
            }
        }
        return;
    }
    // Narrow rows: several runs to a CTA, `wide` threads each.
    const int wide = run_threads(p.D / V), group = threadIdx.x / wide;
    const int64_t col_blocks = (p.D / V + wide - 1) / wide;
    const int64_t runs = (p.M + kRun - 1) / kRun;
    const int64_t run0 = blockIdx.x / col_blocks * (kEmbedThreads / wide);
    const int64_t c = (blockIdx.x % col_blocks * wide + threadIdx.x % wide) * V;
    for (int k = threadIdx.x; k < kEmbedThreads / wide * (kRun + 2); k += kEmbedThreads) {
        const int g = k / (kRun + 2), j = k % (kRun + 2);  // the pair before the run is j = 0
        const int64_t i = (run0 + g) * kRun + j - 1;
        const uint2 q = i >= 0 && i < p.M ? __ldcg(p.pairs[0] + i) : make_uint2(~0u, 0u);
        all_keys[g][j] = q.x;  // ~0: no token
        // Past the last pair, and for padding, any row will do: it is read but not added.
        if (j > 0 && j <= kRun) all_pos[g][j - 1] = q.y;
    }
    __syncthreads();
    const int64_t run = run0 + group, lo = run * kRun;
    if (c >= p.D || run >= runs) return;
    const uint32_t *skey = all_keys[group], *spos = all_pos[group];
    const int n = (int)(p.M - lo < kRun ? p.M - lo : kRun);
    const T *rows = static_cast<const T *>(p.dout) + c;
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
    bool head = skey[0] == skey[1];  // the segment came in from an earlier run
    for (int i0 = 0; i0 < n; i0 += U) {
        if (skey[i0 + 1] >= p.V) break;  // sorted last: no row of the table
        Pack<T, V> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            r[u] = load_pack<T, V>(rows + (int64_t)spos[i0 + u] * p.ld);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u;
            if (i >= n) break;
            const uint32_t key = skey[i + 1];
            if (key >= p.V) break;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += widen(r[u].e[k]);
            const bool same = skey[i + 2] == key;
            if (same && i + 1 < n) continue;
            if (head)
                write_sums<V>(p.partial + (run * 2 + 0) * p.D + c, acc, 1.f);
            else if (same)
                write_sums<V>(p.partial + (run * 2 + 1) * p.D + c, acc, 1.f);
            else
                write_sums<V>(p.dtable + (int64_t)key * p.D + c, acc, p.scale);
            head = false;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = 0.f;
        }
    }
}

}  // namespace seq
}  // namespace rlca

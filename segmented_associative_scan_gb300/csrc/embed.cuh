// Token embedding: rows of a table, scaled; and the table's gradient, a segmented sum over
// the positions sorted by token.
//
// Gradient: the (token, position) pairs are sorted by token, stably, so the positions of a
// token stay in order. The sorted pairs are cut into runs of kRun; a CTA adds up the rows
// of one run segment by segment. A segment inside a run is written at once; what crosses
// a run's border goes to a partial row and is added up, run after run, by a last kernel. So
// the sums are taken in one fixed order whatever the GPU does, frequent tokens are spread
// over many CTAs, and no atomics are needed.
#pragma once

#include "sequence.cuh"

namespace rlca {
namespace seq {

constexpr int kEmbedThreads = 128;
constexpr int kRun = 32;               // sorted pairs of one run
constexpr int kSortCtas = 8;           // one cluster
constexpr int kSortThreads = 1024;
constexpr int kSortItems = 4;          // keys of a thread per sweep

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
    uint32_t *keys[2], *pos[2];  // ping-pong buffers of the sort; the last pass ends in [0]
    float *partial;              // [runs, 2, D]: what a run holds of the segment that came
                                 // in, and of the one that goes on
};

struct EmbedWorkspace {
    size_t keys[2], pos[2], partial, bytes;
};

inline EmbedWorkspace embed_workspace(int64_t M, int64_t D)
{
    EmbedWorkspace w;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t r = at;
        at += align256(n);
        return r;
    };
    for (int i = 0; i < 2; ++i) {
        w.keys[i] = take((size_t)M * 4);
        w.pos[i] = take((size_t)M * 4);
    }
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

template <typename T, int V>
__global__ void __launch_bounds__(kEmbedThreads) embed_kernel(const EmbedParams p)
{
    grid_dependency_sync();
    const int64_t vecs = (p.D + V - 1) / V;
    const int64_t i = (int64_t)blockIdx.x * kEmbedThreads + threadIdx.x;
    const int64_t m = i / vecs, c = (i % vecs) * V;
    if (m >= p.M) return;
    const int64_t tok = token_at(p, m);
    Pack<T, V> o = zero_pack<T, V>();
    if (tok >= 0 && tok < p.V) {
        o = load_pack<T, V>(static_cast<const T *>(p.table) + tok * p.ld + c);
#pragma unroll
        for (int k = 0; k < V; ++k) o.e[k] = narrow<T>(widen(o.e[k]) * p.scale);
    }
    store_pack<T, V>(static_cast<T *>(p.out) + m * p.out_ld + c, o);
}

// Adds V fp32 sums, scaled, to nothing: writes them.
template <int V>
__device__ __forceinline__ void write_sums(float *dst, const float (&acc)[V], float scale)
{
#pragma unroll
    for (int k = 0; k < V; ++k) dst[k] = acc[k] * scale;
}

// One run of sorted pairs and kEmbedThreads vectors of columns per CTA.
template <typename T, int V>
__global__ void __launch_bounds__(kEmbedThreads) embed_runs_kernel(const EmbedParams p)
{
    grid_dependency_sync();
    const int64_t col_blocks = (p.D / V + kEmbedThreads - 1) / kEmbedThreads;
    const int64_t run = blockIdx.x / col_blocks;
    const int64_t c = ((blockIdx.x % col_blocks) * kEmbedThreads + threadIdx.x) * V;
    const int64_t lo = run * kRun, hi = lo + kRun < p.M ? lo + kRun : p.M;
    if (c >= p.D) return;
    const uint32_t *keys = p.keys[0], *pos = p.pos[0];
    const bool comes_in = lo > 0 && __ldcg(keys + lo - 1) == __ldcg(keys + lo);
    const bool goes_on = hi < p.M && __ldcg(keys + hi) == __ldcg(keys + hi - 1);
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
    int64_t begin = lo;
    for (int64_t i = lo; i < hi; ++i) {
        const uint32_t key = __ldcg(keys + i);
        if (key >= p.V) break;  // sorted last: no row of the table
        const Pack<T, V> r = load_pack<T, V>(static_cast<const T *>(p.dout) +
                                             (int64_t)__ldcg(pos + i) * p.ld + c);
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] += widen(r.e[k]);
        if (i + 1 < hi && __ldcg(keys + i + 1) == key) continue;
        if (begin == lo && comes_in)
            write_sums<V>(p.partial + (run * 2 + 0) * p.D + c, acc, 1.f);
        else if (i + 1 == hi && goes_on)
            write_sums<V>(p.partial + (run * 2 + 1) * p.D + c, acc, 1.f);
        else
            write_sums<V>(p.dtable + (int64_t)key * p.D + c, acc, p.scale);
        begin = i + 1;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.f;
    }
}

}  // namespace seq
}  // namespace rlca

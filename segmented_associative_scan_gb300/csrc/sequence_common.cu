// Kernels of the sequence operators that do not depend on the data type: the last sums over
// rows, and the sort of tokens behind the embedding's gradient.
#include <cooperative_groups.h>

#include "conv.cuh"
#include "embed.cuh"
#include "scan.cuh"

namespace cg = cooperative_groups;

namespace rlca {
namespace seq {

constexpr int kSumGroups = 8;

__global__ void __launch_bounds__(32 * kSumGroups) sum_rows_kernel(const SumRows p)
{
    __shared__ float part[kSumGroups][32];
    grid_dependency_sync();
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    int64_t i = (int64_t)blockIdx.x * 32 + lane;
    const bool in = i < p.count[0] + p.count[1] + p.count[2];
    float sum = 0.f;
    if (in) {
        const float *src = p.src + i;
#pragma unroll 8
        for (int64_t r = group; r < p.rows; r += kSumGroups) sum += __ldcg(src + r * p.stride);
    }
    part[group][lane] = sum;
    __syncthreads();
    if (group || !in) return;
#pragma unroll
    for (int g = 1; g < kSumGroups; ++g) sum += part[g][lane];
    if (i < p.count[0]) {
        const int64_t wide = p.tap ? p.count[0] / p.tap : 0;
        if (p.dst[0]) p.dst[0][p.tap ? i % wide * p.tap + i / wide : i] = sum;
        return;
    }
    i -= p.count[0];
    if (i < p.count[1]) {
        if (p.dst[1]) p.dst[1][i] = sum;
    } else if (p.dst[2]) {
        p.dst[2][i - p.count[1]] = sum;
    }
}

cudaError_t launch_sum_rows(const SumRows &p, cudaStream_t stream)
{
    const int64_t n = p.count[0] + p.count[1] + p.count[2];
    return launch_pdl(sum_rows_kernel, (unsigned)((n + 31) / 32), 32 * kSumGroups, 0, stream, p);
}

// ------------------------------------------------------------------ spans of a scan

// A thread owns one state of one channel and walks the row's spans: on entry span_state holds
// what each span leaves from a zero state (the span walked last: not read), on exit what each
// span starts from. A span in which an episode starts passes nothing on.
template <bool REVERSE>
__global__ void __launch_bounds__(256) scan_join_kernel(const ScanParams p)
{
    grid_dependency_sync();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t es = p.E * p.S;
    const int64_t n = i / es, at = i % es;
    if (n >= p.N) return;
    const float a = kLog2e * __ldg(p.A + at);
    const float *from = REVERSE ? p.d_final : p.init;
    float carry = from ? __ldg(from + i) : 0.f;
    if (REVERSE) {
        const int len = row_length(p.rows, n, p.T);
        if (len > 0 && step_ended(p.rows, n, len - 1)) carry = 0.f;
    }
    float *state = p.span_state + n * p.spans * es + at;
    const float *sum = p.span_sum + n * p.spans * p.E + at / p.S;
#pragma unroll 4
    for (int k = 0; k + 1 < p.spans; ++k) {
        const int s = REVERSE ? p.spans - 1 - k : k;
        const float local = __ldcg(state + s * es), d = __ldcg(sum + s * p.E);
        state[s * es] = carry;
        carry = d != d ? local : fmaf(exp2_fast(d * a), carry, local);
    }
    state[(REVERSE ? 0 : p.spans - 1) * es] = carry;
}

cudaError_t launch_scan_join(const ScanParams &p, bool reverse, cudaStream_t stream)
{
    const int64_t n = p.N * p.E * p.S;
    const unsigned grid = (unsigned)((n + 255) / 256);
    return reverse ? launch_pdl(scan_join_kernel<true>, grid, 256, 0, stream, p)
                   : launch_pdl(scan_join_kernel<false>, grid, 256, 0, stream, p);
}

// ------------------------------------------------------------------ sort by token

// Stable radix sort of (token, position), 8 bits a pass, by one cluster of kSortCtas CTAs:
// CTA r owns the r-th part of the pairs. Per pass each CTA counts its digits, reads the
// other CTAs' counts through distributed shared memory to find where its pairs of every
// digit go, and then sweeps its part in order, ranking the pairs of equal digits by warp
// votes. The cluster's barrier stands between passes, so a sort is one launch.
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const EmbedParams p, int passes)
{
    constexpr int kWarps = kSortThreads / 32;
    __shared__ uint32_t hist[256];
    __shared__ uint32_t base[256];
    __shared__ uint32_t wcount[kWarps][256];
    __shared__ uint32_t wsum[8];
    grid_dependency_sync();
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned rank = cluster.block_rank();
    const int64_t part = ((p.M + kSortCtas - 1) / kSortCtas + 31) / 32 * 32;
    const int64_t lo = part * rank < p.M ? part * rank : p.M;
    const int64_t hi = lo + part < p.M ? lo + part : p.M;

    for (int pass = 0; pass < passes; ++pass) {
        const int shift = 8 * pass;
        // The last pass ends in buffer 0.
        const int to = (passes - 1 - pass) & 1, from = to ^ 1;
        auto key_at = [&](int64_t i) -> uint32_t {
            if (pass > 0) return __ldcg(p.keys[from] + i);
            const int64_t t = token_at(p, i);
            return t >= 0 && t < p.V ? (uint32_t)t : (uint32_t)p.V;
        };
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int64_t i = lo + tid; i < hi; i += kSortThreads)
            atomicAdd(&hist[(key_at(i) >> shift) & 255u], 1u);
        cluster.sync();
        // Where this CTA's pairs of digit d go: after all smaller digits, and after the
        // same digit's pairs of the CTAs before it.
        uint32_t total = 0, before = 0;
        if (tid < 256)
            for (unsigned r = 0; r < kSortCtas; ++r) {
                const uint32_t c = cluster.map_shared_rank(hist, r)[tid];
                if (r < rank) before += c;
                total += c;
            }
        uint32_t incl = total;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t v = __shfl_up_sync(kFullMask, incl, d);
            if (lane >= d) incl += v;
        }
        if (tid < 256 && lane == 31) wsum[warp] = incl;
        __syncthreads();
        if (tid < 256) {
            uint32_t off = incl - total + before;
            for (int w = 0; w < warp; ++w) off += wsum[w];
            base[tid] = off;
        }
        for (int64_t t0 = lo; t0 < hi; t0 += kSortThreads * kSortItems) {
            for (int i = tid; i < kWarps * 256; i += kSortThreads) (&wcount[0][0])[i] = 0;
            __syncthreads();
            // A warp's pairs are consecutive: 32 * kSortItems of them, 32 at a time.
            uint32_t key[kSortItems], place[kSortItems];
            const int64_t w0 = t0 + (int64_t)warp * 32 * kSortItems + lane;
#pragma unroll
            for (int k = 0; k < kSortItems; ++k) {
                const int64_t i = w0 + k * 32;
                key[k] = i < hi ? key_at(i) : 0u;
            }
#pragma unroll
            for (int k = 0; k < kSortItems; ++k) {
                const bool in = w0 + k * 32 < hi;
                const uint32_t d = (key[k] >> shift) & 255u;
                unsigned peers = __ballot_sync(kFullMask, in);
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const unsigned v = __ballot_sync(kFullMask, (d >> b) & 1u);
                    peers &= (d >> b) & 1u ? v : ~v;
                }
                uint32_t seen = 0;
                if (in) seen = wcount[warp][d];
                __syncwarp();
                place[k] = seen + __popc(peers & ((1u << lane) - 1u));
                if (in && lane == 31 - __clz(peers)) wcount[warp][d] = place[k] + 1;
                __syncwarp();
            }
            __syncthreads();
            if (tid < 256) {
                uint32_t run = base[tid];
                for (int w = 0; w < kWarps; ++w) {
                    const uint32_t c = wcount[w][tid];
                    wcount[w][tid] = run;
                    run += c;
                }
                base[tid] = run;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kSortItems; ++k) {
                const int64_t i = w0 + k * 32;
                if (i < hi) {
                    const uint32_t at = wcount[warp][(key[k] >> shift) & 255u] + place[k];
                    p.keys[to][at] = key[k];
                    p.pos[to][at] = pass > 0 ? __ldcg(p.pos[from] + i) : (uint32_t)i;
                }
            }
            __syncthreads();
        }
        cluster.sync();  // the pass is written, and no CTA still reads this one's counts
    }
}

// A segment that crosses runs: the run it starts in adds up its share there and those of the
// runs it goes on into, in order.
__global__ void __launch_bounds__(kEmbedThreads) embed_join_kernel(const EmbedParams p)
{
    grid_dependency_sync();
    const int64_t col_blocks = (p.D + kEmbedThreads - 1) / kEmbedThreads;
    const int64_t run = blockIdx.x / col_blocks;
    const int64_t c = (blockIdx.x % col_blocks) * kEmbedThreads + threadIdx.x;
    const uint32_t *keys = p.keys[0];
    const int64_t lo = run * kRun, hi = lo + kRun;
    if (hi >= p.M || c >= p.D) return;
    const uint32_t key = __ldcg(keys + hi - 1);
    if (key >= p.V || __ldcg(keys + hi) != key) return;  // ends here
    if (lo > 0 && __ldcg(keys + lo - 1) == key) return;  // starts in an earlier run
    float sum = __ldcg(p.partial + (run * 2 + 1) * p.D + c);
    int64_t r = run + 1;
    for (bool more = true; more; ++r) {
        sum += __ldcg(p.partial + (r * 2 + 0) * p.D + c);
        const int64_t end = (r + 1) * kRun;
        more = end < p.M && __ldcg(keys + end - 1) == key && __ldcg(keys + end) == key;
    }
    p.dtable[(int64_t)key * p.D + c] = sum * p.scale;
}

cudaError_t launch_embed_sort(const EmbedParams &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSortCtas);
    cfg.blockDim = dim3(kSortThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kSortCtas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, embed_sort_kernel, p, sort_passes(p.V));
}

cudaError_t launch_embed_join(const EmbedParams &p, cudaStream_t stream)
{
    const int64_t col_blocks = (p.D + kEmbedThreads - 1) / kEmbedThreads;
    const int64_t runs = (p.M + kRun - 1) / kRun;
    return launch_pdl(embed_join_kernel, (unsigned)(runs * col_blocks), kEmbedThreads, 0, stream,
                      p);
}

}  // namespace seq
}  // namespace rlca

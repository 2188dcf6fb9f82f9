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
    return launch_grid(sum_rows_kernel, (n + 31) / 32, 32 * kSumGroups, stream, p);
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
    const float a = __ldg(p.A + at);
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
        // A span past the row's end has d = 0 and leaves what comes in, A = -inf or not; where nothing
        // comes in, nothing does at the other end, though exp of the sum may be Inf.
        const float decay = d == 0.f ? 1.f : expf(d * a);
        carry = d != d || carry == 0.f ? local : fmaf(decay, carry, local);
    }
    state[(REVERSE ? 0 : p.spans - 1) * es] = carry;
}

cudaError_t launch_scan_join(const ScanParams &p, bool reverse, cudaStream_t stream)
{
    const int64_t n = p.N * p.E * p.S;
    const int64_t grid = (n + 255) / 256;
    return reverse ? launch_grid(scan_join_kernel<true>, grid, 256, stream, p)
                   : launch_grid(scan_join_kernel<false>, grid, 256, stream, p);
}

// ------------------------------------------------------------------ sort by token

// Stable radix sort of (token, position), 8 bits a pass, by one cluster of CTAS CTAs:
// CTA r owns the r-th part of the pairs. Per pass each warp ranks its pairs among those of the
// same digit by votes, 32 pairs at a time, the CTA's warps add up their counts, and the CTAs
// read one another's through distributed shared memory to find where their pairs of every
// digit go. The cluster's barrier stands between passes, so a sort is one launch. A part of at
// most one sweep (kSortThreads * kSortItems pairs) is read once a pass; a longer one is counted
// first and then swept in order. A pair is written as one 8-byte word: it is the scattered
// stores of a few SMs that a pass waits for. CTAS = 1: few pairs, one CTA, no cluster.
template <int CTAS>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const EmbedParams p, int passes)
{
    constexpr int kWarps = kSortThreads / 32, kSweep = kSortThreads * kSortItems;
    __shared__ uint32_t hist[256];
    __shared__ uint32_t base[256];
    __shared__ uint32_t wcount[kWarps][256];
    __shared__ uint32_t wsum[8];
    grid_dependency_sync();
    auto barrier = [] {
        if constexpr (CTAS > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
    };
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned rank = CTAS > 1 ? blockIdx.x : 0;
    const int64_t part = ((p.M + CTAS - 1) / CTAS + 31) / 32 * 32;
    const int64_t lo = part * rank < p.M ? part * rank : p.M;
    const int64_t hi = lo + part < p.M ? lo + part : p.M;
    for (int64_t i = rank * kSortThreads + tid; i < (p.V + 15) / 16; i += CTAS * kSortThreads)
        reinterpret_cast<uint4 *>(p.present)[i] = make_uint4(0u, 0u, 0u, 0u);

    // Pairs of a warp in a sweep: shared out evenly, in whole rounds of 32.
    const int per = part >= kSweep ? 32 * kSortItems
                                   : (int)((part + kWarps * 32 - 1) / (kWarps * 32)) * 32;
    uint32_t key[kSortItems], pos[kSortItems], place[kSortItems];
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = 8 * pass;
        // The last pass ends in buffer 0.
        const int to = (passes - 1 - pass) & 1, from = to ^ 1;
        auto key_at = [&](int64_t i) -> uint32_t {
            if (pass > 0) return __ldcg(p.pairs[from] + i).x;
            const int64_t t = token_at(p, i);
            return t >= 0 && t < p.V ? (uint32_t)t : (uint32_t)p.V;
        };
        // A warp's pairs of a sweep are consecutive, `per` of them. Leaves each
        // pair's place among its warp's pairs of the digit, and in wcount the warps' counts.
        auto sweep = [&](int64_t t0) {
            const int64_t w0 = t0 + (int64_t)warp * per + lane;
            const int64_t end = t0 + (int64_t)(warp + 1) * per, we = end < hi ? end : hi;
            // All of a thread's loads first: one loop for each kind of source.
            if (pass > 0) {
#pragma unroll
                for (int k = 0; k < kSortItems; ++k) {
                    uint2 q = make_uint2(0u, 0u);
                    if (w0 + k * 32 < we) q = __ldcg(p.pairs[from] + w0 + k * 32);
                    key[k] = q.x, pos[k] = q.y;
                }
            } else {
                auto read = [&](auto *tokens) {
                    std::remove_cv_t<std::remove_pointer_t<decltype(tokens)>> t;
#pragma unroll
                    for (int k = 0; k < kSortItems; ++k) {
                        t = -1;
                        if (w0 + k * 32 < we) t = __ldg(tokens + w0 + k * 32);
                        key[k] = t >= 0 && t < p.V ? (uint32_t)t : (uint32_t)p.V;
                        pos[k] = (uint32_t)(w0 + k * 32);
                    }
                };
                if (p.token_bytes == 8)
                    read(static_cast<const long long *>(p.tokens));
                else
                    read(static_cast<const int *>(p.tokens));
            }
            for (int i = lane; i < 256; i += 32) wcount[warp][i] = 0;
            __syncwarp();
#pragma unroll
            for (int k = 0; k < kSortItems; ++k) {
                if (w0 - lane + k * 32 >= we) break;  // the whole warp
                const bool in = w0 + k * 32 < we;
                const uint32_t d = (key[k] >> shift) & 255u;
                unsigned peers = __ballot_sync(kFullMask, in);
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const unsigned v = __ballot_sync(kFullMask, (d >> b) & 1u);
                    peers &= (d >> b) & 1u ? v : ~v;
                }
                const uint32_t seen = in ? wcount[warp][d] : 0;
                __syncwarp();
                place[k] = seen + __popc(peers & ((1u << lane) - 1u));
                if (in && lane == 31 - __clz(peers)) wcount[warp][d] = place[k] + 1;
                __syncwarp();
            }
            __syncthreads();
        };
        // Turns the warps' counts of every digit into what stands before each warp; returns
        // the sum over warps (of digit tid).
        auto add_warps = [&]() {
            uint32_t run = 0, c[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) c[w] = wcount[w][tid];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                wcount[w][tid] = run;
                run += c[w];
            }
            return run;
        };
        auto scatter = [&](int64_t t0) {
            const int64_t w0 = t0 + (int64_t)warp * per + lane;
            const int64_t end = t0 + (int64_t)(warp + 1) * per, we = end < hi ? end : hi;
#pragma unroll
            for (int k = 0; k < kSortItems; ++k) {
                if (w0 + k * 32 >= we) continue;
                const uint32_t d = (key[k] >> shift) & 255u;
                const uint32_t at = base[d] + wcount[warp][d] + place[k];
                p.pairs[to][at] = make_uint2(key[k], pos[k]);
            }
        };

        const bool once = part <= kSweep;
        if (once) {
            sweep(lo);
            if (tid < 256) hist[tid] = add_warps();
        } else {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int64_t i = lo + tid; i < hi; i += kSortThreads)
                atomicAdd(&hist[(key_at(i) >> shift) & 255u], 1u);
        }
        barrier();
        // Where this CTA's pairs of digit d go: after all smaller digits, and after the
        // same digit's pairs of the CTAs before it.
        uint32_t total = 0, before = 0;
        if (tid < 256) {
            uint32_t c[CTAS];
#pragma unroll
            for (unsigned r = 0; r < CTAS; ++r)
                c[r] = CTAS > 1 ? cg::this_cluster().map_shared_rank(hist, r)[tid] : hist[tid];
#pragma unroll
            for (unsigned r = 0; r < CTAS; ++r) {
                if (r < rank) before += c[r];
                total += c[r];
            }
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
        __syncthreads();
        if (once) {
            scatter(lo);
        } else {
            for (int64_t t0 = lo; t0 < hi; t0 += kSweep) {
                sweep(t0);
                uint32_t count = 0;
                if (tid < 256) count = add_warps();
                __syncthreads();
                scatter(t0);
                __syncthreads();
                if (tid < 256) base[tid] += count;
                __syncthreads();
            }
        }
        barrier();  // the pass is written, and no CTA still reads this one's counts
    }
    // Which tokens occur: the first pair of every token marks its row.
    for (int64_t i0 = lo + tid; i0 < hi; i0 += 8 * kSortThreads) {
        uint32_t k[8], before[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int64_t i = i0 + u * kSortThreads;
            k[u] = i < hi ? __ldcg(p.pairs[0] + i).x : ~0u;
            before[u] = i < hi && i > 0 ? __ldcg(p.pairs[0] + i - 1).x : ~0u;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (k[u] < p.V && k[u] != before[u]) p.present[k[u]] = 1;
    }
}

// A segment that crosses runs: the run it starts in adds up its share there and those of the
// runs it goes on into. A warp takes a run and 128 columns; it looks at the first pairs of 32
// following runs at a time to see how far the segment goes. A segment of more than 32 further
// runs is left to the whole CTA: warp w takes the further runs in blocks of 32, w, w + 8, ...,
// and the warps' sums are added in order.
constexpr int kJoinWarps = 8;

__global__ void __launch_bounds__(32 * kJoinWarps) embed_join_kernel(const EmbedParams p)
{
    constexpr int U = 8;
    __shared__ int longer[kJoinWarps];
    __shared__ float part[kJoinWarps][128];
    grid_dependency_sync();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col_blocks = (p.D + 127) / 128;
    const int64_t run0 = (int64_t)(blockIdx.x / col_blocks) * kJoinWarps;
    const int64_t c = blockIdx.x % col_blocks * 128 + lane;
    auto key_of = [&](int64_t i) { return __ldcg(p.pairs[0] + i).x; };
    bool in[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) in[k] = c + 32 * k < p.D;

    // The key of a segment that starts in `run` and goes on, or ~0.
    auto starts = [&](int64_t run) -> uint32_t {
        const int64_t lo = run * kRun, hi = lo + kRun;
        if (hi >= p.M) return ~0u;
        const uint32_t key = key_of(hi - 1), next = key_of(hi);
        const uint32_t before = lo > 0 ? key_of(lo - 1) : ~0u;
        return key < p.V && next == key && before != key ? key : ~0u;
    };
    // How many of the 32 runs from r0 on begin with `key`, from the first on.
    auto further = [&](int64_t r0, uint32_t key) {
        const int64_t at = (r0 + lane) * kRun;
        const unsigned goes = __ballot_sync(kFullMask, at < p.M && key_of(at) == key);
        return goes == kFullMask ? 32 : __ffs(~goes) - 1;
    };
    auto add_runs = [&](int64_t r0, int n, float (&sum)[4]) {
        for (int r = 0; r < n; r += U) {
            float v[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[u][k] = in[k] && r + u < n
                                  ? __ldcg(p.partial + (r0 + r + u) * 2 * p.D + c + 32 * k)
                                  : 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < 4; ++k) sum[k] += v[u][k];
        }
    };
    auto own_share = [&](int64_t run, float (&sum)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            sum[k] = in[k] ? __ldcg(p.partial + (run * 2 + 1) * p.D + c + 32 * k) : 0.f;
    };

    const int64_t run = run0 + warp;
    const uint32_t key = starts(run);
    int n = 0;
    if (key != ~0u) n = further(run + 1, key);
    if (lane == 0) longer[warp] = n == 32;
    if (n > 0 && n < 32) {
        float sum[4];
        own_share(run, sum);
        add_runs(run + 1, n, sum);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (in[k]) p.dtable[(int64_t)key * p.D + c + 32 * k] = sum[k] * p.scale;
    }
    __syncthreads();
    for (int w = 0; w < kJoinWarps; ++w) {
        if (!longer[w]) continue;
        const uint32_t k0 = starts(run0 + w);
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        if (warp == 0) own_share(run0 + w, sum);
        for (int64_t r0 = run0 + w + 1 + 32 * warp;; r0 += 32 * kJoinWarps) {
            const int m = further(r0, k0);
            add_runs(r0, m, sum);
            if (m < 32) break;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) part[warp][lane + 32 * k] = sum[k];
        __syncthreads();
        const int64_t col = blockIdx.x % col_blocks * 128 + threadIdx.x;
        if (threadIdx.x < 128 && col < p.D) {
            float all = part[0][threadIdx.x];
#pragma unroll
            for (int i = 1; i < kJoinWarps; ++i) all += part[i][threadIdx.x];
            p.dtable[(int64_t)k0 * p.D + col] = all * p.scale;
        }
        __syncthreads();
    }
}

cudaError_t launch_embed_sort(const EmbedParams &p, cudaStream_t stream)
{
    // Measured, 13 bits, the whole gradient, us, one CTA / the cluster: 1 token 12.2 / 14.8, 2048
    // 15.0 / 15.5, 4096 19.7 / 16.1.
    if (p.M <= kSortThreads * kSortItems / 2)
        return launch_grid(embed_sort_kernel<1>, 1, kSortThreads, stream, p, sort_passes(p.V));
    // 16 CTAs are more than every GPU's clusters hold: the kernel has to ask, once per device.
    static std::atomic<bool> asked[kMaxDevices];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= kMaxDevices || !asked[dev].load(std::memory_order_relaxed)) {
        err = cudaFuncSetAttribute(embed_sort_kernel<kSortCtas>,
                                   cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (err != cudaSuccess) return err;
        if (dev < kMaxDevices) asked[dev].store(true, std::memory_order_relaxed);
    }
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
    return cudaLaunchKernelEx(&cfg, embed_sort_kernel<kSortCtas>, p, sort_passes(p.V));
}

cudaError_t launch_embed_join(const EmbedParams &p, cudaStream_t stream)
{
    const int64_t col_blocks = (p.D + 127) / 128;
    const int64_t blocks = ((p.M + kRun - 1) / kRun + kJoinWarps - 1) / kJoinWarps;
    return launch_grid(embed_join_kernel, blocks * col_blocks, 32 * kJoinWarps, stream, p);
}

}  // namespace seq
}  // namespace rlca

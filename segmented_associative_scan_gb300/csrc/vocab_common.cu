// The part of the preference loss that does not depend on the data type: sums over the steps of
// a pair's rows, and the loss of their difference.
#include "vocab.cuh"

namespace rlca {
namespace seq {

constexpr int kPairThreads = 256;

// A CTA owns a pair; the first half of its threads sums the preferred answer's steps, the second
// half the other's. A score is a small difference of long sums, so the log ratios are added
// in 64 bits (T / 128 additions a thread: nothing beside the rows of logits behind them).
__global__ void __launch_bounds__(kPairThreads) vocab_pair_kernel(const PairParams p)
{
    constexpr int HALF = kPairThreads / 2, WARPS = HALF / 32;
    __shared__ double sums[2][WARPS];
    __shared__ int counts[2][WARPS];
    grid_dependency_sync();
    const int64_t pairs = p.N / 2;
    const int side = threadIdx.x / HALF, tid = threadIdx.x % HALF;
    const int64_t n = blockIdx.x + side * pairs;
    double sum = 0.0;
    int count = 0;
    for (int64_t t = tid; t < p.T && inside_row(p, n, t); t += HALF) {
        const int64_t token = vocab_token(p, n, t);
        if (token < 0 || token >= p.V) continue;
        const float logp = __ldcg(p.logp + n * p.T + t);
        // A row of logits without an allowed token does not count.
        if (__ldcg(p.saved + 2 * (n * p.T + t)) == -INFINITY) continue;
        sum += p.ref_logp.ptr ? (double)logp - (double)at(p.ref_logp, n, t) : (double)logp;
        ++count;
    }
#pragma unroll
    for (int w = 16; w >= 1; w /= 2) {
        sum += __shfl_xor_sync(kFullMask, sum, w);
        count += __shfl_xor_sync(kFullMask, count, w);
    }
    if ((tid & 31) == 0) {
        sums[side][tid >> 5] = sum;
        counts[side][tid >> 5] = count;
    }
    __syncthreads();
    if (threadIdx.x) return;
    double score[2], by_logp[2];
    for (int s = 0; s < 2; ++s) {
        sum = 0.0;
        count = 0;
        for (int w = 0; w < WARPS; ++w) {
            sum += sums[s][w];
            count += counts[s][w];
        }
        by_logp[s] = p.by_length ? (double)p.beta / (count > 0 ? count : 1) : (double)p.beta;
        score[s] = by_logp[s] * sum;
    }
    // -log sigmoid(x) = max(-x, 0) + log(1 + e^-|x|); by x: smoothing - sigmoid(-x).
    const double x = score[0] - score[1];
    const double e = exp(-fabs(x)), tail = log1p(e);
    const double eps = p.smoothing;
    const double down = x < 0.0 ? -x : 0.0, up = x < 0.0 ? 0.0 : x;
    // A NaN comes through `tail`; an infinite side without a share adds nothing.
    double loss = tail;
    if (eps < 1.0) loss += (1.0 - eps) * down;
    if (eps > 0.0) loss += eps * up;
    p.loss[blockIdx.x] = (float)loss;
    const double sig = (x < 0.0 ? 1.0 : e) / (1.0 + e);              // sigmoid(-x)
    for (int s = 0; s < 2; ++s) {
        const int64_t row = blockIdx.x + s * pairs;
        p.scores[row] = (float)score[s];
        if (p.slope) p.slope[row] = (float)((s ? sig - eps : eps - sig) * by_logp[s]);
    }
}

cudaError_t launch_pairs(const PairParams &p, cudaStream_t stream)
{
    return launch_grid(vocab_pair_kernel, p.N / 2, kPairThreads, stream, p);
}

}  // namespace seq
}  // namespace rlca

// Losses over a vocabulary in one data type: compiled once per format with RLCA_UNIT_FMT (the
// Fmt value) set by the build.
#include <algorithm>

#include "vocab_parked.cuh"
#include "vocab_tile.cuh"

#if !defined(RLCA_UNIT_FMT)
#error "vocab_unit.cu is compiled with -DRLCA_UNIT_FMT=<0..2>"
#endif

namespace rlca {
namespace seq {

namespace {

using T = DataType<static_cast<Fmt>(RLCA_UNIT_FMT)>::type;

constexpr int W = RowPacks<T>::W;

// Whether all rows begin on 16 bytes.
bool rows_aligned(const VocabParams &p)
{
    return reinterpret_cast<uintptr_t>(p.logits.ptr) % 16 == 0 &&
           (p.N <= 1 || p.logits.row % W == 0) && (p.T <= 1 || p.logits.step % W == 0);
}

// Most packs that a row of V elements covers.
int64_t most_packs(const VocabParams &p)
{
    return (p.V + W - 1 + (rows_aligned(p) ? 0 : W - 1)) / W;
}

// `warps` of U packs a lane to a row, in clusters of `ctas`.
template <VocabOp OP, bool ENT, bool GRAD, int U>
cudaError_t held_rows(const VocabParams &p, int warps, int ctas, cudaStream_t stream)
{
    const auto kernel = vocab_held_kernel<T, OP, ENT, GRAD, U>;
    int each = (warps + ctas - 1) / ctas;
    if (OP == VocabOp::kDistill && each < teach_warps(p.K)) each = teach_warps(p.K);
    const int smem = each * U * 32 * 16;
    if (smem > 40 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    const int fixed = (OP == VocabOp::kDistill ? 11 : 7) * 1024;  // of shared memory, at most
    const int fit = std::min(kHeldMaxThreads / 32 / each, 227 * 1024 / (smem + fixed));
    const int64_t most = (int64_t)sm_count() * fit / ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.M < most ? p.M : most) * ctas));
    cfg.blockDim = dim3(32 * each);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, ctas);
}

constexpr int kParkedBytes = 216 * 1024;  // of a row, at most

template <VocabOp OP, bool ENT, bool GRAD>
cudaError_t parked_rows(VocabParams p, int packs, cudaStream_t stream)
{
    p.even = rows_aligned(p) && p.V % W == 0;
    const auto kernel = vocab_parked_kernel<T, OP, ENT, GRAD>;
    // Four chunks to a warp or more, where that leaves it enough warps: a row costs each of them some
    // 300 instructions. Measured, two / four / eight: policy loss [16, 1024, 32768] bf16 with
    // entropy 448 / 390 / 431 us, [24, 700, 50001] fp16 402 / 403 / 410.
    const int chunks = (packs + kParkedChunk - 1) / kParkedChunk;
    const int most_warps = std::min(kParkedWarps, (chunks + 3) / 4);
    const int turns = (chunks + most_warps - 1) / most_warps;
    int warps = (chunks + turns - 1) / turns;
    if (OP == VocabOp::kDistill && warps < teach_warps(p.K)) warps = teach_warps(p.K);
    const int smem = packs * 16;
    if (smem > 40 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    const int fixed = (OP == VocabOp::kDistill ? 9 : 5) * 1024;  // of shared memory, at most
    const int fit = std::max(1, std::min(2 * kParkedWarps / warps, 227 * 1024 / (smem + fixed)));
    const int64_t most = (int64_t)sm_count() * fit;
    return launch_pdl(kernel, (unsigned)(p.M < most ? p.M : most), 32 * warps, smem, stream, p);
}

// Whether the rows of a tile lie one behind the other, and every tile begins on 16 bytes.
bool tiles_are_linear(const VocabParams &p, const rlca_steps &a)
{
    return reinterpret_cast<uintptr_t>(a.ptr) % 16 == 0 && (p.T <= 1 || a.step == p.V) &&
           (p.N <= 1 || a.row == p.T * p.V);
}

template <VocabOp OP, bool ENT, bool GRAD, int A>
cudaError_t tile_rows(const VocabParams &p, cudaStream_t stream)
{
    TileShape sh;
    const int V = (int)p.V, most = TileLane<T, A>::most;
    sh.group = 1;
    while (sh.group * most < V && !(A == 1 && V <= 32)) sh.group *= 2;
    const int least = 32 / sh.group;
    sh.rows = std::max(least, std::min<int>(32, kTileBytes / (V * (int)sizeof(T))) / least * least);
    // Tiles begin on 16 bytes where their rows come to that.
    const bool even = (int64_t)sh.rows * V * sizeof(T) % 16 == 0;
    sh.linear = (even && tiles_are_linear(p, p.logits) ? 1 : 0) |
                (even && p.grad.ptr && tiles_are_linear(p, p.grad) ? 2 : 0);
    sh.bytes = 512 + (sh.rows * V * (int)sizeof(T) + 15) / 16 * 16;
    const int64_t tiles = (p.M + sh.rows - 1) / sh.rows;
    return launch_pdl(vocab_tile_kernel<T, OP, ENT, GRAD, A>,
                      (unsigned)((tiles + kTileWarps - 1) / kTileWarps), 32 * kTileWarps,
                      kTileWarps * sh.bytes, stream, p, sh);
}

// Rows short enough for a group of lanes.
bool short_rows(const VocabParams &p)
{
    return p.V <= 32 * (p.V % W ? TileLane<T, 1>::most : TileLane<T, W>::most);
}

template <VocabOp OP, bool ENT, bool GRAD>
cudaError_t short_rows(const VocabParams &p, cudaStream_t stream)
{
    return p.V % W ? tile_rows<OP, ENT, GRAD, 1>(p, stream) : tile_rows<OP, ENT, GRAD, W>(p, stream);
}

template <VocabOp OP, bool ENT, bool GRAD>
cudaError_t rows(const VocabParams &p, cudaStream_t stream)
{
    if constexpr (OP != VocabOp::kDistill) {
        if (short_rows(p)) return short_rows<OP, ENT, GRAD>(p, stream);
    }
    const int64_t packs = most_packs(p);
    const int64_t warps = (packs + 255) / 256, thin = (packs + 63) / 64;
    // Few rows: four times the warps to each, in clusters.
    if (thin <= kHeldMaxWarps && p.M * warps <= 4 * sm_count())
        return held_rows<OP, ENT, GRAD, 2>(p, (int)thin, (int)std::min<int64_t>(8, (thin + 7) / 8),
                                           stream);
    if (packs * 16 <= kParkedBytes) return parked_rows<OP, ENT, GRAD>(p, (int)packs, stream);
    if (warps <= kHeldMaxWarps)
        return held_rows<OP, ENT, GRAD, 8>(p, (int)warps,
                                           warps <= 32 ? 1 : (int)(warps + 15) / 16, stream);
    return launch_grid(vocab_stream_kernel<T, OP, ENT, GRAD>, p.M, kStreamThreads, stream, p);
}

template <VocabOp OP, bool ENT>
cudaError_t rows(const VocabParams &p, cudaStream_t stream)
{
    if constexpr (OP == VocabOp::kLogp) return rows<OP, ENT, false>(p, stream);
    else return p.grad.ptr ? rows<OP, ENT, true>(p, stream) : rows<OP, ENT, false>(p, stream);
}

}  // namespace

template <Fmt F>
cudaError_t launch_vocab(const VocabParams &p, VocabOp op, bool entropy, cudaStream_t stream)
{
    switch (op) {
    case VocabOp::kLogp:
        return entropy ? rows<VocabOp::kLogp, true>(p, stream)
                       : rows<VocabOp::kLogp, false>(p, stream);
    case VocabOp::kPolicy:
        return entropy ? rows<VocabOp::kPolicy, true>(p, stream)
                       : rows<VocabOp::kPolicy, false>(p, stream);
    default: return rows<VocabOp::kDistill, false>(p, stream);
    }
}

template <Fmt F>
cudaError_t launch_vocab_slope(const VocabParams &p, cudaStream_t stream)
{
    if (short_rows(p))
        return p.dentropy.ptr ? short_rows<VocabOp::kSlope, true, true>(p, stream)
                              : short_rows<VocabOp::kSlope, false, true>(p, stream);
    const int64_t warps = (most_packs(p) + 32 * kSlopePacks - 1) / (32 * kSlopePacks);
    const int64_t grid = (p.M * warps + kSlopeWarps - 1) / kSlopeWarps;
    const auto kernel = p.dentropy.ptr ? vocab_slope_kernel<T, true> : vocab_slope_kernel<T, false>;
    return launch_grid(kernel, grid, 32 * kSlopeWarps, stream, p, (int)warps);
}

template cudaError_t launch_vocab<static_cast<Fmt>(RLCA_UNIT_FMT)>(const VocabParams &, VocabOp,
                                                                   bool, cudaStream_t);
template cudaError_t launch_vocab_slope<static_cast<Fmt>(RLCA_UNIT_FMT)>(const VocabParams &,
                                                                         cudaStream_t);

}  // namespace seq
}  // namespace rlca

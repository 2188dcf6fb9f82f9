// Losses over a vocabulary in one data type: compiled once per format and operator with RLCA_UNIT_FMT
// (the Fmt value) and RLCA_UNIT_PART (the VocabOp value) set by the build.
#include <algorithm>

#include "vocab_held.cuh"
#include "vocab_parked.cuh"
#include "vocab_tile.cuh"

#if !defined(RLCA_UNIT_FMT) || !defined(RLCA_UNIT_PART)
#error "vocab_unit.cu is compiled with -DRLCA_UNIT_FMT=<0..2> -DRLCA_UNIT_PART=<0..3>"
#endif

namespace rlca {
namespace seq {

namespace {

using T = DataType<static_cast<Fmt>(RLCA_UNIT_FMT)>::type;

constexpr int W = 16 / (int)sizeof(T);

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
    if (p.M > INT32_MAX / ctas) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.M * ctas));
    cfg.blockDim = dim3(32 * each);
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

template <VocabOp OP, bool ENT, bool GRAD>
cudaError_t parked_rows(VocabParams p, int packs, cudaStream_t stream)
{
    p.even = rows_aligned(p) && p.V % W == 0;
    // Half an SM's shared memory at the most: two CTAs hide each other's waits. (Rows of 65536 in bf16,
    // 1 / 2 CTAs to an SM, the second parking in part: policy loss of 268 MB 117 / 102 us. A third part
    // is no gain where rows fit into a half: [24, 700, 50001] fp16 398 / 434 us.)
    const int fixed = (OP == VocabOp::kDistill ? 9 : 5) * 1024;
    const int most_room = (227 * 1024 / 2 - fixed) / 16 / kParkedChunk * kParkedChunk;
    const int room = std::min(packs, most_room), smem = room * 16;
    // Four chunks to a warp or more: a row costs each of them some 300 instructions (two / four /
    // eight: policy loss [16, 1024, 32768] bf16 with entropy 448 / 390 / 431 us). Ten warps at the
    // most, where more CTAs may fit (at most 8 / 10 / 16: [24, 700, 50001] fp16 407 / 398 / 403 us, its
    // log-probabilities 105 / 103 / 108), but where a row is more than an SM's half (rows of 131072 in
    // bf16, 10 / 16: 132 / 125 us).
    const int chunks = (packs + kParkedChunk - 1) / kParkedChunk;
    const int most_warps = std::min(room < packs ? kParkedWarps : 10, (chunks + 3) / 4);
    const int turns = (chunks + most_warps - 1) / most_warps;
    int warps = (chunks + turns - 1) / turns;
    if (OP == VocabOp::kDistill && warps < teach_warps(p.K)) warps = teach_warps(p.K);
    const auto kernel = room < packs ? vocab_parked_kernel<T, OP, ENT, GRAD, true>
                                     : vocab_parked_kernel<T, OP, ENT, GRAD, false>;
    if (smem > 40 * 1024) {
        // Always the most that any call takes: the limit is the kernel's, and another thread may launch
        // it with longer rows at the same time.
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most_room * 16);
        if (e != cudaSuccess) return e;
    }
    const int fit = std::min(32 / warps, 227 * 1024 / (smem + fixed));  // 64 registers: 32 warps
    const int64_t most = (int64_t)sm_count() * fit;
    return launch_pdl(kernel, (unsigned)(p.M < most ? p.M : most), 32 * warps, smem, stream, p, room);
}

// How the rows of a tile lie: one behind the other within a row of steps (1), or altogether (3); 4:
// every row begins on 16 bytes.
[[maybe_unused]] int tile_layout(const VocabParams &p, const rlca_steps &a)
{
    const bool steps = p.T <= 1 || a.step == p.V, all = p.N <= 1 || a.row == p.T * p.V;
    const bool even = reinterpret_cast<uintptr_t>(a.ptr) % 16 == 0 && p.V % W == 0 &&
                      (p.N <= 1 || a.row % W == 0) && (p.T <= 1 || a.step % W == 0);
    return (steps ? all ? 3 : 1 : 0) | (even ? 4 : 0);
}

// How rows of V elements are taken in tiles; no rows: they are too long for that.
TileShape tile_shape(const VocabParams &p)
{
    const int64_t V = p.V;
    TileShape sh = {};
    const int64_t packs = (V + W - 1) / W, bytes = V * (int64_t)sizeof(T);
    if (packs > 32 * kTilePacks) return sh;
    sh.step = 16;
    while (bytes % sh.step) sh.step /= 2;
    if (V % W == 0 || V > kTileOwn) {
        // Eight lanes to a row or more, which read it without bank conflicts, and four packs to
        // each.
        sh.group = 1;
        while (sh.group < packs && (sh.group < 8 || (sh.group < 32 && 4 * sh.group < packs)))
            sh.group *= 2;
    }
    // A multiple of rows that fills a turn of the warp, and that comes to 16 bytes.
    int unit = sh.group ? 32 / sh.group : 32;
    if (V % W) unit = std::max(unit, W);
    if (unit * bytes > kTileMostBytes) return sh;
    sh.rows = std::min(32, std::max(unit, (int)(kTileBytes / bytes) / unit * unit));
    // Few rows: spread over the SMs.
    while (sh.rows / 2 >= unit && p.M < (int64_t)sh.rows * 8 * sm_count()) sh.rows /= 2;
    sh.rows = sh.rows / unit * unit;
    sh.bytes = 512 + 16 + (int)(sh.rows * bytes + 15) / 16 * 16;  // and what lies past the last pack
    return sh;
}

template <VocabOp OP, bool ENT, bool GRAD>
cudaError_t tile_rows(const VocabParams &p, TileShape sh, cudaStream_t stream)
{
    sh.from = tile_layout(p, p.logits);
    sh.to = tile_layout(p, p.grad);
    const int64_t tiles = (p.M + sh.rows - 1) / sh.rows;
    const auto kernel = p.V % W == 0 ? vocab_tile_kernel<T, OP, ENT, GRAD, TileRows::kWhole>
                        : sh.group   ? vocab_tile_kernel<T, OP, ENT, GRAD, TileRows::kAny>
                                     : vocab_tile_kernel<T, OP, ENT, GRAD, TileRows::kOwn>;
    // Small CTAs fill an SM best where a tile takes much of it; a few bytes to a tile make so many
    // CTAs that their launch shows (4 Mi rows of 2 in bf16: 71 us with 2 warps, 43 with 8; 1.3 Mi
    // rows of 100: 308 with 2, 350 with 5).
    const int warps = std::min(kTileWarps, std::max(2, 16 * 1024 / sh.bytes));
    return launch_pdl(kernel, (unsigned)((tiles + warps - 1) / warps), 32 * warps, warps * sh.bytes,
                      stream, p, sh);
}

template <VocabOp OP, bool ENT, bool GRAD>
cudaError_t rows(const VocabParams &p, cudaStream_t stream)
{
    if constexpr (OP != VocabOp::kDistill) {
        const TileShape tile = tile_shape(p);
        if (tile.rows) return tile_rows<OP, ENT, GRAD>(p, tile, stream);
    }
    const int64_t packs = most_packs(p);
    const int64_t warps = (packs + 255) / 256, thin = (packs + 63) / 64;
    // Rows for two fifths of the SMs, or four warps' work for each: many warps to a row, in clusters.
    // Policy loss in bf16, clusters / a CTA to a row, us: 152 rows of 4096 2.9 / 4.8, 64 rows of 32768
    // 5.4 / 5.8, of 131072 10.5 / 13.3, 100 rows of 32768 8.7 / 5.8, of 131072 15.2 / 13.5.
    if (p.M <= sm_count() * 2 / 5 || p.M * warps <= 4 * sm_count()) {
        if (thin <= kHeldMaxWarps)
            return held_rows<OP, ENT, GRAD, 2>(
                p, (int)thin, (int)std::min<int64_t>(8, (thin + 7) / 8), stream);
        if (warps <= kHeldMaxWarps)
            return held_rows<OP, ENT, GRAD, 8>(
                p, (int)warps, (int)std::min<int64_t>(8, (warps + 7) / 8), stream);
    }
    return parked_rows<OP, ENT, GRAD>(p, (int)packs, stream);
}

template <VocabOp OP>
cudaError_t slopes(const VocabParams &p, bool entropy, cudaStream_t stream)
{
    const TileShape tile = tile_shape(p);
    if (tile.rows)
        return entropy ? tile_rows<OP, true, true>(p, tile, stream)
                       : tile_rows<OP, false, true>(p, tile, stream);
    const int64_t warps = (most_packs(p) + 32 * kSlopePacks<T> - 1) / (32 * kSlopePacks<T>);
    const int64_t grid = (p.M * warps + kSlopeWarps - 1) / kSlopeWarps;
    const auto kernel = entropy ? vocab_slope_kernel<T, true> : vocab_slope_kernel<T, false>;
    return launch_grid(kernel, grid, 32 * kSlopeWarps, stream, p, (int)warps);
}

}  // namespace

template <Fmt F, VocabOp OP>
cudaError_t launch_vocab(const VocabParams &p, bool entropy, cudaStream_t stream)
{
    if constexpr (OP == VocabOp::kSlope)
        return slopes<OP>(p, entropy, stream);
    else if constexpr (OP == VocabOp::kLogp)
        return entropy ? rows<OP, true, false>(p, stream) : rows<OP, false, false>(p, stream);
    else if constexpr (OP == VocabOp::kDistill)
        return p.grad.ptr ? rows<OP, false, true>(p, stream) : rows<OP, false, false>(p, stream);
    else if (entropy)
        return p.grad.ptr ? rows<OP, true, true>(p, stream) : rows<OP, true, false>(p, stream);
    else
        return p.grad.ptr ? rows<OP, false, true>(p, stream) : rows<OP, false, false>(p, stream);
}

template cudaError_t launch_vocab<static_cast<Fmt>(RLCA_UNIT_FMT),
                                  static_cast<VocabOp>(RLCA_UNIT_PART)>(const VocabParams &, bool,
                                                                        cudaStream_t);

}  // namespace seq
}  // namespace rlca

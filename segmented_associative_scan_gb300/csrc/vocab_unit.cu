// Losses over a vocabulary in one data type: compiled once per format with RLCA_UNIT_FMT (the
// Fmt value) set by the build.
#include "vocab.cuh"
#include "vocab_held.cuh"

#if !defined(RLCA_UNIT_FMT)
#error "vocab_unit.cu is compiled with -DRLCA_UNIT_FMT=<0..2>"
#endif

namespace rlca {
namespace seq {

namespace {

using T = DataType<static_cast<Fmt>(RLCA_UNIT_FMT)>::type;

constexpr int W = RowPacks<T>::W;

// Most packs that a row of V elements covers.
int64_t most_packs(const VocabParams &p)
{
    const bool even = reinterpret_cast<uintptr_t>(p.logits.ptr) % 16 == 0 &&
                      (p.N <= 1 || p.logits.row % W == 0) && (p.T <= 1 || p.logits.step % W == 0);
    return (p.V + W - 1 + (even ? 0 : W - 1)) / W;
}

template <VocabOp OP, bool ENT, bool GRAD, int U, int MIN>
cudaError_t held_rows(VocabParams p, int packs, int ctas, cudaStream_t stream)
{
    p.share = held_share(packs, ctas * kHeldWarps);
    const auto kernel = vocab_held_kernel<T, OP, ENT, GRAD, U, MIN>;
    if (ctas > 8) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    const int64_t most = (int64_t)sm_count() * MIN / ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.M < most ? p.M : most) * ctas));
    cfg.blockDim = dim3(kHeldThreads);
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
cudaError_t rows(const VocabParams &p, cudaStream_t stream)
{
    const int packs = (int)most_packs(p);
    auto share = [&](int ctas) { return held_share(packs, ctas * kHeldWarps); };
    int ctas = 1;
    while (ctas <= 8 && share(ctas) > 32 * 8) ++ctas;
    if (ctas > 8) ctas = 16;
    // Few rows: more CTAs to each, while their warps have a pack for every lane.
    while (2 * ctas <= 8 && p.M * ctas * 2 <= sm_count() && share(2 * ctas) >= 32) ctas *= 2;
    if (share(ctas) <= 32 * 2) return held_rows<OP, ENT, GRAD, 2, 4>(p, packs, ctas, stream);
    if (share(ctas) <= 32 * 4) return held_rows<OP, ENT, GRAD, 4, 4>(p, packs, ctas, stream);
    if (share(ctas) <= 32 * 8) return held_rows<OP, ENT, GRAD, 8, 3>(p, packs, ctas, stream);
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
    const int64_t grid = p.M * slope_blocks(p.V, RowPacks<T>::W);
    return p.dentropy.ptr
               ? launch_grid(vocab_slope_kernel<T, true>, grid, kSlopeThreads, stream, p)
               : launch_grid(vocab_slope_kernel<T, false>, grid, kSlopeThreads, stream, p);
}

template cudaError_t launch_vocab<static_cast<Fmt>(RLCA_UNIT_FMT)>(const VocabParams &, VocabOp,
                                                                   bool, cudaStream_t);
template cudaError_t launch_vocab_slope<static_cast<Fmt>(RLCA_UNIT_FMT)>(const VocabParams &,
                                                                         cudaStream_t);

}  // namespace seq
}  // namespace rlca

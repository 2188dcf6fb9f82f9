// Losses over a vocabulary in one data type: compiled once per format with RLCA_UNIT_FMT (the
// Fmt value) set by the build.
#include "vocab.cuh"

#if !defined(RLCA_UNIT_FMT)
#error "vocab_unit.cu is compiled with -DRLCA_UNIT_FMT=<0..2>"
#endif

namespace rlca {
namespace seq {

namespace {

using T = DataType<static_cast<Fmt>(RLCA_UNIT_FMT)>::type;

template <VocabOp OP, bool ENT, bool GRAD>
cudaError_t rows(const VocabParams &p, cudaStream_t stream)
{
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

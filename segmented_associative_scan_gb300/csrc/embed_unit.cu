// Token embedding in one data type: compiled once per format with RLCA_UNIT_FMT (the Fmt
// value) set by the build.
#include "embed.cuh"

#if !defined(RLCA_UNIT_FMT)
#error "embed_unit.cu is compiled with -DRLCA_UNIT_FMT=<0..2>"
#endif

namespace rlca {
namespace seq {

namespace {

using T = DataType<static_cast<Fmt>(RLCA_UNIT_FMT)>::type;

template <int V>
cudaError_t lookup(const EmbedParams &p, cudaStream_t stream)
{
    const int64_t n = (p.M + kEmbedRows - 1) / kEmbedRows * (p.D / V);
    return launch_grid(embed_kernel<T, V>, (n + kEmbedThreads - 1) / kEmbedThreads,
                      kEmbedThreads, stream, p);
}

template <int V>
cudaError_t runs(const EmbedParams &p, cudaStream_t stream)
{
    const int wide = run_threads(p.D / V), groups = kEmbedThreads / wide;
    const int64_t col_blocks = (p.D / V + wide - 1) / wide;
    const int64_t runs = ((p.M + kRun - 1) / kRun + groups - 1) / groups * col_blocks;
    const int64_t clears = (p.V + clear_rows(p.D) - 1) / clear_rows(p.D);
    return launch_grid(embed_runs_kernel<T, V>, runs + clears, kEmbedThreads, stream,
                      p, runs);
}

}  // namespace

template <Fmt F>
cudaError_t launch_embed(const EmbedParams &p, bool vec, cudaStream_t stream)
{
    return vec ? lookup<vec_of<T>()>(p, stream) : lookup<1>(p, stream);
}

template <Fmt F>
cudaError_t launch_embed_sum(const EmbedParams &p, bool vec, cudaStream_t stream)
{
    return vec ? runs<vec_of<T>()>(p, stream) : runs<1>(p, stream);
}

template cudaError_t launch_embed<static_cast<Fmt>(RLCA_UNIT_FMT)>(const EmbedParams &, bool,
                                                                   cudaStream_t);
template cudaError_t launch_embed_sum<static_cast<Fmt>(RLCA_UNIT_FMT)>(const EmbedParams &, bool,
                                                                       cudaStream_t);

}  // namespace seq
}  // namespace rlca

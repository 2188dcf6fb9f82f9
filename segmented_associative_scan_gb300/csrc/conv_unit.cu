// Causal convolution in one data type: compiled once per format with RLCA_UNIT_FMT (the
// Fmt value) set by the build.
#include "conv.cuh"

#if !defined(RLCA_UNIT_FMT)
#error "conv_unit.cu is compiled with -DRLCA_UNIT_FMT=<0..2>"
#endif

namespace rlca {
namespace seq {

namespace {

using T = DataType<static_cast<Fmt>(RLCA_UNIT_FMT)>::type;

// One kernel for each number of taps: the windows are registers, and one kernel for all of them
// took 103 us in place of 44 forward and 448 in place of 91 backward ([16, 1024, 2048], 4 taps).
template <int V, int K = RLCA_CONV_MAX_K>
cudaError_t forward(const ConvParams &p, cudaStream_t stream)
{
    if constexpr (K > 1)
        if (p.K < K) return forward<V, K - 1>(p, stream);
    const int64_t lane_blocks = (p.E / V + 31) / 32;
    const int64_t grid = p.N * (p.T ? conv_span_blocks(p.T) : 1) * lane_blocks;
    return launch_grid(conv_forward_kernel<T, V, K>, grid, kConvThreads, stream, p);
}

template <int V, int K = RLCA_CONV_MAX_K>
cudaError_t backward(const ConvParams &p, cudaStream_t stream)
{
    if constexpr (K > 1)
        if (p.K < K) return backward<V, K - 1>(p, stream);
    const int64_t lane_blocks = (p.E / V + 31) / 32;
    const int64_t grid = p.N * conv_span_blocks(p.T) * lane_blocks;
    return launch_grid(conv_backward_kernel<T, V, K>, grid, kConvThreads, stream, p);
}

template <int V>
cudaError_t step(const ConvParams &p, cudaStream_t stream)
{
    const int64_t lane_blocks = (p.E / V + 31) / 32;
    const int64_t grid = ((p.N + kConvWarps - 1) / kConvWarps * lane_blocks);
    return launch_grid(conv_step_kernel<T, V>, grid, kConvThreads, stream, p);
}

}  // namespace

template <Fmt F>
cudaError_t launch_conv_forward(const ConvParams &p, bool vec, cudaStream_t stream)
{
    return vec ? forward<4>(p, stream) : forward<1>(p, stream);
}

template <Fmt F>
cudaError_t launch_conv_backward(const ConvParams &p, bool vec, cudaStream_t stream)
{
    return vec ? backward<4>(p, stream) : backward<1>(p, stream);
}

template <Fmt F>
cudaError_t launch_conv_step(const ConvParams &p, bool vec, cudaStream_t stream)
{
    return vec ? step<4>(p, stream) : step<1>(p, stream);
}

template cudaError_t launch_conv_forward<static_cast<Fmt>(RLCA_UNIT_FMT)>(const ConvParams &, bool,
                                                                          cudaStream_t);
template cudaError_t launch_conv_backward<static_cast<Fmt>(RLCA_UNIT_FMT)>(const ConvParams &,
                                                                           bool, cudaStream_t);
template cudaError_t launch_conv_step<static_cast<Fmt>(RLCA_UNIT_FMT)>(const ConvParams &, bool,
                                                                       cudaStream_t);

}  // namespace seq
}  // namespace rlca

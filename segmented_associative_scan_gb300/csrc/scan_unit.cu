// Selective scan in one data type: compiled once per format with RLCA_UNIT_FMT (the Fmt
// value) set by the build.
#include "scan_backward.cuh"
#include "scan_forward.cuh"
#include "scan_step.cuh"

#if !defined(RLCA_UNIT_FMT)
#error "scan_unit.cu is compiled with -DRLCA_UNIT_FMT=<0..2>"
#endif

namespace rlca {
namespace seq {

namespace {

using T = DataType<static_cast<Fmt>(RLCA_UNIT_FMT)>::type;

template <bool BACKWARD, int V, int SL, int CPT>
cudaError_t launch_walk(ScanParams p, cudaStream_t stream)
{
    const unsigned grid = (unsigned)(p.N * p.G * p.blocks_g);
    if constexpr (BACKWARD)
        return launch_pdl(scan_backward_kernel<T, V, SL, CPT>, grid, kScanThreads, 0, stream, p);
    else
        return launch_pdl(scan_forward_kernel<T, V, SL, CPT>, grid, kScanThreads, 0, stream, p);
}

template <bool BACKWARD, int V>
cudaError_t launch_states(const ScanParams &p, cudaStream_t stream)
{
    switch (scan_state_lanes(p.S)) {
    case 1: return launch_walk<BACKWARD, V, 1, scan_lane_channels(1)>(p, stream);
    case 2: return launch_walk<BACKWARD, V, 2, scan_lane_channels(2)>(p, stream);
    case 4: return launch_walk<BACKWARD, V, 4, scan_lane_channels(4)>(p, stream);
    case 8: return launch_walk<BACKWARD, V, 8, scan_lane_channels(8)>(p, stream);
    default: return launch_walk<BACKWARD, V, 16, scan_lane_channels(16)>(p, stream);
    }
}

template <int SL>
cudaError_t launch_bc(const ScanParams &p, cudaStream_t stream)
{
    const int64_t n = p.N * p.T * p.G * 8 * SL;
    return launch_pdl(scan_bc_kernel<T, 4 * SL>, (unsigned)((n + 255) / 256), 256, 0, stream, p);
}

template <int SL>
cudaError_t launch_step(const ScanParams &p, cudaStream_t stream)
{
    const int64_t n = p.N * p.E * SL;
    return launch_pdl(scan_step_kernel<T, SL>, (unsigned)((n + 127) / 128), 128, 0, stream, p);
}

}  // namespace

template <Fmt F>
cudaError_t launch_scan_forward(const ScanParams &p, bool vec, cudaStream_t stream)
{
    return vec ? launch_states<false, vec_of<T>()>(p, stream) : launch_states<false, 1>(p, stream);
}

template <Fmt F>
cudaError_t launch_scan_backward(const ScanParams &p, bool vec, cudaStream_t stream)
{
    cudaError_t err =
        vec ? launch_states<true, vec_of<T>()>(p, stream) : launch_states<true, 1>(p, stream);
    if (err != cudaSuccess || p.T == 0) return err;
    switch (scan_state_lanes(p.S)) {
    case 1: return launch_bc<1>(p, stream);
    case 2: return launch_bc<2>(p, stream);
    case 4: return launch_bc<4>(p, stream);
    case 8: return launch_bc<8>(p, stream);
    default: return launch_bc<16>(p, stream);
    }
}

template <Fmt F>
cudaError_t launch_scan_step(const ScanParams &p, cudaStream_t stream)
{
    switch (scan_state_lanes(p.S)) {
    case 1: return launch_step<1>(p, stream);
    case 2: return launch_step<2>(p, stream);
    case 4: return launch_step<4>(p, stream);
    case 8: return launch_step<8>(p, stream);
    default: return launch_step<16>(p, stream);
    }
}

template cudaError_t launch_scan_forward<static_cast<Fmt>(RLCA_UNIT_FMT)>(const ScanParams &, bool,
                                                                          cudaStream_t);
template cudaError_t launch_scan_backward<static_cast<Fmt>(RLCA_UNIT_FMT)>(const ScanParams &,
                                                                           bool, cudaStream_t);
template cudaError_t launch_scan_step<static_cast<Fmt>(RLCA_UNIT_FMT)>(const ScanParams &,
                                                                       cudaStream_t);

}  // namespace seq
}  // namespace rlca

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

template <bool VEC, int SL>
cudaError_t forward(const ScanParams &p, cudaStream_t stream)
{
    const int64_t grid = (p.N * p.G * p.blocks_g * p.spans);
    if (p.spans > 1) {
        cudaError_t err = launch_grid(scan_forward_kernel<T, VEC, SL, true, false>, grid,
                                      kForwardThreads, stream, p);
        if (err == cudaSuccess) err = launch_scan_join(p, false, stream);
        if (err != cudaSuccess) return err;
    }
    if (p.z.ptr)
        return launch_grid(scan_forward_kernel<T, VEC, SL, false, true>, grid, kForwardThreads,
                           stream, p);
    return launch_grid(scan_forward_kernel<T, VEC, SL, false, false>, grid, kForwardThreads,
                       stream, p);
}

template <bool VEC>
cudaError_t forward(const ScanParams &p, cudaStream_t stream)
{
    switch (scan_state_lanes(p.S, 8)) {
    case 1: return forward<VEC, 1>(p, stream);
    case 2: return forward<VEC, 2>(p, stream);
    case 4: return forward<VEC, 4>(p, stream);
    default: return forward<VEC, 8>(p, stream);
    }
}

// CTAs to an SM that the registers are cut for. Four (230 registers at 16 states) run a CTA
// fastest, where no more are to be had; six keep more warps at work; eight (128 registers, some
// spilled) take a grid in one wave that six would leave a few stragglers of: only where more than
// six fit beside one another in shared memory, and the grid is one wave of those. Measured, us, four
// / six / eight, 512 steps, 704, 1024, 1152 and 2048 CTAs:
//   8 states   bf16 (5 fit)  440 / 323 / 405   501 / 533 / 706   503 / 536 / 733    924 / 852 / 1115
//              fp32 (4 fit)  578 / 595 / 946   652 / 669 / 1000  661 / 677 / 1004  1279 / 1315 / 1945
//   16 states  bf16 (7 fit)  409 / 310 / 423   472 / 482 / 450   475 / 485 / 673    866 / 777 / 875
//              fp32 (6 fit)  549 / 415 / 538   579 / 659 / 939   595 / 688 / 1002  1133 / 1061 / 1489
//   32 states  bf16 (8 fit)  469 / 395 / 520   556 / 598 / 559   558 / 606 / 573   1016 / 988 / 1036
//   64 states  bf16 (7 fit)                    717 / 820 / 628   722 / 879 / 943   1312 / 1375 / 1230
//              fp32 (7 fit)                    816 / 933 / 754   828 / 1035 / 1253 1555 / 1593 / 1490
// Between 4 and 6 the grid alone decides, as at 16 states in bf16; a grid that is little more than
// one wave of six runs up to a seventh faster at four (fp32, 1024 CTAs).
template <bool VEC, int SL, bool GATE>
cudaError_t backward(const ScanParams &p, cudaStream_t stream)
{
    constexpr int fit = backward_fit<T, SL, GATE>() < 8 ? backward_fit<T, SL, GATE>() : 8;
    const int64_t ctas = p.N * p.G * p.blocks_g * p.spans, sms = sm_count();
    if (ctas <= 4 * sms)
        return launch_grid(scan_backward_kernel<T, VEC, SL, GATE, 4>, ctas, kBackwardThreads,
                           stream, p);
    if constexpr (VEC && fit > 6) {
        if (ctas > 6 * sms && ctas <= fit * sms)
            return launch_grid(scan_backward_kernel<T, VEC, SL, GATE, 8>, ctas, kBackwardThreads,
                               stream, p);
    }
    return launch_grid(scan_backward_kernel<T, VEC, SL, GATE, 6>, ctas, kBackwardThreads, stream,
                       p);
}

template <bool VEC, int SL>
cudaError_t backward(const ScanParams &p, cudaStream_t stream)
{
    return p.z.ptr ? backward<VEC, SL, true>(p, stream) : backward<VEC, SL, false>(p, stream);
}

template <bool VEC>
cudaError_t backward(const ScanParams &p, cudaStream_t stream)
{
    switch (scan_backward_lanes(p.S)) {
    case 2: return backward<VEC, 2>(p, stream);
    case 4: return backward<VEC, 4>(p, stream);
    case 8: return backward<VEC, 8>(p, stream);
    default: return backward<VEC, 16>(p, stream);
    }
}

// The first pass over spans, its CTAs cut as the forward pass cuts channels.
template <int SL>
cudaError_t adjoint(const ScanParams &p, cudaStream_t stream)
{
    ScanParams q = p;
    const int ch = kForwardThreads / SL;
    q.blocks_g = (p.Eg + ch - 1) / ch;
    const int64_t grid = (p.N * p.G * q.blocks_g * p.spans);
    if (p.z.ptr)
        return launch_grid(scan_adjoint_kernel<T, SL, true>, grid, kForwardThreads, stream, q);
    return launch_grid(scan_adjoint_kernel<T, SL, false>, grid, kForwardThreads, stream, q);
}

cudaError_t adjoint(const ScanParams &p, cudaStream_t stream)
{
    switch (scan_state_lanes(p.S, 8)) {
    case 1: return adjoint<1>(p, stream);
    case 2: return adjoint<2>(p, stream);
    case 4: return adjoint<4>(p, stream);
    default: return adjoint<8>(p, stream);
    }
}

template <int SL>
cudaError_t launch_bc(const ScanParams &p, cudaStream_t stream)
{
    const int64_t n = p.N * p.T * p.G * 8 * SL;
    return launch_grid(scan_bc_kernel<T, 4 * SL>, (n + 255) / 256, 256, stream, p);
}

// Rows to a thread: 2 where that still leaves 16 CTAs to an SM, else 1. Measured, 16 states, us,
// two / one: [4096, 1024] 112 / 117, [1024, 2048] 57.3 / 58.8, [512, 2048] 29.8 / 30.6.
template <int SL, bool VEC>
cudaError_t launch_step(const ScanParams &p, cudaStream_t stream)
{
    const int64_t per_row = p.E * SL;
    auto ctas = [&](int64_t rows) { return ((p.N + rows - 1) / rows * per_row + 127) / 128; };
    if (ctas(2) >= 16 * sm_count())
        return launch_grid(scan_step_kernel<T, SL, 2, VEC>, ctas(2), 128, stream, p);
    return launch_grid(scan_step_kernel<T, SL, 1, VEC>, ctas(1), 128, stream, p);
}

template <bool VEC>
cudaError_t launch_step(const ScanParams &p, cudaStream_t stream)
{
    switch (scan_state_lanes(p.S, 8)) {
    case 1: return launch_step<1, VEC>(p, stream);
    case 2: return launch_step<2, VEC>(p, stream);
    case 4: return launch_step<4, VEC>(p, stream);
    default: return launch_step<8, VEC>(p, stream);
    }
}

}  // namespace

template <Fmt F>
cudaError_t launch_scan_forward(const ScanParams &p, bool vec, cudaStream_t stream)
{
    return vec ? forward<true>(p, stream) : forward<false>(p, stream);
}

template <Fmt F>
cudaError_t launch_scan_backward(const ScanParams &p, bool vec, cudaStream_t stream)
{
    cudaError_t err = cudaSuccess;
    if (p.spans > 1) {
        err = adjoint(p, stream);
        if (err == cudaSuccess) err = launch_scan_join(p, true, stream);
        if (err != cudaSuccess) return err;
    }
    err = vec ? backward<true>(p, stream) : backward<false>(p, stream);
    if (err != cudaSuccess || p.T == 0) return err;
    switch (scan_backward_lanes(p.S)) {
    case 2: return launch_bc<2>(p, stream);
    case 4: return launch_bc<4>(p, stream);
    case 8: return launch_bc<8>(p, stream);
    default: return launch_bc<16>(p, stream);
    }
}

template <Fmt F>
cudaError_t launch_scan_step(const ScanParams &p, bool vec, cudaStream_t stream)
{
    return vec ? launch_step<true>(p, stream) : launch_step<false>(p, stream);
}

template cudaError_t launch_scan_forward<static_cast<Fmt>(RLCA_UNIT_FMT)>(const ScanParams &, bool,
                                                                          cudaStream_t);
template cudaError_t launch_scan_backward<static_cast<Fmt>(RLCA_UNIT_FMT)>(const ScanParams &,
                                                                           bool, cudaStream_t);
template cudaError_t launch_scan_step<static_cast<Fmt>(RLCA_UNIT_FMT)>(const ScanParams &, bool,
                                                                       cudaStream_t);

}  // namespace seq
}  // namespace rlca

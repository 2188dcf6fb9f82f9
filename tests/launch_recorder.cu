// The host side of the sequence operators' entry points (csrc/sequence_api.cu) with the CUDA
// runtime's answers and the kernels' launches replaced: a scan's launch records what the kernel
// would get. Built and loaded by test_sequence_launches.py, needs no GPU.
#include <cuda_runtime.h>

static cudaError_t fake_get_device(int *device)
{
    *device = 0;
    return cudaSuccess;
}
static cudaError_t fake_attributes(cudaPointerAttributes *a, const void *)
{
    a->type = cudaMemoryTypeDevice;
    a->device = 0;
    return cudaSuccess;
}
#define cudaGetDevice fake_get_device
#define cudaPointerGetAttributes fake_attributes

#include "../segmented_associative_scan_gb300/csrc/sequence_api.cu"

namespace rlca {
namespace seq {

static ScanParams g_scan;
static int g_vec;

template <Fmt F>
cudaError_t launch_scan_forward(const ScanParams &p, bool vec, cudaStream_t)
{
    g_scan = p;
    g_vec = vec;
    return cudaSuccess;
}
template <Fmt F>
cudaError_t launch_scan_backward(const ScanParams &p, bool vec, cudaStream_t)
{
    g_scan = p;
    g_vec = vec;
    return cudaSuccess;
}
template <Fmt F>
cudaError_t launch_scan_step(const ScanParams &, bool, cudaStream_t)
{
    return cudaSuccess;
}
template <Fmt F>
cudaError_t launch_conv_forward(const ConvParams &, bool, cudaStream_t)
{
    return cudaSuccess;
}
template <Fmt F>
cudaError_t launch_conv_backward(const ConvParams &, bool, cudaStream_t)
{
    return cudaSuccess;
}
template <Fmt F>
cudaError_t launch_conv_step(const ConvParams &, bool, cudaStream_t)
{
    return cudaSuccess;
}
template <Fmt F>
cudaError_t launch_embed(const EmbedParams &, bool, cudaStream_t)
{
    return cudaSuccess;
}
template <Fmt F>
cudaError_t launch_embed_sum(const EmbedParams &, bool, cudaStream_t)
{
    return cudaSuccess;
}
cudaError_t launch_sum_rows(const SumRows &, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_embed_sort(const EmbedParams &, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_embed_join(const EmbedParams &, cudaStream_t) { return cudaSuccess; }

}  // namespace seq
}  // namespace rlca

// Whether the last scan was launched for 16-byte copies.
extern "C" int recorded_vec() { return rlca::seq::g_vec; }

// Its activation `which`, as the kernel would address it.
extern "C" rlca_steps recorded_steps(int which)
{
    const rlca::seq::ScanParams &p = rlca::seq::g_scan;
    const rlca_steps all[] = {p.x, p.dt, p.z, p.out, p.dout, p.dx, p.ddt, p.dz};
    return all[which];
}

// Launchers of the decode attention over a cache of T (bf16 or f32); the
// kernel is in attend_kernel.cuh.
#include "attend_kernel.cuh"

namespace pdattn {

template <int D>
static cudaError_t launch_f32(const AttendArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map, int grid,
                              bool programmatic, cudaStream_t stream) {
    if (a.group <= 1) return launch_one<float, D, 1>(a, k_map, v_map, grid, programmatic, stream);
    if (a.group <= 2) return launch_one<float, D, 2>(a, k_map, v_map, grid, programmatic, stream);
    if (a.group <= 4) return launch_one<float, D, 4>(a, k_map, v_map, grid, programmatic, stream);
    return launch_one<float, D, 8>(a, k_map, v_map, grid, programmatic, stream);
}

cudaError_t launch_attend(const AttendArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map,
                          int dtype, int grid, bool programmatic, cudaStream_t stream) {
    if (dtype == 0 && a.head_dim == 128)
        return launch_one<__nv_bfloat16, 128, kMaxGroup>(a, k_map, v_map, grid, programmatic, stream);
    if (dtype == 0 && a.head_dim == 64)
        return launch_one<__nv_bfloat16, 64, kMaxGroup>(a, k_map, v_map, grid, programmatic, stream);
    if (dtype == 1 && a.head_dim == 128) return launch_f32<128>(a, k_map, v_map, grid, programmatic, stream);
    if (dtype == 1 && a.head_dim == 64) return launch_f32<64>(a, k_map, v_map, grid, programmatic, stream);
    return cudaErrorInvalidValue;
}

// Multi-layer launches: bf16 at head dim 64 / 128 (groups up to 8 on one
// instance) and f32 with one-head groups (plain multi-head attention) or any
// group up to 8.  Always a programmatic dependent of the prep launch.
cudaError_t launch_attend_layers(const AttendArgs& a, const AttendLayers& lay, int dtype, int grid,
                                 cudaStream_t stream) {
    const CUtensorMap& k0 = lay.k[0];
    const CUtensorMap& v0 = lay.v[0];
    if (dtype == 0 && a.head_dim == 128)
        return launch_one<__nv_bfloat16, 128, kMaxGroup, AttendLayers>(a, k0, v0, grid, true, stream, lay);
    if (dtype == 0 && a.head_dim == 64)
        return launch_one<__nv_bfloat16, 64, kMaxGroup, AttendLayers>(a, k0, v0, grid, true, stream, lay);
    if (dtype == 1 && a.head_dim == 128)
        return a.group <= 1 ? launch_one<float, 128, 1, AttendLayers>(a, k0, v0, grid, true, stream, lay)
                            : launch_one<float, 128, 8, AttendLayers>(a, k0, v0, grid, true, stream, lay);
    if (dtype == 1 && a.head_dim == 64)
        return a.group <= 1 ? launch_one<float, 64, 1, AttendLayers>(a, k0, v0, grid, true, stream, lay)
                            : launch_one<float, 64, 8, AttendLayers>(a, k0, v0, grid, true, stream, lay);
    return cudaErrorInvalidValue;
}

size_t attend_smem_bytes(int dtype, int head_dim) {
    if (dtype == 0)
        return head_dim == 128 ? Cfg<__nv_bfloat16, 128, kMaxGroup>::kSmem : Cfg<__nv_bfloat16, 64, kMaxGroup>::kSmem;
    return head_dim == 128 ? Cfg<float, 128, kMaxGroup>::kSmem : Cfg<float, 64, kMaxGroup>::kSmem;
}

}  // namespace pdattn

// Launcher of the decode attention over a coded (8-bit) cache; the kernel is
// in attend_kernel.cuh, its consumer Consumer<T, D, G, Code>.
#include "attend_kernel.cuh"

namespace pdattn {

template <typename T, int D, int G>
static cudaError_t launch_code_type(const AttendArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map, int code,
                                    int grid, cudaStream_t stream) {
    if (code == 0) return launch_one<T, D, G, NoLayers, E4m3>(a, k_map, v_map, grid, true, stream);
    return launch_one<T, D, G, NoLayers, Int8>(a, k_map, v_map, grid, true, stream);
}

cudaError_t launch_attend_coded(const AttendArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map, int dtype,
                                int code, int grid, cudaStream_t stream) {
    if (dtype == 0)
        return a.head_dim == 128 ? launch_code_type<__nv_bfloat16, 128, kMaxGroup>(a, k_map, v_map, code, grid, stream)
                                 : launch_code_type<__nv_bfloat16, 64, kMaxGroup>(a, k_map, v_map, code, grid, stream);
    // f32: both f16 parts of up to four heads in one pass (Consumer<..., Code>)
    if (a.group <= 4)
        return a.head_dim == 128 ? launch_code_type<float, 128, 4>(a, k_map, v_map, code, grid, stream)
                                 : launch_code_type<float, 64, 4>(a, k_map, v_map, code, grid, stream);
    return a.head_dim == 128 ? launch_code_type<float, 128, kMaxGroup>(a, k_map, v_map, code, grid, stream)
                             : launch_code_type<float, 64, kMaxGroup>(a, k_map, v_map, code, grid, stream);
}

}  // namespace pdattn

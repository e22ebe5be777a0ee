// Launcher of the decode attention whose rows share pages (bf16): the kernel
// of attend_kernel.cuh over the rows' own pages, merging the shared pages'
// partials (csrc/shared.cu).
#include "attend_kernel.cuh"

namespace pdattn {

cudaError_t launch_attend_shared(const AttendArgs& a, const AttendShared& sh, const CUtensorMap& k_map,
                                 const CUtensorMap& v_map, int grid, cudaStream_t stream) {
    if (a.head_dim == 128)
        return launch_one<__nv_bfloat16, 128, kMaxGroup, AttendShared>(a, k_map, v_map, grid, true, stream, sh);
    if (a.head_dim == 64)
        return launch_one<__nv_bfloat16, 64, kMaxGroup, AttendShared>(a, k_map, v_map, grid, true, stream, sh);
    return cudaErrorInvalidValue;
}

}  // namespace pdattn

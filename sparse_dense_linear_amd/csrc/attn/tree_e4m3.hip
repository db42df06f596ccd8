// tree_e4m3.hip -- attention of drafted tokens over a paged cache that holds
// floating-point numbers of 8 bits (e4m3): tree_codes.h.
#include "tree_codes.h"

namespace sdl {

hipError_t launch_tree_e4m3(int dtype, const TreeArgs &a, hipStream_t stream)
{
    return dtype == SPMM_DTYPE_BF16 ? launch_codes_sized<__bf16, E4M3>(a, stream) : launch_codes_sized<float, E4M3>(a, stream);
}

}  // namespace sdl

// tree_int8.hip -- attention of drafted tokens over a paged cache that holds
// integers of 8 bits: tree_codes.h.
#include "tree_codes.h"

namespace sdl {

hipError_t launch_tree_int8(int dtype, const TreeArgs &a, hipStream_t stream)
{
    return dtype == SPMM_DTYPE_BF16 ? launch_codes_sized<__bf16, Int8>(a, stream) : launch_codes_sized<float, Int8>(a, stream);
}

}  // namespace sdl

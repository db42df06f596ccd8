// tree.hip -- attention of drafted tokens over a paged cache that holds rows of
// the type of q: tree_impl.h.
#include "tree_impl.h"

namespace sdl {

TreeShape tree_shape(int dtype, int held, int64_t S, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t D)
{
    TreeShape sh = {};
    const int DP = D <= 64 ? 64 : 128;
    // as many queries to a block as the mean sequence fills
    sh.rows = S > 0 ? (Tq + S - 1) / S * (Hq / Hkv) : 0;
    sh.block_rows = sh.rows <= 16 ? 16 : (sh.rows <= 32 ? 32 : (sh.rows <= 64 ? 64 : 128));
    sh.wave_heads = 1;
    // as many workgroups as the 256 CUs hold at once
    if (held != 0 && sh.block_rows == 16) {
        sh.workers = 256 * stream_per_cu(dtype == SPMM_DTYPE_BF16 ? 2 : 4, DP);
        sh.wave_heads = Hkv % 4 == 0 ? 4 : (Hkv % 2 == 0 ? 2 : 1);
    } else if (held != 0) {
        sh.workers = 256 * 2;                  // tree_tiles
        if (dtype != SPMM_DTYPE_BF16 && sh.block_rows > 64)
            sh.block_rows = 64;
    } else if (dtype == SPMM_DTYPE_BF16) {
        sh.workers = 256 * (DP == 64 ? per_cu<__bf16, 64>(sh.block_rows) : per_cu<__bf16, 128>(sh.block_rows));
    } else {
        sh.workers = 256 * (DP == 64 ? per_cu<float, 64>(sh.block_rows) : per_cu<float, 128>(sh.block_rows));
    }
    const int64_t slot_rows = (int64_t)sh.block_rows * sh.wave_heads;
    sh.bytes = 4 * (2 * ((S + 1 + 31) / 32 * 32) + 2 * (int64_t)sh.workers * slot_rows * (2 + DP));
    return sh;
}

int64_t tree_threads(const TreeArgs &a)
{
    const int64_t join = join_numbers(a) * a.Hkv, most = join > a.workers ? join : a.workers;
    return most * kAttnThreads;
}

hipError_t launch_tree(int dtype, const TreeArgs &a, hipStream_t stream)
{
    return dtype == SPMM_DTYPE_BF16 ? launch_sized<__bf16>(a, stream)
                                    : launch_sized<float>(a, stream);
}

}  // namespace sdl

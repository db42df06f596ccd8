// Argument paths of include/attn.h in a host-only build under
// AddressSanitizer and UndefinedBehaviorSanitizer: every call is answered on
// the host.  Sizes and strides at their limits show any overflow.
#include <cstdio>
#include <cstdlib>
#include <limits>

#include "attn.h"

namespace {

int g_failures = 0;

void expect(bool ok, const char *what, int line)
{
    if (!ok) {
        std::fprintf(stderr, "line %d: %s (last error: \"%s\")\n", line, what, spmm_last_error());
        ++g_failures;
    }
}

#define EXPECT(cond) expect((cond), #cond, __LINE__)

void *fake() { return reinterpret_cast<void *>(uintptr_t{0x10000}); }

const int64_t kExtremes[] = {std::numeric_limits<int64_t>::min(), -1, 0, 1, 7, 8, 64, 128,
                             (int64_t{1} << 30) - 1, int64_t{1} << 30, int64_t{1} << 32,
                             std::numeric_limits<int64_t>::max()};

void windows()
{
    const attn_window_t good = {2, 10, 10, 4, 2, 64, 8, 1, 0.1f, 0};
    const attn_rows_t r = {fake(), 256, 64};
    int32_t *p = static_cast<int32_t *>(fake());
    float *f = static_cast<float *>(fake());
    int64_t attn_window_t::*const fields[] = {
        &attn_window_t::S, &attn_window_t::Tq, &attn_window_t::Tk, &attn_window_t::Hq, &attn_window_t::Hkv,
        &attn_window_t::D, &attn_window_t::window, &attn_window_t::sinks};
    for (auto a : fields)
        for (int64_t x : kExtremes)
            for (auto b : fields)
                for (int64_t y : kExtremes) {
                    attn_window_t w = good;
                    w.*a = x;
                    w.*b = y;
                    int64_t bytes = -1;
                    const spmm_status_t st = window_attn_bwd_scratch(&w, &bytes);
                    EXPECT(st == SPMM_SUCCESS ? bytes >= 0 : bytes == -1);
                    // no scratch, an unknown type, a misaligned lse: refused, or nothing to do
                    EXPECT(window_attn_fwd(7, &w, &r, &r, &r, p, p, &r, f, nullptr, 0, nullptr) != SPMM_SUCCESS);
                    int64_t forward = -1;
                    EXPECT(window_attn_fwd_scratch(SPMM_DTYPE_BF16, &w, &forward) == st);
                    EXPECT(st == SPMM_SUCCESS ? forward >= 0 : forward == -1);
                    const spmm_status_t back = window_attn_bwd(SPMM_DTYPE_F32, &w, &r, &r, &r, &r, &r, f, p, p,
                                                               &r, &r, &r, nullptr, 0, nullptr);
                    EXPECT(back != SPMM_SUCCESS || w.S == 0 || (w.Tq == 0 && w.Tk == 0));
                }
    for (int64_t x : kExtremes)
        for (int64_t y : kExtremes) {
            const attn_rows_t odd = {fake(), x, y};
            EXPECT(window_attn_fwd(SPMM_DTYPE_F32, &good, &odd, &r, &r, nullptr, p, &odd, f, nullptr, 0, nullptr) !=
                   SPMM_SUCCESS);
        }
}

void trees()
{
    const attn_tree_t good = {2, 10, 4, 2, 64, 16, 2048, 128, 64, 5, 8, 1, 0.1f, 0};
    const attn_rows_t r = {fake(), 256, 64};
    int32_t *p = static_cast<int32_t *>(fake());
    float *f = static_cast<float *>(fake());
    int64_t attn_tree_t::*const fields[] = {
        &attn_tree_t::S, &attn_tree_t::Tq, &attn_tree_t::Hq, &attn_tree_t::Hkv, &attn_tree_t::D,
        &attn_tree_t::page, &attn_tree_t::page_stride, &attn_tree_t::row_stride, &attn_tree_t::head_stride,
        &attn_tree_t::table_stride, &attn_tree_t::window, &attn_tree_t::sinks};
    for (auto a : fields)
        for (int64_t x : kExtremes)
            for (auto b : fields)
                for (int64_t y : kExtremes) {
                    attn_tree_t w = good;
                    w.*a = x;
                    w.*b = y;
                    int64_t bytes = -1;
                    const spmm_status_t st = tree_attn_scratch(SPMM_DTYPE_BF16, &w, &bytes);
                    EXPECT(st == SPMM_SUCCESS ? bytes >= 0 : bytes == -1);
                    const spmm_status_t run = tree_attn_paged(SPMM_DTYPE_F32, &w, &r, fake(), fake(), p, p, p,
                                                              nullptr, fake(), f, nullptr, 0, nullptr);
                    EXPECT(run != SPMM_SUCCESS || w.S == 0 || w.Tq == 0);
                }
}

void pages()
{
    int32_t *p = static_cast<int32_t *>(fake());
    for (int64_t x : kExtremes)
        for (int64_t y : kExtremes)
            for (int64_t z : kExtremes) {
                const attn_pool_t a = {fake(), fake(), x, y, z, 256}, b = {fake(), fake(), z, 8, x, y};
                EXPECT(pages_copy(&a, nullptr, p, 3, nullptr) != SPMM_SUCCESS || x == 0 || y == 0 || z == 0);
                EXPECT(pages_copy(&b, nullptr, p, x, nullptr) != SPMM_SUCCESS || x == 0 || y == 0 || z == 0);
                EXPECT(pages_compact(&a, p, x, nullptr, p, y, z, nullptr) != SPMM_SUCCESS || x == 0 || y == 0 ||
                       z == 0);
            }
}

}  // namespace

int main()
{
    windows();
    trees();
    pages();
    if (g_failures != 0)
        return 1;
    std::puts("attention argument paths: ok");
    return 0;
}

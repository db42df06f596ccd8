// Argument paths of include/cache.h in a host-only build under
// AddressSanitizer and UndefinedBehaviorSanitizer: every call is answered on
// the host.  Sizes and strides at their limits show any overflow.
#include <cstdio>
#include <limits>

#include "cache.h"

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
int32_t *numbers() { return static_cast<int32_t *>(fake()); }
float *floats() { return static_cast<float *>(fake()); }

const int64_t kExtremes[] = {std::numeric_limits<int64_t>::min(), -1, 0, 1, 7, 8, 16, 64, 128,
                             (int64_t{1} << 30) - 1, int64_t{1} << 30, int64_t{1} << 32,
                             std::numeric_limits<int64_t>::max()};
const int32_t kKinds[] = {CACHE_AS_IS, CACHE_E4M3, CACHE_INT8, 3};

// The last argument that a call looks at is wrong (scratch, scales): nothing is enqueued.
void trees()
{
    const attn_tree_t good = {2, 10, 4, 2, 64, 16, 2048, 128, 64, 5, 8, 1, 0.1f, 0};
    const attn_rows_t r = {fake(), 256, 64};
    const cache_scales_t s = {floats(), floats(), 8, 4, 2, 1};
    int64_t attn_tree_t::*const fields[] = {
        &attn_tree_t::S, &attn_tree_t::Tq, &attn_tree_t::Hq, &attn_tree_t::Hkv, &attn_tree_t::D,
        &attn_tree_t::page, &attn_tree_t::page_stride, &attn_tree_t::row_stride, &attn_tree_t::head_stride,
        &attn_tree_t::table_stride, &attn_tree_t::window, &attn_tree_t::sinks};
    for (int32_t held : kKinds)
        for (auto a : fields)
            for (int64_t x : kExtremes)
                for (auto b : fields)
                    for (int64_t y : kExtremes) {
                        attn_tree_t w = good;
                        w.*a = x;
                        w.*b = y;
                        int64_t bytes = -1;
                        const spmm_status_t st = cache_tree_attn_scratch(SPMM_DTYPE_BF16, held, &w, &bytes);
                        EXPECT(st == SPMM_SUCCESS ? bytes >= 0 : bytes == -1);
                        const spmm_status_t run = cache_tree_attn(SPMM_DTYPE_F32, held, &w, &r, fake(), fake(), &s,
                                                                  numbers(), numbers(), numbers(), nullptr, fake(),
                                                                  floats(), nullptr, 0, nullptr);
                        EXPECT(run != SPMM_SUCCESS || w.S == 0 || w.Tq == 0);
                    }
}

void appends()
{
    const cache_append_t good = {2, 10, 4, 2, 64, 16, 8, 2048, 128, 64, 5, 64, 100, 0, 0};
    const attn_rows_t q = {fake(), 256, 64}, k = {fake(), 128, 64};
    int64_t cache_append_t::*const fields[] = {
        &cache_append_t::S, &cache_append_t::T, &cache_append_t::Hq, &cache_append_t::Hkv, &cache_append_t::D,
        &cache_append_t::page, &cache_append_t::pages, &cache_append_t::page_stride, &cache_append_t::row_stride,
        &cache_append_t::head_stride, &cache_append_t::table_stride, &cache_append_t::rotated,
        &cache_append_t::angles};
    auto call = [&](int32_t held, const cache_append_t &w, const cache_scales_t *s) {
        return cache_append(SPMM_DTYPE_F32, held, &w, &q, &k, &k, floats(), floats(), numbers(), numbers(), numbers(),
                            nullptr, fake(), fake(), s, &q, nullptr);
    };
    const cache_scales_t any = {floats(), floats(), 8, 4, 2, 1};
    for (int32_t held : kKinds)
        for (auto a : fields)
            for (int64_t x : kExtremes)
                for (auto b : fields)
                    for (int64_t y : kExtremes) {
                        cache_append_t w = good;
                        w.*a = x;
                        w.*b = y;
                        // scales where none belong, and none where they do
                        EXPECT(call(held, w, held == CACHE_AS_IS ? &any : nullptr) != SPMM_SUCCESS || w.S == 0 ||
                               w.T == 0);
                    }
    for (int64_t x : kExtremes)
        for (int64_t y : kExtremes)
            for (int64_t z : kExtremes) {
                const cache_scales_t s = {nullptr, floats(), x, y, z, 1}, t = {floats(), nullptr, 8, x, y, z},
                                     u = {floats(), floats(), 16, x, y, 0};
                cache_append_t w = good;
                w.page = x;
                w.pages = y;
                w.page_stride = z;
                EXPECT(call(CACHE_E4M3, good, &s) != SPMM_SUCCESS);
                EXPECT(call(CACHE_INT8, good, &t) != SPMM_SUCCESS);
                EXPECT(call(CACHE_INT8, good, &u) != SPMM_SUCCESS);
                EXPECT(call(CACHE_E4M3, w, &s) != SPMM_SUCCESS);
            }
}

void pages()
{
    for (int64_t x : kExtremes)
        for (int64_t y : kExtremes)
            for (int64_t z : kExtremes) {
                const bool none = x == 0 || y == 0 || z == 0;
                const cache_pool_t a = {{fake(), fake(), x, y, z, 256}, nullptr, floats(), z, 2};
                const cache_pool_t b = {{fake(), fake(), z, 8, x, y}, floats(), nullptr, 1, z};
                EXPECT(cache_copy(&a, nullptr, numbers(), 3, nullptr) != SPMM_SUCCESS || none);
                EXPECT(cache_copy(&b, nullptr, numbers(), x, nullptr) != SPMM_SUCCESS || none);
                for (int32_t held : kKinds) {
                    EXPECT(cache_compact(held, &a, numbers(), x, nullptr, numbers(), y, z, nullptr) != SPMM_SUCCESS ||
                           none);
                    EXPECT(cache_compact(held, &b, numbers(), x, nullptr, numbers(), y, z, nullptr) != SPMM_SUCCESS ||
                           none);
                }
            }
}

}  // namespace

int main()
{
    trees();
    appends();
    pages();
    if (g_failures != 0)
        return 1;
    std::puts("cache argument paths: ok");
    return 0;
}

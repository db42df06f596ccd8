// SeenRows (attn/draft.h) against what the drafts of a sequence see one by
// one: the rows of the cache that are read are those that some draft sees.
#include <cstdio>
#include <random>
#include <vector>

#include "attn/draft.h"

using namespace sdl;

namespace {

int g_failures = 0;

// masks empty: a chain
void check(int ctx, int drafts, int window, int sinks, const std::vector<uint64_t> &masks)
{
    const bool chain = masks.empty();
    int low = chain ? window_low(ctx, window) : ctx, place[64] = {}, flags[64] = {};
    uint64_t named = 0;
    for (int t = 0; !chain && t < drafts; ++t) {
        count_draft(masks.data(), ctx, drafts, window, sinks, t, low, named);
        if (t < 64)
            place[t] = draft_place(ctx, draft_mask(masks[t], drafts));
    }
    for (int d = 0; d < 64; ++d)
        flags[d] = named >> d & 1;
    const SeenRows rows = {ctx, ctx + drafts, low, sinks, chain ? nullptr : flags};
    auto some_sees = [&](int j) {
        for (int t = 0; t < drafts; ++t) {
            const uint64_t mask = chain ? 0 : draft_mask(masks[t], drafts);
            const DraftSeen seen = {ctx, drafts, window, sinks, chain ? ctx + t : draft_place(ctx, mask), mask,
                                    chain ? nullptr : place};
            if (seen(j))
                return true;
        }
        return false;
    };
    const int end = ctx + drafts + 3;
    for (int j = 0; j < end; ++j) {
        if (rows(j) != some_sees(j)) {
            std::fprintf(stderr, "ctx %d, %d drafts, window %d, %d sinks, %s: key %d %s\n", ctx, drafts, window, sinks,
                         chain ? "chain" : "masks", j, rows(j) ? "is read, not seen" : "is seen, not read");
            ++g_failures;
            return;
        }
    }
}

}  // namespace

int main()
{
    std::mt19937_64 r(1);
    auto any = [&](int n) { return (int)(r() % (uint64_t)n); };
    const int windows[] = {1, 2, 5, 16, 40, 63, 64, 65, 200, (1 << 30) - 1};
    // two drafts that see each other stand at ctx + 1: the first key of a
    // window from ctx is behind it
    check(47, 2, 16, 0, {3, 3});
    check(47, 2, 16, 4, {3, 3});
    check(0, 1, 16, 4, {0});
    for (int n = 0; n < 20000 && g_failures < 10; ++n) {
        const int ctx = any(3) == 0 ? any(4) : any(300), drafts = 1 + (any(4) == 0 ? any(90) : any(9));
        const int window = windows[any(10)], sinks = any(2) == 0 ? 0 : any(129);
        std::vector<uint64_t> masks(drafts);
        const int kind = any(4);
        for (int t = 0; t < drafts; ++t) {
            if (kind == 0)
                masks[t] = r();
            else if (kind == 1)
                masks[t] = r() & r() & r();
            else if (kind == 2)                // none names itself
                masks[t] = any(2) == 0 ? 0 : (uint64_t)1 << any(64);
            else {                             // a tree
                const int parent = any(t + 1) - 1;
                masks[t] = (parent < 0 ? 0 : masks[parent]) | (t < 64 ? (uint64_t)1 << t : 0);
            }
        }
        check(ctx, drafts, window, sinks, masks);
        check(ctx, drafts, window, sinks, {});
    }
    if (g_failures != 0)
        return 1;
    std::puts("drafts: ok");
    return 0;
}

// BlockSeen (attn/draft.h), 32 keys at once, against DraftSeen, key by key, and
// division by a prepared number (attn/ops.h) against division.
#include <cstdio>
#include <random>
#include <vector>

#include "attn/draft.h"
#include "attn/ops.h"

using namespace sdl;

namespace {

int g_failures = 0;

// masks empty: a chain
void check(int ctx, int drafts, int window, int sinks, const std::vector<uint64_t> &masks)
{
    const bool chain = masks.empty();
    int place[64] = {};
    for (int t = 0; !chain && t < drafts && t < 64; ++t)
        place[t] = draft_place(ctx, draft_mask(masks[t], drafts));
    for (int t = 0; t < drafts; ++t) {
        const uint64_t mask = chain ? 0 : draft_mask(masks[t], drafts);
        const int pos = chain ? ctx + t : draft_place(ctx, mask);
        const DraftSeen one = {ctx, drafts, window, sinks, pos, mask, chain ? nullptr : place};
        BlockSeen block = {pos, chain ? pos + 1 : ctx, mask};
        if (!chain)
            block.keep_near(place, window, sinks);
        for (int j0 = 0; j0 < ctx + drafts + 64; j0 += 16) {
            const uint32_t bits = block(j0, ctx, window, sinks);
            for (int i = 0; i < 32; ++i)
                if ((bits >> i & 1) != (one(j0 + i) ? 1u : 0u) && ++g_failures < 10)
                    std::fprintf(stderr, "ctx %d drafts %d window %d sinks %d draft %d key %d\n", ctx, drafts, window,
                                 sinks, t, j0 + i);
        }
    }
}

void divisions()
{
    const uint32_t most = 0x7fffffff;
    std::mt19937 r(1);
    std::vector<uint32_t> by;
    for (uint32_t d = 1; d < 300; ++d)
        by.push_back(d);
    for (int s = 8; s < 30; ++s)
        for (int e = -1; e <= 1; ++e)
            by.push_back((1u << s) + e);
    for (uint32_t d : by) {
        const Divisor v = divisor(d);
        auto one = [&](uint32_t x) {
            const uint32_t q = (uint32_t)((uint64_t)(x << 1) * v.factor >> 32) >> v.shift;
            if (q != x / d && ++g_failures < 10)
                std::fprintf(stderr, "%u / %u: %u\n", x, d, q);
        };
        for (int i = 0; i < 200; ++i) {
            const uint32_t x = r() & most, m = x / d * d;
            one(x);
            one(m);
            one(m > 0 ? m - 1 : 0);
        }
        for (uint32_t x : {0u, 1u, d - 1, d, most / d * d, most / d * d - 1, most})
            one(x & most);
    }
}

}  // namespace

int main()
{
    std::mt19937_64 r(7);
    for (int ctx : {0, 1, 5, 31, 32, 33, 100})
        for (int drafts : {1, 2, 7, 32, 63, 64, 70})
            for (int window : {1, 2, 16, 40, 63, 64, 90, 1 << 29})
                for (int sinks : {0, 3, 34, 128}) {
                    check(ctx, drafts, window, sinks, {});
                    for (int kind = 0; kind < 3; ++kind) {
                        std::vector<uint64_t> masks;
                        for (int t = 0; t < drafts; ++t)
                            masks.push_back(kind == 0 ? r() : (kind == 1 ? r() & r() & r() : (t < 64 ? ~0ull >> (63 - t) : 0)));
                        check(ctx, drafts, window, sinks, masks);
                    }
                }
    divisions();
    if (g_failures != 0)
        return 1;
    std::puts("seen: ok");
    return 0;
}

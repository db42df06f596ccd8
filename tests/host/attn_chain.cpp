// Which operands chain() (attn/tile.h) reads: those of its instructions, each
// once and before its use, also where it may read further ahead than there
// are instructions.
#include <cstdio>
#include <vector>

#include "attn/tile.h"

namespace {

int g_failures = 0;

template <int COUNT, int AHEAD>
void check()
{
    std::vector<int> reads, uses;
    bool right = true;
    sdl::chain<COUNT, AHEAD>(
        [&](int i) {
            reads.push_back(i);
            return i;
        },
        [&](int i, int f) {
            uses.push_back(i);
            right = right && f == i;
        });
    right = right && (int)reads.size() == COUNT && (int)uses.size() == COUNT;
    for (int i = 0; right && i < COUNT; ++i)
        right = reads[i] == i && uses[i] == i;
    if (!right) {
        std::fprintf(stderr, "chain<%d, %d>: %d reads, %d uses, last read %d\n", COUNT, AHEAD, (int)reads.size(),
                     (int)uses.size(), reads.empty() ? -1 : reads.back());
        ++g_failures;
    }
}

}  // namespace

int main()
{
    check<1, 1>();
    check<2, 4>();
    check<4, 6>();
    check<6, 6>();
    check<7, 6>();
    check<16, 6>();
    check<16, 3>();
    check<3, 2>();
    if (g_failures != 0)
        return 1;
    std::puts("chain: ok");
    return 0;
}

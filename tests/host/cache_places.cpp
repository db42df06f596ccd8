// Which rows of the rotation's tables a position may read, and which block of
// positions holds it (attn/draft.h), also in front of the sequence.
#include <cstdio>

#include "attn/draft.h"

using namespace sdl;

int main()
{
    int failures = 0;
    const int least = -2147483647 - 1, most = 2147483647;
    for (int angles : {0, 1, 2, 63, 1 << 30})
        for (int place : {least, least + 1, -(1 << 30), -64, -2, -1, 0, 1, 2, 62, 63, 64, 1 << 30, most})
            if (has_angles(place, angles) != (place >= 0 && place < angles)) {
                std::fprintf(stderr, "place %d of %d\n", place, angles);
                ++failures;
            }
    for (int block : {1, 2, 7, 16, 25, 1 << 29})
        for (int64_t near : {(int64_t)least, -(int64_t)block * 3, -(int64_t)block, (int64_t)0, (int64_t)block, (int64_t)most})
            for (int64_t pos = near - 40; pos <= near + 40; ++pos) {
                if (pos < least || pos > most)
                    continue;
                const int64_t b = block_of((int)pos, block);
                if (b * block > pos || (b + 1) * block <= pos) {
                    std::fprintf(stderr, "position %lld, block %d: %lld\n", (long long)pos, block, (long long)b);
                    ++failures;
                }
            }
    if (failures)
        return 1;
    std::puts("places: ok");
    return 0;
}

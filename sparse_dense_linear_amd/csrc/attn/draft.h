// draft.h -- what drafts of a sequence see of its cached keys and of each
// other: by each draft (DraftSeen), and by all of them together (SeenRows).
// The host can run it too.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sdl {

#define SDL_BOTH __host__ __device__ inline

// Which keys draft t sees, and from where.
struct DraftSeen {
    int ctx, drafts, window, sinks;
    int pos;              // of the draft
    uint64_t mask;
    const int *place;     // positions of the drafts' keys (null: a chain)
    __host__ __device__ bool operator()(int j) const
    {
        if (j < ctx || place == nullptr)
            return j <= pos && (pos - j < window || j < sinks);
        const int d = j - ctx;
        if (d >= drafts || d >= 64 || !(mask >> d & 1))
            return false;
        return pos - place[d] < window || place[d] < sinks;
    }
};

// The drafts of its sequence that a mask names.
SDL_BOTH uint64_t draft_mask(uint64_t mask, int drafts)
{
    return drafts < 64 ? mask & (((uint64_t)1 << drafts) - 1) : mask;
}

SDL_BOTH int draft_place(int ctx, uint64_t mask)
{
    const int n = __builtin_popcountll(mask);
    return ctx + (n > 1 ? n - 1 : 0);
}

// The keys that some draft of a sequence sees.  No other row of the cache may
// be read: its page may have been given away, and the table's entry may be
// anything.
struct SeenRows {
    int ctx, end;          // end: ctx + drafts
    int low, sinks;        // of the context: keys from low on, and the first ones
    const int *named;      // [64], of the first drafts: not 0 where one is seen (null: a chain, all are)
    __host__ __device__ bool operator()(int j) const
    {
        if (j < ctx)
            return j >= low || j < sinks;
        return named == nullptr ? j < end : j < end && j - ctx < 64 && named[j - ctx] != 0;
    }
};

// The first key of the context that a draft at position pos sees, sinks apart.
SDL_BOTH int window_low(int pos, int window) { return pos - window + 1 > 0 ? pos - window + 1 : 0; }

// What drafts with masks see together: `low` and the bits of `named` of
// SeenRows.  Counts draft t of a sequence and returns where it stands; at first
// low is ctx and named 0.
// (Positions of drafts differ by less than 64, so that a window which reaches
// as far hides no draft that is named.)
SDL_BOTH int count_draft(const uint64_t *masks, int ctx, int drafts, int window, int sinks, int t, int &low,
                         uint64_t &named)
{
    uint64_t m = draft_mask(masks[t], drafts);
    const int pos = draft_place(ctx, m), from = window_low(pos, window);
    low = from < low ? from : low;
    if (window < 64)
        for (int d = 0; d < drafts && d < 64; ++d) {
            const int place = draft_place(ctx, draft_mask(masks[d], drafts));
            if (pos - place >= window && place >= sinks)
                m &= ~((uint64_t)1 << d);
        }
    named |= m;
    return pos;
}

}  // namespace sdl

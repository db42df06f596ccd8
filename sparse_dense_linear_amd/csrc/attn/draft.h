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

// What draft t sees of 32 keys from j0 on, bit by bit.
struct BlockSeen {
    int pos, cached;      // where it stands; keys before `cached` go by the window alone
    uint64_t mask;        // of the drafts it sees (0: a chain, whose keys all lie before `cached`)
    __host__ __device__ static uint32_t below(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1); }
    // Drops the drafts that the window hides, once for all blocks (further apart than
    // 63 they do not stand).
    __host__ __device__ void keep_near(const int *place, int window, int sinks)
    {
        if (window < 64)
            for (int d = 0; d < 64; ++d)
                if (mask >> d & 1 && pos - place[d] >= window && place[d] >= sinks)
                    mask &= ~((uint64_t)1 << d);
    }
    __host__ __device__ uint32_t operator()(int j0, int ctx, int window, int sinks) const
    {
        const uint32_t near = (~below(pos - window + 1 - j0) | below(sinks - j0)) & below(cached - j0);
        const int d = j0 - ctx;
        const uint64_t drafts = d >= 64 || d <= -32 ? 0 : (d >= 0 ? mask >> d : mask << -d);
        return near | (uint32_t)drafts;
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

// Whether the tables of a rotation have the position where a row stands.
SDL_BOTH bool has_angles(int place, int angles) { return (uint32_t)place < (uint32_t)angles; }

// The block of positions (of `block` each) that holds a position, also one in front of
// the sequence, which no page holds.
SDL_BOTH int64_t block_of(int pos, int block)
{
    // (32 bits: a division of 64 costs some hundred instructions)
    return pos >= 0 ? (int64_t)((uint32_t)pos / (uint32_t)block)
                    : -1 - (int64_t)((uint32_t)~pos / (uint32_t)block);
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

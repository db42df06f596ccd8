// tree.hip -- attention of drafted tokens over a paged cache that holds rows of
// the type of q.  How the work is cut and joined: tree_impl.h.
//
// One answered token of each sequence is bound by the read of the cache: 64
// sequences, 1.39 GB in 225 us = 6.2 TB/s (a plain read reaches 7.1), 6 us
// for the join.  Drafts of up to 64 tokens with 8 heads on one are bound by
// latency, two workgroups to a CU: 23 GFLOP in 73 us and 12 for the join.
#include "tree_impl.h"

namespace sdl {

namespace {

// Where sequences fill one block of 16 queries in the mean, most keys are read
// once, and keeping them in the caches would only push out what is read again.
// (64 answers: 231 us against 255; trees of drafts, several blocks each, 83
// against 76 the other way round.)
template <bool ONCE>
__device__ inline u32x4 load_once(const u32x4 *p)
{
    return ONCE ? __builtin_nontemporal_load(p) : *p;
}

// Workgroups to a CU that registers and LDS allow.
template <class T, int DP>
constexpr int per_cu(int block_rows)
{
    const int tile = 2 * tile_keys(block_rows) * DP * (int)sizeof(T);
    return tile <= 16384 ? 4 : (tile <= 32768 && block_rows == 16 ? 3 : (tile <= 65536 ? 2 : 1));
}

// RG groups of C queries; the 4 / RG wavefronts of a group share the keys of
// a tile.
template <class T, int DP, int DU, int C, int RG>
__global__ __launch_bounds__(kAttnThreads, (per_cu<T, DP>(C * RG))) void tree_attn(TreeArgs a)
{
    constexpr int KS = 4 / RG;                 // wavefronts that share a query group's keys
    constexpr int RB = C * RG;                 // queries of a block
    constexpr int kTileKeys = tile_keys(RB);
    typedef Cols<T, DP, DU, kTileKeys, C> Co;
    typedef typename Co::Acc Acc;
    constexpr int STEPS = Co::kSteps, DB = Co::kBlocks;
    typedef Tile<T, DP, kTileKeys> Tl;
    typedef Tile<float, DP, C> Out;
    constexpr int kPieces = Tl::kPieces, kElems = 16 / (int)sizeof(T);
    constexpr int kPiecesPer = kTileKeys * kPieces / kAttnThreads;
    constexpr int kBytes = 2 * Tl::kBytes > 4 * Out::kBytes ? 2 * Tl::kBytes : 4 * Out::kBytes;
    __shared__ __align__(16) char lds[kBytes];
    __shared__ Drafts drafts;
    __shared__ float tops[4][C], totals[4][C];
    __shared__ int redo[RB];
    __shared__ int64_t place_of[2][kTileKeys];     // of a tile's rows, in the pools

    const int t = threadIdx.x, lane = t & 63, part = lane / C;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int group = a.Hq / a.Hkv;
    const int rg = wave % RG, ks = wave / RG;
    const float c2 = a.scale * kLog2e;
    const Slots slots(a);

    Span span;
    if (!span.begin<T>(a, slots))
        return;
    const int w = span.w;
    int64_t at = span.at, base = span.base;
    const int64_t stop = span.stop;
    int seq = span.seq;

    // ---- the units of the span, one piece after another
    int64_t piece_no = 0;
    while (at < stop) {
        Unit u = unit_of<T>(a, seq);
        int64_t mine = (int64_t)a.Hkv * u.blocks * u.tiles;
        while (at >= base + mine) {            // the next sequence that has tiles
            base += mine;
            ++seq;
            u = unit_of<T>(a, seq);
            mine = (int64_t)a.Hkv * u.blocks * u.tiles;
        }
        const int unit = (int)Spans::divide(at - base, u.tiles);
        const int hk = unit / u.blocks, block = unit % u.blocks;
        const int n0 = (int)(at - base - (int64_t)unit * u.tiles);
        const int n1 = stop - at < u.tiles - n0 ? n0 + (int)(stop - at) : u.tiles;
        const int rows = u.drafts * group;

        // the drafts' positions, and what they see together
        __syncthreads();
        if (t < RB)
            redo[t] = 0;
        if (wave == 3 && a.tree != nullptr)    // (the first ones find the rows)
            find_drafts(a, u, lane, drafts);

        // this lane's query
        const int r = block * RB + C * rg + lane % C;
        const int token = (r < rows ? r : rows - 1) / group, head = hk * group + (r < rows ? r : rows - 1) % group;
        DraftSeen seen;
        seen.ctx = u.ctx;
        seen.drafts = u.drafts;
        seen.window = a.window;
        seen.sinks = a.sinks;
        seen.mask = a.tree != nullptr ? draft_mask(a.tree[u.q_begin + token], u.drafts) : 0;
        seen.pos = a.tree != nullptr ? draft_place(u.ctx, seen.mask) : u.ctx + token;
        seen.place = a.tree != nullptr ? drafts.place : nullptr;
        const T *q = (const T *)a.q + (int64_t)(u.q_begin + token) * a.q_row + head * a.q_head;
        Frag<T> qf[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            qf[s] = Co::kTerms * s + 8 * part < a.D ? load8(q + Co::kTerms * s + 8 * part) : zero_frag<T>();

        Acc O[DB];
#pragma unroll
        for (int d = 0; d < DB; ++d)
            O[d] = Acc(0.0f);
        float top = SDL_NEG_INF, total = 0.0f;

        // Rows pass through registers: a tile's rows are under way while the
        // tile before it is worked on, in both workgroups of a CU, which is
        // what keeps HBM busy (LDS alone could not hold as much).  Where the
        // rows lie is found two tiles ahead, once for each row.
        const int32_t *table = a.table + (int64_t)seq * a.table_stride;
        const T *kp = (const T *)a.k_pages + hk * a.head_stride, *vp = (const T *)a.v_pages + hk * a.head_stride;
        u32x4 pk[kPiecesPer], pv[kPiecesPer];
        int id = 0, in_page = 0;               // in_page < 0: a row that is not read
        auto whole = [&](int n) { return all_seen(a, u, first_key(u, n), first_key(u, n) + kTileKeys - 1); };
        auto find_row = [&](int n) {
            const int j = first_key(u, n) + t;
            in_page = -1;
            if (whole(n) || seen_rows(a, u, drafts)(j)) {
                const int p = j / a.page;
                in_page = j - p * a.page;
                id = table[p];
            }
        };
        auto keep_row = [&](int n) {
            place_of[n & 1][t] = in_page < 0 ? -1 : (int64_t)id * a.page_stride + (int64_t)in_page * a.row_stride;
        };
        auto fetch = [&](int n) {
            const int tt = renewed(t);
            int64_t at[kPiecesPer];            // all of them before the loads, which then go out together
#pragma unroll
            for (int i = 0; i < kPiecesPer; ++i)
                at[i] = place_of[n & 1][(tt + i * kAttnThreads) / kPieces];
            auto load = [&](bool all) {
#pragma unroll
                for (int i = 0; i < kPiecesPer; ++i) {
                    const int p = (tt + i * kAttnThreads) % kPieces;
                    const int d = p * kElems < a.D ? p * kElems : a.D - kElems;
                    if (!all) {
                        pk[i] = u32x4(0);
                        pv[i] = u32x4(0);
                    }
                    if (all || at[i] >= 0) {
                        pk[i] = load_once<C == 16>((const u32x4 *)(kp + at[i] + d));
                        pv[i] = load_once<C == 16>((const u32x4 *)(vp + at[i] + d));
                    }
                }
            };
            if (whole(n))
                load(true);
            else
                load(false);
        };
        if (a.tree != nullptr && !(whole(n0) && (n0 + 1 >= n1 || whole(n0 + 1))))
            __syncthreads();                   // what the drafts see is there
        if (t < kTileKeys) {
            find_row(n0);
            keep_row(n0);
            if (n0 + 1 < n1) {
                find_row(n0 + 1);
                keep_row(n0 + 1);
            }
        }
        __syncthreads();
        fetch(n0);
        for (int n = n0; n < n1; ++n) {
            char *kt = lds, *vt = lds + Tl::kBytes;
#pragma unroll
            for (int i = 0; i < kPiecesPer; ++i) {
                const int m = t + i * kAttnThreads;
                *(u32x4 *)(kt + Tl::at(m / kPieces, m % kPieces)) = pk[i];
                *(u32x4 *)(vt + Tl::at(m / kPieces, m % kPieces)) = pv[i];
            }
            const bool find = t < kTileKeys && n + 2 < n1;
            if (find)
                find_row(n + 2);
            if (n + 1 < n1)
                fetch(n + 1);
            __syncthreads();
#pragma unroll 1
            for (int b = ks; b < kTileKeys / C; b += KS) {
                const int j0 = first_key(u, n) + C * b, j1 = j0 + C - 1;
                if (j0 >= u.end || (j1 < u.low && j0 >= a.sinks) || block * RB + C * rg >= rows)
                    continue;
                const int rows_at = renewed(Co::row_base(lane) + C * b * Tl::kRowBytes);
                const int cols_at = renewed(Co::col_base(lane) + C * b * Tl::kRowBytes);
                Acc x = Acc(0.0f);
                chain<STEPS, 4>([&](int i) { return Co::key_frag(kt, rows_at, i); },
                                [&](int i, Frag<T> f) { x = Co::mul(f, qf[i], x); });
                if (!(j1 < u.ctx && (u.end - 1 - j0 < a.window || j1 < a.sinks))) {
                    const int j = renewed(j0 + 4 * part);
#pragma unroll
                    for (int i = 0; i < Co::kAcc; ++i)
                        if (!seen(j + Co::key_of(i)))
                            x[i] = SDL_NEG_INF;
                }
                const float most = Co::most(x) * c2;
                if (__any(most > top + kLazy)) {
                    const float now = fmaxf(top, most);
                    const float keep = now == SDL_NEG_INF ? 1.0f : __builtin_amdgcn_exp2f(top - now);
                    top = now;
                    total *= keep;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int i = 0; i < Co::kAcc; ++i)
                            O[d][i] *= keep;
                }
                const float ref = top == SDL_NEG_INF ? 0.0f : top;
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < Co::kAcc; ++i) {
                    x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], c2, -ref));
                    sum += x[i];
                }
                total += sum;
                typename Co::Weights pf[Co::kGroups];
#pragma unroll
                for (int i = 0; i < Co::kGroups; ++i)
                    pf[i] = Co::weights(x, i);
                chain<Co::kGroups * DB, 4>(
                    [&](int i) { return Co::val_frag(vt, cols_at, i / DB, i % DB); },
                    [&](int i, typename Co::Weights f) { O[i % DB] = Co::apply(f, pf[i / DB], O[i % DB]); });
            }
            if (find)
                keep_row(n + 2);
            __syncthreads();
        }

        // ---- join the wavefronts of a query group, and write
        total = Co::sum(total);
        if (part == 0) {
            tops[wave][lane] = top;
            totals[wave][lane] = total;
        }
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < Co::kAcc / 4; ++g)
                store4((float *)(lds + wave * Out::kBytes +
                                 Out::at(lane % C, (C * d + Co::key_of(4 * g)) / 4 + part)),
                       O[d][4 * g], O[d][4 * g + 1], O[d][4 * g + 2], O[d][4 * g + 3]);
        __syncthreads();
        join_waves<T, T, DP, DU, C, RG>(a, u, {w, seq, hk, block, n0, n1, piece_no != 0}, slots, lds, tops, totals, redo,
                                        drafts, wave, lane);
        at += n1 - n0;
        ++piece_no;
    }
}

template <class T, int DP, int DU>
hipError_t launch(const TreeArgs &a, hipStream_t stream)
{
    if (a.block_rows == 16)
        tree_attn<T, DP, DU, 16, 1><<<a.workers, kAttnThreads, 0, stream>>>(a);
    else if (a.block_rows == 32)
        tree_attn<T, DP, DU, 32, 1><<<a.workers, kAttnThreads, 0, stream>>>(a);
    else if (a.block_rows == 64)
        tree_attn<T, DP, DU, 32, 2><<<a.workers, kAttnThreads, 0, stream>>>(a);
    else
        tree_attn<T, DP, DU, 32, 4><<<a.workers, kAttnThreads, 0, stream>>>(a);
    return launch_join<T, T, DP, DU>(a, stream);
}

// By the head's size.
template <class T>
hipError_t launch_sized(const TreeArgs &a, hipStream_t stream)
{
    return a.D <= 64 ? launch<T, 64, 64>(a, stream)
                     : (a.D <= 96 ? launch<T, 128, 96>(a, stream) : launch<T, 128, 128>(a, stream));
}

}  // namespace

TreeShape tree_shape(int dtype, int held, int64_t S, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t D)
{
    TreeShape sh = {};
    const int DP = D <= 64 ? 64 : 128;
    // As many queries to a block as the mean sequence fills.  A batch of unlike sequences
    // so costs more than its parts: 64 single tokens over codes 155 us, a piece of 512
    // behind 4096 keys 82, both in one call 300 (q in fp32 169, 186, 614); a piece of 64
    // 46, both 199.  Two calls, over the sequences of either kind, cost the sum.
    sh.rows = S > 0 ? (Tq + S - 1) / S * (Hq / Hkv) : 0;
    sh.block_rows = sh.rows <= 16 ? 16 : (sh.rows <= 32 ? 32 : (sh.rows <= 64 ? 64 : 128));
    sh.wave_heads = 1;
    // as many workgroups as the 256 CUs hold at once
    if (held != 0 && sh.block_rows == 16) {
        // (neighbouring heads together: loads of whole rows of four heads reach 7.0 TB/s,
        // of one 5.9)
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

// window_fwd.hip -- window attention, forward.
//
//   s_ij = scale <q_i, k_j>,  o_i = sum_j softmax_j(s_ij) v_j over the keys
//   that i sees (Seen), lse_i = log sum_j exp(s_ij)
//
// One workgroup takes 32 * RG queries of one head and walks the key tiles
// that any of them sees: the tiles of the first `sinks` keys, then those of
// the window.  Softmax in one pass: running reference and sum in fp32, base 2
// (scale * log2 e is one factor).
//
// Scores are formed transposed, S^T = K q^T, so that a lane holds one query:
// its maximum, its sum and the rescaling of its output are the lane's own
// (the two lanes of a query exchange one value), and the weights are, as
// they lie, the second operand of O^T = V^T P^T.
#include "ops.h"

#include "exact.h"
#include "spmm.h"
#include "tile.h"

namespace sdl {

namespace {

// Keys of a tile.  In bf16, 128 queries to a workgroup, tiles of 32 leave
// room for a third workgroup on a CU (16384 tokens, 32 heads of 128 on 8,
// window 1024: 300 us, against 326 with tiles of 64 and two workgroups, timed in
// turn).
__host__ __device__ constexpr int tile_keys(bool bf16, int rows) { return bf16 && rows == 128 ? 32 : 64; }

// The shape of a call.  128 queries to a workgroup, unless that makes too few
// of them; then either their walks are split, into as many parts as make
// about three rounds of the workgroups that run at once, of at least 512
// keys each, or, where walks are short, 64 queries to a workgroup.  Sequences
// of few queries take 64, and are split too.  (Pieces of 512 queries behind
// 16384 and 9000 keys with two more sequences: 113 us in parts, 141 whole; the
// split of workgroups of 64 takes 129.  257 tokens of 4 heads of 64: 7.8 us
// with 64, 9.3 with 128.)
SplitShape window_split(int dtype, const WindowArgs &a)
{
    SplitShape s = {128, INT32_MAX / 2, 1, nullptr, nullptr};
    if (!few_tiles(a))
        return s;
    const bool bf16 = dtype == SPMM_DTYPE_BF16;
    const int64_t rows = a.Tq >= 96 * (int64_t)a.S ? 128 : 64;
    const int64_t units = (a.Tq / rows + a.S) * a.Hq;
    // no walk is longer than this
    const int64_t reach = (int64_t)a.window + a.sinks + rows;
    const int64_t tiles = (a.Tk < reach ? a.Tk : reach) / tile_keys(bf16, (int)rows) + 3;
    int64_t parts = (2048 + units - 1) / units;
    const int64_t most = tiles * tile_keys(bf16, (int)rows) / 512;
    parts = parts < most ? parts : most;
    if (parts > 1) {
        s.rows = (int32_t)rows;
        s.tiles = (int32_t)((tiles + parts - 1) / parts);
        s.parts = (int32_t)((tiles + s.tiles - 1) / s.tiles);
    } else {
        s.rows = 64;
    }
    return s;
}

// RG groups of 32 queries; the 4 / RG wavefronts of a group share the keys
// of each tile and join their results at the end.
struct Walk {
    int first_tiles, band, count, low;
};

// The key tiles that queries at positions p0 .. p1 see: [0, first_tiles) and
// [band, band + count - first_tiles).
__device__ inline Walk walk_of(const Seen &seen, int p0, int p1, int KT)
{
    Walk w;
    w.low = p0 - seen.window + 1 > 0 ? p0 - seen.window + 1 : 0;
    w.band = w.low / KT;
    w.first_tiles = (seen.sinks + KT - 1) / KT;
    w.first_tiles = w.first_tiles < w.band ? w.first_tiles : w.band;
    w.count = p1 < 0 ? 0 : w.first_tiles + p1 / KT + 1 - w.band;
    return w;
}

// Computes rows again that came out non-finite, where that is called for:
// bits 0 .. 31 (and the same again from 32) of `redo` are queries wi0 .., lane
// n holds the log-sum of query n.
template <class T, int DU>
__device__ inline void again(const WindowArgs &a, const Seen &seen, uint64_t redo, float lse, int wi0, int wp0,
                             int p1, const Walk &walk, int KT, int q_begin, int k_begin, int lk, int shift, int head,
                             int hk, int lane)
{
    if (redo == 0)
        return;
    const T *K = (const T *)a.k.base + (int64_t)k_begin * a.k.row_stride + hk * a.k.head_stride;
    const T *V = (const T *)a.v.base + (int64_t)k_begin * a.v.row_stride + hk * a.v.head_stride;
    auto key_row = [&](int j) { return K + (int64_t)j * a.k.row_stride; };
    auto val_row = [&](int j) { return V + (int64_t)j * a.v.row_stride; };
    const bool odd = odd_masked_keys<T>(seen, key_row, val_row, wp0, p1, walk.first_tiles, walk.band, KT, lk, a.D, lane);
    TooLarge<T> too_large;
    if (!odd && (redo & __ballot(finite(lse))) != 0) {
        const int lo = wp0 - seen.window + 1 > 0 ? wp0 - seen.window + 1 : 0;
        auto every = [](int) { return true; };
        too_large.look(val_row, every, 0, seen.sinks < lo ? seen.sinks : lo, a.D, lane);
        too_large.look(val_row, every, lo, p1 + 1, a.D, lane);
        __threadfence_block();                 // the outputs, which other lanes stored
    }
    for (uint32_t left = (uint32_t)(redo | (redo >> 32)); left != 0; left &= left - 1) {
        const int n = __ffs(left) - 1, i = wi0 + n, p = i + shift;
        T *o = (T *)a.o.base + (int64_t)(q_begin + i) * a.o.row_stride + head * a.o.head_stride;
        // (a sum of weights that is not finite says too little: an infinite
        // score, a score that is no number, or an infinite key times the zeros
        // past D)
        const bool have_lse = finite(__shfl(lse, n));
        if (!odd && have_lse && !too_large(o, a.D, lane))
            continue;
        const int lo = p - seen.window + 1 > 0 ? p - seen.window + 1 : 0;
        exact_row<T>(
            (const T *)a.q.base + (int64_t)(q_begin + i) * a.q.row_stride + head * a.q.head_stride, key_row,
            val_row, [&](int j) { return seen(p, j); }, seen.sinks < lo ? seen.sinks : lo, lo, p + 1, a.D,
            a.scale * kLog2e, o, a.lse + (int64_t)head * a.Tq + q_begin + i, have_lse, lane);
    }
}

// The walk of a workgroup may be split over several (SplitShape): each takes
// split.tiles key tiles of it, and what they leave is joined by window_join.
//
// No unit bounds it alone.  16384 tokens, 32 heads of 128 on 8, window 1024,
// bf16: 303 - 316 us, 770 TFLOP/s of pairs that are seen; matrix instructions
// keep 41 % of the cycles busy, VALU instructions 50 %, and LDS reads take 63 %
// of what they take in a loop of nothing else (a third of that is bank
// conflicts of the transposing reads).  Within a wavefront products, softmax and
// products follow each other, and overlap only between wavefronts of a SIMD, of
// which three workgroups on a CU give three (tile_keys).
template <class T, int DP, int DU, int RG>
__global__ __launch_bounds__(kAttnThreads, sizeof(T) == 2 ? (RG == 4 ? 3 : 2) : 1) void window_fwd(WindowArgs a, int slots, SplitShape split)
{
    constexpr int KT = tile_keys(sizeof(T) == 2, 32 * RG);
    constexpr int KS = 4 / RG;                   // wavefronts of a group
    constexpr int NB = KT / 32 / KS;             // 32-key blocks of a wavefront
    constexpr int STEPS = DU / 16, DB = DU / 32;
    constexpr int kRows = 32 * RG;
    constexpr int kAhead = sizeof(T) == 2 ? 6 : 2;
    typedef Tile<T, DP, KT> Tl;
    // K and V, two buffers of each; four objects, so that the compiler sees
    // that reading one does not wait for loads into another
    __shared__ __align__(16) char k_even[Tl::kBytes], v_even[Tl::kBytes], k_odd[Tl::kBytes], v_odd[Tl::kBytes];
    __shared__ float parked_top[4][32], parked_total[4][32];

    const int group = a.Hq / a.Hkv;
    const int idx = xcd_order(blockIdx.x, gridDim.x);
    const int hk = idx / (slots * group), rest = idx % (slots * group);
    const int head = hk * group + rest % group;
    // late tiles (the long ones without a window) first
    const SeqTile st = find_seq_tile(a.q_rowptr, a.S, kRows, slots - 1 - rest / group);
    if (st.seq < 0)
        return;
    const int q_begin = a.q_rowptr[st.seq], lq = a.q_rowptr[st.seq + 1] - q_begin;
    const int k_begin = a.k_rowptr[st.seq], lk = a.k_rowptr[st.seq + 1] - k_begin;
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ks = KS == 1 ? 0 : wave / RG;
    const Seen seen = {a.window, a.sinks};
    const int shift = lk - lq;
    const int i0 = st.tile * kRows, i1 = (i0 + kRows < lq ? i0 + kRows : lq) - 1;
    const int wi0 = i0 + 32 * (wave % RG);                // the wavefront's queries
    const int qi = wi0 + (lane & 31);
    const int pos = qi + shift;
    const int wp0 = wi0 + shift, wp1 = (wi0 + 31 < i1 ? wi0 + 31 : i1) + shift;
    const float c2 = a.scale * kLog2e;

    const T *K = (const T *)a.k.base + (int64_t)k_begin * a.k.row_stride + hk * a.k.head_stride;
    const T *V = (const T *)a.v.base + (int64_t)k_begin * a.v.row_stride + hk * a.v.head_stride;
    const T *Q = (const T *)a.q.base + (int64_t)(q_begin + (qi < lq ? qi : lq - 1)) * a.q.row_stride +
                 head * a.q.head_stride;

    const int p0 = i0 + shift, p1 = i1 + shift;
    const Walk walk = walk_of(seen, p0, p1, KT);
    const int first_tiles = walk.first_tiles, band = walk.band;
    // this workgroup's part of the walk
    const bool whole_walk = walk.count <= split.tiles;
    const int from = blockIdx.y * split.tiles;
    const int count = walk.count < from + split.tiles ? walk.count : from + split.tiles;
    if (blockIdx.y > 0 && from >= count)
        return;

    const Stager<T, DP, KT, 4> k_in(a.k.row_stride, a.D), v_in(a.v.row_stride, a.D);
    auto first_key = [&](int n) { return (n < first_tiles ? n : band + n - first_tiles) * KT; };
    auto fetch = [&](int n, char *kt, char *vt) {
        k_in.load(kt, K, first_key(n), lk - 1, wave);
        v_in.load(vt, V, first_key(n), lk - 1, wave);
    };
    if (count > from)
        fetch(from, k_even, v_even);

    Frag<T> qf[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
        qf[s] = 16 * s + 8 * half < a.D ? load8(Q + 16 * s + 8 * half) : zero_frag<T>();

    f32x16 O[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
        O[d] = f32x16(0.0f);
    float top = SDL_NEG_INF, total = 0.0f;

    auto compute = [&](int n, const char *kt, const char *vt) {
        const int j0 = first_key(n) + 32 * NB * ks, j1 = j0 + 32 * NB - 1;
        if (wi0 > i1 || seen.none(wp0, wp1, j0, j1))
            return;
        const int rows_at = renewed(Tl::row_base(lane) + 32 * NB * ks * Tl::kRowBytes);
        const int cols_at = renewed(Tl::col_base(lane) + 32 * NB * ks * Tl::kRowBytes);
        f32x16 x[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b)
            x[b] = f32x16(0.0f);
        chain<NB * STEPS, kAhead>(
            [&](int i) { return Tl::row_frag(kt, rows_at, i / STEPS, i % STEPS); },
            [&](int i, Frag<T> f) { x[i / STEPS] = mma(f, qf[i % STEPS], x[i / STEPS]); });
        if (!seen.all(wp0, wp1, j0, j1)) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
                mask_keys(seen, pos, j0 + 32 * b, half, x[b]);
        }
        float most = max_of(x[0]);
#pragma unroll
        for (int b = 1; b < NB; ++b)
            most = fmaxf(most, max_of(x[b]));
        most = max_halves(most) * c2;
        if (__any(most > top + kLazy)) {
            const float now = fmaxf(top, most);
            const float keep = now == SDL_NEG_INF ? 1.0f : __builtin_amdgcn_exp2f(top - now);
            top = now;
            total *= keep;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    O[d][r] *= keep;
        }
        const float base = top == SDL_NEG_INF ? 0.0f : top;
        float sum = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                x[b][r] = __builtin_amdgcn_exp2f(fmaf(x[b][r], c2, -base));
                sum += x[b][r];
            }
        total += sum;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Frag<T> pf = result_frag<T>(x[b], s);
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    O[d] = mma(Tl::col_frag(vt, cols_at, 2 * b + s, d), pf, O[d]);
            }
    };
    wait_loads();
    __syncthreads();
    for (int n = from; n < count; n += 2) {
        if (n + 1 < count)
            fetch(n + 1, k_odd, v_odd);
        compute(n, k_even, v_even);
        wait_loads();
        __syncthreads();
        if (n + 1 >= count)
            break;
        if (n + 2 < count)
            fetch(n + 2, k_even, v_even);
        compute(n + 1, k_odd, v_odd);
        wait_loads();
        __syncthreads();
    }

    total = sum_halves(total);
    if constexpr (KS == 2) {
        static_assert(RG == 2 && Parked<DP, DU>::kBytes <= Tl::kBytes, "a buffer for each group");
        char *room = wave % RG == 0 ? k_even : k_odd;
        if (ks == 1) {
            Parked<DP, DU>::put(room, lane, O);
            if (half == 0) {
                parked_top[wave % RG][lane] = top;
                parked_total[wave % RG][lane] = total;
            }
        }
        __syncthreads();
        if (ks == 1)
            return;
        const float other = parked_top[wave % RG][lane & 31];
        const float now = fmaxf(top, other), base = now == SDL_NEG_INF ? 0.0f : now;
        const float mine = __builtin_amdgcn_exp2f(top - base), theirs = __builtin_amdgcn_exp2f(other - base);
        Parked<DP, DU>::add(room, lane, mine, theirs, O);
        total = fmaf(theirs, parked_total[wave % RG][lane & 31], mine * total);
        top = now;
    }
    if (wi0 > i1)
        return;
    if (!whole_walk) {
        // a part: left for window_join
        const int64_t row = ((int64_t)idx * split.parts + blockIdx.y) * kRows + 32 * (wave % RG) + (lane & 31);
        if (half == 0) {
            split.stat[2 * row] = top;
            split.stat[2 * row + 1] = total;
        }
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                store4(split.out + row * DU + 32 * d + 8 * g + 4 * half, O[d][4 * g], O[d][4 * g + 1],
                       O[d][4 * g + 2], O[d][4 * g + 3]);
        return;
    }
    const bool some = pos >= 0;                 // window >= 1: a query sees its own position
    const float inv = 1.0f / total;
    const float lse = some ? kLn2 * (top + __builtin_amdgcn_logf(total)) : SDL_NEG_INF;
    bool clean = finite(lse);
    T *out = (T *)a.o.base + (int64_t)(q_begin + qi) * a.o.row_stride + head * a.o.head_stride;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            if (32 * d + 8 * g < a.D) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[e] = some ? O[d][4 * g + e] * inv : 0.0f;
                    clean = clean && finite(y[e]);
                }
                if (qi <= i1)
                    store4(out + 32 * d + 8 * g + 4 * half, y[0], y[1], y[2], y[3]);
            }
    if (qi <= i1 && half == 0)
        a.lse[(int64_t)head * a.Tq + q_begin + qi] = lse;

    again<T, DU>(a, seen, __ballot(!clean && some && qi <= i1), lse, wi0, wp0, p1, walk, KT, q_begin, k_begin, lk,
                 shift, head, hk, lane);
}

// Joins the parts of walks that were split: 16 of a workgroup's queries to
// each workgroup, a thread to four elements of two of them.
template <class T, int DU>
__global__ __launch_bounds__(kAttnThreads) void window_join(WindowArgs a, int slots, SplitShape split)
{
    constexpr int kPieces = DU / 4;
    const int kRows = split.rows, KT = tile_keys(sizeof(T) == 2, split.rows);
    __shared__ float sums[16];
    __shared__ int odd[16];
    const int group = a.Hq / a.Hkv;
    const int idx = blockIdx.x, row0 = blockIdx.y * 16;
    const int hk = idx / (slots * group), rest = idx % (slots * group);
    const int head = hk * group + rest % group;
    const SeqTile st = find_seq_tile(a.q_rowptr, a.S, kRows, slots - 1 - rest / group);
    if (st.seq < 0)
        return;
    const int q_begin = a.q_rowptr[st.seq], lq = a.q_rowptr[st.seq + 1] - q_begin;
    const int k_begin = a.k_rowptr[st.seq], lk = a.k_rowptr[st.seq + 1] - k_begin;
    const Seen seen = {a.window, a.sinks};
    const int shift = lk - lq;
    const int i0 = st.tile * kRows, i1 = (i0 + kRows < lq ? i0 + kRows : lq) - 1;
    const Walk walk = walk_of(seen, i0 + shift, i1 + shift, KT);
    if (walk.count <= split.tiles || i0 + row0 > i1)
        return;
    const int parts = (walk.count + split.tiles - 1) / split.tiles;
    if (threadIdx.x < 16)
        odd[threadIdx.x] = 0;
    __syncthreads();
    for (int m = threadIdx.x; m < 16 * kPieces; m += kAttnThreads) {
        const int lr = m / kPieces, p = m % kPieces, i = i0 + row0 + lr;
        if (i > i1)
            break;
        float best = SDL_NEG_INF, sum = 0.0f;
        f32x4 o = f32x4(0.0f);
#pragma unroll 4
        for (int n = 0; n < parts; ++n) {
            const int64_t row = ((int64_t)idx * split.parts + n) * kRows + row0 + lr;
            const float top = split.stat[2 * row], total = split.stat[2 * row + 1];
            const f32x4 x = *(const f32x4 *)(split.out + row * DU + 4 * p);
            const float now = fmaxf(best, top), ref = now == SDL_NEG_INF ? 0.0f : now;
            const float mine = __builtin_amdgcn_exp2f(best - ref), theirs = __builtin_amdgcn_exp2f(top - ref);
            best = now;
            sum = fmaf(theirs, total, mine * sum);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = fmaf(theirs, x[e], mine * o[e]);
        }
        const bool some = i + shift >= 0;
        const float inv = 1.0f / sum;
        const float lse = some ? kLn2 * (best + __builtin_amdgcn_logf(sum)) : SDL_NEG_INF;
        bool clean = finite(lse) || !some;
        if (4 * p < a.D) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[e] = some ? o[e] * inv : 0.0f;
                clean = clean && finite(y[e]);
            }
            store4((T *)a.o.base + (int64_t)(q_begin + i) * a.o.row_stride + head * a.o.head_stride + 4 * p, y[0],
                   y[1], y[2], y[3]);
        }
        if (p == 0) {
            a.lse[(int64_t)head * a.Tq + q_begin + i] = lse;
            sums[lr] = lse;
        }
        if (!clean)
            atomicOr(&odd[lr], 1);
    }
    __syncthreads();
    const int lane = threadIdx.x;
    if (lane >= 64)
        return;
    const bool redo = lane < 16 && odd[lane & 15] != 0;
    again<T, DU>(a, seen, __ballot(redo), sums[lane & 15], i0 + row0, i0 + row0 + shift, i1 + shift, walk, KT, q_begin,
                 k_begin, lk, shift, head, hk, lane);
}

template <class T, int DP, int DU>
hipError_t launch_rows(const WindowArgs &a, hipStream_t stream)
{
    SplitShape split = window_split(sizeof(T) == 2 ? SPMM_DTYPE_BF16 : SPMM_DTYPE_F32, a);
    const int64_t slots = a.Tq / split.rows + a.S;
    const uint32_t units = (uint32_t)(slots * a.Hq);
    split.stat = a.partial;
    split.out = a.partial + (int64_t)units * split.parts * split.rows * 2;
    if (split.rows == 128)
        window_fwd<T, DP, DU, 4><<<dim3(units, split.parts), kAttnThreads, 0, stream>>>(a, (int)slots, split);
    else
        window_fwd<T, DP, DU, 2><<<dim3(units, split.parts), kAttnThreads, 0, stream>>>(a, (int)slots, split);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || split.parts == 1)
        return err;
    window_join<T, DU><<<dim3(units, split.rows / 16), kAttnThreads, 0, stream>>>(a, (int)slots, split);
    return hipGetLastError();
}

}  // namespace

int64_t window_fwd_scratch_bytes(int dtype, const WindowArgs &a)
{
    const SplitShape split = window_split(dtype, a);
    if (split.parts == 1)
        return 0;
    const int64_t DU = a.D <= 64 ? 64 : (a.D <= 96 ? 96 : 128);
    return (a.Tq / split.rows + a.S) * a.Hq * split.parts * split.rows * (2 + DU) * 4;
}

int64_t window_fwd_threads(int dtype, const WindowArgs &a)
{
    return (a.Tq / window_split(dtype, a).rows + a.S) * a.Hq * kAttnThreads;
}

hipError_t launch_window_fwd(int dtype, const WindowArgs &a, hipStream_t stream)
{
    if (dtype == SPMM_DTYPE_BF16)
        return a.D <= 64 ? launch_rows<__bf16, 64, 64>(a, stream)
                         : (a.D <= 96 ? launch_rows<__bf16, 128, 96>(a, stream) : launch_rows<__bf16, 128, 128>(a, stream));
    return a.D <= 64 ? launch_rows<float, 64, 64>(a, stream)
                     : (a.D <= 96 ? launch_rows<float, 128, 96>(a, stream) : launch_rows<float, 128, 128>(a, stream));
}

}  // namespace sdl

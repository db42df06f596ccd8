// window_bwd.hip -- window attention, backward.
//
//   p_ij = exp(s_ij - lse_i)             delta_i = <do_i, o_i>
//   dv_j = sum_i p_ij do_i               ds_ij = p_ij (<do_i, v_j> - delta_i)
//   dq_i = scale sum_j ds_ij k_j         dk_j = scale sum_i ds_ij q_i
//
// Two passes that each form the weights again from q, k and lse: one over
// keys for dq (queries stay with a workgroup, as in the forward), one over
// queries for dk and dv (keys stay).  No sum is spread over workgroups by
// atomic adds, so gradients repeat bit for bit; the price is 7 products of
// the pair matrix instead of 5.  The queries of all heads that share a key
// head are taken one after another by the workgroup that owns the keys.
//
// The first `sinks` keys are seen by every later query.  Their workgroup
// would walk the whole sequence while the others walk one window, so what
// lies past its window is cut into runs of queries with a workgroup each;
// those and the window's part leave fp32 partial sums, which a last small
// launch adds in a fixed order.  Where key tiles are few, their windows are
// taken in parts too (dkv_parts).
//
// delta is formed from o as the forward pass stored it.  In bf16 it carries o's
// rounding, which is what remains in dq and dk where <do_i, v_j> - delta_i
// cancels (windows of few keys: off by 0.0037 of their norm for 2 keys, 0.0025
// from 16 on, where rounding alone is 0.0017).  An exact one would need the
// products with k and v once more before this pass.
//
// 8192 tokens, 32 heads of 128 on 8, window 1024, bf16 (forward 136 us): dq
// 188 us, dk and dv 292, the join 5.  dq keeps the matrix cores busy 41 % of
// the cycles, as the forward does; dk and dv, with 128 accumulator registers
// a lane for two gradients, have two workgroups on a CU and 36 %.  fp32 is nearer
// to its bound (54 % in dk and dv): its matrix instructions are 16 times slower,
// so everything else hides behind them.
#include "ops.h"

#include "exact.h"
#include "spmm.h"
#include "tile.h"

namespace sdl {

namespace {

constexpr int kKeyRows = 64;      // keys of a dk/dv workgroup
constexpr int kStepRows = 64;     // queries of one step of it

template <class T>
__device__ GradRows<T> grad_rows(const WindowArgs &a, int q_begin, int k_begin, int head, int hk)
{
    GradRows<T> r;
    r.q = (const T *)a.q.base + (int64_t)q_begin * a.q.row_stride + head * a.q.head_stride;
    r.k = (const T *)a.k.base + (int64_t)k_begin * a.k.row_stride + hk * a.k.head_stride;
    r.v = (const T *)a.v.base + (int64_t)k_begin * a.v.row_stride + hk * a.v.head_stride;
    r.dout = (const T *)a.dout.base + (int64_t)q_begin * a.dout.row_stride + head * a.dout.head_stride;
    r.q_stride = a.q.row_stride;
    r.k_stride = a.k.row_stride;
    r.v_stride = a.v.row_stride;
    r.dout_stride = a.dout.row_stride;
    r.lse = a.lse + (int64_t)head * a.Tq + q_begin;
    r.delta = a.delta + (int64_t)head * a.Tq + q_begin;
    return r;
}

// lse in base 2, of a query at position pos.  One that sees nothing (pos < 0)
// has -infinity, which against a masked score would be no number; any finite
// value gives it weights of 0.  One whose scores are all -infinity has the
// same sum, and its weights are no numbers.
__device__ inline float base2(float lse, int pos) { return pos < 0 ? 0.0f : lse * kLog2e; }

// ------------------------------------------------------------------- dq

template <class T, int DP, int DU, int RG>
__global__ __launch_bounds__(kAttnThreads, sizeof(T) == 2 ? 2 : 1) void window_dq(WindowArgs a, int slots)
{
    constexpr int KT = 64;                       // keys of a tile
    constexpr int KS = 4 / RG;                   // wavefronts that share a group's keys
    constexpr int NB = KT / 32 / KS;             // 32-key blocks of a wavefront
    constexpr int STEPS = DU / 16, DB = DU / 32;
    constexpr int kRows = 32 * RG;
    constexpr int kAhead = sizeof(T) == 2 ? 6 : 2;
    typedef Tile<T, DP, KT> Tl;
    __shared__ __align__(16) char k_even[Tl::kBytes], v_even[Tl::kBytes], k_odd[Tl::kBytes], v_odd[Tl::kBytes];

    const int group = a.Hq / a.Hkv;
    const int idx = xcd_order(blockIdx.x, gridDim.x);
    const int hk = idx / (slots * group), rest = idx % (slots * group);
    const int head = hk * group + rest % group;
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
    const int wi0 = i0 + 32 * (wave % RG);
    const int qi = wi0 + (lane & 31);
    const int pos = qi + shift;
    const int wp0 = wi0 + shift, wp1 = (wi0 + 31 < i1 ? wi0 + 31 : i1) + shift;
    const float c2 = a.scale * kLog2e;
    const GradRows<T> r = grad_rows<T>(a, q_begin, k_begin, head, hk);
    const int row = qi < lq ? qi : lq - 1;

    const int p0 = i0 + shift, p1 = i1 + shift;
    const int low = p0 - seen.window + 1 > 0 ? p0 - seen.window + 1 : 0;
    const int band = low / KT;
    int first_tiles = (seen.sinks + KT - 1) / KT;
    first_tiles = first_tiles < band ? first_tiles : band;
    const int count = p1 < 0 ? 0 : first_tiles + p1 / KT + 1 - band;

    const Stager<T, DP, KT, 4> k_in(r.k_stride, a.D), v_in(r.v_stride, a.D);
    auto first_key = [&](int n) { return (n < first_tiles ? n : band + n - first_tiles) * KT; };
    auto fetch = [&](int n, char *kt, char *vt) {
        k_in.load(kt, r.k, first_key(n), lk - 1, wave);
        v_in.load(vt, r.v, first_key(n), lk - 1, wave);
    };
    if (count > 0)
        fetch(0, k_even, v_even);

    Frag<T> qf[STEPS], gf[STEPS];
    float delta = 0.0f;
    {
        const T *q = r.q + (int64_t)row * r.q_stride, *g = r.dout + (int64_t)row * r.dout_stride;
        const T *o = (const T *)a.out.base + (int64_t)(q_begin + row) * a.out.row_stride +
                     head * a.out.head_stride;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int d = 16 * s + 8 * half;
            qf[s] = d < a.D ? load8(q + d) : zero_frag<T>();
            gf[s] = d < a.D ? load8(g + d) : zero_frag<T>();
            const Frag<T> of = d < a.D ? load8(o + d) : zero_frag<T>();
#pragma unroll
            for (int e = 0; e < 8; ++e)
                delta = fmaf((float)gf[s][e], (float)of[e], delta);
        }
        delta = sum_halves(delta);
        if (qi <= i1 && half == 0 && ks == 0)
            a.delta[(int64_t)head * a.Tq + q_begin + qi] = delta;
    }
    const float lse2 = base2(r.lse[row], row + shift);

    f32x16 dQ[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
        dQ[d] = f32x16(0.0f);

    auto compute = [&](int n, const char *kt, const char *vt) {
        if (wi0 > i1)
            return;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int j0 = first_key(n) + 32 * (NB * ks + b);
            if (seen.none(wp0, wp1, j0, j0 + 31))
                continue;
            const int rows_at = renewed(Tl::row_base(lane) + 32 * NB * ks * Tl::kRowBytes);
            const int cols_at = renewed(Tl::col_base(lane) + 32 * NB * ks * Tl::kRowBytes);
            f32x16 x = f32x16(0.0f), dp = f32x16(0.0f);
            chain<2 * STEPS, kAhead>(
                [&](int i) { return Tl::row_frag(i & 1 ? vt : kt, rows_at, b, i >> 1); },
                [&](int i, Frag<T> f) {
                    if (i & 1)
                        dp = mma(f, gf[i >> 1], dp);
                    else
                        x = mma(f, qf[i >> 1], x);
                });
            if (!seen.all(wp0, wp1, j0, j0 + 31))
                mask_keys(seen, pos, j0, half, x, dp);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], c2, -lse2)) * (dp[i] - delta);
            const Frag<T> df[2] = {result_frag<T>(x, 0), result_frag<T>(x, 1)};
            chain<2 * DB, kAhead>(
                [&](int i) { return Tl::col_frag(kt, cols_at, 2 * b + i / DB, i % DB); },
                [&](int i, Frag<T> f) { dQ[i % DB] = mma(f, df[i / DB], dQ[i % DB]); });
        }
    };
    wait_loads();
    __syncthreads();
    for (int n = 0; n < count; n += 2) {
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

    if constexpr (KS == 2) {
        static_assert(RG == 2 && Parked<DP, DU>::kBytes <= Tl::kBytes, "a buffer for each group");
        char *room = wave % RG == 0 ? k_even : k_odd;
        if (ks == 1)
            Parked<DP, DU>::put(room, lane, dQ);
        __syncthreads();
        if (ks == 1)
            return;
        Parked<DP, DU>::add(room, lane, 1.0f, 1.0f, dQ);
    }
    if (wi0 > i1)
        return;
    const bool some = pos >= 0;
    bool clean = true;
    T *out = (T *)a.dq.base + (int64_t)(q_begin + qi) * a.dq.row_stride + head * a.dq.head_stride;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            if (32 * d + 8 * g < a.D) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[e] = some ? dQ[d][4 * g + e] * a.scale : 0.0f;
                    clean = clean && finite(y[e]);
                }
                if (qi <= i1)
                    store4(out + 32 * d + 8 * g + 4 * half, y[0], y[1], y[2], y[3]);
            }
    const uint64_t redo = __ballot(!clean && qi <= i1);
    if (redo == 0)
        return;
    // (an infinity times the zeros past D is no number either)
    if (a.D == DU &&
        !odd_masked_keys<T>(
            seen, [&](int j) { return r.k + (int64_t)j * r.k_stride; },
            [&](int j) { return r.v + (int64_t)j * r.v_stride; }, wp0, p1, first_tiles, band, KT, lk, a.D, lane))
        return;
    for (uint32_t left = (uint32_t)(redo | (redo >> 32)); left != 0; left &= left - 1) {
        const int n = __ffs(left) - 1, i = wi0 + n, p = i + shift;
        const int lo = p - seen.window + 1 > 0 ? p - seen.window + 1 : 0;
        // delta of the row, stored above by this wavefront, is not read back:
        // the lane that holds it hands it out
        exact_dq_row<T>(
            r, i, __shfl(delta, n), [&](int j) { return seen(p, j); },
            seen.sinks < lo ? seen.sinks : lo, lo, p + 1, a.D, c2, a.scale,
            (T *)a.dq.base + (int64_t)(q_begin + i) * a.dq.row_stride + head * a.dq.head_stride, lane);
    }
}

// ---------------------------------------------------------------- dk, dv

// The queries that a key tile j0 .. j1 meets within the window, in steps of
// kStepRows: [from, to).  The rest of the sequence is far (first keys only).
struct StepRange {
    int from, to;
};

__device__ inline StepRange window_steps(int j0, int j1, int window, int shift, int lq)
{
    const int lo = j0 - shift > 0 ? j0 - shift : 0;
    int64_t hi = (int64_t)j1 + window - shift;
    hi = hi < lq ? hi : lq;
    hi = hi > 0 ? hi : 0;
    StepRange r;
    r.to = (int)((hi + kStepRows - 1) / kStepRows);
    r.from = lo / kStepRows < r.to ? lo / kStepRows : r.to;
    return r;
}

// fp32 partial sums of the first keys: [run][key head][key][dk | dv][DP];
// run = a far run's number, or far_slots + sequence for the window's part.
__device__ inline float *partial_at(const WindowArgs &a, int run, int hk, int key, int DP)
{
    return a.partial + (((int64_t)run * a.Hkv + hk) * a.sinks + key) * 2 * DP;
}

// Whether one of queries from .. to - 1, of any head that shares key head hk,
// has something that is not finite.
template <class T>
__device__ bool odd_queries(const WindowArgs &a, int q_begin, int k_begin, int hk, int from, int to, int lane)
{
    const int group = a.Hq / a.Hkv;
    bool odd = false;
    for (int g = 0; g < group && !odd; ++g) {
        const GradRows<T> r = grad_rows<T>(a, q_begin, k_begin, hk * group + g, hk);
        for (int i = from + lane; i < to; i += 64)
            odd = odd || r.lse[i] != r.lse[i] || !finite(r.delta[i]);
        odd = __any(odd) ||
              any_odd([&](int i) { return r.q + (int64_t)i * r.q_stride; }, from, to, a.D, lane) ||
              any_odd([&](int i) { return r.dout + (int64_t)i * r.dout_stride; }, from, to, a.D, lane);
    }
    return odd;
}

template <class T>
__device__ void exact_dkv_row(const WindowArgs &a, int q_begin, int k_begin, int lq, int lk, int hk,
                              int j, int lane)
{
    const Seen seen = {a.window, a.sinks};
    const int group = a.Hq / a.Hkv, shift = lk - lq;
    float dk[2] = {0.0f, 0.0f}, dv[2] = {0.0f, 0.0f};
    int64_t end = j < seen.sinks ? lq : (int64_t)j + seen.window - shift;
    end = end < lq ? end : lq;
    for (int g = 0; g < group; ++g)
        exact_dkv_add<T>(
            grad_rows<T>(a, q_begin, k_begin, hk * group + g, hk), j,
            [&](int i) { return seen(i + shift, j); }, j - shift > 0 ? j - shift : 0, (int)end, a.D,
            a.scale * kLog2e, lane, dk, dv);
    T *k = (T *)a.dk.base + (int64_t)(k_begin + j) * a.dk.row_stride + hk * a.dk.head_stride;
    T *v = (T *)a.dv.base + (int64_t)(k_begin + j) * a.dv.row_stride + hk * a.dv.head_stride;
    put_row(k, dk[0] * a.scale, dk[1] * a.scale, a.D, lane);
    put_row(v, dv[0], dv[1], a.D, lane);
}

// Where part `part` of key tile `unit` leaves 32 of its keys' sums (keys 32 * kw
// on): registers in turn, a lane's four elements behind each other.
template <int DU>
__device__ inline float *sums_at(float *sums, int unit, int parts, int part, int kw)
{
    return sums + (((int64_t)unit * parts + part) * 2 + kw) * (2 * DU * 32);
}

// Computes rows of keys again that came out non-finite, where that is called
// for: bits 0 .. 31 (and the same again from 32) of `redo` are keys wj0 .. wj1;
// steps: the queries that the tile met; has_far: for first keys, far runs too.
template <class T, int DU>
__device__ inline void again_dkv(const WindowArgs &a, const Seen &seen, uint64_t redo, const StepRange &steps,
                                 bool has_far, int wj0, int wj1, int q_begin, int k_begin, int lq, int lk, int hk, int lane)
{
    if (redo == 0)
        return;
    // queries of the steps that a key of this wavefront does not see: before
    // the keys, and behind the window (a step's missing rows repeat the last,
    // the last step of the far runs included)
    const int shift = lk - lq;
    const int before = wj1 - shift < lq ? wj1 - shift : lq;
    int behind = wj0 + seen.window - shift < lq - 1 ? wj0 + seen.window - shift : lq - 1;
    behind = behind > 0 ? behind : 0;
    const int end = steps.to * kStepRows < lq ? steps.to * kStepRows : lq;
    if (a.D == DU && !odd_queries<T>(a, q_begin, k_begin, hk, steps.from * kStepRows, before, lane) &&
        !odd_queries<T>(a, q_begin, k_begin, hk, behind, end, lane) &&
        !(has_far && odd_queries<T>(a, q_begin, k_begin, hk, lq - 1, lq, lane)))
        return;
    for (uint32_t left = (uint32_t)(redo | (redo >> 32)); left != 0; left &= left - 1)
        exact_dkv_row<T>(a, q_begin, k_begin, lq, lk, hk, wj0 + __ffs(left) - 1, lane);
}

// Two wavefronts share 32 keys and take the halves of each step's queries;
// their sums are joined at the end.  Where there are few key tiles, the
// queries of a tile are taken in gridDim.y parts (dkv_parts), which leave
// their sums for window_dkv_parts.
template <class T, int DP, int DU>
__global__ __launch_bounds__(kAttnThreads, sizeof(T) == 2 ? 2 : 1) void window_dkv(WindowArgs a, int key_slots,
                                                                                   int far_slots, int far_tiles,
                                                                                   int far_rows, float *sums)
{
    constexpr int QT = kStepRows, STEPS = DU / 16, DB = DU / 32;
    constexpr int kAhead = sizeof(T) == 2 ? 3 : 2;   // 317 us of a training step; 4: 358, 2: 319
    typedef Tile<T, DP, QT> Tl;
    __shared__ __align__(16) char q_even[Tl::kBytes], g_even[Tl::kBytes], q_odd[Tl::kBytes], g_odd[Tl::kBytes];
    __shared__ __align__(16) float stat_even[2 * QT], stat_odd[2 * QT];    // lse, delta

    const int group = a.Hq / a.Hkv;
    const int far_items = far_slots * far_tiles;
    const int per_head = key_slots + far_items;
    const int idx = xcd_order(blockIdx.x, gridDim.x);
    const int hk = idx / per_head, rest = idx % per_head;
    const bool far = rest < far_items;
    const int parts = gridDim.y, part_no = blockIdx.y;
    if (far && part_no > 0)
        return;
    const SeqTile st = far ? find_seq_tile(a.q_rowptr, a.S, far_rows, rest / far_tiles)
                           : find_seq_tile(a.k_rowptr, a.S, kKeyRows, rest - far_items);
    if (st.seq < 0)
        return;
    const int q_begin = a.q_rowptr[st.seq], lq = a.q_rowptr[st.seq + 1] - q_begin;
    const int k_begin = a.k_rowptr[st.seq], lk = a.k_rowptr[st.seq + 1] - k_begin;
    const int j0 = (far ? rest % far_tiles : st.tile) * kKeyRows;
    if (j0 >= lk)
        return;
    const int t = threadIdx.x, lane = t & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int kw = wave & 1, qw = wave >> 1;
    const Seen seen = {a.window, a.sinks};
    const int shift = lk - lq;
    const int j1 = (j0 + kKeyRows < lk ? j0 + kKeyRows : lk) - 1;
    const int wj0 = j0 + 32 * kw, wj1 = wj0 + 31 < j1 ? wj0 + 31 : j1;
    const int key = wj0 + (lane & 31);
    const float c2 = a.scale * kLog2e;

    StepRange steps = window_steps(j0, j1, seen.window, shift, lq);
    const int all_steps = (lq + QT - 1) / QT;
    const bool has_far = j0 < seen.sinks && steps.to < all_steps;
    if (far) {
        const int b = st.tile * (far_rows / QT), e = b + far_rows / QT;
        steps.from = b > steps.to ? b : steps.to;
        steps.to = e < all_steps ? e : all_steps;
        if (steps.from >= steps.to)
            return;
    }
    const bool working = wj0 <= j1 && (!far || wj0 < seen.sinks);

    // items: head of the group, then step
    const int length = steps.to - steps.from;
    int begin = 0, count = group * length;
    if (parts > 1 && !far) {
        begin = (int)((int64_t)count * part_no / parts);
        count = (int)((int64_t)count * (part_no + 1) / parts) - begin;
    }
    float carried = 0.0f;            // lse or delta of one row on its way to LDS
    const Stager<T, DP, QT, 4> q_in(a.q.row_stride, a.D), g_in(a.dout.row_stride, a.D);
    // of the next fetch
    int next_head = hk * group, next_step = steps.from;
    if (begin > 0) {
        next_head += begin / length;
        next_step += begin % length;
    }
    auto fetch = [&](char *qt, char *gt) {
        const int first = next_step * QT;
        const GradRows<T> r = grad_rows<T>(a, q_begin, k_begin, next_head, hk);
        q_in.load(qt, r.q, first, lq - 1, wave);
        g_in.load(gt, r.dout, first, lq - 1, wave);
        if (t < 2 * QT) {
            const int i = first + (t & (QT - 1)) < lq ? first + (t & (QT - 1)) : lq - 1;
            carried = t < QT ? base2(r.lse[i], i + shift) : r.delta[i];
        }
        if (++next_step == steps.to) {
            next_step = steps.from;
            ++next_head;
        }
    };
    auto arrive = [&](float *stat) {
        wait_loads();
        if (t < 2 * QT)
            stat[t] = carried;
        __syncthreads();
    };
    const int next_step0 = next_step;
    if (count > 0)
        fetch(q_even, g_even);

    Frag<T> kf[STEPS], vf[STEPS];
    {
        const int row = key < lk ? key : lk - 1;
        const T *k = (const T *)a.k.base + (int64_t)(k_begin + row) * a.k.row_stride + hk * a.k.head_stride;
        const T *v = (const T *)a.v.base + (int64_t)(k_begin + row) * a.v.row_stride + hk * a.v.head_stride;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int d = 16 * s + 8 * half;
            kf[s] = d < a.D ? load8(k + d) : zero_frag<T>();
            vf[s] = d < a.D ? load8(v + d) : zero_frag<T>();
        }
    }
    f32x16 dK[DB], dV[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d) {
        dK[d] = f32x16(0.0f);
        dV[d] = f32x16(0.0f);
    }

    int this_step = next_step0;
    auto compute = [&](const char *qt, const char *gt, const float *stat) {
        const int first = this_step * QT + 32 * qw;          // the wavefront's rows
        const int last = (first + 32 < lq ? first + 32 : lq) - 1;
        if (++this_step == steps.to)
            this_step = steps.from;
        if (!working || first > last || seen.none(first + shift, last + shift, wj0, wj1))
            return;
        const int rows_at = renewed(Tl::row_base(lane) + 32 * qw * Tl::kRowBytes);
        const int cols_at = renewed(Tl::col_base(lane) + 32 * qw * Tl::kRowBytes);
        f32x16 x = f32x16(0.0f), dp = f32x16(0.0f);
        chain<2 * STEPS, kAhead>(
            [&](int i) { return Tl::row_frag(i & 1 ? gt : qt, rows_at, 0, i >> 1); },
            [&](int i, Frag<T> f) {
                if (i & 1)
                    dp = mma(f, vf[i >> 1], dp);
                else
                    x = mma(f, kf[i >> 1], x);
            });
        if (last < first + 31 || !seen.all(first + shift, last + shift, wj0, wj0 + 31))
            mask_queries(seen, key, first + shift, last + 1 - first, half, x, dp);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const f32x4 l4 = *(const f32x4 *)(stat + 32 * qw + 8 * g + 4 * half);
            const f32x4 d4 = *(const f32x4 *)(stat + QT + 32 * qw + 8 * g + 4 * half);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[4 * g + e] = __builtin_amdgcn_exp2f(fmaf(x[4 * g + e], c2, -l4[e]));
                dp[4 * g + e] = x[4 * g + e] * (dp[4 * g + e] - d4[e]);
            }
        }
        const Frag<T> pf[2] = {result_frag<T>(x, 0), result_frag<T>(x, 1)};
        const Frag<T> df[2] = {result_frag<T>(dp, 0), result_frag<T>(dp, 1)};
        chain<4 * DB, kAhead>(
            [&](int i) { return Tl::col_frag(i & 1 ? qt : gt, cols_at, i / (2 * DB), (i >> 1) % DB); },
            [&](int i, Frag<T> f) {
                const int d = (i >> 1) % DB;
                if (i & 1)
                    dK[d] = mma(f, df[i / (2 * DB)], dK[d]);
                else
                    dV[d] = mma(f, pf[i / (2 * DB)], dV[d]);
            });
    };
    arrive(stat_even);
    for (int n = 0; n < count; n += 2) {
        if (n + 1 < count)
            fetch(q_odd, g_odd);
        compute(q_even, g_even, stat_even);
        arrive(stat_odd);
        if (n + 1 >= count)
            break;
        if (n + 2 < count)
            fetch(q_even, g_even);
        compute(q_odd, g_odd, stat_odd);
        arrive(stat_even);
    }

    static_assert(Parked<DP, DU>::kBytes <= Tl::kBytes, "a buffer for each sum");
    if (qw == 1) {
        Parked<DP, DU>::put(kw == 0 ? q_even : q_odd, lane, dK);
        Parked<DP, DU>::put(kw == 0 ? g_even : g_odd, lane, dV);
    }
    __syncthreads();
    if (qw == 1)
        return;
    Parked<DP, DU>::add(kw == 0 ? q_even : q_odd, lane, 1.0f, 1.0f, dK);
    Parked<DP, DU>::add(kw == 0 ? g_even : g_odd, lane, 1.0f, 1.0f, dV);
    if (!working)
        return;
    if (parts > 1 && !far) {
        float *to = sums_at<DU>(sums, hk * key_slots + rest - far_items, parts, part_no, kw) + 4 * lane;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                store4(to + 256 * (4 * d + g), dK[d][4 * g], dK[d][4 * g + 1], dK[d][4 * g + 2], dK[d][4 * g + 3]);
                store4(to + 256 * (4 * (DB + d) + g), dV[d][4 * g], dV[d][4 * g + 1], dV[d][4 * g + 2],
                       dV[d][4 * g + 3]);
            }
        return;
    }
    bool clean = true;
    const bool part = has_far && key < seen.sinks;    // summed by the last launch
    if (part && key <= j1) {
        float *to = partial_at(a, far ? rest / far_tiles : far_slots + st.seq, hk, key, DP);
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int at = 32 * d + 8 * g + 4 * half;
                store4(to + at, dK[d][4 * g], dK[d][4 * g + 1], dK[d][4 * g + 2], dK[d][4 * g + 3]);
                store4(to + DP + at, dV[d][4 * g], dV[d][4 * g + 1], dV[d][4 * g + 2], dV[d][4 * g + 3]);
            }
    } else if (!far && key <= j1) {
        T *k = (T *)a.dk.base + (int64_t)(k_begin + key) * a.dk.row_stride + hk * a.dk.head_stride;
        T *v = (T *)a.dv.base + (int64_t)(k_begin + key) * a.dv.row_stride + hk * a.dv.head_stride;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (32 * d + 8 * g < a.D) {
                    float y[4], z[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[e] = dK[d][4 * g + e] * a.scale;
                        z[e] = dV[d][4 * g + e];
                        clean = clean && finite(y[e]) && finite(z[e]);
                    }
                    const int at = 32 * d + 8 * g + 4 * half;
                    store4(k + at, y[0], y[1], y[2], y[3]);
                    store4(v + at, z[0], z[1], z[2], z[3]);
                }
    }
    again_dkv<T, DU>(a, seen, __ballot(!clean), steps, false, wj0, wj1, q_begin, k_begin, lq, lk, hk, lane);
}

constexpr int kPartThreads = 512;

// Adds the parts of half a key tile in order, and for first keys their far
// runs.
template <class T, int DP, int DU>
__global__ __launch_bounds__(kPartThreads) void window_dkv_parts(WindowArgs a, int key_slots, int far_rows,
                                                                 int parts, float *sums)
{
    constexpr int DB = DU / 32;
    __shared__ int odd[32];
    const int unit = blockIdx.x, hk = unit / key_slots, kw = blockIdx.y;
    const SeqTile st = find_seq_tile(a.k_rowptr, a.S, kKeyRows, unit % key_slots);
    if (st.seq < 0)
        return;
    const int q_begin = a.q_rowptr[st.seq], lq = a.q_rowptr[st.seq + 1] - q_begin;
    const int k_begin = a.k_rowptr[st.seq], lk = a.k_rowptr[st.seq + 1] - k_begin;
    const int j0 = st.tile * kKeyRows, wj0 = j0 + 32 * kw;
    if (wj0 >= lk)
        return;
    const int j1 = (j0 + kKeyRows < lk ? j0 + kKeyRows : lk) - 1;
    const int wj1 = wj0 + 31 < j1 ? wj0 + 31 : j1;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, key = wj0 + (lane & 31);
    const StepRange steps = window_steps(j0, j1, a.window, lk - lq, lq);
    const bool has_far = j0 < a.sinks && steps.to < (lq + kStepRows - 1) / kStepRows;
    const bool first = has_far && key < a.sinks;
    const int base = q_begin / far_rows + st.seq;      // the sequence's first far run
    const int run0 = steps.to / (far_rows / kStepRows), run1 = (lq + far_rows - 1) / far_rows;
    if (t < 32)
        odd[t] = 0;
    __syncthreads();
    bool clean = true;
    for (int n = wave; n < 8 * DB; n += kPartThreads / 64) {      // dk's registers, then dv's
        const bool of_v = n >= 4 * DB;
        const int at = 8 * (of_v ? n - 4 * DB : n) + 4 * (lane >> 5);
        f32x4 x = f32x4(0.0f);
#pragma unroll 4
        for (int p = 0; p < parts; ++p)
            x += *(const f32x4 *)(sums_at<DU>(sums, unit, parts, p, kw) + 256 * n + 4 * lane);
        if (first)
#pragma unroll 4
            for (int r = run0; r < run1; ++r)
                x += *(const f32x4 *)(partial_at(a, base + r, hk, key, DP) + (of_v ? DP : 0) + at);
        if (key > j1 || at >= a.D)
            continue;
        if (!of_v)
            x *= a.scale;
        const OutRows &out = of_v ? a.dv : a.dk;
        store4((T *)out.base + (int64_t)(k_begin + key) * out.row_stride + hk * out.head_stride + at, x[0], x[1],
               x[2], x[3]);
        clean = clean && finite(x[0]) && finite(x[1]) && finite(x[2]) && finite(x[3]);
    }
    if (!clean)
        atomicOr(&odd[lane & 31], 1);
    __syncthreads();
    if (wave == 0)
        again_dkv<T, DU>(a, Seen{a.window, a.sinks}, __ballot(odd[lane & 31] != 0), steps, has_far, wj0, wj1, q_begin,
                         k_begin, lq, lk, hk, lane);
}

constexpr int kJoinThreads = 64;

// One wavefront for each first key of each sequence and key head.
template <class T, int DP, int DU>
__global__ __launch_bounds__(kJoinThreads) void window_dkv_join(WindowArgs a, int far_slots, int far_rows)
{
    const int lane = threadIdx.x;
    const int j = blockIdx.x % a.sinks, hk = blockIdx.x / a.sinks % a.Hkv;
    const int seq = blockIdx.x / a.sinks / a.Hkv;
    const int q_begin = a.q_rowptr[seq], lq = a.q_rowptr[seq + 1] - q_begin;
    const int k_begin = a.k_rowptr[seq], lk = a.k_rowptr[seq + 1] - k_begin;
    if (j >= lk)
        return;
    const int j0 = j / kKeyRows * kKeyRows;               // its key tile
    const int j1 = (j0 + kKeyRows < lk ? j0 + kKeyRows : lk) - 1;
    const StepRange steps = window_steps(j0, j1, a.window, lk - lq, lq);
    if (steps.to >= (lq + kStepRows - 1) / kStepRows)
        return;                                        // no far part: written already
    const int base = q_begin / far_rows + seq;         // the sequence's first far run
    const int from = steps.to / (far_rows / kStepRows), to = (lq + far_rows - 1) / far_rows;
    float sum[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
    auto add = [&](int run) {
        const float *p = partial_at(a, run, hk, j, DP);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            sum[x][0] += p[x * DP + lane];
            if (DP > 64)
                sum[x][1] += p[x * DP + 64 + lane];
        }
    };
    add(far_slots + seq);
#pragma unroll 4
    for (int r = from; r < to; ++r)
        add(base + r);
    bool clean = true;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        sum[0][e] *= a.scale;
        if (lane + 64 * e < a.D)
            clean = clean && finite(sum[0][e]) && finite(sum[1][e]);
    }
    // queries before the key are all that it does not see, and what repeats the
    // last one behind the sequence
    const int before = j1 - (lk - lq) < lq ? j1 - (lk - lq) : lq;
    if (!__all(clean) && (a.D != DU || odd_queries<T>(a, q_begin, k_begin, hk, 0, before, lane) ||
                          odd_queries<T>(a, q_begin, k_begin, hk, lq - 1, lq, lane))) {
        exact_dkv_row<T>(a, q_begin, k_begin, lq, lk, hk, j, lane);
        return;
    }
    put_row((T *)a.dk.base + (int64_t)(k_begin + j) * a.dk.row_stride + hk * a.dk.head_stride,
            sum[0][0], sum[0][1], a.D, lane);
    put_row((T *)a.dv.base + (int64_t)(k_begin + j) * a.dv.row_stride + hk * a.dv.head_stride,
            sum[1][0], sum[1][1], a.D, lane);
}

// Whether there are fewer key tiles than twice the CUs.
bool few_key_tiles(int64_t S, int64_t Tk, int64_t Hkv) { return (Tk / kKeyRows + S) * Hkv < 512; }

// Parts that a key tile's queries are taken in: where there are few tiles, as
// many as make about two workgroups to a CU, of at least 8 steps each (6 of
// fp32's longer ones), which pay for the launch that adds them.  (2900 tokens,
// 16 heads of 128 on 2, all keys seen, bf16: the backward pass 306 us in parts,
// 730 whole; 2025 tokens, 8 heads of 80 on 4, window 300, fp32: dk and dv 78
// us with the adding, 99 whole.  In bf16, parts of 6 steps cost 8000 pairs
// of a window of 64 60 us against 45 whole.)
int64_t dkv_parts(bool f32, int64_t S, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t window)
{
    const int64_t units = (Tk / kKeyRows + S) * Hkv;
    if (units == 0 || !few_key_tiles(S, Tk, Hkv))
        return 1;
    const int64_t reach = window + kKeyRows < Tq ? window + kKeyRows : Tq;
    const int64_t most = Hq / Hkv * (reach / kStepRows + 1) / (f32 ? 6 : 8);
    const int64_t parts = (512 + units / 2) / units;
    return most < 1 ? 1 : (parts < most ? parts : most);
}

// Queries of a far run: shorter ones where there are few workgroups otherwise.
// (Dk and dv of the fp32 example: 68 us with 256, 80 with 128, 122 with 512.  990
// tokens, 4 heads of 64 on 1, window 100, bf16: the backward pass 40 us with 256,
// 30 with 128, 43 with 512.)
int64_t far_run_rows(bool f32, int64_t S, int64_t Tk, int64_t Hkv)
{
    return few_key_tiles(S, Tk, Hkv) ? (f32 ? 256 : 128) : 512;
}

// Far runs of a call: none without first keys, or where no position can lie
// past the window of the first key.
int64_t far_runs(bool f32, int64_t S, int64_t Tq, int64_t Tk, int64_t Hkv, int64_t window, int64_t sinks)
{
    return sinks > 0 && window < Tk ? Tq / far_run_rows(f32, S, Tk, Hkv) + S : 0;
}

// Floats of the first keys' partial sums, and of the parts' sums.
int64_t far_floats(int64_t S, int64_t Hkv, int64_t D, int64_t sinks, int64_t runs)
{
    return runs == 0 ? 0 : (runs + S) * Hkv * sinks * 2 * (D <= 64 ? 64 : 128);
}

int64_t parts_floats(int64_t S, int64_t Tk, int64_t Hkv, int64_t D, int64_t parts)
{
    const int64_t DU = D <= 64 ? 64 : (D <= 96 ? 96 : 128);
    return parts == 1 ? 0 : (Tk / kKeyRows + S) * Hkv * parts * kKeyRows * 2 * DU;
}

// The launches of dk and dv.
struct DkvShape {
    int64_t key_slots, far, far_tiles, parts;
    int far_rows;
};

DkvShape dkv_shape(bool f32, const WindowArgs &a)
{
    DkvShape s;
    s.key_slots = a.Tk / kKeyRows + a.S;
    s.far = far_runs(f32, a.S, a.Tq, a.Tk, a.Hkv, a.window, a.sinks);
    s.far_rows = (int)far_run_rows(f32, a.S, a.Tk, a.Hkv);
    s.far_tiles = s.far > 0 ? (a.sinks + kKeyRows - 1) / kKeyRows : 0;
    s.parts = dkv_parts(f32, a.S, a.Tq, a.Tk, a.Hq, a.Hkv, a.window);
    return s;
}

template <class T, int DP, int DU, int RG>
hipError_t launch_dq(const WindowArgs &a, hipStream_t stream)
{
    const int64_t slots = a.Tq / (32 * RG) + a.S;
    window_dq<T, DP, DU, RG><<<dim3((uint32_t)(slots * a.Hq)), kAttnThreads, 0, stream>>>(a, (int)slots);
    return hipGetLastError();
}

template <class T, int DP, int DU>
hipError_t launch(const WindowArgs &a, hipStream_t stream)
{
    constexpr bool f32 = sizeof(T) == 4;
    const DkvShape s = dkv_shape(f32, a);
    hipError_t err;
    if (a.Tq > 0) {
        err = few_tiles(a) ? launch_dq<T, DP, DU, 2>(a, stream) : launch_dq<T, DP, DU, 4>(a, stream);
        if (err != hipSuccess)
            return err;
    }
    if (a.Tk > 0) {
        float *sums = a.partial + far_floats(a.S, a.Hkv, a.D, a.sinks, s.far);
        window_dkv<T, DP, DU><<<dim3((uint32_t)((s.key_slots + s.far * s.far_tiles) * a.Hkv), (uint32_t)s.parts),
                                kAttnThreads, 0, stream>>>(a, (int)s.key_slots, (int)s.far, (int)s.far_tiles,
                                                           s.far_rows, sums);
        if ((err = hipGetLastError()) != hipSuccess)
            return err;
        if (s.parts > 1) {
            window_dkv_parts<T, DP, DU><<<dim3((uint32_t)(s.key_slots * a.Hkv), 2), kPartThreads, 0, stream>>>(
                a, (int)s.key_slots, s.far_rows, (int)s.parts, sums);
            return hipGetLastError();
        }
        if (s.far > 0) {
            window_dkv_join<T, DP, DU><<<dim3((uint32_t)(a.S * a.Hkv * a.sinks)), kJoinThreads, 0, stream>>>(
                a, (int)s.far, s.far_rows);
            if ((err = hipGetLastError()) != hipSuccess)
                return err;
        }
    }
    return hipSuccess;
}

}  // namespace

int64_t window_bwd_delta_bytes(int64_t Tq, int64_t Hq) { return (Tq * Hq * 4 + 255) / 256 * 256; }

int64_t window_bwd_partial_bytes(int64_t S, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D,
                                 int64_t window, int64_t sinks)
{
    // enough for both types: bf16 has more runs, fp32 more parts
    return 4 * (far_floats(S, Hkv, D, sinks, far_runs(false, S, Tq, Tk, Hkv, window, sinks)) +
                parts_floats(S, Tk, Hkv, D, dkv_parts(true, S, Tq, Tk, Hq, Hkv, window)));
}

int64_t window_bwd_threads(int dtype, const WindowArgs &a)
{
    const DkvShape s = dkv_shape(dtype == SPMM_DTYPE_F32, a);
    auto most = [](int64_t x, int64_t y) { return x > y ? x : y; };
    int64_t n = 0;
    if (a.Tq > 0)
        n = (a.Tq / (few_tiles(a) ? 64 : 128) + a.S) * a.Hq * kAttnThreads;
    if (a.Tk > 0) {
        n = most(n, (s.key_slots + s.far * s.far_tiles) * a.Hkv * kAttnThreads);
        n = most(n, s.parts > 1 ? s.key_slots * a.Hkv * kPartThreads : 0);
        n = most(n, s.parts == 1 && s.far > 0 ? (int64_t)a.S * a.Hkv * a.sinks * kJoinThreads : 0);
    }
    return n;
}

hipError_t launch_window_bwd(int dtype, const WindowArgs &a, hipStream_t stream)
{
    if (dtype == SPMM_DTYPE_BF16)
        return a.D <= 64 ? launch<__bf16, 64, 64>(a, stream)
                         : (a.D <= 96 ? launch<__bf16, 128, 96>(a, stream) : launch<__bf16, 128, 128>(a, stream));
    return a.D <= 64 ? launch<float, 64, 64>(a, stream)
                     : (a.D <= 96 ? launch<float, 128, 96>(a, stream) : launch<float, 128, 128>(a, stream));
}

}  // namespace sdl

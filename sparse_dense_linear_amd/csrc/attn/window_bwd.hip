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
// lies past its window is cut into runs of kFarRows queries with a workgroup
// each; those and the window's part leave fp32 partial sums, which a last
// small launch adds in a fixed order.
#include "ops.h"
#include "exact.h"
#include "tile.h"
#include "spmm.h"

namespace sdl {

namespace {

constexpr int kKeyRows = 128;     // keys of a dk/dv workgroup
constexpr int kStepRows = 32;     // queries of one step of it
constexpr int kFarRows = 512;     // queries of a far run

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

// ------------------------------------------------------------------- dq

template <class T, int DP>
__global__ __launch_bounds__(kAttnThreads, sizeof(T) == 2 ? 2 : 1) void window_dq(WindowArgs a, int slots)
{
    constexpr int KT = sizeof(T) == 2 ? 64 : (DP == 64 ? 64 : 32);
    constexpr int SB = KT / 32, STEPS = DP / 16, DB = DP / 32;
    typedef Tile<T, DP, KT> Tl;
    __shared__ __align__(16) char lds[2][2][Tl::kBytes];

    const int group = a.Hq / a.Hkv;
    const int idx = xcd_order(blockIdx.x, gridDim.x);
    const int hk = idx / (slots * group), rest = idx % (slots * group);
    const int head = hk * group + rest % group;
    const SeqTile st = find_seq_tile(a.q_rowptr, a.S, kFwdRows, slots - 1 - rest / group);
    if (st.seq < 0)
        return;
    const int q_begin = a.q_rowptr[st.seq], lq = a.q_rowptr[st.seq + 1] - q_begin;
    const int k_begin = a.k_rowptr[st.seq], lk = a.k_rowptr[st.seq + 1] - k_begin;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, half = lane >> 5;
    const Seen seen = {a.window, a.sinks};
    const int shift = lk - lq;
    const int i0 = st.tile * kFwdRows, i1 = (i0 + kFwdRows < lq ? i0 + kFwdRows : lq) - 1;
    const int wi0 = i0 + 32 * wave;
    const int qi = wi0 + (lane & 31);
    const int pos = qi + shift;
    const int wp0 = wi0 + shift, wp1 = (wi0 + 31 < i1 ? wi0 + 31 : i1) + shift;
    const float c2 = a.scale * kLog2e;
    const GradRows<T> r = grad_rows<T>(a, q_begin, k_begin, head, hk);
    const int row = qi < lq ? qi : lq - 1;

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
        if (qi <= i1 && half == 0)
            a.delta[(int64_t)head * a.Tq + q_begin + qi] = delta;
    }
    const float lse2 = r.lse[row] * kLog2e;

    f32x16 dQ[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
        dQ[d] = f32x16(0.0f);

    const int p0 = i0 + shift, p1 = i1 + shift;
    const int low = p0 - seen.window + 1 > 0 ? p0 - seen.window + 1 : 0;
    const int band = low / KT;
    int first_tiles = (seen.sinks + KT - 1) / KT;
    first_tiles = first_tiles < band ? first_tiles : band;
    const int count = p1 < 0 ? 0 : first_tiles + p1 / KT + 1 - band;

    Carrier<T, DP, KT, kAttnThreads> ck, cv;
    if (count > 0) {
        const int j0 = (first_tiles > 0 ? 0 : band) * KT;
        ck.load(r.k, r.k_stride, j0, lk - 1, a.D, t);
        cv.load(r.v, r.v_stride, j0, lk - 1, a.D, t);
        ck.store(lds[0][0], t);
        cv.store(lds[0][1], t);
    }
    __syncthreads();
    for (int n = 0; n < count; ++n) {
        const int j0 = (n < first_tiles ? n : band + n - first_tiles) * KT;
        if (n + 1 < count) {
            const int next = (n + 1 < first_tiles ? n + 1 : band + n + 1 - first_tiles) * KT;
            ck.load(r.k, r.k_stride, next, lk - 1, a.D, t);
            cv.load(r.v, r.v_stride, next, lk - 1, a.D, t);
        }
        if (wi0 <= i1 && !seen.none(wp0, wp1, j0, j0 + KT - 1)) {
            const char *kt = lds[n & 1][0], *vt = lds[n & 1][1];
            const bool whole = seen.all(wp0, wp1, j0, j0 + KT - 1);
#pragma unroll
            for (int b = 0; b < SB; ++b) {
                f32x16 x = f32x16(0.0f), dp = f32x16(0.0f);
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    x = mma(Tl::row_frag(kt, 32 * b + (lane & 31), s, half), qf[s], x);
                    dp = mma(Tl::row_frag(vt, 32 * b + (lane & 31), s, half), gf[s], dp);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float p = __builtin_amdgcn_exp2f(fmaf(x[i], c2, -lse2));
                    float ds = p * (dp[i] - delta);
                    if (!whole && !seen(pos, j0 + 32 * b + 8 * (i >> 2) + 4 * half + (i & 3)))
                        ds = 0.0f;
                    x[i] = ds;
                }
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const Frag<T> df = result_frag<T>(x, s);
#pragma unroll
                    for (int d = 0; d < DB; ++d)
                        dQ[d] = mma(Tl::col_frag(kt, 32 * b + 16 * s, d, lane), df, dQ[d]);
                }
            }
        }
        if (n + 1 < count) {
            ck.store(lds[(n + 1) & 1][0], t);
            cv.store(lds[(n + 1) & 1][1], t);
        }
        __syncthreads();
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
    for (uint32_t left = (uint32_t)(redo | (redo >> 32)); left != 0; left &= left - 1) {
        const int i = wi0 + __ffs(left) - 1, p = i + shift;
        const int lo = p - seen.window + 1 > 0 ? p - seen.window + 1 : 0;
        // delta of the row, stored above by this wavefront, is not read back:
        // the lane that holds it hands it out
        exact_dq_row<T>(
            r, i, __shfl(delta, i - wi0), [&](int j) { return seen(p, j); },
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

template <class T, int DP>
__global__ __launch_bounds__(kAttnThreads, 1) void window_dkv(WindowArgs a, int key_slots, int far_slots)
{
    constexpr int QT = kStepRows, STEPS = DP / 16, DB = DP / 32;
    typedef Tile<T, DP, QT> Tl;
    __shared__ __align__(16) char lds[2][2][Tl::kBytes];
    __shared__ float row_lse[2][QT], row_delta[2][QT];

    const int group = a.Hq / a.Hkv;
    const int per_head = key_slots + far_slots;
    const int idx = xcd_order(blockIdx.x, gridDim.x);
    const int hk = idx / per_head, rest = idx % per_head;
    const bool far = rest < far_slots;
    const SeqTile st = far ? find_seq_tile(a.q_rowptr, a.S, kFarRows, rest)
                           : find_seq_tile(a.k_rowptr, a.S, kKeyRows, rest - far_slots);
    if (st.seq < 0)
        return;
    const int q_begin = a.q_rowptr[st.seq], lq = a.q_rowptr[st.seq + 1] - q_begin;
    const int k_begin = a.k_rowptr[st.seq], lk = a.k_rowptr[st.seq + 1] - k_begin;
    if (lk <= 0)
        return;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, half = lane >> 5;
    const Seen seen = {a.window, a.sinks};
    const int shift = lk - lq;
    const int j0 = far ? 0 : st.tile * kKeyRows;
    const int j1 = (j0 + kKeyRows < lk ? j0 + kKeyRows : lk) - 1;
    const int wj0 = j0 + 32 * wave, wj1 = wj0 + 31 < j1 ? wj0 + 31 : j1;
    const int key = wj0 + (lane & 31);
    const float c2 = a.scale * kLog2e;

    StepRange steps = window_steps(j0, j1, seen.window, shift, lq);
    const int all_steps = (lq + QT - 1) / QT;
    const bool has_far = j0 == 0 && seen.sinks > 0 && steps.to < all_steps;
    if (far) {
        const int b = st.tile * (kFarRows / QT), e = b + kFarRows / QT;
        steps.from = b > steps.to ? b : steps.to;
        steps.to = e < all_steps ? e : all_steps;
        if (steps.from >= steps.to)
            return;
    }
    const bool working = wj0 <= j1 && (!far || wj0 < seen.sinks);

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

    // items: head of the group, then step
    const int n_steps = steps.to - steps.from;
    const int count = group * n_steps;
    Carrier<T, DP, QT, kAttnThreads> cq, cg;
    float stat = 0.0f;
    auto fetch = [&](int n) {
        const int head = hk * group + n / n_steps, first = (steps.from + n % n_steps) * QT;
        const GradRows<T> r = grad_rows<T>(a, q_begin, k_begin, head, hk);
        cq.load(r.q, r.q_stride, first, lq - 1, a.D, t);
        cg.load(r.dout, r.dout_stride, first, lq - 1, a.D, t);
        if (t < 2 * QT) {
            const int i = first + (t & (QT - 1)) < lq ? first + (t & (QT - 1)) : lq - 1;
            stat = t < QT ? r.lse[i] * kLog2e : r.delta[i];
        }
    };
    auto stash = [&](int buf) {
        cq.store(lds[buf][0], t);
        cg.store(lds[buf][1], t);
        if (t < QT)
            row_lse[buf][t] = stat;
        else if (t < 2 * QT)
            row_delta[buf][t - QT] = stat;
    };
    if (count > 0) {
        fetch(0);
        stash(0);
    }
    __syncthreads();
    for (int n = 0; n < count; ++n) {
        if (n + 1 < count)
            fetch(n + 1);
        const int first = (steps.from + n % n_steps) * QT;
        const int last = (first + QT < lq ? first + QT : lq) - 1;
        if (working && !seen.none(first + shift, last + shift, wj0, wj1)) {
            const char *qt = lds[n & 1][0], *gt = lds[n & 1][1];
            f32x16 x = f32x16(0.0f), dp = f32x16(0.0f);
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                x = mma(Tl::row_frag(qt, lane & 31, s, half), kf[s], x);
                dp = mma(Tl::row_frag(gt, lane & 31, s, half), vf[s], dp);
            }
            const bool whole =
                last == first + QT - 1 && seen.all(first + shift, last + shift, wj0, wj0 + 31);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 l4 = *(const f32x4 *)(row_lse[n & 1] + 8 * g + 4 * half);
                const f32x4 d4 = *(const f32x4 *)(row_delta[n & 1] + 8 * g + 4 * half);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = first + 8 * g + 4 * half + e;
                    float p = __builtin_amdgcn_exp2f(fmaf(x[4 * g + e], c2, -l4[e]));
                    float ds = p * (dp[4 * g + e] - d4[e]);
                    if (!whole && !(i <= last && seen(i + shift, key)))
                        p = ds = 0.0f;
                    x[4 * g + e] = p;
                    dp[4 * g + e] = ds;
                }
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Frag<T> pf = result_frag<T>(x, s), df = result_frag<T>(dp, s);
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    dV[d] = mma(Tl::col_frag(gt, 16 * s, d, lane), pf, dV[d]);
                    dK[d] = mma(Tl::col_frag(qt, 16 * s, d, lane), df, dK[d]);
                }
            }
        }
        if (n + 1 < count)
            stash((n + 1) & 1);
        __syncthreads();
    }

    if (!working)
        return;
    bool clean = true;
    const bool part = has_far && key < seen.sinks;    // summed by the last launch
    if (part && key <= j1) {
        float *to = partial_at(a, far ? rest : far_slots + st.seq, hk, key, DP);
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
    const uint64_t redo = __ballot(!clean);
    for (uint32_t left = (uint32_t)(redo | (redo >> 32)); left != 0; left &= left - 1)
        exact_dkv_row<T>(a, q_begin, k_begin, lq, lk, hk, wj0 + __ffs(left) - 1, lane);
}

// One wavefront for each first key of each sequence and key head.
template <class T, int DP>
__global__ __launch_bounds__(64) void window_dkv_join(WindowArgs a, int far_slots)
{
    const int lane = threadIdx.x;
    const int j = blockIdx.x % a.sinks, hk = blockIdx.x / a.sinks % a.Hkv;
    const int seq = blockIdx.x / a.sinks / a.Hkv;
    const int q_begin = a.q_rowptr[seq], lq = a.q_rowptr[seq + 1] - q_begin;
    const int k_begin = a.k_rowptr[seq], lk = a.k_rowptr[seq + 1] - k_begin;
    if (j >= lk)
        return;
    const int j1 = (kKeyRows < lk ? kKeyRows : lk) - 1;
    const StepRange steps = window_steps(0, j1, a.window, lk - lq, lq);
    if (steps.to >= (lq + kStepRows - 1) / kStepRows)
        return;                                        // no far part: written already
    const int base = q_begin / kFarRows + seq;         // the sequence's first far run
    const int from = steps.to / (kFarRows / kStepRows), to = (lq + kFarRows - 1) / kFarRows;
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
    for (int r = from; r < to; ++r)
        add(base + r);
    bool clean = true;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        sum[0][e] *= a.scale;
        if (lane + 64 * e < a.D)
            clean = clean && finite(sum[0][e]) && finite(sum[1][e]);
    }
    if (!__all(clean)) {
        exact_dkv_row<T>(a, q_begin, k_begin, lq, lk, hk, j, lane);
        return;
    }
    put_row((T *)a.dk.base + (int64_t)(k_begin + j) * a.dk.row_stride + hk * a.dk.head_stride,
            sum[0][0], sum[0][1], a.D, lane);
    put_row((T *)a.dv.base + (int64_t)(k_begin + j) * a.dv.row_stride + hk * a.dv.head_stride,
            sum[1][0], sum[1][1], a.D, lane);
}

// Far runs of a call: none without first keys, or where no position can lie
// past the window of the first key.
int64_t far_runs(int64_t S, int64_t Tq, int64_t Tk, int64_t window, int64_t sinks)
{
    return sinks > 0 && window < Tk ? Tq / kFarRows + S : 0;
}

template <class T, int DP>
hipError_t launch(const WindowArgs &a, hipStream_t stream)
{
    const int64_t slots = a.Tq / kFwdRows + a.S;
    const int64_t key_slots = a.Tk / kKeyRows + a.S;
    const int64_t far = far_runs(a.S, a.Tq, a.Tk, a.window, a.sinks);
    hipError_t err;
    if (a.Tq > 0) {
        window_dq<T, DP><<<dim3((uint32_t)(slots * a.Hq)), kAttnThreads, 0, stream>>>(a, (int)slots);
        if ((err = hipGetLastError()) != hipSuccess)
            return err;
    }
    if (a.Tk > 0) {
        window_dkv<T, DP><<<dim3((uint32_t)((key_slots + far) * a.Hkv)), kAttnThreads, 0, stream>>>(
            a, (int)key_slots, (int)far);
        if ((err = hipGetLastError()) != hipSuccess)
            return err;
        if (far > 0) {
            window_dkv_join<T, DP><<<dim3((uint32_t)(a.S * a.Hkv * a.sinks)), 64, 0, stream>>>(a, (int)far);
            if ((err = hipGetLastError()) != hipSuccess)
                return err;
        }
    }
    return hipSuccess;
}

}  // namespace

int64_t window_bwd_delta_bytes(int64_t Tq, int64_t Hq) { return (Tq * Hq * 4 + 255) / 256 * 256; }

int64_t window_bwd_partial_bytes(int64_t S, int64_t Tq, int64_t Tk, int64_t Hkv, int64_t D,
                                 int64_t window, int64_t sinks)
{
    const int64_t runs = far_runs(S, Tq, Tk, window, sinks);
    return runs == 0 ? 0 : (runs + S) * Hkv * sinks * 2 * (D <= 64 ? 64 : 128) * 4;
}

hipError_t launch_window_bwd(int dtype, const WindowArgs &a, hipStream_t stream)
{
    if (dtype == SPMM_DTYPE_BF16)
        return a.D <= 64 ? launch<__bf16, 64>(a, stream) : launch<__bf16, 128>(a, stream);
    return a.D <= 64 ? launch<float, 64>(a, stream) : launch<float, 128>(a, stream);
}

}  // namespace sdl

// window_fwd.hip -- window attention, forward.
//
//   s_ij = scale <q_i, k_j>,  o_i = sum_j softmax_j(s_ij) v_j over the keys
//   that i sees (Seen), lse_i = log sum_j exp(s_ij)
//
// One workgroup takes 128 queries of one head, 32 per wavefront, and walks
// the key tiles that any of them sees: the tiles of the first `sinks` keys,
// then those of the window.  Softmax in one pass: running maximum and sum in
// fp32, base 2 (scale * log2 e is one factor).
//
// Scores are formed transposed, S^T = K q^T, so that a lane holds one query:
// its maximum, its sum and the rescaling of its output are the lane's own
// (the two lanes of a query exchange one value), and the weights are, as
// they lie, the second operand of O^T = V^T P^T.
#include "ops.h"
#include "exact.h"
#include "tile.h"
#include "spmm.h"

namespace sdl {

namespace {

template <class T, int DP>
struct FwdShape {
    // keys of a tile: two buffers of K and V within half of the CU's LDS
    static constexpr int kKeys = sizeof(T) == 2 ? 64 : (DP == 64 ? 64 : 32);
};

template <class T, int DP>
__global__ __launch_bounds__(kAttnThreads, sizeof(T) == 2 ? 2 : 1) void window_fwd(WindowArgs a, int slots)
{
    constexpr int KT = FwdShape<T, DP>::kKeys;
    constexpr int SB = KT / 32, STEPS = DP / 16, DB = DP / 32;
    typedef Tile<T, DP, KT> Tl;
    __shared__ __align__(16) char lds[2][2][Tl::kBytes];

    const int group = a.Hq / a.Hkv;
    const int idx = xcd_order(blockIdx.x, gridDim.x);
    const int hk = idx / (slots * group), rest = idx % (slots * group);
    const int head = hk * group + rest % group;
    // late tiles (the long ones without a window) first
    const SeqTile st = find_seq_tile(a.q_rowptr, a.S, kFwdRows, slots - 1 - rest / group);
    if (st.seq < 0)
        return;
    const int q_begin = a.q_rowptr[st.seq], lq = a.q_rowptr[st.seq + 1] - q_begin;
    const int k_begin = a.k_rowptr[st.seq], lk = a.k_rowptr[st.seq + 1] - k_begin;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, half = lane >> 5;
    const Seen seen = {a.window, a.sinks};
    const int shift = lk - lq;
    const int i0 = st.tile * kFwdRows, i1 = (i0 + kFwdRows < lq ? i0 + kFwdRows : lq) - 1;
    const int wi0 = i0 + 32 * wave;                       // the wavefront's queries
    const int qi = wi0 + (lane & 31);
    const int pos = qi + shift;
    const int wp0 = wi0 + shift, wp1 = (wi0 + 31 < i1 ? wi0 + 31 : i1) + shift;
    const float c2 = a.scale * kLog2e;

    const T *K = (const T *)a.k.base + (int64_t)k_begin * a.k.row_stride + hk * a.k.head_stride;
    const T *V = (const T *)a.v.base + (int64_t)k_begin * a.v.row_stride + hk * a.v.head_stride;
    const T *Q = (const T *)a.q.base + (int64_t)(q_begin + (qi < lq ? qi : lq - 1)) * a.q.row_stride +
                 head * a.q.head_stride;

    Frag<T> qf[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
        qf[s] = 16 * s + 8 * half < a.D ? load8(Q + 16 * s + 8 * half) : zero_frag<T>();

    f32x16 O[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
        O[d] = f32x16(0.0f);
    float top = SDL_NEG_INF, total = 0.0f;

    // key tiles: [0, first_tiles) and [band, band + ...)
    const int p0 = i0 + shift, p1 = i1 + shift;
    const int low = p0 - seen.window + 1 > 0 ? p0 - seen.window + 1 : 0;
    const int band = low / KT;
    int first_tiles = (seen.sinks + KT - 1) / KT;
    first_tiles = first_tiles < band ? first_tiles : band;
    const int count = p1 < 0 ? 0 : first_tiles + p1 / KT + 1 - band;

    Carrier<T, DP, KT, kAttnThreads> ck, cv;
    if (count > 0) {
        const int j0 = (first_tiles > 0 ? 0 : band) * KT;
        ck.load(K, a.k.row_stride, j0, lk - 1, a.D, t);
        cv.load(V, a.v.row_stride, j0, lk - 1, a.D, t);
        ck.store(lds[0][0], t);
        cv.store(lds[0][1], t);
    }
    __syncthreads();
    for (int n = 0; n < count; ++n) {
        const int j0 = (n < first_tiles ? n : band + n - first_tiles) * KT;
        if (n + 1 < count) {
            const int next = (n + 1 < first_tiles ? n + 1 : band + n + 1 - first_tiles) * KT;
            ck.load(K, a.k.row_stride, next, lk - 1, a.D, t);
            cv.load(V, a.v.row_stride, next, lk - 1, a.D, t);
        }
        if (wi0 <= i1 && !seen.none(wp0, wp1, j0, j0 + KT - 1)) {
            const char *kt = lds[n & 1][0], *vt = lds[n & 1][1];
            f32x16 x[SB];
#pragma unroll
            for (int b = 0; b < SB; ++b) {
                x[b] = f32x16(0.0f);
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
                    x[b] = mma(Tl::row_frag(kt, 32 * b + (lane & 31), s, half), qf[s], x[b]);
            }
            const bool whole = seen.all(wp0, wp1, j0, j0 + KT - 1);
            float most = SDL_NEG_INF;
#pragma unroll
            for (int b = 0; b < SB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float y = x[b][r] * c2;
                    if (!whole && !seen(pos, j0 + 32 * b + 8 * (r >> 2) + 4 * half + (r & 3)))
                        y = SDL_NEG_INF;
                    x[b][r] = y;
                    most = fmaxf(most, y);
                }
            const float now = fmaxf(top, max_halves(most));
            const float base = now == SDL_NEG_INF ? 0.0f : now;
            const float keep = __builtin_amdgcn_exp2f(top - base);
            top = now;
            float sum = 0.0f;
#pragma unroll
            for (int b = 0; b < SB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    x[b][r] = __builtin_amdgcn_exp2f(x[b][r] - base);
                    sum += x[b][r];
                }
            total = total * keep + sum;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    O[d][r] *= keep;
#pragma unroll
            for (int b = 0; b < SB; ++b)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const Frag<T> pf = result_frag<T>(x[b], s);
#pragma unroll
                    for (int d = 0; d < DB; ++d)
                        O[d] = mma(Tl::col_frag(vt, 32 * b + 16 * s, d, lane), pf, O[d]);
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
    total = sum_halves(total);
    const bool some = pos >= 0;                 // window >= 1: a query sees its own position
    const float inv = 1.0f / total;
    const float lse = some ? kLn2 * (top + __builtin_amdgcn_logf(total)) : SDL_NEG_INF;
    bool clean = finite(lse);
    T *out = (T *)a.o.base + (int64_t)(q_begin + qi) * a.o.row_stride + head * a.o.head_stride;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[e] = some ? O[d][4 * g + e] * inv : 0.0f;
                if (32 * d + 8 * g < a.D)
                    clean = clean && finite(y[e]);
            }
            if (qi <= i1 && 32 * d + 8 * g < a.D)
                store4(out + 32 * d + 8 * g + 4 * half, y[0], y[1], y[2], y[3]);
        }
    if (qi <= i1 && half == 0)
        a.lse[(int64_t)head * a.Tq + q_begin + qi] = lse;

    const uint64_t redo = __ballot(!clean && some && qi <= i1);
    for (uint32_t left = (uint32_t)(redo | (redo >> 32)); left != 0; left &= left - 1) {
        const int i = wi0 + __ffs(left) - 1, p = i + shift;
        const int lo = p - seen.window + 1 > 0 ? p - seen.window + 1 : 0;
        const T *row = (const T *)a.q.base + (int64_t)(q_begin + i) * a.q.row_stride +
                       head * a.q.head_stride;
        exact_row<T>(
            row, [&](int j) { return K + (int64_t)j * a.k.row_stride; },
            [&](int j) { return V + (int64_t)j * a.v.row_stride; },
            [&](int j) { return seen(p, j); }, seen.sinks < lo ? seen.sinks : lo, lo, p + 1, a.D, c2,
            (T *)a.o.base + (int64_t)(q_begin + i) * a.o.row_stride + head * a.o.head_stride,
            a.lse + (int64_t)head * a.Tq + q_begin + i, lane);
    }
}

template <class T, int DP>
hipError_t launch(const WindowArgs &a, hipStream_t stream)
{
    const int64_t slots = a.Tq / kFwdRows + a.S;
    window_fwd<T, DP><<<dim3((uint32_t)(slots * a.Hq)), kAttnThreads, 0, stream>>>(a, (int)slots);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_window_fwd(int dtype, const WindowArgs &a, hipStream_t stream)
{
    if (dtype == SPMM_DTYPE_BF16)
        return a.D <= 64 ? launch<__bf16, 64>(a, stream) : launch<__bf16, 128>(a, stream);
    return a.D <= 64 ? launch<float, 64>(a, stream) : launch<float, 128>(a, stream);
}

}  // namespace sdl

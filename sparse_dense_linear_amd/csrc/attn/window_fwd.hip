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

// RG groups of 32 queries; the 4 / RG wavefronts of a group share the keys
// of each tile and join their results at the end.
//
// What bounds it is the issue of instructions: matrix instructions take about
// as long as the softmax between them, and overlap only between wavefronts
// of a SIMD.  In bf16, 128 queries to a workgroup, tiles of 32 keys leave
// room for a third workgroup on a CU (16384 tokens, 32 heads of 128 on 8,
// window 1024: 300 us, against 326 with tiles of 64 and two).
template <class T, int DP, int DU, int RG>
__global__ __launch_bounds__(kAttnThreads, sizeof(T) == 2 ? (RG == 4 ? 3 : 2) : 1) void window_fwd(WindowArgs a, int slots)
{
    constexpr int KT = RG == 4 && sizeof(T) == 2 ? 32 : 64;   // keys of a tile
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

    // key tiles: [0, first_tiles) and [band, band + ...)
    const int p0 = i0 + shift, p1 = i1 + shift;
    const int low = p0 - seen.window + 1 > 0 ? p0 - seen.window + 1 : 0;
    const int band = low / KT;
    int first_tiles = (seen.sinks + KT - 1) / KT;
    first_tiles = first_tiles < band ? first_tiles : band;
    const int count = p1 < 0 ? 0 : first_tiles + p1 / KT + 1 - band;

    const Stager<T, DP, KT, 4> k_in(a.k.row_stride, a.D), v_in(a.v.row_stride, a.D);
    auto first_key = [&](int n) { return (n < first_tiles ? n : band + n - first_tiles) * KT; };
    auto fetch = [&](int n, char *kt, char *vt) {
        k_in.load(kt, K, first_key(n), lk - 1, wave);
        v_in.load(vt, V, first_key(n), lk - 1, wave);
    };
    if (count > 0)
        fetch(0, k_even, v_even);

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
                mask_keys(x[b], seen, pos, j0 + 32 * b, half);
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

    uint64_t redo = __ballot(!clean && some && qi <= i1);
    if (redo == 0)
        return;
    auto key_row = [&](int j) { return K + (int64_t)j * a.k.row_stride; };
    auto val_row = [&](int j) { return V + (int64_t)j * a.v.row_stride; };
    // (a sum that is not finite says too little: an infinite score, a score
    // that is no number, or an infinite key times the zeros past D)
    if (!odd_masked_keys<T, KT>(seen, key_row, val_row, wp0, p1, first_tiles, band, lk, a.D, lane))
        redo &= __ballot(!finite(lse));
    for (uint32_t left = (uint32_t)(redo | (redo >> 32)); left != 0; left &= left - 1) {
        const int n = __ffs(left) - 1, i = wi0 + n, p = i + shift;
        const int lo = p - seen.window + 1 > 0 ? p - seen.window + 1 : 0;
        exact_row<T>(
            (const T *)a.q.base + (int64_t)(q_begin + i) * a.q.row_stride + head * a.q.head_stride, key_row,
            val_row, [&](int j) { return seen(p, j); }, seen.sinks < lo ? seen.sinks : lo, lo, p + 1, a.D, c2,
            (T *)a.o.base + (int64_t)(q_begin + i) * a.o.row_stride + head * a.o.head_stride,
            a.lse + (int64_t)head * a.Tq + q_begin + i, finite(__shfl(lse, n)), lane);
    }
}

template <class T, int DP, int DU, int RG>
hipError_t launch(const WindowArgs &a, hipStream_t stream)
{
    const int64_t slots = a.Tq / (32 * RG) + a.S;
    window_fwd<T, DP, DU, RG><<<dim3((uint32_t)(slots * a.Hq)), kAttnThreads, 0, stream>>>(a, (int)slots);
    return hipGetLastError();
}

template <class T, int DP, int DU>
hipError_t launch_rows(const WindowArgs &a, hipStream_t stream)
{
    return few_tiles(a) ? launch<T, DP, DU, 2>(a, stream) : launch<T, DP, DU, 4>(a, stream);
}

}  // namespace

hipError_t launch_window_fwd(int dtype, const WindowArgs &a, hipStream_t stream)
{
    if (dtype == SPMM_DTYPE_BF16)
        return a.D <= 64 ? launch_rows<__bf16, 64, 64>(a, stream)
                         : (a.D <= 96 ? launch_rows<__bf16, 128, 96>(a, stream) : launch_rows<__bf16, 128, 128>(a, stream));
    return a.D <= 64 ? launch_rows<float, 64, 64>(a, stream)
                     : (a.D <= 96 ? launch_rows<float, 128, 96>(a, stream) : launch_rows<float, 128, 128>(a, stream));
}

}  // namespace sdl

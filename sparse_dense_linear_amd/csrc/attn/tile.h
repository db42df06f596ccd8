// tile.h -- device pieces shared by the attention kernels: matrix
// fragments, tiles of rows in LDS, and what a query sees.
//
// Everything is built on one matrix shape, 32 x 32 with 16 terms a step.
//   A operand  lane l holds row l % 32, terms 8 * (l / 32) .. + 7
//   B operand  lane l holds column l % 32, the same terms
//   result     lane l holds column l % 32, rows 8 * (r / 4) + 4 * (l / 32)
//              + r % 4 of register r = 0 .. 15
// bf16 takes one instruction a step.  fp32 takes eight of 2 terms each:
// instruction e contracts terms e and 8 + e, so that both types have the
// same fragments, and one kernel text serves both.
//
// The product of two products (softmax weights times V) needs no exchange
// between lanes: a result register group of the first product is, lane for
// lane, a B operand of the second one whose 16 terms come in the order
// {0-3, 8-11 | 4-7, 12-15} (terms of lanes 0-31 | of lanes 32-63), and the
// A operand of the second product is read from LDS in that order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sdl {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
#define SDL_NEG_INF (-__builtin_inff())

template <class T> struct FragOf;
template <> struct FragOf<__bf16> { typedef bf16x8 type; };
template <> struct FragOf<float> { typedef f32x8 type; };
template <class T> using Frag = typename FragOf<T>::type;

__device__ inline f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ inline f32x16 mma(f32x8 a, f32x8 b, f32x16 c)
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
    return c;
}

// Registers 8 * half .. + 7 of a result as a B operand (order above).  bf16:
// weights and score gradients are rounded to nearest even here, once, as
// the matrix instructions take them; their sums stay in fp32.
template <class T>
__device__ inline Frag<T> result_frag(const f32x16 &c, int half)
{
    Frag<T> f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] = (T)c[8 * half + e];
    return f;
}

template <class T>
__device__ inline Frag<T> zero_frag()
{
    Frag<T> f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] = (T)0.0f;
    return f;
}

// x of this lane and of the lane 32 away.
__device__ inline float max_halves(float x)
{
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ inline float sum_halves(float x)
{
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Eight consecutive elements of global memory (16-byte aligned).
__device__ inline bf16x8 load8(const __bf16 *p) { return *(const bf16x8 *)p; }
__device__ inline f32x8 load8(const float *p)
{
    const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ inline void store4(__bf16 *p, float a, float b, float c, float d)
{
    bf16x4 v = {(__bf16)a, (__bf16)b, (__bf16)c, (__bf16)d};
    *(bf16x4 *)p = v;
}

__device__ inline void store4(float *p, float a, float b, float c, float d)
{
    f32x4 v = {a, b, c, d};
    *(f32x4 *)p = v;
}

// ------------------------------------------------------------ LDS tiles

// A tile of ROWS rows of DP elements.  The 16-byte pieces of a row are
// exchanged among themselves by its row number, so that lanes reading one
// piece of 16 consecutive rows, or one row across, touch different banks.
template <class T, int DP, int ROWS>
struct Tile {
    static constexpr int kRowBytes = DP * (int)sizeof(T);
    static constexpr int kPieces = kRowBytes / 16;            // per row
    static constexpr int kElems = 16 / (int)sizeof(T);        // per piece
    static constexpr int kBytes = ROWS * kRowBytes;
    static constexpr int kShift = kRowBytes <= 128 ? 1 : 0;   // rows per 256 bytes
    static constexpr int kMask = (kPieces < 16 ? kPieces : 16) - 1;

    __device__ static int at(int row, int piece)
    {
        return row * kRowBytes + ((piece ^ ((row >> kShift) & kMask)) << 4);
    }

    // A operand with the tile's rows as rows: row `row`, terms 16 * step +
    // 8 * half .. + 7 along D.
    __device__ static Frag<T> row_frag(const char *base, int row, int step, int half)
    {
        if constexpr (sizeof(T) == 2) {
            return *(const bf16x8 *)(base + at(row, 2 * step + half));
        } else {
            const f32x4 a = *(const f32x4 *)(base + at(row, 4 * step + 2 * half));
            const f32x4 b = *(const f32x4 *)(base + at(row, 4 * step + 2 * half + 1));
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }

    // A operand with D as rows (32 * block + l % 32) and 16 of the tile's
    // rows, from `first` on, as terms in the order of result_frag.  bf16: two
    // transposing reads (each group of 16 lanes hands in 4 rows of 16
    // elements and takes one column of them per lane).
    __device__ static Frag<T> col_frag(const char *base, int first, int block, int lane)
    {
        const int half = lane >> 5;
        if constexpr (sizeof(T) == 2) {
            const int i = lane & 15;
            const int row = first + 4 * half + (i >> 2);
            const int d = 32 * block + (lane & 16) + 4 * (i & 3);
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4 *)(base + at(row, d >> 3) + 2 * (d & 7)));
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4 *)(base + at(row + 8, d >> 3) + 2 * (d & 7)));
            const auto ab = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(bf16x8, ab);
        } else {
            const int d = 32 * block + (lane & 31);
            f32x8 f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int row = first + 4 * half + (e & 3) + 8 * (e >> 2);
                f[e] = *(const float *)(base + at(row, d >> 2) + 4 * (d & 3));
            }
            return f;
        }
    }
};

// Pieces of a tile's rows on their way from global memory to LDS: thread t
// of THREADS carries pieces t, t + THREADS, ...
template <class T, int DP, int ROWS, int THREADS>
struct Carrier {
    typedef Tile<T, DP, ROWS> Tl;
    static constexpr int kCount = ROWS * Tl::kPieces / THREADS;
    static_assert(ROWS * Tl::kPieces % THREADS == 0, "whole pieces per thread");
    u32x4 piece[kCount];

    // Row r of the tile is row min(first + r, last) of `base` (element
    // stride `stride`); pieces past D repeat the row's last one, whose
    // products meet zeros of the other operand.
    __device__ void load(const T *base, int64_t stride, int first, int last, int D, int t)
    {
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const int n = t + i * THREADS;
            const int r = n / Tl::kPieces, p = n % Tl::kPieces;
            const int row = first + r < last ? first + r : last;
            const int d = p * Tl::kElems < D ? p * Tl::kElems : D - Tl::kElems;
            piece[i] = *(const u32x4 *)(base + (int64_t)row * stride + d);
        }
    }

    __device__ void store(char *tile, int t) const
    {
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const int n = t + i * THREADS;
            *(u32x4 *)(tile + Tl::at(n / Tl::kPieces, n % Tl::kPieces)) = piece[i];
        }
    }
};

// --------------------------------------------------------------- window

// What a query at position p sees: keys j <= p with p - j < window or
// j < sinks (positions count from the sequence's first key).
struct Seen {
    int window, sinks;
    __device__ bool operator()(int p, int j) const
    {
        return j <= p && (p - j < window || j < sinks);
    }
    // every key of j0 .. j1 seen from every position of p0 .. p1
    __device__ bool all(int p0, int p1, int j0, int j1) const
    {
        return j1 <= p0 && (p1 - j0 < window || j1 < sinks);
    }
    // no key of j0 .. j1 seen from any position of p0 .. p1
    __device__ bool none(int p0, int p1, int j0, int j1) const
    {
        return j0 > p1 || (p0 - j1 >= window && j0 >= sinks);
    }
};

// ------------------------------------------------------------- sequences

// The tiles of `rows` consecutive rows that packed sequences are cut into
// are numbered without a list: sequence s owns the numbers from
// rowptr[s] / rows + s on, which are enough for its own tiles (numbers past
// them hold nothing), and total / rows + S numbers serve every batch.
struct SeqTile {
    int seq;      // -1: nothing
    int tile;     // tile of the sequence
};

__device__ inline SeqTile find_seq_tile(const int32_t *rowptr, int S, int rows, int number)
{
    // the last sequence whose first number is <= number
    int lo = 0, hi = S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (rowptr[mid] / rows + mid <= number)
            lo = mid;
        else
            hi = mid;
    }
    SeqTile r;
    const int tile = number - (rowptr[lo] / rows + lo);
    r.seq = tile >= 0 && (int64_t)tile * rows < (int64_t)rowptr[lo + 1] - rowptr[lo] ? lo : -1;
    r.tile = tile;
    return r;
}

// Workgroups reach the 8 XCDs in turn; numbering them so that each XCD takes
// consecutive work keeps the keys of one head in one XCD's L2.
__device__ inline int xcd_order(int block, int count)
{
    const int per = count / 8, rest = count % 8;
    const int x = block % 8, i = block / 8;
    return x * per + (x < rest ? x : rest) + i;
}

__device__ inline bool finite(float x) { return fabsf(x) < __builtin_inff(); }

}  // namespace sdl

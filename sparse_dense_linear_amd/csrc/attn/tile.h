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

#include <type_traits>

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
// the matrix instructions take them; their sums stay in fp32.  (What is rounded
// away of the score gradients, as a second product: a training step 870 us
// instead of 620.)
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

// The 16 x 16 shape, for few columns: lane l holds row or column l % 16 and
// terms 8 * (l / 16) .. + 7 of 32 (4 * (l / 16) .. + 3 of 16 for the shorter
// step), and of the result column l % 16, rows 4 * (l / 16) + register.
// Again a result is, as it lies, the second operand of the shorter step.
__device__ inline f32x4 mma16(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ inline f32x4 mma16(f32x8 a, f32x8 b, f32x4 c)
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
}

__device__ inline f32x4 mma16_short(s16x4 a, s16x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(a, b, c, 0, 0, 0);
}

__device__ inline f32x4 mma16_short(f32x4 a, f32x4 b, f32x4 c)
{
#pragma unroll
    for (int e = 0; e < 4; ++e)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
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

// x of the four lanes of a column of the 16 x 16 shape.
__device__ inline float max_quarters(float x)
{
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}

__device__ inline float sum_quarters(float x)
{
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return sum_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

__device__ inline float max_of(const f32x16 &x)
{
    float m = fmaxf(fmaxf(x[0], x[1]), x[2]);
#pragma unroll
    for (int r = 3; r < 15; r += 2)
        m = fmaxf(fmaxf(m, x[r]), x[r + 1]);
    return fmaxf(m, x[15]);
}

// The running maximum of a softmax is a reference, not an exact maximum: it
// moves (and the output so far is rescaled) only when a score passes it by
// more than this, in base 2.  Weights then reach up to 2^8, which fp32 sums
// and bf16 operands hold with the same relative precision.  Without it some
// query of a wavefront finds a new maximum in almost every tile.
constexpr float kLazy = 8.0f;

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

// 16 bytes a lane from `from` (any address) to `to` + 16 * lane, where `to`
// is the same for the whole wavefront.
__device__ inline void load_to_lds(const void *from, char *to)
{
    typedef __attribute__((address_space(1))) const uint32_t global_u32;
    typedef __attribute__((address_space(3))) uint32_t lds_u32;
    __builtin_amdgcn_global_load_lds((global_u32 *)from, (lds_u32 *)to, 16, 0, 0);
}

// Until every load of this wavefront has arrived.
__device__ inline void wait_loads()
{
    __builtin_amdgcn_s_waitcnt(0x0f70);      // vmcnt(0), nothing else
}

// A number that the compiler takes to be new here.  Addresses of fragments
// differ from a lane's base by an exclusive or and a constant; left alone,
// the compiler computes all of them (some 60) once before a loop over tiles
// and has no registers left for the tiles themselves.
__device__ inline int renewed(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// A tile of ROWS rows of DP elements, of which the kernels work on the first
// DU (D of 65 .. 96 lies in rows of 128 and costs three quarters of them: of
// a training step in fp32 with D = 80 that saved 48 of 249 us).
// The 16-byte pieces of a row are exchanged among themselves by its row number:
// neighbouring rows differ by a pair of pieces and every eighth one by the order
// within the pair, so that 8 lanes that read one piece of 8 consecutive rows,
// and 32 lanes that read across a row and across the one 4 further, touch
// different banks: loops of nothing but these reads count no conflicts.  bf16's
// transposing reads (16 lanes, 32 bytes of 4 rows) count half of their cycles as
// conflicts.  Rows 16 apart are exchanged alike.
template <class T, int DP, int ROWS>
struct Tile {
    static constexpr int kRowBytes = DP * (int)sizeof(T);
    static constexpr int kPieces = kRowBytes / 16;            // per row
    static constexpr int kElems = 16 / (int)sizeof(T);        // per piece
    static constexpr int kBytes = ROWS * kRowBytes;
    static constexpr int kShift = kRowBytes <= 128 ? 1 : 0;   // rows per 256 bytes
    static constexpr int kMask = (kPieces < 16 ? kPieces : 16) / 2 - 1;

    __device__ static int exchange(int row)
    {
        return ((row >> kShift) & kMask) << 1 | ((row >> 3) & 1);
    }

    __device__ static int at(int row, int piece)
    {
        return row * kRowBytes + ((piece ^ exchange(row)) << 4);
    }

    // Where a lane's fragments start: row_frag and col_frag add the rest.
    __device__ static int row_base(int lane)
    {
        return at(lane & 31, (sizeof(T) == 2 ? 1 : 2) * (lane >> 5));
    }
    __device__ static int col_base(int lane)
    {
        if constexpr (sizeof(T) == 2) {
            const int i = lane & 15;
            const int row = 4 * (lane >> 5) + (i >> 2), d = (lane & 16) + 4 * (i & 3);
            return at(row, d >> 3) + 2 * (d & 7);
        } else {
            return at(4 * (lane >> 5), (lane & 31) >> 2) + 4 * (lane & 3);
        }
    }

    // A operand with the tile's rows as rows: row 32 * block + lane % 32,
    // terms 16 * step + 8 * half .. + 7 along D.
    __device__ static Frag<T> row_frag(const char *tile, int row_base, int block, int step)
    {
        const char *p = tile + 32 * block * kRowBytes;
        if constexpr (sizeof(T) == 2) {
            return *(const bf16x8 *)(p + (row_base ^ (step << 5)));
        } else {
            const f32x4 a = *(const f32x4 *)(p + (row_base ^ (step << 6)));
            const f32x4 b = *(const f32x4 *)(p + (row_base ^ (step << 6 | 16)));
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }

    // A operand with D as rows (32 * block + l % 32) and the tile's rows
    // 16 * group .. + 15 as terms in the order of result_frag.  bf16: two
    // transposing reads (each group of 16 lanes hands in 4 rows of 16
    // elements and takes one column of them per lane).
    __device__ static Frag<T> col_frag(const char *tile, int col_base, int group, int block)
    {
        const char *p = tile + 16 * group * kRowBytes;
        if constexpr (sizeof(T) == 2) {
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4 *)(p + (col_base ^ (block << 6))));
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4 *)(p + 8 * kRowBytes + (col_base ^ exchanged(8) ^ (block << 6))));
            const auto ab = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(bf16x8, ab);
        } else {
            f32x8 f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int row = (e & 3) + 8 * (e >> 2);
                f[e] = *(const float *)(p + row * kRowBytes + (col_base ^ exchanged(row) ^ (block << 7)));
            }
            return f;
        }
    }

    // The exchange of a row r + c against that of row r, where c = 0 .. 3 or
    // 8 .. 11 is added to a multiple of 4 below 8, in bytes.  (c and the
    // multiple share no bit, so the exchange of their sum is that of c
    // applied to that of the multiple.)
    __device__ static constexpr int exchanged(int c)
    {
        return (((c >> kShift) & kMask) << 1 | ((c >> 3) & 1)) << 4;
    }
};

// A tile's rows on their way from global memory into LDS without passing
// through registers: a wavefront's lanes write 16 consecutive bytes each, so
// the exchange of pieces is done on the side of the addresses that are read.
// Each of WAVES wavefronts moves its share; the tile is whole once all of
// them have passed wait_loads() and a barrier.
//
// Row r of the tile at `first` is row min(first + r, last) of the operand;
// pieces past D repeat the row's last one, whose products meet zeros of the
// other operand.
template <class T, int DP, int ROWS, int WAVES>
struct Stager {
    typedef Tile<T, DP, ROWS> Tl;
    static constexpr int kThreads = 64 * WAVES;
    static constexpr int kCount = ROWS * Tl::kPieces / kThreads;
    static constexpr int kStep = kThreads / Tl::kPieces;      // rows of one turn
    static_assert(ROWS * Tl::kPieces % kThreads == 0, "whole pieces per thread");
    static_assert(kStep * Tl::kPieces == kThreads, "whole rows per turn");

    static_assert(kStep % 8 == 0, "every second turn is exchanged alike");

    int64_t stride;
    int D;
    uint32_t offset[kStep % 16 == 0 ? 1 : 2];   // the lane's bytes of even and odd turns
    bool near;                                  // which fit 32 bits

    // the lane's row of a turn, and its element in turn i
    __device__ static int row_of(int n) { return n / Tl::kPieces; }
    __device__ int elem_of(int n, int i) const
    {
        const int p = (n % Tl::kPieces) ^ Tl::exchange(row_of(n) + i * kStep);
        return p * Tl::kElems < D ? p * Tl::kElems : D - Tl::kElems;
    }

    __device__ Stager(int64_t stride_, int D_) : stride(stride_), D(D_)
    {
        const int n = threadIdx.x;
        near = kStep * stride * (int64_t)sizeof(T) < ((int64_t)1 << 31);
#pragma unroll
        for (int i = 0; i < (kStep % 16 == 0 ? 1 : 2); ++i)
            offset[i] = (uint32_t)((row_of(n) * stride + elem_of(n, i)) * (int64_t)sizeof(T));
    }

    __device__ void load(char *tile, const T *base, int first, int last, int wave) const
    {
        char *to = tile + wave * 1024;
        if (near && first + ROWS - 1 <= last) {
            // all rows are there: one scalar address a turn, one offset a lane
            const char *from = (const char *)(base + first * stride);
#pragma unroll
            for (int i = 0; i < kCount; ++i)
                load_to_lds(from + i * kStep * stride * (int64_t)sizeof(T) +
                                offset[kStep % 16 == 0 ? 0 : i & 1],
                            to + i * kThreads * 16);
        } else {
            const int n = renewed(threadIdx.x);
#pragma unroll
            for (int i = 0; i < kCount; ++i) {
                const int r = first + i * kStep + row_of(n);
                load_to_lds(base + (r < last ? r : last) * stride + elem_of(n, i), to + i * kThreads * 16);
            }
        }
    }
};

// One wavefront's share of attention with C = 32 or 16 queries as columns:
// the shapes, fragments and reductions that depend on C.  A block of keys is
// C keys; `part` is the lane's share of the terms, lane / C.
template <class T, int DP, int DU, int ROWS, int C> struct Cols;

template <class T, int DP, int DU, int ROWS>
struct Cols<T, DP, DU, ROWS, 32> {
    typedef Tile<T, DP, ROWS> Tl;
    typedef f32x16 Acc;
    static constexpr int kAcc = 16, kSteps = DU / 16, kTerms = 16, kBlocks = DU / 32, kGroups = 2;
    __device__ static int key_of(int r) { return 8 * (r >> 2) + (r & 3); }    // + 4 * part
    __device__ static int row_base(int lane) { return Tl::row_base(lane); }
    __device__ static int col_base(int lane) { return Tl::col_base(lane); }
    __device__ static Frag<T> key_frag(const char *tile, int base, int step)
    {
        return Tl::row_frag(tile, base, 0, step);
    }
    __device__ static Acc mul(Frag<T> a, Frag<T> b, Acc c) { return mma(a, b, c); }
    __device__ static float most(const Acc &x) { return max_halves(max_of(x)); }
    __device__ static float sum(float x) { return sum_halves(x); }
    typedef Frag<T> Weights;
    __device__ static Weights weights(const Acc &x, int group) { return result_frag<T>(x, group); }
    __device__ static Weights val_frag(const char *tile, int base, int group, int block)
    {
        return Tl::col_frag(tile, base, group, block);
    }
    __device__ static Acc apply(Weights v, Weights p, Acc o) { return mma(v, p, o); }
};

template <class T, int DP, int DU, int ROWS>
struct Cols<T, DP, DU, ROWS, 16> {
    typedef Tile<T, DP, ROWS> Tl;
    typedef f32x4 Acc;
    static constexpr int kAcc = 4, kSteps = DU / 32, kTerms = 32, kBlocks = DU / 16, kGroups = 1;
    __device__ static int key_of(int r) { return r; }                          // + 4 * part
    __device__ static int row_base(int lane)
    {
        return Tl::at(lane & 15, (sizeof(T) == 2 ? 1 : 2) * (lane >> 4));
    }
    __device__ static int col_base(int lane)
    {
        const int i = lane & 15, part = lane >> 4;
        if constexpr (sizeof(T) == 2)
            return Tl::at(4 * part + (i >> 2), (i & 3) >> 1) + 8 * (i & 1);
        else
            return Tl::at(4 * part, i >> 2) + 4 * (i & 3);
    }
    __device__ static Frag<T> key_frag(const char *tile, int base, int step)
    {
        if constexpr (sizeof(T) == 2) {
            return *(const bf16x8 *)(tile + (base ^ (step << 6)));
        } else {
            const f32x4 a = *(const f32x4 *)(tile + (base ^ (step << 7)));
            const f32x4 b = *(const f32x4 *)(tile + (base ^ (step << 7 | 16)));
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    __device__ static Acc mul(Frag<T> a, Frag<T> b, Acc c) { return mma16(a, b, c); }
    __device__ static float most(const Acc &x)
    {
        return max_quarters(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
    }
    __device__ static float sum(float x) { return sum_quarters(x); }
    typedef std::conditional_t<sizeof(T) == 2, s16x4, f32x4> Weights;
    __device__ static Weights weights(const Acc &x, int)
    {
        if constexpr (sizeof(T) == 2) {
            const bf16x4 p = {(__bf16)x[0], (__bf16)x[1], (__bf16)x[2], (__bf16)x[3]};
            return __builtin_bit_cast(s16x4, p);
        } else {
            return x;
        }
    }
    __device__ static Weights val_frag(const char *tile, int base, int, int block)
    {
        if constexpr (sizeof(T) == 2) {
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(tile + (base ^ (block << 5))));
        } else {
            f32x4 f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = *(const float *)(tile + e * Tl::kRowBytes + (base ^ Tl::exchanged(e) ^ (block << 6)));
            return f;
        }
    }
    __device__ static Acc apply(Weights v, Weights p, Acc o) { return mma16_short(v, p, o); }
};

// A wavefront's 32 columns of DU results to LDS and back, for the wavefronts
// that share them: `block` of the results is rows 32 * block .. of D.
template <int DP, int DU>
struct Parked {
    typedef Tile<float, DP, 32> Tl;
    static constexpr int kBytes = Tl::kBytes;
    __device__ static void put(char *to, int lane, const f32x16 (&x)[DU / 32])
    {
#pragma unroll
        for (int d = 0; d < DU / 32; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                store4((float *)(to + Tl::at(lane & 31, 8 * d + 2 * g + (lane >> 5))), x[d][4 * g],
                       x[d][4 * g + 1], x[d][4 * g + 2], x[d][4 * g + 3]);
    }
    // x = mine * x + theirs * what was put
    __device__ static void add(const char *from, int lane, float mine, float theirs,
                               f32x16 (&x)[DU / 32])
    {
#pragma unroll
        for (int d = 0; d < DU / 32; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 y =
                    *(const f32x4 *)(from + Tl::at(lane & 31, 8 * d + 2 * g + (lane >> 5)));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[d][4 * g + e] = fmaf(theirs, y[e], mine * x[d][4 * g + e]);
            }
    }
};

// The compiler moves no instruction across this point.
__host__ __device__ inline void keep_order()
{
#ifdef __HIP_DEVICE_COMPILE__
    __builtin_amdgcn_sched_barrier(0);
#endif
}

// COUNT matrix instructions in a row, use(i, read(i)), with the LDS reads of
// the next AHEAD of them under way (of all of them, where they are no more).
// Left to itself the compiler keeps one operand's registers and waits out the
// latency of LDS before every instruction, where registers are scarce; the
// order here is therefore fixed.
template <int COUNT, int AHEAD, class Read, class Use>
__host__ __device__ inline void chain(Read read, Use use)
{
    constexpr int kAhead = AHEAD < COUNT ? AHEAD : COUNT;
    decltype(read(0)) f[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        f[i] = read(i);
    keep_order();
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
        use(i, f[i % kAhead]);
        if (i + kAhead < COUNT)
            f[i % kAhead] = read(i + kAhead);
        keep_order();
    }
}

// --------------------------------------------------------------- window

// What a query at position p sees: keys j <= p with p - j < window or
// j < sinks (positions count from the sequence's first key).
struct Seen {
    int window, sinks;
    __device__ bool operator()(int p, int j) const
    {
        // p - j as unsigned: a later key is past every limit
        return (uint32_t)(p - j) < (uint32_t)(j < sinks ? 0x7fffffff : window);
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

// Scores of one 32 x 32 result whose pair is not seen become -infinity, and
// its elements of `zeroed` 0: what the weight of 0 multiplies later must not be
// an infinity.  Lane: one query at position p; rows: keys from j0 on.
// (renewed() keeps the comparisons on the caller's side of its branch: most
// tiles lie within the window and skip them.)
template <class... Zeroed>
__device__ inline void mask_keys(const Seen &seen, int p, int j0, int half, f32x16 &x, Zeroed &...zeroed)
{
    const int t = renewed(p - j0 - 4 * half);
    if (j0 >= seen.sinks) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if ((uint32_t)(t - (8 * (r >> 2) + (r & 3))) >= (uint32_t)seen.window) {
                x[r] = SDL_NEG_INF;
                ((zeroed[r] = 0.0f), ...);
            }
    } else {
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if (!seen(p, p - t + 8 * (r >> 2) + (r & 3))) {
                x[r] = SDL_NEG_INF;
                ((zeroed[r] = 0.0f), ...);
            }
    }
}

// The same with one key a lane, rows: queries from position p0 on, of which
// `count` exist.
__device__ inline void mask_queries(const Seen &seen, int key, int p0, int count, int half, f32x16 &x,
                                    f32x16 &zeroed)
{
    const int t = renewed(p0 - key + 4 * half);
    const uint32_t limit = key < seen.sinks ? 0x7fffffff : seen.window;
#pragma unroll
    for (int r = 0; r < 16; ++r)
        if ((uint32_t)(t + 8 * (r >> 2) + (r & 3)) >= limit) {
            x[r] = SDL_NEG_INF;
            zeroed[r] = 0.0f;
        }
    if (count < 32) {
        const int left = renewed(count - 4 * half);
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if (8 * (r >> 2) + (r & 3) >= left) {
                x[r] = SDL_NEG_INF;
                zeroed[r] = 0.0f;
            }
    }
}

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

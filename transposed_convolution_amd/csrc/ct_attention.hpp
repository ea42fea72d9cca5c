// ct_attention.hpp -- what the attention kernels share: tiles in LDS that are read by rows and by
// columns, fragments of the matrix instructions, and the launchers' declarations.
//
// The mathematics of all three kernels is laid out so that no value changes its lane.  A 32 x 32
// product leaves lane l with column l % 32 and, in register r, row 8 (r / 4) + 4 (l / 32) + r % 4.
// Its next use is as the right operand of a product whose sum runs over those rows: there lane l
// has to bring 8 values of column l % 32 a step, and any 8 rows will do if the left operand brings
// the same ones.  So registers 8 s .. 8 s + 7 go in as they are, and the left operand is read from
// LDS by columns at the rows 16 s + 4 (l / 32) + {0..3, 8..11}: for 16-bit types two transposing
// reads (ds_read_b64_tr_b16) an operand, for float32 eight words.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "ct_vec.hpp"

namespace ct {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kMaxHead = 256;  // elements of a head that the kernels' registers hold

// Strides (elements) of the image, token and head axes of an (N, T, H, D) tensor whose D is dense.  A
// token's is at most 2^24, so that the 64 rows of a tile are 32-bit byte offsets from its start.
struct Strided {
    const void *p = nullptr;
    int64_t n = 0, t = 0, h = 0;
};
constexpr int64_t kMaxTokenStride = int64_t(1) << 24;

// Division of u < 2^31 by d >= 1: with s = ceil(log2 d) and m = ceil(2^(31 + s) / d) the error of m is
// below 2^s / d, that of 2 u m / 2^(32 + s) below 1 / d.
struct Div31 {
    unsigned m = 0x80000000u;
    int s = 0, d = 1;
    Div31() = default;
    explicit Div31(int dv) : d(dv)
    {
        while ((int64_t(1) << s) < d) ++s;
        m = unsigned(((uint64_t(1) << (31 + s)) + d - 1) / d);
    }
    __device__ __forceinline__ int div(int u) const { return int(__umulhi(unsigned(u) << 1, m) >> s); }
};

// One call, either direction.  The G = H / Hkv query heads of a key head and the Tq tokens are
// one axis of R = Tq * G rows, row = token * G + head: a tile of keys serves all of them, and a
// single token still has G rows for the matrix instructions.  Tokens, rows and keys are below 2^30.
struct Attention {
    Strided q, k, v, o, d_o;   // o, d_o: the gradient's inputs
    int N = 0, Tq = 0, Tk = 0, H = 0, Hkv = 0, G = 1, D = 0, R = 0;
    Div31 by_g;
    float scale = 1.0f;
    int causal = 0;
    const int *lengths = nullptr, *starts = nullptr;
    void *out = nullptr;       // forward: (N, Tq, H, D) dense
    float *lse = nullptr;      // (N, H, Tq): written by the forward call, read by the gradient
    void *dq = nullptr, *dk = nullptr, *dv = nullptr;

    // The place of an image's first query among the keys, within what makes a difference.
    __device__ __forceinline__ int start(int n) const { return starts ? max(-Tq, min(starts[n], Tk)) : Tk - Tq; }
    // An image's keys: those that one of its tokens sees at all.
    __device__ __forceinline__ int length(int n, int start) const
    {
        return Tq == 0 ? 0 : seen(lengths ? max(0, min(lengths[n], Tk)) : Tk, start, Tq - 1);
    }
    // Keys that token t of an image sees: the first seen(...) ones.
    __device__ __forceinline__ int seen(int len, int start, int t) const
    {
        return causal ? max(0, min(start + t + 1, len)) : len;
    }
    // The first token that sees a key at all.
    __device__ __forceinline__ int first_token(int len, int start) const
    {
        return len == 0 ? Tq : causal ? max(0, -start) : 0;
    }
};

// The i-th tile of rows that an image's key head gives out.  In a causal call later rows see more keys: the longest
// go first.  Where the heads do not come out even over the 8 XCDs, some of which then take parts of a head, long and
// short ones take turns, so that every part is a fair one (4 heads of 129 tiles in whole order
// gave one XCD three times the work of the next).
__device__ __forceinline__ int long_first(int i, int tiles, int heads)
{
    return heads & 7 ? (i & 1 ? i >> 1 : tiles - 1 - (i >> 1)) : tiles - 1 - i;
}

using f32x16 = float __attribute__((ext_vector_type(16)));
using f32x4 = float __attribute__((ext_vector_type(4)));

template <class T>
using Frag = T __attribute__((ext_vector_type(8)));  // 8 values of one row or column for a step of 16

// A 32 x 32 product over 16, in float32 (float32 operands: 8 instructions over 2 each; the sum
// runs over the same 16 whatever place a value has in it, as long as both operands agree).
__device__ __forceinline__ f32x16 mma(Frag<_Float16> a, Frag<_Float16> b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(Frag<__bf16> a, Frag<__bf16> b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(Frag<float> a, Frag<float> b, f32x16 c)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
    return c;
}

// Registers 8 s .. 8 s + 7 of a product as an operand, one rounding to T.
template <class T>
__device__ __forceinline__ Frag<T> operand(const f32x16 &c, int s)
{
    Frag<float> v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c[8 * s + j];
    return __builtin_convertvector(v, Frag<T>);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Row of register r of a product.
__device__ __forceinline__ constexpr int c_row(int r, int half) { return 8 * (r / 4) + 4 * half + r % 4; }

// The values of lane l % 32 and of the lane 32 above it, in both.  (The elements go through
// variables: a bit cast of a vector's element takes its first one.)
__device__ __forceinline__ void both_halves(float x, float &low, float &high)
{
    const unsigned u = __builtin_bit_cast(unsigned, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned a = r[0], b = r[1];
    low = __builtin_bit_cast(float, a);
    high = __builtin_bit_cast(float, b);
}
__device__ __forceinline__ float half_max(float x)
{
    float a, b;
    both_halves(x, a, b);
    return fmaxf(a, b);
}
__device__ __forceinline__ float half_sum(float x)
{
    float a, b;
    both_halves(x, a, b);
    return a + b;
}

// 16 bytes of a row, of which the first `valid` elements exist; the others are 0.  Where a row does not end
// with a whole chunk its last one has `tail` elements, the same number everywhere: loads of 4, 2 and
// 1 of them as it takes, not one an element.
template <class T>
__device__ __forceinline__ Raw<T, kVec<T>> load_chunk(const T *p, int valid, int tail)
{
    constexpr int V = kVec<T>;
    Raw<T, V> r = {};
    if (valid >= V) r = *reinterpret_cast<const Raw<T, V> *>(p);
    if (tail && valid > 0 && valid < V) {
        using U1 = std::conditional_t<sizeof(T) == 2, unsigned short, unsigned>;
        using U2 = U1 __attribute__((ext_vector_type(2), aligned(sizeof(T))));
        using U4 = U1 __attribute__((ext_vector_type(4), aligned(sizeof(T))));
        const U1 *q = reinterpret_cast<const U1 *>(p);
        U4 four = {};
        U2 two = {};
        U1 one = 0;
        if (V == 8 && tail & 4) four = *reinterpret_cast<const U4 *>(q);
        if (tail & 2) two = *reinterpret_cast<const U2 *>(q + (tail & 4));
        if (tail & 1) one = q[tail & 6];
        U1 u[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int in2 = j - (tail & 4), in1 = j - (tail & 6);
            U1 v = in1 == 0 && tail & 1 ? one : U1(0);
            if (tail & 2) v = in2 == 0 ? two[0] : in2 == 1 ? two[1] : v;
            if (V == 8 && j < 4 && tail & 4) v = four[j & 3];
            u[j] = v;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) r[j] = __builtin_bit_cast(T, u[j]);
    }
    return r;
}

// 8 elements d .. d + 7 of a row of D, 0 behind it.
template <class T>
__device__ __forceinline__ Frag<T> load_frag(const T *row, int d, int D)
{
    constexpr int V = kVec<T>;
    Frag<T> f;
#pragma unroll
    for (int c = 0; c < 8 / V; ++c) {
        const Raw<T, V> r = load_chunk<T>(row + d + c * V, D - d - c * V, D % V);
#pragma unroll
        for (int j = 0; j < V; ++j) f[c * V + j] = r[j];
    }
    return f;
}

// A tile of rows of DP elements in LDS, in 16-byte chunks.  Chunk c of row r lies at c ^ turn(r),
// which keeps both kinds of read free of bank conflicts: by rows, 16 lanes read one chunk of 16
// consecutive rows; by columns, 32 lanes read 4 chunks of 4 consecutive rows.  A row has 4 g
// chunks; g odd: 4 rows cover the 64 banks 4 chunks each and 2 bits are turned; g = 2 (mod 4):
// 2 rows cover them, 3 bits; g = 0 (mod 4): 4 bits.
template <class T, int DP>
struct Tile {
    static constexpr int kChunk = int(16 / sizeof(T)), kChunks = DP / kChunk, kG = kChunks / 4;
    static_assert(DP % 32 == 0, "whole products over columns");
    __device__ static __forceinline__ int turn(int row)
    {
        const int low = row >> 2 & 3;
        return kG % 2 ? low : kG % 4 == 2 ? low | (row & 2) << 1 : low | (row & 3) << 2;
    }
    __device__ static __forceinline__ int at(int row, int chunk) { return row * DP + (chunk ^ turn(row)) * kChunk; }
    // the 8 values of `row` for step ks: the elements 16 ks + 8 half ..
    __device__ static __forceinline__ Frag<T> by_rows(const T *tile, int row, int ks, int half)
    {
        Frag<T> f;
        if constexpr (sizeof(T) == 2) {
            f = *reinterpret_cast<const Frag<T> *>(tile + at(row, ks * 2 + half));
        } else {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const Raw<T, 4> r = *reinterpret_cast<const __attribute__((aligned(16))) Raw<T, 4> *>(tile + at(row, ks * 4 + half * 2 + c));
#pragma unroll
                for (int j = 0; j < 4; ++j) f[c * 4 + j] = r[j];
            }
        }
        return f;
    }
    // their place in the tile
    __device__ static __forceinline__ void put(T *tile, int row, int ks, int half, const Frag<T> &f)
    {
#pragma unroll
        for (int c = 0; c < 8 / kChunk; ++c) {
            Raw<T, kChunk> r;
#pragma unroll
            for (int j = 0; j < kChunk; ++j) r[j] = f[c * kChunk + j];
            *reinterpret_cast<__attribute__((aligned(16))) Raw<T, kChunk> *>(tile + at(row, (ks * 2 + half) * (8 / kChunk) + c)) = r;
        }
    }
    // the 8 values of column 32 db + lane % 32 at the rows row0 + 4 (lane / 32) + {0..3, 8..11};
    // row0 a multiple of 16
    __device__ static __forceinline__ Frag<T> by_columns(const T *tile, int row0, int db, int lane)
    {
        const int half = lane >> 5;
        Frag<T> f;
        if constexpr (sizeof(T) == 2) {
            // 16 lanes read 4 rows of 16 elements; lane i gets column i of them
            using V4 = short __attribute__((ext_vector_type(4)));
            const int in = lane & 15, col = db * 32 + (lane & 16) + (in & 3) * 4;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = row0 + 8 * c + 4 * half + (in >> 2);
                const T *p = tile + at(row, col / 8) + (col & 7);
                const V4 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) V4 *)(const_cast<T *>(p)));
                const Raw<T, 4> v = __builtin_bit_cast(Raw<T, 4>, r);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[c * 4 + j] = v[j];
            }
        } else {
            const int col = db * 32 + (lane & 31);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int row = row0 + 4 * half + (j & 3) + (j & 4) * 2;
                f[j] = tile[at(row, col / 4) + (col & 3)];
            }
        }
        return f;
    }
};

// N operands read from LDS, each for a matrix instruction, P of them ahead of their use.  Left to itself the compiler
// asks for an operand right before its instruction when registers are short, and every instruction
// then waits for LDS; here reads and matrix instructions keep the order they are written in.
template <class T, int N, int P>
struct Ahead {
    Frag<T> f[P];
    template <class L>
    __device__ __forceinline__ void prime(L &&load)
    {
#pragma unroll
        for (int i = 0; i < P && i < N; ++i) f[i] = load(i);
        keep_order();
    }
    template <class L, class U>
    __device__ __forceinline__ void run(L &&load, U &&use)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            use(i, f[i % P]);
            if (i + P < N) f[i % P] = load(i + P);
            keep_order();
        }
    }
    // vector, scalar and transcendental instructions and global loads may pass
    __device__ static __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0x416); }
};

// ROWS rows on their way from memory to a tile, 16 bytes a thread and piece; the threads of a row are a
// power of two, so that a thread keeps its column.
template <class T, int DP, int ROWS, int THREADS>
struct Mover {
    using L = Tile<T, DP>;
    using Chunk = Raw<T, L::kChunk>;
    static constexpr int kLanes = L::kChunks <= 4 ? 4 : L::kChunks <= 8 ? 8 : L::kChunks <= 16 ? 16 : L::kChunks <= 32 ? 32 : 64;
    static constexpr int kStep = THREADS / kLanes, kPieces = ROWS / kStep;
    static_assert(ROWS % kStep == 0 && THREADS % kLanes == 0, "every thread has as many pieces");
    Chunk r[kPieces];
    int row0, column;  // of the thread: first row, first element
    __device__ __forceinline__ explicit Mover(int tid) : row0(tid / kLanes), column(tid % kLanes * L::kChunk)
    {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) r[i] = Chunk{};
    }
    // Rows base + row * stride, of which the first `valid` exist; the others become zeros.
    __device__ __forceinline__ void load(const T *base, int64_t stride, int valid, int D)
    {
        const unsigned at = unsigned(row0 * int(stride) + column) * unsigned(sizeof(T));
        const char *p = reinterpret_cast<const char *>(base);
        const int64_t step = kStep * stride * int64_t(sizeof(T));
        if (valid >= ROWS && D % L::kChunk == 0) {
            whole(D, [&](int i) { return p + i * step + at; });
        } else {
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                r[i] = load_chunk<T>(reinterpret_cast<const T *>(p + i * step + at), row0 + i * kStep < valid ? D - column : 0, D % L::kChunk);
        }
    }
    // Pieces that all exist, of rows of whole chunks, from at(i).
    template <class F>
    __device__ __forceinline__ void whole(int D, F &&at)
    {
        if (L::kChunks == kLanes && D == DP) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) r[i] = *reinterpret_cast<const Chunk *>(at(i));
        } else if (column < D) {
            // threads behind the row's end keep the zeros they began with
#pragma unroll
            for (int i = 0; i < kPieces; ++i) r[i] = *reinterpret_cast<const Chunk *>(at(i));
        }
    }
    // Rows row(i), null for zeros.
    template <class F>
    __device__ __forceinline__ void load(int D, F &&row)
    {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const T *p = row(row0 + i * kStep);
            r[i] = load_chunk<T>(p + column, p ? D - column : 0, D % L::kChunk);
        }
    }
    // Values that are not finite become zeros; were there any in the wave?  Their exponent is all ones: one more at its
    // lowest bit carries into the sign's, two elements a word where they have 16 bits.
    __device__ __forceinline__ bool drop_not_finite()
    {
        using U = std::conditional_t<sizeof(T) == 2, unsigned short, unsigned>;
        constexpr U ONES = std::is_same_v<T, _Float16> ? 0x7c00 : sizeof(T) == 2 ? 0x7f80 : U(0x7f800000);
        constexpr U LOWEST = std::is_same_v<T, _Float16> ? 0x0400 : sizeof(T) == 2 ? 0x0080 : U(0x00800000);
        constexpr unsigned TWICE = sizeof(T) == 2 ? 0x10001u : 1u;
        using Words = unsigned __attribute__((ext_vector_type(4)));
        unsigned carry = 0;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const Words w = __builtin_bit_cast(Words, r[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) carry |= (w[j] & ONES * TWICE) + LOWEST * TWICE;
        }
        const bool found = __any(carry & (sizeof(T) == 2 ? 0x80008000u : 0x80000000u));
        if (__builtin_expect(found, 0)) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
#pragma unroll
                for (int j = 0; j < L::kChunk; ++j) {
                    const T x = r[i][j];
                    r[i][j] = (__builtin_bit_cast(U, x) & ONES) == ONES ? T(0.0f) : x;
                }
        }
        return found;
    }
    __device__ __forceinline__ void store(T *tile) const
    {
        if (L::kChunks == kLanes || column < DP) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                *reinterpret_cast<__attribute__((aligned(16))) Chunk *>(tile + L::at(row0 + i * kStep, column / L::kChunk)) = r[i];
        }
    }
};

// Column `lane % 32` of a (DP x 32) product as a row of D elements of T.
template <class T, int DB>
__device__ __forceinline__ void store_columns(T *row, const f32x16 (&c)[DB], float factor, int D, int half)
{
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int d = db * 32 + 8 * k + 4 * half;
            Raw<T, 4> v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = T(c[db][4 * k + j] * factor);
            if (d + 4 <= D) {
                *reinterpret_cast<Raw<T, 4> *>(row + d) = v;
            } else {
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (d + j < D) row[d + j] = v[j];
            }
        }
}

inline int padded_head(int64_t D) { return D <= 32 ? 32 : D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : 256; }

// Calls f with the padded head size as a constant.
template <class F>
inline void with_head(int64_t D, F &&f)
{
    switch (padded_head(D)) {
    case 32: f(std::integral_constant<int, 32>{}); break;
    case 64: f(std::integral_constant<int, 64>{}); break;
    case 96: f(std::integral_constant<int, 96>{}); break;
    case 128: f(std::integral_constant<int, 128>{}); break;
    default: f(std::integral_constant<int, 256>{}); break;
    }
}

// How a call's work is cut.  Forward: calls of up to 32 rows a key head (a few tokens) have a kernel
// whose waves take keys each; others give a wave 32 rows.  `splits` parts of the keys (or
// rows) go to different blocks and are joined by a second kernel.
struct AttendPlan {
    bool few = false;
    int tiles = 0, splits = 1, chunk = 1;  // chunk: keys a split
    size_t bytes = 0;    // workspace: the parts of splits
};
AttendPlan attend_plan(const Attention &a, int dtype);
template <class T>
void launch_attend(const Attention &a, const AttendPlan &p, float *part, hipStream_t st);

// The gradient: key blocks take the rows in chunks, row blocks the keys; more than one chunk leaves
// parts that are joined.
struct AttendGradPlan {
    int waves = 4, key_span = 128, row_span = 128;  // keys and rows of a block
    int row_chunk = 1, key_chunk = 1;
    int key_splits = 1, row_splits = 1;             // of the query gradient, of the key and value gradient
    size_t stat = 0, top = 0, key_part = 0, row_part = 0, bytes = 0;  // offsets in the workspace, and its size
};
constexpr size_t kOneWaveBytes = 256;  // longer heads do not fit the registers of the one-wave kernel

// Heads (padded) of 129 to 256 bytes: a block of the key gradient has 8 waves, one block a compute unit, so that its
// keys and values fit LDS.
constexpr bool wide_keys(size_t bytes) { return bytes > 128 && bytes <= 256; }
AttendGradPlan attend_grad_plan(const Attention &a, int dtype);
template <class T>
void launch_attend_grad(const Attention &a, const AttendGradPlan &p, char *ws, hipStream_t st);

}  // namespace ct

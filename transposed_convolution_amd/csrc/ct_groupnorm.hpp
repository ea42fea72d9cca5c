// ct_groupnorm.hpp -- what the group norm kernels share: moments, activations, how a call
// is cut into blocks and how a thread finds its elements.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ct_vec.hpp"

namespace ct {
namespace norm {

// (count, mean, sum of squared distances from the mean).  A thread's own are in float32, its mean
// relative to a value of its own (Moments<float>); where those of threads and blocks are
// joined, means are absolute and 64 bits wide, so that neither a mean far from zero nor a
// single value far from the others costs digits (Moments<double>).
template <class M>
struct Moments {
    float n = 0.0f;
    M mean = 0;
    float m2 = 0.0f;
    __device__ __forceinline__ void join(float bn, M bmean, float bm2)
    {
        const float total = n + bn;
        if (bn > 0.0f) {
            const float d = float(bmean - mean);
            const float w = bn * __builtin_amdgcn_rcpf(total);  // counts: one rounding more is nothing
            mean = n > 0.0f ? mean + M(d * w) : bmean;
            m2 += n > 0.0f ? bm2 + d * d * n * w : bm2;
            n = total;
        }
    }
};

// Activation and its derivative.  Kernels are compiled for SiLU and for the piecewise linear
// kinds (none among them), which are told apart by selects: a switch inside a kernel made
// the compiler hoist the unpacking of every held value above it, into spilled registers.
//
// SiLU by the hardware's 2^x and reciprocal: z log2(e) is rounded before 2^x, so y is off by up to
// (|z| + 5) 2^-24 of itself for negative z (30 at z = -30, where y is 3e-12) and 2.5 * 2^-24
// for others, measured; beside z, about 2^-24.  exp and a division (2.6 * 2^-24
// everywhere) took 50.7 us for 40.2 in an 8 x 256 x 16384 float16 call and 88.6 for 67.5 in
// its gradient.
struct Silu {
    __device__ __forceinline__ float y(float z) const { return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }
    __device__ __forceinline__ float d(float z) const
    {
        const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-z));
        return __builtin_fmaf(z * s, 1.0f - s, s);
    }
};
// A NaN stays NaN in both, ReLU's comparison included: a group with a value that is not finite
// is not to leave as zeros.
struct Piecewise {
    ct::Act a;
    __device__ __forceinline__ float y(float z) const
    {
        // one instruction for a maximum that keeps NaN, where a comparison and a select are two
        const float relu = __builtin_elementwise_maximum(z, 0.0f);
        const float leaky = z >= 0.0f ? z : a.p0 * z;
        const float clip = __builtin_elementwise_minimum(__builtin_elementwise_maximum(z, a.p0), a.p1);
        return a.kind == CT_ACT_RELU ? relu : a.kind == CT_ACT_LEAKY_RELU ? leaky : a.kind == CT_ACT_CLIP ? clip : z;
    }
    __device__ __forceinline__ float d(float z) const
    {
        const float relu = z > 0.0f ? 1.0f : 0.0f;
        const float leaky = z >= 0.0f ? 1.0f : a.p0;
        const float clip = z >= a.p0 && z <= a.p1 ? 1.0f : 0.0f;
        const float d = a.kind == CT_ACT_RELU ? relu : a.kind == CT_ACT_LEAKY_RELU ? leaky : clip;
        return a.identity() ? 1.0f : z == z ? d : z;
    }
};
template <class F>
void with_act(const ct::Act &a, F &&f)
{
    if (a.kind == CT_ACT_SILU) f(Silu{});
    else f(Piecewise{a});
}

// x - mu, and x * f: the value times an opaque 1 (or f) plus a term, which for float16 is one
// mixed-precision FMA on the packed half where the plain forms unpack it first.
__device__ __forceinline__ float opaque_one()
{
    float one = 1.0f;
    asm("" : "+v"(one));
    return one;
}
template <class T>
__device__ __forceinline__ float minus(T x, float mu, float one)
{
    return __builtin_fmaf(float(x), one, -mu);
}
template <class T>
__device__ __forceinline__ float times(T x, float f)
{
    return __builtin_fmaf(float(x), f, 0.0f);
}

// V elements of which the first `valid` exist.
template <class T, int V>
__device__ __forceinline__ Raw<T, V> load_first(const T *p, int valid)
{
    if (valid >= V) return *reinterpret_cast<const Raw<T, V> *>(p);
    Raw<T, V> r{};
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (j < valid) r[j] = p[j];
    return r;
}
template <class T, int V>
__device__ __forceinline__ void store_first(T *p, const Raw<T, V> &r, int valid)
{
    if (valid >= V) {
        __builtin_nontemporal_store(r, reinterpret_cast<Raw<T, V> *>(p));  // nobody here reads it again
        return;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (j < valid) p[j] = r[j];
}

// ------------------------------------------------------------------------------------
// How (N, P, C) is cut
// ------------------------------------------------------------------------------------
// Slabs of whole groups, as many as a tile's row holds (or, where one group is wider than
// that, of a part of a group), and chunks of `tiles` tiles of `rows` positions.  A thread
// owns the V consecutive elements at e = V * thread of every tile (a tile's elements run
// through its rows), so its channels are the same in all of them.  One slab holding all
// channels may have any width: its tile is contiguous and a vector may run over a row's end.
constexpr int kMostGroups = 1024;  // groups of a slab
struct Cut {
    int64_t P;
    int C, G, Cg;
    int width, slabs;  // channels of a slab (the last, or a group's last, may be narrower)
    int per;           // groups of a slab
    int split;         // slabs of a group: 1, or more when a group is wider than a slab
    int rows, tiles, chunks;
    int last_tiles, last_rows;  // tiles of the last chunk, positions of its last tile
    int lanes;  // threads that share a group when partials are joined: a power of two

    __host__ __device__ int64_t span() const { return int64_t(tiles) * rows; }  // positions of a chunk
};

// A block's image, chunk and slab, and the thread's vector within a tile.  An address is
// kept as a block-uniform tile offset (scalar registers) and the thread's 32-bit offset in
// the tile: 64-bit addresses of every tile would take the registers that hold the tiles.
template <int V>
struct Place {
    int64_t n;
    int chunk, sub;
    int g0, groups;  // groups of the slab
    int c0, width;   // its channels
    int e, col;
    unsigned off;  // elements
    bool active;
    __device__ Place(const Cut &k, unsigned b)
    {
        const unsigned rest = b / unsigned(k.slabs);
        const int slab = int(b - rest * unsigned(k.slabs));
        n = rest / unsigned(k.chunks);
        chunk = int(rest - unsigned(n) * unsigned(k.chunks));
        if (k.split == 1) {
            sub = 0;
            g0 = slab * k.per;
            groups = k.G - g0 < k.per ? k.G - g0 : k.per;
            c0 = g0 * k.Cg;
            width = groups * k.Cg;
        } else {
            g0 = slab / k.split;
            sub = slab - g0 * k.split;
            groups = 1;
            c0 = g0 * k.Cg + sub * k.width;
            width = k.Cg - sub * k.width < k.width ? k.Cg - sub * k.width : k.width;
        }
        e = int(threadIdx.x) * V;
        active = e < k.rows * width;
        if (!active) e = 0;
        const int row = e / width;
        col = e - row * width;
        off = unsigned(row) * unsigned(k.C) + unsigned(col);
    }
    // element offset of the block's tile i
    __device__ __forceinline__ int64_t tile(const Cut &k, int i) const
    {
        return (n * k.P + (int64_t(chunk) * k.tiles + i) * k.rows) * k.C + c0;
    }
    // how many of the V elements exist in tile i
    __device__ __forceinline__ int valid(const Cut &k, int i) const
    {
        const int64_t left = k.P - (int64_t(chunk) * k.tiles + i) * k.rows;
        const int there = i >= k.tiles || left <= 0 ? 0 : int(left < k.rows ? left : k.rows) * width;
        const int mine = active ? there - e : 0;
        return mine >= V ? V : mine > 0 ? mine : 0;
    }
    // tiles first .. first + count - 1 exist and hold all their positions
    __device__ __forceinline__ bool full(const Cut &k, int first, int count) const
    {
        return first + count <= k.tiles && (int64_t(chunk) * k.tiles + first + count) * k.rows <= k.P;
    }
    // Calls f(i, channel of the slab, group of the slab) for the first of each S elements.
    template <int S, class F>
    __device__ __forceinline__ void each(const Cut &k, F f) const
    {
        int c = col, g = k.split > 1 ? 0 : col / k.Cg, left = k.split > 1 ? width : (g + 1) * k.Cg - col;
#pragma unroll
        for (int i = 0; i < V / S; ++i) {
            f(i, c, g);
            c += S;
            left -= S;
            if (left == 0) {
                ++g;
                left = k.Cg;
            }
            if (c == width) {
                c = 0;
                g = 0;
                left = k.Cg;
            }
        }
    }
    // The parameter's values of the thread's channels.
    template <class T>
    __device__ __forceinline__ void params(float (&out)[V], const Cut &k, const Param<T> &p, float absent) const
    {
        if (width % V == 0) p.template run<V>(out, c0 + col, absent);
        else each<1>(k, [&](int j, int c, int) { out[j] = p.at(c0 + c, absent); });
    }
};

// S: so many consecutive elements of a vector are known to share a group (V, 4 or 1), so the
// thread keeps V / S triples, means and the like.  With S > 1 every vector starts at a
// multiple of V elements.
template <int S, int V>
constexpr int kOwn = V / S;
template <int S, int V>
using OwnMoments = Moments<float>[kOwn<S, V>];
template <int S, int V>
using OwnFloats = float[kOwn<S, V>];
template <int THREADS, int S, int V>
using JoinBuffer = float[3][THREADS * kOwn<S, V>];
// A vector as registers: 16 bytes, or a single element.
using Bits = unsigned __attribute__((ext_vector_type(4)));
template <int V>
using Held = std::conditional_t<V == 1, unsigned, Bits>;
template <class T, int V>
__device__ __forceinline__ Held<V> hold(const Raw<T, V> &r)
{
    Held<V> b{};
    __builtin_memcpy(&b, &r, sizeof(T) * V);
    return b;
}
// Held registers as a new value: what was computed from them before is computed again
// after this, and what is computed from them after is not begun before.  Without it the
// compiler unpacks all held vectors at once, or keeps them unpacked, and spills them.
template <class T, int V>
__device__ __forceinline__ Raw<T, V> held(Held<V> &b)
{
    asm volatile("" : "+v"(b));
    Raw<T, V> r;
    __builtin_memcpy(&r, &b, sizeof(T) * V);
    return r;
}

// Keeps the compiler from working on several tiles at a time, whose temporaries would not
// fit the registers; other waves fill the gaps.
__device__ __forceinline__ void one_by_one() { __builtin_amdgcn_sched_barrier(0); }

// What a thread's moments are relative to: the first value of each of its runs.  A first tile
// in which a run does not exist has none of it anywhere.
template <class T, int V, int S>
__device__ __forceinline__ void first_values(OwnFloats<S, V> &pivot, const Held<V> &b)
{
    Raw<T, V> r;
    __builtin_memcpy(&r, &b, sizeof(T) * V);
#pragma unroll
    for (int a = 0; a < V / S; ++a) pivot[a] = float(r[a * S]);
}

// The thread's moments over `tiles` tiles, updated tile by tile: get(i) is tile i's vector,
// valid(i) how much of it exists.  An element that exists in a tile exists in all tiles
// before, so the counts are known constants where the loop is unrolled.
template <class T, int V, int S, int UNROLL, class Get, class Valid>
__device__ __forceinline__ void own_moments(OwnMoments<S, V> &m, const OwnFloats<S, V> &pivot, int tiles, Get get, Valid valid)
{
    const float one = opaque_one();
#pragma unroll UNROLL
    for (int i = 0; i < tiles; ++i) {
        const int w = valid(i);
        const Raw<T, V> r = get(i);
        const float share = 1.0f / float(i + 1);
#pragma unroll
        for (int a = 0; a < V / S; ++a) {
            // the run's own moments (all of it exists or nothing), then joined
            float v[S], sum = 0.0f, m2 = 0.0f;
#pragma unroll
            for (int j = 0; j < S; ++j) {
                v[j] = minus(r[a * S + j], pivot[a], one);
                sum += v[j];
            }
            const float mean = sum * (1.0f / S), d = mean - m[a].mean;
            if (S > 1) {
#pragma unroll
                for (int j = 0; j < S; ++j) {
                    const float e = v[j] - mean;
                    m2 = __builtin_fmaf(e, e, m2);
                }
            }
            const bool in = a * S < w;
            m[a].n = in ? float(S * (i + 1)) : m[a].n;
            m[a].mean = in ? __builtin_fmaf(d, share, m[a].mean) : m[a].mean;
            m[a].m2 = in ? m[a].m2 + __builtin_fmaf(d * d, float(S * i) * share, m2) : m[a].m2;
        }
    }
}

// K tiles from `first` on as registers.
template <class T, int K, int V>
__device__ __forceinline__ void load_tiles(Held<V> (&raw)[K], const T *x, const Cut &k, const Place<V> &pl, int first)
{
    if (pl.full(k, first, K)) {
#pragma unroll
        for (int i = 0; i < K; ++i) raw[i] = hold<T, V>(*reinterpret_cast<const Raw<T, V> *>(x + pl.tile(k, first + i) + pl.off));
    } else {  // whole tiles, then at most one that ends inside, then none
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const T *const p = x + pl.tile(k, first + i) + pl.off;
            raw[i] = Held<V>{};
            if (pl.full(k, first + i, 1)) raw[i] = hold<T, V>(*reinterpret_cast<const Raw<T, V> *>(p));
            else if (first + i < k.tiles) raw[i] = hold<T, V>(load_first<T, V>(p, pl.valid(k, first + i)));
        }
    }
}

// ------------------------------------------------------------------------------------
// A call and its plan
// ------------------------------------------------------------------------------------
// A call of either direction (dy, dx, dgamma and dbeta: the gradient).
struct Call {
    int64_t N = 0;
    int dt = CT_FLOAT32;
    bool params_f32 = true;
    const void *x = nullptr, *dy = nullptr, *gamma = nullptr, *beta = nullptr;
    void *y = nullptr, *dx = nullptr, *dgamma = nullptr, *dbeta = nullptr;
    float eps = 0.0f;
    float *mean = nullptr, *rstd = nullptr;
    Act act;
    Dropout drop;
};

// Threads of a block and tiles held at once.  Statistics: 512 threads of 128 registers, 64 of
// which hold 16 vectors, so a compute unit has 256 KB of x on its way.  `one`: the kernels
// in which a block has all positions of its groups.
// Chunks of up to kStatShort tiles take a kernel that holds as many (its load, of tiles that are
// not there, and its arithmetic cost the longer one 19.2 against 15.5 us in an 8 x 256 x 2304
// float16 call, 14.4 against 12.2 in a 4 x 36 x 1001 float32 one).
constexpr int kStatThreads = 512, kStatTiles = 16, kStatShort = 4;
constexpr int kApplyThreads = 256, kApplyTiles = 4;
constexpr int kOneThreads = 512, kOneGradThreads = 256, kOneTiles = 4;
constexpr int kGradThreads = 256, kGradTiles = 4;
// Blocks that make dgamma and dbeta, 16 channels each.
inline int64_t param_blocks(int64_t C) { return (C + 15) / 16; }

struct Plan {
    bool vec = true;   // 16-byte vectors, else single elements
    int run = 1;       // consecutive elements of a vector that share a group: all, 4 or 1
    bool one = false;  // a block has all positions of its groups: one kernel
    int threads = 0;   // of its blocks: as many as a tile needs
    bool finish = false;  // many parts a group: a kernel joins them before the second pass
    Cut s, a;          // the pass for the statistics, the pass that writes (or the only one)
    // places in the workspace (bytes)
    size_t part = 0, stats = 0, sums = 0, bytes = 0;
};

void launch_forward(const Call &c, const Plan &p, char *ws, hipStream_t st);
void launch_gradient(const Call &c, const Plan &p, char *ws, hipStream_t st);
void launch_no_gradient(int dt, bool params_f32, int C, void *dgamma, void *dbeta, hipStream_t st);  // zeros

// Calls f(vector width, run) with the instance for the plan.
template <class T, class F>
void with_vector(const Plan &p, F &&f)
{
    constexpr int V = kVec<T>;
    if (!p.vec) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
    else if (p.run == V) f(std::integral_constant<int, V>{}, std::integral_constant<int, V>{});
    else if (p.run == 4) f(std::integral_constant<int, V>{}, std::integral_constant<int, 4>{});
    else f(std::integral_constant<int, V>{}, std::integral_constant<int, 1>{});
}

}  // namespace norm
}  // namespace ct

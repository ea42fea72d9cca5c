// ct_groupnorm.hpp -- what the group norm kernels share: moments, activations, the cut of
// the one-pass kernels and the exchange between their blocks.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ct_vec.hpp"

namespace ct {
namespace norm {

// (count, mean, sum of squared distances from the mean)
struct Moments {
    float n = 0.0f, mean = 0.0f, m2 = 0.0f;
    __device__ __forceinline__ void join(float bn, float bmean, float bm2)
    {
        const float total = n + bn;
        if (bn > 0.0f) {
            const float d = bmean - mean, w = bn / total;
            mean += d * w;
            m2 += bm2 + d * d * n * w;
            n = total;
        }
    }
};

// Activation and its derivative.  Kernels are compiled for SiLU, for none and for the
// piecewise linear kinds, which are told apart by selects: a switch inside a kernel made
// the compiler hoist the unpacking of every held value above it, into spilled registers.
struct Silu {
    __device__ __forceinline__ float y(float z) const { return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }
    __device__ __forceinline__ float d(float z) const
    {
        const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-z));
        return s * (1.0f + z * (1.0f - s));
    }
};
struct Identity {
    __device__ __forceinline__ float y(float z) const { return z; }
    __device__ __forceinline__ float d(float) const { return 1.0f; }
};
struct Piecewise {
    ct::Act a;
    __device__ __forceinline__ float y(float z) const { return a(z); }
    __device__ __forceinline__ float d(float z) const
    {
        const float relu = z > 0.0f ? 1.0f : 0.0f;
        const float leaky = z >= 0.0f ? 1.0f : a.p0;
        const float clip = z >= a.p0 && z <= a.p1 ? 1.0f : 0.0f;
        return a.kind == CT_ACT_RELU ? relu : a.kind == CT_ACT_LEAKY_RELU ? leaky : clip;
    }
};
template <class F>
void with_act(const ct::Act &a, F &&f)
{
    if (a.kind == CT_ACT_SILU) f(Silu{});
    else if (a.kind == CT_ACT_IDENTITY) f(Identity{});
    else f(Piecewise{a});
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
        *reinterpret_cast<Raw<T, V> *>(p) = r;
        return;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (j < valid) p[j] = r[j];
}

// ------------------------------------------------------------------------------------
// One pass: every value is read once and held in registers until it is written
// ------------------------------------------------------------------------------------
// A block holds `tiles` <= K tiles of a slab of whole groups.  When one block holds all
// positions of its groups (chunks == 1) it finishes alone.  Otherwise the blocks of an
// image exchange one 64-bit word per group and chunk: two float32 partials, stored and
// loaded as one relaxed device-scope atomic, so a word that is not kEmpty is complete and
// no fence or flag is needed.  The words are set to kEmpty by a kernel before.
//
// Waiting: a block waits only for blocks of its own image, which are launched next to it,
// and the host takes this path only when all blocks of an image fit the chip together.  The
// wait is bounded all the same: after `limit` looks a block computes what is missing
// itself, from memory, by the same operations (so the result is the same bits).  Every
// wait therefore ends whatever else runs on the device.
constexpr unsigned long long kEmpty = ~0ull;
// Threads of a block: two blocks share a compute unit, so a forward thread has 128 registers
// (64 of them hold 16 vectors) and a gradient thread 256 (128 hold 16 vectors of x and dy).
constexpr int kHeld = 512, kHeldGrad = 256;
constexpr int kMostGroups = 1024;  // groups of a slab


constexpr int kSmallHeld = 4;  // tiles held by the instances for short chunks
constexpr int held_tiles(bool uni, bool backward) { return uni || backward ? 16 : 8; }

struct OneCut {
    int64_t P;
    int C, G, Cg;
    int width, slabs, groups;  // channels and groups of a slab
    int rows, tiles;
    int chunks;
    int lanes;  // threads that share a group when partials are joined: a power of two
    int limit;
};

// A call of either direction (dy, dx and sums: the gradient).
struct Call {
    int dt = CT_FLOAT32;
    bool params_f32 = true;
    const void *x = nullptr, *dy = nullptr, *gamma = nullptr, *beta = nullptr;
    void *y = nullptr, *dx = nullptr;
    float eps = 0.0f;
    float *mean = nullptr, *rstd = nullptr;
    Act act;
    Dropout drop;
    unsigned long long *words = nullptr;
    float2 *sums = nullptr;
};

// The one-pass kernels over `blocks` blocks; uni: every 16-byte vector lies inside one group.
void launch_held(const Call &c, const OneCut &k, bool uni, int64_t blocks, hipStream_t st);
void launch_held_grad(const Call &c, const OneCut &k, bool uni, int64_t blocks, hipStream_t st);

__device__ __forceinline__ unsigned long long pack2(float a, float b)
{
    const unsigned long long w =
        (static_cast<unsigned long long>(__float_as_uint(b)) << 32) | static_cast<unsigned long long>(__float_as_uint(a));
    return w == kEmpty ? w - 1 : w;  // a pair of NaN of another payload
}
__device__ __forceinline__ void publish(unsigned long long *p, float a, float b)
{
    __hip_atomic_store(p, pack2(a, b), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned long long look(const unsigned long long *p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float low2(unsigned long long w) { return __uint_as_float(unsigned(w)); }
__device__ __forceinline__ float high2(unsigned long long w) { return __uint_as_float(unsigned(w >> 32)); }

// A block's place: image, chunk, slab, and the thread's vector within a tile.  An address is
// kept as a block-uniform tile offset (scalar registers) and the thread's 32-bit offset in
// the tile: 64-bit addresses of every tile would take the registers that hold the tiles.
template <int V>
struct HeldPlace {
    int64_t n;
    int chunk, slab, c0;
    int e, col;
    unsigned off;  // elements
    bool active;
    __device__ HeldPlace(const OneCut &k, int64_t b)
    {
        slab = int(b % k.slabs);
        b /= k.slabs;
        chunk = int(b % k.chunks);
        n = b / k.chunks;
        c0 = slab * k.width;
        e = int(threadIdx.x) * V;
        active = e < k.rows * k.width;
        if (!active) e = 0;
        const int row = e / k.width;
        col = e - row * k.width;
        off = unsigned(row) * unsigned(k.C) + unsigned(col);
    }
    // element offset of tile i of chunk q
    __device__ __forceinline__ int64_t tile(const OneCut &k, int q, int i) const
    {
        return (n * k.P + (int64_t(q) * k.tiles + i) * k.rows) * k.C + c0;
    }
    // how many of the V elements exist in tile i of chunk q
    __device__ __forceinline__ int valid(const OneCut &k, int q, int i) const
    {
        const int64_t left = k.P - (int64_t(q) * k.tiles + i) * k.rows;
        const int there = i >= k.tiles || left <= 0 ? 0 : int(left < k.rows ? left : k.rows) * k.width;
        const int mine = active ? there - e : 0;
        return mine >= V ? V : mine > 0 ? mine : 0;
    }
    // all tiles of chunk q hold all their positions
    __device__ __forceinline__ bool full(const OneCut &k, int q) const
    {
        return (int64_t(q) + 1) * k.tiles * k.rows <= k.P;
    }
};

// UNI: a vector lies inside one group, so the thread keeps one triple for all its values.
template <bool UNI, int V>
constexpr int kOwn = UNI ? 1 : V;

// 16 bytes of elements as registers.
using Bits = unsigned __attribute__((ext_vector_type(4)));
// Held registers as a new value: what was computed from them before is computed again
// after this, and what is computed from them after is not begun before.  Without it the
// compiler unpacks all held vectors at once, or keeps them unpacked, and spills them.
template <class T>
__device__ __forceinline__ Raw<T, ct::kVec<T>> held(Bits &b)
{
    asm volatile("" : "+v"(b));
    return __builtin_bit_cast(Raw<T, ct::kVec<T>>, b);
}

// Keeps the compiler from working on several tiles at a time, whose temporaries would not
// fit the registers; other waves fill the gaps.
__device__ __forceinline__ void one_by_one() { __builtin_amdgcn_sched_barrier(0); }

// Waits until every chunk's words of the block's groups are there.  use(g, complete word of
// chunk q, q) sees them in a fixed order per lane, after begin(g) and before end(g); what
// they made of an incomplete look is thrown away.  make(q) publishes chunk q from memory.
template <int THREADS, class Begin, class Use, class End, class Make>
__device__ __forceinline__ void gather_words(const OneCut &k, const unsigned long long *words, Begin begin, Use use, End end,
                                             Make make)
{
    const int lane = threadIdx.x & (k.lanes - 1);
    for (int looks = 0;; ++looks) {
        bool missing = false;
        for (int g = int(threadIdx.x) / k.lanes; g < k.groups; g += THREADS / k.lanes) {
            begin(g);
            for (int q = lane; q < k.chunks; q += k.lanes) {
                const unsigned long long w = look(words + int64_t(g) * k.chunks + q);
                missing |= w == kEmpty;
                use(g, w, q);
            }
            end(g, lane);
        }
        // (the second test is never met: the words made below are all there at the next look)
        if (!__syncthreads_or(missing) || looks > k.limit + 8) return;
        if (looks < k.limit) {
            __builtin_amdgcn_s_sleep(8);
            continue;
        }
        for (int q = 0; q < k.chunks; ++q) {
            bool gone = false;
            for (int g = threadIdx.x; g < k.groups; g += THREADS) gone |= look(words + int64_t(g) * k.chunks + q) == kEmpty;
            if (__syncthreads_or(gone)) make(q);
        }
        __threadfence();  // the words made here have arrived before anybody looks again
        __syncthreads();
    }
}

// Which elements of the thread's K vectors stay, V bits a vector, four vectors a word.  The
// words' loops are not unrolled further: sixteen copies of the generator are slower to fetch
// than to run.
template <int V, int K, class First>
__device__ __forceinline__ void draw(unsigned (&keep)[K / 4], const Dropout &drop, First first)
{
#pragma unroll
    for (int w = 0; w < K / 4; ++w) keep[w] = ~0u;
    if (!drop.threshold) return;
    const uint64_t counter = drop.counter();
#pragma unroll
    for (int w = 0; w < K / 4; ++w) {
        unsigned bits = 0;
#pragma unroll 1
        for (int i = 0; i < 4; ++i)
            bits |= (keep_bits<V>(drop, counter, uint64_t(first(4 * w + i))) & ((1u << V) - 1)) << (8 * i);
        keep[w] = bits;
    }
}
__device__ __forceinline__ bool stays(const unsigned *keep, int i, int j) { return (keep[i / 4] >> (8 * (i % 4) + j)) & 1; }

// Calls launch(vector inside a group?, tiles held) with the instance for the cut.
template <bool BACKWARD, class F>
void with_instance(const OneCut &k, bool uni, F &&launch)
{
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    if (uni && k.tiles <= kSmallHeld) launch(yes, std::integral_constant<int, kSmallHeld>{});
    else if (uni) launch(yes, std::integral_constant<int, held_tiles(true, BACKWARD)>{});
    else if (k.tiles <= kSmallHeld) launch(no, std::integral_constant<int, kSmallHeld>{});
    else launch(no, std::integral_constant<int, held_tiles(false, BACKWARD)>{});
}

}  // namespace norm
}  // namespace ct

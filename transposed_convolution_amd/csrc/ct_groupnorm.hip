// ct_groupnorm.hip -- group norm with an activation and dropout, channels-last, and its
// gradient.
//
// x is stored (N, P, C), P the product of the spatial axes; group g holds the C/G channels
// g*C/G .. and all P positions of an image.
//   mean = average of x over the group, rstd = 1 / sqrt(average of (x - mean)^2 + eps)
//   y = drop(act((x - mean) * rstd * gamma[c] + beta[c]))
// Gradient, with xhat = (x - mean) rstd, z = xhat gamma + beta, dz = drop(dy) act'(z):
//   dbeta[c] = sum dz,  dgamma[c] = sum dz xhat            (over images and positions)
//   c1 = average of dz gamma over the group, c2 = average of dz gamma xhat
//   dx = rstd (dz gamma - c1 - xhat c2)
//
// Statistics: a thread takes the mean and the sum of squared distances from it of the
// values it holds, and such triples (count, mean, m2) are joined pairwise (Chan, Golub,
// LeVeque 1983).  The values are first taken relative to the group's first one, so a mean
// far from zero costs no digits of the spread around it.
// Everything is float32 between the one load and the one store of an element.
//
// Both directions need every value of a group before the first output: a pass that reads
// for the statistics and one that reads again and writes.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <numeric>
#include <string>
#include <type_traits>

#include "ct_vec.hpp"

namespace {

using ct::Dropout;
using ct::Raw;

constexpr int kThreads = 256;
constexpr int kTiles = 8;          // tiles of a thread in flight at once

// A launch's cut of (N, P, C): slabs of `width` channels (the last may be narrower) and
// chunks of `tiles` tiles of `rows` positions.  A thread owns the V consecutive elements
// at e = V * thread of every tile (a tile's elements run through its rows), so its
// channels are the same in all of them.  One slab holding all channels may have any width:
// its tile is contiguous and a vector may run over a row's end.
struct Cut {
    int64_t P;
    int C, G, Cg;
    int width, slabs;
    int rows;
    int64_t tiles_per_chunk, chunks;
    int parts;  // slabs one group may touch
};

struct Block {
    int64_t n, chunk;
    int slab, c0, width;  // first channel, channels
    __device__ explicit Block(const Cut &k, int64_t b)
    {
        slab = int(b % k.slabs);
        b /= k.slabs;
        chunk = b % k.chunks;
        n = b / k.chunks;
        c0 = slab * k.width;
        width = k.C - c0 < k.width ? k.C - c0 : k.width;
    }
};

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

// Activation and its derivative, one instance of f per kind.
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
struct Relu {
    __device__ __forceinline__ float y(float z) const { return z > 0.0f ? z : 0.0f; }
    __device__ __forceinline__ float d(float z) const { return z > 0.0f ? 1.0f : 0.0f; }
};
struct Leaky {
    float slope;
    __device__ __forceinline__ float y(float z) const { return z >= 0.0f ? z : slope * z; }
    __device__ __forceinline__ float d(float z) const { return z >= 0.0f ? 1.0f : slope; }
};
struct Clip {
    float lo, hi;
    __device__ __forceinline__ float y(float z) const { return z < lo ? lo : (z > hi ? hi : z); }
    __device__ __forceinline__ float d(float z) const { return z >= lo && z <= hi ? 1.0f : 0.0f; }
};
template <class F>
__device__ __forceinline__ void with_act(const ct::Act &a, F &&f)
{
    switch (a.kind) {
    case CT_ACT_RELU: f(Relu{}); break;
    case CT_ACT_LEAKY_RELU: f(Leaky{a.p0}); break;
    case CT_ACT_CLIP: f(Clip{a.p0, a.p1}); break;
    case CT_ACT_SILU: f(Silu{}); break;
    default: f(Identity{}); break;
    }
}

// A thread's place in its block's tiles.
template <int V>
struct Place {
    int e, row, col;
    bool active;
    int64_t at;  // element offset of tile 0 in the image
    __device__ Place(const Cut &k, const Block &b)
    {
        e = int(threadIdx.x) * V;
        active = e < k.rows * b.width;
        if (!active) e = 0;
        row = e / b.width;
        col = e - row * b.width;
        at = (b.chunk * k.tiles_per_chunk * k.rows + row) * k.C + b.c0 + col;
    }
};

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

// How many of the thread's V elements of the tile at position p0 exist.
template <int V>
__device__ __forceinline__ int valid_of(const Cut &k, const Block &b, const Place<V> &pl, int64_t p0)
{
    if (!pl.active) return 0;
    const int64_t left = (k.P - p0 < k.rows ? k.P - p0 : int64_t(k.rows)) * b.width - pl.e;
    return left >= V ? V : left > 0 ? int(left) : 0;
}

// ------------------------------------------------------------------------------------
// Forward
// ------------------------------------------------------------------------------------
// What a group's moments are relative to: its first value.
template <class T>
__device__ __forceinline__ float pivot_of(const T *x, const Cut &k, int64_t n, int g)
{
    return float(x[n * k.P * k.C + int64_t(g) * k.Cg]);
}

// The moments of every (chunk, slab) part of every group.
template <class T, int V>
__global__ __launch_bounds__(kThreads) void stats_kernel(const T *x, Cut k, float *part)
{
    __shared__ float lds[3][kThreads * V];
    const Block b(k, blockIdx.x);
    const Place<V> pl(k, b);
    const T *src = x + b.n * k.P * k.C + pl.at;
    const int64_t step = int64_t(k.rows) * k.C;
    float pivot[V];
#pragma unroll
    for (int j = 0; j < V; ++j) pivot[j] = pivot_of(x, k, b.n, (b.c0 + (pl.col + j) % b.width) / k.Cg);
    Moments m[V];
    int64_t p0 = b.chunk * k.tiles_per_chunk * k.rows;
    for (int64_t t = 0; t < k.tiles_per_chunk && p0 < k.P; t += kTiles) {
        Raw<T, V> raw[kTiles];
        int valid[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            valid[i] = t + i < k.tiles_per_chunk ? valid_of(k, b, pl, p0 + int64_t(i) * k.rows) : 0;
            raw[i] = load_first<T, V>(src + i * step, valid[i]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float n = 0.0f, sum = 0.0f, m2 = 0.0f;
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                n += j < valid[i] ? 1.0f : 0.0f;
                sum += j < valid[i] ? float(raw[i][j]) - pivot[j] : 0.0f;
            }
            const float mean = n > 0.0f ? sum / n : 0.0f;
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                const float d = j < valid[i] ? float(raw[i][j]) - pivot[j] - mean : 0.0f;
                m2 += d * d;
            }
            m[j].join(n, mean, m2);
        }
        p0 += int64_t(kTiles) * k.rows;
        src += kTiles * step;
    }
    if (pl.active) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            lds[0][pl.e + j] = m[j].n;
            lds[1][pl.e + j] = m[j].mean;
            lds[2][pl.e + j] = m[j].m2;
        }
    }
    __syncthreads();
    // a wave joins the entries of one group: its columns in every row
    const int g0 = b.c0 / k.Cg, g1 = (b.c0 + b.width - 1) / k.Cg;
    const int lane = threadIdx.x & 63;
    for (int g = g0 + int(threadIdx.x) / 64; g <= g1; g += kThreads / 64) {
        const int lo = g * k.Cg > b.c0 ? g * k.Cg - b.c0 : 0;
        const int hi = (g + 1) * k.Cg < b.c0 + b.width ? (g + 1) * k.Cg - b.c0 : b.width;
        const int w = hi - lo;
        Moments s;
        for (int i = lane; i < w * k.rows; i += 64) {
            const int r = i / w, at = r * b.width + lo + (i - r * w);
            s.join(lds[0][at], lds[1][at], lds[2][at]);
        }
        for (int o = 1; o < 64; o *= 2) s.join(__shfl_xor(s.n, o), __shfl_xor(s.mean, o), __shfl_xor(s.m2, o));
        if (lane == 0) {
            const int first_slab = int((int64_t(g) * k.Cg) / k.width);
            float *out = part + (((b.n * k.G + g) * k.chunks + b.chunk) * k.parts + (b.slab - first_slab)) * 3;
            out[0] = s.n;
            out[1] = s.mean;
            out[2] = s.m2;
        }
    }
}

// Joins the parts of a group: one wave a group.
template <class T>
__global__ __launch_bounds__(kThreads) void finish_kernel(const T *x, const float *part, Cut k, int64_t groups, float eps,
                                                          float *mean, float *rstd)
{
    const int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / 64;
    const int lane = threadIdx.x & 63;
    if (i >= groups) return;
    const int g = int(i % k.G);
    const int64_t first = (int64_t(g) * k.Cg) / k.width, last = (int64_t(g + 1) * k.Cg - 1) / k.width;
    const int64_t own = last - first + 1, count = k.chunks * own;
    Moments s;
    for (int64_t q = lane; q < count; q += 64) {
        const float *p = part + ((i * k.chunks + q / own) * k.parts + q % own) * 3;
        s.join(p[0], p[1], p[2]);
    }
    for (int o = 1; o < 64; o *= 2) s.join(__shfl_xor(s.n, o), __shfl_xor(s.mean, o), __shfl_xor(s.m2, o));
    if (lane == 0) {
        mean[i] = pivot_of(x, k, i / k.G, g) + s.mean;
        rstd[i] = 1.0f / sqrtf(s.m2 / s.n + eps);
    }
}

template <class T, int V>
__global__ __launch_bounds__(kThreads) void apply_kernel(const T *x, Cut k, const float *mean, const float *rstd,
                                                         ct::Param<T> gamma, ct::Param<T> beta, ct::Act act, Dropout drop,
                                                         T *y)
{
    const Block b(k, blockIdx.x);
    const Place<V> pl(k, b);
    float mu[V], a[V], sh[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = b.c0 + (pl.col + j) % b.width;
        const int64_t i = b.n * k.G + c / k.Cg;
        mu[j] = mean[i];
        a[j] = rstd[i] * gamma.at(c, 1.0f);
        sh[j] = beta.at(c, 0.0f);
    }
    const int64_t image = b.n * k.P * k.C + pl.at;
    const int64_t step = int64_t(k.rows) * k.C;
    const uint64_t counter = drop.threshold ? drop.counter() : 0;
    with_act(act, [&](auto f) {
        int64_t p0 = b.chunk * k.tiles_per_chunk * k.rows, at = image;
        for (int64_t t = 0; t < k.tiles_per_chunk && p0 < k.P; ++t, p0 += k.rows, at += step) {
            const int valid = valid_of(k, b, pl, p0);
            if (valid == 0) continue;
            const Raw<T, V> v = load_first<T, V>(x + at, valid);
            const unsigned keep = drop.threshold ? ct::keep_bits<V>(drop, counter, uint64_t(at)) : 0xffu;
            Raw<T, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float r = f.y((float(v[j]) - mu[j]) * a[j] + sh[j]);
                o[j] = T((keep >> j) & 1 ? r * drop.factor : 0.0f);
            }
            store_first<T, V>(y + at, o, valid);
        }
    });
}

// ------------------------------------------------------------------------------------
// Gradient
// ------------------------------------------------------------------------------------
// Per thread: the constants of its V channels.
template <class T, int V>
struct Channels {
    float mu[V], rs[V], ga[V], be[V];
    __device__ Channels(const Cut &k, const Block &b, int col, const float *mean, const float *rstd, const ct::Param<T> &gamma,
                        const ct::Param<T> &beta)
    {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = b.c0 + (col + j) % b.width;
            const int64_t i = b.n * k.G + c / k.Cg;
            mu[j] = mean[i];
            rs[j] = rstd[i];
            ga[j] = gamma.at(c, 1.0f);
            be[j] = beta.at(c, 0.0f);
        }
    }
};

// sums[n][chunk][c] = (sum dz, sum dz xhat) over the chunk's positions.
template <class T, int V>
__global__ __launch_bounds__(kThreads) void grad_stats_kernel(const T *dy, const T *x, Cut k, const float *mean,
                                                              const float *rstd, ct::Param<T> gamma, ct::Param<T> beta,
                                                              ct::Act act, Dropout drop, float2 *sums)
{
    __shared__ float2 lds[kThreads * V];
    const Block b(k, blockIdx.x);
    const Place<V> pl(k, b);
    const Channels<T, V> ch(k, b, pl.col, mean, rstd, gamma, beta);
    const int64_t image = b.n * k.P * k.C + pl.at;
    const int64_t step = int64_t(k.rows) * k.C;
    const uint64_t counter = drop.threshold ? drop.counter() : 0;
    float s1[V] = {}, s2[V] = {};
    with_act(act, [&](auto f) {
        int64_t p0 = b.chunk * k.tiles_per_chunk * k.rows, at = image;
        for (int64_t t = 0; t < k.tiles_per_chunk && p0 < k.P; ++t, p0 += k.rows, at += step) {
            const int valid = valid_of(k, b, pl, p0);
            if (valid == 0) continue;
            const Raw<T, V> xv = load_first<T, V>(x + at, valid), dv = load_first<T, V>(dy + at, valid);
            const unsigned keep = drop.threshold ? ct::keep_bits<V>(drop, counter, uint64_t(at)) : 0xffu;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = (float(xv[j]) - ch.mu[j]) * ch.rs[j];
                const float e = (keep >> j) & 1 ? float(dv[j]) * drop.factor : 0.0f;
                const float dz = e * f.d(xh * ch.ga[j] + ch.be[j]);
                s1[j] += j < valid ? dz : 0.0f;
                s2[j] += j < valid ? dz * xh : 0.0f;
            }
        }
    });
    if (pl.active)
        for (int j = 0; j < V; ++j) lds[pl.e + j] = make_float2(s1[j], s2[j]);
    __syncthreads();
    for (int c = threadIdx.x; c < b.width; c += kThreads) {
        float2 s = make_float2(0.0f, 0.0f);
        for (int r = 0; r < k.rows; ++r) {
            const float2 v = lds[r * b.width + c];
            s.x += v.x;
            s.y += v.y;
        }
        sums[(b.n * k.chunks + b.chunk) * k.C + b.c0 + c] = s;
    }
}

// total[n][c] = the chunks' sums, joined; 16 threads a channel.
constexpr int kJoin = 16;
__global__ __launch_bounds__(1024) void grad_join_kernel(const float2 *sums, Cut k, float2 *total)
{
    __shared__ float2 lds[kJoin][64];
    const int tiles = (k.C + 63) / 64;
    const int64_t n = blockIdx.x / tiles;
    const int c = int(blockIdx.x % tiles) * 64 + (threadIdx.x & 63), q = threadIdx.x / 64;
    float2 s = make_float2(0.0f, 0.0f);
    if (c < k.C)
        for (int64_t i = q; i < k.chunks; i += kJoin) {
            const float2 v = sums[(n * k.chunks + i) * k.C + c];
            s.x += v.x;
            s.y += v.y;
        }
    lds[q][threadIdx.x & 63] = s;
    __syncthreads();
    if (q == 0 && c < k.C) {
        for (int i = 1; i < kJoin; ++i) {
            s.x += lds[i][threadIdx.x].x;
            s.y += lds[i][threadIdx.x].y;
        }
        total[n * k.C + c] = s;
    }
}

// dgamma and dbeta: the images' sums, in their order.
template <class T>
__global__ __launch_bounds__(kThreads) void param_grad_kernel(const float2 *total, int64_t N, int C, bool f32, void *dgamma,
                                                              void *dbeta)
{
    const int c = int(blockIdx.x) * kThreads + threadIdx.x;
    if (c >= C) return;
    float2 s = make_float2(0.0f, 0.0f);
    for (int64_t n = 0; n < N; ++n) {
        const float2 v = total[n * C + c];
        s.x += v.x;
        s.y += v.y;
    }
    if (dgamma) {
        if (f32) static_cast<float *>(dgamma)[c] = s.y;
        else static_cast<T *>(dgamma)[c] = T(s.y);
    }
    if (dbeta) {
        if (f32) static_cast<float *>(dbeta)[c] = s.x;
        else static_cast<T *>(dbeta)[c] = T(s.x);
    }
}

// c1 and c2 of every group, from the channels' sums: one wave a group.
template <class T>
__global__ __launch_bounds__(kThreads) void grad_groups_kernel(const float2 *total, Cut k, int64_t groups,
                                                               ct::Param<T> gamma, float2 *coef)
{
    const int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / 64;
    const int lane = threadIdx.x & 63;
    if (i >= groups) return;
    const int64_t n = i / k.G;
    const int g = int(i % k.G);
    float a = 0.0f, b = 0.0f;
    for (int j = lane; j < k.Cg; j += 64) {
        const int c = g * k.Cg + j;
        const float2 v = total[n * k.C + c];
        const float ga = gamma.at(c, 1.0f);
        a += v.x * ga;
        b += v.y * ga;
    }
    for (int o = 1; o < 64; o *= 2) {
        a += __shfl_xor(a, o);
        b += __shfl_xor(b, o);
    }
    const float count = float(k.P) * float(k.Cg);
    if (lane == 0) coef[i] = make_float2(a / count, b / count);
}

template <class T, int V>
__global__ __launch_bounds__(kThreads) void grad_apply_kernel(const T *dy, const T *x, Cut k, const float *mean,
                                                              const float *rstd, ct::Param<T> gamma, ct::Param<T> beta,
                                                              ct::Act act, Dropout drop, const float2 *coef, T *dx)
{
    const Block b(k, blockIdx.x);
    const Place<V> pl(k, b);
    const Channels<T, V> ch(k, b, pl.col, mean, rstd, gamma, beta);
    float c1[V], c2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float2 v = coef[b.n * k.G + (b.c0 + (pl.col + j) % b.width) / k.Cg];
        c1[j] = v.x;
        c2[j] = v.y;
    }
    const int64_t image = b.n * k.P * k.C + pl.at;
    const int64_t step = int64_t(k.rows) * k.C;
    const uint64_t counter = drop.threshold ? drop.counter() : 0;
    with_act(act, [&](auto f) {
        int64_t p0 = b.chunk * k.tiles_per_chunk * k.rows, at = image;
        for (int64_t t = 0; t < k.tiles_per_chunk && p0 < k.P; ++t, p0 += k.rows, at += step) {
            const int valid = valid_of(k, b, pl, p0);
            if (valid == 0) continue;
            const Raw<T, V> xv = load_first<T, V>(x + at, valid), dv = load_first<T, V>(dy + at, valid);
            const unsigned keep = drop.threshold ? ct::keep_bits<V>(drop, counter, uint64_t(at)) : 0xffu;
            Raw<T, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = (float(xv[j]) - ch.mu[j]) * ch.rs[j];
                const float e = (keep >> j) & 1 ? float(dv[j]) * drop.factor : 0.0f;
                const float dz = e * f.d(xh * ch.ga[j] + ch.be[j]);
                o[j] = T(ch.rs[j] * (dz * ch.ga[j] - c1[j] - xh * c2[j]));
            }
            store_first<T, V>(dx + at, o, valid);
        }
    });
}

// ------------------------------------------------------------------------------------
// Host
// ------------------------------------------------------------------------------------
// Vector width 1 serves the channel counts that no short tile of whole vectors fits (odd
// counts above 256): V = 1 and slabs of 256 channels.
template <int V>
bool make_cut(int64_t N, int64_t P, int64_t C, int64_t G, Cut *k)
{
    k->P = P;
    k->C = int(C);
    k->G = int(G);
    k->Cg = int(C / G);
    const int64_t unit = V / std::gcd(C, int64_t(V));  // rows after which a vector starts a row again
    if (unit * C <= int64_t(kThreads) * V) {
        k->width = int(C);
    } else {
        if (C % V) return false;
        k->width = kThreads * V;
    }
    k->slabs = int((C + k->width - 1) / k->width);
    const int64_t fit = int64_t(kThreads) * V / k->width / unit * unit;
    const int64_t need = (P + unit - 1) / unit * unit;
    k->rows = int(fit < need ? fit : need);
    const int64_t tiles = (P + k->rows - 1) / k->rows;
    // eight tiles a block, and no more than about 2048 blocks in all
    int64_t chunks = (tiles + kTiles - 1) / kTiles;
    const int64_t most_chunks = std::max<int64_t>(1, 2048 / std::max<int64_t>(1, N * k->slabs));
    if (chunks > most_chunks) chunks = most_chunks;
    k->tiles_per_chunk = (tiles + chunks - 1) / chunks;
    k->chunks = (tiles + k->tiles_per_chunk - 1) / k->tiles_per_chunk;
    k->parts = k->slabs == 1 ? 1 : int((k->Cg - 1) / k->width) + 2;
    return true;
}

struct Sizes {
    int64_t N = 0, C = 0, P = 1, G = 1;
    int dt = CT_FLOAT32;
    bool empty() const { return N == 0 || C == 0 || P == 0; }
};

struct Plan {
    bool vec = true;
    Cut k;
    size_t part = 0, stats = 0, total = 0, coef = 0, bytes = 0;
};

Plan make_plan(const Sizes &s, bool backward)
{
    Plan p;
    if (s.empty()) return p;
    p.vec = s.dt == CT_FLOAT32 ? make_cut<4>(s.N, s.P, s.C, s.G, &p.k) : make_cut<8>(s.N, s.P, s.C, s.G, &p.k);
    if (!p.vec) make_cut<1>(s.N, s.P, s.C, s.G, &p.k);
    size_t at = 0;
    auto place = [&](size_t bytes) {
        const size_t q = at;
        at += (bytes + 255) & ~size_t(255);
        return q;
    };
    if (backward) {
        p.part = place(size_t(s.N) * p.k.chunks * s.C * 8);
        p.total = place(size_t(s.N) * s.C * 8);
        p.coef = place(size_t(s.N) * s.G * 8);
    } else {
        p.part = place(size_t(s.N) * s.G * p.k.chunks * p.k.parts * 12);
        p.stats = place(size_t(s.N) * s.G * 8);
    }
    p.bytes = at;
    return p;
}

ct_status fail(ct_status st, const std::string &msg)
{
    ct::set_last_error(msg);
    return st;
}

ct_status check_sizes(int dt, int nsp, const int64_t *shape, int64_t groups, Sizes *s)
{
    if (!ct::is_float_type(dt)) return fail(CT_EUNSUPPORTED, "dtype must be CT_FLOAT32, CT_FLOAT16 or CT_BFLOAT16");
    if (nsp < 1 || nsp > 3) return fail(CT_EINVAL, "the spatial rank must be 1, 2 or 3");
    if (!shape) return fail(CT_EINVAL, "x_shape is NULL");
    for (int a = 0; a < nsp + 2; ++a)
        if (shape[a] < 0) return fail(CT_EINVAL, "sizes must not be negative");
    s->dt = dt;
    s->N = shape[0];
    s->C = shape[1];
    s->G = groups;
    int64_t total = 1;
    for (int a = 0; a < nsp + 2; ++a) {
        if (shape[a] > 0 && total > (int64_t(1) << 58) / shape[a]) return fail(CT_EUNSUPPORTED, "more than 2^58 elements");
        total *= shape[a] > 0 ? shape[a] : 1;
    }
    for (int a = 0; a < nsp; ++a) s->P *= shape[2 + a];
    if (groups < 1 || s->C % groups != 0) return fail(CT_EINVAL, "groups must be at least 1 and divide the channels");
    // a launch holds fewer than 2^32 threads; the smallest work item of a channel tile is a
    // block of 1024 and that of a group a wave
    const int64_t tiles = s->C / 64 + 1;
    if (s->C > (1 << 30) || s->N > (int64_t(1) << 21) / tiles || (s->N > 0 && groups > (int64_t(1) << 25) / s->N))
        return fail(CT_EUNSUPPORTED, "more than 2^21 images times tiles of 64 channels, or 2^25 images times groups");
    return CT_OK;
}

ct_status check_act(int kind, float p0, float p1, ct::Act *act)
{
    act->kind = kind;
    act->p0 = p0;
    act->p1 = p1;
    switch (kind) {
    case CT_ACT_IDENTITY:
    case CT_ACT_RELU:
    case CT_ACT_SILU: return CT_OK;
    case CT_ACT_LEAKY_RELU:
        return std::isfinite(p0) ? CT_OK : fail(CT_EINVAL, "leaky ReLU slope must be finite");
    case CT_ACT_CLIP:
        return std::isfinite(p0) && std::isfinite(p1) && p0 <= p1
                   ? CT_OK
                   : fail(CT_EINVAL, "clip bounds must be finite with lower <= upper");
    default: return fail(CT_EINVAL, "unknown activation");
    }
}

ct_status check_params(int dt, int pt, const void *gamma, const void *beta)
{
    if (pt != dt && pt != CT_FLOAT32) return fail(CT_EUNSUPPORTED, "param_dtype must be dtype or CT_FLOAT32");
    if (!ct::aligned_to(gamma, ct::float_size(pt)) || !ct::aligned_to(beta, ct::float_size(pt)))
        return fail(CT_EINVAL, "gamma and beta must be aligned to their element size");
    return CT_OK;
}

unsigned blocks_of(int64_t items, int64_t per) { return unsigned((items + per - 1) / per); }

}  // namespace

extern "C" {

ct_status group_norm_workspace_size(ct_dtype dtype, int nsp, const int64_t *x_shape, int64_t groups, int backward,
                                    size_t *bytes_out)
{
    ct::set_last_error(std::string());
    if (!bytes_out) return fail(CT_EINVAL, "bytes_out is NULL");
    if (backward != 0 && backward != 1) return fail(CT_EINVAL, "backward must be 0 or 1");
    Sizes s;
    const ct_status st = check_sizes(ct::enum_int(dtype), nsp, x_shape, groups, &s);
    if (st != CT_OK) return st;
    *bytes_out = make_plan(s, backward != 0).bytes;
    return CT_OK;
}

ct_status group_norm_nd(ct_dtype dtype, int nsp, const void *x, const int64_t *x_shape, int64_t groups,
                        ct_dtype param_dtype, const void *gamma, const void *beta, float eps, ct_activation activation,
                        float act_p0, float act_p1, double dropout_p, uint64_t seed, uint64_t offset,
                        const uint64_t *step, void *y, float *mean, float *rstd, void *workspace, size_t workspace_bytes,
                        void *stream)
{
    ct::set_last_error(std::string());
    const int dt = ct::enum_int(dtype), pt = ct::enum_int(param_dtype);
    Sizes s;
    ct::Act act;
    Dropout drop;
    std::string err;
    ct_status st = check_sizes(dt, nsp, x_shape, groups, &s);
    if (st == CT_OK) st = check_params(dt, pt, gamma, beta);
    if (st == CT_OK) st = check_act(ct::enum_int(activation), act_p0, act_p1, &act);
    if (st != CT_OK) return st;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(CT_EINVAL, "eps must be finite and not negative");
    st = ct::make_dropout(dropout_p, seed, offset, step, &drop, &err);
    if (st != CT_OK) return fail(st, err);
    const size_t esz = ct::float_size(dt);
    if (!ct::aligned_to(x, esz) || !ct::aligned_to(y, esz) || !ct::aligned_to(mean, 4) || !ct::aligned_to(rstd, 4))
        return fail(CT_EINVAL, "tensor pointers must be aligned to the element size");
    if (workspace && !ct::aligned_to(workspace, 16)) return fail(CT_EINVAL, "workspace must be 16-byte aligned");
    if (s.empty()) return CT_OK;
    if (!x || !y) return fail(CT_EINVAL, "x or y is NULL");
    const Plan p = make_plan(s, false);
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    ct::Scratch ws;
    st = ws.take(workspace, workspace_bytes, p.bytes, hs, &err);
    if (st != CT_OK) return fail(st, err);
    char *const base = static_cast<char *>(ws.p);
    float *const part = reinterpret_cast<float *>(base + p.part);
    if (!mean) mean = reinterpret_cast<float *>(base + p.stats);
    if (!rstd) rstd = reinterpret_cast<float *>(base + p.stats) + s.N * s.G;
    const int64_t blocks = s.N * p.k.chunks * p.k.slabs;
    ct::with_type(dt, [&](auto t) {
        using T = decltype(t);
        const T *xp = static_cast<const T *>(x);
        const ct::Param<T> ga{gamma, pt == CT_FLOAT32}, be{beta, pt == CT_FLOAT32};
        auto go = [&](auto v) {
            constexpr int V = decltype(v)::value;
            stats_kernel<T, V><<<unsigned(blocks), kThreads, 0, hs>>>(xp, p.k, part);
            finish_kernel<T><<<blocks_of(s.N * s.G, kThreads / 64), kThreads, 0, hs>>>(xp, part, p.k, s.N * s.G, eps, mean, rstd);
            ct::mark_before(hs);
            apply_kernel<T, V><<<unsigned(blocks), kThreads, 0, hs>>>(xp, p.k, mean, rstd, ga, be, act, drop,
                                                                     static_cast<T *>(y));
            ct::mark_after(hs);
        };
        if (p.vec) go(std::integral_constant<int, ct::kVec<T>>{});
        else go(std::integral_constant<int, 1>{});
    });
    st = ct::launch_status("group norm launch failed", &err);
    return st == CT_OK ? CT_OK : fail(st, err);
}

ct_status group_norm_backward_nd(ct_dtype dtype, int nsp, const void *dy, const void *x, const int64_t *x_shape,
                                 int64_t groups, const float *mean, const float *rstd, ct_dtype param_dtype,
                                 const void *gamma, const void *beta, ct_activation activation, float act_p0,
                                 float act_p1, double dropout_p, uint64_t seed, uint64_t offset, const uint64_t *step,
                                 void *dx, void *dgamma, void *dbeta, void *workspace, size_t workspace_bytes,
                                 void *stream)
{
    ct::set_last_error(std::string());
    const int dt = ct::enum_int(dtype), pt = ct::enum_int(param_dtype);
    Sizes s;
    ct::Act act;
    Dropout drop;
    std::string err;
    ct_status st = check_sizes(dt, nsp, x_shape, groups, &s);
    if (st == CT_OK) st = check_params(dt, pt, gamma, beta);
    if (st == CT_OK) st = check_params(dt, pt, dgamma, dbeta);
    if (st == CT_OK) st = check_act(ct::enum_int(activation), act_p0, act_p1, &act);
    if (st != CT_OK) return st;
    st = ct::make_dropout(dropout_p, seed, offset, step, &drop, &err);
    if (st != CT_OK) return fail(st, err);
    const size_t esz = ct::float_size(dt);
    if (!ct::aligned_to(x, esz) || !ct::aligned_to(dy, esz) || !ct::aligned_to(dx, esz) || !ct::aligned_to(mean, 4) ||
        !ct::aligned_to(rstd, 4))
        return fail(CT_EINVAL, "tensor pointers must be aligned to the element size");
    if (workspace && !ct::aligned_to(workspace, 16)) return fail(CT_EINVAL, "workspace must be 16-byte aligned");
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    if (s.C == 0) return CT_OK;
    if (!s.empty() && (!x || !dy || !dx || !mean || !rstd)) return fail(CT_EINVAL, "x, dy, dx, mean or rstd is NULL");
    const Plan p = make_plan(s, true);
    ct::Scratch ws;
    st = ws.take(workspace, workspace_bytes, p.bytes, hs, &err);
    if (st != CT_OK) return fail(st, err);
    char *const base = static_cast<char *>(ws.p);
    float2 *const part = reinterpret_cast<float2 *>(base + p.part);
    float2 *const total = reinterpret_cast<float2 *>(base + p.total);
    float2 *const coef = reinterpret_cast<float2 *>(base + p.coef);
    const int64_t blocks = s.empty() ? 0 : s.N * p.k.chunks * p.k.slabs;
    ct::with_type(dt, [&](auto t) {
        using T = decltype(t);
        const T *xp = static_cast<const T *>(x), *dp = static_cast<const T *>(dy);
        const ct::Param<T> ga{gamma, pt == CT_FLOAT32}, be{beta, pt == CT_FLOAT32};
        auto go = [&](auto v) {
            constexpr int V = decltype(v)::value;
            grad_stats_kernel<T, V><<<unsigned(blocks), kThreads, 0, hs>>>(dp, xp, p.k, mean, rstd, ga, be, act, drop, part);
            grad_join_kernel<<<unsigned(s.N * blocks_of(s.C, 64)), 1024, 0, hs>>>(part, p.k, total);
            grad_groups_kernel<T><<<blocks_of(s.N * s.G, kThreads / 64), kThreads, 0, hs>>>(total, p.k, s.N * s.G, ga, coef);
            ct::mark_before(hs);
            grad_apply_kernel<T, V><<<unsigned(blocks), kThreads, 0, hs>>>(dp, xp, p.k, mean, rstd, ga, be, act, drop, coef,
                                                                          static_cast<T *>(dx));
            ct::mark_after(hs);
        };
        if (!s.empty()) {
            if (p.vec) go(std::integral_constant<int, ct::kVec<T>>{});
            else go(std::integral_constant<int, 1>{});
        }
        if (dgamma || dbeta)
            param_grad_kernel<T><<<blocks_of(s.C, kThreads), kThreads, 0, hs>>>(total, s.empty() ? 0 : s.N, int(s.C),
                                                                               pt == CT_FLOAT32, dgamma, dbeta);
    });
    st = ct::launch_status("group norm gradient launch failed", &err);
    return st == CT_OK ? CT_OK : fail(st, err);
}

}  // extern "C"

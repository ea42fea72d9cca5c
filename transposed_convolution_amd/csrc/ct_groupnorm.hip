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
// Both directions need every value of a group before the first output.  Where an image fits
// the chip's registers it is read once and held there (ct_groupnorm.hpp); here are the
// kernels for the others: a pass that reads for the statistics and one that reads again and
// writes; and the entry points.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <numeric>
#include <string>
#include <type_traits>

#include "ct_groupnorm.hpp"

namespace {

using namespace ct::norm;
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

template <class T, int V, class ACT>
__global__ __launch_bounds__(kThreads) void apply_kernel(const T *x, Cut k, const float *mean, const float *rstd,
                                                         ct::Param<T> gamma, ct::Param<T> beta, ACT f, Dropout drop,
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
template <class T, int V, class ACT>
__global__ __launch_bounds__(kThreads) void grad_stats_kernel(const T *dy, const T *x, Cut k, const float *mean,
                                                              const float *rstd, ct::Param<T> gamma, ct::Param<T> beta,
                                                              ACT f, Dropout drop, float2 *sums)
{
    __shared__ float2 lds[kThreads * V];
    const Block b(k, blockIdx.x);
    const Place<V> pl(k, b);
    const Channels<T, V> ch(k, b, pl.col, mean, rstd, gamma, beta);
    const int64_t image = b.n * k.P * k.C + pl.at;
    const int64_t step = int64_t(k.rows) * k.C;
    const uint64_t counter = drop.threshold ? drop.counter() : 0;
    float s1[V] = {}, s2[V] = {};
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

template <class T, int V, class ACT>
__global__ __launch_bounds__(kThreads) void grad_apply_kernel(const T *dy, const T *x, Cut k, const float *mean,
                                                              const float *rstd, ct::Param<T> gamma, ct::Param<T> beta,
                                                              ACT f, Dropout drop, const float2 *coef, T *dx)
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
}

__global__ __launch_bounds__(kThreads) void empty_kernel(unsigned long long *p, int64_t count)
{
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < count; i += int64_t(gridDim.x) * kThreads) p[i] = kEmpty;
}

// dgamma and dbeta from the chunks' channel sums: 16 channels a block, 16 threads a channel.
template <class T>
__global__ __launch_bounds__(kThreads) void held_param_kernel(const float2 *sums, int64_t parts, int C, bool f32, void *dgamma,
                                                              void *dbeta)
{
    __shared__ float2 lds[16][16];
    const int c = int(blockIdx.x) * 16 + int(threadIdx.x & 15), q = threadIdx.x / 16;
    float2 s = make_float2(0.0f, 0.0f);
    if (c < C) {
#pragma unroll 8
        for (int64_t i = q; i < parts; i += 16) {
            const float2 v = sums[i * C + c];
            s.x += v.x;
            s.y += v.y;
        }
    }
    lds[q][threadIdx.x & 15] = s;
    __syncthreads();
    if (q != 0 || c >= C) return;
    for (int i = 1; i < 16; ++i) {
        s.x += lds[i][threadIdx.x].x;
        s.y += lds[i][threadIdx.x].y;
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

// Controls for tests and tuning (group_norm_set_control).
std::atomic<int> g_one_pass{-1}, g_wait_limit{-1};
constexpr int kWaitLimit = 4096;  // looks, about a microsecond each

// Blocks of kHeld threads the current device holds at once, two a compute unit (the
// kernels' register bound).
int64_t resident_blocks()
{
    int dev = 0, units = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 0;
    if (hipDeviceGetAttribute(&units, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
    return 2 * int64_t(units);
}

// The one-pass cut, if there is one.
bool make_one(const Sizes &s, bool backward, bool in_place, OneCut *k, bool *uni)
{
    const int want = g_one_pass.load(std::memory_order_relaxed);
    if (want == 0 || in_place) return false;
    const int V = s.dt == CT_FLOAT32 ? 4 : 8;
    const int64_t Cg = s.C / s.G;
    *uni = Cg % V == 0;
    const int64_t K = held_tiles(*uni, backward), threads = backward ? kHeldGrad : kHeld, most = threads * V;  // elements of a tile
    // groups of the narrowest slab whose rows are whole vectors, or all of them
    int64_t nb = V / std::gcd(Cg, int64_t(V));
    if (nb > s.G || s.G % nb) nb = s.G;
    auto try_slab = [&](int64_t groups, int64_t max_chunks) {
        const int64_t width = groups * Cg;
        if (groups > kMostGroups || width > most) return false;
        const int64_t unit = V / std::gcd(width, int64_t(V));
        if (unit > 1 && groups != s.G) return false;
        const int64_t fit = most / width / unit * unit;
        if (fit < 1 || fit * s.C > (int64_t(1) << 29)) return false;  // 32-bit offsets in a tile
        const int64_t need = (s.P + unit - 1) / unit * unit;
        k->rows = int(std::min(fit, need));
        const int64_t tiles = (s.P + k->rows - 1) / k->rows;
        const int64_t chunks = (tiles + K - 1) / K;
        if (chunks > max_chunks) return false;
        k->tiles = int((tiles + chunks - 1) / chunks);
        k->chunks = int((tiles + k->tiles - 1) / k->tiles);
        k->width = int(width);
        k->groups = int(groups);
        k->slabs = int(s.G / groups);
        return true;
    };
    k->P = s.P;
    k->C = int(s.C);
    k->G = int(s.G);
    k->Cg = int(Cg);
    bool ok = try_slab(nb, 1);
    if (!ok) {
        // as many groups a slab as fit: whole rows where possible
        int64_t wide = s.G;
        while (wide > nb && (wide * Cg > most || wide > kMostGroups || s.G % wide)) --wide;
        const int64_t room = resident_blocks();
        ok = try_slab(wide, room / std::max<int64_t>(1, s.G / wide));
        if (ok && int64_t(k->chunks) * k->slabs > room) ok = false;
    }
    if (!ok || s.N > (int64_t(1) << 22) / (int64_t(k->chunks) * k->slabs)) return false;
    k->lanes = 1;
    while (k->lanes < 64 && 2 * k->lanes * k->groups <= threads) k->lanes *= 2;
    const int limit = g_wait_limit.load(std::memory_order_relaxed);
    k->limit = limit < 0 ? kWaitLimit : limit;
    return true;
}

struct Plan {
    bool vec = true, one = false, uni = false;
    Cut k;
    OneCut h;
    size_t part = 0, stats = 0, total = 0, coef = 0, words = 0, bytes = 0;
};

Plan make_plan(const Sizes &s, bool backward, bool in_place)
{
    Plan p;
    if (s.empty()) return p;
    size_t at = 0;
    auto place = [&](size_t bytes) {
        const size_t q = at;
        at += (bytes + 255) & ~size_t(255);
        return q;
    };
    p.one = make_one(s, backward, in_place, &p.h, &p.uni);
    if (p.one) {
        p.words = place(p.h.chunks > 1 ? size_t(s.N) * s.G * p.h.chunks * 8 : 0);
        if (backward) p.part = place(size_t(s.N) * p.h.chunks * s.C * 8);
        p.bytes = at;
        return p;
    }
    p.vec = s.dt == CT_FLOAT32 ? make_cut<4>(s.N, s.P, s.C, s.G, &p.k) : make_cut<8>(s.N, s.P, s.C, s.G, &p.k);
    if (!p.vec) make_cut<1>(s.N, s.P, s.C, s.G, &p.k);
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

// Empties the exchanged words, if blocks exchange any.
void empty_words(const Plan &p, const Sizes &s, unsigned long long *words, hipStream_t hs)
{
    if (p.h.chunks == 1) return;
    const int64_t count = s.N * s.G * p.h.chunks;
    empty_kernel<<<std::min<unsigned>(blocks_of(count, kThreads), 1024), kThreads, 0, hs>>>(words, count);
}

}  // namespace

extern "C" {

ct_status group_norm_set_control(int one_pass, int wait_limit)
{
    ct::set_last_error(std::string());
    if (one_pass < -1 || one_pass > 0) return fail(CT_EINVAL, "one_pass must be -1 (automatic) or 0 (never)");
    if (wait_limit < -1) return fail(CT_EINVAL, "wait_limit must be -1 (the default) or a number of looks");
    g_one_pass.store(one_pass, std::memory_order_relaxed);
    g_wait_limit.store(wait_limit, std::memory_order_relaxed);
    return CT_OK;
}

ct_status group_norm_workspace_size(ct_dtype dtype, int nsp, const int64_t *x_shape, int64_t groups, int backward,
                                    size_t *bytes_out)
{
    ct::set_last_error(std::string());
    if (!bytes_out) return fail(CT_EINVAL, "bytes_out is NULL");
    if (backward != 0 && backward != 1) return fail(CT_EINVAL, "backward must be 0 or 1");
    Sizes s;
    const ct_status st = check_sizes(ct::enum_int(dtype), nsp, x_shape, groups, &s);
    if (st != CT_OK) return st;
    // in place or not, and with any control: the larger
    *bytes_out = std::max(make_plan(s, backward != 0, false).bytes, make_plan(s, backward != 0, true).bytes);
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
    const Plan p = make_plan(s, false, x == y);
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    ct::Scratch ws;
    st = ws.take(workspace, workspace_bytes, p.bytes, hs, &err);
    if (st != CT_OK) return fail(st, err);
    char *const base = static_cast<char *>(ws.p);
    float *const part = reinterpret_cast<float *>(base + p.part);
    unsigned long long *const words = reinterpret_cast<unsigned long long *>(base + p.words);
    if (!p.one && !mean) mean = reinterpret_cast<float *>(base + p.stats);
    if (!p.one && !rstd) rstd = reinterpret_cast<float *>(base + p.stats) + s.N * s.G;
    const int64_t blocks = p.one ? s.N * p.h.chunks * p.h.slabs : s.N * p.k.chunks * p.k.slabs;
    if (p.one) {
        Call c;
        c.dt = dt;
        c.params_f32 = pt == CT_FLOAT32;
        c.x = x;
        c.y = y;
        c.gamma = gamma;
        c.beta = beta;
        c.eps = eps;
        c.mean = mean;
        c.rstd = rstd;
        c.act = act;
        c.drop = drop;
        c.words = words;
        empty_words(p, s, words, hs);
        ct::mark_before(hs);
        launch_held(c, p.h, p.uni, blocks, hs);
        ct::mark_after(hs);
        st = ct::launch_status("group norm launch failed", &err);
        return st == CT_OK ? CT_OK : fail(st, err);
    }
    ct::with_type(dt, [&](auto t) {
        using T = decltype(t);
        const T *xp = static_cast<const T *>(x);
        const ct::Param<T> ga{gamma, pt == CT_FLOAT32}, be{beta, pt == CT_FLOAT32};
        auto go = [&](auto v) {
            constexpr int V = decltype(v)::value;
            stats_kernel<T, V><<<unsigned(blocks), kThreads, 0, hs>>>(xp, p.k, part);
            finish_kernel<T><<<blocks_of(s.N * s.G, kThreads / 64), kThreads, 0, hs>>>(xp, part, p.k, s.N * s.G, eps, mean, rstd);
            ct::mark_before(hs);
            with_act(act, [&](auto f) {
                apply_kernel<T, V, decltype(f)>
                    <<<unsigned(blocks), kThreads, 0, hs>>>(xp, p.k, mean, rstd, ga, be, f, drop, static_cast<T *>(y));
            });
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
    const Plan p = make_plan(s, true, dx == x || dx == dy);
    ct::Scratch ws;
    st = ws.take(workspace, workspace_bytes, p.bytes, hs, &err);
    if (st != CT_OK) return fail(st, err);
    char *const base = static_cast<char *>(ws.p);
    float2 *const part = reinterpret_cast<float2 *>(base + p.part);
    float2 *const total = reinterpret_cast<float2 *>(base + p.total);
    float2 *const coef = reinterpret_cast<float2 *>(base + p.coef);
    unsigned long long *const words = reinterpret_cast<unsigned long long *>(base + p.words);
    const int64_t blocks = s.empty() ? 0 : p.one ? s.N * p.h.chunks * p.h.slabs : s.N * p.k.chunks * p.k.slabs;
    if (p.one) {
        Call c;
        c.dt = dt;
        c.params_f32 = pt == CT_FLOAT32;
        c.x = x;
        c.dy = dy;
        c.dx = dx;
        c.gamma = gamma;
        c.beta = beta;
        c.mean = const_cast<float *>(mean);
        c.rstd = const_cast<float *>(rstd);
        c.act = act;
        c.drop = drop;
        c.words = words;
        c.sums = part;
        empty_words(p, s, words, hs);
        ct::mark_before(hs);
        launch_held_grad(c, p.h, p.uni, blocks, hs);
        ct::mark_after(hs);
    }
    ct::with_type(dt, [&](auto t) {
        using T = decltype(t);
        const T *xp = static_cast<const T *>(x), *dp = static_cast<const T *>(dy);
        const ct::Param<T> ga{gamma, pt == CT_FLOAT32}, be{beta, pt == CT_FLOAT32};
        if (p.one) {
            if (dgamma || dbeta)
                held_param_kernel<T><<<blocks_of(s.C, 16), kThreads, 0, hs>>>(part, s.N * p.h.chunks, int(s.C),
                                                                             pt == CT_FLOAT32, dgamma, dbeta);
            return;
        }
        auto go = [&](auto v) {
            constexpr int V = decltype(v)::value;
            with_act(act, [&](auto f) {
                grad_stats_kernel<T, V, decltype(f)>
                    <<<unsigned(blocks), kThreads, 0, hs>>>(dp, xp, p.k, mean, rstd, ga, be, f, drop, part);
            });
            grad_join_kernel<<<unsigned(s.N * blocks_of(s.C, 64)), 1024, 0, hs>>>(part, p.k, total);
            grad_groups_kernel<T><<<blocks_of(s.N * s.G, kThreads / 64), kThreads, 0, hs>>>(total, p.k, s.N * s.G, ga, coef);
            ct::mark_before(hs);
            with_act(act, [&](auto f) {
                grad_apply_kernel<T, V, decltype(f)><<<unsigned(blocks), kThreads, 0, hs>>>(
                    dp, xp, p.k, mean, rstd, ga, be, f, drop, coef, static_cast<T *>(dx));
            });
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

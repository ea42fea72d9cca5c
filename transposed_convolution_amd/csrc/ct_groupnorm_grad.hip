// ct_groupnorm_grad.hip -- the kernels of group norm's gradient (what they share is in
// ct_groupnorm.hpp, the entry points are in ct_groupnorm.hip).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ct_groupnorm.hpp"

namespace {

using namespace ct::norm;
using ct::Dropout;
using ct::Raw;

// The constants of a thread's channels: z = (x - mu) a + be, a = rstd gamma.
template <class T, int V, int S>
struct Constants {
    float mu[kOwn<S, V>], rs[kOwn<S, V>], a[V], be[V];
    __device__ Constants(const Cut &k, const Place<V> &pl, const float *mean, const float *rstd, const ct::Param<T> &gamma,
                         const ct::Param<T> &beta)
    {
        pl.params(a, k, gamma, 1.0f);
        pl.params(be, k, beta, 0.0f);
        const int64_t first = pl.n * k.G + pl.g0;
        pl.template each<S>(k, [&](int j, int, int g) {
            mu[j] = mean[first + g];
            rs[j] = rstd[first + g];
        });
#pragma unroll
        for (int j = 0; j < V; ++j) a[j] *= rs[j / S];
    }
};

// dz of one tile, before the dropout factor.
template <class T, int V, int S, class ACT>
__device__ __forceinline__ void tile_dz(float (&dz)[V], float (&d)[V], const Raw<T, V> &xv, const Raw<T, V> &dv,
                                        const Constants<T, V, S> &ch, const ACT &f, const Dropout &drop, uint64_t counter,
                                        int64_t first)
{
    const float one = opaque_one();
#pragma unroll
    for (int j = 0; j < V; ++j) {
        d[j] = minus(xv[j], ch.mu[j / S], one);
        dz[j] = times(dv[j], f.d(__builtin_fmaf(d[j], ch.a[j], ch.be[j])));
    }
    if (drop.threshold) {  // a select: a dropped dy may be anything
        const ct::Fields keep = ct::draw_fields<V, (S > 1)>(drop, counter, uint64_t(first));
#pragma unroll
        for (int j = 0; j < V; ++j) dz[j] = keep.stays(j, drop.limit()) ? dz[j] : 0.0f;
    }
}

// The block's sums: every channel's (sum dz, sum dz xhat) to column(channel of the slab, sums),
// every group's (sum dz gamma, sum dz gamma xhat) to out(group of the slab, a, b), on one
// thread each.
template <int THREADS, class T, int V, class Column, class Out>
__device__ __forceinline__ void join_sums(const Cut &k, const Place<V> &pl, const float (&s1)[V], const float (&s2)[V],
                                          float2 (&lds)[THREADS * V], const ct::Param<T> &gamma, Column column, Out out)
{
    if (pl.active)
#pragma unroll
        for (int j = 0; j < V; ++j) lds[pl.e + j] = make_float2(s1[j], s2[j]);
    __syncthreads();
    // a narrow slab has many rows and few columns: first up to 16 threads a column, rows apart
    const int parts = min(min(16, k.rows), int(blockDim.x) / pl.width);
    if (parts > 1) {
        const int q = int(threadIdx.x) / pl.width, c = int(threadIdx.x) - q * pl.width;
        float2 s = make_float2(0.0f, 0.0f);
        if (q < parts)
            for (int r = q; r < k.rows; r += parts) {
                const float2 v = lds[r * pl.width + c];
                s.x += v.x;
                s.y += v.y;
            }
        __syncthreads();
        if (q < parts) lds[q * pl.width + c] = s;
        __syncthreads();
    }
    const int rows = parts > 1 ? parts : k.rows;
    for (int c = threadIdx.x; c < pl.width; c += int(blockDim.x)) {
        float2 s = lds[c];
        for (int r = 1; r < rows; ++r) {
            const float2 v = lds[r * pl.width + c];
            s.x += v.x;
            s.y += v.y;
        }
        column(c, s);
        const float w = gamma.at(pl.c0 + c, 1.0f);
        lds[c] = make_float2(s.x * w, s.y * w);  // nobody else reads this column
    }
    __syncthreads();
    const int per = k.split > 1 ? pl.width : k.Cg, lane = threadIdx.x & (k.lanes - 1);
    for (int g = int(threadIdx.x) / k.lanes; g < pl.groups; g += int(blockDim.x) / k.lanes) {
        float a = 0.0f, b = 0.0f;
        for (int c = lane; c < per; c += k.lanes) {
            const float2 v = lds[g * per + c];
            a += v.x;
            b += v.y;
        }
        for (int o = 1; o < k.lanes; o *= 2) {
            a += __shfl_xor(a, o);
            b += __shfl_xor(b, o);
        }
        if (lane == 0) out(g, a, b);
    }
}

// dx = rstd (dz gamma - c1 - xhat c2) = dz a - k1 - (x - mu) k2, from coef = (c1, c2) of the
// slab's groups; a gets the dropout factor.
template <class T, int V, int S>
__device__ __forceinline__ void output_constants(OwnFloats<S, V> &k1, OwnFloats<S, V> &k2,
                                                 Constants<T, V, S> &ch, const Cut &k, const Place<V> &pl, const float2 *coef,
                                                 float factor)
{
    pl.template each<S>(k, [&](int j, int, int g) {
        const float2 v = coef[g];
        k1[j] = v.x * ch.rs[j];
        k2[j] = v.y * ch.rs[j] * ch.rs[j];
    });
#pragma unroll
    for (int j = 0; j < V; ++j) ch.a[j] *= factor;
}

// One block has all positions of its groups: x and dy are read once, x is held in registers
// and so is dz, in float32.  sums[n][c] = (sum dz, sum dz xhat).  Bound by its chain of load,
// join and store, and the launch for the parameters: 1 x 256 x 1024 float16 10.9 us.
template <class T, int V, int S, class ACT>
__global__ __launch_bounds__(kOneGradThreads, 2) void one_grad_kernel(const T *dy, const T *x, Cut k, const float *mean,
                                                                      const float *rstd, ct::Param<T> gamma,
                                                                      ct::Param<T> beta, ACT f, Dropout drop, float2 *sums,
                                                                      T *dx)
{
    constexpr int K = kOneTiles;
    __shared__ float2 lds[kOneGradThreads * V];
    __shared__ float2 coef[kMostGroups];
    const Place<V> pl(k, blockIdx.x);
    Held<V> xr[K], dr[K];
    load_tiles<T, K, V>(xr, x, k, pl, 0);
    load_tiles<T, K, V>(dr, dy, k, pl, 0);
    const bool full = pl.full(k, 0, K);
    Constants<T, V, S> ch(k, pl, mean, rstd, gamma, beta);
    const uint64_t counter = drop.threshold ? drop.counter() : 0;
    // elements that do not exist are zeros in dy and add nothing
    float s1[V] = {}, s2[V] = {}, dz[K][V];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        float d[V];
        tile_dz<T, V, S>(dz[i], d, held<T, V>(xr[i]), held<T, V>(dr[i]), ch, f, drop, counter, pl.tile(k, i) + pl.off);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s1[j] += dz[i][j];
            s2[j] = __builtin_fmaf(dz[i][j], d[j], s2[j]);
        }
        one_by_one();
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s1[j] *= drop.factor;
        s2[j] *= drop.factor * ch.rs[j / S];
    }
    const float count = float(k.P) * float(k.Cg);
    join_sums<kOneGradThreads, T, V>(
        k, pl, s1, s2, lds, gamma, [&](int c, float2 s) { sums[pl.n * k.C + pl.c0 + c] = s; },
        [&](int g, float a, float b) { coef[g] = make_float2(a / count, b / count); });
    __syncthreads();
    if (!pl.active) return;
    float k1[kOwn<S, V>], k2[kOwn<S, V>];
    output_constants<T, V, S>(k1, k2, ch, k, pl, coef, drop.factor);
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int valid = full ? V : pl.valid(k, i);
        if (valid == 0) continue;
        const Raw<T, V> xv = held<T, V>(xr[i]);
        Raw<T, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int q = j / S;
            o[j] = T(__builtin_fmaf(dz[i][j], ch.a[j], __builtin_fmaf(ch.mu[q] - float(xv[j]), k2[q], -k1[q])));
        }
        store_first<T, V>(dx + pl.tile(k, i) + pl.off, o, valid);
        one_by_one();
    }
}

// The first pass.  A thread owns the same channels in all its tiles, so sums by channel stay in
// registers and the groups' follow from them at the end, with gamma.  In a trace, 8 x 256 x 16384
// float16 with SiLU and dropout (134 MB): 38.3 us, 3.5 TB/s, the vector units 69 % busy (SiLU's
// derivative takes an exponential and a reciprocal, the generator ten rounds for eight elements);
// 2 x 64 x 131072 bfloat16 without dropout (67 MB): 16.8 us, 4.0 TB/s.
// Sums of more than kSumTiles tiles are made in two levels, in float32: equal terms are all rounded
// the same way, and n of them one after another may cost n / 4 roundings of their sum.
// part[n][g][chunk][slab of the group] = (sum dz gamma, sum dz gamma xhat),
// sums[n][chunk][c] = (sum dz, sum dz xhat).
constexpr int kSumTiles = 64;
template <class T, int V, int S, class ACT>
__global__ __launch_bounds__(kGradThreads, S > 1 ? 4 : 3) void grad_stats_kernel(const T *dy, const T *x, Cut k, const float *mean,
                                                                     const float *rstd, ct::Param<T> gamma,
                                                                     ct::Param<T> beta, ACT f, Dropout drop, float2 *part,
                                                                     float2 *sums)
{
    constexpr int K = kGradTiles;
    static_assert(kSumTiles % K == 0, "a level ends between two rounds of loads");
    __shared__ float2 lds[kGradThreads * V];
    const Place<V> pl(k, blockIdx.x);
    const Constants<T, V, S> ch(k, pl, mean, rstd, gamma, beta);
    const uint64_t counter = drop.threshold ? drop.counter() : 0;
    float s1[V] = {}, s2[V] = {};
    float2 *const own = lds + threadIdx.x * V;  // until the join, the thread's sums of the tiles before
    for (int first = 0; first < k.tiles; first += K) {
        if (first > 0 && first % kSumTiles == 0) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 before = first > kSumTiles ? own[j] : make_float2(0.0f, 0.0f);
                own[j] = make_float2(before.x + s1[j], before.y + s2[j]);
                s1[j] = s2[j] = 0.0f;
            }
        }
        Held<V> xr[K], dr[K];
        load_tiles<T, K, V>(xr, x, k, pl, first);
        load_tiles<T, K, V>(dr, dy, k, pl, first);
#pragma unroll
        for (int i = 0; i < K; ++i) {
            float dz[V], d[V];
            tile_dz<T, V, S>(dz, d, held<T, V>(xr[i]), held<T, V>(dr[i]), ch, f, drop, counter,
                               pl.tile(k, first + i) + pl.off);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s1[j] += dz[j];
                s2[j] = __builtin_fmaf(dz[j], d[j], s2[j]);
            }
            one_by_one();
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (k.tiles > kSumTiles) {
            s1[j] += own[j].x;
            s2[j] += own[j].y;
        }
        s1[j] *= drop.factor;
        s2[j] *= drop.factor * ch.rs[j / S];
    }
    join_sums<kGradThreads, T, V>(
        k, pl, s1, s2, lds, gamma,
        [&](int c, float2 s) { sums[(pl.n * k.chunks + pl.chunk) * k.C + pl.c0 + c] = s; },
        [&](int g, float a, float b) {
            part[((pl.n * k.G + pl.g0 + g) * k.chunks + pl.chunk) * k.split + pl.sub] = make_float2(a, b);
        });
}

// (c1, c2) of one group from its parts, `lanes` threads together.
__device__ __forceinline__ float2 join_parts(const float2 *part, const Cut &s, int64_t group, int lane, int lanes)
{
    const int count = s.chunks * s.split;
    const float2 *p = part + group * count;
    float2 t = make_float2(0.0f, 0.0f);
    constexpr int kAtOnce = 16;  // on their way together
    for (int q = lane; q < count; q += kAtOnce * lanes) {
        float2 v[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) v[j] = p[q + j * lanes < count ? q + j * lanes : q];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const bool in = q + j * lanes < count;
            t.x += in ? v[j].x : 0.0f;
            t.y += in ? v[j].y : 0.0f;
        }
    }
    for (int o = 1; o < lanes; o *= 2) {
        t.x += __shfl_xor(t.x, o);
        t.y += __shfl_xor(t.y, o);
    }
    const float n = float(s.P) * float(s.Cg);
    return make_float2(t.x / n, t.y / n);
}

__global__ __launch_bounds__(256) void grad_finish_kernel(const float2 *part, Cut s, int64_t groups, float2 *coef)
{
    const int64_t g = (int64_t(blockIdx.x) * 256 + threadIdx.x) / 64;
    if (g >= groups) return;
    const float2 v = join_parts(part, s, g, threadIdx.x & 63, 64);
    if ((threadIdx.x & 63) == 0) coef[g] = v;
}

// dgamma and dbeta of 16 channels from their `parts` sums, by one block: 16 threads a channel.
// Added in 64 bits: a thread may have 2^17 parts (an image each), and equal ones would all be
// rounded the same way.
template <class T>
__device__ __forceinline__ void param_gradients(const float2 *sums, int64_t parts, int C, int tile, bool f32, void *dgamma,
                                                void *dbeta)
{
    __shared__ double2 lds[16][16];
    const int c = tile * 16 + int(threadIdx.x & 15), q = threadIdx.x / 16;
    double2 s = make_double2(0.0, 0.0);
    if (c < C) {
#pragma unroll 8
        for (int64_t i = q; i < parts; i += 16) {
            const float2 v = sums[i * C + c];
            s.x += double(v.x);
            s.y += double(v.y);
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
        if (f32) static_cast<float *>(dgamma)[c] = float(s.y);
        else static_cast<T *>(dgamma)[c] = T(float(s.y));
    }
    if (dbeta) {
        if (f32) static_cast<float *>(dbeta)[c] = float(s.x);
        else static_cast<T *>(dbeta)[c] = T(float(s.x));
    }
}

template <class T>
__global__ __launch_bounds__(256) void param_kernel(const float2 *sums, int64_t parts, int C, bool f32, void *dgamma,
                                                    void *dbeta)
{
    param_gradients<T>(sums, parts, C, blockIdx.x, f32, dgamma, dbeta);
}

// The second pass makes dz again (stored, it would be two more passes over memory) and dx from
// it.  In a trace, 8 x 256 x 16384 float16 with SiLU and dropout (201 MB): 42.2 us, 4.8 TB/s, the
// vector units 71 % busy; 2 x 64 x 131072 bfloat16 (101 MB): 20.4 us, 4.9 TB/s, a copy's rate.  The
// first `head` blocks make dgamma and dbeta; the others write dx.
// finished: c1 and c2 are there; else every block joins the parts of its groups, before it asks for
// its values: behind those the parts took 8 us of a block's 20 to arrive.
template <class T, int V, int S, class ACT>
__global__ __launch_bounds__(kApplyThreads, S > 1 ? 4 : 3) void grad_apply_kernel(const T *dy, const T *x, Cut k, Cut s, const float *mean,
                                                                      const float *rstd, ct::Param<T> gamma,
                                                                      ct::Param<T> beta, ACT f, Dropout drop,
                                                                      const float2 *part, bool finished, const float2 *sums,
                                                                      int64_t parts, int head, void *dgamma, void *dbeta, T *dx)
{
    constexpr int K = kGradTiles;
    __shared__ float2 coef[kMostGroups];
    if (int(blockIdx.x) < head) {
        param_gradients<T>(sums, parts, k.C, blockIdx.x, gamma.f32, dgamma, dbeta);
        return;
    }
    const Place<V> pl(k, blockIdx.x - unsigned(head));
    if (finished) {
        for (int g = threadIdx.x; g < pl.groups; g += kApplyThreads) coef[g] = part[pl.n * k.G + pl.g0 + g];
    } else {
        const int lane = threadIdx.x & (k.lanes - 1);
        for (int g = int(threadIdx.x) / k.lanes; g < pl.groups; g += kApplyThreads / k.lanes) {
            const float2 v = join_parts(part, s, pl.n * k.G + pl.g0 + g, lane, k.lanes);
            if (lane == 0) coef[g] = v;
        }
    }
    Held<V> xr[K], dr[K];
    load_tiles<T, K, V>(xr, x, k, pl, 0);
    load_tiles<T, K, V>(dr, dy, k, pl, 0);
    Constants<T, V, S> ch(k, pl, mean, rstd, gamma, beta);
    __syncthreads();
    if (!pl.active) return;
    const uint64_t counter = drop.threshold ? drop.counter() : 0;
    float k1[kOwn<S, V>], k2[kOwn<S, V>];
    output_constants<T, V, S>(k1, k2, ch, k, pl, coef, 1.0f);  // the factor goes to dz here
    const float factor = drop.factor;
    for (int first = 0;;) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int valid = pl.valid(k, first + i);
            if (valid == 0) continue;
            const int64_t at = pl.tile(k, first + i) + pl.off;
            float dz[V], d[V];
            tile_dz<T, V, S>(dz, d, held<T, V>(xr[i]), held<T, V>(dr[i]), ch, f, drop, counter, at);
            Raw<T, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int q = j / S;
                o[j] = T(__builtin_fmaf(dz[j] * factor, ch.a[j], __builtin_fmaf(-d[j], k2[q], -k1[q])));
            }
            store_first<T, V>(dx + at, o, valid);
            one_by_one();
        }
        first += K;
        if (first >= k.tiles) break;
        load_tiles<T, K, V>(xr, x, k, pl, first);
        load_tiles<T, K, V>(dr, dy, k, pl, first);
    }
}

}  // namespace

void ct::norm::launch_gradient(const Call &c, const Plan &p, char *ws, hipStream_t st)
{
    float2 *const part = reinterpret_cast<float2 *>(ws + p.part);
    float2 *const coef = reinterpret_cast<float2 *>(ws + p.stats);
    float2 *const sums = reinterpret_cast<float2 *>(ws + p.sums);
    const bool params = c.dgamma || c.dbeta;
    const int head = params ? int(param_blocks(p.a.C)) : 0;
    const int64_t groups = c.N * p.a.G, blocks = c.N * p.a.chunks * p.a.slabs;
    with_type(c.dt, [&](auto t) {
        using T = decltype(t);
        const T *const x = static_cast<const T *>(c.x), *const dy = static_cast<const T *>(c.dy);
        T *const dx = static_cast<T *>(c.dx);
        const Param<T> gamma{c.gamma, c.params_f32}, beta{c.beta, c.params_f32};
        if (p.one) {
            with_vector<T>(p, [&](auto v, auto run) {
                constexpr int V = decltype(v)::value, S = decltype(run)::value;
                if constexpr (V == kVec<T>)
                    with_act(c.act, [&](auto f) {
                        using F = decltype(f);
                        mark_before(st);
                        one_grad_kernel<T, V, S, F><<<unsigned(blocks), p.threads, 0, st>>>(
                            dy, x, p.a, c.mean, c.rstd, gamma, beta, f, c.drop, sums, dx);
                        mark_after(st);
                    });
            });
            if (params) param_kernel<T><<<unsigned(head), 256, 0, st>>>(sums, c.N, p.a.C, c.params_f32, c.dgamma, c.dbeta);
            return;
        }
        with_vector<T>(p, [&](auto v, auto run) {
            constexpr int V = decltype(v)::value;
            constexpr int S = decltype(run)::value;
            with_act(c.act, [&](auto f) {
                using F = decltype(f);
                grad_stats_kernel<T, V, S, F><<<unsigned(c.N * p.s.chunks * p.s.slabs), kGradThreads, 0, st>>>(
                    dy, x, p.s, c.mean, c.rstd, gamma, beta, f, c.drop, part, sums);
                if (p.finish) grad_finish_kernel<<<unsigned((groups + 3) / 4), 256, 0, st>>>(part, p.s, groups, coef);
                mark_before(st);
                grad_apply_kernel<T, V, S, F><<<unsigned(blocks + head), kApplyThreads, 0, st>>>(
                    dy, x, p.a, p.s, c.mean, c.rstd, gamma, beta, f, c.drop, p.finish ? coef : part, p.finish, sums,
                    c.N * p.s.chunks, head, c.dgamma, c.dbeta, dx);
                mark_after(st);
            });
        });
    });
}

void ct::norm::launch_no_gradient(int dt, bool params_f32, int C, void *dgamma, void *dbeta, hipStream_t st)
{
    with_type(dt, [&](auto t) {
        param_kernel<decltype(t)><<<unsigned(param_blocks(C)), 256, 0, st>>>(nullptr, 0, C, params_f32, dgamma, dbeta);
    });
}

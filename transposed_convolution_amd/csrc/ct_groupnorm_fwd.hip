// ct_groupnorm_fwd.hip -- the kernels of group norm with an activation and dropout (what they
// share is in ct_groupnorm.hpp, the entry points are in ct_groupnorm.hip).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ct_groupnorm.hpp"

namespace {

using namespace ct::norm;
using ct::Dropout;
using ct::Raw;

// Joins the block's moments of each group of the slab and calls out(group of the slab,
// moments), on one thread a group.  How many values a run has follows from its row.
template <int THREADS, int V, int S, class Out>
__device__ __forceinline__ void join_block(const Cut &k, const Place<V> &pl, const OwnFloats<S, V> &pivot,
                                           const OwnMoments<S, V> &m, JoinBuffer<THREADS, S, V> &lds, Out out)
{
    constexpr int A = kOwn<S, V>, unit = S;  // elements a run has in a tile
    if (pl.active) {
#pragma unroll
        for (int a = 0; a < A; ++a) {
            lds[0][threadIdx.x * A + a] = pivot[a];
            lds[1][threadIdx.x * A + a] = m[a].mean;
            lds[2][threadIdx.x * A + a] = m[a].m2;
        }
    }
    __syncthreads();
    const int per = (k.split > 1 ? pl.width : k.Cg) / unit, row = pl.width / unit, lane = threadIdx.x & (k.lanes - 1);
    const bool last = pl.chunk + 1 == k.chunks;  // a run past the image's end is in one tile less
    const int tiles = last ? k.last_tiles : k.tiles, end = last ? k.last_rows : k.rows;
    for (int g = int(threadIdx.x) / k.lanes; g < pl.groups; g += int(blockDim.x) / k.lanes) {
        Moments<double> s;
        for (int i = lane; i < per * k.rows; i += k.lanes) {
            const int r = i / per, at = r * row + g * per + (i - r * per);
            s.join(float(unit) * float(r < end ? tiles : tiles - 1), double(lds[0][at]) + double(lds[1][at]), lds[2][at]);
        }
        for (int o = 1; o < k.lanes; o *= 2) s.join(__shfl_xor(s.n, o), __shfl_xor(s.mean, o), __shfl_xor(s.m2, o));
        if (lane == 0) out(g, s);
    }
}

// y of one tile from its x.
template <class T, int V, int S, class ACT>
__device__ __forceinline__ Raw<T, V> outputs(const Raw<T, V> &v, const OwnFloats<S, V> &mu, const float (&a)[V],
                                             const float (&be)[V], const ACT &f, const Dropout &drop, uint64_t counter,
                                             int64_t first)
{
    const float one = opaque_one();
    Raw<T, V> o;
    float r[V];
#pragma unroll
    for (int j = 0; j < V; ++j) r[j] = f.y(__builtin_fmaf(minus(v[j], mu[j / S], one), a[j], be[j]));
    if (drop.threshold) {
        const ct::Fields keep = ct::draw_fields<V, (S > 1)>(drop, counter, uint64_t(first));
#pragma unroll
        for (int j = 0; j < V; ++j) r[j] = keep.stays(j, drop.limit()) ? r[j] * drop.factor : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = T(r[j]);
    return o;
}

// The constants of a thread's channels, z = (x - mu) a + be, from a = gamma and the groups'
// statistics.
template <int V, int S>
__device__ __forceinline__ void channel_constants(OwnFloats<S, V> &mu, float (&a)[V], const Cut &k, const Place<V> &pl,
                                                  const float2 *stat)
{
    float rs[kOwn<S, V>];
    pl.template each<S>(k, [&](int j, int, int g) {
        const float2 v = stat[g];
        mu[j] = v.x;
        rs[j] = v.y;
    });
#pragma unroll
    for (int j = 0; j < V; ++j) a[j] *= rs[j / S];
}

// One block has all positions of its groups: x is read once and held in registers.  Bound by
// the launch and one chain of load, join and store: 256 channels of 8 x 8 positions,
// float16 (64 KB in all), 5.3 us.
template <class T, int V, int S, class ACT>
__global__ __launch_bounds__(kOneThreads, 4) void one_kernel(const T *x, Cut k, float eps, ct::Param<T> gamma,
                                                             ct::Param<T> beta, ACT f, Dropout drop, T *y, float *mean,
                                                             float *rstd)
{
    constexpr int A = kOwn<S, V>, K = kOneTiles;
    __shared__ float lds[3][kOneThreads * A];
    __shared__ float2 stat[kMostGroups];
    const Place<V> pl(k, blockIdx.x);
    Held<V> raw[K];
    load_tiles<T, K, V>(raw, x, k, pl, 0);
    const bool full = pl.full(k, 0, K);
    float pivot[A], a[V], be[V];
    pl.params(a, k, gamma, 1.0f);
    pl.params(be, k, beta, 0.0f);
    first_values<T, V, S>(pivot, raw[0]);
    Moments<float> m[A];
    own_moments<T, V, S, K>(m, pivot, K, [&](int i) { return held<T, V>(raw[i]); },
                              [&](int i) { return full ? (pl.active ? V : 0) : pl.valid(k, i); });
    join_block<kOneThreads, V, S>(k, pl, pivot, m, lds, [&](int g, const Moments<double> &s) {
        const float mu = float(s.mean), r = 1.0f / sqrtf(s.m2 / s.n + eps);
        stat[g] = make_float2(mu, r);
        const int64_t at = pl.n * k.G + pl.g0 + g;
        if (mean) mean[at] = mu;
        if (rstd) rstd[at] = r;
    });
    __syncthreads();
    if (!pl.active) return;
    float mu[A];
    channel_constants<V, S>(mu, a, k, pl, stat);
    const uint64_t counter = drop.threshold ? drop.counter() : 0;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int valid = full ? V : pl.valid(k, i);
        if (valid == 0) continue;
        const int64_t at = pl.tile(k, i) + pl.off;
        store_first<T, V>(y + at, outputs<T, V, S>(held<T, V>(raw[i]), mu, a, be, f, drop, counter, at), valid);
        one_by_one();
    }
}

// The first pass: x is read once, 16 vectors of a thread on their way at a time (a block of 512
// threads has 128 KB in flight), and leaves 8 bytes a group and chunk.  Bound by memory: 8 x 256 x
// 16384 float16 (67 MB) 14.6 us in a trace, 4.6 TB/s.  A loop that starts the next tile's load when it
// has used one was no faster.
// part[n][g][chunk][slab of the group] = (mean, m2), the mean rounded to float32 (it is off by no
// more than the call's own mean may be); the counts follow from the cut.
template <class T, int V, int S, int K>
__global__ __launch_bounds__(kStatThreads, 4) void stats_kernel(const T *x, Cut k, float2 *part)
{
    constexpr int A = kOwn<S, V>;
    __shared__ float lds[3][kStatThreads * A];
    const Place<V> pl(k, blockIdx.x);
    float pivot[A];
    Moments<float> m[A];
    for (int first = 0; first < k.tiles; first += K) {
        Held<V> raw[K];
        load_tiles<T, K, V>(raw, x, k, pl, first);
        if (first == 0) first_values<T, V, S>(pivot, raw[0]);
        const bool full = pl.full(k, first, K);
        Moments<float> t[A];
        own_moments<T, V, S, K>(t, pivot, K, [&](int i) { return held<T, V>(raw[i]); },
                                  [&](int i) { return full ? (pl.active ? V : 0) : pl.valid(k, first + i); });
#pragma unroll
        for (int a = 0; a < A; ++a) m[a].join(t[a].n, t[a].mean, t[a].m2);
    }
    join_block<kStatThreads, V, S>(k, pl, pivot, m, lds, [&](int g, const Moments<double> &s) {
        const int64_t group = pl.n * k.G + pl.g0 + g;
        part[(group * k.chunks + pl.chunk) * k.split + pl.sub] = make_float2(float(s.mean), s.m2);
    });
}

// Joins the parts of one group, `lanes` threads together; the moments on every one of them.
__device__ __forceinline__ Moments<double> join_parts(const float2 *part, const Cut &s, int64_t group, int lane, int lanes)
{
    constexpr int kAtOnce = 8;  // on their way together
    const float2 *p = part + group * s.chunks * s.split;
    const int count = s.chunks * s.split;
    Moments<double> m;
    for (int q = lane; q < count; q += kAtOnce * lanes) {
        float2 v[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) v[j] = p[q + j * lanes < count ? q + j * lanes : q];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int at = q + j * lanes;
            if (at >= count) break;
            const int chunk = at / s.split, sub = at - chunk * s.split;
            const int64_t left = s.P - chunk * s.span();
            const int channels = s.split == 1 ? s.Cg : s.Cg - sub * s.width < s.width ? s.Cg - sub * s.width : s.width;
            m.join(float(channels) * float(left < s.span() ? left : s.span()), double(v[j].x), v[j].y);
        }
    }
    for (int o = 1; o < lanes; o *= 2) m.join(__shfl_xor(m.n, o), __shfl_xor(m.mean, o), __shfl_xor(m.m2, o));
    return m;
}

// mean and rstd of every group, one wave a group.
__global__ __launch_bounds__(256) void finish_kernel(const float2 *part, Cut s, int64_t groups, float eps,
                                                     float *mean, float *rstd)
{
    const int64_t g = (int64_t(blockIdx.x) * 256 + threadIdx.x) / 64;
    if (g >= groups) return;
    const Moments<double> m = join_parts(part, s, g, threadIdx.x & 63, 64);
    if ((threadIdx.x & 63) == 0) {
        mean[g] = float(m.mean);
        rstd[g] = 1.0f / sqrtf(m.m2 / m.n + eps);
    }
}

// The second pass: x is read again and y written, bound by memory: 8 x 256 x 16384 float16
// (134 MB) 26.3 us in a trace, 5.1 TB/s, a copy's rate.  The whole call takes 40.2 us; one pass that keeps x
// in registers while the blocks exchange their parts would read x once, but the exchange
// (6 to 13 us an image, while its blocks wait) cost more than the second read.
// finished: mean and rstd are there; else every block joins the parts of its
// groups, before it asks for its values (behind those they would arrive late), and the first
// chunk's blocks write mean and rstd down.
template <class T, int V, int S, class ACT>
__global__ __launch_bounds__(kApplyThreads, 4) void apply_kernel(const T *x, Cut k, Cut s, const float2 *part,
                                                                 bool finished, float eps, ct::Param<T> gamma,
                                                                 ct::Param<T> beta, ACT f, Dropout drop,
                                                                 T *y, float *mean, float *rstd)
{
    constexpr int A = kOwn<S, V>, K = kApplyTiles;
    __shared__ float2 stat[kMostGroups];
    const Place<V> pl(k, blockIdx.x);
    if (finished) {
        for (int g = threadIdx.x; g < pl.groups; g += kApplyThreads) {
            const int64_t at = pl.n * k.G + pl.g0 + g;
            stat[g] = make_float2(mean[at], rstd[at]);
        }
    } else {
        const int lane = threadIdx.x & (k.lanes - 1);
        for (int g = int(threadIdx.x) / k.lanes; g < pl.groups; g += kApplyThreads / k.lanes) {
            const int64_t group = pl.n * k.G + pl.g0 + g;
            const Moments<double> m = join_parts(part, s, group, lane, k.lanes);
            if (lane == 0) {
                const float mu = float(m.mean), r = 1.0f / sqrtf(m.m2 / m.n + eps);
                stat[g] = make_float2(mu, r);
                if (pl.chunk == 0 && pl.sub == 0) {
                    if (mean) mean[group] = mu;
                    if (rstd) rstd[group] = r;
                }
            }
        }
    }
    Held<V> raw[K];
    load_tiles<T, K, V>(raw, x, k, pl, 0);
    float a[V], be[V];
    pl.params(a, k, gamma, 1.0f);
    pl.params(be, k, beta, 0.0f);
    __syncthreads();
    if (!pl.active) return;
    float mu[A];
    channel_constants<V, S>(mu, a, k, pl, stat);
    const uint64_t counter = drop.threshold ? drop.counter() : 0;
    for (int first = 0;;) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int valid = pl.valid(k, first + i);
            if (valid == 0) continue;
            const int64_t at = pl.tile(k, first + i) + pl.off;
            store_first<T, V>(y + at, outputs<T, V, S>(held<T, V>(raw[i]), mu, a, be, f, drop, counter, at), valid);
        }
        first += K;
        if (first >= k.tiles) break;
        load_tiles<T, K, V>(raw, x, k, pl, first);
    }
}

}  // namespace

void ct::norm::launch_forward(const Call &c, const Plan &p, char *ws, hipStream_t st)
{
    float2 *const part = reinterpret_cast<float2 *>(ws + p.part);
    float *const stats = reinterpret_cast<float *>(ws + p.stats);
    const int64_t groups = c.N * p.a.G, blocks = c.N * p.a.chunks * p.a.slabs;
    with_type(c.dt, [&](auto t) {
        using T = decltype(t);
        const T *const x = static_cast<const T *>(c.x);
        T *const y = static_cast<T *>(c.y);
        const Param<T> gamma{c.gamma, c.params_f32}, beta{c.beta, c.params_f32};
        if (p.one) {
            with_vector<T>(p, [&](auto v, auto run) {
                constexpr int V = decltype(v)::value, S = decltype(run)::value;
                if constexpr (V == kVec<T>)
                    with_act(c.act, [&](auto f) {
                        using F = decltype(f);
                        mark_before(st);
                        one_kernel<T, V, S, F><<<unsigned(blocks), p.threads, 0, st>>>(
                            x, p.a, c.eps, gamma, beta, f, c.drop, y, c.mean, c.rstd);
                        mark_after(st);
                    });
            });
            return;
        }
        with_vector<T>(p, [&](auto v, auto run) {
            constexpr int V = decltype(v)::value;
            constexpr int S = decltype(run)::value;
            const unsigned stat_blocks = unsigned(c.N * p.s.chunks * p.s.slabs);
            if (p.s.tiles <= kStatShort)
                stats_kernel<T, V, S, kStatShort><<<stat_blocks, kStatThreads, 0, st>>>(x, p.s, part);
            else stats_kernel<T, V, S, kStatTiles><<<stat_blocks, kStatThreads, 0, st>>>(x, p.s, part);
            float *mean = c.mean, *rstd = c.rstd;
            if (p.finish) {
                if (!mean) mean = stats;
                if (!rstd) rstd = stats + groups;
                finish_kernel<<<unsigned((groups + 3) / 4), 256, 0, st>>>(part, p.s, groups, c.eps, mean, rstd);
            }
            mark_before(st);
            with_act(c.act, [&](auto f) {
                using F = decltype(f);
                apply_kernel<T, V, S, F><<<unsigned(blocks), kApplyThreads, 0, st>>>(
                    x, p.a, p.s, part, p.finish, c.eps, gamma, beta, f, c.drop, y, mean, rstd);
            });
            mark_after(st);
        });
    });
}

// ct_groupnorm_held.hip -- group norm in one pass over x (see ct_groupnorm.hpp).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ct_groupnorm.hpp"

namespace {

using namespace ct::norm;
using ct::Dropout;
using ct::Raw;

template <bool UNI, int V>
using OwnMoments = Moments[kOwn<UNI, V>];
template <bool UNI, int V>
using OwnPivots = float[kOwn<UNI, V>];
template <bool UNI, int V>
using JoinBuffer = float[3][kHeld * kOwn<UNI, V>];

// The thread's moments over `tiles` tiles, updated tile by tile: get(i) is tile i's vector,
// valid(i) how much of it exists.  An element that exists in a tile exists in all tiles
// before, so the counts are known constants where the loop is unrolled.
template <class T, int V, bool UNI, int UNROLL, class Get, class Valid>
__device__ __forceinline__ void own_moments(OwnMoments<UNI, V> &m, const OwnPivots<UNI, V> &pivot, int tiles, Get get,
                                            Valid valid)
{
#pragma unroll UNROLL
    for (int i = 0; i < tiles; ++i) {
        const int w = valid(i);
        const Raw<T, V> r = get(i);
        if (UNI) {  // all of the vector or nothing of it: its own moments, then joined
            float v[V], sum = 0.0f, m2 = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[j] = float(r[j]) - pivot[0];
                sum += v[j];
            }
            const float mean = sum * (1.0f / V);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = v[j] - mean;
                m2 = __builtin_fmaf(d, d, m2);
            }
            const float share = 1.0f / float(i + 1), d = mean - m[0].mean;
            if (w) {
                m[0].n = float(V * (i + 1));
                m[0].mean = __builtin_fmaf(d, share, m[0].mean);
                m[0].m2 += __builtin_fmaf(d * d, float(V * i) * share, m2);
            }
        } else {  // one value of each channel
            const float share = 1.0f / float(i + 1);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int a = UNI ? 0 : j;
                const float v = float(r[j]) - pivot[a], d = v - m[a].mean;
                const float mean = __builtin_fmaf(d, share, m[a].mean);
                m[a].m2 = j < w ? __builtin_fmaf(d, v - mean, m[a].m2) : m[a].m2;
                m[a].mean = j < w ? mean : m[a].mean;
                m[a].n = j < w ? float(i + 1) : m[a].n;
            }
        }
    }
}

// Joins the block's triples of each group and calls out(group of the slab, moments), on one
// thread a group.
template <int V, bool UNI, class Out>
__device__ __forceinline__ void join_block(const OneCut &k, const HeldPlace<V> &pl, const OwnMoments<UNI, V> &m, JoinBuffer<UNI, V> &lds,
                                           Out out)
{
    constexpr int A = kOwn<UNI, V>, unit = UNI ? V : 1;  // elements a triple stands for
    __syncthreads();
    if (pl.active) {
#pragma unroll
        for (int a = 0; a < A; ++a) {
            lds[0][threadIdx.x * A + a] = m[a].n;
            lds[1][threadIdx.x * A + a] = m[a].mean;
            lds[2][threadIdx.x * A + a] = m[a].m2;
        }
    }
    __syncthreads();
    const int per = k.Cg / unit, row = k.width / unit, lane = threadIdx.x & (k.lanes - 1);
    for (int g = int(threadIdx.x) / k.lanes; g < k.groups; g += kHeld / k.lanes) {
        Moments s;
        for (int i = lane; i < per * k.rows; i += k.lanes) {
            const int r = i / per, at = r * row + g * per + (i - r * per);
            s.join(lds[0][at], lds[1][at], lds[2][at]);
        }
        for (int o = 1; o < k.lanes; o *= 2) s.join(__shfl_xor(s.n, o), __shfl_xor(s.mean, o), __shfl_xor(s.m2, o));
        if (lane == 0) out(g, s);
    }
}

template <class T, int V, bool UNI, int K, class ACT>
__global__ __launch_bounds__(kHeld, 4) void held_kernel(const T *x, OneCut k, float eps, ct::Param<T> gamma, ct::Param<T> beta,
                                                        ACT f, Dropout drop, unsigned long long *words, T *y,
                                                        float *mean, float *rstd)
{
    constexpr int A = kOwn<UNI, V>;
    __shared__ float lds[3][kHeld * A];
    __shared__ float2 stat[kMostGroups];
    const HeldPlace<V> pl(k, blockIdx.x);
    auto tile = [&](int i) { return pl.tile(k, pl.chunk, i); };
    const bool full = pl.full(k, pl.chunk) && k.tiles == K;
    Bits raw[K];
    if (full) {
#pragma unroll
        for (int i = 0; i < K; ++i)
            raw[i] = __builtin_bit_cast(Bits, *reinterpret_cast<const Raw<T, V> *>(x + tile(i) + pl.off));
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i)
            raw[i] = __builtin_bit_cast(Bits, load_first<T, V>(x + tile(i) + pl.off, pl.valid(k, pl.chunk, i)));
    }
    const int g_first = pl.slab * k.groups;
    float pivot[A];
#pragma unroll
    for (int a = 0; a < A; ++a)
        pivot[a] = float(x[pl.n * k.P * k.C + int64_t(g_first + (UNI ? pl.col : (pl.col + a) % k.width) / k.Cg) * k.Cg]);
    Moments m[A];
    own_moments<T, V, UNI, K>(m, pivot, K, [&](int i) { return held<T>(raw[i]); },
                              [&](int i) { return full ? (pl.active ? V : 0) : pl.valid(k, pl.chunk, i); });

    const int64_t first_group = pl.n * k.G + g_first;
    unsigned keep[K / 4];
    auto draw_all = [&]() { draw<V, K>(keep, drop, [&](int i) { return tile(i) + pl.off; }); };
    auto finish = [&](int g, const Moments &s) {
        const float mu = float(x[pl.n * k.P * k.C + int64_t(g_first + g) * k.Cg]) + s.mean, r = 1.0f / sqrtf(s.m2 / s.n + eps);
        stat[g] = make_float2(mu, r);
        if (pl.chunk == 0) {
            if (mean) mean[first_group + g] = mu;
            if (rstd) rstd[first_group + g] = r;
        }
    };
    if (k.chunks == 1) {
        join_block<V, UNI>(k, pl, m, lds, finish);
        draw_all();
    } else {
        unsigned long long *const mine = words + first_group * k.chunks;
        auto send = [&](int q) { return [&, q](int g, const Moments &s) { publish(mine + int64_t(g) * k.chunks + q, s.mean, s.m2); }; };
        join_block<V, UNI>(k, pl, m, lds, send(pl.chunk));
        draw_all();  // while the words are on their way
        const int64_t span = int64_t(k.tiles) * k.rows;
        Moments s;
        gather_words<kHeld>(
            k, mine, [&](int) { s = Moments(); },
            [&](int, unsigned long long w, int q) {
                const int64_t left = k.P - q * span;
                s.join(float(k.Cg) * float(left < span ? left : span), low2(w), high2(w));
            },
            [&](int g, int lane) {
                for (int o = 1; o < k.lanes; o *= 2) s.join(__shfl_xor(s.n, o), __shfl_xor(s.mean, o), __shfl_xor(s.m2, o));
                if (lane == 0) finish(g, s);
            },
            [&](int q) {
                auto valid = [&](int i) { return pl.valid(k, q, i); };
                Moments t[A];
                own_moments<T, V, UNI, 1>(t, pivot, k.tiles, [&](int i) { return load_first<T, V>(x + pl.tile(k, q, i) + pl.off, valid(i)); },
                                          valid);
                join_block<V, UNI>(k, pl, t, lds, send(q));
            });
    }
    __syncthreads();
    if (!pl.active) return;
    float mu[A], rs[A], ga[V], be[V];
#pragma unroll
    for (int a = 0; a < A; ++a) {
        const float2 v = stat[(UNI ? pl.col : (pl.col + a) % k.width) / k.Cg];
        mu[a] = v.x;
        rs[a] = v.y;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = pl.c0 + (UNI ? pl.col + j : (pl.col + j) % k.width);
        ga[j] = gamma.at(c, 1.0f) * rs[UNI ? 0 : j];
        be[j] = beta.at(c, 0.0f);
    }
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int valid = full ? V : pl.valid(k, pl.chunk, i);
        if (valid == 0) continue;
        const Raw<T, V> v = held<T>(raw[i]);
        Raw<T, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float r = f.y((float(v[j]) - mu[UNI ? 0 : j]) * ga[j] + be[j]);
            o[j] = T(stays(keep, i, j) ? r * drop.factor : 0.0f);
        }
        store_first<T, V>(y + tile(i) + pl.off, o, valid);
        one_by_one();
    }
}

}  // namespace

void ct::norm::launch_held(const Call &c, const OneCut &k, bool uni, int64_t blocks, hipStream_t st)
{
    ct::with_type(c.dt, [&](auto t) {
        using T = decltype(t);
        constexpr int V = ct::kVec<T>;
        const ct::Param<T> gamma{c.gamma, c.params_f32}, beta{c.beta, c.params_f32};
        with_act(c.act, [&](auto f) {
            using F = decltype(f);
            auto go = [&](auto u, auto tiles) {
                held_kernel<T, V, decltype(u)::value, decltype(tiles)::value, F><<<unsigned(blocks), kHeld, 0, st>>>(
                    static_cast<const T *>(c.x), k, c.eps, gamma, beta, f, c.drop, c.words, static_cast<T *>(c.y), c.mean, c.rstd);
            };
            with_instance<false>(k, uni, go);
        });
    });
}

// ct_groupnorm_held_grad.hip -- the gradient of group norm in one pass over x and dy (see
// ct_groupnorm.hpp).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ct_groupnorm.hpp"

namespace {

using namespace ct::norm;
using ct::Dropout;
using ct::Raw;

// The gradient likewise: x and dy are held; the exchanged words are the chunk's
// (sum dz gamma, sum dz gamma xhat).  sums[n][chunk][c] = (sum dz, sum dz xhat) for the
// parameters' gradients.
template <class T, int V, bool UNI, int K, class ACT>
__global__ __launch_bounds__(kHeldGrad, 2) void held_grad_kernel(const T *dy, const T *x, OneCut k, const float *mean,
                                                             const float *rstd, ct::Param<T> gamma, ct::Param<T> beta,
                                                             ACT f, Dropout drop, unsigned long long *words,
                                                             float2 *sums, T *dx)
{
    constexpr int A = kOwn<UNI, V>;
    __shared__ float2 lds[kHeldGrad * V];
    __shared__ float2 coef[kMostGroups];
    const HeldPlace<V> pl(k, blockIdx.x);
    auto tile = [&](int i) { return pl.tile(k, pl.chunk, i); };
    const bool full = pl.full(k, pl.chunk) && k.tiles == K;
    Bits xr[K], dr[K];
    if (full) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            xr[i] = __builtin_bit_cast(Bits, *reinterpret_cast<const Raw<T, V> *>(x + tile(i) + pl.off));
            dr[i] = __builtin_bit_cast(Bits, *reinterpret_cast<const Raw<T, V> *>(dy + tile(i) + pl.off));
        }
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int valid = pl.valid(k, pl.chunk, i);
            xr[i] = __builtin_bit_cast(Bits, load_first<T, V>(x + tile(i) + pl.off, valid));
            dr[i] = __builtin_bit_cast(Bits, load_first<T, V>(dy + tile(i) + pl.off, valid));
        }
    }
    const int g_first = pl.slab * k.groups;
    const int64_t first_group = pl.n * k.G + g_first;
    float mu[A], rs[A], ga[V], be[V];
#pragma unroll
    for (int a = 0; a < A; ++a) {
        const int64_t g = first_group + (UNI ? pl.col : (pl.col + a) % k.width) / k.Cg;
        mu[a] = mean[g];
        rs[a] = rstd[g];
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = pl.c0 + (UNI ? pl.col + j : (pl.col + j) % k.width);
        ga[j] = gamma.at(c, 1.0f);
        be[j] = beta.at(c, 0.0f);
    }
    unsigned keep[K / 4];
    draw<V, K>(keep, drop, [&](int i) { return tile(i) + pl.off; });  // while the values are on their way
    // (sum dz, sum dz xhat) of the thread's channels, over the tiles of a chunk; elements that do
    // not exist are zeros in dy and add nothing
    auto own_sums = [&](auto unroll, int tiles, float (&s1)[V], float (&s2)[V], auto get_x, auto get_dy, auto bits) {
        constexpr int UNROLL = decltype(unroll)::value;
#pragma unroll UNROLL
        for (int i = 0; i < tiles; ++i) {
            const Raw<T, V> xv = get_x(i), dv = get_dy(i);
            const unsigned b = bits(i);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = (float(xv[j]) - mu[UNI ? 0 : j]) * rs[UNI ? 0 : j];
                const float e = (b >> j) & 1 ? float(dv[j]) * drop.factor : 0.0f;
                const float dz = e * f.d(__builtin_fmaf(xh, ga[j], be[j]));
                s1[j] += dz;
                s2[j] = __builtin_fmaf(dz, xh, s2[j]);
            }
            one_by_one();
        }
    };
    // the block's channel sums in lds[channel of the slab], its group sums to out
    auto join = [&](const float (&s1)[V], const float (&s2)[V], auto out) {
        __syncthreads();
        if (pl.active)
#pragma unroll
            for (int j = 0; j < V; ++j) lds[pl.e + j] = make_float2(s1[j], s2[j]);
        __syncthreads();
        for (int c = threadIdx.x; c < k.width; c += kHeldGrad) {
            float2 s = lds[c];
            for (int r = 1; r < k.rows; ++r) {
                const float2 v = lds[r * k.width + c];
                s.x += v.x;
                s.y += v.y;
            }
            lds[c] = s;  // nobody else reads this column
        }
        __syncthreads();
        const int lane = threadIdx.x & (k.lanes - 1);
        for (int g = int(threadIdx.x) / k.lanes; g < k.groups; g += kHeldGrad / k.lanes) {
            float a = 0.0f, b = 0.0f;
            for (int c = lane; c < k.Cg; c += k.lanes) {
                const float2 v = lds[g * k.Cg + c];
                const float w = gamma.at(pl.c0 + g * k.Cg + c, 1.0f);
                a = __builtin_fmaf(v.x, w, a);
                b = __builtin_fmaf(v.y, w, b);
            }
            for (int o = 1; o < k.lanes; o *= 2) {
                a += __shfl_xor(a, o);
                b += __shfl_xor(b, o);
            }
            if (lane == 0) out(g, a, b);
        }
    };
    float s1[V] = {}, s2[V] = {};
    own_sums(std::integral_constant<int, K>{}, K, s1, s2, [&](int i) { return held<T>(xr[i]); },
             [&](int i) { return held<T>(dr[i]); },
             [&](int i) { return keep[i / 4] >> (8 * (i % 4)); });
    const float count = float(k.P) * float(k.Cg);
    auto finish = [&](int g, float a, float b) { coef[g] = make_float2(a / count, b / count); };
    auto store_sums = [&]() {
        for (int c = threadIdx.x; c < k.width; c += kHeldGrad) sums[(pl.n * k.chunks + pl.chunk) * k.C + pl.c0 + c] = lds[c];
    };
    if (k.chunks == 1) {
        join(s1, s2, finish);
        store_sums();
    } else {
        unsigned long long *const mine = words + first_group * k.chunks;
        auto send = [&](int q) { return [&, q](int g, float a, float b) { publish(mine + int64_t(g) * k.chunks + q, a, b); }; };
        join(s1, s2, send(pl.chunk));
        store_sums();
        float a = 0.0f, b = 0.0f;
        gather_words<kHeldGrad>(
            k, mine, [&](int) { a = b = 0.0f; },
            [&](int, unsigned long long w, int) {
                a += low2(w);
                b += high2(w);
            },
            [&](int g, int lane) {
                for (int o = 1; o < k.lanes; o *= 2) {
                    a += __shfl_xor(a, o);
                    b += __shfl_xor(b, o);
                }
                if (lane == 0) finish(g, a, b);
            },
            [&](int q) {
                float t1[V] = {}, t2[V] = {};
                auto from = [&](const T *p, int i) { return load_first<T, V>(p + pl.tile(k, q, i) + pl.off, pl.valid(k, q, i)); };
                own_sums(std::integral_constant<int, 1>{}, k.tiles, t1, t2, [&](int i) { return from(x, i); },
                         [&](int i) { return from(dy, i); },
                         [&](int i) {
                             const uint64_t first = uint64_t(pl.tile(k, q, i) + pl.off);
                             return drop.threshold ? ct::keep_bits<V>(drop, drop.counter(), first) : 0xffu;
                         });
                join(t1, t2, send(q));
            });
    }
    __syncthreads();
    if (!pl.active) return;
    float c1[A], c2[A];
#pragma unroll
    for (int a = 0; a < A; ++a) {
        const float2 v = coef[(UNI ? pl.col : (pl.col + a) % k.width) / k.Cg];
        c1[a] = v.x;
        c2[a] = v.y;
    }
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int valid = full ? V : pl.valid(k, pl.chunk, i);
        if (valid == 0) continue;
        const Raw<T, V> xv = held<T>(xr[i]), dv = held<T>(dr[i]);
        Raw<T, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int a = UNI ? 0 : j;
            const float xh = (float(xv[j]) - mu[a]) * rs[a];
            const float e = stays(keep, i, j) ? float(dv[j]) * drop.factor : 0.0f;
            const float dz = e * f.d(__builtin_fmaf(xh, ga[j], be[j]));
            o[j] = T(rs[a] * (dz * ga[j] - c1[a] - xh * c2[a]));
        }
        store_first<T, V>(dx + tile(i) + pl.off, o, valid);
        one_by_one();
    }
}

}  // namespace

void ct::norm::launch_held_grad(const Call &c, const OneCut &k, bool uni, int64_t blocks, hipStream_t st)
{
    ct::with_type(c.dt, [&](auto t) {
        using T = decltype(t);
        constexpr int V = ct::kVec<T>;
        const ct::Param<T> gamma{c.gamma, c.params_f32}, beta{c.beta, c.params_f32};
        with_act(c.act, [&](auto f) {
            using F = decltype(f);
            auto go = [&](auto u, auto tiles) {
                held_grad_kernel<T, V, decltype(u)::value, decltype(tiles)::value, F><<<unsigned(blocks), kHeldGrad, 0, st>>>(
                    static_cast<const T *>(c.dy), static_cast<const T *>(c.x), k, c.mean, c.rstd, gamma, beta, f, c.drop, c.words,
                    c.sums, static_cast<T *>(c.dx));
            };
            with_instance<true>(k, uni, go);
        });
    });
}

// ct_rotary.hip -- rotary positions with several axes.
//
// Pair p of a head's 2 R turning elements (x0, x1) goes by axis a(p) and becomes
//   (x0 cos A - x1 sin A, x0 sin A + x1 cos A),   A = position[a(p)] * base^(-e(p)),
// the gradient (inverse) the same with -A.
//
// The angle is kept in turns as a 64-bit fraction: position (an integer) times base^(-e) / 2 pi in
// units of 2^-64 wraps by itself, so a far position loses nothing; float32 products would be off
// by 0.06 at a position of a million.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <string>
#include <type_traits>

#include "ct_vec.hpp"

namespace {

using ct::Raw;

constexpr int kThreads = 256, kMaxPairs = 256, kFewPairs = 64, kMaxAxes = 4, AHEAD = 2;

// The table of angles is an argument of the launch, whose time grows with its arguments: up to 64 pairs have
// a kernel of their own.
template <int PAIRS>
struct Rotary {
    const void *x;
    void *y;
    int64_t xn, xt, xh, yn, yt, yh, pn, pt;  // strides in elements
    const void *positions;
    int64_t tokens, T;           // N * T, T
    int H, D, pairs, head_run;   // head_run: heads a thread turns
    int units;                   // threads along a head: runs of V pairs, then of 2 V elements that stay
    int inverse;
    int axis_end[kMaxAxes];      // pairs up to the end of an axis
    uint64_t turn[PAIRS];
};

// One thread keeps the sines and cosines of V pairs of one token and turns them in `head_run` heads.  Bound by memory
// where there is much: 2 x 16384 tokens, 20 heads of 128, bfloat16, 336 MB in 71 us, 4.7 TB/s, where a copy of as many
// bytes runs at 5.4; a token of 8 sequences, 10 heads of 64: 5.4 us, a launch whose arguments hold the table (4.4 for
// one without) and a chain of position, sine and store.  Four heads on their way instead of two: 32768 tokens, 16 heads
// of 64, 31.1 -> 27.2 us, but 16382 tokens, 32 heads of 128, 53.9 -> 60.5.
template <class T, class I, bool BY_TWOS, int PAIRS>
__global__ __launch_bounds__(kThreads) void rotary_kernel(Rotary<PAIRS> a)
{
    constexpr int V = ct::kVec<T>;
    const int64_t id = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    const int runs = (a.H + a.head_run - 1) / a.head_run;
    const int unit = int(id % a.units);
    const int64_t rest = id / a.units, token = rest / runs;
    if (token >= a.tokens) return;
    const int h0 = int(rest % runs) * a.head_run, h1 = min(h0 + a.head_run, a.H);
    const int64_t n = token / a.T, t = token % a.T;
    const T *x = static_cast<const T *>(a.x) + n * a.xn + t * a.xt;
    T *y = static_cast<T *>(a.y) + n * a.yn + t * a.yt;

    const int turning = (a.pairs + V - 1) / V;
    auto load = [](const T *p, int valid) {
        Raw<T, V> r = {};
        if (valid >= V) return *reinterpret_cast<const Raw<T, V> *>(p);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < valid) r[j] = p[j];
        return r;
    };
    auto store = [](T *p, int valid, const Raw<T, V> &r) {
        if (valid >= V) {
            *reinterpret_cast<Raw<T, V> *>(p) = r;
            return;
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < valid) p[j] = r[j];
    };
    if (unit >= turning) {  // behind the pairs: copied
        const int d = 2 * a.pairs + (unit - turning) * 2 * V;
        for (int h = h0; h < h1; ++h) {
            const Raw<T, V> u = load(x + h * a.xh + d, a.D - d), w = load(x + h * a.xh + d + V, a.D - d - V);
            store(y + h * a.yh + d, a.D - d, u);
            store(y + h * a.yh + d + V, a.D - d - V, w);
        }
        return;
    }
    const int p0 = unit * V, count = min(V, a.pairs - p0);
    const int d0 = BY_TWOS ? 2 * p0 : p0, d1 = BY_TWOS ? 2 * p0 + V : p0 + a.pairs;
    const int n0 = BY_TWOS ? 2 * count : count, n1 = BY_TWOS ? 2 * count - V : count;
    // the first heads' loads go out before the sines and cosines are made, the next ones' before these are turned
    Raw<T, V> u[AHEAD], w[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (h0 + i < h1) {
            u[i] = load(x + (h0 + i) * a.xh + d0, n0);
            w[i] = load(x + (h0 + i) * a.xh + d1, n1);
        }
    const I *position = static_cast<const I *>(a.positions) + n * a.pn + t * a.pt;
    float c[V], s[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int p = min(p0 + j, a.pairs - 1);
        int axis = 0;
#pragma unroll
        for (int i = 0; i < kMaxAxes - 1; ++i) axis += p >= a.axis_end[i];
        const uint64_t turn = uint64_t(int64_t(position[axis])) * a.turn[p];
        // half turns in [-1, 1)
        const float half_turns = float(int32_t(turn >> 32)) * 0x1p-31f;
        sincospif(half_turns, &s[j], &c[j]);
        if (a.inverse) s[j] = -s[j];
    }
    for (int h = h0; h < h1; h += AHEAD) {
        Raw<T, V> un[AHEAD], wn[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (h + AHEAD + i < h1) {
                un[i] = load(x + (h + AHEAD + i) * a.xh + d0, n0);
                wn[i] = load(x + (h + AHEAD + i) * a.xh + d1, n1);
            }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (h + i >= h1) break;
            Raw<T, V> uo, wo;
            if constexpr (BY_TWOS) {
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    const float a0 = float(u[i][2 * j]), b0 = float(u[i][2 * j + 1]), a1 = float(w[i][2 * j]), b1 = float(w[i][2 * j + 1]);
                    const int k = V / 2 + j;
                    uo[2 * j] = T(a0 * c[j] - b0 * s[j]);
                    uo[2 * j + 1] = T(a0 * s[j] + b0 * c[j]);
                    wo[2 * j] = T(a1 * c[k] - b1 * s[k]);
                    wo[2 * j + 1] = T(a1 * s[k] + b1 * c[k]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float a0 = float(u[i][j]), b0 = float(w[i][j]);
                    uo[j] = T(a0 * c[j] - b0 * s[j]);
                    wo[j] = T(a0 * s[j] + b0 * c[j]);
                }
            }
            store(y + (h + i) * a.yh + d0, n0, uo);
            store(y + (h + i) * a.yh + d1, n1, wo);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) u[i] = un[i], w[i] = wn[i];
    }
}

ct_status fail(ct_status st, const std::string &msg)
{
    ct::set_last_error(msg);
    return st;
}

}  // namespace

extern "C" ct_status rotary_nd(ct_dtype dtype, const int64_t *shape, const void *x, const int64_t *x_strides,
                               ct_dtype position_dtype, int axes, const void *positions, const int64_t *position_strides,
                               const int64_t *sections, double base, int whole_ladder, int interleaved, int inverse, void *y,
                               const int64_t *y_strides, void *stream)
{
    ct::set_last_error(std::string());
    const int dt = ct::enum_int(dtype), pt = ct::enum_int(position_dtype);
    if (!ct::is_float_type(dt)) return fail(CT_EUNSUPPORTED, "dtype must be CT_FLOAT32, CT_FLOAT16 or CT_BFLOAT16");
    if (pt != CT_INT32 && pt != CT_INT64) return fail(CT_EUNSUPPORTED, "position_dtype must be CT_INT32 or CT_INT64");
    if (!shape || !sections || !x_strides || !y_strides || !position_strides)
        return fail(CT_EINVAL, "shape, sections or strides are NULL");
    if (axes < 1 || axes > kMaxAxes) return fail(CT_EINVAL, "there must be 1 to 4 axes");
    for (int i = 0; i < 4; ++i)
        if (shape[i] < 0) return fail(CT_EINVAL, "sizes must not be negative");
    constexpr int64_t most = int64_t(1) << 31;
    if (shape[0] >= most || shape[1] >= most || shape[2] >= most || shape[3] >= most ||
        (shape[1] && shape[0] >= most / shape[1]) ||
        (shape[3] && (shape[2] >= most / shape[3])))
        return fail(CT_EUNSUPPORTED, "more than 2^31 tokens or elements of a token");
    // (the sum of two counts of heads is an int)
    if (shape[2] > most / 2) return fail(CT_EUNSUPPORTED, "more than 2^30 heads are not served");
    for (int i = 0; i < 3; ++i)
        if (x_strides[i] < 0 || y_strides[i] < 0 || x_strides[i] > (int64_t(1) << 40) || y_strides[i] > (int64_t(1) << 40))
            return fail(CT_EINVAL, "strides must lie in 0 .. 2^40");
    for (int i = 0; i < 2; ++i)
        if (position_strides[i] < 0 || position_strides[i] > (int64_t(1) << 40))
            return fail(CT_EINVAL, "strides must lie in 0 .. 2^40");
    if (!(base > 0.0 && base <= 1e300)) return fail(CT_EINVAL, "base must be positive and finite");
    if ((whole_ladder != 0 && whole_ladder != 1) || (interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1))
        return fail(CT_EINVAL, "whole_ladder, interleaved and inverse must be 0 or 1");
    Rotary<kMaxPairs> a{};
    int64_t pairs = 0;
    for (int i = 0; i < axes; ++i) {
        if (sections[i] < 0 || sections[i] > kMaxPairs) return fail(CT_EINVAL, "a section must have 0 to 256 pairs");
        pairs += sections[i];
        a.axis_end[i] = int(pairs);
    }
    for (int i = axes; i < kMaxAxes; ++i) a.axis_end[i] = int(pairs);
    if (pairs > kMaxPairs) return fail(CT_EUNSUPPORTED, "more than 256 pairs are not served");
    if (2 * pairs > shape[3]) return fail(CT_EINVAL, "the sections have more pairs than half a head's elements");
    const size_t esz = ct::float_size(dt);
    if (!ct::aligned_to(x, esz) || !ct::aligned_to(y, esz) || !ct::aligned_to(positions, pt == CT_INT32 ? 4 : 8))
        return fail(CT_EINVAL, "tensor pointers must be aligned to the element size");
    if (shape[0] == 0 || shape[1] == 0 || shape[2] == 0 || shape[3] == 0) return CT_OK;
    if (!x || !y || !positions) return fail(CT_EINVAL, "x, y or positions is NULL");

    const long double two_pi = 6.283185307179586476925286766559L;
    int p = 0;
    // turns a position, without whole ones (a position is an integer); each from the one before, which
    // costs 256 roundings of 2^-64 at most and one power an axis instead of one a pair
    long double e = 0.0L;
    for (int i = 0; i < axes; ++i) {
        const long double ratio = sections[i] ? powl((long double)base, -1.0L / (whole_ladder ? pairs : sections[i])) : 1.0L;
        if (i == 0 || !whole_ladder) e = 1.0L / two_pi;
        for (int j = 0; j < int(sections[i]); ++j, ++p, e *= ratio) {
            const long double f = (e < 1.0L ? e : fmodl(e, 1.0L)) * 0x1p64L;
            a.turn[p] = f >= 0x1p64L - 1.0L ? ~uint64_t(0) : uint64_t(f + 0.5L);
        }
    }
    a.x = x;
    a.y = y;
    a.xn = x_strides[0], a.xt = x_strides[1], a.xh = x_strides[2];
    a.yn = y_strides[0], a.yt = y_strides[1], a.yh = y_strides[2];
    a.pn = position_strides[0], a.pt = position_strides[1];
    a.positions = positions;
    a.T = shape[1];
    a.tokens = shape[0] * shape[1];
    a.H = int(shape[2]);
    a.D = int(shape[3]);
    a.pairs = int(pairs);
    a.inverse = inverse;
    const int V = esz == 4 ? 4 : 8;
    const int64_t stay = shape[3] - 2 * pairs;
    a.units = int((pairs + V - 1) / V + (stay + 2 * V - 1) / (2 * V));
    // a thread turns several heads with the sines and cosines it has, as long as the threads fill the chip
    a.head_run = 1;
    while (a.head_run < a.H && a.tokens * a.units * ((a.H + 2 * a.head_run - 1) / (2 * a.head_run)) >= 512 * 1024) a.head_run *= 2;
    // equal shares: 20 heads as 10 and 10, not 16 and 4 (2 x 16384 tokens of 128: 71.2 us for 74.6)
    const int runs = (a.H + a.head_run - 1) / a.head_run;
    a.head_run = (a.H + runs - 1) / runs;
    const int64_t threads = a.tokens * a.units * ((a.H + a.head_run - 1) / a.head_run);
    if (threads >= int64_t(1) << 32) return fail(CT_EUNSUPPORTED, "too many tokens and heads for one launch");
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    ct::mark_before(hs);
    ct::with_type(dt, [&](auto t) {
        using T = decltype(t);
        auto launch = [&](auto i, auto twos, const auto &args) {
            constexpr int P = int(sizeof(args.turn) / sizeof(args.turn[0]));
            rotary_kernel<T, decltype(i), decltype(twos)::value, P>
                <<<unsigned((threads + kThreads - 1) / kThreads), kThreads, 0, hs>>>(args);
        };
        auto go = [&](auto i, auto twos) {
            if (a.pairs <= kFewPairs) {
                Rotary<kFewPairs> few;
                std::memcpy(static_cast<void *>(&few), &a, sizeof few);  // the table is the last member
                launch(i, twos, few);
            } else {
                launch(i, twos, a);
            }
        };
        if (pt == CT_INT32) interleaved ? go(int32_t{}, std::true_type{}) : go(int32_t{}, std::false_type{});
        else interleaved ? go(int64_t{}, std::true_type{}) : go(int64_t{}, std::false_type{});
    });
    ct::mark_after(hs);
    std::string err;
    const ct_status ls = ct::launch_status("rotary launch failed", &err);
    return ls == CT_OK ? CT_OK : fail(ls, err);
}

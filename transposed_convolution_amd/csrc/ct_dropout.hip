// ct_dropout.hip -- dropout with a counter-based generator, optionally added to a residual.
//
//   y[i] = (residual[i] +) (keep(i) ? factor * x[i] : 0)
//
// keep(i) depends on (seed, offset, i) alone (see ct_vec.hpp), so no mask is stored: the
// gradient of x is the same call on the gradient of y, with the same seed and offset.
#include <hip/hip_runtime.h>

#include <string>
#include <type_traits>

#include "ct_vec.hpp"

namespace {

using ct::Dropout;
using ct::Raw;

constexpr int kThreads = 256;

// One thread makes the eight elements of one generator block: the loads go out first and the
// generator runs while they are on their way.  Bound by memory: with a residual, 33.5 M
// float16 elements (201 MB) take 36 us, 5.6 TB/s, a copy's rate; the vector units, ten rounds
// for eight elements and one compare and select each, are 42 % busy meanwhile.  Streaming
// stores gained nothing (float32: 26 us became 30).
template <class T, bool RES, bool DROP>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const T *x, const T *res, T *y, int64_t count, Dropout d)
{
    constexpr int V = ct::kVec<T>;
    const uint64_t counter = DROP ? d.counter() : 0;
    const uint32_t limit = d.limit();
    for (int64_t b = int64_t(blockIdx.x) * kThreads + threadIdx.x; b * 8 < count; b += int64_t(gridDim.x) * kThreads) {
        const int64_t i = b * 8;
        if (count - i >= 8) {
            Raw<T, V> v[8 / V], r[8 / V], o;
#pragma unroll
            for (int h = 0; h < 8 / V; ++h) {
                v[h] = *reinterpret_cast<const Raw<T, V> *>(x + i + h * V);
                if (RES) r[h] = *reinterpret_cast<const Raw<T, V> *>(res + i + h * V);
            }
            const ct::Fields f = DROP ? ct::draw_fields<8, true>(d, counter, uint64_t(i)) : ct::Fields{};
#pragma unroll
            for (int h = 0; h < 8 / V; ++h) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    // a select, not a product: what is dropped may be anything
                    const float t = !DROP ? float(v[h][j]) : f.stays(h * V + j, limit) ? float(v[h][j]) * d.factor : 0.0f;
                    o[j] = T(RES ? float(r[h][j]) + t : t);
                }
                *reinterpret_cast<Raw<T, V> *>(y + i + h * V) = o;
            }
        } else {
            const ct::Fields f = DROP ? ct::draw_fields<8, true>(d, counter, uint64_t(i)) : ct::Fields{};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j >= count - i) break;
                const float t = !DROP ? float(x[i + j]) : f.stays(j, limit) ? float(x[i + j]) * d.factor : 0.0f;
                y[i + j] = T(RES ? float(res[i + j]) + t : t);
            }
        }
    }
}

ct_status fail(ct_status st, const std::string &msg)
{
    ct::set_last_error(msg);
    return st;
}

}  // namespace

extern "C" ct_status dropout_nd(ct_dtype dtype, int64_t count, const void *x, const void *residual, void *y, double p,
                                uint64_t seed, uint64_t offset, const uint64_t *step, void *stream)
{
    ct::set_last_error(std::string());
    const int dt = ct::enum_int(dtype);
    if (!ct::is_float_type(dt)) return fail(CT_EUNSUPPORTED, "dtype must be CT_FLOAT32, CT_FLOAT16 or CT_BFLOAT16");
    if (count < 0) return fail(CT_EINVAL, "count must not be negative");
    Dropout d;
    std::string err;
    const ct_status st = ct::make_dropout(p, seed, offset, step, &d, &err);
    if (st != CT_OK) return fail(st, err);
    const size_t esz = ct::float_size(dt);
    if (!ct::aligned_to(x, esz) || !ct::aligned_to(residual, esz) || !ct::aligned_to(y, esz))
        return fail(CT_EINVAL, "tensor pointers must be aligned to the element size");
    if (count == 0) return CT_OK;
    if (!x || !y) return fail(CT_EINVAL, "x or y is NULL");
    // a launch holds fewer than 2^32 threads: beyond that the blocks go round again
    const int64_t want = (count / 8 + kThreads) / kThreads, blocks = want < (1 << 23) ? want : 1 << 23;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    ct::mark_before(hs);
    ct::with_type(dt, [&](auto t) {
        using T = decltype(t);
        const T *xp = static_cast<const T *>(x), *rp = static_cast<const T *>(residual);
        auto go = [&](auto r, auto dr) {
            dropout_kernel<T, decltype(r)::value, decltype(dr)::value>
                <<<unsigned(blocks), kThreads, 0, hs>>>(xp, rp, static_cast<T *>(y), count, d);
        };
        constexpr std::true_type yes{};
        constexpr std::false_type no{};
        if (residual && d.threshold) go(yes, yes);
        else if (residual) go(yes, no);
        else if (d.threshold) go(no, yes);
        else go(no, no);
    });
    ct::mark_after(hs);
    const ct_status ls = ct::launch_status("dropout launch failed", &err);
    return ls == CT_OK ? CT_OK : fail(ls, err);
}

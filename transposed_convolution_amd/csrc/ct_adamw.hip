// ct_adamw.hip -- an AdamW step (Loshchilov, Hutter 2019) over many tensors at once.
//
//   g = grad_scale * gradient,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr decay) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// in float32, one rounding into each output.  States in 8 bits are e4m3 values with a float32 scale
// for 256 consecutive elements (of m, and of the root of v, whose range e4m3 holds twice over);
// the step itself takes the new states before they are rounded.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "ct_vec.hpp"

namespace {

using ct::Raw;

constexpr int kThreads = 256, kScaleBlock = 256;
// Tensors a launch takes: their descriptions are its arguments (below 4 KB), and a launch with few arguments is
// quicker.
constexpr int kEntries = 40, kFewEntries = 8;
constexpr int kRun32 = 1024, kRun8 = 2048;  // elements a block updates
constexpr float kTop = 448.0f, kLeastScale = 0x1p-126f, kLeastCode = 0x1p-9f;

struct Entry {
    void *p;
    const void *g;
    void *m, *v;
    float *m_scale, *v_scale;
    void *copy;
    int64_t count;
    float keep;  // 1 - lr decay, with the host's lr
    float decay;
};

struct Hyper {
    int entries;
    float b1, c1, b2, c2, eps, lr, grad_scale;  // c1 = 1 - b1, c2 = 1 - b2
    float first_bias, second_root;              // 1 - b1^t and 1 / sqrt(1 - b2^t) of a host step
    double log_b1, log_b2;
    const int64_t *step;
    const float *lr_at, *scale_at;  // device values in place of lr and grad_scale, or null
    int copy_type;
};
template <int N>
struct Step : Hyper {
    unsigned first[N + 1];  // first block of each tensor
    Entry e[N];
};

// lr / (1 - b1^t), 1 / sqrt(1 - b2^t), grad_scale, lr: by one thread a block, behind its loads.
__device__ __forceinline__ void constants(const Hyper &s, float (&out)[4])
{
    float first = s.first_bias, root = s.second_root;
    if (s.step) {
        const double t = double(*s.step);
        first = -expm1f(float(t * s.log_b1));
        root = 1.0f / sqrtf(-expm1f(float(t * s.log_b2)));
    }
    const float lr = s.lr_at ? *s.lr_at : s.lr;
    out[0] = lr / first;
    out[1] = root;
    out[2] = s.scale_at ? *s.scale_at : s.grad_scale;
    out[3] = lr;
}

// m and v as written, in that order and without fused steps, so that a plain float32 form gives the same bits.
__device__ __forceinline__ void moments(const Hyper &s, float g, float &m, float &v)
{
#pragma clang fp contract(off)
    m = m * s.b1 + g * s.c1;
    v = v * s.b2 + (g * g) * s.c2;
}

template <int N>
__device__ __forceinline__ int entry_of(const Step<N> &s, unsigned block)
{
    int lo = 0, hi = s.entries - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.first[mid] <= block) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <class T, int V>
__device__ __forceinline__ Raw<T, V> load(const void *p, int64_t i, int valid)
{
    const T *at = static_cast<const T *>(p) + i;
    if (valid >= V) return *reinterpret_cast<const Raw<T, V> *>(at);
    Raw<T, V> r = {};
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (j < valid) r[j] = at[j];
    return r;
}
template <class T, int V>
__device__ __forceinline__ void store(void *p, int64_t i, int valid, const Raw<T, V> &r)
{
    T *at = static_cast<T *>(p) + i;
    if (valid >= V) {
        *reinterpret_cast<Raw<T, V> *>(at) = r;
        return;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (j < valid) at[j] = r[j];
}
template <int V>
__device__ __forceinline__ void store_copy(const Hyper &s, const Entry &e, int64_t i, int valid, const float (&p)[V])
{
    if (!e.copy) return;
    if (s.copy_type == CT_FLOAT16) {
        Raw<_Float16, V> r;
#pragma unroll
        for (int j = 0; j < V; ++j) r[j] = _Float16(p[j]);
        store<_Float16, V>(e.copy, i, valid, r);
    } else {
        Raw<__bf16, V> r;
#pragma unroll
        for (int j = 0; j < V; ++j) r[j] = __bf16(p[j]);
        store<__bf16, V>(e.copy, i, valid, r);
    }
}

// Bound by memory: 48 tensors of 50 million float32 parameters, bfloat16 gradients and copies, 1.41 GB in 267 us, 5.3 TB/s,
// a copy's rate.  A small call (3 matrices, 3 vectors, 98 496 elements) is a launch: 4.4-5.3 us.
template <class P, class G, int TENSORS>
__global__ __launch_bounds__(kThreads) void adamw32_kernel(Step<TENSORS> s)
{
    constexpr int V = 4, N = kRun32 / (kThreads * V);
    const int k = entry_of(s, blockIdx.x);
    const Entry &e = s.e[k];
    const int64_t from = int64_t(blockIdx.x - s.first[k]) * kRun32 + threadIdx.x * V;
    Raw<P, V> p[N];
    Raw<G, V> g[N];
    Raw<float, V> m[N], v[N];
    int valid[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int64_t i = from + n * (kThreads * V), left = e.count - i;
        valid[n] = left >= V ? V : left > 0 ? int(left) : 0;
        p[n] = load<P, V>(e.p, i, valid[n]);
        g[n] = load<G, V>(e.g, i, valid[n]);
        m[n] = load<float, V>(e.m, i, valid[n]);
        v[n] = load<float, V>(e.v, i, valid[n]);
    }
    __shared__ float shared[4];
    if (threadIdx.x == 0) {
        float c[4];
        constants(s, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) shared[j] = c[j];
    }
    __syncthreads();
    const float rate = shared[0], root = shared[1], gs = shared[2], keep = s.lr_at ? 1.0f - shared[3] * e.decay : e.keep;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int64_t i = from + n * (kThreads * V);
        float out[V];
        Raw<P, V> po;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float mm = m[n][j], vv = v[n][j];
            moments(s, float(g[n][j]) * gs, mm, vv);
            m[n][j] = mm;
            v[n][j] = vv;
            out[j] = float(p[n][j]) * keep - mm / (sqrtf(vv) * root + s.eps) * rate;
            po[j] = P(out[j]);
        }
        store<P, V>(e.p, i, valid[n], po);
        store<float, V>(e.m, i, valid[n], m[n]);
        store<float, V>(e.v, i, valid[n], v[n]);
        store_copy<V>(s, e, i, valid[n], out);
    }
}

// Four e4m3 values in a word, and back.
__device__ __forceinline__ void from_code(unsigned w, float (&x)[4])
{
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
    x[0] = lo[0], x[1] = lo[1], x[2] = hi[0], x[3] = hi[1];
}
__device__ __forceinline__ unsigned to_code(const float (&x)[4])
{
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true);
    return unsigned(w);
}

// The largest magnitudes of a wave's values of x and of y, by their bits: a NaN is above everything.  The halves
// of the wave are exchanged once, then one reduces x and the other y, within rows of 16 lanes by rotations.
__device__ __forceinline__ unsigned top_of(const float (&x)[4])
{
    unsigned t = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) t = max(t, __builtin_bit_cast(unsigned, x[j]) & 0x7fffffffu);
    return t;
}
template <int N>
__device__ __forceinline__ unsigned row_rotate_max(unsigned t)
{
    const unsigned r = unsigned(__builtin_amdgcn_update_dpp(0, int(t), 0x120 + N, 0xf, 0xf, false));
    return max(t, r);
}
__device__ __forceinline__ void wave_tops(const float (&x)[4], const float (&y)[4], float &x_top, float &y_top)
{
    const auto halves = __builtin_amdgcn_permlane32_swap(top_of(x), top_of(y), false, false);
    unsigned t = max(halves[0], halves[1]);
    const auto rows = __builtin_amdgcn_permlane16_swap(t, t, false, false);
    t = max(rows[0], rows[1]);
    t = row_rotate_max<8>(t);
    t = row_rotate_max<4>(t);
    t = row_rotate_max<2>(t);
    t = row_rotate_max<1>(t);
    const int a = __builtin_amdgcn_readlane(int(t), 0), b = __builtin_amdgcn_readlane(int(t), 32);
    x_top = __builtin_bit_cast(float, a);
    y_top = __builtin_bit_cast(float, b);
}
// The scale of values whose largest magnitude is `top` (NaN stays).
__device__ __forceinline__ float scale_of(float top)
{
    const float s = top / kTop;
    return s < kLeastScale ? kLeastScale : s;
}

// x / s from 1 / s, good to a unit (s is 2^-126 at least and 2^120 at most): the product, and its remainder's share.
// A division each would take three times the instructions, and the call is as much bound by them as by memory.
__device__ __forceinline__ float quotient(float x, float s, float inv)
{
    const float q = x * inv;
    return fmaf(fmaf(-q, s, x), inv, q);
}

// m over the denominator: sqrt(v) is at least 2^-75 where v is not 0, so the reciprocal instruction, good to
// a unit, never meets a denormal number.
__device__ __forceinline__ float update(float m, float root_v, float root, float eps, float rate)
{
    return m * __builtin_amdgcn_rcpf(fmaf(root_v, root, eps)) * rate;
}

// A wave updates the 256 elements of a scale at a time, four a lane.  50 million bfloat16 parameters: 506 MB in 108 us,
// 4.7 TB/s.  Bound by the vector unit as much as by memory: an element takes about 70 instructions, a fifth of them its
// square root (139 us with a division an element, 117 with 12 exchanges a wave for the two maxima in place of 6).
template <class P, class G, int TENSORS>
__global__ __launch_bounds__(kThreads) void adamw8_kernel(Step<TENSORS> s)
{
    constexpr int V = 4, WAVES = kThreads / 64, N = kRun8 / (kScaleBlock * WAVES);
    const int k = entry_of(s, blockIdx.x), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Entry &e = s.e[k];
    const int64_t from = int64_t(blockIdx.x - s.first[k]) * kRun8 + wave * kScaleBlock;
    Raw<P, V> p[N];
    Raw<G, V> g[N];
    Raw<unsigned char, V> m8[N], v8[N];
    float ms[N], vs[N];
    int valid[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int64_t b = from + n * (kScaleBlock * WAVES), i = b + lane * V, left = e.count - i;
        valid[n] = left >= V ? V : left > 0 ? int(left) : 0;
        p[n] = load<P, V>(e.p, i, valid[n]);
        g[n] = load<G, V>(e.g, i, valid[n]);
        m8[n] = load<unsigned char, V>(e.m, i, valid[n]);
        v8[n] = load<unsigned char, V>(e.v, i, valid[n]);
        ms[n] = b < e.count ? e.m_scale[b / kScaleBlock] : 0.0f;
        vs[n] = b < e.count ? e.v_scale[b / kScaleBlock] : 0.0f;
    }
    __shared__ float shared[4];
    if (threadIdx.x == 0) {
        float c[4];
        constants(s, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) shared[j] = c[j];
    }
    __syncthreads();
    const float rate = shared[0], root = shared[1], gs = shared[2], keep = s.lr_at ? 1.0f - shared[3] * e.decay : e.keep;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int64_t b = from + n * (kScaleBlock * WAVES), i = b + lane * V;
        if (b >= e.count) break;
        float m[V], r[V], out[V];
        from_code(__builtin_bit_cast(unsigned, m8[n]), m);
        from_code(__builtin_bit_cast(unsigned, v8[n]), r);
        Raw<P, V> po;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float mm = m[j] * ms[n];
            const float rr = r[j] * vs[n];
            float vv = rr * rr;
            moments(s, float(g[n][j]) * gs, mm, vv);
            if (j >= valid[n]) mm = vv = 0.0f;  // behind the tensor's end
            m[j] = mm;
            r[j] = sqrtf(vv);
            out[j] = float(p[n][j]) * keep - update(mm, r[j], root, s.eps, rate);
            po[j] = P(out[j]);
        }
        float m_top, r_top;
        wave_tops(m, r, m_top, r_top);
        const float m_scale = scale_of(m_top), v_scale = scale_of(r_top);
        const float m_inv = __builtin_amdgcn_rcpf(m_scale), v_inv = __builtin_amdgcn_rcpf(v_scale);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const bool some = r[j] > 0.0f;
            m[j] = quotient(m[j], m_scale, m_inv);
            r[j] = quotient(r[j], v_scale, v_inv);
            // a positive root never becomes 0: what is divided by it would grow without bound
            if (some && r[j] < kLeastCode) r[j] = kLeastCode;
        }
        store<P, V>(e.p, i, valid[n], po);
        store<unsigned char, V>(e.m, i, valid[n], __builtin_bit_cast(Raw<unsigned char, V>, to_code(m)));
        store<unsigned char, V>(e.v, i, valid[n], __builtin_bit_cast(Raw<unsigned char, V>, to_code(r)));
        if (lane == 0) {
            e.m_scale[b / kScaleBlock] = m_scale;
            e.v_scale[b / kScaleBlock] = v_scale;
        }
        store_copy<V>(s, e, i, valid[n], out);
    }
}

ct_status fail(ct_status st, const std::string &msg)
{
    ct::set_last_error(msg);
    return st;
}

}  // namespace

extern "C" ct_status adamw_nd(ct_dtype dtype, ct_dtype grad_dtype, int state_bits, ct_dtype copy_dtype, int64_t tensors,
                              const ct_adamw_tensor *list, double lr, const float *lr_device, double beta1, double beta2,
                              double eps, int64_t step, const int64_t *step_device, double grad_scale,
                              const float *grad_scale_device, void *stream)
{
    ct::set_last_error(std::string());
    const int dt = ct::enum_int(dtype), gt = ct::enum_int(grad_dtype), cp = ct::enum_int(copy_dtype);
    if (!ct::is_float_type(dt) || !ct::is_float_type(gt))
        return fail(CT_EUNSUPPORTED, "dtype and grad_dtype must be CT_FLOAT32, CT_FLOAT16 or CT_BFLOAT16");
    if (state_bits != 8 && state_bits != 32) return fail(CT_EUNSUPPORTED, "state_bits must be 8 or 32");
    if (tensors < 0) return fail(CT_EINVAL, "the number of tensors must not be negative");
    if (tensors && !list) return fail(CT_EINVAL, "the list of tensors is NULL");
    if (!std::isfinite(float(lr)) || !std::isfinite(float(grad_scale))) return fail(CT_EINVAL, "lr and grad_scale must be finite");
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0)) return fail(CT_EINVAL, "the betas must lie in [0, 1)");
    // (the update's reciprocal takes no denormal number)
    if (!(eps == 0.0 || (eps >= 1e-30 && eps <= 1e30))) return fail(CT_EINVAL, "eps must be 0 or lie in 1e-30 .. 1e30");
    if (!step_device && step < 1) return fail(CT_EINVAL, "step counts from 1");
    if (!ct::aligned_to(step_device, 8) || !ct::aligned_to(lr_device, 4) || !ct::aligned_to(grad_scale_device, 4))
        return fail(CT_EINVAL, "device scalars must be aligned to their size");
    const size_t ps = ct::float_size(dt), gs = ct::float_size(gt);
    for (int64_t i = 0; i < tensors; ++i) {
        const ct_adamw_tensor &t = list[i];
        const std::string at = " (tensor " + std::to_string(i) + ")";
        if (t.count < 0) return fail(CT_EINVAL, "count must not be negative" + at);
        if (t.count > (int64_t(1) << 40)) return fail(CT_EUNSUPPORTED, "more than 2^40 elements are not served" + at);
        if (!std::isfinite(t.weight_decay)) return fail(CT_EINVAL, "weight_decay must be finite" + at);
        if (t.count == 0) continue;
        if (!t.param || !t.grad || !t.m || !t.v) return fail(CT_EINVAL, "param, grad, m or v is NULL" + at);
        if (state_bits == 8 && (!t.m_scale || !t.v_scale)) return fail(CT_EINVAL, "states in 8 bits need their scales" + at);
        if (t.copy && cp != CT_FLOAT16 && cp != CT_BFLOAT16)
            return fail(CT_EUNSUPPORTED, "copy_dtype must be CT_FLOAT16 or CT_BFLOAT16" + at);
        const size_t ss = state_bits == 32 ? 4 : 1;
        if (!ct::aligned_to(t.param, ps) || !ct::aligned_to(t.grad, gs) || !ct::aligned_to(t.m, ss) || !ct::aligned_to(t.v, ss) ||
            !ct::aligned_to(t.m_scale, 4) || !ct::aligned_to(t.v_scale, 4) || !ct::aligned_to(t.copy, 2))
            return fail(CT_EINVAL, "tensor pointers must be aligned to the element size" + at);
    }
    if (std::all_of(list, list + tensors, [](const ct_adamw_tensor &t) { return t.count == 0; })) return CT_OK;
    Step<kEntries> s{};
    s.b1 = float(beta1), s.c1 = float(1.0 - beta1), s.b2 = float(beta2), s.c2 = float(1.0 - beta2);
    s.eps = float(eps), s.lr = float(lr), s.grad_scale = float(grad_scale);
    s.log_b1 = std::log(beta1), s.log_b2 = std::log(beta2);
    if (!step_device) {
        s.first_bias = float(-std::expm1(double(step) * s.log_b1));
        s.second_root = float(1.0 / std::sqrt(-std::expm1(double(step) * s.log_b2)));
    }
    s.step = step_device;
    s.lr_at = lr_device;
    s.scale_at = grad_scale_device;
    s.copy_type = cp;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    const int64_t run = state_bits == 32 ? kRun32 : kRun8, most = int64_t(1) << 23;  // blocks of a launch
    auto launch = [&] {
        if (!s.entries) return;
        const unsigned blocks = s.first[s.entries];
        auto go = [&](const auto &args) {
            constexpr int N = int(sizeof(args.e) / sizeof(args.e[0]));
            ct::with_type(dt, [&](auto p) {
                ct::with_type(gt, [&](auto g) {
                    if (state_bits == 32) adamw32_kernel<decltype(p), decltype(g), N><<<blocks, kThreads, 0, hs>>>(args);
                    else adamw8_kernel<decltype(p), decltype(g), N><<<blocks, kThreads, 0, hs>>>(args);
                });
            });
        };
        if (s.entries <= kFewEntries) {
            Step<kFewEntries> few;
            static_cast<Hyper &>(few) = s;
            std::copy(s.first, s.first + kFewEntries + 1, few.first);
            std::copy(s.e, s.e + kFewEntries, few.e);
            go(few);
        } else {
            go(s);
        }
        s.entries = 0;
    };
    ct::mark_before(hs);
    for (int64_t i = 0; i < tensors; ++i) {
        const ct_adamw_tensor &t = list[i];
        // a tensor that one launch cannot hold is cut at whole runs
        for (int64_t done = 0; done < t.count;) {
            const int64_t used = s.entries ? int64_t(s.first[s.entries]) : 0;
            if (s.entries == kEntries || used == most) {
                launch();
                continue;
            }
            const int64_t left = t.count - done, blocks = std::min((left + run - 1) / run, most - used);
            const int64_t count = std::min(left, blocks * run);
            auto at = [&](const void *p, size_t size) {
                return p ? const_cast<char *>(static_cast<const char *>(p)) + size_t(done) * size : nullptr;
            };
            const size_t ss = state_bits == 32 ? 4 : 1;
            s.e[s.entries] = {at(t.param, ps), at(t.grad, gs), at(t.m, ss), at(t.v, ss),
                              state_bits == 8 ? t.m_scale + done / kScaleBlock : nullptr,
                              state_bits == 8 ? t.v_scale + done / kScaleBlock : nullptr, at(t.copy, 2), count,
                              float(1.0 - lr * double(t.weight_decay)), t.weight_decay};
            s.first[s.entries] = unsigned(used);
            s.first[++s.entries] = unsigned(used + blocks);
            done += count;
        }
    }
    launch();
    ct::mark_after(hs);
    std::string err;
    const ct_status ls = ct::launch_status("adamw launch failed", &err);
    return ls == CT_OK ? CT_OK : fail(ls, err);
}

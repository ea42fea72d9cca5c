// ct_vec.hpp -- element types, 16-byte vectors, the counter-based generator and the small
// host helpers shared by the group norm, dropout and embedding kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "ct_internal.hpp"

namespace ct {

// V elements as one register vector; the type's alignment is the element's, so a load or
// store through it takes any element address (the hardware splits what crosses a line).
template <class T, int V>
using Raw = T __attribute__((ext_vector_type(V), aligned(sizeof(T))));

// 16 bytes' worth of elements: 8 of the 16-bit types, 4 of float32.
template <class T>
constexpr int kVec = int(16 / sizeof(T));

// Calls f with a value of the element type dt stands for (float32, float16, bfloat16).
template <class F>
inline void with_type(int dt, F &&f)
{
    if (dt == CT_FLOAT32) f(float{});
    else if (dt == CT_FLOAT16) f(_Float16{});
    else f(__bf16{});
}

inline size_t float_size(int dt) { return dt == CT_FLOAT32 ? 4 : 2; }
inline bool is_float_type(int dt) { return dt == CT_FLOAT32 || dt == CT_FLOAT16 || dt == CT_BFLOAT16; }
inline bool aligned_to(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Status of the launches since the last check.
inline ct_status launch_status(const char *what, std::string *err)
{
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) return CT_OK;
    *err = std::string(what) + ": " + hipGetErrorString(e);
    return CT_EDEVICE;
}

// Caller workspace, or stream-ordered scratch released on the same stream at the end of
// the call.
struct Scratch {
    void *p = nullptr;
    hipStream_t st = nullptr;
    bool own = false;
    ct_status take(void *workspace, size_t have, size_t need, hipStream_t stream, std::string *err)
    {
        if (need == 0) return CT_OK;
        if (workspace) {
            if (have < need) {
                *err = "workspace too small: " + std::to_string(have) + " bytes, " + std::to_string(need) + " needed";
                return CT_EINVAL;
            }
            p = workspace;
            return CT_OK;
        }
        const hipError_t e = scratch_malloc(&p, need, stream);
        if (e != hipSuccess) {
            p = nullptr;
            *err = std::string("scratch allocation failed: ") + hipGetErrorString(e);
            return CT_EDEVICE;
        }
        st = stream;
        own = true;
        return CT_OK;
    }
    ~Scratch()
    {
        if (own) (void)hipFreeAsync(p, st);
    }
    Scratch() = default;
    Scratch(const Scratch &) = delete;
    Scratch &operator=(const Scratch &) = delete;
};

// A parameter (gamma, beta) stored as float32 or in the tensor's own type, or absent.
template <class T>
struct Param {
    const void *p;
    bool f32;
    __device__ __forceinline__ float at(int64_t i, float absent) const
    {
        if (!p) return absent;
        return f32 ? static_cast<const float *>(p)[i] : float(static_cast<const T *>(p)[i]);
    }
    // V consecutive values: one choice of type and one wide load, where V calls of at() would
    // be V branches with a wait in each.
    template <int V>
    __device__ __forceinline__ void run(float (&out)[V], int64_t i, float absent) const
    {
        if (!p) {
#pragma unroll
            for (int j = 0; j < V; ++j) out[j] = absent;
        } else if (f32) {
            const Raw<float, V> r = *reinterpret_cast<const Raw<float, V> *>(static_cast<const float *>(p) + i);
#pragma unroll
            for (int j = 0; j < V; ++j) out[j] = r[j];
        } else {
            const Raw<T, V> r = *reinterpret_cast<const Raw<T, V> *>(static_cast<const T *>(p) + i);
#pragma unroll
            for (int j = 0; j < V; ++j) out[j] = float(r[j]);
        }
    }
};

// ------------------------------------------------------------------------------------
// Dropout's random numbers: Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011).  Element i of the tensor in storage order takes
// field i % 8 of the block of counter (i / 8, offset) under key seed; a block's four
// words are eight 16-bit fields, low half first.  The element is dropped when its field
// is below threshold = round(65536 p), so the drop probability is exactly
// threshold / 65536 and the factor of the others 65536 / (65536 - threshold).
//
// 16 bits an element: one block serves a 16-byte vector of the 16-bit types.  A block takes
// 274 cycles of a SIMD for a wave (20 wide integer multiplies are most of it), 353 with the
// eight compares: for 33.5 M elements 9 us of the whole chip, hidden under a pass that is bound
// by memory.  With 32 bits an element it would be nearly twice that in both passes of the
// norm's gradient, whose vector units are 70 % busy as it is.
// ------------------------------------------------------------------------------------
struct Dropout {
    uint32_t threshold = 0;          // 0: no dropout
    float factor = 1.0f;             // 0 when everything is dropped
    uint64_t seed = 0, offset = 0;
    const uint64_t *step = nullptr;  // device value added to offset when the kernel runs
    __device__ __forceinline__ uint32_t limit() const { return threshold - 1; }  // with dropout only
    __device__ __forceinline__ uint64_t counter() const { return step ? offset + *step : offset; }
};

// CT_OK with *d filled, or CT_EINVAL for p outside [0, 1].
inline ct_status make_dropout(double p, uint64_t seed, uint64_t offset, const uint64_t *step, Dropout *d,
                              std::string *err)
{
    if (!(p >= 0.0 && p <= 1.0)) {
        *err = "the dropout probability must lie in [0, 1]";
        return CT_EINVAL;
    }
    if (!aligned_to(step, 8)) {
        *err = "step must be aligned to 8 bytes";
        return CT_EINVAL;
    }
    d->threshold = uint32_t(std::floor(p * 65536.0 + 0.5));
    d->factor = d->threshold >= 65536u ? 0.0f : float(65536.0 / double(65536u - d->threshold));
    d->seed = seed;
    d->offset = offset;
    d->step = step;
    return CT_OK;
}

__device__ __forceinline__ void philox(uint64_t block, uint64_t offset, uint64_t seed, uint32_t (&w)[4])
{
    uint32_t c0 = uint32_t(block), c1 = uint32_t(block >> 32), c2 = uint32_t(offset), c3 = uint32_t(offset >> 32);
    uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = uint64_t(c0) * 0xD2511F53u, p1 = uint64_t(c2) * 0xCD9E8D57u;
        c0 = uint32_t(p1 >> 32) ^ c1 ^ k0;
        c1 = uint32_t(p1);
        c2 = uint32_t(p0 >> 32) ^ c3 ^ k1;
        c3 = uint32_t(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    w[0] = c0;
    w[1] = c1;
    w[2] = c2;
    w[3] = c3;
}

// The fields of V elements, in the places the generator's words have them: element j is
// field j.  It stays when its field is above `limit` = threshold - 1, which fits 16 bits, so
// a low half is compared as it stands and a high half by the whole word.
struct Fields {
    uint32_t w[4];
    __device__ __forceinline__ bool stays(int j, uint32_t limit) const
    {
        return j & 1 ? w[j >> 1] > (limit << 16 | 0xffffu) : uint16_t(w[j >> 1]) > uint16_t(limit);
    }
};

// The fields of elements first .. first + V - 1; ALIGNED: first is known to be a multiple of V.
template <int V, bool ALIGNED>
__device__ __forceinline__ Fields draw_fields(const Dropout &d, uint64_t counter, uint64_t first)
{
    static_assert(V <= 8, "at most two blocks are looked at");
    Fields f;
    philox(first >> 3, counter, d.seed, f.w);
    const int sh = int(first & 7);
    if (V == 4) {
        f.w[0] = sh == 4 ? f.w[2] : f.w[0];
        f.w[1] = sh == 4 ? f.w[3] : f.w[1];
    }
    if (ALIGNED || sh == 0 || (V == 4 && sh == 4)) return f;
    // a vector that starts inside a block: field sh + j, of this block or the next
    Fields next = f, out;
    if (sh + V > 8) philox((first >> 3) + 1, counter, d.seed, next.w);
#pragma unroll
    for (int j = 0; j < 4; ++j) out.w[j] = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int s = 1; s < 8; ++s) {
            const int at = s + j;
            const uint32_t word = at < 8 ? f.w[(at & 7) >> 1] : next.w[(at & 7) >> 1];
            const uint32_t field = at & 1 ? word >> 16 : word & 0xffffu;
            out.w[j >> 1] |= s == sh ? field << (16 * (j & 1)) : 0u;
        }
    }
    return out;
}

}  // namespace ct

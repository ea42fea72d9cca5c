// ct_embedding.hip -- embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward   y[t] = scale * table[ids[t]]
//   gradient  dtable[v] = scale * sum over t with ids[t] = v of dy[t], t ascending
//
// Each sum is made in float32 in a fixed order (no floating atomics), so the gradient of
// the same inputs is the same every time.  An id outside [0, rows) gives a row of zeros
// and no gradient: nothing outside the table is read or written.
#include <hip/hip_runtime.h>

#include <string>

#include "ct_vec.hpp"

namespace {

using ct::Raw;

constexpr int kThreads = 256;
constexpr int kWave = 64;

// A row of `width` elements as whole vectors and then single elements: slot s < full is
// vector s, the others are elements full * V + (s - full).
struct RowSlots {
    int64_t width;
    int64_t full, slots;
    int lanes;  // lanes that share a row: a power of two, at most a wave
};

template <int V>
RowSlots row_slots(int64_t width)
{
    RowSlots r;
    r.width = width;
    r.full = width / V;
    r.slots = r.full + width % V;
    r.lanes = 1;
    while (r.lanes < kWave && r.lanes < r.slots) r.lanes *= 2;
    return r;
}

template <class T, class I>
__global__ __launch_bounds__(kThreads) void lookup_kernel(const I *ids, const T *table, T *y, int64_t tokens,
                                                          int64_t rows, RowSlots rs, float scale)
{
    constexpr int V = ct::kVec<T>;
    const int lane = threadIdx.x & (rs.lanes - 1);
    const int per = kThreads / rs.lanes;
    for (int64_t t = int64_t(blockIdx.x) * per + threadIdx.x / rs.lanes; t < tokens; t += int64_t(gridDim.x) * per) {
        const int64_t id = int64_t(ids[t]);
        const bool ok = id >= 0 && id < rows;
        const T *src = table + (ok ? id : 0) * rs.width;
        T *dst = y + t * rs.width;
        for (int64_t s = lane; s < rs.slots; s += rs.lanes) {
            if (s < rs.full) {
                Raw<T, V> v{}, o;
                if (ok) v = *reinterpret_cast<const Raw<T, V> *>(src + s * V);
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = T(ok ? float(v[j]) * scale : 0.0f);
                *reinterpret_cast<Raw<T, V> *>(dst + s * V) = o;
            } else {
                const int64_t e = rs.full * V + (s - rs.full);
                dst[e] = T(ok ? float(src[e]) * scale : 0.0f);
            }
        }
    }
}

// ------------------------------------------------------------------------------------
// The gradient: a stable radix sort of (id, token) by 8 bits a pass, then the rows' sums
// ------------------------------------------------------------------------------------
constexpr int kDigits = 256;
constexpr int kMaxSortBlocks = 256;

// The sort key of a token: its row, or `rows` (past every row) when it has no gradient.
template <class I>
__device__ __forceinline__ uint32_t key_of(const I *ids, int64_t t, int64_t rows, int64_t padding)
{
    const int64_t id = int64_t(ids[t]);
    return uint32_t(id >= 0 && id < rows && id != padding ? id : rows);
}

// Keys for one pass: the ids themselves in the first, the last pass's output in the others.
template <class I>
struct Source {
    const I *ids;          // first pass
    const uint32_t *keys;  // later passes (ids null)
    const uint32_t *toks;
    int64_t rows, padding;
    __device__ __forceinline__ uint32_t key(int64_t i) const { return keys ? keys[i] : key_of(ids, i, rows, padding); }
    __device__ __forceinline__ uint32_t tok(int64_t i) const { return keys ? toks[i] : uint32_t(i); }
};

template <class I>
__global__ __launch_bounds__(kThreads) void histogram_kernel(Source<I> src, int64_t count, int per_block, int shift,
                                                             uint32_t *hist)
{
    __shared__ uint32_t h[kDigits];
    h[threadIdx.x] = 0;
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * per_block;
    for (int k = threadIdx.x; k < per_block; k += kThreads)
        if (first + k < count) atomicAdd(&h[(src.key(first + k) >> shift) & (kDigits - 1)], 1u);
    __syncthreads();
    hist[blockIdx.x * kDigits + threadIdx.x] = h[threadIdx.x];
}

// Orders a wave's own LDS reads and writes, lane against lane (they execute in order; this
// keeps the compiler from moving them).
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

template <class I>
__global__ __launch_bounds__(kThreads) void scatter_kernel(Source<I> src, int64_t count, int per_block, int shift,
                                                           const uint32_t *hist, uint32_t *keys_out, uint32_t *toks_out)
{
    constexpr int kWaves = kThreads / kWave;
    __shared__ uint32_t off[kWaves][kDigits];
    __shared__ uint32_t scan[kDigits];
    const int d = threadIdx.x, lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    // where this block's tokens of digit d start: all smaller digits, then d in earlier blocks
    uint32_t total = 0, before = 0;
    for (int b = 0; b < int(gridDim.x); ++b) {
        const uint32_t v = hist[b * kDigits + d];
        before += b < int(blockIdx.x) ? v : 0u;
        total += v;
    }
    scan[d] = total;
    for (int w = 0; w < kWaves; ++w) off[w][d] = 0;
    __syncthreads();
    for (int s = 1; s < kDigits; s *= 2) {
        const uint32_t v = d >= s ? scan[d - s] : 0u;
        __syncthreads();
        scan[d] += v;
        __syncthreads();
    }
    const uint32_t base = scan[d] - total + before;
    // a wave's tokens are consecutive, so the order within a digit is wave, round, lane
    const int per_wave = per_block / kWaves;
    const int64_t first = int64_t(blockIdx.x) * per_block + int64_t(wave) * per_wave;
    for (int r = 0; r < per_wave; r += kWave) {
        const int64_t i = first + r + lane;
        if (i < count) atomicAdd(&off[wave][(src.key(i) >> shift) & (kDigits - 1)], 1u);
    }
    __syncthreads();
    uint32_t sum = base;
    for (int w = 0; w < kWaves; ++w) {
        const uint32_t v = off[w][d];
        off[w][d] = sum;
        sum += v;
    }
    __syncthreads();
    for (int r = 0; r < per_wave; r += kWave) {
        const int64_t i = first + r + lane;
        const bool in = i < count;
        const uint32_t key = in ? src.key(i) : 0u;
        const uint32_t digit = (key >> shift) & (kDigits - 1);
        unsigned long long same = __ballot(in);
#pragma unroll
        for (int bit = 0; bit < 8; ++bit) {
            const unsigned long long set = __ballot((digit >> bit) & 1);
            same &= (digit >> bit) & 1 ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        uint32_t at = 0;
        if (in) at = off[wave][digit] + uint32_t(rank);
        wave_fence();
        if (in && rank == 0) off[wave][digit] += uint32_t(__popcll(same));
        wave_fence();
        if (in) {
            keys_out[at] = key;
            toks_out[at] = src.tok(i);
        }
    }
}

// First position of the sorted keys that is not below `key`.
__device__ __forceinline__ int64_t lower_bound(const uint32_t *keys, int64_t count, uint32_t key)
{
    int64_t lo = 0, hi = count;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (keys[mid] < key) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// Adds dy[toks[i]] for i in [begin, end) into acc, slot s of the row.
template <class T, int V>
__device__ __forceinline__ void add_rows(float (&acc)[V], const T *dy, const uint32_t *toks, int64_t begin, int64_t end,
                                         const RowSlots &rs, int64_t s)
{
    if (s < rs.full) {
#pragma unroll 4
        for (int64_t i = begin; i < end; ++i) {
            const Raw<T, V> v = *reinterpret_cast<const Raw<T, V> *>(dy + int64_t(toks[i]) * rs.width + s * V);
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] += float(v[j]);
        }
    } else {
        const int64_t e = rs.full * V + (s - rs.full);
        for (int64_t i = begin; i < end; ++i) acc[0] += float(dy[int64_t(toks[i]) * rs.width + e]);
    }
}

// The sorted tokens in chunks: a row inside one chunk is summed by the kernel that writes
// the rows; of a row that crosses a chunk's border every chunk makes a partial sum here,
// slot 0 for the row at its start and slot 1 for the one at its end.
template <class T>
__global__ __launch_bounds__(kThreads) void partial_kernel(const T *dy, const uint32_t *keys, const uint32_t *toks,
                                                           int64_t count, int64_t rows, int chunk, RowSlots rs,
                                                           float *partial)
{
    constexpr int V = ct::kVec<T>;
    const int64_t a = int64_t(blockIdx.x) * chunk, b = a + chunk < count ? a + chunk : count;
    const uint32_t first = keys[a], last = keys[b - 1];
    const int per = kThreads / rs.lanes;  // 1 < rows of lanes: they share nothing, only the first works
    if (int(threadIdx.x) / rs.lanes > 0 && per > 1) return;
    const int lane = threadIdx.x & (rs.lanes - 1);
    for (int slot = 0; slot < 2; ++slot) {
        const uint32_t key = slot ? last : first;
        if (key >= uint32_t(rows) || (slot && first == last)) continue;
        const int64_t lo = slot ? a + lower_bound(keys + a, b - a, key) : a;
        const int64_t hi = slot ? b : a + lower_bound(keys + a, b - a, key + 1);
        const bool crosses = (lo == a && a > 0 && keys[a - 1] == key) || (hi == b && b < count && keys[b] == key);
        if (!crosses) continue;
        float *out = partial + (int64_t(blockIdx.x) * 2 + slot) * rs.width;
        for (int64_t s = lane; s < rs.slots; s += rs.lanes) {
            float acc[V] = {};
            add_rows<T, V>(acc, dy, toks, lo, hi, rs, s);
            if (s < rs.full) {
                for (int j = 0; j < V; ++j) out[s * V + j] = acc[j];
            } else {
                out[rs.full * V + (s - rs.full)] = acc[0];
            }
        }
    }
}

template <class T, class G>
__global__ __launch_bounds__(kThreads) void rows_kernel(const T *dy, const uint32_t *keys, const uint32_t *toks,
                                                        int64_t count, int64_t rows, int chunk, RowSlots rs,
                                                        const float *partial, float scale, G *dtable)
{
    constexpr int V = ct::kVec<T>;
    const int lane = threadIdx.x & (rs.lanes - 1);
    const int per = kThreads / rs.lanes;
    for (int64_t v = int64_t(blockIdx.x) * per + threadIdx.x / rs.lanes; v < rows; v += int64_t(gridDim.x) * per) {
        const int64_t lo = lower_bound(keys, count, uint32_t(v)), hi = lower_bound(keys, count, uint32_t(v) + 1);
        const int64_t c0 = lo / chunk, c1 = (hi - 1) / chunk;
        G *dst = dtable + v * rs.width;
        for (int64_t s = lane; s < rs.slots; s += rs.lanes) {
            float acc[V] = {};
            const bool vec = s < rs.full;
            const int64_t e = vec ? s * V : rs.full * V + (s - rs.full);
            if (hi > lo && c0 == c1) {
                add_rows<T, V>(acc, dy, toks, lo, hi, rs, s);
            } else if (hi > lo) {
                for (int64_t c = c0; c <= c1; ++c) {
                    const float *src = partial + (c * 2 + (c == c0 && lo > c0 * chunk ? 1 : 0)) * rs.width + e;
                    for (int j = 0; j < (vec ? V : 1); ++j) acc[j] += src[j];
                }
            }
            if (vec) {
                Raw<G, V> o;
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = G(acc[j] * scale);
                *reinterpret_cast<Raw<G, V> *>(dst + e) = o;
            } else {
                dst[e] = G(acc[0] * scale);
            }
        }
    }
}

// How a gradient is cut up, and where its workspace's parts are.
struct GradPlan {
    int64_t tokens = 0, rows = 0, width = 0;
    int passes = 0, sort_blocks = 0, per_block = 0, chunk = 0;
    int64_t chunks = 0;
    size_t keys[2] = {}, toks[2] = {}, hist = 0, partial = 0, bytes = 0;
};

GradPlan grad_plan(int64_t tokens, int64_t rows, int64_t width)
{
    GradPlan g;
    g.tokens = tokens;
    g.rows = rows;
    g.width = width;
    while (g.passes < 4 && (uint64_t(rows) >> (8 * g.passes)) != 0) ++g.passes;  // keys run from 0 to rows
    if (g.passes == 0) g.passes = 1;
    int64_t per = 4 * kThreads;
    while ((tokens + per - 1) / per > kMaxSortBlocks) per *= 2;
    g.per_block = int(per);
    g.sort_blocks = int((tokens + per - 1) / per);
    g.chunk = 64;
    while (int64_t(g.chunk) * g.chunk < tokens) g.chunk *= 2;
    g.chunks = (tokens + g.chunk - 1) / g.chunk;
    size_t at = 0;
    auto place = [&](size_t bytes) {
        const size_t p = at;
        at += (bytes + 255) & ~size_t(255);
        return p;
    };
    for (int k = 0; k < 2; ++k) {
        g.keys[k] = place(size_t(tokens) * 4);
        g.toks[k] = place(size_t(tokens) * 4);
    }
    g.hist = place(size_t(g.sort_blocks) * kDigits * 4);
    g.partial = place(g.chunks > 1 ? size_t(g.chunks) * 2 * size_t(width) * 4 : 0);
    g.bytes = at;
    return g;
}

ct_status fail(ct_status st, const std::string &msg)
{
    ct::set_last_error(msg);
    return st;
}

// Sizes both directions share; every byte offset below stays inside 63 bits.
ct_status check_sizes(int index, int64_t tokens, int64_t rows, int64_t width)
{
    if (index != CT_INT32 && index != CT_INT64) return fail(CT_EUNSUPPORTED, "ids must be CT_INT32 or CT_INT64");
    if (tokens < 0 || rows < 0 || width < 0) return fail(CT_EINVAL, "sizes must not be negative");
    const int64_t most = int64_t(1) << 31;
    if (tokens >= most || rows >= most - 1 || width >= most)
        return fail(CT_EUNSUPPORTED, "tokens, rows and width must be below 2^31 - 1");
    if (width > 0 && (tokens > (int64_t(1) << 58) / width || rows > (int64_t(1) << 58) / width))
        return fail(CT_EUNSUPPORTED, "tensors of more than 2^58 elements");
    return CT_OK;
}

template <class F>
void with_index(int index, F &&f)
{
    if (index == CT_INT32) f(int32_t{});
    else f(int64_t{});
}

unsigned blocks_for(int64_t rows, int per)
{
    const int64_t want = (rows + per - 1) / per;
    return unsigned(want < (1 << 23) ? want : 1 << 23);
}

}  // namespace

extern "C" {

ct_status embedding_nd(ct_dtype dtype, ct_dtype index_dtype, int64_t tokens, const void *ids, int64_t rows,
                       int64_t width, const void *table, float scale, void *y, void *stream)
{
    ct::set_last_error(std::string());
    const int dt = ct::enum_int(dtype), index = ct::enum_int(index_dtype);
    if (!ct::is_float_type(dt)) return fail(CT_EUNSUPPORTED, "dtype must be CT_FLOAT32, CT_FLOAT16 or CT_BFLOAT16");
    const ct_status st = check_sizes(index, tokens, rows, width);
    if (st != CT_OK) return st;
    if (!std::isfinite(scale)) return fail(CT_EINVAL, "scale must be finite");
    const size_t esz = ct::float_size(dt);
    if (!ct::aligned_to(table, esz) || !ct::aligned_to(y, esz) || !ct::aligned_to(ids, index == CT_INT32 ? 4 : 8))
        return fail(CT_EINVAL, "tensor pointers must be aligned to the element size");
    if (tokens == 0 || width == 0) return CT_OK;
    if (!ids || !y || (!table && rows > 0)) return fail(CT_EINVAL, "ids, table or y is NULL");
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    ct::mark_before(hs);
    ct::with_type(dt, [&](auto t) {
        using T = decltype(t);
        with_index(index, [&](auto i) {
            using I = decltype(i);
            const RowSlots rs = row_slots<ct::kVec<T>>(width);
            lookup_kernel<T, I><<<blocks_for(tokens, kThreads / rs.lanes), kThreads, 0, hs>>>(
                static_cast<const I *>(ids), static_cast<const T *>(table), static_cast<T *>(y), tokens, rows, rs, scale);
        });
    });
    ct::mark_after(hs);
    std::string err;
    const ct_status ls = ct::launch_status("embedding launch failed", &err);
    return ls == CT_OK ? CT_OK : fail(ls, err);
}

ct_status embedding_workspace_size(int64_t tokens, int64_t rows, int64_t width, size_t *bytes_out)
{
    ct::set_last_error(std::string());
    if (!bytes_out) return fail(CT_EINVAL, "bytes_out is NULL");
    const ct_status st = check_sizes(CT_INT64, tokens, rows, width);
    if (st != CT_OK) return st;
    *bytes_out = tokens > 0 && rows > 0 && width > 0 ? grad_plan(tokens, rows, width).bytes : 0;
    return CT_OK;
}

ct_status embedding_backward_nd(ct_dtype dtype, ct_dtype index_dtype, int64_t tokens, const void *ids, int64_t rows,
                                int64_t width, const void *dy, float scale, int64_t padding_idx, ct_dtype grad_dtype,
                                void *dtable, void *workspace, size_t workspace_bytes, void *stream)
{
    ct::set_last_error(std::string());
    const int dt = ct::enum_int(dtype), index = ct::enum_int(index_dtype), gt = ct::enum_int(grad_dtype);
    if (!ct::is_float_type(dt)) return fail(CT_EUNSUPPORTED, "dtype must be CT_FLOAT32, CT_FLOAT16 or CT_BFLOAT16");
    if (gt != dt && gt != CT_FLOAT32) return fail(CT_EUNSUPPORTED, "grad_dtype must be dtype or CT_FLOAT32");
    ct_status st = check_sizes(index, tokens, rows, width);
    if (st != CT_OK) return st;
    if (!std::isfinite(scale)) return fail(CT_EINVAL, "scale must be finite");
    if (padding_idx < -1 || padding_idx >= rows)
        return fail(CT_EINVAL, "padding_idx must be a row, or -1 for none");
    if (!ct::aligned_to(dy, ct::float_size(dt)) || !ct::aligned_to(dtable, ct::float_size(gt)) ||
        !ct::aligned_to(ids, index == CT_INT32 ? 4 : 8))
        return fail(CT_EINVAL, "tensor pointers must be aligned to the element size");
    if (workspace && !ct::aligned_to(workspace, 16)) return fail(CT_EINVAL, "workspace must be 16-byte aligned");
    if (rows == 0 || width == 0) return CT_OK;
    if (!dtable || (tokens > 0 && (!ids || !dy))) return fail(CT_EINVAL, "ids, dy or dtable is NULL");
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    const GradPlan g = grad_plan(tokens, rows, width);
    ct::Scratch ws;
    std::string err;
    st = ws.take(workspace, workspace_bytes, tokens > 0 ? g.bytes : 0, hs, &err);
    if (st != CT_OK) return fail(st, err);
    char *const base = static_cast<char *>(ws.p);
    auto words = [&](size_t at) { return reinterpret_cast<uint32_t *>(base + at); };
    const uint32_t *keys = nullptr, *toks = nullptr;
    if (tokens > 0) {
        with_index(index, [&](auto i) {
            using I = decltype(i);
            Source<I> src{static_cast<const I *>(ids), nullptr, nullptr, rows, padding_idx};
            for (int p = 0; p < g.passes; ++p) {
                histogram_kernel<I><<<g.sort_blocks, kThreads, 0, hs>>>(src, tokens, g.per_block, 8 * p, words(g.hist));
                scatter_kernel<I><<<g.sort_blocks, kThreads, 0, hs>>>(src, tokens, g.per_block, 8 * p, words(g.hist),
                                                                     words(g.keys[p & 1]), words(g.toks[p & 1]));
                src.keys = words(g.keys[p & 1]);
                src.toks = words(g.toks[p & 1]);
            }
            keys = src.keys;
            toks = src.toks;
        });
    }
    ct::with_type(dt, [&](auto t) {
        using T = decltype(t);
        const RowSlots rs = row_slots<ct::kVec<T>>(width);
        float *const partial = reinterpret_cast<float *>(base + g.partial);
        const T *const dyp = static_cast<const T *>(dy);
        if (tokens > 0 && g.chunks > 1)
            partial_kernel<T><<<unsigned(g.chunks), kThreads, 0, hs>>>(dyp, keys, toks, tokens, rows, g.chunk, rs, partial);
        const unsigned blocks = blocks_for(rows, kThreads / rs.lanes);
        ct::mark_before(hs);
        if (gt == CT_FLOAT32)
            rows_kernel<T, float><<<blocks, kThreads, 0, hs>>>(dyp, keys, toks, tokens, rows, g.chunk, rs, partial, scale,
                                                              static_cast<float *>(dtable));
        else
            rows_kernel<T, T><<<blocks, kThreads, 0, hs>>>(dyp, keys, toks, tokens, rows, g.chunk, rs, partial, scale,
                                                          static_cast<T *>(dtable));
        ct::mark_after(hs);
    });
    st = ct::launch_status("embedding gradient launch failed", &err);
    return st == CT_OK ? CT_OK : fail(st, err);
}

}  // extern "C"

// ct_embedding.hip -- embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward   y[t] = scale * table[ids[t]]
//   gradient  dtable[v] = scale * sum over t with ids[t] = v of dy[t], t ascending
//
// Each sum is made in float32 in a fixed order (no floating atomics), so the gradient of
// the same inputs is the same every time.  An id outside [0, rows) gives a row of zeros
// and no gradient: nothing outside the table is read or written.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "ct_vec.hpp"

namespace {

using ct::Raw;

constexpr int kThreads = 256;
constexpr int kWave = 64;

template <int V>
__device__ __forceinline__ Raw<float, V> as_floats(const float (&a)[V])
{
    Raw<float, V> r;
#pragma unroll
    for (int j = 0; j < V; ++j) r[j] = a[j];
    return r;
}

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

// The lookup: up to a wave's lanes share a row, 16 bytes each, and a block's rows are
// consecutive tokens, so y is written in one stream.  Bound by memory: 32768 rows of 512
// float16 (1 KB each) out of 16384 take 10.2 us, 42.7 MB, 4.2 TB/s; the id is one more read
// in front of the row's, which the block's other waves hide.  One token is a launch, 4.4 us.
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
//
// Sorted, a row's tokens stand together in ascending order: every row of dy is read once,
// every row of the table is written once, and no sum depends on which block came first.
// 32768 tokens of 512 float16 into 16384 rows (50.6 MB) take 37.8 us.  A trace, which keeps the
// kernels further apart, has the counts at 3.9 and 2.6, the moves at 6.2 and 6.1, the chunks at
// 13.1 and the rows at 9.7 (medians; more than the untraced call when added).  The sort and the rows
// are bound by chains of dependent reads (an id to a place, a row's begin to its key to its
// partial sums) of about a microsecond a link, not by bytes; the chunks by memory.
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

// One pass is two kernels: how many tokens of each digit a block has, then, with all blocks'
// counts, where each of its tokens goes.
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

// Where the lane's token goes: the next place of its digit after the lanes before it with the
// same digit.  off[digit] is the wave's next place of each digit and moves on.
__device__ __forceinline__ uint32_t place_in_order(uint32_t *off, uint32_t digit, bool in, int lane)
{
    unsigned long long same = __ballot(in);
#pragma unroll
    for (int bit = 0; bit < 8; ++bit) {
        const unsigned long long set = __ballot((digit >> bit) & 1);
        same &= (digit >> bit) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    uint32_t at = 0;
    if (in) at = off[digit] + uint32_t(rank);
    wave_fence();
    if (in && rank == 0) off[digit] += uint32_t(__popcll(same));
    wave_fence();
    return at;
}

template <class I>
__global__ __launch_bounds__(kThreads) void scatter_kernel(Source<I> src, int64_t count, int per_block, int shift,
                                                           const uint32_t *hist, uint32_t *keys_out, uint32_t *toks_out)
{
    constexpr int kWaves = kThreads / kWave;
    __shared__ uint32_t off[kWaves][kDigits];
    __shared__ uint32_t wave_sum[kWaves];
    const int d = threadIdx.x, lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    // a wave's tokens are consecutive, so the order within a digit is wave, round, lane
    const int per_wave = per_block / kWaves;
    const int64_t first = int64_t(blockIdx.x) * per_block + int64_t(wave) * per_wave;
    constexpr int kEarly = 2;  // rounds whose tokens are asked for first: all of them but in very long sorts
    uint32_t early_key[kEarly], early_tok[kEarly];
#pragma unroll
    for (int r = 0; r < kEarly; ++r) {
        const int64_t i = first + r * kWave + lane;
        const bool in = r * kWave < per_wave && i < count;
        early_key[r] = in ? src.key(i) : 0u;
        early_tok[r] = in ? src.tok(i) : 0u;
    }
    auto key_at = [&](int r, int64_t i) { return r == 0 ? early_key[0] : r == kWave ? early_key[1] : src.key(i); };
    auto tok_at = [&](int r, int64_t i) { return r == 0 ? early_tok[0] : r == kWave ? early_tok[1] : src.tok(i); };
    // where this block's tokens of digit d start: all smaller digits, then d in earlier blocks
    uint32_t total = 0, before = 0;
#pragma unroll 16
    for (int b = 0; b < int(gridDim.x); ++b) {
        const uint32_t v = hist[b * kDigits + d];
        before += b < int(blockIdx.x) ? v : 0u;
        total += v;
    }
    for (int w = 0; w < kWaves; ++w) off[w][d] = 0;
    uint32_t upto = total;  // of this wave's digits up to d
    for (int s = 1; s < kWave; s *= 2) {
        const uint32_t v = __shfl_up(upto, s);
        upto += lane >= s ? v : 0u;
    }
    if (lane == kWave - 1) wave_sum[wave] = upto;
    __syncthreads();
    uint32_t base = upto - total + before;
    for (int w = 0; w < wave; ++w) base += wave_sum[w];
    for (int r = 0; r < per_wave; r += kWave) {
        const int64_t i = first + r + lane;
        if (i < count) atomicAdd(&off[wave][(key_at(r, i) >> shift) & (kDigits - 1)], 1u);
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
        const uint32_t key = in ? key_at(r, i) : 0u;
        const uint32_t at = place_in_order(off[wave], (key >> shift) & (kDigits - 1), in, lane);
        if (in) {
            keys_out[at] = key;
            toks_out[at] = tok_at(r, i);
        }
    }
}

// Where each row's tokens begin and end in the sorted order, written by the thread that sees
// the border.  Rows without tokens are not written: who reads a row's begin looks whether
// the row is there.
struct Bounds {
    uint32_t *begin, *end;
    __device__ __forceinline__ void mark(const uint32_t *keys, int64_t i, int64_t count, int64_t rows) const
    {
        const uint32_t k = keys[i];
        if (k >= uint32_t(rows)) return;
        if (i == 0 || keys[i - 1] != k) begin[k] = uint32_t(i);
        if (i + 1 == count || keys[i + 1] != k) end[k] = uint32_t(i + 1);
    }
};

// Up to kOneSort tokens (their keys and places twice fill 64 KB of LDS): the whole sort in one
// block, one launch instead of two a pass.  The whole gradient, one block / kernels a pass, us:
// 600 tokens into 8000 rows 17.4 / 24.1, 2000 20.2 / 26.6, 4000 24.4 / 29.2, 4000 into 200 rows
// (one pass) 19.0 / 19.7.
constexpr int kOneSort = 4096, kSortThreads = 1024;
template <class I>
__global__ __launch_bounds__(kSortThreads) void one_sort_kernel(Source<I> src, int count, int passes, bool mark, Bounds bounds,
                                                                uint32_t *keys_out, uint32_t *toks_out)
{
    constexpr int kWaves = kSortThreads / kWave;
    __shared__ uint32_t keys[2][kOneSort], toks[2][kOneSort];
    __shared__ uint32_t off[kWaves][kDigits], scan[kDigits];
    const int t = threadIdx.x, lane = t & (kWave - 1), wave = t / kWave;
    for (int i = t; i < count; i += kSortThreads) {
        keys[0][i] = src.key(i);
        toks[0][i] = uint32_t(i);
    }
    const int per_wave = (count + kWaves * kWave - 1) / (kWaves * kWave) * kWave;  // consecutive tokens of a wave
    for (int p = 0; p < passes; ++p) {
        const uint32_t *const key = keys[p & 1], *const tok = toks[p & 1];
        uint32_t *const key_to = keys[1 - (p & 1)], *const tok_to = toks[1 - (p & 1)];
        const int shift = 8 * p;
        for (int i = t; i < kWaves * kDigits; i += kSortThreads) (&off[0][0])[i] = 0;
        __syncthreads();
        for (int r = 0; r < per_wave; r += kWave) {
            const int i = wave * per_wave + r + lane;
            if (i < count) atomicAdd(&off[wave][(key[i] >> shift) & (kDigits - 1)], 1u);
        }
        __syncthreads();
        uint32_t total = 0;
        if (t < kDigits) {
            for (int w = 0; w < kWaves; ++w) total += off[w][t];
            scan[t] = total;
        }
        __syncthreads();
        for (int d = 1; d < kDigits; d *= 2) {
            const uint32_t v = t < kDigits && t >= d ? scan[t - d] : 0u;
            __syncthreads();
            if (t < kDigits) scan[t] += v;
            __syncthreads();
        }
        if (t < kDigits) {
            uint32_t sum = scan[t] - total;
            for (int w = 0; w < kWaves; ++w) {
                const uint32_t v = off[w][t];
                off[w][t] = sum;
                sum += v;
            }
        }
        __syncthreads();
        for (int r = 0; r < per_wave; r += kWave) {
            const int i = wave * per_wave + r + lane;
            const bool in = i < count;
            const uint32_t k = in ? key[i] : 0u;
            const uint32_t at = place_in_order(off[wave], (k >> shift) & (kDigits - 1), in, lane);
            if (in) {
                key_to[at] = k;
                tok_to[at] = tok[i];
            }
        }
        __syncthreads();
    }
    for (int i = t; i < count; i += kSortThreads) {
        keys_out[i] = keys[passes & 1][i];
        toks_out[i] = toks[passes & 1][i];
        if (mark) bounds.mark(keys[passes & 1], i, count, src.rows);
    }
}

// Adds dy[toks[i]] for i in [begin, end) into acc, slot s of the row: kAtOnce tokens' loads at
// a time, added in order.
template <int kAtOnce, class T, int V>
__device__ __forceinline__ void add_rows(float (&acc)[V], const T *dy, const uint32_t *toks, int64_t begin, int64_t end,
                                         const RowSlots &rs, int64_t s)
{
    if (s < rs.full) {
        const T *const src = dy + s * V;
        int64_t i = begin;
        for (; i + kAtOnce <= end; i += kAtOnce) {
            uint32_t tok[kAtOnce];
            Raw<T, V> v[kAtOnce];
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) tok[q] = toks[i + q];
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) v[q] = *reinterpret_cast<const Raw<T, V> *>(src + int64_t(tok[q]) * rs.width);
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q)
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] += float(v[q][j]);
        }
        if (i < end) {  // the rest together too: what is past the end is the last token, not added
            uint32_t tok[kAtOnce];
            Raw<T, V> v[kAtOnce];
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) tok[q] = toks[i + q < end ? i + q : end - 1];
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q)
                if (q == 0 || i + q < end) v[q] = *reinterpret_cast<const Raw<T, V> *>(src + int64_t(tok[q]) * rs.width);
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q)
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] += i + q < end ? float(v[q][j]) : 0.0f;
        }
    } else {
        const int64_t e = rs.full * V + (s - rs.full);
#pragma unroll 4
        for (int64_t i = begin; i < end; ++i) acc[0] += float(dy[int64_t(toks[i]) * rs.width + e]);
    }
}

// Adds the partial sums of chunks from .. to - 1 of a row that begins in chunk `first`, there
// in slot `head`, slot s of the row.
template <int V>
__device__ __forceinline__ void add_partials(float (&acc)[V], const float *partial, int from, int to, int first, int head,
                                             const RowSlots &rs, int64_t s)
{
    constexpr int kAtOnce = 8;  // on their way together; past the end the last one, not added
    const bool vec = s < rs.full;
    const float *const src = partial + (vec ? s * V : rs.full * V + (s - rs.full));
    for (int c = from; c < to; c += kAtOnce) {
        Raw<float, V> p[kAtOnce];
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
            const int at = c + q < to ? c + q : to - 1;
            const float *const one = src + (int64_t(at) * 2 + (at == first ? head : 0)) * rs.width;
            p[q] = Raw<float, V>{};
            if (vec) p[q] = *reinterpret_cast<const Raw<float, V> *>(one);
            else p[q][0] = *one;
        }
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q)
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] += c + q < to ? p[q][j] : 0.0f;
    }
}

// Stores slot s of a table row.
template <class G, int V>
__device__ __forceinline__ void store_slot(G *dst, const RowSlots &rs, int64_t s, const float (&acc)[V], float scale)
{
    if (s < rs.full) {
        Raw<G, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = G(acc[j] * scale);
        *reinterpret_cast<Raw<G, V> *>(dst + s * V) = o;
    } else {
        dst[rs.full * V + (s - rs.full)] = G(acc[0] * scale);
    }
}

// The sorted tokens in chunks.  The groups of lanes take consecutive shares of a chunk's tokens
// and walk them, kAtOnce rows of dy on their way together: a sum that begins and ends inside a
// share is stored at once, those at a share's borders are joined in their order over LDS, and
// of a row that crosses a chunk's border every chunk leaves a partial sum, in slot 0 of the
// chunk for a row that is there from its start and in slot 1 for one that begins later.
// The work is cut by tokens, so a frequent row and many rare ones take the same time; the
// kernel reads all of dy: 33.5 MB and 9 MB of the table's rows in 13.1 us (traced), 3.2 TB/s (16
// rows on their way made the whole gradient 40.5 us instead of 39.4).
constexpr int kMostChunk = 1024;
template <class T, class G>
__global__ __launch_bounds__(kThreads) void chunk_kernel(const T *dy, const uint32_t *keys, const uint32_t *toks,
                                                         int64_t count, int64_t rows, int chunk, RowSlots rs, int64_t steps,
                                                         int64_t work, Bounds bounds, float *partial, float scale, G *dtable)
{
    constexpr int V = ct::kVec<T>, kAtOnce = 8;
    __shared__ uint32_t key[kMostChunk], tok[kMostChunk];
    __shared__ float ends[2][kThreads * V];  // a share's first sum, and its last if that is another
    __shared__ int valid;
    const int groups = kThreads / rs.lanes, group = threadIdx.x / rs.lanes, lane = threadIdx.x & (rs.lanes - 1);
    for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
        const int64_t c = w / steps, s = (w - c * steps) * rs.lanes + lane, a = c * chunk;
        const int n = int(count - a < chunk ? count - a : chunk);
        const uint32_t left = a > 0 ? keys[a - 1] : uint32_t(rows), right = a + n < count ? keys[a + n] : uint32_t(rows);
        __syncthreads();
        if (threadIdx.x == 0) valid = 0;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            key[i] = keys[a + i];
            tok[i] = toks[a + i];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const uint32_t k = key[i];
            if (k >= uint32_t(rows)) continue;
            const uint32_t before = i > 0 ? key[i - 1] : left, after = i + 1 < n ? key[i + 1] : right;
            if (i + 1 == n || after >= uint32_t(rows)) valid = i + 1;
            if (s != lane) continue;  // one step a chunk marks
            if (before != k) bounds.begin[k] = uint32_t(a + i);
            if (after != k) bounds.end[k] = uint32_t(a + i + 1);
        }
        __syncthreads();
        const int m = valid;
        if (m == 0) continue;
        const bool vec = s < rs.full, there = s < rs.slots;
        const int64_t at = vec ? s * V : rs.full * V + (s - rs.full);  // the slot's first element
        const int share = (m + groups - 1) / groups;
        const int from = group * share < m ? group * share : m, to = from + share < m ? from + share : m;
        float acc[V] = {};
        int run = from;  // where the sum in acc began
        auto keep = [&](int part) {
#pragma unroll
            for (int j = 0; j < V; ++j) ends[part][threadIdx.x * V + j] = acc[j];
        };
        auto put = [&](uint32_t k) {
            if (there) store_slot<G, V>(dtable + int64_t(k) * rs.width, rs, s, acc, scale);
        };
        for (int i = from; i < to; i += kAtOnce) {
            Raw<T, V> v[kAtOnce];
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {  // past the end the last token, not added
                const T *const src = dy + int64_t(tok[i + q < to ? i + q : to - 1]) * rs.width + at;
                v[q] = Raw<T, V>{};
                if (vec) v[q] = *reinterpret_cast<const Raw<T, V> *>(src);
                else if (there) v[q][0] = *src;
            }
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                if (i + q >= to) break;
                if (i + q > run && key[i + q] != key[i + q - 1]) {
                    if (run == from) keep(0);
                    else put(key[run]);
                    run = i + q;
#pragma unroll
                    for (int j = 0; j < V; ++j) acc[j] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] += float(v[q][j]);
            }
        }
        if (from < to) keep(run == from ? 0 : 1);
        __syncthreads();
        // each share's groups of lanes write the rows that begin in its first or last sum
        for (int part = 0; part < 2 && from < to; ++part) {
            const uint32_t k = part ? key[to - 1] : key[from];
            if (part ? k == key[from] : from > 0 && key[from - 1] == k) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] = ends[part][threadIdx.x * V + j];
            if (key[to - 1] == k)
                for (int g = group + 1; g * share < m && key[g * share] == k; ++g)
#pragma unroll
                    for (int j = 0; j < V; ++j) acc[j] += ends[0][(g * rs.lanes + lane) * V + j];
            if (!((k == key[0] && left == k) || (k == key[m - 1] && m == n && right == k))) {
                put(k);
            } else if (there) {
                float *const out = partial + (c * 2 + (k == key[0] ? 0 : 1)) * rs.width + at;
                if (vec) *reinterpret_cast<Raw<float, V> *>(out) = as_floats(acc);
                else *out = acc[0];
            }
        }
    }
}

// The table's rows, one by each `lanes` threads: zeros, or the sum of the chunks' partial sums
// of it; the rows inside a chunk are written already.  With one chunk there is no kernel
// before this one, and a row is the sum of its tokens.  Many partial sums (a frequent row) are shared out over the block:
// consecutive ones to each group of lanes, joined in their order, kJoin reads of LDS on their way
// together and only those of groups that have a share: a narrow row has up to 256 groups, and
// all of them one after another took 9 us a row (6225 tokens into 90 rows of one float32 84.7 us a
// call, now 30.3; 8 at a time 30.5).
// kFewPartials: as many as are on their way together (4 / 16: 39.4 / 39.6 us for 32768 x 512).
constexpr int kFewPartials = 8, kBlockRows = 1024, kJoin = 4;
template <class T, class G>
__global__ __launch_bounds__(kThreads) void rows_kernel(const T *dy, const uint32_t *keys, const uint32_t *toks,
                                                        int64_t count, int64_t rows, int chunk, RowSlots rs, Bounds bounds,
                                                        const float *partial, bool inner, int ahead, float scale, G *dtable)
{
    constexpr int V = ct::kVec<T>;
    __shared__ float lds[kThreads * V];
    __shared__ int low[kBlockRows], high[kBlockRows], many[kBlockRows], found;
    const int lane = threadIdx.x & (rs.lanes - 1), group = threadIdx.x / rs.lanes;
    const int groups = kThreads / rs.lanes;
    const int64_t stride = int64_t(gridDim.x) * groups;  // from a group's row to its next
    for (int64_t v0 = int64_t(blockIdx.x) * groups; v0 < rows; v0 += stride * ahead) {
        __syncthreads();
        for (int t = threadIdx.x; t < groups * ahead; t += kThreads) {
            const int64_t v = v0 + t / groups * stride + t % groups;
            int lo = 0, hi = 0;
            if (count > 0 && v < rows) {
                const uint32_t begin = bounds.begin[v], end = bounds.end[v];
                if (begin < uint32_t(count) && keys[begin] == uint32_t(v)) {
                    lo = int(begin);
                    hi = int(end);
                }
            }
            low[t] = lo;
            high[t] = hi;
        }
        if (threadIdx.x == 0) found = 0;
        __syncthreads();
        for (int q = 0; q < ahead; ++q) {
            const int t = q * groups + group;
            const int64_t v = v0 + q * stride + group;
            if (v >= rows) break;
            const int lo = low[t], hi = high[t], c0 = lo / chunk, c1 = hi > lo ? (hi - 1) / chunk : c0;
            if (inner && hi > lo && c0 == c1) continue;
            if (c1 - c0 >= kFewPartials) {
                if (lane == 0) many[atomicAdd(&found, 1)] = t;  // any order: each row is summed by itself
                continue;
            }
            G *const dst = dtable + v * rs.width;
            for (int64_t s = lane; s < rs.slots; s += rs.lanes) {
                float acc[V] = {};
                if (hi > lo && c0 == c1) add_rows<4, T, V>(acc, dy, toks, lo, hi, rs, s);
                else if (hi > lo) add_partials<V>(acc, partial, c0, c1 + 1, c0, lo > c0 * chunk ? 1 : 0, rs, s);
                store_slot<G, V>(dst, rs, s, acc, scale);
            }
        }
        __syncthreads();
        for (int m = 0; m < found; ++m) {
            const int t = many[m], first = low[t] / chunk, n = (high[t] - 1) / chunk - first + 1;
            const int share = (n + groups - 1) / groups, head = low[t] > first * chunk ? 1 : 0;
            const int from = group * share < n ? group * share : n, to = from + share < n ? from + share : n;
            const int used = (n + share - 1) / share;  // groups of lanes that have a share
            G *const dst = dtable + (v0 + t / groups * stride + t % groups) * rs.width;
            for (int64_t s0 = 0; s0 < rs.slots; s0 += rs.lanes) {
                const int64_t s = s0 + lane;
                float acc[V] = {};
                if (s < rs.slots) add_partials<V>(acc, partial, first + from, first + to, first, head, rs, s);
                __syncthreads();
#pragma unroll
                for (int j = 0; j < V; ++j) lds[threadIdx.x * V + j] = acc[j];
                __syncthreads();
                if (group == 0 && s < rs.slots) {
                    for (int g = 1; g < used; g += kJoin) {
                        float p[kJoin][V];
#pragma unroll
                        for (int q = 0; q < kJoin; ++q) {
                            const int at = g + q < used ? g + q : used - 1;
#pragma unroll
                            for (int j = 0; j < V; ++j) p[q][j] = lds[(at * rs.lanes + lane) * V + j];
                        }
#pragma unroll
                        for (int q = 0; q < kJoin; ++q)
#pragma unroll
                            for (int j = 0; j < V; ++j) acc[j] += g + q < used ? p[q][j] : 0.0f;
                    }
                    store_slot<G, V>(dst, rs, s, acc, scale);
                }
            }
        }
    }
}

// How a gradient is cut up, and where its workspace's parts are.
struct GradPlan {
    int64_t tokens = 0, rows = 0, width = 0;
    int passes = 0, sort_blocks = 0, per_block = 0, chunk = 0;
    int64_t chunks = 0;
    bool one_sort = false;
    size_t keys[2] = {}, toks[2] = {}, hist = 0, begin = 0, end = 0, partial = 0, bytes = 0;
};

GradPlan grad_plan(int64_t tokens, int64_t rows, int64_t width)
{
    GradPlan g;
    g.tokens = tokens;
    g.rows = rows;
    g.width = width;
    while (g.passes < 4 && (uint64_t(rows) >> (8 * g.passes)) != 0) ++g.passes;  // keys run from 0 to rows
    if (g.passes == 0) g.passes = 1;
    int64_t per = 2 * kThreads;  // tokens of a sorting block (60000 tokens: 54.5, 48.0, 51.4 us for 1, 2, 4 a thread)
    while ((tokens + per - 1) / per > kMaxSortBlocks) per *= 2;
    g.per_block = int(per);
    g.sort_blocks = int((tokens + per - 1) / per);
    g.one_sort = tokens <= kOneSort;
    // Short chunks spread the sums over many blocks, long ones leave fewer partial sums of a
    // frequent row to add (ids by 1/rank, us at 32 / 64 / 128 / 256 tokens a chunk: 2000 tokens x
    // 1024 bfloat16 24.0 / 26.5 / 31.6 / 41.0; float16 32768 x 512 39.6 / 39.4 / 42.0 / 51.3,
    // 60000 x 256 48.1 / 44.9 / 45.1 / 48.8, 400000 x 64 120 / 91 / 76 / 69).  Up to 512 tokens the
    // rows' own threads add them and a launch is saved (500 tokens x 256 12.9 against 17.7).
    g.chunk = 32;
    while (g.chunk < kMostChunk && int64_t(g.chunk) * g.chunk * 16 < tokens) g.chunk *= 2;
    if (tokens <= 512) g.chunk = 512;
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
    g.begin = place(size_t(rows) * 4);
    g.end = place(size_t(rows) * 4);
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
    auto words = [&](size_t at) { return base ? reinterpret_cast<uint32_t *>(base + at) : nullptr; };
    const Bounds bounds{words(g.begin), words(g.end)};
    const uint32_t *keys = nullptr, *toks = nullptr;
    if (tokens > 0) {
        with_index(index, [&](auto i) {
            using I = decltype(i);
            Source<I> src{static_cast<const I *>(ids), nullptr, nullptr, rows, padding_idx};
            if (g.one_sort) {
                one_sort_kernel<I><<<1, kSortThreads, 0, hs>>>(src, int(tokens), g.passes, g.chunks == 1, bounds,
                                                              words(g.keys[0]), words(g.toks[0]));
                src.keys = words(g.keys[0]);
                src.toks = words(g.toks[0]);
            }
            for (int p = 0; p < g.passes && !g.one_sort; ++p) {
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
        float *const partial = reinterpret_cast<float *>(words(g.partial));
        const T *const dyp = static_cast<const T *>(dy);
        const bool inner = g.chunks > 1;
        const int64_t steps = (rs.slots + rs.lanes - 1) / rs.lanes, work = g.chunks * steps;
        auto go = [&](auto *grad) {
            using G = std::remove_reference_t<decltype(*grad)>;
            ct::mark_before(hs);
            if (inner)
                chunk_kernel<T, G><<<blocks_for(work, 1), kThreads, 0, hs>>>(dyp, keys, toks, tokens, rows, g.chunk, rs, steps,
                                                                            work, bounds, partial, scale, grad);
            // Where the table is long a block takes several rows in turn, so that few rounds of
            // blocks wait for begin and end (float16, us at 2 / 4 / 8 / 16 rows: 2000 tokens into
            // 128000 x 512 69.9 / 65.2 / 58.7 / 55.3, 32768 into 16384 x 512 40.0 / 39.1 / 40.3 /
            // 44.1; 400000 into 30000 x 64 at 1 / 2 / 4 71.2 / 71.8 / 74.2): as many as leave 1024
            // blocks, at most 16.
            const int64_t groups = kThreads / rs.lanes, turns = std::min({rows / (groups * 1024), kBlockRows / groups, int64_t(16)});
            const int ahead = int(std::max(turns, int64_t(1)));
            rows_kernel<T, G><<<blocks_for(rows, int(groups) * ahead), kThreads, 0, hs>>>(
                dyp, keys, toks, tokens, rows, g.chunk, rs, bounds, partial, inner, ahead, scale, grad);
            ct::mark_after(hs);
        };
        if (gt == CT_FLOAT32) go(static_cast<float *>(dtable));
        else go(static_cast<T *>(dtable));
    });
    st = ct::launch_status("embedding gradient launch failed", &err);
    return st == CT_OK ? CT_OK : fail(st, err);
}

}  // extern "C"

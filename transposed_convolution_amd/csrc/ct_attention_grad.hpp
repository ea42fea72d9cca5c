// ct_attention_grad.hpp -- attention's gradient, from the forward call's outputs o and lse:
//
//   P_ij = exp(s_ij - lse_i),  dP_ij = do_i . v_j,  delta_i = do_i . o_i,
//   dS_ij = scale P_ij (dP_ij - delta_i),
//   dv_j = sum_i P_ij do_i,  dk_j = sum_i dS_ij q_i,  dq_i = sum_j dS_ij k_j.
//
// Nothing of size Tq x Tk is stored: both kernels compute P and dP again.  One holds a block of keys
// and sums dk and dv over the rows, those of all query heads of its key head among them; the other
// holds a block of rows and sums dq over the keys.  That is 7 products where one kernel that also
// added into dq would take 5, but every sum has one owner and a fixed order: no atomics, the
// same bits every time.  8 x 4096 tokens, 8 heads of 64, float16: 1230 us, 22 of them for the rows'
// statistics, 764 for the keys (matrix unit busy 33 %), 496 for the rows (41 %); 560 TFLOP/s of the 5 products, 780
// of the 7.  Both kernels are bound as the forward one is, by the vector instructions of a score (8 here) and
// by waiting between dependent steps at two or three waves a SIMD.
//
// float16 has few exponents, and P is about 1 / Tk: P is held 2^15 times larger, and dS by a power of two
// that takes its largest possible value, scale * 2 |do| max|v|, to 2^15: of its row in the sum for dq, of its tile of
// rows in the sum for dk, which is scaled where that power changes.  So a row's gradient keeps its digits whatever
// size that of other rows has.  Both powers are taken out of the float32 sums at the end.  (One power for a whole
// head took 1217 us in the call above, and 1156 for 1207 with 4 x 4096 tokens and heads of 128; rows 2^22 smaller
// than another lost all digits.)
#pragma once

#include "ct_attention.hpp"

namespace ct {

template <class T>
constexpr bool kHalf = std::is_same_v<T, _Float16>;
constexpr int kHalfBias = 15;  // P of float16 is held 2^15 times larger

// What the kernels read of a row: lse in powers of two (+inf where the row sees nothing, which
// makes its P 0) and delta.
struct RowStat {
    float lse2, delta;
};

// Operands asked for ahead.  Gradient with heads of 64 / 128 / 256 (float16, 4096 tokens; with one power of dS a head), 2:
// 1242 / 1204 / 1280 us, 3: 1240 / 1140 / 1424, 4: 1230 / 1180 / 1305; registers are short in long heads.
template <class T, int DP>
constexpr int kAhead = DP * sizeof(T) > 256 ? 2 : DP * sizeof(T) > 128 ? 3 : 4;

constexpr int kStatRows = 64;  // rows or keys a block of stat_kernel looks at

// RowStat of the rows, and for float16 log2 of the largest norm of 64 rows' do, or of 64 keys' values, for each
// image and key head.  LANES lanes a row, 16 bytes a lane; one pass over o, do and v, 4.6 TB/s of 100 MB.
template <class T, int LANES>
__global__ __launch_bounds__(256) void stat_kernel(Attention a, RowStat *stat, float *top, int row_blocks, int blocks)
{
    constexpr int V = kVec<T>;
    const int in = threadIdx.x & (LANES - 1), first = threadIdx.x / LANES;
    const int nh = blockIdx.x / blocks, b = blockIdx.x - nh * blocks, n = nh / a.Hkv, hk = nh - n * a.Hkv;
    const int start = a.start(n), len = a.length(n, start), from = a.first_token(len, start);
    float most = 0.0f;
    const bool rows = b < row_blocks;
    const int base = (rows ? b : b - row_blocks) * kStatRows;
#pragma unroll
    for (int i = 0; i < kStatRows * LANES / 256; ++i) {
        const int at = base + first + i * (256 / LANES);
        float sum = 0.0f, sq = 0.0f;
        if (rows) {
            const int t = a.by_g.div(at), h = hk * a.G + at - t * a.G;
            const bool sees = at < a.R && t >= from;
            if (sees) {
                const T *po = static_cast<const T *>(a.o.p) + n * a.o.n + t * a.o.t + h * a.o.h;
                const T *pd = static_cast<const T *>(a.d_o.p) + n * a.d_o.n + t * a.d_o.t + h * a.d_o.h;
                for (int d = in * V; d < a.D; d += LANES * V) {
                    const Raw<T, V> x = load_chunk<T>(pd + d, a.D - d, a.D % V), y = load_chunk<T>(po + d, a.D - d, a.D % V);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        sum = fmaf(float(x[j]), float(y[j]), sum);
                        if (kHalf<T>) sq = fmaf(float(x[j]), float(x[j]), sq);
                    }
                }
            }
#pragma unroll
            for (int s = LANES / 2; s; s >>= 1) sum += __shfl_xor(sum, s);
            if (in == 0 && at < a.R)
                stat[int64_t(nh) * a.R + at] = {sees ? a.lse[(int64_t(n) * a.H + h) * a.Tq + t] * kLog2e : INFINITY, sum};
        } else if (at < len) {
            const T *p = static_cast<const T *>(a.v.p) + n * a.v.n + at * a.v.t + hk * a.v.h;
            for (int d = in * V; d < a.D; d += LANES * V) {
                const Raw<T, V> x = load_chunk<T>(p + d, a.D - d, a.D % V);
#pragma unroll
                for (int j = 0; j < V; ++j) sq = fmaf(float(x[j]), float(x[j]), sq);
            }
        }
        if (kHalf<T>) {
#pragma unroll
            for (int s = LANES / 2; s; s >>= 1) sq += __shfl_xor(sq, s);
            // one that is not finite says nothing about the others, whose score gradients would become zeros
            most = fmaxf(most, sq < INFINITY ? sq : 0.0f);
        }
    }
    if constexpr (kHalf<T>) {
        __shared__ float shared[256 / LANES];
        if (in == 0) shared[first] = most;
        __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int i = 1; i < 256 / LANES; ++i) most = fmaxf(most, shared[i]);
            top[blockIdx.x] = 0.5f * log2f(most);
        }
    }
}

// log2 of the largest norm of the values of an image and key head, of its first `count` blocks of 64 keys.
template <class T, int THREADS>
__device__ __forceinline__ float value_top(const float *top, int count)
{
    if constexpr (!kHalf<T>) {
        return 0.0f;
    } else {
        __shared__ float shared[THREADS / 64];
        float most = -INFINITY;
        for (int b = threadIdx.x; b < count; b += THREADS) most = fmaxf(most, top[b]);
#pragma unroll
        for (int s = 32; s; s >>= 1) most = fmaxf(most, __shfl_xor(most, s));
        if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = most;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < THREADS / 64; ++i) most = fmaxf(most, shared[i]);
        return most;
    }
}
// A value that a wave's lanes share, in a scalar register.
__device__ __forceinline__ float uniform(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}
// The power of two by which dS is held whose magnitude has log2 below `bound`.  2^60 is enough for any: what is below
// 2^-25 there is 2^-85 and nothing in float16, however many are summed.  (A row that is not finite ends at either end;
// its score gradients are not finite then.)
__device__ __forceinline__ int grad_shift(float bound)
{
    return kHalfBias - int(ceilf(fminf(fmaxf(bound, float(kHalfBias - 60)), 200.0f)));
}
// c / 2^shift
template <class T, int DB>
__device__ __forceinline__ void unshift(f32x16 (&c)[DB], int shift)
{
    if constexpr (kHalf<T>) {
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int r = 0; r < 16; ++r) c[db][r] = ldexpf(c[db][r], -shift);
    }
}

// What the blocks of a call share, and how the work of one kind of block is cut.
struct GradShared {
    const RowStat *stat;
    const float *top;
    int row_blocks, blocks;
};
struct Share {
    int tiles, splits, chunk;
};

// How long heads are held: the two accumulators of a wave's 32 keys take a register for each element of the
// head, and its keys' and values' operands an eighth of one a byte.  Up to 128 bytes a head all of it fits beside
// the scores at two waves a SIMD.  Beyond, the values' operands are read from LDS each time, at 256 bytes the keys'
// too: 8 waves share the rows' tile then, so that one block of 16-bit heads of 128 has 147 KB (4096 tokens, 4 x 8
// heads, float16: 1410 us with 4 waves and the keys in registers, some of them in scratch, 1325 with 8, 1204 with the keys
// in LDS).  At 256 elements of 16 bits two waves share the 32 keys, each with half of the columns: both make all
// scores, 6 products for 4, but one wave kept 900 bytes in scratch (2 x 4096 tokens, 4 heads, float16: 3927 us, now 1326).
template <class T, int DP>
struct KeyPlan {
    static constexpr int kBytes = DP * int(sizeof(T));
    static constexpr int kParts = DP == 256 && sizeof(T) == 2 ? 2 : 1;
    static constexpr bool kValues = kBytes > 128 && kBytes <= 512, kKeys = kParts == 2 || kBytes == 256;  // in LDS
    static constexpr int kWaves = wide_keys(kBytes) ? 8 : 4;
};

// dk and dv of a block of keys from RT rows at a time.
template <class T, int DP, int WAVES, int RT>
struct KeyGrad {
    using Plan = KeyPlan<T, DP>;
    static constexpr int PARTS = WAVES == 1 ? 1 : Plan::kParts, KEYS = WAVES / PARTS * 32;
    static constexpr bool LDSV = Plan::kValues, LDSK = Plan::kKeys;
    // two buffers where other waves are to be waited for and registers are not short
    static constexpr int BUFS = WAVES == 1 || Plan::kBytes > 128 ? 1 : 2;
    struct Lds {
        T tile[BUFS][2][RT * DP], values[LDSV ? KEYS * DP : 8], keys[LDSK ? KEYS * DP : 8];
        float lse2[BUFS][RT], delta[BUFS][RT];
        int ends[BUFS][RT];
    };
    __device__ static __forceinline__ void run(const Attention &a, const GradShared &shared, float *part, Share sh, int block,
                                               int count, Lds &lds)
    {
        using L = Tile<T, DP>;
        constexpr int KS = DP / 16, DB = DP / 32 / PARTS, RB = RT / 32, THREADS = WAVES * 64;
        constexpr int P = kAhead<T, DP>;
        const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = lane >> 5;
        const int tiles = sh.tiles, splits = sh.splits, chunk = sh.chunk;

        int w = xcd_remap(block, count);
        const int split = w % splits;
        w /= splits;
        const int nh = w / tiles, tile = tiles - 1 - long_first(w - nh * tiles, tiles, a.N * a.Hkv), n = nh / a.Hkv, hk = nh - n * a.Hkv;
        const int start = a.start(n), len = a.length(n, start), from_token = a.first_token(len, start);
        const int group = wave / PARTS * 32 + (lane & 31), column = wave % PARTS * DB;  // the lane's key, the wave's first 32 columns
        const int block_key = tile * KEYS, key0 = block_key + wave / PARTS * 32, key = block_key + group;
        // rows from the first that sees the block's first key on, of this split's chunk
        const int from = a.causal ? max(0, min(block_key - start, a.Tq)) * a.G : 0;
        const int rt0 = max(from, split * chunk) / RT, rt1 = block_key < len ? (min(a.R, split * chunk + chunk) + RT - 1) / RT : 0;
        if (splits > 1 && rt0 >= rt1) return;  // the join passes over it

        Frag<T> k[LDSK ? 1 : KS], v[LDSV ? 1 : KS];
        const T *kp = static_cast<const T *>(a.k.p) + n * a.k.n + key * a.k.t + hk * a.k.h;
        const T *vp = static_cast<const T *>(a.v.p) + n * a.v.n + key * a.v.t + hk * a.v.h;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            // a lane reads from LDS what it put there (or the other wave of its keys, behind the loop's first barrier)
            const Frag<T> f = load_frag<T>(kp, ks * 16 + half * 8, key < len ? a.D : 0);
            if constexpr (LDSK) L::put(lds.keys, group, ks, half, f);
            else k[ks] = f;
            const Frag<T> g = load_frag<T>(vp, ks * 16 + half * 8, key < len ? a.D : 0);
            if constexpr (LDSV) L::put(lds.values, group, ks, half, g);
            else v[ks] = g;
        }
        f32x16 dk[DB], dv[DB];
#pragma unroll
        for (int db = 0; db < DB; ++db) dk[db] = dv[db] = f32x16{};

        const float bias = kHalf<T> ? float(kHalfBias) : 0.0f, c = a.scale * kLog2e;
        // float16: the power of the sums so far, that of the tile in LDS, log2 of what goes with a row's norm in dS
        const float *top = shared.top + int64_t(nh) * shared.blocks;
        const float rest = uniform(1.0f + log2f(a.scale) + value_top<T, THREADS>(top + shared.row_blocks, shared.blocks - shared.row_blocks));
        int shift = 0, next = 60;
        float factor = a.scale, norm = 0.0f;

        const T *qp = static_cast<const T *>(a.q.p) + n * a.q.n + hk * a.G * a.q.h;
        const T *dp = static_cast<const T *>(a.d_o.p) + n * a.d_o.n + hk * a.G * a.d_o.h;
        const RowStat *sp = shared.stat + int64_t(nh) * a.R;
        Mover<T, DP, RT, THREADS> qm(tid), dm(tid);
        RowStat mine{INFINITY, 0.0f};
        int end = 0;
        auto load = [&](int rt) {
            if constexpr (kHalf<T>) norm = top[rt * RT / kStatRows];
            if (a.G == 1 && rt * RT >= from_token) {
                qm.load(qp + int64_t(rt) * RT * a.q.t, a.q.t, a.R - rt * RT, a.D);
                dm.load(dp + int64_t(rt) * RT * a.d_o.t, a.d_o.t, a.R - rt * RT, a.D);
            } else {
                // rows that see nothing are zeros: what stands there takes no part
                auto place = [&](int r, const T *p, const Strided &s) -> const T * {
                    const int row = rt * RT + r, t = a.by_g.div(row);
                    return row < a.R && t >= from_token ? p + t * s.t + (row - t * a.G) * s.h : nullptr;
                };
                qm.load(a.D, [&](int r) { return place(r, qp, a.q); });
                dm.load(a.D, [&](int r) { return place(r, dp, a.d_o); });
            }
            if (tid < RT) {
                const int row = rt * RT + tid;
                mine = row < a.R ? sp[row] : RowStat{INFINITY, 0.0f};
                // how many of the keys from the block's first on the row sees
                end = row < a.R ? a.seen(len, start, a.by_g.div(row)) - block_key : 0;
            }
        };
        auto store = [&](int buf) {
            qm.store(lds.tile[buf][0]);
            dm.store(lds.tile[buf][1]);
            float by = a.scale;
            if constexpr (kHalf<T>) {
                // it stays while it is at most 2 below what the tile allows: norms of like size change nothing
                const int allowed = __builtin_amdgcn_readfirstlane(grad_shift(norm + rest));
                if (next > allowed || (next < allowed - 2 && norm > -INFINITY)) next = allowed;
                by = ldexpf(a.scale, next - kHalfBias);
            }
            if (tid < RT) {
                lds.lse2[buf][tid] = mine.lse2 - bias;
                lds.delta[buf][tid] = mine.delta * by;
                lds.ends[buf][tid] = end;
            }
        };

        if (rt0 < rt1) {
            load(rt0);
            if (BUFS == 2) store(0);
        }
        for (int rt = rt0; rt < rt1; ++rt) {
            __syncthreads();
            const int buf = BUFS == 2 ? (rt - rt0) & 1 : 0;
            if (BUFS == 1) {
                store(0);
                __syncthreads();
            }
            const int held = next;  // this tile's
            if (rt + 1 < rt1) load(rt + 1);
            const T *ql = lds.tile[buf][0], *dl = lds.tile[buf][1];
            if (WAVES > 4 && a.causal && a.seen(len, start, a.by_g.div(min(rt * RT + RT, a.R) - 1)) <= key0) {
                // nothing of this wave's (the test costs shorter blocks more than it saves)
                if (BUFS == 2 && rt + 1 < rt1) store(buf ^ 1);
                continue;
            }
            if (kHalf<T> && shift != held) {
                unshift<T, DB>(dk, shift - held);
                shift = held;
                factor = uniform(ldexpf(a.scale, shift - kHalfBias));
            }
            // the tile's first row sees fewest keys; rows that do not exist have P = 0
            const bool whole = key0 + 32 <= a.seen(len, start, a.by_g.div(rt * RT));
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                f32x16 s = {}, g = {};
                Ahead<T, 2 * KS, P> rows;
                auto row = [&](int i) { return L::by_rows(i < KS ? ql : dl, rb * 32 + (lane & 31), i % KS, half); };
                rows.prime(row);
                rows.run(row, [&](int i, const Frag<T> &f) {
                    if (i < KS) {
                        if constexpr (LDSK) s = mma(f, L::by_rows(lds.keys, group, i, half), s);
                        else s = mma(f, k[i], s);
                    } else {
                        if constexpr (LDSV) g = mma(f, L::by_rows(lds.values, group, i - KS, half), g);
                        else g = mma(f, v[i - KS], g);
                    }
                });
                Ahead<T, 4 * DB, P> columns;
                auto col = [&](int i) { return L::by_columns(i & 1 ? ql : dl, rb * 32 + i / (2 * DB) * 16, column + i / 2 % DB, lane); };
                columns.prime(col);
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4) {
                    const int at = rb * 32 + 8 * r4 + 4 * half;
                    const f32x4 le = *reinterpret_cast<const f32x4 *>(lds.lse2[buf] + at), de = *reinterpret_cast<const f32x4 *>(lds.delta[buf] + at);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = 4 * r4 + j;
                        const float p = exp2_fast(fmaf(s[r], c, -le[j]));
                        s[r] = p;
                        g[r] = p * fmaf(g[r], factor, -de[j]);
                    }
                }
                if (!whole) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const bool sees = key - block_key < lds.ends[buf][rb * 32 + c_row(r, half)];
                        s[r] = sees ? s[r] : 0.0f;
                        g[r] = sees ? g[r] : 0.0f;
                    }
                }
                Frag<T> pf, gf;
                columns.run(col, [&](int i, const Frag<T> &f) {
                    if (i % (2 * DB) == 0) pf = operand<T>(s, i / (2 * DB)), gf = operand<T>(g, i / (2 * DB));
                    if (i & 1) dk[i / 2 % DB] = mma(f, gf, dk[i / 2 % DB]);
                    else dv[i / 2 % DB] = mma(f, pf, dv[i / 2 % DB]);
                });
            }
            if (BUFS == 2 && rt + 1 < rt1) store(buf ^ 1);
        }
        if (key >= a.Tk) return;
        unshift<T, DB>(dk, shift);
        const float undo_v = exp2f(-bias);
        const int64_t at = ((int64_t(n) * a.Tk + key) * a.Hkv + hk) * a.D + column * 32;
        const int D = a.D - column * 32;
        if (splits == 1) {
            store_columns<T, DB>(static_cast<T *>(a.dk) + at, dk, 1.0f, D, half);
            store_columns<T, DB>(static_cast<T *>(a.dv) + at, dv, undo_v, D, half);
        } else {
            const int64_t all = int64_t(a.N) * a.Tk * a.Hkv * a.D;
            float *to = part + int64_t(split) * 2 * all + at;
            store_columns<float, DB>(to, dk, 1.0f, D, half);
            store_columns<float, DB>(to + all, dv, undo_v, D, half);
        }
    }
};

// dq of a block of rows, a wave 32 of them, from KT keys at a time.
template <class T, int DP, int WAVES, int KT>
struct RowGrad {
    static constexpr int BUFS = WAVES == 1 ? 1 : 2;
    struct Lds {
        T tile[BUFS][2][KT * DP];
    };
    __device__ static __forceinline__ void run(const Attention &a, const GradShared &shared, float *part, Share sh, int block,
                                               int count, Lds &lds)
    {
        using L = Tile<T, DP>;
        constexpr int KS = DP / 16, DB = DP / 32, KB = KT / 32, THREADS = WAVES * 64, ROWS = WAVES * 32;
        constexpr int P = kAhead<T, DP>;
        const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = lane >> 5;
        const int tiles = sh.tiles, splits = sh.splits, chunk = sh.chunk;

        int w = xcd_remap(block, count);
        const int split = w % splits;
        w /= splits;
        const int nh = w / tiles, tile = long_first(w - nh * tiles, tiles, a.N * a.Hkv), n = nh / a.Hkv, hk = nh - n * a.Hkv;
        const int start = a.start(n), len = a.length(n, start), from_token = a.first_token(len, start);
        const int block_row = tile * ROWS, row0 = block_row + wave * 32;
        // keys the block looks at, of this split's chunk
        const int most_seen = a.seen(len, start, a.by_g.div(min(block_row + ROWS, a.R) - 1)), want = min(most_seen, split * chunk + chunk);
        const int kt0 = split * chunk / KT, kt1 = (want + KT - 1) / KT;
        if (splits > 1 && kt0 >= kt1) return;  // the join passes over it

        const float bias = kHalf<T> ? float(kHalfBias) : 0.0f, c = a.scale * kLog2e;
        // of the keys that the block's rows see, whatever this split has of them: delta is of all
        const float most = value_top<T, THREADS>(shared.top + int64_t(nh) * shared.blocks + shared.row_blocks, (most_seen + kStatRows - 1) / kStatRows);

        const int row = row0 + (lane & 31), t = a.by_g.div(row), h = hk * a.G + row - t * a.G;
        const bool sees = row < a.R && t >= from_token;
        const int seen = sees ? a.seen(len, start, t) : 0;
        const RowStat mine = row < a.R ? shared.stat[int64_t(nh) * a.R + row] : RowStat{INFINITY, 0.0f};
        Frag<T> q[KS], d_o[KS];
        const T *qp = static_cast<const T *>(a.q.p) + n * a.q.n + t * a.q.t + h * a.q.h;
        const T *dp = static_cast<const T *>(a.d_o.p) + n * a.d_o.n + t * a.d_o.t + h * a.d_o.h;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            q[ks] = load_frag<T>(qp, ks * 16 + half * 8, sees ? a.D : 0);
            d_o[ks] = load_frag<T>(dp, ks * 16 + half * 8, sees ? a.D : 0);
        }
        int shift = 0;
        float factor = a.scale;
        if constexpr (kHalf<T>) {  // a row is a lane's and the lane's 32 above
            float square = 0.0f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int j = 0; j < 8; ++j) square = fmaf(float(d_o[ks][j]), float(d_o[ks][j]), square);
            shift = grad_shift(1.0f + log2f(a.scale) + most + 0.5f * log2f(half_sum(square)));
            factor = ldexpf(a.scale, shift - kHalfBias);
        }
        const float lse2 = mine.lse2 - bias, delta = mine.delta * factor;
        const bool rows = row0 < a.R;
        const int whole = rows ? a.seen(len, start, a.by_g.div(row0)) / KT : 0;
        const int none = rows ? (a.seen(len, start, a.by_g.div(min(row0 + 32, a.R) - 1)) + KT - 1) / KT : 0;

        const T *kp = static_cast<const T *>(a.k.p) + n * a.k.n + hk * a.k.h;
        const T *vp = static_cast<const T *>(a.v.p) + n * a.v.n + hk * a.v.h;
        Mover<T, DP, KT, THREADS> km(tid), vm(tid);
        auto load = [&](int kt) {
            km.load(kp + int64_t(kt) * KT * a.k.t, a.k.t, len - kt * KT, a.D);
            vm.load(vp + int64_t(kt) * KT * a.v.t, a.v.t, len - kt * KT, a.D);
        };
        f32x16 dq[DB];
#pragma unroll
        for (int db = 0; db < DB; ++db) dq[db] = f32x16{};

        auto store = [&](int buf) {
            km.store(lds.tile[buf][0]);
            vm.store(lds.tile[buf][1]);
        };
        if (kt0 < kt1) {
            load(kt0);
            if (BUFS == 2) store(0);
        }
        for (int kt = kt0; kt < kt1; ++kt) {
            __syncthreads();
            const int buf = BUFS == 2 ? (kt - kt0) & 1 : 0;
            if (BUFS == 1) {
                store(0);
                __syncthreads();
            }
            if (kt + 1 < kt1) load(kt + 1);
            if (kt < none) {
                const T *kl = lds.tile[buf][0], *vl = lds.tile[buf][1];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    f32x16 s = {}, g = {};
                    Ahead<T, 2 * KS, P> rows;
                    auto row = [&](int i) { return L::by_rows(i < KS ? kl : vl, kb * 32 + (lane & 31), i % KS, half); };
                    rows.prime(row);
                    rows.run(row, [&](int i, const Frag<T> &f) {
                        if (i < KS) s = mma(f, q[i], s);
                        else g = mma(f, d_o[i - KS], g);
                    });
                    Ahead<T, 2 * DB, P> columns;
                    auto col = [&](int i) { return L::by_columns(kl, kb * 32 + i / DB * 16, i % DB, lane); };
                    columns.prime(col);
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const float p = exp2_fast(fmaf(s[r], c, -lse2));
                        g[r] = p * fmaf(g[r], factor, -delta);
                    }
                    if (kt >= whole) {
                        const int end = seen - kt * KT;
#pragma unroll
                        for (int r = 0; r < 16; ++r) g[r] = kb * 32 + c_row(r, half) < end ? g[r] : 0.0f;
                    }
                    Frag<T> gf;
                    columns.run(col, [&](int i, const Frag<T> &f) {
                        if (i % DB == 0) gf = operand<T>(g, i / DB);
                        dq[i % DB] = mma(f, gf, dq[i % DB]);
                    });
                }
            }
            if (BUFS == 2 && kt + 1 < kt1) store(buf ^ 1);
        }
        if (row >= a.R) return;
        unshift<T, DB>(dq, shift);
        const int64_t at = ((int64_t(n) * a.Tq + t) * a.H + h) * a.D;
        if (splits == 1) store_columns<T, DB>(static_cast<T *>(a.dq) + at, dq, 1.0f, a.D, half);
        else store_columns<float, DB>(part + int64_t(split) * a.N * a.Tq * a.H * a.D + at, dq, 1.0f, a.D, half);
    }
};

// The kernels: each kind of block by itself, or, for small calls, both in one launch (4 x 257 tokens, 3 heads of 36,
// float32: 32 us, 44.6 with a launch each).  Row blocks of heads of 128 with 8 waves took 461 us where 4 take 446.
template <class T, int DP, int WAVES, int RT>
__global__ __launch_bounds__(WAVES * 64, DP * sizeof(T) <= 256 ? 2 : 1) void key_grad_kernel(Attention a, GradShared shared, float *part, Share sh)
{
    using K = KeyGrad<T, DP, WAVES, RT>;
    __shared__ __attribute__((aligned(16))) char lds[sizeof(typename K::Lds)];
    K::run(a, shared, part, sh, blockIdx.x, gridDim.x, *reinterpret_cast<typename K::Lds *>(lds));
}
template <class T, int DP, int WAVES, int KT>
__global__ __launch_bounds__(WAVES * 64, DP * sizeof(T) <= 128 ? 3 : DP * sizeof(T) <= 256 ? 2 : 1) void row_grad_kernel(
    Attention a, GradShared shared, float *part, Share sh)
{
    using K = RowGrad<T, DP, WAVES, KT>;
    __shared__ __attribute__((aligned(16))) char lds[sizeof(typename K::Lds)];
    K::run(a, shared, part, sh, blockIdx.x, gridDim.x, *reinterpret_cast<typename K::Lds *>(lds));
}
template <class T, int DP>
__global__ __launch_bounds__(64) void both_grad_kernel(Attention a, GradShared shared, float *key_part, Share keys, int key_count,
                                                       float *row_part, Share rows)
{
    using K = KeyGrad<T, DP, 1, 32>;
    using R = RowGrad<T, DP, 1, 32>;
    constexpr size_t BYTES = sizeof(typename K::Lds) > sizeof(typename R::Lds) ? sizeof(typename K::Lds) : sizeof(typename R::Lds);
    __shared__ __attribute__((aligned(16))) char lds[BYTES];
    const int b = blockIdx.x;
    if (b < key_count) K::run(a, shared, key_part, keys, b, key_count, *reinterpret_cast<typename K::Lds *>(lds));
    else R::run(a, shared, row_part, rows, b - key_count, int(gridDim.x) - key_count, *reinterpret_cast<typename R::Lds *>(lds));
}

// Sums of partial results, in their order, a block a token: first the tokens of the keys (dk and dv), then
// those of the queries.  Chunks that a block of keys or rows had nothing of are passed over.  Bound by memory: 4097
// causal tokens, 16 heads over 4 of 128, leave 184 MB of parts that take 49 us.
template <class T>
__global__ __launch_bounds__(256) void grad_join_kernel(Attention a, AttendGradPlan p, const float *key_part, const float *row_part,
                                                        int key_tokens, Div31 by_d)
{
    int token = blockIdx.x;
    if (token < key_tokens) {
        const int n = token / a.Tk, block_key = (token - n * a.Tk) / p.key_span * p.key_span;
        const int start = a.start(n), len = a.length(n, start);
        const int from = a.causal ? max(0, min(block_key - start, a.Tq)) * a.G : 0;
        const int s0 = from / p.row_chunk, s1 = block_key < len ? p.row_splits : 0;
        const int count = a.Hkv * a.D;
        const int64_t all = int64_t(a.N) * a.Tk * count, base = int64_t(token) * count;
        for (int i = threadIdx.x; i < 2 * count; i += 256) {
            const int64_t at = i < count ? base + i : all + base + i - count;
            float sum = 0.0f;
#pragma unroll 4
            for (int s = s0; s < s1; ++s) sum += key_part[s * 2 * all + at];
            (i < count ? static_cast<T *>(a.dk)[at] : static_cast<T *>(a.dv)[at - all]) = T(sum);
        }
    } else {
        token -= key_tokens;
        const int n = token / a.Tq, t = token - n * a.Tq, start = a.start(n), len = a.length(n, start);
        const int count = a.H * a.D;
        const int64_t all = int64_t(a.N) * a.Tq * count, base = int64_t(token) * count;
        for (int i = threadIdx.x; i < count; i += 256) {
            const int h = by_d.div(i), row = t * a.G + h - a.by_g.div(h) * a.G;
            const int want = a.seen(len, start, a.by_g.div(min(row / p.row_span * p.row_span + p.row_span, a.R) - 1));
            const int s1 = min(p.key_splits, (want + p.key_chunk - 1) / p.key_chunk);
            float sum = 0.0f;
#pragma unroll 4
            for (int s = 0; s < s1; ++s) sum += row_part[s * all + base + i];
            static_cast<T *>(a.dq)[base + i] = T(sum);
        }
    }
}

template <class T>
void launch_attend_grad(const Attention &a, const AttendGradPlan &p, char *ws, hipStream_t st)
{
    RowStat *stat = reinterpret_cast<RowStat *>(ws + p.stat);
    float *top = reinterpret_cast<float *>(ws + p.top);
    float *key_part = reinterpret_cast<float *>(ws + p.key_part), *row_part = reinterpret_cast<float *>(ws + p.row_part);
    const int heads = a.N * a.Hkv, row_blocks = (a.R + kStatRows - 1) / kStatRows;
    const int blocks = row_blocks + (kHalf<T> ? (a.Tk + kStatRows - 1) / kStatRows : 0);
    if (heads * int64_t(blocks) > 0) {
        if (a.D * int(sizeof(T)) <= 128) stat_kernel<T, 8><<<unsigned(heads * blocks), 256, 0, st>>>(a, stat, top, row_blocks, blocks);
        else stat_kernel<T, 16><<<unsigned(heads * blocks), 256, 0, st>>>(a, stat, top, row_blocks, blocks);
    }
    const GradShared shared = {stat, top, row_blocks, blocks};
    const int key_tiles = (a.Tk + p.key_span - 1) / p.key_span, row_tiles = (a.R + p.row_span - 1) / p.row_span;
    const Share keys = {key_tiles, p.row_splits, p.row_chunk}, rows = {row_tiles, p.key_splits, p.key_chunk};
    const int key_count = heads * key_tiles * p.row_splits, row_count = heads * row_tiles * p.key_splits;
    with_head(a.D, [&](auto head) {
        constexpr int DP = decltype(head)::value, TILE = DP * sizeof(T) > 128 ? 32 : 64;
        if constexpr (DP * sizeof(T) <= kOneWaveBytes) {
            if (p.waves == 1) {
                both_grad_kernel<T, DP><<<unsigned(key_count + row_count), 64, 0, st>>>(a, shared, key_part, keys, key_count, row_part, rows);
                return;
            }
        }
        if (key_count) key_grad_kernel<T, DP, KeyPlan<T, DP>::kWaves, TILE><<<unsigned(key_count), KeyPlan<T, DP>::kWaves * 64, 0, st>>>(a, shared, key_part, keys);
        if (row_count) row_grad_kernel<T, DP, 4, TILE><<<unsigned(row_count), 256, 0, st>>>(a, shared, row_part, rows);
    });
    const int key_tokens = p.row_splits > 1 ? a.N * a.Tk : 0, row_tokens = p.key_splits > 1 ? a.N * a.Tq : 0;
    if (key_tokens + row_tokens > 0)
        grad_join_kernel<T><<<unsigned(key_tokens + row_tokens), 256, 0, st>>>(a, p, key_part, row_part, key_tokens, Div31(a.D));
}

}  // namespace ct

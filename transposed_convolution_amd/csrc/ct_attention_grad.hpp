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
// same bits every time.
//
// float16 has few exponents, and P is about 1 / Tk: P is held 2^15 times larger, and dS by the power
// of two that takes its largest possible value, scale * 2 max|do| max|v|, to 2^15.  Both are divided
// out of the float32 sums at the end.
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

constexpr int kStatRows = 64;  // rows or keys a block of stat_kernel looks at

// A wave a row: RowStat of the rows, and for float16 the largest norm of 64 rows' do, or of 64 keys'
// values, for each image and key head.
template <class T>
__global__ __launch_bounds__(256) void stat_kernel(Attention a, RowStat *stat, float *top, int64_t row_blocks, int64_t blocks)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t nh = blockIdx.x / blocks, b = blockIdx.x % blocks, n = nh / a.Hkv, hk = nh % a.Hkv;
    const int64_t len = a.length(n), start = a.start(n);
    float most = 0.0f;
    __shared__ float shared[4];
    if (b < row_blocks) {
        for (int i = wave; i < kStatRows; i += 4) {
            const int64_t row = b * kStatRows + i;
            if (row >= a.R) break;
            const int64_t t = row / a.G, h = hk * a.G + row % a.G;
            const bool sees = a.seen(len, start, t) > 0;
            float sum = 0.0f, sq = 0.0f;
            if (sees) {
                const T *po = static_cast<const T *>(a.o.p) + n * a.o.n + t * a.o.t + h * a.o.h;
                const T *pd = static_cast<const T *>(a.d_o.p) + n * a.d_o.n + t * a.d_o.t + h * a.d_o.h;
                for (int d = lane; d < a.D; d += 64) {
                    const float g = float(pd[d]);
                    sum = fmaf(g, float(po[d]), sum);
                    sq = fmaf(g, g, sq);
                }
            }
#pragma unroll
            for (int s = 32; s; s >>= 1) {
                sum += __shfl_xor(sum, s);
                sq += __shfl_xor(sq, s);
            }
            most = fmaxf(most, sq);
            if (lane == 0)
                stat[nh * a.R + row] = {sees ? a.lse[(n * a.H + h) * a.Tq + t] * kLog2e : INFINITY, sum};
        }
    } else {
        for (int i = wave; i < kStatRows; i += 4) {
            const int64_t j = (b - row_blocks) * kStatRows + i;
            if (j >= len) break;
            const T *p = static_cast<const T *>(a.v.p) + n * a.v.n + j * a.v.t + hk * a.v.h;
            float sq = 0.0f;
            for (int d = lane; d < a.D; d += 64) sq = fmaf(float(p[d]), float(p[d]), sq);
#pragma unroll
            for (int s = 32; s; s >>= 1) sq += __shfl_xor(sq, s);
            most = fmaxf(most, sq);
        }
    }
    if constexpr (kHalf<T>) {
        if (lane == 0) shared[wave] = most;
        __syncthreads();
        if (threadIdx.x == 0)
            top[blockIdx.x] = sqrtf(fmaxf(fmaxf(shared[0], shared[1]), fmaxf(shared[2], shared[3])));
    }
}

// The power of two dS of an image and key head is held by; the same in both kernels.
template <class T, int THREADS>
__device__ __forceinline__ int grad_shift(const Attention &a, const float *top, int64_t nh, int64_t row_blocks, int64_t blocks)
{
    if constexpr (!kHalf<T>) {
        return 0;
    } else {
        __shared__ float shared[2][THREADS / 64];
        float most[2] = {0.0f, 0.0f};
        for (int64_t b = threadIdx.x; b < blocks; b += THREADS) {
            const int of = b < row_blocks ? 0 : 1;
            most[of] = fmaxf(most[of], top[nh * blocks + b]);
        }
#pragma unroll
        for (int of = 0; of < 2; ++of) {
#pragma unroll
            for (int s = 32; s; s >>= 1) most[of] = fmaxf(most[of], __shfl_xor(most[of], s));
            if ((threadIdx.x & 63) == 0) shared[of][threadIdx.x >> 6] = most[of];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < THREADS / 64; ++i) {
            most[0] = fmaxf(most[0], shared[0][i]);
            most[1] = fmaxf(most[1], shared[1][i]);
        }
        // logarithms, not products: the norms' product may leave float32
        const float bound = log2f(most[0]) + log2f(most[1]) + log2f(a.scale) + 1.0f;
        // (nothing but zeros, or a value that is not finite: any shift will do)
        return bound > -100.0f && bound < 100.0f ? kHalfBias - int(ceilf(bound)) : 0;
    }
}

// dk and dv of a block of keys, from the rows [rt0, rt1) of RT.
template <class T, int DP, int KB, int WAVES, int RT>
__global__ __launch_bounds__(WAVES * 64) void key_grad_kernel(Attention a, const RowStat *stat, const float *top,
                                                              int64_t row_blocks, int64_t blocks, int64_t tiles)
{
    using L = Tile<T, DP>;
    constexpr int KS = DP / 16, DB = DP / 32, RB = RT / 32, THREADS = WAVES * 64;
    __shared__ __attribute__((aligned(16))) T lds[2][RT * DP];
    __shared__ __attribute__((aligned(16))) float lse2[RT], delta[RT];
    __shared__ int ends[RT];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, half = lane >> 5;

    int64_t w = xcd_remap(blockIdx.x, gridDim.x);
    const int split = int(w % a.splits);
    w /= a.splits;
    const int64_t tile = w % tiles, nh = w / tiles, n = nh / a.Hkv, hk = nh % a.Hkv;
    const int64_t len = a.length(n), start = a.start(n);
    const int64_t block_key = tile * (WAVES * KB * 32), key0 = block_key + wave * (KB * 32);

    Frag<T> k[KB][KS], v[KB][KS];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        const int64_t key = key0 + kb * 32 + (lane & 31);
        const T *kp = static_cast<const T *>(a.k.p) + n * a.k.n + key * a.k.t + hk * a.k.h;
        const T *vp = static_cast<const T *>(a.v.p) + n * a.v.n + key * a.v.t + hk * a.v.h;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            k[kb][ks] = load_frag<T>(kp, ks * 16 + half * 8, key < len ? a.D : 0);
            v[kb][ks] = load_frag<T>(vp, ks * 16 + half * 8, key < len ? a.D : 0);
        }
    }
    f32x16 dk[KB][DB], dv[KB][DB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int db = 0; db < DB; ++db) dk[kb][db] = dv[kb][db] = f32x16{};

    const int shift = grad_shift<T, THREADS>(a, top, nh, row_blocks, blocks);
    const float bias = kHalf<T> ? float(kHalfBias) : 0.0f, c = a.scale * kLog2e;
    const float factor = a.scale * exp2f(float(shift) - bias);

    // rows from the first that sees the block's first key on; this split's share of them
    int64_t from = 0;
    if (a.causal) from = max(int64_t(0), min(block_key - start, a.Tq)) * a.G;
    const int64_t t0 = from / RT, t1 = block_key < len ? (a.R + RT - 1) / RT : 0, each = t1 > t0 ? (t1 - t0 + a.splits - 1) / a.splits : 0;
    const int64_t rt0 = t0 + split * each, rt1 = min(t1, rt0 + each);

    const T *qp = static_cast<const T *>(a.q.p) + n * a.q.n + hk * a.G * a.q.h;
    const T *dp = static_cast<const T *>(a.d_o.p) + n * a.d_o.n + hk * a.G * a.d_o.h;
    Mover<T, DP, RT, THREADS> qm, dm;
    RowStat mine{INFINITY, 0.0f};
    int end = 0;
    auto load = [&](int64_t rt) {
        // rows that see nothing are zeros: what stands there takes no part
        auto place = [&](int r, const T *p, const Strided &s) -> const T * {
            const int64_t row = rt * RT + r, t = row / a.G;
            return row < a.R && a.seen(len, start, t) > 0 ? p + t * s.t + row % a.G * s.h : nullptr;
        };
        qm.load(tid, a.D, [&](int r) { return place(r, qp, a.q); });
        dm.load(tid, a.D, [&](int r) { return place(r, dp, a.d_o); });
        if (tid < RT) {
            const int64_t row = rt * RT + tid;
            mine = row < a.R ? stat[nh * a.R + row] : RowStat{INFINITY, 0.0f};
            // how many of the keys from the block's first on the row sees
            end = row < a.R ? int(max(int64_t(0), min(a.seen(len, start, row / a.G) - block_key, int64_t(WAVES * KB * 32)))) : 0;
        }
    };
    auto store = [&]() {
        qm.store(lds[0], tid);
        dm.store(lds[1], tid);
        if (tid < RT) {
            lse2[tid] = mine.lse2 - bias;
            delta[tid] = mine.delta * factor;
            ends[tid] = end;
        }
    };

    if (rt0 < rt1) load(rt0);
    for (int64_t rt = rt0; rt < rt1; ++rt) {
        __syncthreads();
        store();
        __syncthreads();
        if (rt + 1 < rt1) load(rt + 1);
        const T *ql = lds[0], *dl = lds[1];
        // the tile's first row sees fewest keys, and its last row exists or there are rows to hide
        const bool whole = key0 + KB * 32 <= a.seen(len, start, rt * RT / a.G);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            f32x16 s[KB], g[KB];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) s[kb] = g[kb] = f32x16{};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const Frag<T> qf = L::by_rows(ql, rb * 32 + (lane & 31), ks, half);
                const Frag<T> df = L::by_rows(dl, rb * 32 + (lane & 31), ks, half);
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    s[kb] = mma(qf, k[kb][ks], s[kb]);
                    g[kb] = mma(df, v[kb][ks], g[kb]);
                }
            }
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) {
                const int at = rb * 32 + 8 * r4 + 4 * half;
                const f32x4 le = *reinterpret_cast<const f32x4 *>(lse2 + at), de = *reinterpret_cast<const f32x4 *>(delta + at);
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = 4 * r4 + j;
                        const float p = exp2_fast(fmaf(s[kb][r], c, -le[j]));
                        s[kb][r] = p;
                        g[kb][r] = p * fmaf(g[kb][r], factor, -de[j]);
                    }
                if (!whole) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int e = ends[at + j] - wave * (KB * 32) - (lane & 31);
#pragma unroll
                        for (int kb = 0; kb < KB; ++kb) {
                            s[kb][4 * r4 + j] = kb * 32 < e ? s[kb][4 * r4 + j] : 0.0f;
                            g[kb][4 * r4 + j] = kb * 32 < e ? g[kb][4 * r4 + j] : 0.0f;
                        }
                    }
                }
            }
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                Frag<T> pf[KB], gf[KB];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    pf[kb] = operand<T>(s[kb], st);
                    gf[kb] = operand<T>(g[kb], st);
                }
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    const Frag<T> df = L::by_columns(dl, rb * 32 + st * 16, db, lane);
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) dv[kb][db] = mma(df, pf[kb], dv[kb][db]);
                    const Frag<T> qf = L::by_columns(ql, rb * 32 + st * 16, db, lane);
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) dk[kb][db] = mma(qf, gf[kb], dk[kb][db]);
                }
            }
        }
    }
    const float undo_k = exp2f(-float(shift)), undo_v = exp2f(-bias);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        const int64_t key = key0 + kb * 32 + (lane & 31);
        if (key >= a.Tk) continue;
        if (a.splits == 1) {
            const int64_t at = ((n * a.Tk + key) * a.Hkv + hk) * a.D;
            store_columns<T, DB>(static_cast<T *>(a.dk) + at, dk[kb], undo_k, a.D, half);
            store_columns<T, DB>(static_cast<T *>(a.dv) + at, dv[kb], undo_v, a.D, half);
        } else {
            const int64_t all = a.N * a.Tk * a.Hkv * a.D, at = ((n * a.Tk + key) * a.Hkv + hk) * a.D;
            float *part = a.part + int64_t(split) * 2 * all + at;
            store_columns<float, DB>(part, dk[kb], undo_k, a.D, half);
            store_columns<float, DB>(part + all, dv[kb], undo_v, a.D, half);
        }
    }
}

// dq of a block of rows, from the keys of this split.
template <class T, int DP, int QB, int WAVES, int KT>
__global__ __launch_bounds__(WAVES * 64) void row_grad_kernel(Attention a, const RowStat *stat, const float *top,
                                                              int64_t row_blocks, int64_t blocks, int64_t tiles)
{
    using L = Tile<T, DP>;
    constexpr int KS = DP / 16, DB = DP / 32, KB = KT / 32, THREADS = WAVES * 64;
    __shared__ __attribute__((aligned(16))) T lds[2][KT * DP];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, half = lane >> 5;

    int64_t w = xcd_remap(blockIdx.x, gridDim.x);
    const int split = int(w % a.splits);
    w /= a.splits;
    const int64_t tile = tiles - 1 - w % tiles, nh = w / tiles, n = nh / a.Hkv, hk = nh % a.Hkv;
    const int64_t len = a.length(n), start = a.start(n);
    const int64_t row0 = tile * (WAVES * QB * 32) + wave * (QB * 32);

    const int shift = grad_shift<T, THREADS>(a, top, nh, row_blocks, blocks);
    const float bias = kHalf<T> ? float(kHalfBias) : 0.0f, c = a.scale * kLog2e;
    const float factor = a.scale * exp2f(float(shift) - bias);

    Frag<T> q[QB][KS], d_o[QB][KS];
    int64_t seen[QB];
    float lse2[QB], delta[QB];
#pragma unroll
    for (int qb = 0; qb < QB; ++qb) {
        const int64_t row = row0 + qb * 32 + (lane & 31), t = row / a.G, h = hk * a.G + row % a.G;
        seen[qb] = row < a.R ? a.seen(len, start, t) : 0;
        const RowStat st = row < a.R ? stat[nh * a.R + row] : RowStat{INFINITY, 0.0f};
        lse2[qb] = st.lse2 - bias;
        delta[qb] = st.delta * factor;
        const T *qp = static_cast<const T *>(a.q.p) + n * a.q.n + t * a.q.t + h * a.q.h;
        const T *dp = static_cast<const T *>(a.d_o.p) + n * a.d_o.n + t * a.d_o.t + h * a.d_o.h;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            q[qb][ks] = load_frag<T>(qp, ks * 16 + half * 8, seen[qb] > 0 ? a.D : 0);
            d_o[qb][ks] = load_frag<T>(dp, ks * 16 + half * 8, seen[qb] > 0 ? a.D : 0);
        }
    }
    const int64_t last = min(tile * (WAVES * QB * 32) + WAVES * QB * 32, a.R) - 1;
    const int64_t want = (a.seen(len, start, last / a.G) + KT - 1) / KT, each = (want + a.splits - 1) / a.splits;
    const int64_t kt0 = split * each, kt1 = min(want, kt0 + each);
    const int64_t first_seen = row0 < a.R ? a.seen(len, start, row0 / a.G) : 0;
    const int64_t last_seen = row0 < a.R ? a.seen(len, start, (min(row0 + QB * 32, a.R) - 1) / a.G) : 0;
    const int64_t whole = first_seen / KT, none = (last_seen + KT - 1) / KT;

    const T *kp = static_cast<const T *>(a.k.p) + n * a.k.n + hk * a.k.h;
    const T *vp = static_cast<const T *>(a.v.p) + n * a.v.n + hk * a.v.h;
    Mover<T, DP, KT, THREADS> km, vm;
    auto load = [&](int64_t kt) {
        km.load(tid, a.D, [&](int r) { return kt * KT + r < len ? kp + (kt * KT + r) * a.k.t : nullptr; });
        vm.load(tid, a.D, [&](int r) { return kt * KT + r < len ? vp + (kt * KT + r) * a.v.t : nullptr; });
    };
    f32x16 dq[QB][DB];
#pragma unroll
    for (int qb = 0; qb < QB; ++qb)
#pragma unroll
        for (int db = 0; db < DB; ++db) dq[qb][db] = f32x16{};

    if (kt0 < kt1) load(kt0);
    for (int64_t kt = kt0; kt < kt1; ++kt) {
        __syncthreads();
        km.store(lds[0], tid);
        vm.store(lds[1], tid);
        __syncthreads();
        if (kt + 1 < kt1) load(kt + 1);
        if (kt >= none) continue;
        const T *kl = lds[0], *vl = lds[1];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            f32x16 s[QB], g[QB];
#pragma unroll
            for (int qb = 0; qb < QB; ++qb) s[qb] = g[qb] = f32x16{};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const Frag<T> kf = L::by_rows(kl, kb * 32 + (lane & 31), ks, half);
                const Frag<T> vf = L::by_rows(vl, kb * 32 + (lane & 31), ks, half);
#pragma unroll
                for (int qb = 0; qb < QB; ++qb) {
                    s[qb] = mma(kf, q[qb][ks], s[qb]);
                    g[qb] = mma(vf, d_o[qb][ks], g[qb]);
                }
            }
#pragma unroll
            for (int qb = 0; qb < QB; ++qb) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float p = exp2_fast(fmaf(s[qb][r], c, -lse2[qb]));
                    g[qb][r] = p * fmaf(g[qb][r], factor, -delta[qb]);
                }
                if (kt >= whole) {
                    const int end = int(max(int64_t(0), min(seen[qb] - kt * KT, int64_t(KT))));
#pragma unroll
                    for (int r = 0; r < 16; ++r) g[qb][r] = kb * 32 + c_row(r, half) < end ? g[qb][r] : 0.0f;
                }
            }
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                Frag<T> gf[QB];
#pragma unroll
                for (int qb = 0; qb < QB; ++qb) gf[qb] = operand<T>(g[qb], st);
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    const Frag<T> kf = L::by_columns(kl, kb * 32 + st * 16, db, lane);
#pragma unroll
                    for (int qb = 0; qb < QB; ++qb) dq[qb][db] = mma(kf, gf[qb], dq[qb][db]);
                }
            }
        }
    }
    const float undo = exp2f(-float(shift));
#pragma unroll
    for (int qb = 0; qb < QB; ++qb) {
        const int64_t row = row0 + qb * 32 + (lane & 31), t = row / a.G, h = hk * a.G + row % a.G;
        if (row >= a.R) continue;
        const int64_t at = ((n * a.Tq + t) * a.H + h) * a.D;
        if (a.splits == 1) store_columns<T, DB>(static_cast<T *>(a.dq) + at, dq[qb], undo, a.D, half);
        else store_columns<float, DB>(a.part + int64_t(split) * a.N * a.Tq * a.H * a.D + at, dq[qb], undo, a.D, half);
    }
}

// Sums of `splits` partial results of `count` values each, in their order; the first `first` of
// them go to y0, the others to y1.
template <class T>
__global__ __launch_bounds__(256) void grad_join_kernel(const float *part, int splits, int64_t count, int64_t first, T *y0, T *y1)
{
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < count; i += int64_t(gridDim.x) * 256) {
        float sum = 0.0f;
        for (int s = 0; s < splits; ++s) sum += part[s * count + i];
        (i < first ? y0[i] : y1[i - first]) = T(sum);
    }
}

template <class T>
void launch_attend_grad(Attention a, const AttendGradPlan &p, char *ws, hipStream_t st)
{
    RowStat *stat = reinterpret_cast<RowStat *>(ws + p.stat);
    float *top = reinterpret_cast<float *>(ws + p.top);
    const int64_t row_blocks = (a.R + kStatRows - 1) / kStatRows;
    const int64_t blocks = row_blocks + (kHalf<T> ? (a.Tk + kStatRows - 1) / kStatRows : 0);
    const int64_t heads = a.N * a.Hkv;
    if (a.R > 0 && heads * blocks > 0) stat_kernel<T><<<unsigned(heads * blocks), 256, 0, st>>>(a, stat, top, row_blocks, blocks);
    a.part = reinterpret_cast<float *>(ws + p.part);
    auto join = [&](int splits, int64_t count, int64_t first, void *y0, void *y1) {
        const int64_t want = (count + 255) / 256;
        grad_join_kernel<T><<<unsigned(want < 4096 ? want : 4096), 256, 0, st>>>(a.part, splits, count, first, static_cast<T *>(y0),
                                                                                 static_cast<T *>(y1));
    };
    with_head(a.D, [&](auto head) {
        constexpr int DP = decltype(head)::value;
        constexpr int TILE = DP * sizeof(T) > 512 ? 32 : 64;
        constexpr int BLOCK = 128;
        const int64_t key_tiles = (a.Tk + BLOCK - 1) / BLOCK, row_tiles = (a.R + BLOCK - 1) / BLOCK;
        if (key_tiles > 0) {
            a.splits = p.row_splits;
            key_grad_kernel<T, DP, 1, 4, TILE><<<unsigned(heads * key_tiles * a.splits), 256, 0, st>>>(a, stat, top, row_blocks, blocks, key_tiles);
            const int64_t count = a.N * a.Tk * a.Hkv * a.D;
            if (a.splits > 1) join(a.splits, 2 * count, count, a.dk, a.dv);
        }
        if (row_tiles > 0) {
            a.splits = p.key_splits;
            row_grad_kernel<T, DP, 1, 4, TILE><<<unsigned(heads * row_tiles * a.splits), 256, 0, st>>>(a, stat, top, row_blocks, blocks, row_tiles);
            const int64_t count = a.N * a.R * a.Hkv * a.D;
            if (a.splits > 1) join(a.splits, count, count, a.dq, a.dq);
        }
    });
}

}  // namespace ct

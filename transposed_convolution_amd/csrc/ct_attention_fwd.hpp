// ct_attention_fwd.hpp -- attention in one pass over the keys:
//
//   s_ij = scale q_i . k_j,  lse_i = log sum_j exp s_ij,  o_i = sum_j exp(s_ij - lse_i) v_j
//
// over the keys j that row i sees.  Keys and values go through LDS; a running reference m
// (near the largest score so far) keeps the exponentials in range, and the sum l and the output o
// are scaled when it moves.  Scores, sums and outputs stay in float32 registers; the weights are
// rounded once to the values' type for the second product.
#pragma once

#include "ct_attention.hpp"

namespace ct {

// The reference only moves when a score exceeds it by more than 2^kSlack, so most tiles scale
// nothing; weights are up to 2^(kSlack + bias).
constexpr float kSlack = 8.0f;
// float16 weights are held 2^7 times larger, so that small ones keep their digits (the largest is 2^15).
template <class T>
constexpr float kWeightBias = std::is_same_v<T, _Float16> ? 7.0f : 0.0f;

// References from here on (in powers of two) are those of scores whose product with c is rounded by itself.  One fused
// step, s c - m, keeps what the reference's own rounding left out, half a unit: 2^-5 here, which does no harm, but
// from 2^24 on it takes float16 weights beyond their range and from 2^31 on any: the largest score's is not 1 then
// but infinite or nothing.
constexpr float kFar = 0x1p20f;

// The softmax of a row so far: reference m (in powers of two, the bias taken off where it is not far), sum l of 2^(s c - m), this
// lane's half of it.
struct Running {
    float m = -INFINITY, l = 0.0f;
    // Moves the reference for a tile's scores, and scales the output where it does.
    template <class T, int KB, int DB>
    __device__ __forceinline__ void look(const f32x16 (&s)[KB], f32x16 (&o)[DB], float c)
    {
        float top = s[0][0];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[kb][r]);
        top = half_max(top) * c;
        const bool moves = top - m > kSlack + kWeightBias<T>;  // exact where they are near each other
        if (__any(moves)) {
            const float to = moves ? fabsf(top) < kFar ? top - kWeightBias<T> : top : m;
            const float f = moves ? exp2_fast(m - to) : 1.0f;
            m = to;
            l *= f;
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[db][r] *= f;
        }
    }
    // Scores times c, rounded: the product of the largest is the reference itself.
    template <int KB>
    __device__ __forceinline__ static void far(f32x16 (&s)[KB], float c)
    {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[kb][r] *= c;
    }
    // Scores become weights.
    template <class T, int KB>
    __device__ __forceinline__ void weigh(f32x16 (&s)[KB], float c)
    {
        const float base = m == -INFINITY ? 0.0f : m;
        float by = c;
        if (__builtin_expect(__any(fabsf(base) >= kFar), 0)) {
            far(s, c);
            by = 1.0f;
        }
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float e = exp2_fast(fmaf(s[kb][r], by, -base));
                s[kb][r] = e;
                sum[r & 1] += e;
            }
        l += sum[0] + sum[1];
    }
};

// Scores of keys at or behind `end` (of the tile's) become -inf.
template <int KB>
__device__ __forceinline__ void hide(f32x16 (&s)[KB], int end, int half)
{
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[kb][r] = kb * 32 + c_row(r, half) < end ? s[kb][r] : -INFINITY;
}

// Where a row's parts lie in the workspace: (m, l) of every split and row, then the outputs.
struct Parts {
    float *stat, *out;
    int64_t rows;
    int D;
    __device__ __forceinline__ Parts(float *p, const Attention &a, int splits)
        : stat(p), out(p + 2 * int64_t(splits) * a.N * a.Hkv * a.R), rows(int64_t(a.N) * a.Hkv * a.R), D(a.D)
    {
    }
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// The result of a row: stored, or left as a part.
template <class T, int DB>
__device__ __forceinline__ void finish(const Attention &a, float *part, int splits, int split, int nh, int n, int hk, int row,
                                       int half, float m, float l, const f32x16 (&o)[DB])
{
    const int t = a.by_g.div(row), h = hk * a.G + row - t * a.G;
    if (splits == 1) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        store_columns<T, DB>(static_cast<T *>(a.out) + ((int64_t(n) * a.Tq + t) * a.H + h) * a.D, o, inv, a.D, half);
        if (half == 0) a.lse[(int64_t(n) * a.H + h) * a.Tq + t] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * kLn2;
    } else {
        const Parts ps(part, a, splits);
        const int64_t at = split * ps.rows + int64_t(nh) * a.R + row;
        if (half == 0) {
            ps.stat[2 * at] = l == 0.0f ? -INFINITY : m;
            ps.stat[2 * at + 1] = l;
        }
        store_columns<float, DB>(ps.out + at * a.D, o, 1.0f, a.D, half);
    }
}

// A weight of 0 times a value that is not finite is NaN, so in a causal call such a value would reach rows that do not
// see it.  The tiles that some rows see in part (two or three a block) therefore have zeros in such places, and what
// stood there is added at the end to the rows that see it: a weight leaves neither an infinity nor a NaN
// otherwise.  In tiles that every row sees it takes part as it is.
//
// This happens only where such a value was found: a lane looks at one of 64 keys, then those that have any are taken
// from memory, several at a time where heads are short.  `end`: how many of the keys the lane's row sees.  2048 causal
// tokens, 4 heads of 64, float16: 35 us, as many with a NaN that all rows see, 100 with nothing but infinities.
template <class T, int DB>
__device__ __forceinline__ void add_not_finite(f32x16 (&o)[DB], const T *v, int64_t stride, int keys, int end, int D, int lane)
{
    constexpr int K = DB == 1 ? 8 : DB == 2 ? 4 : DB <= 4 ? 2 : 1;
    const int half = lane >> 5;
    for (int j0 = 0; j0 < keys; j0 += 64) {
        bool odd = false;
        if (j0 + lane < keys)
            for (int d = 0; d < D; d += kVec<T>) {
                const Raw<T, kVec<T>> r = load_chunk<T>(v + (j0 + lane) * stride + d, D - d, D % kVec<T>);
#pragma unroll
                for (int i = 0; i < kVec<T>; ++i) odd |= !finite(float(r[i]));
            }
        for (uint64_t left = __ballot(odd); left;) {
            const int first = __builtin_ctzll(left) / K * K, j = j0 + first;
            left &= ~(((uint64_t(1) << K) - 1) << first);
#pragma unroll
            for (int db = 0; db < DB; ++db) {
                Raw<T, 4> x[K][4];
#pragma unroll
                for (int key = 0; key < K; ++key)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // every lane loads, whatever its row sees: no load is in a branch of its own
                        const int d = db * 32 + 8 * k + 4 * half;
                        const T *p = v + min(j + key, keys - 1) * stride + d;
                        x[key][k] = Raw<T, 4>{};
                        if (D == DB * 32 || d + 4 <= D) {
                            x[key][k] = *reinterpret_cast<const Raw<T, 4> *>(p);
                        } else {
#pragma unroll
                            for (int i = 0; i < 3; ++i)
                                if (d + i < D) x[key][k][i] = p[i];
                        }
                    }
#pragma unroll
                for (int key = 0; key < K; ++key)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const Raw<T, 4> seen = j + key < end ? x[key][k] : Raw<T, 4>{};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float f = float(seen[i]);
                            o[db][4 * k + i] += finite(f) ? 0.0f : f;
                        }
                    }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
}

// A wave holds 32 rows, a block goes through the keys KT at a time; the next tile is on its way while one
// is worked on.  8 x 4096 tokens, 8 heads of 64, float16: 400 to 433 us by card, 635 to 690 TFLOP/s; 2 x 8191 causal
// tokens, 16 heads over 4 of 128, bfloat16: 656 to 695 us; heads of 256, 2 x 4096 tokens, 4 heads, float16: 350 us, 390 (one
// wave a SIMD).  Bound by the vector unit beside the matrix unit: a score takes 6 vector instructions, one of them the
// exponential at a half of their rate, so that 32 x 32 scores take 500 cycles of them and, with heads of 64, 256 of matrix
// instructions; the two are busy 60 and 30 % of the time (heads of 128: 44 and 34 %), the rest is steps that wait for
// the one before.
// Other cuts, us for the first and the second call (438 and 695 then): 64 rows a wave 408 and 1112, 32 keys a tile 452 and
// 835, 128 keys 427 and 1144, 8 waves a block 500 and 738, three buffers 469 and 1140.  Three waves a SIMD
// (168 registers) took heads of 64 from 521 to 441.  Heads of 32 have four (128 registers): 4 x 4096 tokens, 8 heads, float16, 131 us, 155
// with three; causal bfloat16 122, 96 with three.
template <class T, int DP, int WAVES, int KT>
__global__ __launch_bounds__(WAVES * 64, DP * sizeof(T) <= 64 ? 4 : DP * sizeof(T) <= 128 ? 3 : DP * sizeof(T) <= 256 ? 2 : 1) void attend_kernel(
    Attention a, float *part, int tiles, int splits, int chunk)
{
    using L = Tile<T, DP>;
    constexpr int KS = DP / 16, DB = DP / 32, KB = KT / 32, THREADS = WAVES * 64, ROWS = WAVES * 32;
    // Operands asked for ahead: heads of 128 took 727 us without, 699, 692, 687 and 690 with 2, 3, 4 and 6.
    constexpr int P = 4;
    __shared__ __attribute__((aligned(16))) T lds[2][2][KT * DP];
    __shared__ int odd[WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = lane >> 5;

    // an XCD takes a contiguous run of blocks: those of one image and key head share its L2
    int w = xcd_remap(blockIdx.x, gridDim.x);
    const int split = w % splits;
    w /= splits;
    const int nh = w / tiles, tile = long_first(w - nh * tiles, tiles, a.N * a.Hkv), n = nh / a.Hkv, hk = nh % a.Hkv;
    const int start = a.start(n), len = a.length(n, start);
    const int block_row = tile * ROWS, row0 = block_row + wave * 32;

    const int row = row0 + (lane & 31), t = a.by_g.div(row);
    const bool there = row < a.R;
    const int seen = there ? a.seen(len, start, t) : 0;
    Frag<T> q[KS];
    const T *qp = static_cast<const T *>(a.q.p) + n * a.q.n + t * a.q.t + (hk * a.G + row - t * a.G) * a.q.h;
    // a row that sees nothing is not read: without keys there may be no q
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q[ks] = load_frag<T>(qp, ks * 16 + half * 8, seen > 0 ? a.D : 0);
    // keys the block looks at, of this split's chunk
    const int want = min(a.seen(len, start, a.by_g.div(min(block_row + ROWS, a.R) - 1)), split * chunk + chunk);
    if (split > 0 && split * chunk >= want) return;  // the join passes over it
    const int kt0 = split * chunk / KT, kt1 = (want + KT - 1) / KT;
    // of this wave's rows: tiles before `whole` are seen by every row, tiles from `none` on by none
    const bool rows = row0 < a.R;
    const int whole = rows ? a.seen(len, start, a.by_g.div(row0)) / KT : 0;
    const int none = rows ? (a.seen(len, start, a.by_g.div(min(row0 + 32, a.R) - 1)) + KT - 1) / KT : 0;
    // tiles from here on some rows of the block see in part, but for those behind the length
    const int mixed = a.causal ? a.seen(len, start, a.by_g.div(block_row)) / KT : kt1;

    const T *kp = static_cast<const T *>(a.k.p) + n * a.k.n + hk * a.k.h;
    const T *vp = static_cast<const T *>(a.v.p) + n * a.v.n + hk * a.v.h;
    Mover<T, DP, KT, THREADS> km(tid), vm(tid);
    // keys behind the length are zeros: what stands there takes no part
    auto load = [&](int kt) {
        km.load(kp + int64_t(kt) * KT * a.k.t, a.k.t, len - kt * KT, a.D);
        vm.load(vp + int64_t(kt) * KT * a.v.t, a.v.t, len - kt * KT, a.D);
    };
    int found = 0;  // did this wave bring values that are not finite in such tiles
    auto store = [&](int buf, int kt) {
        if (kt >= mixed) {
            found |= vm.drop_not_finite();
            if (lane == 0) odd[wave] = found;
        }
        km.store(lds[buf][0]);
        vm.store(lds[buf][1]);
    };

    f32x16 o[DB];
    Running run;
#pragma unroll
    for (int db = 0; db < DB; ++db) o[db] = f32x16{};
    const float c = a.scale * kLog2e;
    if (kt0 < kt1) {
        load(kt0);
        store(0, kt0);
    }
    for (int kt = kt0; kt < kt1; ++kt) {
        __syncthreads();
        const int buf = (kt - kt0) & 1;
        if (kt + 1 < kt1) load(kt + 1);
        if (kt < none) {
            const T *kl = lds[buf][0], *vl = lds[buf][1];
            f32x16 s[KB];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) s[kb] = f32x16{};
            Ahead<T, KB * KS, P> keys;
            auto key = [&](int i) { return L::by_rows(kl, i / KS * 32 + (lane & 31), i % KS, half); };
            keys.prime(key);
            keys.run(key, [&](int i, const Frag<T> &f) { s[i / KS] = mma(f, q[i % KS], s[i / KS]); });
            Ahead<T, KT / 16 * DB, P> values;
            auto value = [&](int i) { return L::by_columns(vl, i / DB * 16, i % DB, lane); };
            values.prime(value);
            if (kt >= whole) hide(s, seen - kt * KT, half);
            run.template look<T>(s, o, c);
            run.template weigh<T>(s, c);
            Frag<T> p;
            values.run(value, [&](int i, const Frag<T> &f) {
                if (i % DB == 0) p = operand<T>(s[i / DB / 2], i / DB % 2);
                o[i % DB] = mma(f, p, o[i % DB]);
            });
        }
        if (kt + 1 < kt1) store(buf ^ 1, kt + 1);
    }
    const int odd0 = max(mixed, kt0);
    if (odd0 < kt1) {
#pragma unroll
        for (int i = 0; i < WAVES; ++i) found |= odd[i];  // complete since the last tile's barrier
        if (__builtin_expect(__builtin_amdgcn_readfirstlane(found), 0))
            add_not_finite<T, DB>(o, vp + int64_t(odd0) * KT * a.v.t, a.v.t, min(kt1 * KT, len) - odd0 * KT, seen - odd0 * KT, a.D, lane);
    }
    const float l = half_sum(run.l);
    if (there) finish<T, DB>(a, part, splits, split, nh, n, hk, row, half, run.m, l, o);
}

// Memory accesses of a wave's lanes on both sides stay there: what one lane stored before, another reads after.
__device__ __forceinline__ void in_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Up to 32 rows a key head (a token or a few over a cache): every wave takes 32 keys of its own at a
// time, through LDS of its own, and the block's waves are joined at the end.  Nothing waits for another wave
// on the way.  One token, 4 images of up to 32768 keys, 16 heads over 4 of 128, bfloat16: 45 us with the join,
// 2.9 TB/s of the keys and values that are seen.  Bound by latency in short calls: 8 images of up to 4096 keys,
// 8 heads over 2 of 64, take 7.4 us for the chain length, keys, scores, values, join of waves, and 4 for the join of splits.
template <class T, int DP, int WAVES>
__global__ __launch_bounds__(WAVES * 64, DP * sizeof(T) <= 256 ? 2 : 1) void attend_few_kernel(Attention a, float *part, int splits, int chunk)
{
    using L = Tile<T, DP>;
    constexpr int KS = DP / 16, DB = DP / 32;
    // the waves' tiles of keys and values, and then their outputs: 32 rows of DP float32
    __shared__ __attribute__((aligned(16))) char lds[WAVES * 32 * DP * 2 * sizeof(T)];
    __shared__ float ms[WAVES][32], ls[WAVES][32];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = lane >> 5;
    T *kl = reinterpret_cast<T *>(lds) + wave * 64 * DP, *vl = kl + 32 * DP;

    int w = xcd_remap(blockIdx.x, gridDim.x);
    const int split = w % splits, nh = w / splits, n = nh / a.Hkv, hk = nh % a.Hkv;
    const int start = a.start(n), len = a.length(n, start);
    const int row = lane & 31, t = a.by_g.div(row), g = row - t * a.G;
    const bool there = row < a.R;
    const int seen = there ? a.seen(len, start, t) : 0;

    // tiles of 32 keys of this split's chunk, dealt to the block's waves in turn
    const int want = min(a.seen(len, start, a.Tq - 1), split * chunk + chunk);
    if (split > 0 && split * chunk >= want) return;  // the join passes over it
    const int kt0 = split * chunk / 32 + wave, kt1 = (want + 31) / 32;
    const int whole = a.seen(len, start, 0) / 32, mixed = a.causal ? whole : kt1;
    const T *kp = static_cast<const T *>(a.k.p) + n * a.k.n + hk * a.k.h;
    const T *vp = static_cast<const T *>(a.v.p) + n * a.v.n + hk * a.v.h;

    Frag<T> q[KS];
    // one tile on its way at a time: the values while the scores are made, the next keys while the values
    // are added, in the same registers
    Mover<T, DP, 32, 64> mv(lane);
    if (kt0 < kt1) mv.load(kp + int64_t(kt0) * 32 * a.k.t, a.k.t, len - kt0 * 32, a.D);
    const T *qp = static_cast<const T *>(a.q.p) + n * a.q.n + t * a.q.t + (hk * a.G + g) * a.q.h;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q[ks] = load_frag<T>(qp, ks * 16 + half * 8, seen > 0 ? a.D : 0);

    f32x16 o[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db) o[db] = f32x16{};
    Running run;
    const float c = a.scale * kLog2e;
    bool odd = false;
    for (int kt = kt0; kt < kt1; kt += WAVES) {
        // The tiles are the wave's own, whose LDS accesses are done in order; in_order keeps the compiler from changing
        // it, here and for the next tiles' stores: each tile's reads lie before the other's.
        mv.store(kl);
        mv.load(vp + int64_t(kt) * 32 * a.v.t, a.v.t, len - kt * 32, a.D);
        in_order();
        f32x16 s[1] = {f32x16{}};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) s[0] = mma(L::by_rows(kl, lane & 31, ks, half), q[ks], s[0]);
        if (kt >= whole) hide(s, seen - kt * 32, half);
        run.template look<T>(s, o, c);
        run.weigh<T>(s, c);
        if (kt >= mixed) odd |= mv.drop_not_finite();
        mv.store(vl);
        const int next = kt + WAVES;
        if (next < kt1) mv.load(kp + int64_t(next) * 32 * a.k.t, a.k.t, len - next * 32, a.D);
        in_order();
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const Frag<T> p = operand<T>(s[0], st);
#pragma unroll
            for (int db = 0; db < DB; ++db) o[db] = mma(L::by_columns(vl, st * 16, db, lane), p, o[db]);
        }
    }
    if (odd)
        for (int kt = kt0; kt < kt1; kt += WAVES)
            if (kt >= mixed) add_not_finite<T, DB>(o, vp + int64_t(kt) * 32 * a.v.t, a.v.t, min(32, len - kt * 32), seen - kt * 32, a.D, lane);
    float l = half_sum(run.l), m = run.m;
    if constexpr (WAVES > 1) {
        if (half == 0) {
            ms[wave][row] = m;
            ls[wave][row] = l;
        }
        __syncthreads();  // the tiles are done with
        float *ol = reinterpret_cast<float *>(lds) + wave * 32 * DP;
        if (wave > 0 && there)
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x4 v = {o[db][4 * k], o[db][4 * k + 1], o[db][4 * k + 2], o[db][4 * k + 3]};
                    // chunks turned by the row, so that rows do not meet in the banks
                    *reinterpret_cast<f32x4 *>(ol + row * DP + (((db * 8 + 2 * k + half) ^ (row & 7)) * 4)) = v;
                }
        __syncthreads();
        if (wave > 0) return;
        float top = m;
#pragma unroll
        for (int i = 1; i < WAVES; ++i) top = fmaxf(top, ms[i][row]);
        const float f0 = m == -INFINITY ? 0.0f : exp2_fast(m - top);
        l *= f0;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[db][r] *= f0;
        if (there)
#pragma unroll
            for (int i = 1; i < WAVES; ++i) {
                const float mi = ms[i][row], f = mi == -INFINITY ? 0.0f : exp2_fast(mi - top);
                l = fmaf(ls[i][row], f, l);
                const float *oi = reinterpret_cast<const float *>(lds) + i * 32 * DP;
#pragma unroll
                for (int db = 0; db < DB; ++db)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const f32x4 v = *reinterpret_cast<const f32x4 *>(oi + row * DP + (((db * 8 + 2 * k + half) ^ (row & 7)) * 4));
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[db][4 * k + j] = fmaf(v[j], f, o[db][4 * k + j]);
                    }
            }
        m = top;
    }
    if (there) finish<T, DB>(a, part, splits, split, nh, n, hk, row, half, m, l, o);
}

// The splits of a row, a block a row: weights 2^(m - largest m).  A lane reads the statistics of one split; the
// waves (one for a few splits, four for many) take the parts in turn, 8 asked for at a time.  Chunks that a block of
// `span` rows had nothing of are passed over.  A launch and two dependent reads: 4 us for 64 rows of 32 parts, 5 for 1155
// rows of 9.
template <class T, int C, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void attend_join_kernel(Attention a, float *part, int splits, int chunk, int span)
{
    const Parts ps(part, a, splits);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t id = blockIdx.x;
    const int nh = int(id / a.R), row = int(id - int64_t(nh) * a.R), n = nh / a.Hkv, t = a.by_g.div(row);
    const int h = (nh - n * a.Hkv) * a.G + row - t * a.G;
    const int start = a.start(n), want = a.seen(a.length(n, start), start, a.by_g.div(min(row / span * span + span, a.R) - 1));
    const int count = max(1, (want + chunk - 1) / chunk);  // the first split always leaves its part
    // a plan has at most 64 splits: one a lane
    const bool mine = lane < count;
    const float m = mine ? ps.stat[2 * (lane * ps.rows + id)] : -INFINITY, l = mine ? ps.stat[2 * (lane * ps.rows + id) + 1] : 0.0f;
    constexpr int AT_ONCE = 8;
    float acc[C] = {};
    for (int s0 = wave; s0 < count; s0 += WAVES * AT_ONCE) {
        float v[AT_ONCE][C];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int s = s0 + WAVES * k, d = i * 64 + lane;
                v[k][i] = s < count && d < a.D ? ps.out[(s * ps.rows + id) * a.D + d] : 0.0f;
            }
        float top = m;
#pragma unroll
        for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
        const float f = l == 0.0f ? 0.0f : exp2_fast(m - top);  // nothing seen there: nothing to add
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const float wt = __shfl(f, (s0 + WAVES * k) & 63);
#pragma unroll
            for (int i = 0; i < C; ++i) acc[i] = fmaf(v[k][i], wt, acc[i]);
        }
    }
    if constexpr (WAVES > 1) {
        __shared__ float shared[WAVES - 1][C][64];
        if (wave > 0) {
#pragma unroll
            for (int i = 0; i < C; ++i) shared[wave - 1][i][lane] = acc[i];
        }
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int x = 0; x < WAVES - 1; ++x)
#pragma unroll
            for (int i = 0; i < C; ++i) acc[i] += shared[x][i][lane];
    }
    float top = m;
#pragma unroll
    for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    float sum = l == 0.0f ? 0.0f : l * exp2_fast(m - top);
#pragma unroll
    for (int x = 32; x; x >>= 1) sum += __shfl_xor(sum, x);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    T *out = static_cast<T *>(a.out) + ((int64_t(n) * a.Tq + t) * a.H + h) * a.D;
#pragma unroll
    for (int i = 0; i < C; ++i)
        if (i * 64 + lane < a.D) out[i * 64 + lane] = T(acc[i] * inv);
    if (lane == 0) a.lse[(int64_t(n) * a.H + h) * a.Tq + t] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * kLn2;
}

template <class T>
void launch_attend(const Attention &a, const AttendPlan &p, float *part, hipStream_t st)
{
    const int heads = a.N * a.Hkv;
    with_head(a.D, [&](auto head) {
        constexpr int DP = decltype(head)::value, KT = DP * sizeof(T) > 256 ? 32 : 64, C = (DP + 63) / 64;
        constexpr int FW = DP * sizeof(T) > 512 ? 2 : 4;  // their tiles fit LDS
        const int span = p.few ? 32 : 128;
        if (p.few) attend_few_kernel<T, DP, FW><<<unsigned(heads * p.splits), FW * 64, 0, st>>>(a, part, p.splits, p.chunk);
        else attend_kernel<T, DP, 4, KT><<<unsigned(heads * p.tiles * p.splits), 256, 0, st>>>(a, part, p.tiles, p.splits, p.chunk);
        if (p.splits > 16) attend_join_kernel<T, C, 4><<<unsigned(heads * a.R), 256, 0, st>>>(a, part, p.splits, p.chunk, span);
        else if (p.splits > 1) attend_join_kernel<T, C, 1><<<unsigned(heads * a.R), 64, 0, st>>>(a, part, p.splits, p.chunk, span);
    });
}

}  // namespace ct

// ct_attention_fwd.hpp -- attention in one pass over the keys:
//
//   s_ij = scale q_i . k_j,  lse_i = log sum_j exp s_ij,  o_i = sum_j exp(s_ij - lse_i) v_j
//
// over the keys j that row i sees.  Tiles of keys and values go through LDS; a running reference m
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

template <class T, int DP, int QB, int WAVES, int KT>
__global__ __launch_bounds__(WAVES * 64) void attend_kernel(Attention a, int64_t tiles)
{
    using L = Tile<T, DP>;
    constexpr int KS = DP / 16, DB = DP / 32, KB = KT / 32, THREADS = WAVES * 64;
    __shared__ __attribute__((aligned(16))) T lds[2][2][KT * DP];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, half = lane >> 5;

    // an XCD takes a contiguous run of blocks: those of one image and key head share its L2; a
    // causal call's long tiles go first
    int64_t w = xcd_remap(blockIdx.x, gridDim.x);
    const int split = int(w % a.splits);
    w /= a.splits;
    const int64_t tile = tiles - 1 - w % tiles, nh = w / tiles;
    const int64_t n = nh / a.Hkv, hk = nh % a.Hkv;
    const int64_t len = a.length(n), start = a.start(n);
    const int64_t row0 = tile * (WAVES * QB * 32) + wave * (QB * 32);

    Frag<T> q[QB][KS];
    int64_t seen[QB];
#pragma unroll
    for (int qb = 0; qb < QB; ++qb) {
        const int64_t row = row0 + qb * 32 + (lane & 31), t = row / a.G, g = row % a.G;
        const bool there = row < a.R;
        seen[qb] = there ? a.seen(len, start, t) : 0;
        const T *p = static_cast<const T *>(a.q.p) + n * a.q.n + t * a.q.t + (hk * a.G + g) * a.q.h;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) q[qb][ks] = load_frag<T>(p, ks * 16 + half * 8, there ? a.D : 0);
    }
    // keys the block looks at, and this split's share of them in whole tiles
    const int64_t last = min(tile * (WAVES * QB * 32) + WAVES * QB * 32, a.R) - 1;
    const int64_t want = (a.seen(len, start, last / a.G) + KT - 1) / KT, each = (want + a.splits - 1) / a.splits;
    const int64_t kt0 = split * each, kt1 = min(want, kt0 + each);
    // of this wave's rows: tiles before `whole` are seen by every row, tiles from `none` on by none
    const int64_t first_seen = row0 < a.R ? a.seen(len, start, row0 / a.G) : 0;
    const int64_t last_seen = row0 < a.R ? a.seen(len, start, (min(row0 + QB * 32, a.R) - 1) / a.G) : 0;
    const int64_t whole = first_seen / KT, none = (last_seen + KT - 1) / KT;

    const T *kp = static_cast<const T *>(a.k.p) + n * a.k.n + hk * a.k.h;
    const T *vp = static_cast<const T *>(a.v.p) + n * a.v.n + hk * a.v.h;
    Mover<T, DP, KT, THREADS> km, vm;
    auto load = [&](int64_t kt) {
        // rows behind the length are zeros: what stands there takes no part
        km.load(tid, a.D, [&](int r) { return kt * KT + r < len ? kp + (kt * KT + r) * a.k.t : nullptr; });
        vm.load(tid, a.D, [&](int r) { return kt * KT + r < len ? vp + (kt * KT + r) * a.v.t : nullptr; });
    };

    f32x16 o[QB][DB];
    float m[QB], l[QB];
#pragma unroll
    for (int qb = 0; qb < QB; ++qb) {
        m[qb] = -INFINITY;
        l[qb] = 0.0f;
#pragma unroll
        for (int db = 0; db < DB; ++db) o[qb][db] = f32x16{};
    }
    const float c = a.scale * kLog2e;

    if (kt0 < kt1) {
        load(kt0);
        km.store(lds[0][0], tid);
        vm.store(lds[0][1], tid);
    }
    for (int64_t kt = kt0; kt < kt1; ++kt) {
        __syncthreads();
        const int buf = int(kt - kt0) & 1;
        if (kt + 1 < kt1) load(kt + 1);
        if (kt < none) {
            const T *kl = lds[buf][0], *vl = lds[buf][1];
            f32x16 s[QB][KB];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                for (int qb = 0; qb < QB; ++qb) s[qb][kb] = f32x16{};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const Frag<T> kf = L::by_rows(kl, kb * 32 + (lane & 31), ks, half);
#pragma unroll
                    for (int qb = 0; qb < QB; ++qb) s[qb][kb] = mma(kf, q[qb][ks], s[qb][kb]);
                }
            }
            if (kt >= whole) {
#pragma unroll
                for (int qb = 0; qb < QB; ++qb) {
                    const int end = int(max(int64_t(0), min(seen[qb] - kt * KT, int64_t(KT))));
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                        for (int r = 0; r < 16; ++r) s[qb][kb][r] = kb * 32 + c_row(r, half) < end ? s[qb][kb][r] : -INFINITY;
                }
            }
#pragma unroll
            for (int qb = 0; qb < QB; ++qb) {
                float top = s[qb][0][0];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int r = 0; r < 16; ++r) top = fmaxf(top, s[qb][kb][r]);
                top = half_max(top) * c;
                const bool moves = top > m[qb] + kSlack || (m[qb] == -INFINITY && top > -INFINITY);
                if (__any(moves)) {
                    const float to = moves ? top : m[qb];
                    const float f = moves ? exp2_fast(m[qb] - to) : 1.0f;
                    m[qb] = to;
                    l[qb] *= f;
#pragma unroll
                    for (int db = 0; db < DB; ++db)
#pragma unroll
                        for (int r = 0; r < 16; ++r) o[qb][db][r] *= f;
                }
                const float base = m[qb] == -INFINITY ? 0.0f : m[qb] - kWeightBias<T>;
                float sum = 0.0f;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const float e = exp2_fast(fmaf(s[qb][kb][r], c, -base));
                        s[qb][kb][r] = e;
                        sum += e;
                    }
                l[qb] += sum;
            }
#pragma unroll
            for (int st = 0; st < KT / 16; ++st) {
                Frag<T> p[QB];
#pragma unroll
                for (int qb = 0; qb < QB; ++qb) p[qb] = operand<T>(s[qb][st / 2], st % 2);
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    const Frag<T> vf = L::by_columns(vl, st * 16, db, lane);
#pragma unroll
                    for (int qb = 0; qb < QB; ++qb) o[qb][db] = mma(vf, p[qb], o[qb][db]);
                }
            }
        }
        if (kt + 1 < kt1) {
            km.store(lds[buf ^ 1][0], tid);
            vm.store(lds[buf ^ 1][1], tid);
        }
    }

#pragma unroll
    for (int qb = 0; qb < QB; ++qb) {
        const int64_t row = row0 + qb * 32 + (lane & 31), t = row / a.G, g = row % a.G;
        if (row >= a.R) continue;
        const float sum = half_sum(l[qb]), to = m[qb] - kWeightBias<T>;
        if (a.splits == 1) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            const int64_t h = hk * a.G + g;
            store_columns<T, DB>(static_cast<T *>(a.out) + ((n * a.Tq + t) * a.H + h) * a.D, o[qb], inv, a.D, half);
            if (half == 0) a.lse[(n * a.H + h) * a.Tq + t] = sum == 0.0f ? -INFINITY : (to + __log2f(sum)) * kLn2;
        } else {
            // (o, m, l) of this split: the join takes them
            const int64_t place = (int64_t(split) * a.N * a.Hkv + nh) * a.R + row;
            float *stat = a.part + 2 * place, *part = a.part + 2 * a.splits * a.N * a.Hkv * a.R + place * a.D;
            if (half == 0) {
                stat[0] = sum == 0.0f ? -INFINITY : to;
                stat[1] = sum;
            }
            store_columns<float, DB>(part, o[qb], 1.0f, a.D, half);
        }
    }
}

// The splits of a row, one wave a row: weights 2^(m - largest m).
template <class T>
__global__ __launch_bounds__(256) void attend_join_kernel(Attention a)
{
    const int64_t rows = a.N * a.Hkv * a.R;
    const int lane = threadIdx.x & 63;
    const int64_t id = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (id >= rows) return;
    const int64_t nh = id / a.R, row = id % a.R, n = nh / a.Hkv, h = nh % a.Hkv * a.G + row % a.G, t = row / a.G;
    const float *stat = a.part, *part = a.part + 2 * a.splits * rows;
    float top = -INFINITY;
    for (int s = 0; s < a.splits; ++s) top = fmaxf(top, stat[2 * (s * rows + id)]);
    float acc[kMaxHead / 64] = {}, sum = 0.0f;
    for (int s = 0; s < a.splits; ++s) {
        const float m = stat[2 * (s * rows + id)], l = stat[2 * (s * rows + id) + 1];
        if (l == 0.0f) continue;  // nothing seen there
        const float f = exp2_fast(m - top);
        sum = fmaf(l, f, sum);
#pragma unroll
        for (int i = 0; i < kMaxHead / 64; ++i)
            if (i * 64 + lane < a.D) acc[i] = fmaf(part[(s * rows + id) * a.D + i * 64 + lane], f, acc[i]);
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    T *out = static_cast<T *>(a.out) + ((n * a.Tq + t) * a.H + h) * a.D;
#pragma unroll
    for (int i = 0; i < kMaxHead / 64; ++i)
        if (i * 64 + lane < a.D) out[i * 64 + lane] = T(acc[i] * inv);
    if (lane == 0) a.lse[(n * a.H + h) * a.Tq + t] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * kLn2;
}

template <class T>
void launch_attend(Attention a, const AttendPlan &p, hipStream_t st)
{
    a.splits = p.splits;
    const unsigned blocks = unsigned(a.N * a.Hkv * p.tiles * p.splits);
    with_head(a.D, [&](auto head) {
        constexpr int DP = decltype(head)::value, KT = DP * sizeof(T) > 512 ? 32 : 64;
        if (p.waves == 1) attend_kernel<T, DP, 1, 1, KT><<<blocks, 64, 0, st>>>(a, p.tiles);
        else attend_kernel<T, DP, 1, 4, KT><<<blocks, 256, 0, st>>>(a, p.tiles);
    });
    if (p.splits > 1) {
        const int64_t rows = a.N * a.Hkv * a.R;
        attend_join_kernel<T><<<unsigned((rows + 3) / 4), 256, 0, st>>>(a);
    }
}

}  // namespace ct

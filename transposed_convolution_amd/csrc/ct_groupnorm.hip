// ct_groupnorm.hip -- group norm with an activation and dropout, channels-last, and its
// gradient.
//
// x is stored (N, P, C), P the product of the spatial axes; group g holds the C/G channels
// g*C/G .. and all P positions of an image.
//   mean = average of x over the group, rstd = 1 / sqrt(average of (x - mean)^2 + eps)
//   y = drop(act((x - mean) * rstd * gamma[c] + beta[c]))
// Gradient, with xhat = (x - mean) rstd, z = xhat gamma + beta, dz = drop(dy) act'(z):
//   dbeta[c] = sum dz,  dgamma[c] = sum dz xhat            (over images and positions)
//   c1 = average of dz gamma over the group, c2 = average of dz gamma xhat
//   dx = rstd (dz gamma - c1 - xhat c2)
//
// Statistics: a thread takes the mean and the sum of squared distances from it of the
// values it holds, and such triples (count, mean, m2) are joined pairwise (Chan, Golub,
// LeVeque 1983).  A thread takes its values relative to its own first one, so a mean far from
// zero costs no digits of the spread around it, and a value far from the others costs digits
// of the few values only that share its thread; the joins hold means in 64 bits, and in 64
// bits the parameters' gradients are added over images and chunks.
// Everything else is float32 between the one load and the one store of an element.
//
// Both directions need every value of a group before the first output.  Small groups fit the
// registers of one block, which reads them once; for the others a first pass over the
// tensor makes partial sums and a second one reads it again, joins the partial sums at the
// start of every block and writes.  Here are the plan and the entry points, the kernels are
// in ct_groupnorm_fwd.hip and ct_groupnorm_grad.hip.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <numeric>
#include <string>

#include "ct_groupnorm.hpp"

namespace {

using namespace ct::norm;
using ct::Dropout;

struct Sizes {
    int64_t N = 0, C = 0, P = 1, G = 1;
    int dt = CT_FLOAT32;
    bool empty() const { return N == 0 || C == 0 || P == 0; }
};

// Controls for tests and tuning (group_norm_set_control).
std::atomic<int> g_one_block{-1}, g_finish{-1};

void set_lanes(Cut *k, int threads)
{
    k->lanes = 1;
    while (k->lanes < 64 && 2 * k->lanes * k->per <= threads) k->lanes *= 2;
}

// The slabs and the tile of blocks of `threads` threads; false when whole vectors of V
// elements do not fit this channel count.
bool cut_tiles(const Sizes &s, int V, int threads, int64_t most_groups, Cut *k)
{
    const int64_t Cg = s.C / s.G, most = int64_t(threads) * V;
    k->P = s.P;
    k->C = int(s.C);
    k->G = int(s.G);
    k->Cg = int(Cg);
    k->split = 1;
    int64_t unit = 1;  // rows after which a vector starts a row again
    most_groups = std::min<int64_t>(most_groups, kMostGroups);
    if (Cg > most) {
        if (Cg % V) return false;
        k->per = 1;
        k->width = int(most);
        k->split = int((Cg + most - 1) / most);
        k->slabs = int(s.G * k->split);
    } else {
        int64_t per = std::min<int64_t>(most_groups, most / Cg);
        if (per >= s.G) {
            per = s.G;
            unit = V / std::gcd(s.C, int64_t(V));
            if (unit * s.C > most) return false;
        } else if (s.C % V) {
            return false;
        } else {
            const int64_t step = V / std::gcd(Cg, int64_t(V));  // groups of whole vectors
            per = per / step * step;
            if (per == 0) return false;
        }
        k->per = int(per);
        k->width = int(per * Cg);
        k->slabs = int((s.G + per - 1) / per);
    }
    const int64_t fit = std::min<int64_t>(most / k->width, (int64_t(1) << 30) / s.C) / unit * unit;
    if (fit < 1) return false;
    k->rows = int(std::min(fit, (s.P + unit - 1) / unit * unit));
    set_lanes(k, threads);
    return true;
}

int64_t tiles_of(const Cut &k) { return (k.P + k.rows - 1) / k.rows; }

// Chunks of about `tiles` tiles, at most 2^30: tiles and chunks fit 32 bits for every size that is
// let through (2^58 elements), as a query for a workspace may name sizes no memory holds.
void cut_chunks(Cut *k, int64_t tiles)
{
    tiles = std::min(tiles, int64_t(1) << 30);
    const int64_t all = tiles_of(*k), chunks = (all + tiles - 1) / tiles;
    k->tiles = int((all + chunks - 1) / chunks);
    k->chunks = int((all + k->tiles - 1) / k->tiles);
    k->last_tiles = int(all - int64_t(k->chunks - 1) * k->tiles);
    k->last_rows = int(k->P - (all - 1) * k->rows);
}

// One block for a group's slab where a thread holds at most four vectors and the reads stay
// small.  The slab of a block may be only 16 bytes wide, and each block reads the whole
// 128-byte lines it touches: what counts is those.  Measured (float16, 256 channels in 32
// groups, N images of P positions; one block / two passes, us): N 1, P 2048 9.0 / 12.6,
// P 4096 (eight vectors) 15.2 / 12.6; N 8, P 1024 (32 MiB of lines) 13.8 / 16.4, P 2048
// 25.0 / 17.1; N 32, P 256 (32 MiB) 12.8 / 14.2, P 1024 44.5 / 15.8.  Gradient: N 1, P 1024
// 10.5 / 11.4, P 2048 (eight vectors) 15.3 / 12.6; N 8, P 256 (16 MiB) 10.2 / 10.9, P 1024
// (64 MiB) 21.1 / 16.2; 64 channels in 16 groups, float32, N 8, P 1024 (32 MiB) 12.2 / 11.6.
constexpr int64_t kOneBytes = 32 << 20, kOneGradBytes = 16 << 20;
int64_t line_bytes(const Sizes &s, const Cut &k, bool backward)
{
    const int64_t run = int64_t(k.width) * int64_t(ct::float_size(s.dt));
    const int64_t dense = s.N * s.P * s.C * int64_t(ct::float_size(s.dt));  // no line is read less than once
    if (dense > kOneBytes) return dense;
    const int64_t lines = s.N * s.P * ((s.C + k.width - 1) / k.width) * ((run + 127) / 128 * 128);
    return backward ? 2 * lines : lines;
}

// Parts that every block of the second pass joins by itself; more are joined by a kernel
// between the passes.  Joined by every block / by a kernel, us, with SiLU: 36 x 1001 float32, 4
// images (a few parts) 12.2 / 13.8, gradient 13.0 / 14.8; float16, 8 x 256 x 16384 in 32 groups
// (16 KB a block) 40.5 / 40.7, gradient 65.9 / 67.7; bfloat16, 2 x 64 x 131072 in 16 groups (32 KB)
// 31.9 / 28.4, gradient 36.0 / 37.3; float16, 64 x 1048576 in 16 groups (64 KB) 90.1 / 82.8,
// gradient 119.6 / 119.0; 256 x 131072 in 32 groups (128 KB) 59.3 / 41.9, gradient 71.5 / 68.6;
// 256 x 65536 in 256 groups (1 MB) 287 / 34, gradient 302 / 45.
constexpr int64_t kPartBytes = 32 << 10;
// Blocks of a first pass, at most about.  The forward call's have 512 threads, and 512 of them are one
// round of the chip; the gradient's have 256, so 512 are half a round of what its registers
// allow, and a whole one gained as much in one call as it lost in the other (us at 256 / 512 /
// 768 / 1024, whole call: forward 8 x 256 x 16384 float16 43.5 / 41.2 / 47 / 48, its gradient
// 83.4 / 76.9 / 81.7 / 75.9, gradient 2 x 64 x 131072 39.2 / 37.4 / 40.2 / 38.9).
constexpr int64_t kStatBlocks = 512;
// and of a second one, 1024 blocks of 256 threads (us at 512 / 768 / 1024 / 1536 / 2048, the same
// calls: 41.0 / 40.2 / 40.8 / 40.2 / 41.1, 78.9 / 75.7 / 75.8 / 74.7 / 74.2, 39.5 / 38.6 / 36.6 /
// 39.5 / 39.3).
constexpr int64_t kApplyBlocks = 1024;

Plan make_plan(const Sizes &s, bool backward)
{
    Plan p;
    if (s.empty()) return p;
    const int V = s.dt == CT_FLOAT32 ? 4 : 8;
    const int64_t Cg = s.C / s.G;
    size_t at = 0;
    auto place = [&](size_t bytes) {
        const size_t q = at;
        at += (bytes + 255) & ~size_t(255);
        return q;
    };
    p.run = Cg % V == 0 ? V : Cg % 4 == 0 && s.C % V == 0 ? 4 : 1;
    // one block for all positions of as few groups as make whole vectors
    const int want_one = g_one_block.load(std::memory_order_relaxed);
    if (want_one != 0) {
        const int64_t step = V / std::gcd(Cg, int64_t(V));
        const int threads = backward ? kOneGradThreads : kOneThreads;
        if (cut_tiles(s, V, threads, step, &p.a) && p.a.split == 1 && tiles_of(p.a) <= kOneTiles &&
            line_bytes(s, p.a, backward) <= (backward ? kOneGradBytes : kOneBytes)) {
            p.one = true;
            cut_chunks(&p.a, kOneTiles);
            p.threads = (int(int64_t(p.a.rows) * p.a.width / V) + 63) / 64 * 64;
            set_lanes(&p.a, p.threads);
            p.s = p.a;
            if (backward) p.sums = place(size_t(s.N) * s.C * 8);
            p.bytes = at;
            return p;
        }
    }
    const int stat_threads = backward ? kGradThreads : kStatThreads;
    p.vec = cut_tiles(s, V, kApplyThreads, kMostGroups, &p.a) && cut_tiles(s, V, stat_threads, kMostGroups, &p.s);
    if (!p.vec) {
        cut_tiles(s, 1, kApplyThreads, kMostGroups, &p.a);
        cut_tiles(s, 1, stat_threads, kMostGroups, &p.s);
    }
    const int64_t stat_rows = s.N * p.s.slabs * tiles_of(p.s), apply_rows = s.N * p.a.slabs * tiles_of(p.a);
    cut_chunks(&p.s, std::max<int64_t>(1, (stat_rows + kStatBlocks - 1) / kStatBlocks));
    cut_chunks(&p.a, std::max<int64_t>(1, (apply_rows + kApplyBlocks - 1) / kApplyBlocks));
    const int want_finish = g_finish.load(std::memory_order_relaxed);
    p.finish = want_finish >= 0 ? want_finish != 0 : int64_t(p.s.chunks) * p.s.split * p.a.per * 8 > kPartBytes;
    p.part = place(size_t(s.N) * s.G * p.s.chunks * p.s.split * 8);
    p.stats = place(size_t(s.N) * s.G * 8);
    if (backward) p.sums = place(size_t(s.N) * p.s.chunks * s.C * 8);
    p.bytes = at;
    return p;
}

ct_status fail(ct_status st, const std::string &msg)
{
    ct::set_last_error(msg);
    return st;
}

ct_status check_sizes(int dt, int nsp, const int64_t *shape, int64_t groups, Sizes *s)
{
    if (!ct::is_float_type(dt)) return fail(CT_EUNSUPPORTED, "dtype must be CT_FLOAT32, CT_FLOAT16 or CT_BFLOAT16");
    if (nsp < 1 || nsp > 3) return fail(CT_EINVAL, "the spatial rank must be 1, 2 or 3");
    if (!shape) return fail(CT_EINVAL, "x_shape is NULL");
    for (int a = 0; a < nsp + 2; ++a)
        if (shape[a] < 0) return fail(CT_EINVAL, "sizes must not be negative");
    s->dt = dt;
    s->N = shape[0];
    s->C = shape[1];
    s->G = groups;
    int64_t total = 1;
    for (int a = 0; a < nsp + 2; ++a) {
        if (shape[a] > 0 && total > (int64_t(1) << 58) / shape[a]) return fail(CT_EUNSUPPORTED, "more than 2^58 elements");
        total *= shape[a] > 0 ? shape[a] : 1;
    }
    for (int a = 0; a < nsp; ++a) s->P *= shape[2 + a];
    if (groups < 1 || s->C % groups != 0) return fail(CT_EINVAL, "groups must be at least 1 and divide the channels");
    if (s->C > (1 << 30)) return fail(CT_EUNSUPPORTED, "more than 2^30 channels");
    return CT_OK;
}

ct_status check_act(int kind, float p0, float p1, ct::Act *act)
{
    act->kind = kind;
    act->p0 = p0;
    act->p1 = p1;
    switch (kind) {
    case CT_ACT_IDENTITY:
    case CT_ACT_RELU:
    case CT_ACT_SILU: return CT_OK;
    case CT_ACT_LEAKY_RELU:
        return std::isfinite(p0) ? CT_OK : fail(CT_EINVAL, "leaky ReLU slope must be finite");
    case CT_ACT_CLIP:
        return std::isfinite(p0) && std::isfinite(p1) && p0 <= p1
                   ? CT_OK
                   : fail(CT_EINVAL, "clip bounds must be finite with lower <= upper");
    default: return fail(CT_EINVAL, "unknown activation");
    }
}

ct_status check_params(int dt, int pt, const void *gamma, const void *beta)
{
    if (pt != dt && pt != CT_FLOAT32) return fail(CT_EUNSUPPORTED, "param_dtype must be dtype or CT_FLOAT32");
    if (!ct::aligned_to(gamma, ct::float_size(pt)) || !ct::aligned_to(beta, ct::float_size(pt)))
        return fail(CT_EINVAL, "gamma and beta must be aligned to their element size");
    return CT_OK;
}

// A launch holds fewer than 2^32 threads; here each of the call's launches at most 2^31: the two
// passes (512 threads a block in the forward call's first one, else 256), the blocks for the
// parameters' gradients that go before the second, and a wave a group where the parts are
// joined between.
ct_status check_launches(const Sizes &s, const Plan &p, bool backward)
{
    constexpr int64_t most = int64_t(1) << 31;
    const int64_t head = backward ? param_blocks(s.C) : 0;
    int64_t first = 0, second = 0;
    if (!s.empty()) {
        first = s.N * p.s.chunks * p.s.slabs;
        second = s.N * p.a.chunks * p.a.slabs;
    }
    if (first > most / (backward ? kGradThreads : kStatThreads) || second > most / kApplyThreads - head ||
        (p.finish && s.N * s.G > most / 64))
        return fail(CT_EUNSUPPORTED, "more than 2^31 threads in a launch: too many images, channels or groups");
    return CT_OK;
}

}  // namespace

extern "C" {

ct_status group_norm_set_control(int one_block, int join)
{
    ct::set_last_error(std::string());
    if (one_block < -1 || one_block > 0) return fail(CT_EINVAL, "one_block must be -1 (automatic) or 0 (never)");
    if (join < -1 || join > 1) return fail(CT_EINVAL, "join must be -1 (automatic), 0 or 1");
    g_one_block.store(one_block, std::memory_order_relaxed);
    g_finish.store(join, std::memory_order_relaxed);
    return CT_OK;
}

ct_status group_norm_workspace_size(ct_dtype dtype, int nsp, const int64_t *x_shape, int64_t groups, int backward,
                                    size_t *bytes_out)
{
    ct::set_last_error(std::string());
    if (!bytes_out) return fail(CT_EINVAL, "bytes_out is NULL");
    if (backward != 0 && backward != 1) return fail(CT_EINVAL, "backward must be 0 or 1");
    Sizes s;
    const ct_status st = check_sizes(ct::enum_int(dtype), nsp, x_shape, groups, &s);
    if (st != CT_OK) return st;
    const Plan p = make_plan(s, backward != 0);
    const ct_status ls = check_launches(s, p, backward != 0);
    if (ls == CT_OK) *bytes_out = p.bytes;
    return ls;
}

ct_status group_norm_nd(ct_dtype dtype, int nsp, const void *x, const int64_t *x_shape, int64_t groups,
                        ct_dtype param_dtype, const void *gamma, const void *beta, float eps, ct_activation activation,
                        float act_p0, float act_p1, double dropout_p, uint64_t seed, uint64_t offset,
                        const uint64_t *step, void *y, float *mean, float *rstd, void *workspace, size_t workspace_bytes,
                        void *stream)
{
    ct::set_last_error(std::string());
    const int dt = ct::enum_int(dtype), pt = ct::enum_int(param_dtype);
    Sizes s;
    ct::Act act;
    Dropout drop;
    std::string err;
    ct_status st = check_sizes(dt, nsp, x_shape, groups, &s);
    if (st == CT_OK) st = check_params(dt, pt, gamma, beta);
    if (st == CT_OK) st = check_act(ct::enum_int(activation), act_p0, act_p1, &act);
    if (st != CT_OK) return st;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(CT_EINVAL, "eps must be finite and not negative");
    st = ct::make_dropout(dropout_p, seed, offset, step, &drop, &err);
    if (st != CT_OK) return fail(st, err);
    const size_t esz = ct::float_size(dt);
    if (!ct::aligned_to(x, esz) || !ct::aligned_to(y, esz) || !ct::aligned_to(mean, 4) || !ct::aligned_to(rstd, 4))
        return fail(CT_EINVAL, "tensor pointers must be aligned to the element size");
    if (workspace && !ct::aligned_to(workspace, 16)) return fail(CT_EINVAL, "workspace must be 16-byte aligned");
    if (s.empty()) return CT_OK;
    if (!x || !y) return fail(CT_EINVAL, "x or y is NULL");
    const Plan p = make_plan(s, false);
    st = check_launches(s, p, false);
    if (st != CT_OK) return st;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    ct::Scratch ws;
    st = ws.take(workspace, workspace_bytes, p.bytes, hs, &err);
    if (st != CT_OK) return fail(st, err);
    Call c;
    c.N = s.N;
    c.dt = dt;
    c.params_f32 = pt == CT_FLOAT32;
    c.x = x;
    c.y = y;
    c.gamma = gamma;
    c.beta = beta;
    c.eps = eps;
    c.mean = mean;
    c.rstd = rstd;
    c.act = act;
    c.drop = drop;
    launch_forward(c, p, static_cast<char *>(ws.p), hs);
    st = ct::launch_status("group norm launch failed", &err);
    return st == CT_OK ? CT_OK : fail(st, err);
}

ct_status group_norm_backward_nd(ct_dtype dtype, int nsp, const void *dy, const void *x, const int64_t *x_shape,
                                 int64_t groups, const float *mean, const float *rstd, ct_dtype param_dtype,
                                 const void *gamma, const void *beta, ct_activation activation, float act_p0,
                                 float act_p1, double dropout_p, uint64_t seed, uint64_t offset, const uint64_t *step,
                                 void *dx, void *dgamma, void *dbeta, void *workspace, size_t workspace_bytes,
                                 void *stream)
{
    ct::set_last_error(std::string());
    const int dt = ct::enum_int(dtype), pt = ct::enum_int(param_dtype);
    Sizes s;
    ct::Act act;
    Dropout drop;
    std::string err;
    ct_status st = check_sizes(dt, nsp, x_shape, groups, &s);
    if (st == CT_OK) st = check_params(dt, pt, gamma, beta);
    if (st == CT_OK) st = check_params(dt, pt, dgamma, dbeta);
    if (st == CT_OK) st = check_act(ct::enum_int(activation), act_p0, act_p1, &act);
    if (st != CT_OK) return st;
    st = ct::make_dropout(dropout_p, seed, offset, step, &drop, &err);
    if (st != CT_OK) return fail(st, err);
    const size_t esz = ct::float_size(dt);
    if (!ct::aligned_to(x, esz) || !ct::aligned_to(dy, esz) || !ct::aligned_to(dx, esz) || !ct::aligned_to(mean, 4) ||
        !ct::aligned_to(rstd, 4))
        return fail(CT_EINVAL, "tensor pointers must be aligned to the element size");
    if (workspace && !ct::aligned_to(workspace, 16)) return fail(CT_EINVAL, "workspace must be 16-byte aligned");
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    if (s.C == 0) return CT_OK;
    if (!s.empty() && (!x || !dy || !dx || !mean || !rstd)) return fail(CT_EINVAL, "x, dy, dx, mean or rstd is NULL");
    const Plan p = make_plan(s, true);
    st = check_launches(s, p, true);
    if (st != CT_OK) return st;
    if (s.empty()) {  // no element: the parameters' gradients are 0
        if (dgamma || dbeta) launch_no_gradient(dt, pt == CT_FLOAT32, int(s.C), dgamma, dbeta, hs);
        st = ct::launch_status("group norm gradient launch failed", &err);
        return st == CT_OK ? CT_OK : fail(st, err);
    }
    ct::Scratch ws;
    st = ws.take(workspace, workspace_bytes, p.bytes, hs, &err);
    if (st != CT_OK) return fail(st, err);
    Call c;
    c.N = s.N;
    c.dt = dt;
    c.params_f32 = pt == CT_FLOAT32;
    c.x = x;
    c.dy = dy;
    c.dx = dx;
    c.gamma = gamma;
    c.beta = beta;
    c.dgamma = dgamma;
    c.dbeta = dbeta;
    c.mean = const_cast<float *>(mean);  // read only there
    c.rstd = const_cast<float *>(rstd);
    c.act = act;
    c.drop = drop;
    launch_gradient(c, p, static_cast<char *>(ws.p), hs);
    st = ct::launch_status("group norm gradient launch failed", &err);
    return st == CT_OK ? CT_OK : fail(st, err);
}

}  // extern "C"

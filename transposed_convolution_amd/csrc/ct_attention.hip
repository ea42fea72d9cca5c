// ct_attention.hip -- attention and its gradient: checks, the split of the work, entry points.
#include "ct_attention.hpp"

#include <algorithm>
#include <string>

namespace ct {

namespace {
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align16(size_t n) { return (n + 15) & ~size_t(15); }
}  // namespace

constexpr int kMostSplits = 64;  // attend_join_kernel has a lane for each

AttendPlan attend_plan(const Attention &a, int dtype)
{
    AttendPlan p;
    const int64_t heads = int64_t(a.N) * a.Hkv;
    p.few = a.R <= 32;
    p.tiles = p.few ? 1 : int(ceil_div(a.R, 128));
    // Blocks wanted before a call's work is split over its keys (and joined by a second kernel: 4 us), and the keys a
    // split should have.  Few rows, 8 heads over 4 of 64: 200 keys took 7.2 us in one block a head and 9.5 split, 4096
    // keys 10.9 in splits of 128 and 13.7 in splits of 512.  Many rows: a chunk is to outweigh its part of the output, and
    // float32 products take 8 times as long (5 heads of 40, 77 rows, 1001 keys, float32: 28.6 us whole, 15 in 9 parts).
    const int64_t base = heads * p.tiles, wanted = p.few && padded_head(a.D) * float_size(dtype) > 256 ? 256 : 512,
                  least = p.few ? 128 : dtype == CT_FLOAT32 ? 64 : 256;
    int64_t splits = 1;
    if (base > 0 && base < wanted && !(p.few && a.Tk <= 512))
        splits = std::max<int64_t>(1, std::min({ceil_div(wanted, base), ceil_div(a.Tk, least), int64_t(kMostSplits)}));
    // chunks are whole steps of a block
    const int64_t step = p.few ? 128 : 64;
    p.chunk = int(splits > 1 ? ceil_div(ceil_div(a.Tk, splits), step) * step : std::max(1, a.Tk));
    p.splits = int(std::max<int64_t>(1, ceil_div(a.Tk, p.chunk)));
    if (p.splits > 1) p.bytes = size_t(p.splits) * size_t(heads * a.R) * size_t(a.D + 2) * 4;
    return p;
}

AttendGradPlan attend_grad_plan(const Attention &a, int dtype)
{
    AttendGradPlan p;
    const int64_t heads = int64_t(a.N) * a.Hkv;
    // Blocks of several waves share what they read, blocks of one wave make more of a small call: those
    // are taken where the former, split as far as is sensible, would not fill the chip (4 x 257 tokens, 3 heads of 36,
    // float32: 116 us with 4 waves, 44.6 with one).
    const size_t bytes = padded_head(a.D) * float_size(dtype);
    const int64_t most = std::max(a.Tk, a.R);
    const bool fills = heads * ceil_div(most, 128) * std::max<int64_t>(1, std::min<int64_t>(a.Tk, a.R) / 512) >= 256;
    p.waves = fills || bytes > kOneWaveBytes ? 4 : 1;
    p.key_span = p.waves == 1 ? 32 : wide_keys(bytes) ? 256 : padded_head(a.D) == 256 && dtype != CT_FLOAT32 ? 64 : 128;
    p.row_span = p.waves == 1 ? 32 : 128;
    // 2048 waves (2 a SIMD) fill the chip.  In a causal call half of the (tile, chunk) pairs have nothing to do and
    // the others differ, so three times as many are given out: the gradient of 4097 tokens, 16 heads over 4 of 128, took
    // 511, 470, 446 and 494 us with 8, 10, 12 and 16 parts for its key blocks (8 waves each); its row blocks (4
    // waves) alone 325, 204, 257 and 219 with 2, 3, 4 and 6.
    auto chunk = [&](int64_t blocks, int64_t length, int waves) {
        const int64_t wanted = (waves > 1 && a.causal ? 6144 : 2048) / waves, least = fills ? 512 : 64, step = 64;
        if (blocks == 0 || length == 0 || blocks >= wanted) return std::max<int64_t>(1, length);
        const int64_t splits = std::max<int64_t>(1, std::min({ceil_div(wanted, blocks), ceil_div(length, least), int64_t(kMostSplits)}));
        return splits == 1 ? length : ceil_div(ceil_div(length, splits), step) * step;
    };
    p.row_chunk = int(chunk(heads * ceil_div(a.Tk, p.key_span), a.R, p.waves > 1 && wide_keys(bytes) ? 8 : p.waves));
    p.key_chunk = int(chunk(heads * ceil_div(a.R, p.row_span), a.Tk, p.waves));
    p.row_splits = int(std::max<int64_t>(1, ceil_div(a.R, p.row_chunk)));
    p.key_splits = int(std::max<int64_t>(1, ceil_div(a.Tk, p.key_chunk)));
    size_t at = 0;
    p.stat = at;
    at = align16(at + size_t(heads * a.R) * 8);
    p.top = at;
    if (dtype == CT_FLOAT16) at = align16(at + size_t(heads * (ceil_div(a.R, 64) + ceil_div(a.Tk, 64))) * 4);
    p.key_part = at;
    if (p.row_splits > 1) at = align16(at + size_t(p.row_splits) * size_t(2 * a.Tk * heads * a.D) * 4);
    p.row_part = at;
    if (p.key_splits > 1) at = align16(at + size_t(p.key_splits) * size_t(a.R * heads * a.D) * 4);
    p.bytes = at;
    return p;
}

}  // namespace ct

namespace {

using ct::Attention;

ct_status fail(ct_status st, const std::string &msg)
{
    ct::set_last_error(msg);
    return st;
}

// Sizes of a call, checked.
ct_status sizes(int dt, const int64_t *q_shape, int64_t tk, int64_t kv_heads, Attention *a, std::string *err)
{
    auto bad = [&](ct_status st, const char *msg) {
        *err = msg;
        return st;
    };
    if (!ct::is_float_type(dt)) return bad(CT_EUNSUPPORTED, "dtype must be CT_FLOAT32, CT_FLOAT16 or CT_BFLOAT16");
    if (!q_shape) return bad(CT_EINVAL, "q_shape is NULL");
    for (int i = 0; i < 4; ++i)
        if (q_shape[i] < 0) return bad(CT_EINVAL, "sizes must not be negative");
    if (tk < 0) return bad(CT_EINVAL, "sizes must not be negative");
    if (q_shape[2] < 1 || kv_heads < 1 || q_shape[2] % kv_heads)
        return bad(CT_EINVAL, "there must be at least one key head, and the heads must be a multiple of the key heads");
    if (q_shape[3] < 1) return bad(CT_EINVAL, "a head needs at least one element");
    if (q_shape[3] > ct::kMaxHead) return bad(CT_EUNSUPPORTED, "heads of more than 256 elements are not served");
    // rows of either side below 2^30: places and counts of them fit an int, sums of two too
    constexpr int64_t most = (int64_t(1) << 30) - 1;
    auto product = [&](int64_t x, int64_t y, int64_t z) {
        if (x == 0 || y == 0 || z == 0) return int64_t(0);
        return x > most || y > most || z > most || x > most / y || x * y > most / z ? most + 1 : x * y * z;
    };
    if (q_shape[0] > most || q_shape[1] > most || q_shape[2] > most || tk > most || product(q_shape[0], q_shape[1], q_shape[2]) > most ||
        product(q_shape[0], tk, kv_heads) > most || product(q_shape[0], kv_heads, 1) > (1 << 22) ||
        product(q_shape[1], q_shape[2], 1) > most)
        return bad(CT_EUNSUPPORTED, "2^30 rows of queries or keys and more, or more than 2^22 images times key heads");
    a->N = int(q_shape[0]);
    a->Tq = int(q_shape[1]);
    a->H = int(q_shape[2]);
    a->D = int(q_shape[3]);
    a->Tk = int(tk);
    a->Hkv = int(kv_heads);
    a->G = a->H / a->Hkv;
    a->R = a->Tq * a->G;
    a->by_g = ct::Div31(a->G);
    return CT_OK;
}

ct_status options(float scale, const int32_t *lengths, int causal, const int32_t *starts, Attention *a, std::string *err)
{
    if (!(scale > 0.0f && scale <= 1.0e38f)) {  // times log2(e) it still is a float32
        *err = "scale must lie in (0, 1e38]";
        return CT_EINVAL;
    }
    if (causal != 0 && causal != 1) {
        *err = "causal must be 0 or 1";
        return CT_EINVAL;
    }
    if (starts && !causal) {
        *err = "starts are for causal calls";
        return CT_EINVAL;
    }
    if (!ct::aligned_to(lengths, 4) || !ct::aligned_to(starts, 4)) {
        *err = "lengths and starts must be aligned to 4 bytes";
        return CT_EINVAL;
    }
    a->scale = scale;
    a->causal = causal;
    a->lengths = lengths;
    a->starts = starts;
    return CT_OK;
}

// Blocks of a launch of 256 threads each, which holds fewer than 2^32 threads.
ct_status launchable(int64_t blocks, std::string *err)
{
    if (blocks < (int64_t(1) << 24)) return CT_OK;
    *err = "too many images, heads and tokens for one launch";
    return CT_EUNSUPPORTED;
}

// A strided operand: (n, t, h) strides in elements, none negative.
ct_status operand(const char *name, const void *p, const int64_t *strides, bool needed, size_t esz, ct::Strided *s, std::string *err)
{
    if (needed && (!p || !strides)) {
        *err = std::string(name) + " or its strides are NULL";
        return CT_EINVAL;
    }
    if (!ct::aligned_to(p, esz)) {
        *err = "tensor pointers must be aligned to the element size";
        return CT_EINVAL;
    }
    if (!needed || !strides) return CT_OK;
    for (int i = 0; i < 3; ++i)
        if (strides[i] < 0 || strides[i] > (int64_t(1) << 40)) {
            *err = std::string("the strides of ") + name + " must lie in 0 .. 2^40";
            return CT_EINVAL;
        }
    if (strides[1] > ct::kMaxTokenStride) {
        *err = std::string("more than 2^24 elements from token to token of ") + name + " are not served";
        return CT_EUNSUPPORTED;
    }
    *s = {p, strides[0], strides[1], strides[2]};
    return CT_OK;
}

}  // namespace

extern "C" ct_status attention_nd(ct_dtype dtype, const int64_t *q_shape, int64_t kv_tokens, int64_t kv_heads, const void *q,
                                  const int64_t *q_strides, const void *k, const int64_t *k_strides, const void *v,
                                  const int64_t *v_strides, float scale, int causal, const int32_t *lengths,
                                  const int32_t *starts, void *out, float *lse, void *workspace, size_t workspace_bytes,
                                  void *stream)
{
    ct::set_last_error(std::string());
    const int dt = ct::enum_int(dtype);
    Attention a;
    std::string err;
    ct_status st = sizes(dt, q_shape, kv_tokens, kv_heads, &a, &err);
    if (st == CT_OK) st = options(scale, lengths, causal, starts, &a, &err);
    if (st != CT_OK) return fail(st, err);
    const size_t esz = ct::float_size(dt);
    const bool some = a.N > 0 && a.Tq > 0, keys = some && a.Tk > 0;
    st = operand("q", q, q_strides, keys, esz, &a.q, &err);
    if (st == CT_OK) st = operand("k", k, k_strides, keys, esz, &a.k, &err);
    if (st == CT_OK) st = operand("v", v, v_strides, keys, esz, &a.v, &err);
    if (st != CT_OK) return fail(st, err);
    if (!ct::aligned_to(out, esz) || !ct::aligned_to(lse, 4) || !ct::aligned_to(workspace, 16))
        return fail(CT_EINVAL, "out must be aligned to the element size, lse to 4 bytes and the workspace to 16");
    if (!some) return CT_OK;
    if (!out || !lse) return fail(CT_EINVAL, "out or lse is NULL");
    a.out = out;
    a.lse = lse;
    const ct::AttendPlan p = ct::attend_plan(a, dt);
    st = launchable(int64_t(a.N) * a.Hkv * p.tiles * p.splits, &err);
    if (st != CT_OK) return fail(st, err);
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    ct::Scratch ws;
    st = ws.take(workspace, workspace_bytes, p.bytes, hs, &err);
    if (st != CT_OK) return fail(st, err);
    ct::mark_before(hs);
    ct::with_type(dt, [&](auto t) { ct::launch_attend<decltype(t)>(a, p, static_cast<float *>(ws.p), hs); });
    ct::mark_after(hs);
    st = ct::launch_status("attention launch failed", &err);
    return st == CT_OK ? CT_OK : fail(st, err);
}

extern "C" ct_status attention_backward_nd(ct_dtype dtype, const int64_t *q_shape, int64_t kv_tokens, int64_t kv_heads,
                                           const void *dout, const int64_t *dout_strides, const void *q,
                                           const int64_t *q_strides, const void *k, const int64_t *k_strides,
                                           const void *v, const int64_t *v_strides, const void *out,
                                           const int64_t *out_strides, const float *lse, float scale, int causal,
                                           const int32_t *lengths, const int32_t *starts, void *dq, void *dk, void *dv,
                                           void *workspace, size_t workspace_bytes, void *stream)
{
    ct::set_last_error(std::string());
    const int dt = ct::enum_int(dtype);
    Attention a;
    std::string err;
    ct_status st = sizes(dt, q_shape, kv_tokens, kv_heads, &a, &err);
    if (st == CT_OK) st = options(scale, lengths, causal, starts, &a, &err);
    if (st != CT_OK) return fail(st, err);
    const size_t esz = ct::float_size(dt);
    const bool rows = a.N > 0 && a.Tq > 0, keys = a.N > 0 && a.Tk > 0, both = rows && keys;
    st = operand("dout", dout, dout_strides, both, esz, &a.d_o, &err);
    if (st == CT_OK) st = operand("q", q, q_strides, both, esz, &a.q, &err);
    if (st == CT_OK) st = operand("k", k, k_strides, both, esz, &a.k, &err);
    if (st == CT_OK) st = operand("v", v, v_strides, both, esz, &a.v, &err);
    if (st == CT_OK) st = operand("out", out, out_strides, both, esz, &a.o, &err);
    if (st != CT_OK) return fail(st, err);
    if (!ct::aligned_to(dq, esz) || !ct::aligned_to(dk, esz) || !ct::aligned_to(dv, esz) || !ct::aligned_to(lse, 4) ||
        !ct::aligned_to(workspace, 16))
        return fail(CT_EINVAL, "the gradients must be aligned to the element size, lse to 4 bytes and the workspace to 16");
    if (!rows && !keys) return CT_OK;
    if ((rows && !dq) || (keys && (!dk || !dv)) || (both && !lse)) return fail(CT_EINVAL, "dq, dk, dv or lse is NULL");
    a.lse = const_cast<float *>(lse);
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    const ct::AttendGradPlan p = ct::attend_grad_plan(a, dt);
    const int64_t heads = int64_t(a.N) * a.Hkv;
    const auto blocks = [](int64_t n, int64_t each) { return (n + each - 1) / each; };
    // (a block of 8 waves counts twice)
    st = launchable(heads * std::max(blocks(a.R, 64) + blocks(a.Tk, 64), blocks(a.Tk, std::min(p.key_span, 128)) * p.row_splits +
                                                                             blocks(a.R, p.row_span) * p.key_splits), &err);
    if (st != CT_OK) return fail(st, err);
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    ct::Scratch ws;
    st = ws.take(workspace, workspace_bytes, p.bytes, hs, &err);
    if (st != CT_OK) return fail(st, err);
    ct::mark_before(hs);
    ct::with_type(dt, [&](auto t) { ct::launch_attend_grad<decltype(t)>(a, p, static_cast<char *>(ws.p), hs); });
    ct::mark_after(hs);
    st = ct::launch_status("attention gradient launch failed", &err);
    return st == CT_OK ? CT_OK : fail(st, err);
}

extern "C" ct_status attention_workspace_size(ct_dtype dtype, const int64_t *q_shape, int64_t kv_tokens, int64_t kv_heads,
                                              int backward, size_t *bytes_out)
{
    ct::set_last_error(std::string());
    if (!bytes_out) return fail(CT_EINVAL, "bytes_out is NULL");
    if (backward != 0 && backward != 1) return fail(CT_EINVAL, "backward must be 0 or 1");
    const int dt = ct::enum_int(dtype);
    Attention a;
    std::string err;
    const ct_status st = sizes(dt, q_shape, kv_tokens, kv_heads, &a, &err);
    if (st != CT_OK) return fail(st, err);
    const bool rows = a.N > 0 && a.Tq > 0, keys = a.N > 0 && a.Tk > 0;
    a.causal = 1;  // whose plans have at least as many parts
    *bytes_out = backward ? (rows || keys ? ct::attend_grad_plan(a, dt).bytes : 0) : (rows ? ct::attend_plan(a, dt).bytes : 0);
    return CT_OK;
}

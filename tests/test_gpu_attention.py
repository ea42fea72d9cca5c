"""Attention and its gradient on the GPU against plain 64-bit forms (attention_refs), at every
element within bounds derived from the kernels' arithmetic."""
import numpy as np
import pytest
import torch

import attention_refs as A
import layer_refs as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def T():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import transposed_convolution_amd as T
    T.load_library()
    return T


def dev(a, dtype):
    """A float64 array as a device tensor of dtype, and the values it holds there."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DT[dtype])
    return t.cuda(), t.double().numpy()


def host(t):
    return t.double().cpu().numpy()


def ints(a):
    return None if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")


def inputs(dtype, n, tq, tk, h, hk, d, seed, gain=1.5):
    rng = np.random.default_rng(seed)
    made = [dev(rng.normal(size=s) * f, dtype) for s, f in (((n, tq, h, d), gain), ((n, tk, hk, d), 1.0), ((n, tk, hk, d), 1.0),
                                                            ((n, tq, h, d), 1.0))]
    return [t for t, _ in made], [a for _, a in made]


def check_forward(T, dtype, tensors, arrays, seen, scale, what, **mask):
    q, k, v = tensors[:3]
    out, lse = T.attention_nd(q, k, v, scale=scale, **mask)
    torch.cuda.synchronize()
    (o, l), (otol, ltol) = A.attend(*arrays[:3], scale or q.shape[3] ** -0.5, seen, dtype)
    assert out.dtype == q.dtype and out.is_contiguous() and lse.dtype == torch.float32
    R.assert_close(host(out), o, otol, dtype, f"{what} out")
    got = host(lse)
    assert np.array_equal(got == -np.inf, l == -np.inf), what
    fine = np.isfinite(l)
    R.assert_close(got[fine], l[fine], ltol[fine], "f32", f"{what} lse")
    return out, lse


def check_backward(T, dtype, tensors, arrays, seen, scale, what, **mask):
    (q, k, v, do), real = tensors, scale or tensors[0].shape[3] ** -0.5
    (o, l), _ = A.attend(*arrays[:3], real, seen, dtype)
    out, o = dev(o, dtype)
    lse, l = dev(l, "f32")
    grads = T.attention_backward_nd(do, q, k, v, out, lse, scale=scale, **mask)
    torch.cuda.synchronize()
    want, tol = A.attend_grad(arrays[3], *arrays[:3], o, l, real, seen, dtype)
    for name, got, w, t, like in zip(("dq", "dk", "dv"), grads, want, tol, (q, k, v)):
        assert got.dtype == q.dtype and got.shape == like.shape and got.is_contiguous()
        R.assert_close(host(got), w, t, dtype, f"{what} {name}")
    return grads


# n, tq, tk, h, hk, d, causal, lengths, starts
SHAPES = [
    (1, 1, 1, 1, 1, 1, False, None, None),
    (1, 1, 1, 2, 1, 64, True, None, None),
    (2, 1, 77, 4, 2, 64, False, None, None),
    (3, 5, 130, 6, 2, 40, True, (130, 5, 64), (125, 0, 59)),
    (2, 33, 31, 3, 3, 8, False, None, None),
    (2, 64, 64, 2, 2, 32, True, None, None),
    (1, 129, 129, 4, 1, 96, True, None, None),
    (3, 77, 200, 5, 5, 36, False, (200, 0, 131), None),
    (2, 200, 77, 2, 1, 80, True, None, None),            # the first 123 tokens see nothing
    (2, 31, 65, 2, 2, 128, True, (65, 40), (-3, 20)),
    (1, 140, 300, 2, 1, 256, False, (257,), None),
    (2, 50, 70, 3, 1, 129, True, None, None),
    (1, 300, 300, 1, 1, 33, True, None, None),
    (2, 9, 500, 8, 8, 160, False, (-4, 900), None),      # lengths outside are brought inside
    (1, 2, 3000, 12, 3, 64, True, None, None),           # split over the keys
    (2, 150, 1300, 2, 2, 72, False, (1300, 700), None),
    (9, 17, 23, 4, 4, 31, False, tuple(range(0, 27, 3)), None),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=[str(s[:6]) for s in SHAPES])
def test_forward(T, shape, dtype):
    n, tq, tk, h, hk, d, causal, lengths, starts = shape
    seen = A.visible(n, tq, tk, causal, lengths, starts)
    tensors, arrays = inputs(dtype, n, tq, tk, h, hk, d, seed=11)
    check_forward(T, dtype, tensors, arrays, seen, None, str(shape), causal=causal, lengths=ints(lengths), starts=ints(starts))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=[str(s[:6]) for s in SHAPES])
def test_backward(T, shape, dtype):
    n, tq, tk, h, hk, d, causal, lengths, starts = shape
    seen = A.visible(n, tq, tk, causal, lengths, starts)
    tensors, arrays = inputs(dtype, n, tq, tk, h, hk, d, seed=12)
    check_backward(T, dtype, tensors, arrays, seen, None, str(shape), causal=causal, lengths=ints(lengths), starts=ints(starts))


# calls that fill the chip: blocks of several waves, in one piece and split over rows and keys
LARGE = [
    (8, 150, 140, 16, 16, 64, True, (140, 3, 0, 77, 140, 64, 65, 139), None),
    (3, 530, 540, 22, 11, 128, True, None, (10, 300, -40)),
    (2, 300, 700, 48, 24, 96, False, (700, 401), None),
    (16, 257, 129, 8, 8, 33, True, None, None),          # the first 128 tokens see nothing
    (1, 260, 520, 66, 66, 120, True, None, None),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", LARGE, ids=[str(s[:6]) for s in LARGE])
def test_large(T, shape, dtype):
    test_forward(T, shape, dtype)
    test_backward(T, shape, dtype)


def test_layouts(T):
    """Parts of one projection, heads in front of tokens, and repeated keys."""
    n, t, h, hk, d = 2, 90, 4, 2, 40
    rng = np.random.default_rng(21)
    packed, pv = dev(rng.normal(size=(n, t, h + 2 * hk, d)), "bf16")
    do, dov = dev(rng.normal(size=(n, h, t, d)), "bf16")
    cut = lambda a: [a[:, :, :h], a[:, :, h:h + hk], a[:, :, h + hk:]]  # noqa: E731
    seen = A.visible(n, t, t, True, None, None)
    tensors, arrays = cut(packed) + [do.transpose(1, 2)], cut(pv) + [dov.transpose(0, 2, 1, 3)]
    check_forward(T, "bf16", tensors, arrays, seen, 0.2, "parts", causal=True)
    check_backward(T, "bf16", tensors, arrays, seen, 0.2, "parts", causal=True)
    one, ov = dev(rng.normal(size=(1, t, 1, d)), "f16")  # one key head of one image for all
    q, qv = dev(rng.normal(size=(n, h, 7, d)), "f16")
    kv = one.expand(n, t, 2, d)
    tensors = [q.transpose(1, 2), kv, kv, q.transpose(1, 2)]
    arrays = [qv.transpose(0, 2, 1, 3)] + [np.broadcast_to(ov, (n, t, 2, d))] * 2 + [qv.transpose(0, 2, 1, 3)]
    seen = A.visible(n, 7, t, False, None, None)
    check_forward(T, "f16", tensors, arrays, seen, None, "repeated")
    check_backward(T, "f16", tensors, arrays, seen, None, "repeated")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("tq", [3, 150])
def test_hidden_places_hold_anything(T, dtype, tq):
    """NaN and infinities behind the lengths, in keys no query sees, and in queries that see nothing."""
    n, tk, h, hk, d = 3, 200, 4, 2, 48
    lengths, starts = (200, 0, 77), (-1, 0, 77 - tq)
    seen = A.visible(n, tq, tk, True, lengths, starts)
    tensors, arrays = inputs(dtype, n, tq, tk, h, hk, d, seed=31)
    mask = dict(causal=True, lengths=ints(lengths), starts=ints(starts))
    unseen, blind = torch.from_numpy(~seen.any(1)).cuda(), torch.from_numpy(~seen.any(2)).cuda()
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(DT[dtype]).min):
        q, k, v, do = (t.clone() for t in tensors)
        k[unseen] = bad
        v[unseen] = bad
        q[blind] = bad
        do[blind] = bad
        out, _ = check_forward(T, dtype, [q, k, v], [np.where(np.isfinite(a), a, 0) for a in arrays], seen, None, f"{bad}", **mask)
        grads = check_backward(T, dtype, [q, k, v, do], arrays, seen, None, f"{bad}", **mask)
        assert not out[blind].any() and not grads[0][blind].any() and not grads[1][unseen].any() and not grads[2][unseen].any()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(130, 130, 2, 2), (6, 400, 8, 2), (200, 3000, 1, 1)], ids=str)
def test_values_that_are_not_finite_reach_those_that_see_them(T, dtype, shape):
    tq, tk, h, hk = shape
    d = 64
    seen = A.visible(1, tq, tk, True, None, None)
    tensors, arrays = inputs(dtype, 1, tq, tk, h, hk, d, seed=33)
    (o, l), (otol, ltol) = A.attend(*arrays[:3], d ** -0.5, seen, dtype)
    at = tk - tq + tq // 2  # the first key that only the later half of the tokens sees
    for which, bad in ((1, float("nan")), (2, float("nan")), (2, float("inf"))):
        changed = [t.clone() for t in tensors]
        changed[which][0, at, 0, 5] = bad
        out, lse = T.attention_nd(*changed[:3], causal=True)
        torch.cuda.synchronize()
        sees = torch.from_numpy(seen[0, :, at].copy()).cuda()
        mine, other = slice(0, h // hk), slice(h // hk, None)  # the query heads of key head 0
        if which == 1:
            assert out[0, sees][:, mine].isnan().all() and lse[0, mine][:, sees].isnan().all()
        else:
            reached = out[0, sees][:, mine, 5]
            assert (reached.isnan() if bad != bad else reached == float("inf")).all()
        kept = host(out)
        R.assert_close(kept[0, ~seen[0, :, at]], o[0, ~seen[0, :, at]], otol[0, ~seen[0, :, at]], dtype, f"{which} {bad} out")
        R.assert_close(kept[:, :, other], o[:, :, other], otol[:, :, other], dtype, f"{which} {bad} other heads")
        R.assert_close(host(lse)[0][:, ~seen[0, :, at]], l[0][:, ~seen[0, :, at]], ltol[0][:, ~seen[0, :, at]], "f32", "lse")


@pytest.mark.parametrize("gain", [2.0 ** -12, 2.0 ** 9])
def test_float16_gradients_keep_their_digits(T, gain):
    """Gradients of an unscaled mean over many keys, and ones near float16's upper end."""
    n, tq, tk, h, d = 1, 64, 2000, 1, 64
    seen = A.visible(n, tq, tk, False, None, None)
    tensors, arrays = inputs("f16", n, tq, tk, h, h, d, seed=41, gain=0.2)
    do, dov = dev(arrays[3] * gain, "f16")
    tensors[3], arrays[3] = do, dov
    check_backward(T, "f16", tensors, arrays, seen, None, f"gain {gain}")


def test_large_scores(T):
    """Scores of hundreds: the weights are those of the largest keys alone."""
    for dtype in DT:
        tensors, arrays = inputs(dtype, 1, 40, 300, 2, 1, 64, seed=43, gain=60.0)
        seen = A.visible(1, 40, 300, True, None, None)
        check_forward(T, dtype, tensors, arrays, seen, None, dtype, causal=True)
        check_backward(T, dtype, tensors, arrays, seen, None, dtype, causal=True)


def test_gradient_against_differences(T):
    n, tq, tk, h, hk, d = 2, 5, 9, 4, 2, 8
    tensors, _ = inputs("f32", n, tq, tk, h, hk, d, seed=51, gain=1.0)
    q, k, v, do = tensors
    out, lse = T.attention_nd(q, k, v, causal=True)
    grads = T.attention_backward_nd(do, q, k, v, out, lse, causal=True)
    loss = lambda *a: float((T.attention_nd(*a, causal=True)[0].double() * do.double()).sum())  # noqa: E731
    gen = torch.Generator().manual_seed(3)
    for which in range(3):
        u = torch.randn(tensors[which].shape, generator=gen).cuda()
        step = 2.0 ** -7
        moved = [[t + s * u if i == which else t for i, t in enumerate((q, k, v))] for s in (step, -step, 2 * step, -2 * step)]
        a, b, c, e = (loss(*m) for m in moved)
        slope = (8 * (a - b) - (c - e)) / (12 * step)
        want = float((grads[which].double() * u.double()).sum())
        # float32 losses of order 50 over the step: 50 * 2^-22 / 2^-7, and the formula's step^4 times derivatives of
        # the fifth order, which scores of this size keep below 10^4
        assert abs(slope - want) <= 50 * 2.0 ** -15 + 1e4 * step ** 4, which


def test_same_bits_prepared_streamed_and_captured(T):
    n, tq, tk, h, hk, d = 3, 2, 1500, 8, 2, 64
    tensors, arrays = inputs("bf16", n, tq, tk, h, hk, d, seed=61)
    q, k, v, do = tensors
    lengths, starts = ints((1500, 900, 3)), ints((1498, 898, 1))
    mask = dict(causal=True, lengths=lengths, starts=starts)
    out, lse = T.attention_nd(q, k, v, **mask)
    grads = T.attention_backward_nd(do, q, k, v, out, lse, **mask)
    again = T.attention_nd(q, k, v, **mask) + T.attention_backward_nd(do, q, k, v, out, lse, **mask)
    assert all(torch.equal(a, b) for a, b in zip((out, lse) + grads, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = T.attention_nd(q, k, v, stream=side, **mask)
    side.synchronize()
    assert torch.equal(other[0], out) and torch.equal(other[1], lse)
    # a graph of the step, replayed as the cache grows
    with torch.cuda.stream(side):
        forward = T.PreparedCall(T.attention_nd, q, k, v, **mask)
        forward()
        backward = T.PreparedCall(T.attention_backward_nd, do, q, k, v, *forward.out, **mask)
        backward()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        forward()
        backward()
    for place in ((1500, 900, 3), (700, 2, 1500), (2, 1400, 130)):
        lengths.copy_(torch.tensor(place, dtype=torch.int32))
        starts.copy_(lengths - 2)
        graph.replay()
        torch.cuda.synchronize()
        want = T.attention_nd(q, k, v, **mask)
        want += T.attention_backward_nd(do, q, k, v, *want, **mask)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(forward.out + backward.out, want)), place


def test_empty_sides(T):
    q, kv = torch.ones((2, 3, 4, 8), device="cuda"), torch.ones((2, 0, 2, 8), device="cuda")
    out, lse = T.attention_nd(q, kv, kv)
    assert not out.any() and (lse == -float("inf")).all()
    dq, dk, dv = T.attention_backward_nd(q, q, kv, kv, out, lse)
    assert not dq.any() and dk.shape == kv.shape == dv.shape
    k = torch.ones((2, 5, 2, 8), device="cuda")
    none = q[:, :0]
    out, lse = T.attention_nd(none, k, k)
    dq, dk, dv = T.attention_backward_nd(none, none, k, k, out, lse)
    torch.cuda.synchronize()
    assert out.shape == none.shape and not dk.any() and not dv.any()


def test_out_is_not_an_input(T):
    x = torch.ones((2, 3, 4, 8), device="cuda")
    for k, out in (((x + 1), x), (x, x)):
        with pytest.raises(T.ConvTransposeError, match="one of the inputs"):
            T.attention_nd(x, k, k, out=out)
    with pytest.raises(T.ConvTransposeError, match="one of the inputs"):
        T.attention_nd(x + 1, x, x + 2, out=x)
    with pytest.raises(T.ConvTransposeError, match="scale"):
        T.attention_nd(x, x, x, scale=2e38)
    # the largest scale keeps the formula: scores of 0 weigh alike (lse: 8 roundings of log 3 are 5.3e-7)
    out, lse = T.attention_nd(torch.zeros_like(x), x, x, scale=1e38)
    torch.cuda.synchronize()
    assert torch.equal(out, x) and bool((lse - np.log(3.0)).abs().max() < 5.3e-7)


def test_long_cache(T):
    """Keys more than 2^31 elements from the first: two million tokens of 8 heads of 128."""
    tk, hk, d = (1 << 21) + 70, 8, 128
    cache = torch.zeros((2, 1, tk, hk, d), dtype=torch.float16, device="cuda")
    rng = np.random.default_rng(71)
    tail, _ = dev(rng.normal(size=(2, 1, 70, hk, d)), "f16")
    cache[:, :, -70:] = tail
    q, qv = dev(rng.normal(size=(1, 2, hk, d)) * 8, "f16")
    # the tail's scores are of order 8 and its head's 0: those 2^21 keys weigh 2^21 e^-top of the tail's largest
    out, lse = T.attention_nd(q, cache[0], cache[1], scale=1.0, causal=True)
    torch.cuda.synchronize()
    seen = A.visible(1, 2, 70, True, None, np.array([68]))
    k, v = (host(t) for t in tail)
    (o, l), (otol, ltol) = A.attend(qv, k, v, 1.0, seen, "f16")
    assert l.min() > 60  # so they weigh 2^21 e^-60 < 2^-65: nothing
    R.assert_close(host(out), o, otol, "f16", "long cache")
    R.assert_close(host(lse), l, ltol, "f32", "long cache lse")

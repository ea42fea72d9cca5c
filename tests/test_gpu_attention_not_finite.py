"""Attention over keys and values that are not finite: who sees them gets them, nobody else does, and it
takes no longer."""
import time

import numpy as np
import pytest
import torch

import attention_refs as A
import layer_refs as R
from test_gpu_attention import DT, T, dev, host, inputs  # noqa: F401  (T: the fixture)

pytestmark = pytest.mark.gpu


# tq, tk, h, hk, d: whole blocks, a few rows, a split over the keys, shared heads whose rows of a token differ
CALLS = [(200, 200, 2, 2, 64), (130, 130, 4, 1, 40), (6, 400, 8, 2, 128), (32, 90, 1, 1, 256), (200, 1500, 1, 1, 96), (9, 3000, 2, 1, 33)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("call", CALLS, ids=str)
def test_each_element_is_what_its_row_sees(T, dtype, call):  # noqa: F811
    """NaN in one element of a value that all rows see, infinities in others that some see: by element."""
    tq, tk, h, hk, d = call
    seen = A.visible(1, tq, tk, True, None, None)
    tensors, arrays = inputs(dtype, 1, tq, tk, h, hk, d, seed=91)
    (o, l), (otol, ltol) = A.attend(*arrays[:3], d ** -0.5, seen, dtype)
    v, first = tensors[2].clone(), tk - tq  # key `first` is the last that row 0 sees
    late, last, nan, inf = first + tq // 2, tk - 1, float("nan"), float("inf")
    odd = [(0, 0, nan), (0, 1, inf), (first, 2, -inf), (late, 3, inf), (late, 4, nan), (late + 1, 3, -inf), (last, 5, nan), (last, d - 1, inf)]
    for key, column, bad in odd:
        v[0, key, 0, column] = bad
    out, lse = T.attention_nd(*tensors[:2], v, causal=True)
    torch.cuda.synchronize()
    want = o.copy()
    for key, column, bad in odd:  # a weight is positive: it leaves infinities and NaN as they are, and they add up
        rows = seen[0, :, key]
        for head in range(h // hk):
            with np.errstate(invalid="ignore"):
                want[0, rows, head, column] += bad
    got, fine = host(out), np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    assert np.array_equal(np.isfinite(got), fine)
    R.assert_close(got[fine], want[fine], otol[fine], dtype, f"{call} out")
    R.assert_close(host(lse), l, ltol, "f32", f"{call} lse")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("call", [(300, 300, 2, 2, 64), (5, 700, 8, 2, 64)], ids=str)
def test_queries_that_are_not_finite_reach_their_own_row(T, dtype, call):  # noqa: F811
    tq, tk, h, hk, d = call
    seen = A.visible(1, tq, tk, True, None, None)
    tensors, arrays = inputs(dtype, 1, tq, tk, h, hk, d, seed=92)
    (o, l), (otol, ltol) = A.attend(*arrays[:3], d ** -0.5, seen, dtype)
    q = tensors[0].clone()
    q[0, tq // 2, 0, 3] = float("nan")
    out, lse = T.attention_nd(q, *tensors[1:3], causal=True)
    torch.cuda.synchronize()
    hit = np.zeros((1, tq, h), bool)
    hit[0, tq // 2, 0] = True
    got = host(out)
    assert np.isnan(got[hit]).all() and np.isnan(host(lse).transpose(0, 2, 1)[hit]).all()
    R.assert_close(got[~hit], o[~hit], otol[~hit], dtype, "out")
    at = ~hit.transpose(0, 2, 1)
    R.assert_close(host(lse)[at], l[at], ltol[at], "f32", "lse")


@pytest.mark.parametrize("where", ["key", "value", "query", "every value"])
def test_they_take_no_longer(T, where):  # noqa: F811
    """A value that every row sees, and values everywhere: within four times the call without them (whose medians
    vary by a few percent)."""
    tensors, _ = inputs("f16", 1, 2048, 2048, 4, 4, 64, seed=93)
    q, k, v = (t.clone() for t in tensors[:3])
    if where == "query":
        q[:, :, :, 1] = float("nan")
    elif where == "every value":
        v.fill_(float("inf"))
    else:
        (k if where == "key" else v)[0, 0, 0, 1] = float("nan")

    def micros(*a):
        call, found = T.PreparedCall(T.attention_nd, *a, causal=True), []
        for _ in range(8):
            torch.cuda.synchronize()
            begin = time.perf_counter()
            call()
            torch.cuda.synchronize()
            found.append((time.perf_counter() - begin) * 1e6)
        return sorted(found[1:])[3]

    plain, odd = micros(*tensors[:3]), micros(q, k, v)
    print(f"{where}: {odd:.0f} us, {plain:.0f} without")
    assert odd <= 4 * plain


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(200, 2, 1, 40), (600, 24, 24, 64), (600, 24, 12, 128)], ids=str)
@pytest.mark.parametrize("which", ["k", "v", "q", "do"])
def test_gradients_are_right_or_not_finite(T, shape, dtype, which):  # noqa: F811
    """A value that is not finite may reach the gradients of its image and key head, as NaN or infinities: what is
    finite is right.  NaN is there where its sums are.  Other images and key heads are right."""
    t, h, hk, d = shape
    seen = A.visible(2, t, t, True, None, None)
    tensors, arrays = inputs(dtype, 2, t, t, h, hk, d, seed=97)
    (o, l), _ = A.attend(*arrays[:3], d ** -0.5, seen, dtype)
    out, o = dev(o, dtype)
    lse, l = dev(l, "f32")
    want, tol = A.attend_grad(arrays[3], *arrays[:3], o, l, d ** -0.5, seen, dtype)
    at, g = t // 3, h // hk
    rows = slice(at, at + 1) if which in ("q", "do") else slice(at, None)  # the tokens that it is in
    for bad in (float("nan"), float("inf")):
        q, k, v, do = (x.clone() for x in tensors)
        dict(q=q, k=k, v=v, do=do)[which][1, at, 0, 2] = bad
        given = (out.clone(), lse.clone())
        if which != "do":  # those tokens' out and lse are what the forward call leaves
            made = T.attention_nd(q, k, v, causal=True)
            given[0][1, rows, :g], given[1][1, :g, rows] = made[0][1, rows, :g], made[1][1, :g, rows]
        grads = T.attention_backward_nd(do, q, k, v, *given, causal=True)
        torch.cuda.synchronize()
        for name, got, w, bound in zip(("dq", "dk", "dv"), map(host, grads), want, tol):
            mine, sums = np.zeros(got.shape, bool), np.zeros(got.shape, bool)
            mine[1, :, :g if name == "dq" else 1] = True
            if name == "dq":  # the sums that it is in
                sums[1, rows, :g] = True
            elif name == "dk" or which != "v":
                sums[1, :, 0] = True
            assert np.isfinite(got[~mine]).all(), (name, bad)
            if bad != bad and name == "dq":
                assert np.isnan(got[1, rows, 0]).any(-1).all(), name
            elif bad != bad and sums.any():
                assert np.isnan(got[1, :at + 1, 0]).any(-1).all(), name
            fine = np.isfinite(got) & ~sums
            R.assert_close(np.where(fine, got, 0.0), np.where(fine, w, 0.0), bound, dtype, f"{name} {bad}")

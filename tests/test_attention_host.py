"""Argument checks of attention, rotary positions and AdamW that need no GPU: every call here is refused,
or has nothing to do, before anything is launched; and the plain forms against differences."""
import ctypes
import os

import numpy as np
import pytest
import torch

import attention_refs as A


@pytest.fixture(scope="module")
def T():
    import transposed_convolution_amd as T
    if not os.path.exists(T.library_path()):
        from transposed_convolution_amd import build
        build.build()
    T.load_library()
    return T


P = ctypes.c_void_p(256)  # an aligned stand-in: no call here gets as far as a launch
ODD = ctypes.c_void_p(257)
NAN, INF = float("nan"), float("inf")


def _forward(T, dtype=1, shape=(2, 3, 4, 8), tk=5, hk=2, q=P, qs=(96, 32, 8), k=P, ks=(80, 16, 8), v=P, vs=(80, 16, 8), scale=1.0,
             causal=1, lengths=P, starts=P, out=P, lse=P, ws=None, wsb=0):
    i = lambda s: None if s is None else T._i64(s)  # noqa: E731
    return T.load_library().attention_nd(dtype, i(shape), tk, hk, q, i(qs), k, i(ks), v, i(vs), scale, causal, lengths, starts, out,
                                         lse, ws, wsb, None)


def _backward(T, dtype=1, shape=(2, 3, 4, 8), tk=5, hk=2, do=P, dos=(96, 32, 8), q=P, qs=(96, 32, 8), k=P, ks=(80, 16, 8), v=P,
              vs=(80, 16, 8), out=P, outs=(96, 32, 8), lse=P, scale=1.0, causal=1, lengths=P, starts=P, dq=P, dk=P, dv=P, ws=None, wsb=0):
    i = lambda s: None if s is None else T._i64(s)  # noqa: E731
    return T.load_library().attention_backward_nd(dtype, i(shape), tk, hk, do, i(dos), q, i(qs), k, i(ks), v, i(vs), out, i(outs), lse,
                                                  scale, causal, lengths, starts, dq, dk, dv, ws, wsb, None)


def test_attention_refusals(T):
    big = 1 << 31
    bad = [(dict(dtype=2), 3), (dict(dtype=9), 3), (dict(dtype=-1), 3), (dict(shape=None), 1), (dict(shape=(2, -3, 4, 8)), 1),
           (dict(tk=-1), 1), (dict(hk=0), 1), (dict(hk=3), 1), (dict(shape=(2, 3, 0, 8)), 1), (dict(shape=(2, 3, 4, 0)), 1),
           (dict(shape=(2, 3, 4, 257)), 3), (dict(tk=big), 3), (dict(shape=(2, big, 4, 8)), 3), (dict(shape=(big, 3, 4, 8)), 3),
           (dict(shape=(1 << 22, 1, 4, 8)), 3), (dict(shape=(1 << 20, 1 << 9, 2, 8)), 3), (dict(shape=(1 << 40, 1 << 40, 2, 8)), 3),
           (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=NAN), 1), (dict(scale=INF), 1), (dict(causal=2), 1),
           (dict(causal=0), 1), (dict(lengths=ctypes.c_void_p(258)), 1), (dict(starts=ctypes.c_void_p(258)), 1), (dict(q=None), 1),
           (dict(k=None), 1), (dict(v=None), 1), (dict(q=ODD), 1), (dict(qs=None), 1), (dict(qs=(96, -32, 8)), 1),
           (dict(ks=(80, 1 << 25, 8)), 3), (dict(vs=(1 << 41, 16, 8)), 1), (dict(out=None), 1), (dict(out=ODD), 1), (dict(lse=None), 1),
           (dict(lse=ctypes.c_void_p(258)), 1), (dict(ws=ctypes.c_void_p(264), wsb=1 << 20), 1)]
    for kw, want in bad:
        assert _forward(T, **kw) == want, kw
        assert T.convtranspose_last_error(), kw
        assert _backward(T, **kw) == want, kw
    for kw in (dict(do=None), dict(dos=None), dict(do=ODD), dict(outs=(96, 32, -8)), dict(dq=None), dict(dk=None), dict(dv=None),
               dict(dv=ODD), dict(ws=P, wsb=8)):
        assert _backward(T, **kw) == 1, kw
    for shape in ((0, 3, 4, 8), (2, 0, 4, 8)):  # nothing to write
        assert _forward(T, shape=shape, q=None, k=None, v=None, out=None, lse=None) == 0
    assert _backward(T, shape=(0, 3, 4, 8), do=None, q=None, k=None, v=None, out=None, lse=None, dq=None, dk=None, dv=None) == 0
    assert _backward(T, shape=(2, 0, 4, 8), tk=0, do=None, q=None, k=None, v=None, out=None, lse=None, dq=None, dk=None, dv=None) == 0


def test_attention_workspace(T):
    lib, n = T.load_library(), ctypes.c_size_t(0)
    for dtype in (0, 1, 4):
        for shape, tk, hk in (((1, 1, 8, 64), 65536, 2), ((8, 4096, 8, 64), 4096, 8), ((1, 4097, 16, 128), 4097, 4), ((2, 5, 4, 256), 9, 1)):
            for backward in (0, 1):
                assert lib.attention_workspace_size(dtype, T._i64(shape), tk, hk, backward, ctypes.byref(n)) == 0
                rows, keys = shape[0] * shape[1] * shape[2], shape[0] * tk * hk
                # at most 64 float32 parts of each result, and the rows' statistics
                assert n.value <= 64 * 4 * (shape[3] + 2) * (rows + 2 * keys) + 16 * (rows + keys) + 4096
    assert lib.attention_workspace_size(1, T._i64((8, 4096, 8, 64)), 4096, 8, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.attention_workspace_size(1, T._i64((0, 1, 8, 64)), 4096, 8, 1, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.attention_workspace_size(1, T._i64((1, 1, 8, 64)), 4096, 8, 2, ctypes.byref(n)) == 1
    assert lib.attention_workspace_size(1, T._i64((1, 1, 8, 64)), 4096, 8, 0, None) == 1
    assert lib.attention_workspace_size(1, T._i64((1, 1, 8, 64)), 4096, 3, 0, ctypes.byref(n)) == 1


def _rotary(T, dtype=1, shape=(2, 3, 4, 16), x=P, xs=(192, 64, 16), ptype=5, axes=2, pos=P, ps=(6, 2), sections=(3, 5), base=1e4,
            whole=0, inter=0, inverse=0, y=P, ys=(192, 64, 16)):
    i = lambda s: None if s is None else T._i64(s)  # noqa: E731
    return T.load_library().rotary_nd(dtype, i(shape), x, i(xs), ptype, axes, pos, i(ps), i(sections), base, whole, inter, inverse, y,
                                      i(ys), None)


def test_scales_and_rates_that_leave_float32(T):
    # 2e38 log2(e), and the reciprocal of a denormal eps, are infinite
    assert _forward(T, scale=2e38) == 1 and _backward(T, scale=2e38) == 1
    for kw in (dict(eps=1e-40), dict(eps=1e31), dict(lr=1e39), dict(lr=-1e39), dict(scale=1e39)):
        assert _adamw(T, **kw) == 1, kw
    assert _adamw(T, eps=0.0, entry=dict(count=0)) == 0 and _adamw(T, eps=1e-30, entry=dict(count=0)) == 0


def test_rotary_refusals(T):
    bad = [(dict(dtype=2), 3), (dict(dtype=7), 3), (dict(ptype=0), 3), (dict(shape=None), 1), (dict(sections=None), 1), (dict(xs=None), 1),
           (dict(axes=0), 1), (dict(axes=5, sections=(1,) * 5), 1), (dict(shape=(2, 3, 4, -1)), 1), (dict(sections=(3, -1)), 1),
           (dict(sections=(4, 5)), 1), (dict(sections=(200, 100), shape=(2, 3, 4, 1024)), 3), (dict(sections=(257, 0), shape=(2, 3, 4, 1024)), 1),
           (dict(base=0.0), 1), (dict(base=-2.0), 1), (dict(base=NAN), 1), (dict(base=INF), 1), (dict(whole=2), 1), (dict(inter=-1), 1),
           (dict(inverse=3), 1), (dict(x=ODD), 1), (dict(y=ODD), 1), (dict(pos=ctypes.c_void_p(258)), 1), (dict(x=None), 1), (dict(pos=None), 1),
           (dict(ps=(-1, 2)), 1), (dict(ys=(192, 64, -16)), 1), (dict(shape=(1 << 20, 1 << 20, 4, 16)), 3),
           (dict(shape=(1 << 20, 1 << 10, 1, 128)), 3)]
    for kw, want in bad:
        assert _rotary(T, **kw) == want, kw
        assert T.convtranspose_last_error(), kw
    for shape in ((0, 3, 4, 16), (2, 3, 0, 16)):
        assert _rotary(T, shape=shape, x=None, y=None, pos=None) == 0


def _adamw(T, dtype=0, gtype=1, bits=8, ctype=1, tensors=1, entry=None, lr=1e-3, lr_at=None, b1=0.9, b2=0.99, eps=1e-8, step=1, step_at=None,
           scale=1.0, scale_at=None, none=False):
    table = (T._AdamWTensor * max(1, tensors))()
    for i in range(tensors):
        e = dict(param=256, grad=256, m=256, v=256, m_scale=256, v_scale=256, copy=256, count=300, weight_decay=0.1)
        e.update(entry or {})
        table[i] = T._AdamWTensor(**e)
    return T.load_library().adamw_nd(dtype, gtype, bits, ctype, tensors, None if none else table, lr, lr_at, b1, b2, eps, step, step_at,
                                     scale, scale_at, None)


def test_adamw_refusals(T):
    bad = [(dict(dtype=2), 3), (dict(gtype=5), 3), (dict(bits=16), 3), (dict(none=True), 1), (dict(lr=NAN), 1), (dict(lr=INF), 1),
           (dict(b1=1.0), 1), (dict(b1=-0.1), 1), (dict(b2=NAN), 1), (dict(eps=-1.0), 1), (dict(eps=INF), 1), (dict(step=0), 1),
           (dict(step_at=ctypes.c_void_p(260)), 1), (dict(lr_at=ctypes.c_void_p(258)), 1), (dict(scale=NAN), 1),
           (dict(scale_at=ctypes.c_void_p(258)), 1), (dict(entry=dict(count=-1)), 1), (dict(entry=dict(count=1 << 41)), 3),
           (dict(entry=dict(weight_decay=INF)), 1), (dict(entry=dict(param=None)), 1), (dict(entry=dict(grad=None)), 1),
           (dict(entry=dict(m=None)), 1), (dict(entry=dict(v_scale=None)), 1), (dict(ctype=0), 3), (dict(entry=dict(param=258)), 1),
           (dict(entry=dict(grad=257)), 1), (dict(entry=dict(m_scale=258)), 1), (dict(entry=dict(copy=257)), 1),
           (dict(bits=32, entry=dict(m=258)), 1)]
    for kw, want in bad:
        assert _adamw(T, **kw) == want, kw
        assert T.convtranspose_last_error(), kw
    assert _adamw(T, tensors=0, none=True) == 0
    assert _adamw(T, tensors=3, entry=dict(count=0, param=None, grad=None, m=None, v=None)) == 0


def test_binding_refuses_host_tensors(T):
    x = torch.zeros((1, 2, 2, 8))
    with pytest.raises(T.ConvTransposeError, match="HIP device"):
        T.attention_nd(x, x, x)
    with pytest.raises(T.ConvTransposeError, match="HIP device"):
        T.rotary_nd(x, torch.zeros((1, 2, 1), dtype=torch.int32), (4,))
    with pytest.raises(T.ConvTransposeError, match="HIP device"):
        T.adamw_nd([x], [x], [x], [x], lr=1e-3, step=1)
    with pytest.raises(T.ConvTransposeError, match="one tensor a parameter"):
        T.adamw_nd([x], [], [x], [x], lr=1e-3, step=1)
    assert T.adamw_nd([], [], [], [], lr=1e-3, step=1) == ()


def test_gradient_formula_against_differences():
    """The plain gradient, shared heads and masked rows included, against central differences of the plain forward."""
    rng = np.random.default_rng(1)
    n, tq, tk, h, hk, d = 2, 4, 6, 4, 2, 3
    q, k, v, do = (rng.normal(size=s) for s in ((n, tq, h, d), (n, tk, hk, d), (n, tk, hk, d), (n, tq, h, d)))
    seen = A.visible(n, tq, tk, True, (6, 4), (2, -2))
    forward = lambda *a: (A.attend(*a, 0.7, seen, "f32")[0][0] * do).sum()  # noqa: E731
    (out, lse), _ = A.attend(q, k, v, 0.7, seen, "f32")
    grads, _ = A.attend_grad(do, q, k, v, out, lse, 0.7, seen, "f32")
    for which, g in enumerate(grads):
        for _ in range(4):
            u = rng.normal(size=g.shape)
            e = 1e-5
            up, down = ([t + s * u if i == which else t for i, t in enumerate((q, k, v))] for s in (e, -e))
            # roundings of 2^-53 over the step, and its square times third derivatives
            assert abs((forward(*up) - forward(*down)) / (2 * e) - (g * u).sum()) < 1e-8


def test_rotary_formula_turns_back_and_keeps_angles():
    rng = np.random.default_rng(2)
    x, pos = rng.normal(size=(2, 3, 2, 14)), rng.integers(-9, 1 << 40, size=(2, 3, 2))
    for whole in (False, True):
        for inter in (False, True):
            y = A.rotary(x, pos, (2, 4), 1e4, whole, inter, False)
            assert np.allclose(A.rotary(y, pos, (2, 4), 1e4, whole, inter, True), x, atol=1e-14)
            # only differences of positions matter to a product of two turned heads
            a = A.rotary(x, pos, (2, 4), 1e4, whole, inter, False) * A.rotary(x[::-1], pos - 5, (2, 4), 1e4, whole, inter, False)
            b = A.rotary(x, pos + 77, (2, 4), 1e4, whole, inter, False) * A.rotary(x[::-1], pos + 72, (2, 4), 1e4, whole, inter, False)
            assert np.allclose(a[..., :12].sum(-1), b[..., :12].sum(-1), atol=1e-6)

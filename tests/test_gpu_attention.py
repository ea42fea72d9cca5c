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

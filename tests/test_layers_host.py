"""Argument checks of group norm, dropout and the embedding that need no GPU: every call
here is refused, or has nothing to do, before anything is launched."""
import ctypes
import os

import pytest
import torch

import layer_refs as R


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


def _norm(T, dtype=1, nsp=2, x=P, shape=(2, 8, 3, 3), groups=2, ptype=0, gamma=P, beta=P, eps=1e-5, act=0, p0=0.0, p1=0.0,
          p=0.0, step=None, y=P, mean=P, rstd=P, ws=None, wsb=0):
    return T.load_library().group_norm_nd(dtype, nsp, x, None if shape is None else T._i64(shape), groups, ptype, gamma,
                                          beta, eps, act, p0, p1, p, 1, 2, step, y, mean, rstd, ws, wsb, None)


def _norm_grad(T, dtype=1, nsp=2, dy=P, x=P, shape=(2, 8, 3, 3), groups=2, mean=P, rstd=P, ptype=0, gamma=P, beta=P, act=0,
               p0=0.0, p1=0.0, p=0.0, step=None, dx=P, dgamma=P, dbeta=P, ws=None, wsb=0):
    return T.load_library().group_norm_backward_nd(dtype, nsp, dy, x, T._i64(shape), groups, mean, rstd, ptype, gamma, beta,
                                                   act, p0, p1, p, 1, 2, step, dx, dgamma, dbeta, ws, wsb, None)


def test_group_norm_refusals(T):
    bad = [(dict(dtype=2), 3), (dict(dtype=9), 3), (dict(dtype=-1), 3), (dict(dtype=5), 3), (dict(nsp=0), 1), (dict(nsp=4), 1),
           (dict(shape=(2, -8, 3, 3)), 1), (dict(groups=0), 1), (dict(groups=3), 1), (dict(groups=-2), 1), (dict(ptype=4), 3),
           (dict(ptype=2), 3), (dict(gamma=ctypes.c_void_p(258)), 1), (dict(act=5), 1), (dict(act=-1), 1),
           (dict(act=2, p0=INF), 1), (dict(act=3, p0=1.0, p1=0.0), 1), (dict(act=3, p0=NAN), 1), (dict(p=-0.1), 1),
           (dict(p=1.01), 1), (dict(p=NAN), 1), (dict(step=ctypes.c_void_p(260)), 1), (dict(x=ODD), 1),
           (dict(mean=ctypes.c_void_p(258)), 1), (dict(x=None), 1), (dict(ws=ctypes.c_void_p(264), wsb=1 << 20), 1),
           (dict(ws=P, wsb=8, shape=(2, 8, 300, 300)), 1), (dict(shape=(1 << 24, 8, 1, 1)), 3), (dict(shape=(2, 1 << 31, 1, 1), groups=1), 3)]
    for kw, want in bad:
        assert _norm(T, **kw) == want, kw
        assert T.convtranspose_last_error(), kw
        assert _norm_grad(T, **kw) == want, kw
    for kw in (dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(y=None), dict(y=ODD), dict(shape=None)):
        assert _norm(T, **kw) == 1, kw
    for kw in (dict(dy=None), dict(dx=None), dict(mean=None), dict(rstd=None), dict(dy=ODD), dict(dx=ODD),
               dict(dgamma=ctypes.c_void_p(258))):
        assert _norm_grad(T, **kw) == 1, kw
    for shape in ((0, 8, 3, 3), (2, 0, 3, 3), (2, 8, 0, 3)):  # nothing to do
        assert _norm(T, shape=shape, x=None, y=None) == 0
    assert _norm_grad(T, shape=(2, 0, 3, 3), x=None, dy=None) == 0


def test_group_norm_workspace(T):
    lib, n = T.load_library(), ctypes.c_size_t(0)
    for dtype in (0, 1, 4):
        for shape in ((1, 8, 1, 1), (8, 256, 128, 128), (2, 4104, 5, 5), (3, 1001, 9, 9)):
            for backward in (0, 1):
                assert lib.group_norm_workspace_size(dtype, 2, T._i64(shape), 1, backward, ctypes.byref(n)) == 0
                # at most two float32 sums an element, where a chunk is one position
                assert 0 <= n.value <= 8 * shape[0] * shape[1] * shape[2] * shape[3] + (1 << 16)
    assert lib.group_norm_workspace_size(1, 2, T._i64((0, 8, 4, 4)), 1, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.group_norm_workspace_size(1, 2, T._i64((1, 8, 4, 4)), 1, 2, ctypes.byref(n)) == 1
    assert lib.group_norm_workspace_size(1, 2, T._i64((1, 8, 4, 4)), 1, 0, None) == 1
    assert lib.group_norm_workspace_size(1, 2, T._i64((1, 8, 4, 4)), 3, 0, ctypes.byref(n)) == 1


def test_group_norm_control(T):
    lib = T.load_library()
    try:
        assert lib.group_norm_set_control(1, -1) == 1 and lib.group_norm_set_control(-2, -1) == 1
        assert lib.group_norm_set_control(-1, -2) == 1 and T.convtranspose_last_error()
        assert lib.group_norm_set_control(-1, 2) == 1 and lib.group_norm_set_control(0, 1) == 0
    finally:
        T.set_group_norm_control()


def test_dropout_refusals(T):
    def call(dtype=1, count=8, x=P, res=None, y=P, p=0.5, step=None):
        return T.load_library().dropout_nd(dtype, count, x, res, y, p, 1, 2, step, None)

    for kw, want in ((dict(dtype=3), 3), (dict(dtype=6), 3), (dict(dtype=-5), 3), (dict(count=-1), 1), (dict(x=None), 1),
                     (dict(y=None), 1), (dict(x=ODD), 1), (dict(res=ODD), 1), (dict(y=ODD), 1), (dict(p=1.5), 1),
                     (dict(p=-1e-9), 1), (dict(p=NAN), 1), (dict(step=ODD), 1)):
        assert call(**kw) == want, kw
        assert T.convtranspose_last_error(), kw
    assert call(count=0, x=None, y=None) == 0


def test_embedding_refusals(T):
    lib = T.load_library()

    def look(dtype=1, index=6, tokens=4, ids=P, rows=5, width=8, table=P, scale=1.0, y=P):
        return lib.embedding_nd(dtype, index, tokens, ids, rows, width, table, scale, y, None)

    def grad(dtype=1, index=6, tokens=4, ids=P, rows=5, width=8, dy=P, scale=1.0, padding=-1, gt=1, out=P, ws=None, wsb=0):
        return lib.embedding_backward_nd(dtype, index, tokens, ids, rows, width, dy, scale, padding, gt, out, ws, wsb, None)

    both = [(dict(dtype=2), 3), (dict(dtype=6), 3), (dict(index=1), 3), (dict(index=-1), 3), (dict(tokens=-1), 1),
            (dict(rows=-1), 1), (dict(width=-1), 1), (dict(tokens=1 << 31), 3), (dict(rows=1 << 31), 3), (dict(scale=INF), 1),
            (dict(scale=NAN), 1), (dict(ids=ctypes.c_void_p(260)), 1), (dict(ids=None), 1)]
    for kw, want in both:
        assert look(**kw) == want, kw
        assert T.convtranspose_last_error(), kw
        assert grad(**kw) == want, kw
    for kw in (dict(table=None), dict(y=None), dict(table=ODD), dict(y=ODD)):
        assert look(**kw) == 1, kw
    for kw, want in ((dict(gt=4), 3), (dict(gt=2), 3), (dict(padding=5), 1), (dict(padding=-2), 1), (dict(dy=None), 1),
                     (dict(out=None), 1), (dict(dy=ODD), 1), (dict(out=ODD), 1), (dict(ws=P, wsb=16), 1),
                     (dict(ws=ctypes.c_void_p(264), wsb=1 << 20), 1)):
        assert grad(**kw) == want, kw
    assert look(tokens=0, ids=None, y=None) == 0 and look(width=0) == 0
    assert grad(rows=0) == 0 and grad(width=0) == 0
    n = ctypes.c_size_t(0)
    assert lib.embedding_workspace_size(1000, 50, 64, ctypes.byref(n)) == 0 and n.value >= 16 * 1000
    assert lib.embedding_workspace_size(0, 50, 64, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.embedding_workspace_size(10, 50, 64, None) == 1
    assert lib.embedding_workspace_size(-1, 50, 64, ctypes.byref(n)) == 1


def test_convolutions_refuse_the_new_types_and_activation(T):
    lib = T.load_library()
    at = T._attr_args(2, strides=[2, 2])

    def nd(dtype=1, act=0):
        return lib.convtranspose_nd_fused(0, dtype, 2, 0, P, T._i64((1, 4, 5, 5)), P, T._i64((4, 2, 3, 3)), None, P,
                                          T._i64((1, 2, 11, 11)), *at, act, 0.0, 0.0, None, 0, None)

    assert nd(dtype=4) == 3 and nd(dtype=5) == 3 and nd(dtype=6) == 3 and nd(act=4) == 1


def test_tensors_are_checked(T):
    """The binding refuses what the kernels would read wrongly (host tensors stand for all)."""
    x = T.to_channels_last(torch.zeros(2, 8, 3, 3))
    for call in (lambda: T.group_norm_nd(x, 2), lambda: T.dropout_nd(x, 0.5, seed=1),
                 lambda: T.embedding_nd(torch.zeros(3, dtype=torch.int64), torch.zeros(4, 8)),
                 lambda: T.embedding_backward_nd(torch.zeros(3, 8), torch.zeros(3, dtype=torch.int64), 4),
                 lambda: T.group_norm_backward_nd(x, x, x, x, 2)):
        with pytest.raises(T.ConvTransposeError, match="HIP device"):
            call()
    for call in (lambda: T.group_norm_nd(x.double(), 2), lambda: T.dropout_nd(x.int(), 0.5, seed=1),
                 lambda: T.embedding_nd(torch.zeros(3, dtype=torch.int64), torch.zeros(4, 8).double()),
                 lambda: T.embedding_backward_nd(torch.zeros(3, 8).int(), torch.zeros(3, dtype=torch.int64), 4)):
        with pytest.raises(T.ConvTransposeError, match="not served"):
            call()
    assert T._storage_order(x) is not None and T._storage_order(x[:, :, 1:]) is None
    assert T._storage_order(torch.zeros(3, 1, 4).expand(3, 2, 4)) is None
    assert set(T.NORM_ACTIVATIONS) == set(T.ACTIVATIONS) | {"silu"}


def test_reference_generator_known_answers():
    """Published Philox4x32-10 vectors pin both generators the kernels are compared with."""
    m = 0xFFFFFFFF
    assert R.philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert R.philox([m] * 4, [m] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert R.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]
    seed, offset = 0x123456789ABCDEF0, 0xFEDCBA9876543210
    for first in (0, 8, (1 << 35) + 16):
        words = R.philox([first // 8 & m, first // 8 >> 32, offset & m, offset >> 32], [seed & m, seed >> 32])
        fields = [w >> s & 0xFFFF for w in words for s in (0, 16)]
        assert list(R.keep_mask(8, 0.5, seed, offset, first)) == [f >= 32768 for f in fields]

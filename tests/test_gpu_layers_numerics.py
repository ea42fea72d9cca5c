"""Group norm where float32 arithmetic can go wrong: values that are not finite, under every
activation, single values far from all others, and sums of many equal terms, whose roundings
all go the same way; and the embedding's gradient of narrow rows with very many tokens."""
import numpy as np
import pytest
import torch

import layer_refs as R
from test_gpu_layers import ACTS, T, host, norm_inputs, path, rows_of  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("kind,params", ACTS)
def test_a_diverged_group_is_seen(T, path, kind, params, bad):
    """One value that is not finite leaves its group without statistics: every output of the group
    is NaN under every activation, and so are its gradients, but dbeta of the identity, whose
    derivative depends on nothing.  The other groups and images keep their bits."""
    x, _, dy, _, ga, _, be, _ = norm_inputs(2, 32, (6, 5), "f16", "f32", 3)
    kw = dict(activation=kind, act_params=params)
    clean = T.group_norm_nd(x, 4, ga, be, **kw)
    grads = T.group_norm_backward_nd(dy, x, clean[1], clean[2], 4, ga, be, **kw)
    x = x.clone(memory_format=torch.preserve_format)
    x[1, 9, 2, 2] = float(bad)
    y, mean, rstd = T.group_norm_nd(x, 4, ga, be, **kw)
    dx, dgamma, dbeta = T.group_norm_backward_nd(dy, x, mean, rstd, 4, ga, be, **kw)
    assert torch.isnan(y[1, 8:16]).all()
    assert torch.isnan(dx[1, 8:16]).all() and torch.isnan(dgamma[8:16]).all()
    assert torch.equal(dbeta, grads[2]) if kind == "identity" else torch.isnan(dbeta[8:16]).all()
    for got, want in ((y, clean[0]), (dx, grads[0])):
        assert torch.equal(got[0], want[0])
        for part in (slice(0, 8), slice(16, 32)):
            assert torch.equal(got[1, part], want[1, part])
    for got, want in ((dgamma, grads[1]), (dbeta, grads[2])):
        for part in (slice(0, 8), slice(16, 32)):
            assert torch.equal(got[part], want[part])


@pytest.mark.parametrize("far", [1e3, -1e5])
@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("shape", [(2, 32, (9, 7), 4), (1, 12, (3001,), 2), (1, 256, (64, 64), 32), (1, 24, (20011,), 3),
                                   (2, 64, (4, 6, 5), 1), (1, 4104, (3, 3), 1), (2, 1001, (13,), 7), (5, 8, (129,), 2)])
def test_group_norm_one_value_far_from_the_others(T, path, shape, where, far):
    """Standard normals and one large value a group, the first or the last of it.

    The large value A leaves the group of n values a spread s of A / sqrt(n).  What it costs are
    roundings of A in the few values that are summed next to it, at most 2^-24 A a value, and
    those are few of the n: together less than 2^-24 s.  The mean of the group comes to a few
    2^-24 of itself and of s, and so does each x - mean."""
    n, c, dims, groups = shape
    rng = np.random.default_rng(17)
    xv = rng.normal(size=(n,) + dims + (c,)).astype(np.float32)
    by_group = xv.reshape(n, -1, groups, c // groups)
    by_group[:, 0 if where == "first" else -1, :, 0 if where == "first" else -1] = far
    x = torch.from_numpy(xv).cuda().movedim(-1, 1)
    y, mean, rstd = T.group_norm_nd(x, groups, eps=0.0)
    v = by_group.astype(np.float64)
    m, s = v.mean((1, 3)), v.std((1, 3))
    assert (np.abs(host(mean) - m) <= 4 * R.EPS * (np.abs(m) + s)).all(), np.abs(host(mean) - m).max()
    assert (np.abs(host(rstd) * s - 1) <= R.FACTOR * R.EPS).all()
    wide = lambda a: a[:, None, :, None]  # noqa: E731
    z = (v - wide(m)) / wide(s)
    bound = (8 * (1 + np.abs(wide(m)) / wide(s)) + R.FACTOR * np.abs(z)) * R.EPS
    assert (np.abs(rows_of(y).reshape(v.shape) - z) <= bound).all()


@pytest.mark.parametrize("n,c,dims,groups", [((1 << 21) + 5, 2, (2,), 1), (300001, 16, (3,), 4), (1, 4, (1 << 28,), 2),
                                             (600, 24, (60, 1000), 3)])
def test_parameter_gradients_of_a_constant_gradient(T, n, c, dims, groups):
    """dy = 0.1 everywhere and no activation: dbeta is 0.1 times the number of positions, to the
    roundings of a sum in a tree.  One sum of 2^17 terms after another would be off by hundreds
    of times that."""
    print(f"[case] constant gradient {(n, c, dims)} f32", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((n,) + dims + (c,), generator=gen, device="cuda").movedim(-1, 1)
    dy = torch.full_like(x, 0.1)
    gamma = torch.ones(c, device="cuda")
    _, mean, rstd = T.group_norm_nd(x, groups, gamma, gamma)
    _, dgamma, dbeta = T.group_norm_backward_nd(dy, x, mean, rstd, groups, gamma, gamma, out=dy)
    want = float(np.float32(0.1)) * n * int(np.prod(dims))
    print(f"dbeta off by {np.abs(host(dbeta) / want - 1).max() / R.EPS:.1f} roundings", flush=True)
    assert (np.abs(host(dbeta) - want) <= R.FACTOR * R.EPS * want).all()
    # the sums of 0.1 xhat by group vanish, and those by channel are small beside the terms'
    # magnitudes, 0.1 sqrt(2 / pi) on average
    by_group = host(dgamma).reshape(groups, -1).sum(1)
    assert (np.abs(by_group) <= R.FACTOR * R.EPS * want * (c // groups)).all()


@pytest.mark.parametrize("tokens,rows,width", [(6225, 90, 1), (3003, 6, 1), (22634, 19, 2), (29915, 63, 18), (70001, 2, 3),
                                               (40000, 1, 9), (5000, 300, 130)])
def test_embedding_gradient_of_frequent_narrow_rows(T, tokens, rows, width):
    """A row's partial sums are shared out over up to 256 groups of lanes, some without a share: whole
    numbers, so every partial sum is counted exactly once."""
    rng = np.random.default_rng(tokens)
    ids = np.minimum((rows + 1) ** rng.random(tokens) - 1, rows - 1).astype(np.int64)
    dy = rng.integers(-2, 3, size=(tokens, width)).astype(np.float64)
    want, _ = R.embedding_grad(dy, ids, rows, 1.0)
    for dtype in (torch.float32, torch.bfloat16):
        d = torch.from_numpy(dy).to(dtype).cuda()
        got = T.embedding_backward_nd(d, torch.from_numpy(ids).cuda(), rows, grad_dtype=torch.float32)
        assert np.array_equal(host(got), want), dtype

"""Group norm with an activation, dropout and the embedding on the GPU against plain 64-bit
forms (layer_refs): values at every element within bounds derived from the kernels'
float32 arithmetic, masks and selections exactly."""
import numpy as np
import pytest
import torch

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


def rows_of(t):
    """A logical (N, C, D..) tensor as the float64 array (N, P, C)."""
    return host(t.movedim(1, -1).reshape(t.shape[0], -1, t.shape[1]))


@pytest.fixture(params=["automatic", "two_passes", "joined_between"])
def path(T, request):
    """How group norm is computed: by its own choice, or always in two passes, the partial sums
    joined in the second one or between them."""
    T.set_group_norm_control(request.param == "automatic", {"two_passes": False, "joined_between": True}.get(request.param))
    yield request.param
    T.set_group_norm_control()


def norm_inputs(n, c, dims, dtype, params, seed, mean=0.5, spread=1.0):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(n,) + dims + (c,)) * spread * rng.uniform(0.5, 1.5, c) + mean * rng.normal(size=c)
    tx, x = dev(x, dtype)
    ga, gav = dev(1.0 + 0.3 * rng.normal(size=c), params)
    be, bev = dev(0.3 * rng.normal(size=c), params)
    tdy, dy = dev(rng.normal(size=x.shape), dtype)
    flat = lambda a: a.reshape(n, -1, c)  # noqa: E731
    return tx.movedim(-1, 1), flat(x), tdy.movedim(-1, 1), flat(dy), ga, gav, be, bev


# every kind of cut: single values, vectors that run over a row's end, channel counts no vector
# divides, several slabs, groups that cross slabs, many chunks
SHAPES = [
    (1, 1, (1,), 1), (1, 8, (1,), 1), (2, 6, (5,), 3), (3, 4, (1, 2), 4), (2, 36, (7, 9), 4), (1, 256, (8, 8), 32),
    (3, 320, (31,), 32), (2, 64, (4, 6, 5), 16), (2, 33, (1000,), 3), (1, 24, (20011,), 3), (5, 8, (129,), 8),
    (1, 2112, (7,), 4), (2, 4096, (5,), 2), (1, 4104, (3, 3), 1), (2, 1001, (13,), 7), (1, 300, (257,), 300),
    (1, 1030, (11,), 5), (2, 128, (33, 65), 32), (17, 16, (3, 5), 2), (1, 512, (64, 64), 32),
]
ACTS = [("silu", ()), ("identity", ()), ("relu", ()), ("leaky_relu", (0.2,)), ("clip", (-0.5, 0.75))]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_group_norm(T, path, case, dtype):
    n, c, dims, groups = SHAPES[case]
    kind, params = ACTS[case % len(ACTS)]
    p = (0.0, 0.3)[case % 2]
    ptype = "f32" if case % 3 else dtype
    print(f"[case] group_norm {SHAPES[case]} {dtype} {kind} p={p} params {ptype} {path}", flush=True)
    x, xv, _, _, ga, gav, be, bev = norm_inputs(n, c, dims, dtype, ptype, case)
    seed, offset = 0x9E3779B97F4A7C15, (7 << 40) + case
    y, mean, rstd = T.group_norm_nd(x, groups, ga, be, activation=kind, act_params=params, dropout_p=p, seed=seed,
                                    offset=offset)
    torch.cuda.synchronize()
    want, tol = R.group_norm(xv, groups, gav, bev, 1e-5, kind, params, p, seed, offset)
    assert y.shape == x.shape and y.stride() == T.channels_last_empty(x.shape, x.dtype, x.device).stride()
    R.assert_close(rows_of(y), want[0], tol[0], dtype, "y")
    R.assert_close(host(mean), want[1], tol[1], "f32", "mean")
    R.assert_close(host(rstd), want[2], tol[2], "f32", "rstd")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_group_norm_gradient(T, path, case, dtype):
    n, c, dims, groups = SHAPES[case]
    kind, params = ACTS[(case + 2) % len(ACTS)]
    p = (0.3, 0.0)[case % 2]
    ptype = dtype if case % 3 else "f32"
    print(f"[case] group_norm gradient {SHAPES[case]} {dtype} {kind} p={p} params {ptype} {path}", flush=True)
    x, xv, dy, dyv, ga, gav, be, bev = norm_inputs(n, c, dims, dtype, ptype, 100 + case)
    (_, mean, rstd), _ = R.group_norm(xv, groups, gav, bev, 1e-5, "identity")
    mean, rstd = (torch.from_numpy(a).float().cuda() for a in (mean, rstd))
    # a value at a kink of the activation may fall on either side of it: none is there
    xhat = (xv - np.repeat(host(mean), c // groups, 1)[:, None]) * np.repeat(host(rstd), c // groups, 1)[:, None]
    z = xhat * gav + bev
    kinks = {"relu": [0.0], "leaky_relu": [0.0], "clip": list(params)}.get(kind, [])
    for q in kinks:
        near = np.abs(z - q) < 1e-4
        dyv[near] = 0.0
    dy = torch.from_numpy(dyv.reshape((n,) + dims + (c,))).to(DT[dtype]).cuda().movedim(-1, 1)
    seed, offset = 12345, case
    dx, dgamma, dbeta = T.group_norm_backward_nd(dy, x, mean, rstd, groups, ga, be, activation=kind, act_params=params,
                                                 dropout_p=p, seed=seed, offset=offset)
    torch.cuda.synchronize()
    want, tol = R.group_norm_grad(dyv, xv, host(mean), host(rstd), groups, gav, bev, kind, params, p, seed, offset)
    R.assert_close(rows_of(dx), want[0], tol[0], dtype, "dx")
    R.assert_close(host(dgamma), want[1], tol[1], ptype, "dgamma")
    R.assert_close(host(dbeta), want[2], tol[2], ptype, "dbeta")


@pytest.mark.parametrize("given", ["gamma", "beta", "none"])
def test_group_norm_absent_parameters(T, given):
    x, xv, dy, dyv, ga, gav, be, bev = norm_inputs(2, 24, (9, 5), "f16", "f32", 5)
    ga, gav = (ga, gav) if given == "gamma" else (None, None)
    be, bev = (be, bev) if given == "beta" else (None, None)
    y, mean, rstd = T.group_norm_nd(x, 3, ga, be, eps=1e-3, activation="silu")
    want, tol = R.group_norm(xv, 3, gav, bev, 1e-3, "silu")
    R.assert_close(rows_of(y), want[0], tol[0], "f16", "y")
    dx, dgamma, dbeta = T.group_norm_backward_nd(dy, x, mean, rstd, 3, ga, be, activation="silu")
    assert (dgamma is None) == (ga is None) and (dbeta is None) == (be is None)
    want, tol = R.group_norm_grad(dyv, xv, host(mean), host(rstd), 3, gav, bev, "silu")
    R.assert_close(rows_of(dx), want[0], tol[0], "f16", "dx")
    for got, w, t in ((dgamma, want[1], tol[1]), (dbeta, want[2], tol[2])):
        if got is not None:
            R.assert_close(host(got), w, t, "f32", "parameter gradient")


@pytest.mark.parametrize("shape", [(2, 32, (9, 7), 4), (1, 12, (3001,), 2), (1, 256, (64, 64), 32)])
def test_group_norm_mean_far_from_zero(T, path, shape):
    """Values of spread 1 around 4096: the variance is not a difference of large sums."""
    n, c, dims, groups = shape
    x, xv, _, _, ga, gav, be, bev = norm_inputs(n, c, dims, "f32", "f32", 9, mean=0.0)
    x = x + 4096.0
    xv = rows_of(x)
    y, mean, rstd = T.group_norm_nd(x, groups, ga, be)
    want, tol = R.group_norm(xv, groups, gav, bev, 1e-5, "identity")
    # the values themselves are exact; the mean may be off by a few roundings of 4096
    assert np.abs(host(mean) - want[1]).max() <= 4 * 2.0 ** -24 * 4200
    assert np.abs(host(rstd) / want[2] - 1).max() <= 2e-5
    R.assert_close(rows_of(y), want[0], tol[0], "f32", "y")


def test_group_norm_constant_and_non_finite_groups(T, path):
    """A constant group gives beta; NaN and infinities stay inside their own group and image."""
    x, xv, _, _, ga, gav, be, bev = norm_inputs(2, 32, (6, 5), "f16", "f32", 3)
    x = x.clone(memory_format=torch.preserve_format)
    x[0, 0:8] = 3.0
    clean, _, _ = T.group_norm_nd(x, 4, ga, be)
    assert torch.equal(clean[0, 0:8], be[:8].half()[:, None, None].expand_as(clean[0, 0:8]))
    x[1, 9, 2, 2] = float("nan")
    x[1, 17, 1, 1] = float("inf")
    y, mean, rstd = T.group_norm_nd(x, 4, ga, be)
    assert torch.equal(y[0], clean[0]) and torch.equal(y[1, 0:8], clean[1, 0:8]) and torch.equal(y[1, 24:], clean[1, 24:])
    assert torch.isnan(y[1, 8:16]).all() and not torch.isfinite(y[1, 16:24]).any()
    assert torch.isnan(rstd[1, 1]) and not torch.isfinite(mean[1, 2])


def test_group_norm_unaligned_storage_in_place_and_streams(T):
    n, c, dims, groups = 2, 40, (17, 3), 5
    x, xv, dy, dyv, ga, gav, be, bev = norm_inputs(n, c, dims, "f16", "f16", 8)
    want = [t.clone() for t in T.group_norm_nd(x, groups, ga, be, activation="silu", dropout_p=0.2, seed=5)]
    grads = [t.clone() for t in T.group_norm_backward_nd(dy, x, want[1], want[2], groups, ga, be, activation="silu",
                                                         dropout_p=0.2, seed=5)]

    def shifted(t, by):
        """A channels-last copy whose storage starts `by` elements off a 16-byte boundary."""
        flat = torch.empty(t.numel() + 16, dtype=t.dtype, device=t.device)
        v = flat[by:by + t.numel()].view((n,) + dims + (c,))
        v.copy_(t.movedim(1, -1))
        return v.movedim(-1, 1)

    side = torch.cuda.Stream()
    for by in (1, 3, 4):
        xs, out = shifted(x, by), shifted(torch.zeros_like(x), by + 1)
        gs, bs = torch.cat([ga[:1], ga])[1:], torch.cat([be[:1], be])[1:]
        side.wait_stream(torch.cuda.current_stream())
        y, mean, rstd = T.group_norm_nd(xs, groups, gs, bs, activation="silu", dropout_p=0.2, seed=5, out=out, stream=side)
        dx, dg, db = T.group_norm_backward_nd(shifted(dy, by), xs, want[1], want[2], groups, gs, bs, activation="silu",
                                              dropout_p=0.2, seed=5)
        torch.cuda.synchronize()
        assert y is out
        for got, w in ((y, want[0]), (mean, want[1]), (rstd, want[2]), (dx, grads[0]), (dg, grads[1]), (db, grads[2])):
            assert torch.equal(got, w)
    for into in ("dy", "x"):
        xs, ds = shifted(x, 0), shifted(dy, 0)
        dx, dg, db = T.group_norm_backward_nd(ds, xs, want[1], want[2], groups, ga, be, activation="silu", dropout_p=0.2,
                                              seed=5, out=ds if into == "dy" else xs)
        assert dx is (ds if into == "dy" else xs)
        assert torch.equal(dx, grads[0]) and torch.equal(dg, grads[1]) and torch.equal(db, grads[2])
    xs = shifted(x, 0)
    y, _, _ = T.group_norm_nd(xs, groups, ga, be, activation="silu", dropout_p=0.2, seed=5, out=xs)
    assert torch.equal(xs, want[0])


@pytest.mark.parametrize("shape", [(2, 16, (6, 7), 4), (1, 64, (33, 31), 8)])
def test_group_norm_gradient_against_differences(T, path, shape):
    """The directional derivative of sum(w y) by central differences of the forward call."""
    n, c, dims, groups = shape
    x, _, w, wv, ga, _, be, _ = norm_inputs(n, c, dims, "f32", "f32", 77)
    kw = dict(activation="silu", dropout_p=0.25, seed=3, offset=11)
    value = lambda a, g, b: float((T.group_norm_nd(a, groups, g, b, **kw)[0].double() * w.double()).sum())  # noqa: E731
    _, mean, rstd = T.group_norm_nd(x, groups, ga, be, **kw)
    grads = T.group_norm_backward_nd(w, x, mean, rstd, groups, ga, be, **kw)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for k, grad in enumerate(grads):
        args = [x, ga, be]
        u = torch.randn(args[k].shape, generator=gen, device="cuda") if k else torch.randn(
            x.movedim(1, -1).shape, generator=gen, device="cuda").movedim(-1, 1)
        h = 2.0 ** -7
        up, down = list(args), list(args)
        up[k], down[k] = args[k] + h * u, args[k] - h * u
        slope = (value(*up) - value(*down)) / (2 * h)
        want = float((grad.double() * u.double()).sum())
        # h^2/6 of a third derivative of order |w| per element, and float32 sums over 2 h
        count = x.numel()
        bound = 4 * h * h * count ** 0.5 + 2.0 ** -20 * count ** 0.5 / h
        assert abs(slope - want) <= bound, (k, slope, want, bound)


def test_group_norm_repeats_its_bits(T, path):
    for shape in ((1, 256, (64, 64), 32), (2, 36, (90, 91), 4), (3, 64, (17, 33, 20), 16)):
        n, c, dims, groups = shape
        x, _, dy, _, ga, _, be, _ = norm_inputs(n, c, dims, "f16", "f32", 13)
        kw = dict(activation="silu", dropout_p=0.1, seed=4)

        def both():
            y, mean, rstd = T.group_norm_nd(x, groups, ga, be, **kw)
            return [y, mean, rstd, *T.group_norm_backward_nd(dy, x, mean, rstd, groups, ga, be, **kw)]

        want = both()
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(both(), want)), shape


def test_group_norm_empty(T):
    for shape in ((0, 8, 3, 3), (2, 8, 0, 3)):
        x = T.channels_last_empty(shape, torch.float16, "cuda")
        ga, be = torch.ones(8, device="cuda"), torch.ones(8, device="cuda")
        y, mean, rstd = T.group_norm_nd(x, 2, ga, be)
        assert y.shape == x.shape and mean.shape == (shape[0], 2)
        dx, dg, db = T.group_norm_backward_nd(x, x, mean, rstd, 2, ga, be)
        assert not dg.any() and not db.any()


# ------------------------------------------------------------------------------------
# dropout
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("count", [1, 2, 7, 8, 9, 255, 2048, 2049, 100003])
def test_dropout(T, count, dtype):
    rng = np.random.default_rng(count)
    x, xv = dev(rng.normal(size=count), dtype)
    r, rv = dev(rng.normal(size=count), dtype)
    for p, seed, offset in ((0.1, 1, 0), (0.5, (1 << 64) - 3, (1 << 64) - 1), (1 / 65536, 9, 1 << 33), (0.999, 7, 7)):
        want = R.drop(xv, p, seed, offset)
        y = T.dropout_nd(x, p, seed=seed, offset=offset)
        R.assert_close(host(y), want, 2 * R.EPS * np.abs(want), dtype, "y")
        assert np.array_equal(host(y) == 0, want == 0)
        y = T.dropout_nd(x, p, seed=seed, offset=offset, residual=r)
        R.assert_close(host(y), want + rv, 4 * R.EPS * (np.abs(want) + np.abs(rv)), dtype, "y with residual")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_one_rounding_to_nearest_even(T, dtype):
    """x + residual in float32 and one rounding: torch's conversion of the same sum, bit for bit."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, r = (torch.randn(4099, generator=gen, device="cuda").to(DT[dtype]) for _ in range(2))
    assert torch.equal(T.dropout_nd(x, 0.0, seed=0, residual=r), (x.float() + r.float()).to(DT[dtype]))


def test_dropout_none_all_and_non_finite(T):
    x = torch.randn(1000, device="cuda", dtype=torch.float16)
    assert torch.equal(T.dropout_nd(x, 0.0, seed=1), x)
    assert torch.equal(T.dropout_nd(x, 2.0 ** -18, seed=1), x)  # below the smallest step
    x[::3] = float("nan")
    x[1::3] = float("inf")
    assert not T.dropout_nd(x, 1.0, seed=1).any()
    y = T.dropout_nd(x, 0.5, seed=4)
    keep = torch.from_numpy(R.keep_mask(1000, 0.5, 4, 0)).cuda()
    assert torch.equal(y == 0, ~keep)
    z = T.dropout_nd(x, 1.0, seed=1, residual=torch.ones_like(x))
    assert torch.equal(z, torch.ones_like(x))


def test_dropout_is_its_own_gradient_and_keeps_the_mean(T):
    """y = D x with D diagonal: <D x, w> = <x, D w>, and the share that stays is 1 - p."""
    x, w = torch.randn(1 << 20, device="cuda"), torch.randn(1 << 20, device="cuda")
    kw = dict(seed=21, offset=5)
    a = (T.dropout_nd(x, 0.3, **kw).double() * w).sum()
    b = (x.double() * T.dropout_nd(w, 0.3, **kw)).sum()
    assert abs(float(a - b)) <= 1e-5 * float((x.double() * w).abs().sum())
    ones = T.dropout_nd(torch.ones_like(x), 0.3, **kw)
    n, q = x.numel(), R.threshold(0.3) / 65536
    assert abs(float((ones > 0).float().mean()) - (1 - q)) <= 6 * (q * (1 - q) / n) ** 0.5
    other = T.dropout_nd(torch.ones_like(x), 0.3, seed=21, offset=6)
    both = float(((ones > 0) & (other > 0)).float().mean())
    assert abs(both - (1 - q) ** 2) <= 6 / n ** 0.5  # another offset: independent


def test_dropout_storage_order_in_place_and_step(T):
    x = T.to_channels_last(torch.randn(2, 24, 5, 7, device="cuda"))
    y = T.dropout_nd(x, 0.4, seed=3, offset=1 << 40)
    flat = x.permute(0, 2, 3, 1).reshape(-1)
    want = T.dropout_nd(flat, 0.4, seed=3, offset=1 << 40)
    assert y.stride() == x.stride() and torch.equal(y.permute(0, 2, 3, 1).reshape(-1), want)
    step = torch.tensor([5], device="cuda")
    assert torch.equal(T.dropout_nd(flat, 0.4, seed=3, offset=(1 << 40) - 5, step=step), want)
    res = torch.randn_like(flat)
    both = T.dropout_nd(flat, 0.4, seed=3, offset=1 << 40, residual=res)
    r = res.clone()
    assert T.dropout_nd(flat, 0.4, seed=3, offset=1 << 40, residual=r, out=r) is r and torch.equal(r, both)
    f = flat.clone()
    T.dropout_nd(f, 0.4, seed=3, offset=1 << 40, out=f)
    assert torch.equal(f, want)
    g = torch.cat([flat[:1], flat])[1:]  # storage off a 16-byte boundary
    assert torch.equal(T.dropout_nd(g, 0.4, seed=3, offset=1 << 40), want)


# ------------------------------------------------------------------------------------
# embedding
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 9, 512), (5, 3, 3), (300, 17, 77), (64, 1000, 8), (7, 5, 1024),
                                   (3, 4, 2500), (4097, 50, 31)])
def test_embedding(T, shape, dtype):
    tokens, rows, width = shape
    rng = np.random.default_rng(sum(shape))
    table, tv = dev(rng.normal(size=(rows, width)), dtype)
    ids = rng.integers(-2, rows + 2, size=tokens)
    ids[0] = rows - 1
    ok = (ids >= 0) & (ids < rows)
    want = np.where(ok[:, None], tv[np.clip(ids, 0, rows - 1)] * np.float64(np.float32(1.7)), 0.0)
    for it in (torch.int32, torch.int64):
        y = T.embedding_nd(torch.from_numpy(ids).to(it).cuda(), table, scale=1.7)
        R.assert_close(host(y), want, R.EPS * np.abs(want), dtype, "y")
    grid = torch.from_numpy(ids).cuda().reshape(1, 1, tokens)
    y2 = T.embedding_nd(grid, table, scale=1.7)
    assert y2.shape == (1, 1, tokens, width) and torch.equal(y2.reshape(tokens, width), y)


def _ids(kind, tokens, rows, rng):
    if kind == "one":
        return np.full(tokens, rows // 2)
    if kind == "skewed":
        return np.minimum((rows + 1) ** rng.random(tokens) - 1, rows - 1).astype(np.int64)
    if kind == "sorted":
        return np.sort(rng.integers(0, rows, tokens))
    return rng.integers(-1, rows + 1, tokens)


GRADS = [
    (1, 1, 1, "any"), (1, 300, 5, "any"), (64, 2, 8, "any"), (65, 255, 16, "any"), (257, 1025, 77, "any"),
    (5000, 3, 40, "skewed"), (5000, 70000, 9, "any"), (4097, 256, 512, "skewed"), (3000, 10, 64, "one"),
    (20000, 500, 24, "skewed"), (8192, 64, 33, "sorted"), (1024, 1 << 17, 4, "skewed"), (70000, 40, 3, "any"),
    (300000, 9, 1, "skewed"), (200, 7, 3000, "skewed"),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", range(len(GRADS)))
def test_embedding_gradient(T, case, dtype):
    tokens, rows, width, kind = GRADS[case]
    print(f"[case] embedding gradient {GRADS[case]} {dtype}", flush=True)
    rng = np.random.default_rng(1000 + case)
    dy, dv = dev(rng.normal(size=(tokens, width)), dtype)
    ids = _ids(kind, tokens, rows, rng)
    padding = None if case % 2 else int(ids[-1]) if 0 <= ids[-1] < rows else 0
    gt = dtype if case % 3 else "f32"
    ti = torch.from_numpy(ids).cuda().to(torch.int32 if case % 2 else torch.int64)
    got = T.embedding_backward_nd(dy, ti, rows, scale=0.5, padding_idx=padding, grad_dtype=DT[gt])
    want, mag = R.embedding_grad(dv, ids, rows, 0.5, padding)
    # tokens one after another within a chunk, then the chunks: at most the longest run of both
    n = max(64, int(2 * tokens ** 0.5) + 2)
    R.assert_close(host(got), want, R.EPS * min(n, 4096) * mag, gt, "gradient")
    again = T.embedding_backward_nd(dy, ti, rows, scale=0.5, padding_idx=padding, grad_dtype=DT[gt])
    assert torch.equal(again, got)  # a fixed order


def test_embedding_gradient_sums_in_token_order(T):
    """Small whole numbers: sums are exact, so every token is counted exactly once."""
    rng = np.random.default_rng(2)
    ids = np.minimum(1001 ** rng.random(30000) - 1, 999).astype(np.int64)
    dy = rng.integers(-2, 3, size=(30000, 20)).astype(np.float64)
    want, _ = R.embedding_grad(dy, ids, 1000, 1.0)
    got = T.embedding_backward_nd(torch.from_numpy(dy).float().cuda(), torch.from_numpy(ids).cuda(), 1000)
    assert np.array_equal(host(got), want)


@pytest.mark.parametrize("tokens,rows,width,top", [
    (513, 20000, 260, 3), (4096, 9000, 512, 9000), (5000, 50, 1030, 50), (9000, 40000, 8, 900), (2000, 30000, 300, 1),
    (20000, 5, 100, 5),
])
def test_embedding_gradient_of_tokens_without_a_row(T, tokens, rows, width, top):
    """Sums of small whole numbers are exact, and what padding or an id outside the table has for a
    gradient (NaN here) goes nowhere; rows without tokens, the last ones too, are zeros."""
    rng = np.random.default_rng(tokens)
    ids = np.minimum((top + 1) ** rng.random(tokens) - 1, top - 1).astype(np.int64)
    ids[rng.random(tokens) < 0.2] = -5
    ids[rng.random(tokens) < 0.2] = rows
    padding = top // 2
    dy = rng.integers(-2, 3, size=(tokens, width)).astype(np.float64)
    none = (ids < 0) | (ids >= rows) | (ids == padding)
    want, _ = R.embedding_grad(np.where(none[:, None], 0.0, dy), ids, rows, 1.0, padding)
    dy[none] = np.nan
    for dtype in ("f32", "f16"):
        d = torch.from_numpy(dy).to(DT[dtype]).cuda()
        got = T.embedding_backward_nd(d, torch.from_numpy(ids).cuda(), rows, padding_idx=padding, grad_dtype=DT["f32"])
        assert np.array_equal(host(got), want), dtype


def test_embedding_gradient_against_differences(T):
    """The lookup is linear: sum(w y(table + h u)) changes by h <gradient, u> exactly."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.randint(0, 50, (700,), generator=gen, device="cuda")
    table, u = (torch.randn((50, 24), generator=gen, device="cuda") for _ in range(2))
    w = torch.randn((700, 24), generator=gen, device="cuda")
    value = lambda t: float((T.embedding_nd(ids, t, scale=3.0).double() * w.double()).sum())  # noqa: E731
    slope = (value(table + u) - value(table - u)) / 2
    grad = T.embedding_backward_nd(w, ids, 50, scale=3.0)
    want = float((grad.double() * u.double()).sum())
    assert abs(slope - want) <= 2.0 ** -18 * 3.0 * float(w.abs().sum())


def test_embedding_empty(T):
    table = torch.randn(5, 8, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert T.embedding_nd(none, table).shape == (0, 8)
    out = torch.full((5, 8), 3.0, device="cuda")
    assert not T.embedding_backward_nd(torch.empty(0, 8, device="cuda"), none, 5, out=out).any()
    ids = torch.tensor([0, 3], device="cuda")
    assert not T.embedding_nd(ids, torch.empty(0, 8, device="cuda")).any()  # no rows: every id is outside
    assert T.embedding_backward_nd(torch.ones(2, 8, device="cuda"), ids, 0).shape == (0, 8)


# ------------------------------------------------------------------------------------
# prepared and captured calls
# ------------------------------------------------------------------------------------
def test_prepared_and_captured_calls(T):
    """Prepared calls repeat the direct call's bits, alone and replayed from a captured graph
    with a step that counts up between eager work."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    ids = torch.randint(0, 100, (2, 9, 11), generator=gen, device="cuda")
    table = torch.randn((100, 64), generator=gen, device="cuda").half()
    ga, be = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    kw = dict(activation="silu", dropout_p=0.3, seed=8, step=step)
    look = T.PreparedCall(T.embedding_nd, ids, table, scale=8.0)
    x = look.out.movedim(-1, 1)
    norm = T.PreparedCall(T.group_norm_nd, x, 8, ga, be, **kw)
    y, mean, rstd = norm.out
    res = T.PreparedCall(T.dropout_nd, y, 0.2, seed=9, step=step, residual=x)
    grad = T.PreparedCall(T.group_norm_backward_nd, res.out, x, mean, rstd, 8, ga, be, **kw)
    dx = grad.out[0].movedim(1, -1)
    emb = T.PreparedCall(T.embedding_backward_nd, dx, ids, 100, scale=8.0)
    calls = (look, norm, res, grad, emb)

    def eager():
        x = T.embedding_nd(ids, table, scale=8.0).movedim(-1, 1)
        y, mean, rstd = T.group_norm_nd(x, 8, ga, be, **kw)
        r = T.dropout_nd(y, 0.2, seed=9, step=step, residual=x)
        g = T.group_norm_backward_nd(r, x, mean, rstd, 8, ga, be, **kw)
        return [y, mean, rstd, r, *g, T.embedding_backward_nd(g[0].movedim(1, -1).contiguous(), ids, 100, scale=8.0)]

    def outputs():
        return [*norm.out, res.out, *grad.out, emb.out]

    for c in calls:
        c()
    torch.cuda.synchronize()
    for got, want in zip(outputs(), eager()):
        assert torch.equal(got, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        look = T.PreparedCall(T.embedding_nd, ids, table, scale=8.0, out=look.out)
        norm = T.PreparedCall(T.group_norm_nd, x, 8, ga, be, **kw)
        y, mean, rstd = norm.out
        res = T.PreparedCall(T.dropout_nd, y, 0.2, seed=9, step=step, residual=x)
        grad = T.PreparedCall(T.group_norm_backward_nd, res.out, x, mean, rstd, 8, ga, be, **kw)
        emb = T.PreparedCall(T.embedding_backward_nd, grad.out[0].movedim(1, -1), ids, 100, scale=8.0)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            for c in (look, norm, res, grad, emb):
                c()
    torch.cuda.synchronize()
    seen = []
    for k in range(4):
        step.fill_(k)
        for t in outputs():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = eager()
        torch.cuda.synchronize()
        for got, w in zip(outputs(), want):
            assert torch.equal(got, w), k
        seen.append(outputs()[0].clone())
    assert not torch.equal(seen[0], seen[1])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape,groups", [((2, 16, 10, 9), 4), ((1, 24, 40000), 3), ((2, 9, 77), 3)])
def test_dropped_gradients_may_be_anything(T, shape, groups, dtype):
    """A value of dy that dropout hides adds nothing, infinite or NaN: the gradients are those of 0."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    store = (shape[0],) + shape[2:] + (shape[1],)
    x, dy = (torch.randn(store, generator=gen, device="cuda").to(DT[dtype]).movedim(-1, 1) for _ in range(2))
    gamma = torch.rand(shape[1], generator=gen, device="cuda") + 0.5
    kw = dict(activation="silu", dropout_p=0.3, seed=11, offset=5)
    _, mean, rstd = T.group_norm_nd(x, groups, gamma, gamma, **kw)
    keep = torch.from_numpy(R.keep_mask(x.numel(), 0.3, 11, 5)).cuda().reshape(store).movedim(-1, 1)
    zero, bad = torch.where(keep, dy, 0), torch.where(keep, dy, float("nan"))
    bad[0, 0] = torch.where(keep[0, 0], dy[0, 0], float("-inf"))
    want = T.group_norm_backward_nd(zero, x, mean, rstd, groups, gamma, gamma, **kw)
    got = T.group_norm_backward_nd(bad, x, mean, rstd, groups, gamma, gamma, **kw)
    for w, g in zip(want, got):
        assert torch.isfinite(w).all() and torch.equal(w, g)


def test_offsets_beyond_32_bits(T):
    """Tensors of more than 2^31 elements: the last elements are read, drawn and written."""
    n = (1 << 31) + 40
    x = torch.zeros(n, dtype=torch.float16, device="cuda")
    x[-40:] = torch.arange(1, 41, device="cuda")
    y = T.dropout_nd(x, 0.5, seed=1)
    keep = R.keep_mask(40, 0.5, 1, 0, first=n - 40)
    assert np.array_equal(host(y[-40:]), np.where(keep, 2.0 * np.arange(1, 41), 0.0))
    del y
    # a table of that size: its last row, looked up and given a gradient
    table, rows = x.view(-1, 8), n // 8
    ids = torch.tensor([rows - 1, 0, rows], device="cuda")
    got = T.embedding_nd(ids, table)
    assert torch.equal(got[0], table[-1]) and not got[1:].any()
    grad = T.embedding_backward_nd(torch.ones(3, 8, dtype=torch.float16, device="cuda"), ids, rows)
    assert bool((grad[-1] == 1).all()) and bool((grad[0] == 1).all()) and float(grad.sum(dtype=torch.float64)) == 16
    del grad, got, table
    # one image of that many values: 0 but for the last positions of each group
    xs = x.view(1, n // 8, 8).movedim(-1, 1)
    y, mean, rstd = T.group_norm_nd(xs, 2)
    v = host(xs[0, :, -5:])
    for g in range(2):
        part = v[4 * g:4 * g + 4]
        m = part.sum() / (n / 2)
        var = (part ** 2).sum() / (n / 2) - m * m
        r = 1 / np.sqrt(var + 1e-5)
        assert abs(float(mean[0, g]) - m) <= 1e-5 * abs(m) and abs(float(rstd[0, g]) / r - 1) <= 1e-5
        want = (part - m) * r
        assert np.abs(host(y[0, 4 * g:4 * g + 4, -5:]) - want).max() <= 2.0 ** -10 * np.abs(want).max()
    dx, _, _ = T.group_norm_backward_nd(xs, xs, mean, rstd, 2)
    xhat = (v[:4] - float(mean[0, 0])) * float(rstd[0, 0])
    c1, c2 = v[:4].sum() / (n / 2), (v[:4] * xhat).sum() / (n / 2)
    want = float(rstd[0, 0]) * (v[:4] - c1 - xhat * c2)
    assert np.abs(host(dx[0, :4, -5:]) - want).max() <= 2.0 ** -10 * np.abs(want).max() + 1e-3

"""Plain 64-bit forms of group norm, dropout and the embedding, for the tests of the kernels.

The bounds are what the kernels' arithmetic allows, from its float32 operations: EPS is one
float32 rounding; a sum of n values joined in a tree costs a few roundings of the sum of
their magnitudes, for which 32 are allowed; the one rounding to the result's type costs
half a unit in its last place.
"""
import numpy as np

EPS = 2.0 ** -24
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # 24, 11 and 8 significant bits
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half the smallest step
FACTOR = 32


def threshold(p):
    return int(np.floor(p * 65536 + 0.5))


def philox(counter, key):
    """Philox4x32-10 of one counter (4 words) under one key (2 words), in Python integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep_mask(count, p, seed, offset, first=0):
    """Which of the elements first .. first + count - 1 stay (first a multiple of 8)."""
    n = (count + 7) // 8
    m = np.uint64(0xFFFFFFFF)
    i = np.arange(n, dtype=np.uint64) + np.uint64(first // 8)
    a, b = i & m, i >> np.uint64(32)
    c, d = np.full(n, offset & 0xFFFFFFFF, np.uint64), np.full(n, offset >> 32, np.uint64)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        e, f = a * np.uint64(0xD2511F53), c * np.uint64(0xCD9E8D57)
        a, b, c, d = ((f >> np.uint64(32)) ^ b ^ np.uint64(k0), f & m, (e >> np.uint64(32)) ^ d ^ np.uint64(k1), e & m)
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    fields = np.stack([a, b, c, d], 1).astype("<u4").view("<u2").reshape(-1)[:count]
    return fields.astype(np.int64) >= threshold(p)


def drop(v, p, seed, offset):
    """Dropout of an array whose elements are numbered in its own order."""
    if p == 0.0:
        return v
    t = threshold(p)
    factor = 0.0 if t == 65536 else 65536.0 / (65536 - t)
    return np.where(keep_mask(v.size, p, seed, offset).reshape(v.shape), v * factor, 0.0)


def act(z, kind, params=()):
    if kind == "identity":
        return z
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "leaky_relu":
        return np.where(z >= 0, z, params[0] * z)
    if kind == "clip":
        return np.clip(z, *params)
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z))


def act_grad(z, kind, params=()):
    if kind == "identity":
        return np.ones_like(z)
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "leaky_relu":
        return np.where(z >= 0, 1.0, params[0])
    if kind == "clip":
        return ((z >= params[0]) & (z <= params[1])).astype(np.float64)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-z))
    return s + z * s * (1.0 - s)


def group_norm(x, groups, gamma, beta, eps, kind, params=(), p=0.0, seed=0, offset=0):
    """x (N, P, C) float64.  Returns y, mean, rstd and a bound on the float32 error of each."""
    N, P, C = x.shape
    cg = C // groups
    v = x.reshape(N, P, groups, cg)
    mean = v.mean((1, 3))
    var = ((v - mean[:, None, :, None]) ** 2).mean((1, 3))
    rstd = 1.0 / np.sqrt(var + eps)
    ga = np.ones(C) if gamma is None else gamma
    be = np.zeros(C) if beta is None else beta
    a = (np.repeat(rstd, cg, 1) * ga)[:, None, :]
    z = (x - np.repeat(mean, cg, 1)[:, None, :]) * a + be
    y = drop(act(z, kind, params), p, seed, offset)
    big = np.abs(v).max((1, 3))  # of the group
    spread = np.abs(v - mean[:, None, :, None]).max((1, 3))
    mean_tol = FACTOR * EPS * big
    # m2 is a sum of squares of distances that are off by a few roundings of big
    rstd_tol = FACTOR * EPS * rstd * (1.0 + rstd * rstd * spread * big)
    zmag = np.repeat(big, cg, 1)[:, None, :] * np.abs(a) + np.abs(be)
    z_tol = FACTOR * EPS * zmag + np.abs(z - be) * np.repeat(rstd_tol / rstd, cg, 1)[:, None, :]
    slope = max([1.1] + [abs(q) for q in (params[:1] if kind == "leaky_relu" else ())])
    t = threshold(p)
    factor = 65536.0 / (65536 - t) if t < 65536 else 0.0
    y_tol = factor * (slope * z_tol + FACTOR * EPS * np.abs(act(z, kind, params)) * (1.0 + np.abs(z)))
    return (y, mean, rstd), (y_tol, mean_tol, rstd_tol)


def group_norm_grad(dy, x, mean, rstd, groups, gamma, beta, kind, params=(), p=0.0, seed=0, offset=0):
    """dy, x (N, P, C), mean and rstd (N, groups), all float64.  Returns dx, dgamma, dbeta and bounds."""
    N, P, C = x.shape
    cg = C // groups
    wide = lambda s: np.repeat(s, cg, 1)[:, None, :]  # noqa: E731
    ga = np.ones(C) if gamma is None else gamma
    be = np.zeros(C) if beta is None else beta
    xhat = (x - wide(mean)) * wide(rstd)
    z = xhat * ga + be
    e = drop(dy, p, seed, offset)
    dz = e * act_grad(z, kind, params)
    average = lambda s: s.reshape(N, P, groups, cg).mean((1, 3))  # noqa: E731
    g = dz * ga
    c1, c2 = average(g), average(g * xhat)
    dx = wide(rstd) * (g - wide(c1) - xhat * wide(c2))
    # dz is off by the roundings of z times |act''| <= 0.5, and by its own
    xmag = (np.abs(x) + np.abs(wide(mean))) * wide(rstd)
    dz_mag = np.abs(e) * (1.0 + xmag * np.abs(ga) + np.abs(be))
    gm = dz_mag * np.abs(ga)
    tol_dx = FACTOR * EPS * wide(rstd) * (gm + wide(average(gm)) + xmag * wide(average(gm * (1.0 + xmag))))
    tol_dgamma = FACTOR * EPS * (dz_mag * (1.0 + xmag)).sum((0, 1))
    tol_dbeta = FACTOR * EPS * dz_mag.sum((0, 1))
    return (dx, (dz * xhat).sum((0, 1)), dz.sum((0, 1))), (tol_dx, tol_dgamma, tol_dbeta)


def embedding_grad(dy, ids, rows, scale, padding=None):
    """dy (T, D) float64, ids (T,).  Returns the table's gradient and the sum of magnitudes."""
    out, mag = np.zeros((rows, dy.shape[1])), np.zeros((rows, dy.shape[1]))
    ok = (ids >= 0) & (ids < rows)
    if padding is not None:
        ok &= ids != padding
    np.add.at(out, ids[ok], dy[ok])
    np.add.at(mag, ids[ok], np.abs(dy[ok]))
    return out * scale, mag * abs(scale)


def assert_close(got, want, tol, dtype, what=""):
    """|got - want| <= tol and the rounding to dtype, at every element."""
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if got.size == 0:
        return
    bound = tol + (HALF_ULP[dtype] * (np.abs(want) + tol)) * 1.0001 + TINY[dtype]
    bad = ~(np.abs(got - want) <= bound)
    if bad.any():
        i = np.unravel_index(int(np.argmax(np.where(bad, np.abs(got - want) - bound, -np.inf))), got.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.size} off, at {i}: {got[i]!r} for {want[i]!r}, bound "
                             f"{np.broadcast_to(bound, got.shape)[i]:.3e}")

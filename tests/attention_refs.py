"""Plain 64-bit forms of attention and its gradient, rotary positions and AdamW, for the tests of the
kernels, with bounds on what the kernels' arithmetic may be off by.

EPS is one float32 rounding, HALF_ULP one rounding to a type.  A score is a float32 sum of D
products, so it is off by at most (D + 4) EPS of the sum of their magnitudes; the exponential's
argument is rounded at its own size and the exponential itself to 2 units.  Weights and score gradients are
rounded to the operands' type once, before their matrix product (float32: not at all); products and
sums over n terms add n EPS of the sum of magnitudes.
"""
import numpy as np

from layer_refs import EPS, HALF_ULP

# An exponential below float32's normal range is 0: a probability is off by up to this beside its relative error.
FLUSH = 2.0 ** -126
ROUND = {"f32": 0.0, "f16": HALF_ULP["f16"], "bf16": HALF_ULP["bf16"]}  # of an operand in the second product


def visible(n, tq, tk, causal, lengths, starts):
    """(N, Tq, Tk) truth values."""
    length = np.full(n, tk) if lengths is None else np.clip(lengths, 0, tk)
    start = np.full(n, tk - tq) if starts is None else np.asarray(starts)
    i, j = np.arange(tq)[None, :, None], np.arange(tk)[None, None, :]
    seen = j < length[:, None, None]
    if causal:
        seen = seen & (j <= start[:, None, None] + i)
    return np.broadcast_to(seen, (n, tq, tk))


def _heads(q, k, v):
    """Each query head beside its key head: three (N, H, T, D) arrays."""
    g = q.shape[2] // k.shape[2]
    return q.transpose(0, 2, 1, 3), np.repeat(k, g, 2).transpose(0, 2, 1, 3), np.repeat(v, g, 2).transpose(0, 2, 1, 3)


def _where(seen, k, v):
    """k and v with zeros at what no query of their image sees: there may be anything."""
    used = seen.any(1)[:, :, None, None]
    return np.where(used, k, 0.0), np.where(used, v, 0.0)


def _scores(qh, kh, scale, seen):
    s = np.matmul(qh, kh.swapaxes(2, 3)) * scale
    mag = np.matmul(np.abs(qh), np.abs(kh).swapaxes(2, 3)) * scale
    return np.where(seen[:, None], s, -np.inf), mag


def _weight_error(mag, d):
    """Relative error of exp(s - reference) in float32, for scores of this magnitude."""
    return (d + 4) * EPS * mag + 4 * EPS * (mag + mag.max(initial=0.0) + 12.0)


def attend(q, k, v, scale, seen, dtype):
    """q (N, Tq, H, D), k, v (N, Tk, Hkv, D) float64.  Returns (out, lse) and a bound on each's error."""
    d, tk = q.shape[3], k.shape[1]
    k, v = _where(seen, k, v)
    qh, kh, vh = _heads(q, k, v)
    s, mag = _scores(qh, kh, scale, seen)
    top = s.max(3, keepdims=True, initial=-np.inf)
    top = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(s - top)
    total = e.sum(3, keepdims=True)
    p = e / np.where(total == 0.0, 1.0, total)
    with np.errstate(divide="ignore"):
        lse = (top + np.log(total))[..., 0]
    rel = np.where(seen[:, None], _weight_error(mag, d), 0.0).max(3, keepdims=True, initial=0.0)
    out = np.matmul(p, vh)
    big = np.abs(vh).max((2, 3), keepdims=True, initial=0.0)
    # the last term: float16 weights below its normal range, 2^-32 of the largest one
    tol = np.matmul(p, np.abs(vh)) * (ROUND[dtype] + 2 * rel + 2 * (tk + 64) * EPS) + tk * 2.0 ** -32 * big
    lse_tol = rel[..., 0] + (tk + 16) * EPS + 8 * EPS * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return (out.transpose(0, 2, 1, 3), lse), (tol.transpose(0, 2, 1, 3), lse_tol)


def attend_grad(do, q, k, v, out, lse, scale, seen, dtype, least=None):
    """The gradient from out and lse as they are given.  Returns (dq, dk, dv) and a bound on each's error.  `least`:
    what float16 score gradients below its normal range may be off by, in the sums for dq and for dk, where the
    largest of all rows says too little."""
    n, tq, h, d = q.shape
    tk, hk = k.shape[1], k.shape[2]
    k, v = _where(seen, k, v)
    sees = seen.any(2)[:, :, None, None]
    q, do, out = (np.where(sees, t, 0.0) for t in (q, do, out))
    qh, kh, vh = _heads(q, k, v)
    doh, oh = do.transpose(0, 2, 1, 3), out.transpose(0, 2, 1, 3)
    s, mag = _scores(qh, kh, scale, seen)
    p = np.exp(s - np.where(np.isfinite(lse), lse, 0.0)[..., None])
    rel = np.where(seen[:, None], _weight_error(mag, d), 0.0) + 4 * EPS * np.abs(np.where(np.isfinite(lse), lse, 0.0))[..., None]
    dp = np.matmul(doh, vh.swapaxes(2, 3))
    delta = (doh * oh).sum(3, keepdims=True)
    ds = scale * p * (dp - delta)
    parts = np.matmul(np.abs(doh), np.abs(vh).swapaxes(2, 3)) + (np.abs(doh) * np.abs(oh)).sum(3, keepdims=True)
    norm = lambda t: np.sqrt((t * t).sum(3)).max(2, initial=0.0)[..., None, None]  # noqa: E731
    if least is None:
        least = [2.0 ** -36 * scale * norm(doh) * norm(vh) if dtype == "f16" else 0.0] * 2  # below float16's normal range
    ds_tol = np.abs(ds) * (ROUND[dtype] + rel + 8 * EPS) + scale * (p * (d + 16) * EPS + FLUSH) * parts
    dq_ds_tol, dk_ds_tol = (ds_tol + t * seen[:, None] for t in least)
    sum_heads = lambda t: t.reshape(n, hk, h // hk, tk, d).sum(2).transpose(0, 2, 1, 3)  # noqa: E731
    by_key = lambda a, b: sum_heads(np.matmul(a.swapaxes(2, 3), b))  # noqa: E731
    dq = np.matmul(ds, kh).transpose(0, 2, 1, 3)
    dk, dv = by_key(ds, qh), by_key(p, doh)
    n_q, n_k = (tk + 64) * EPS, (tq * h // hk + 64) * EPS
    dq_tol = np.matmul(dq_ds_tol + n_q * np.abs(ds), np.abs(kh)).transpose(0, 2, 1, 3)
    dk_tol = by_key(dk_ds_tol + n_k * np.abs(ds), np.abs(qh))
    dv_tol = by_key(p * (ROUND[dtype] + rel + n_k) + (FLUSH + (2.0 ** -40 if dtype == "f16" else 0.0)) * seen[:, None], np.abs(doh))
    return (dq, dk, dv), (dq_tol, dk_tol, dv_tol)


def rotary(x, positions, sections, base, whole, interleaved, inverse):
    """x (N, T, H, D) float64, positions (N, T, axes) whole numbers.  Angles in extended precision."""
    total, y, p = sum(sections), x.copy(), 0
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    for axis, size in enumerate(sections):
        for j in range(size):
            e = np.longdouble(p) / total if whole else np.longdouble(j) / size
            turns = positions[:, :, axis].astype(np.longdouble) * (np.longdouble(base) ** -e / two_pi)
            a = ((turns - np.round(turns)) * two_pi).astype(np.float64)[:, :, None]
            c, s = np.cos(a), -np.sin(a) if inverse else np.sin(a)
            i0, i1 = (2 * p, 2 * p + 1) if interleaved else (p, p + total)
            y[..., i0], y[..., i1] = x[..., i0] * c - x[..., i1] * s, x[..., i0] * s + x[..., i1] * c
            p += 1
    return y


def adamw(p, g, m, v, lr, b1, b2, eps, step, decay, grad_scale):
    """float64 arrays.  Returns p, m, v."""
    g = g * grad_scale
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    mh, vh = m / (1 - b1 ** step), v / (1 - b2 ** step)
    return p - lr * decay * p - lr * mh / (np.sqrt(vh) + eps), m, v

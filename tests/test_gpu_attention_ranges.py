"""Attention where scores are far from zero and its gradient where rows are of very different sizes, against the plain
64-bit form."""
import numpy as np
import pytest
import torch

import attention_refs as A
import layer_refs as R
from test_gpu_attention import DT, T, dev, host, inputs  # noqa: F401  (T: the fixture)

pytestmark = pytest.mark.gpu


def least_by_row(do, v, seen, scale, h):
    """What float16 score gradients below its normal range are off by.  Each is held by a power of two that takes
    bound = 2 scale |do| max|v| above 2^14, so its smallest half step, 2^-25, stands for at most 2^-39 bound: by
    row in the sum for dq; in the sum for dk by the largest of 64 rows (token by token, the heads of a key head
    together), from where it may lie up to 2^2 lower."""
    n, tq = do.shape[:2]
    g = h // v.shape[2]
    norm = np.sqrt((np.where(seen.any(2)[:, :, None, None], do, 0.0) ** 2).sum(3))  # (N, Tq, H)
    used = np.where(seen.any(1)[:, :, None, None], v, 0.0)
    top = np.repeat(np.sqrt((used ** 2).sum(3)).max(1), g, 1)[:, :, None, None]  # (N, H, 1, 1)
    rows = norm.reshape(n, tq, -1, g).transpose(0, 2, 1, 3).reshape(n, h // g, tq * g)
    tiles = np.arange(tq * g) // 64
    most = np.stack([np.where(tiles == t, rows, 0.0).max(2) for t in range(tiles[-1] + 1)], 2)[:, :, tiles]
    most = most.reshape(n, h // g, tq, g).transpose(0, 1, 3, 2).reshape(n, h, tq, 1)
    by_row = norm.transpose(0, 2, 1)[..., None]
    return 2.0 ** -38 * scale * by_row * top, 2.0 ** -36 * scale * most * top


# t, h, hk, d, causal: blocks of one wave, and of several (two keys' halves, operands in registers and in LDS)
SPREAD = [(512, 2, 1, 36, True), (1024, 16, 16, 64, True), (1024, 16, 16, 64, False), (1024, 16, 4, 128, True),
          (1024, 16, 16, 96, False), (700, 12, 6, 256, True), (333, 4, 4, 64, False)]


@pytest.mark.parametrize("shape", SPREAD, ids=str)
def test_float16_rows_keep_their_digits_beside_much_larger_ones(T, shape):  # noqa: F811
    """Two rows whose gradients are 2^22 times the others': each row's dq, and the dk of keys those rows do not see
    or give little to, keep what rounding leaves."""
    t, h, hk, d, causal = shape
    seen = A.visible(1, t, t, causal, None, None)
    tensors, arrays = inputs("f16", 1, t, t, h, hk, d, seed=81)
    rows = np.full((1, t, 1, 1), 2.0 ** -9)
    rows[0, [5, t // 3]] = 2.0 ** 13
    tensors[3], arrays[3] = dev(np.clip(arrays[3], -3, 3) * rows, "f16")
    tensors[1], arrays[1] = dev(arrays[1] * 4, "f16")
    tensors[0], arrays[0] = dev(arrays[0] / 4, "f16")
    q, k, v, do = tensors
    (o, l), _ = A.attend(*arrays[:3], d ** -0.5, seen, "f16")
    out, o = dev(o, "f16")
    lse, l = dev(l, "f32")
    grads = T.attention_backward_nd(do, q, k, v, out, lse, causal=causal)
    torch.cuda.synchronize()
    least = least_by_row(arrays[3], arrays[2], seen, d ** -0.5, h)
    want, tol = A.attend_grad(arrays[3], *arrays[:3], o, l, d ** -0.5, seen, "f16", least)
    for name, got, w, bound in zip(("dq", "dk", "dv"), grads, want, tol):
        # a large row's result may lie behind 65504, the largest value; from 65520 on, half a step (32 / 2) further, it
        # rounds to infinity.  Both sides are brought to 65504, which takes no two values further from each other
        most = 65504.0
        R.assert_close(np.clip(host(got), -most, most), np.clip(w, -most, most), bound, "f16", f"{shape} {name}")


@pytest.mark.parametrize("shape", [(60, 2, 36), (1024, 16, 64)], ids=str)
def test_float16_score_gradients_beyond_any_power(T, shape):  # noqa: F811
    """scale * |dout| |v| far above float32's middle: score gradients are held by a smaller power, not left to overflow.
    Queries and keys are zeros, so their gradients are."""
    t, h, d = shape
    tensors, arrays = inputs("f16", 1, t, t, h, h, d, seed=83)
    tensors[0].zero_(), tensors[1].zero_()
    arrays[0][...] = arrays[1][...] = 0.0
    tensors[3], arrays[3] = dev(arrays[3] * 64, "f16")
    tensors[2], arrays[2] = dev(arrays[2] * 64, "f16")
    q, k, v, do = tensors
    seen = A.visible(1, t, t, True, None, None)
    (o, l), _ = A.attend(*arrays[:3], 1.0, seen, "f16")
    out, o = dev(o, "f16")
    lse, l = dev(l, "f32")
    dq, dk, dv = T.attention_backward_nd(do, q, k, v, out, lse, scale=1e38, causal=True)
    torch.cuda.synchronize()
    assert not dq.any() and not dk.any()
    want, tol = A.attend_grad(arrays[3], *arrays[:3], o, l, 1.0, seen, "f16")  # dv has no scale where scores are 0
    R.assert_close(host(dv), want[2], tol[2], "f16", "dv")


# tq, tk, h, hk, causal: whole blocks, a few rows, split over the keys
FAR = [(150, 150, 2, 1, True), (3, 90, 8, 2, True), (2, 2000, 4, 2, True), (130, 1400, 1, 1, False)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("power", [9, 14, 17, 24, 60])
@pytest.mark.parametrize("call", FAR, ids=str)
def test_scores_far_from_zero(T, dtype, power, call):  # noqa: F811
    """Scores that are multiples of 2^power, up to 127 of them either way: the largest take all, in equal parts.  Every
    third token's scores are zeros, beside the others in its wave."""
    tq, tk, h, hk, causal = call
    rng = np.random.default_rng(85)
    q, k = np.zeros((1, tq, h, 64)), rng.normal(size=(1, tk, hk, 64))
    q[:, :, :, 0] = np.where(np.arange(tq) % 3 == 0, 0.0, 16.0)[None, :, None]
    k[..., 0] = rng.integers(-127, 128, size=(1, tk, hk))
    (tq_, qv), (tk_, kv), (tv_, vv) = (dev(a, dtype) for a in (q, k, rng.normal(size=k.shape)))
    scale = 2.0 ** (power - 4)
    seen = A.visible(1, tq, tk, causal, None, None)
    (o, l), _ = A.attend(qv, kv, vv, scale, seen, dtype)
    out, lse = T.attention_nd(tq_, tk_, tv_, scale=scale, causal=causal)
    torch.cuda.synchronize()
    # weights are 1 and 0 (2^-700 and less), but for the zero scores' rows in float16, which are 2^7: out is a float32
    # sum of up to tk values, their count's reciprocal and a product
    tol = (tk + 4) * R.EPS * np.abs(vv).max()
    if power < 24:
        # references below 2^20 were rounded, by up to 2^-5, and the scores' products with c are not: a weight is then
        # 2^(+-2^-5) of a power of two, the same for equal scores, and is rounded to dtype beside the products but not in
        # the sum of weights
        tol += A.ROUND[dtype] * np.abs(vv).max()
    R.assert_close(host(out), o, tol, dtype, f"{call} 2^{power} out")
    # scale log2(e), its product with the score, the sum with the count's logarithm, the way back: 6 roundings
    R.assert_close(host(lse), l, 6 * R.EPS * np.abs(l) + 8 * R.EPS, "f32", f"{call} 2^{power} lse")

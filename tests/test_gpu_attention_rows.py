"""Attention's rows: places that nothing may come from, and many heads of one key head."""
import pytest
import torch

import attention_refs as A
from test_gpu_attention import DT, T, check_backward, check_forward, inputs, ints  # noqa: F401  (T: the fixture)

pytestmark = pytest.mark.gpu


# Images, heads and key heads: blocks of one wave and of several, a query head a key head (whose tiles of rows are read
# without looking at each row once they all see something) and two.
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("heads", [(4, 4, 4), (4, 4, 2), (64, 2, 2), (64, 4, 2)], ids=str)
@pytest.mark.parametrize("d", [48, 128])
def test_queries_that_see_nothing_hold_anything(T, dtype, heads, d):  # noqa: F811
    """The first token that sees a key lies inside a tile of 32 or 64 rows, on its border, and behind the first one."""
    n, h, hk = heads
    tq, tk = 150, 140
    firsts, ends = (20, 32, 64, 100), (140, 33, 140, 0)  # of the images in turn; keys
    starts, lengths = tuple(-firsts[i % 4] for i in range(n)), tuple(ends[i // 4 % 4] for i in range(n))
    seen = A.visible(n, tq, tk, True, lengths, starts)
    tensors, arrays = inputs(dtype, n, tq, tk, h, hk, d, seed=95)
    mask = dict(causal=True, lengths=ints(lengths), starts=ints(starts))
    unseen, blind = torch.from_numpy(~seen.any(1)).cuda(), torch.from_numpy(~seen.any(2)).cuda()
    for bad in (float("nan"), float("inf"), torch.finfo(DT[dtype]).min):
        q, k, v, do = (t.clone() for t in tensors)
        k[unseen], v[unseen], q[blind], do[blind] = bad, bad, bad, bad
        grads = check_backward(T, dtype, [q, k, v, do], arrays, seen, None, f"{bad}", **mask)
        assert not grads[0][blind].any() and not grads[1][unseen].any() and not grads[2][unseen].any()


# n, tq, tk, h, hk, d, lengths: more than 32 rows of a key head, tokens fewer than its heads
SHARED = [(1, 1, 300, 64, 1, 64, None), (2, 1, 2000, 96, 1, 40, (2000, 700)), (3, 5, 400, 40, 5, 128, (400, 5, 77)),
          (1, 2, 513, 33, 1, 256, None), (2, 3, 1500, 200, 2, 64, (3, 1500)), (1, 1, 33, 128, 1, 96, None)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHARED, ids=[str(s[:6]) for s in SHARED])
def test_tokens_of_many_heads_over_one_key_head(T, shape, dtype):  # noqa: F811
    n, tq, tk, h, hk, d, lengths = shape
    starts = None if lengths is None else tuple(x - tq for x in lengths)
    seen = A.visible(n, tq, tk, True, lengths, starts)
    tensors, arrays = inputs(dtype, n, tq, tk, h, hk, d, seed=96)
    mask = dict(causal=True, lengths=ints(lengths), starts=ints(starts))
    check_forward(T, dtype, tensors, arrays, seen, None, str(shape), **mask)
    check_backward(T, dtype, tensors, arrays, seen, None, str(shape), **mask)

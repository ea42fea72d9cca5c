"""Rotary calls that are large enough for a thread to turn several heads with the sines and cosines it has."""
import numpy as np
import pytest
import torch

import attention_refs as A
import layer_refs as R
from test_gpu_rotary_adamw import DT, T, host, rotary_bound  # noqa: F401  (T: the fixture)

pytestmark = pytest.mark.gpu

# dtype, n, t, heads, d, sections, interleaved, inverse, in place, heads of one thread
CALLS = [
    ("f16", 1, 65536, 7, 64, (16, 16), False, False, False, 4),          # shares of 4 and 3
    ("bf16", 2, 16411, 11, 128, (16, 24, 24), False, True, False, 6),    # 6 and 5
    ("bf16", 2, 16411, 11, 128, (64,), True, False, True, 6),
    ("f16", 1, 40009, 20, 80, (20, 20), True, True, False, 7),           # 7, 7 and 6
    ("f32", 1, 40009, 19, 96, (5, 0, 11), False, False, True, 10),       # 10 and 9; 64 elements stay behind the pairs
    ("f32", 3, 30011, 3, 36, (9, 8), True, False, False, 3),             # an odd run; a pair behind the last whole vector
    ("f16", 1, 120001, 5, 33, (7,), False, True, False, 3),              # elements that stay end inside a vector
    ("bf16", 1, 262144, 16, 32, (16,), False, False, True, 16),
]


def heads_of_a_thread(dtype, tokens, heads, d, sections):
    """As the call's own rule has it: doubled while half as many threads are 512 * 1024 still, then in equal shares."""
    v, pairs = (4 if dtype == "f32" else 8), sum(sections)
    units = -(-pairs // v) + -(-(d - 2 * pairs) // (2 * v))
    run = 1
    while run < heads and tokens * units * -(-heads // (2 * run)) >= 512 * 1024:
        run *= 2
    return -(-heads // -(-heads // run))


@pytest.mark.parametrize("call", CALLS, ids=str)
def test_several_heads_a_thread(T, call):  # noqa: F811
    dtype, n, t, h, d, sections, interleaved, inverse, in_place, run = call
    assert heads_of_a_thread(dtype, n * t, h, d, sections) == run and run > 1
    gen = torch.Generator(device="cuda").manual_seed(7)
    whole = torch.randn((n, t, h + 2, d), generator=gen, device="cuda").to(DT[dtype])
    pos = torch.randint(-(1 << 20), 1 << 30, (n, t, len(sections)), generator=gen, device="cuda")
    options = dict(interleaved=interleaved, inverse=inverse)
    x = whole[:, :, 1:h + 1]
    # One head by itself is one head a thread.  Each side rounds once, and a fused step may leave out the float32 rounding
    # before it: both lie within half a step and the float32 bound of the exact value, so within twice that of each other.
    one = torch.stack([T.rotary_nd(x[:, :, i:i + 1], pos, sections, **options)[:, :, 0] for i in range(h)], 2)
    before = whole.clone()
    y = T.rotary_nd(x, pos, sections, out=x if in_place else None, **options)
    torch.cuda.synchronize()
    size = before[:, :, 1:h + 1].double().abs().amax(3, keepdim=True)
    bound = (np.pi + 8) * R.EPS * 2.0 ** 0.5 * size
    far = (y.double() - one.double()).abs() > 2 * (bound + R.HALF_ULP[dtype] * (one.double().abs() + bound) * 1.001 + R.TINY[dtype])
    assert not far.any(), (call, far.nonzero()[0].tolist(), int(far.sum()))
    assert torch.equal(whole[:, :, 0], before[:, :, 0]) and torch.equal(whole[:, :, -1], before[:, :, -1])
    assert in_place or torch.equal(whole, before)
    some = torch.arange(0, t, 4001, device="cuda")
    some = torch.cat((some, torch.tensor([t - 1], device="cuda")))
    xv = host(before[:, :, 1:h + 1][:, some])
    want = A.rotary(xv, pos[:, some].cpu().numpy(), sections, 10000.0, False, interleaved, inverse)
    R.assert_close(host(y[:, some]), want, rotary_bound(xv), dtype, str(call))

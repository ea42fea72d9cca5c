"""Rotary positions and the AdamW step on the GPU against plain forms (attention_refs): values within
bounds derived from float32 arithmetic, 8-bit states code for code."""
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
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DT[dtype])
    return t.cuda(), t.double().numpy()


def host(t):
    return t.double().cpu().numpy()


def rotary_bound(x):
    # the angle is off by 2^-32 of a turn and its float32 rounding, half a unit of half a turn: together
    # pi 2^-24 and less; sine and cosine by 2 units, the two products and their sum by a rounding each
    return (np.pi + 8) * R.EPS * np.sqrt(2.0) * np.abs(x).max(3, keepdims=True, initial=0.0)


# n, t, h, d, sections
ROTARY = [(1, 1, 1, 2, (1,)), (2, 3, 4, 64, (8, 12, 12)), (1, 7, 3, 33, (5, 0, 11)), (2, 5, 10, 128, (16, 24, 24)),
          (3, 1, 2, 40, (3, 4, 5, 2)), (1, 300, 20, 80, (20, 20)), (1, 2, 1, 512, (256,)), (2, 2, 3, 17, (0, 3))]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", ROTARY, ids=str)
@pytest.mark.parametrize("options", [(False, False, False), (True, False, True), (False, True, True), (True, True, False)], ids=str)
def test_rotary(T, shape, dtype, options):
    n, t, h, d, sections = shape
    whole, interleaved, inverse = options
    rng = np.random.default_rng(5)
    x, xv = dev(rng.normal(size=(n, t, h + 1, d)), dtype)
    x, xv = x[:, :, :h], xv[:, :, :h]  # strided heads
    pos = rng.integers(-(1 << 20), 1 << 31, size=(n, t, len(sections)))
    for index in (torch.int32, torch.int64):
        y = T.rotary_nd(x, torch.from_numpy(pos).to(index).cuda(), sections, whole_ladder=whole, interleaved=interleaved,
                        inverse=inverse)
        torch.cuda.synchronize()
        want = A.rotary(xv, pos, sections, 10000.0, whole, interleaved, inverse)
        turned = 2 * sum(sections)
        assert np.array_equal(host(y)[..., turned:], xv[..., turned:])
        R.assert_close(host(y), want, rotary_bound(xv), dtype, str(shape))


def test_rotary_in_place_and_bases(T):
    rng = np.random.default_rng(6)
    x, xv = dev(rng.normal(size=(2, 9, 5, 48)), "f32")
    pos = rng.integers(0, 100, size=(1, 9, 2))
    tp = torch.from_numpy(pos).cuda().expand(2, 9, 2)
    for base in (0.25, 1.0, 500000.0):  # below one a position turns by more than one angle a step
        y = x.clone()
        part = y[:, :, 1:4]
        assert T.rotary_nd(part, tp, (9, 15), base=base, out=part) is part
        want = A.rotary(xv[:, :, 1:4], np.broadcast_to(pos, (2, 9, 2)), (9, 15), base, False, False, False)
        torch.cuda.synchronize()
        R.assert_close(host(part), want, rotary_bound(xv[:, :, 1:4]), "f32", f"base {base}")
        assert torch.equal(y[:, :, 0], x[:, :, 0]) and torch.equal(y[:, :, 4], x[:, :, 4])  # the others stay
        back = T.rotary_nd(part, tp, (9, 15), base=base, inverse=True)
        R.assert_close(host(back), xv[:, :, 1:4], 2 * rotary_bound(xv[:, :, 1:4]) * 1.5, "f32", "turned back")


def adamw_inputs(sizes, dtype, grad, seed, copies=None):
    rng = np.random.default_rng(seed)
    made = []
    for k, size in enumerate(sizes):
        p, pv = dev(rng.normal(size=size), dtype)
        g, gv = dev(rng.normal(size=size) * 10.0 ** rng.uniform(-3, 1), grad)
        m, v = (rng.normal(size=size) * 0.1).astype(np.float32), (rng.normal(size=size) ** 2 * 0.01).astype(np.float32)
        made.append((p, pv, g, gv, m, v))
    return made


SIZES = [(5,), (256,), (257,), (3, 1001), (70, 64), (1,), (2048,), (4097,)]
HYPER = dict(lr=2e-3, betas=(0.9, 0.98), eps=1e-7)


def param_bound(want, before, update):
    # the update's chain (a quotient, a root, four products, a sum, the corrections) is off by 16 roundings
    return 16 * R.EPS * (np.abs(before) + np.abs(update))


@pytest.mark.parametrize("dtype,grad", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("f16", "f32"), ("bf16", "f16")])
@pytest.mark.parametrize("device_values", [False, True])
def test_adamw_32_bits(T, dtype, grad, device_values):
    made = adamw_inputs(SIZES, dtype, grad, seed=3)
    decay = [0.1 if k % 2 else 0.0 for k in range(len(made))]
    p, g = [a[0] for a in made], [a[2] for a in made]
    m, v = [torch.from_numpy(a[4]).cuda() for a in made], [torch.from_numpy(a[5]).cuda() for a in made]
    copies = [torch.zeros(a[0].shape, dtype=torch.bfloat16, device="cuda") if k % 3 else None for k, a in enumerate(made)]
    wrap = (lambda x, t: torch.tensor([x], dtype=t, device="cuda")) if device_values else (lambda x, t: x)
    got = T.adamw_nd(p, g, m, v, lr=wrap(HYPER["lr"], torch.float32), betas=HYPER["betas"], eps=HYPER["eps"],
                     step=wrap(7, torch.int64), weight_decay=decay, grad_scale=wrap(0.25, torch.float32), copies=copies)
    torch.cuda.synchronize()
    assert all(a is b for a, b in zip(got, p))
    for k, (tp, pv, _, gv, m0, v0) in enumerate(made):
        want, wm, wv = A.adamw(pv, gv, m0.astype(np.float64), v0.astype(np.float64), HYPER["lr"], *HYPER["betas"], HYPER["eps"], 7,
                               decay[k], 0.25)
        tol = param_bound(want, pv, want - pv)
        R.assert_close(host(tp), want, tol, dtype, f"param {k}")
        R.assert_close(host(m[k]), wm, 4 * R.EPS * (np.abs(0.9 * m0) + np.abs(0.1 * 0.25 * gv)), "f32", f"m {k}")
        R.assert_close(host(v[k]), wv, 6 * R.EPS * np.abs(wv), "f32", f"v {k}")
        if copies[k] is not None:
            R.assert_close(host(copies[k]), want, tol, "bf16", f"copy {k}")


def coded(x, root):
    """Blocks of 256 of a float32 array as (e4m3 tensor, scales), by single float32 operations."""
    flat = np.zeros(-(-x.size // 256) * 256, np.float32)
    flat[:x.size] = x.reshape(-1)
    rows = flat.reshape(-1, 256)
    scale = np.maximum((np.abs(rows).max(1) / np.float32(448.0)).astype(np.float32), np.float32(2.0 ** -126))
    q = rows / scale[:, None]
    if root:
        q = np.where(rows > 0, np.maximum(q, np.float32(2.0 ** -9)), q)
    return torch.from_numpy(q.reshape(-1)[:x.size].astype(np.float32)).to(torch.float8_e4m3fn), torch.from_numpy(scale)


@pytest.mark.parametrize("dtype,grad", [("f32", "f32"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")])
def test_adamw_8_bits(T, dtype, grad):
    made = adamw_inputs(SIZES, dtype, grad, seed=4)
    p, g = [a[0] for a in made], [a[2] for a in made]
    flat = lambda t: t.reshape(-1)  # noqa: E731
    cm = [coded(a[4], False) for a in made]
    cv = [coded(np.sqrt(a[5]), True) for a in made]
    m, v = [c.cuda() for c, _ in cm], [c.cuda() for c, _ in cv]
    ms, vs = [s.cuda() for _, s in cm], [s.cuda() for _, s in cv]
    T.adamw_nd([flat(t) for t in p], [flat(t) for t in g], m, v, step=3, weight_decay=0.05, m_scales=ms, v_scales=vs, **HYPER)
    torch.cuda.synchronize()
    f = np.float32
    for k, (tp, pv, _, gv, _, _) in enumerate(made):
        wide = lambda s: np.repeat(s.numpy(), 256)[:pv.size]  # noqa: E731
        m0 = cm[k][0].float().numpy() * wide(cm[k][1])
        r0 = cv[k][0].float().numpy() * wide(cv[k][1])
        g32 = gv.reshape(-1).astype(f)
        # one float32 operation after the other: the same bits as the kernel's
        wm = m0 * f(0.9) + g32 * f(1 - 0.9)
        wv = (r0 * r0) * f(0.98) + (g32 * g32) * f(1 - 0.98)
        (mc, msc), (vc, vsc) = coded(wm, False), coded(np.sqrt(wv), True)
        assert torch.equal(ms[k].cpu(), msc) and torch.equal(vs[k].cpu(), vsc), k
        assert torch.equal(m[k].cpu().view(torch.uint8), mc.view(torch.uint8)), k
        assert torch.equal(v[k].cpu().view(torch.uint8), vc.view(torch.uint8)), k
        want, _, _ = A.adamw(pv.reshape(-1), gv.reshape(-1), m0.astype(np.float64), (r0 * r0).astype(np.float64), HYPER["lr"],
                             *HYPER["betas"], HYPER["eps"], 3, 0.05, 1.0)
        R.assert_close(host(tp).reshape(-1), want, param_bound(want, pv.reshape(-1), want - pv.reshape(-1)), dtype, f"param {k}")


def test_adamw_8_bit_codes_of_every_magnitude(T):
    """The conversion to e4m3 at every exponent, ties and the smallest codes among them."""
    rng = np.random.default_rng(8)
    x = (448.0 * 2.0 ** -rng.uniform(0, 22, size=65536)).astype(np.float32)
    x[::2] = (np.round(x[::2] * 16) / 16)  # many ties
    x[::256] = 448.0  # every scale is 1
    x[1::3] *= -1
    p = torch.zeros(65536, device="cuda")
    m, v = (torch.zeros(65536, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ms, vs = torch.zeros(256, device="cuda"), torch.zeros(256, device="cuda")
    T.adamw_nd([p], [torch.from_numpy(x).cuda()], [m], [v], lr=0.0, step=1, betas=(0.0, 0.0), m_scales=[ms], v_scales=[vs])
    torch.cuda.synchronize()
    want, scale = coded(np.float32(0.0) + x, False)  # m = 0 m + 1 g: a negative zero becomes zero
    assert torch.equal(ms.cpu(), scale) and float(ms.max()) == 1.0
    assert torch.equal(m.cpu().view(torch.uint8), want.view(torch.uint8))
    want, scale = coded(np.sqrt(x * x), True)
    assert torch.equal(v.cpu().view(torch.uint8), want.view(torch.uint8))
    assert int((v.cpu().float() == 0).sum()) == int((x == 0).sum())


@pytest.mark.parametrize("count", [1, 8, 9, 40, 41, 131])
def test_adamw_many_tensors(T, count):
    """More tensors than a launch's arguments describe; each is updated once."""
    rng = np.random.default_rng(count)
    sizes = rng.integers(1, 1500, size=count)
    sizes[0] = 40000
    p0 = [rng.normal(size=s).astype(np.float32) for s in sizes]
    g0 = [rng.normal(size=s).astype(np.float32) for s in sizes]
    p, g = ([torch.from_numpy(a).cuda() for a in part] for part in (p0, g0))
    m, v = ([torch.zeros_like(t) for t in p] for _ in range(2))
    T.adamw_nd(p, g, m, v, step=1, weight_decay=0.0, **HYPER)
    torch.cuda.synchronize()
    for k in range(count):
        want, wm, wv = A.adamw(p0[k].astype(np.float64), g0[k].astype(np.float64), 0.0, 0.0, HYPER["lr"], *HYPER["betas"], HYPER["eps"],
                               1, 0.0, 1.0)
        R.assert_close(host(p[k]), want, param_bound(want, p0[k], want - p0[k]), "f32", f"param {k}")
        R.assert_close(host(m[k]), wm, 4 * R.EPS * np.abs(wm), "f32", f"m {k}")
        R.assert_close(host(v[k]), wv, 6 * R.EPS * np.abs(wv), "f32", f"v {k}")


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_and_rotary_captured_follow_device_values(T, bits):
    """A graph of a turn and a step: replays with new step numbers, rates, gradients and positions equal eager calls."""
    state = torch.float32 if bits == 32 else torch.float8_e4m3fn
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((2, 6, 4, 32), generator=gen, device="cuda")
    pos = torch.zeros((2, 6, 2), dtype=torch.int64, device="cuda")
    make = lambda: dict(p=[torch.ones(n, device="cuda") for n in (700, 2 * 6 * 4 * 32)],  # noqa: E731
                        m=[torch.zeros(n, dtype=state, device="cuda") for n in (700, 1536)],
                        v=[torch.zeros(n, dtype=state, device="cuda") for n in (700, 1536)],
                        ms=[torch.zeros(n, device="cuda") for n in (3, 6)], vs=[torch.zeros(n, device="cuda") for n in (3, 6)])
    grad = torch.zeros(700, device="cuda")
    lr, step, scale = torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(1, device="cuda")
    turned = torch.empty_like(x)

    def arguments(s, **options):
        if bits == 8:
            options.update(m_scales=s["ms"], v_scales=s["vs"])
        return (s["p"], [grad, turned.reshape(-1)], s["m"], s["v"]), options

    kept, eager = make(), make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        turn = T.PreparedCall(T.rotary_nd, x, pos, (6, 10), out=turned)
        args, options = arguments(kept, lr=lr, step=step, grad_scale=scale, weight_decay=[0.1, 0.0])
        update = T.PreparedCall(T.adamw_nd, *args, **options)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        turn()
        update()
    for k in range(1, 5):
        grad.copy_(torch.randn(700, generator=gen, device="cuda"))
        pos.copy_(torch.randint(0, 1 << 30, pos.shape, generator=gen, device="cuda"))
        lr.fill_(0.01 * k), step.fill_(k), scale.fill_(1.0 / k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(turned, T.rotary_nd(x, pos, (6, 10)))
        args, options = arguments(eager, lr=lr, step=step, grad_scale=scale, weight_decay=[0.1, 0.0])
        T.adamw_nd(*args, **options)
        torch.cuda.synchronize()
        bits_of = lambda t: t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t  # noqa: E731
        for name in ("p", "m", "v") + (("ms", "vs") if bits == 8 else ()):
            assert all(torch.equal(bits_of(a), bits_of(b)) for a, b in zip(kept[name], eager[name])), (k, name)
        assert not torch.equal(kept["p"][0], torch.ones(700, device="cuda"))


def test_adamw_values_that_are_not_finite_stay_in_their_block(T):
    for bad in (float("nan"), float("inf")):
        p, g = torch.ones(1000, device="cuda"), torch.ones(1000, device="cuda")
        g[300] = bad
        m, v = (torch.zeros(1000, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
        ms, vs = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")
        T.adamw_nd([p], [g], [m], [v], lr=0.1, step=1, m_scales=[ms], v_scales=[vs])
        torch.cuda.synchronize()
        held, root = m.float() * ms.repeat_interleave(256)[:1000], v.float() * vs.repeat_interleave(256)[:1000]
        block = torch.zeros(1000, dtype=torch.bool, device="cuda")
        block[256:512] = True
        assert not torch.isfinite(held[block]).any() and not torch.isfinite(root[block]).any(), bad
        assert torch.isfinite(held[~block]).all() and torch.isfinite(root[~block]).all() and not torch.isfinite(p[300])
        others = torch.cat((p[:300], p[301:]))  # the step itself takes the states before they are held in 8 bits
        assert torch.isfinite(others).all()


def test_adamw_zero_states_and_refusals(T):
    p = torch.ones(300, device="cuda")
    zero = lambda: torch.zeros(300, dtype=torch.float8_e4m3fn, device="cuda")  # noqa: E731
    m, v, ms, vs = zero(), zero(), torch.zeros(2, device="cuda"), torch.zeros(2, device="cuda")
    T.adamw_nd([p], [torch.zeros(300, device="cuda")], [m], [v], lr=0.5, step=1, weight_decay=0.5, m_scales=[ms], v_scales=[vs])
    torch.cuda.synchronize()
    assert torch.equal(p, torch.full((300,), 0.75, device="cuda")) and not m.float().any() and not v.float().any()
    f = lambda: torch.zeros(300, device="cuda")  # noqa: E731
    for what, call in {
        "twice": lambda: T.adamw_nd([p, p], [f(), f()], [f(), f()], [f(), f()], lr=0.1, step=1),
        "dense": lambda: T.adamw_nd([p[::2]], [f()[:150]], [f()[:150]], [f()[:150]], lr=0.1, step=1),
        "dense with 300": lambda: T.adamw_nd([p], [f()], [f()[:10]], [f()], lr=0.1, step=1),
        "scales": lambda: T.adamw_nd([p], [f()], [zero()], [zero()], lr=0.1, step=1),
        "float8": lambda: T.adamw_nd([p], [f()], [f().half()], [f().half()], lr=0.1, step=1),
        "copies must": lambda: T.adamw_nd([p], [f()], [f()], [f()], lr=0.1, step=1, copies=[f()]),
        "one value": lambda: T.adamw_nd([p], [f()], [f()], [f()], lr=f(), step=1),
        "counts from 1": lambda: T.adamw_nd([p], [f()], [f()], [f()], lr=0.1, step=0),
    }.items():
        with pytest.raises(T.ConvTransposeError, match=what):
            call()
    x, pos = torch.zeros((2, 3, 4, 16), device="cuda"), torch.zeros((2, 3, 1), dtype=torch.int32, device="cuda")
    for what, call in {
        "half a head": lambda: T.rotary_nd(x, pos, (9,)),
        "one section an axis": lambda: T.rotary_nd(x, pos, (2, 2)),
        "int32 or int64": lambda: T.rotary_nd(x, pos.float(), (4,)),
        "dense": lambda: T.rotary_nd(x.transpose(2, 3), pos, (1,)),
        "x's strides": lambda: T.rotary_nd(x, pos, (4,), out=x.as_strided((2, 3, 4, 16), (16, 32, 96, 1))),
    }.items():
        with pytest.raises(T.ConvTransposeError, match=what):
            call()

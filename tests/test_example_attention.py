"""The attention decoder example: its gradients against automatic differentiation of the same network in
float64 on the CPU, its steps in both widths of state; and a sequence decoded token by token over a cache."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import attention_refs as A
import layer_refs as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("attention_decoder", os.path.join(ROOT, "examples", "attention_decoder.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def turned(x, codes_shape, sections):
    """Rotary positions by row and column in torch float64: x (N, T, H, D)."""
    n, h, w = codes_shape
    row, col = torch.arange(h).repeat_interleave(w), torch.arange(w).repeat(h)
    angle = torch.cat([p[:, None] * 10000.0 ** (-torch.arange(s, dtype=torch.float64) / s) for p, s in zip((row, col), sections)], 1)
    c, s = angle.cos()[None, :, None], angle.sin()[None, :, None]
    half = sum(sections)
    a, b = x[..., :half], x[..., half:2 * half]
    return torch.cat((a * c - b * s, a * s + b * c, x[..., 2 * half:]), -1)


def test_gradients_of_the_whole_step(example):
    model = example.AttentionDecoder(codes=40, width=32, heads=4, kv_heads=2, head=16, out=16, groups=4, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(5)
    codes = torch.randint(0, 40, (2, 6, 5), generator=gen, device="cuda")
    y, saved = model.forward(codes)
    dy = torch.randn((2, 12, 10, 16), generator=gen, device="cuda").half().movedim(-1, 1)
    grads = model.backward(dy, saved)
    torch.cuda.synchronize()

    book = model.lookup.double().cpu().requires_grad_()
    ga, be = (p.double().cpu().requires_grad_() for p in (model.gamma, model.beta))
    w1, w2, w3 = (w.double().cpu() for w in (model.w_qkv, model.w_back, model.w_up))
    x = book[codes.cpu()].movedim(-1, 1)
    p = torch.nn.functional.conv2d(torch.nn.functional.group_norm(x, 4, ga, be, 1e-5), w1)
    q, k, v = model.split(p.movedim(1, -1).reshape(2, 30, 8, 16))
    q, k = (turned(t, codes.shape, model.sections) for t in (q, k))
    k, v = (t.repeat_interleave(2, 2) for t in (k, v))
    s = torch.matmul(q.transpose(1, 2), k.permute(0, 2, 3, 1)) / 4.0
    a = torch.matmul(s.softmax(-1), v.transpose(1, 2)).transpose(1, 2)
    z = torch.nn.functional.conv2d(a.reshape(2, 6, 5, 64).movedim(-1, 1), w2) + x
    want = torch.nn.functional.conv_transpose2d(z, w3, stride=2, padding=1)
    # float16 holds the activations between the operators: a few roundings of 2^-11 each way, as independent errors
    err = lambda got, ref: float((got.double().cpu() - ref).norm() / ref.norm())  # noqa: E731
    assert err(y, want.detach()) <= 6 * 2.0 ** -11
    want.backward(dy.double().cpu())
    for name, got, ref in zip(("codebook", "gamma", "beta"), grads, (book.grad, ga.grad, be.grad)):
        assert got.dtype == torch.float32 and err(got, ref) <= 12 * 2.0 ** -11, name


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_run(example, bits):
    model = example.AttentionDecoder(codes=40, state_bits=bits)
    before = [p.clone() for p in model.parameters()]
    losses = example.train(steps=3, images=2, grid=6, model=model)
    assert np.isfinite(losses).all() and int(model.steps) == 3
    assert torch.equal(model.lookup, model.codebook.half())
    assert all(torch.isfinite(p).all() and not torch.equal(p, b) for p, b in zip(model.parameters(), before))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_token_by_token_over_a_cache(example, dtype):
    """A causal pass over whole sequences, and the same one token at a time: rotary, cache, attention."""
    T = example.T
    kind = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    n, t, h, hk, d = 3, 70, 6, 2, 32
    gen = torch.Generator(device="cuda").manual_seed(7)
    packed = torch.randn((n, t, h + 2 * hk, d), generator=gen, device="cuda").to(kind)
    first = torch.tensor([0, 40, 69], dtype=torch.int32, device="cuda")  # where each sequence's decoding begins
    places = torch.arange(t, device="cuda", dtype=torch.int64)[None, :, None].expand(n, -1, 1)
    turning = packed[:, :, :h + hk]
    T.rotary_nd(turning, places, (d // 2,), out=turning)
    whole, lse = T.attention_nd(packed[:, :, :h], packed[:, :, h:h + hk], packed[:, :, h + hk:], causal=True)
    cache = torch.full((2, n, t + 5, hk, d), float("nan"), dtype=kind, device="cuda")  # what is not written yet may be anything
    for i in range(n):
        cache[0, i, :first[i]], cache[1, i, :first[i]] = packed[i, :first[i], h:h + hk], packed[i, :first[i], h + hk:]
    lengths = first.clone()
    got = {}
    for _ in range(t):
        active = (lengths < t).nonzero().flatten()
        if not len(active):
            break
        at = torch.clamp(lengths, max=t - 1).long()
        token = packed[torch.arange(n, device="cuda"), at][:, None]
        cache[0, active, at[active]], cache[1, active, at[active]] = token[active, 0, h:h + hk], token[active, 0, h + hk:]
        lengths = torch.clamp(lengths + 1, max=t)
        out, l = T.attention_nd(token[:, :, :h], cache[0], cache[1], causal=True, lengths=lengths, starts=lengths - 1)
        for i in active.tolist():
            got[i, int(at[i])] = (out[i, 0], l[i, :, 0])
    assert len(got) == sum(t - int(f) for f in first)
    q, k, v = (a.double().cpu().numpy() for a in (packed[:, :, :h], packed[:, :, h:h + hk], packed[:, :, h + hk:]))
    (o, ls), (otol, ltol) = A.attend(q, k, v, d ** -0.5, A.visible(n, t, t, True, None, None), dtype)
    R.assert_close(whole.double().cpu().numpy(), o, otol, dtype, "whole")
    for (i, j), (a, b) in got.items():
        R.assert_close(a.double().cpu().numpy(), o[i, j], otol[i, j], dtype, f"token {j} of {i}")
        R.assert_close(b.double().cpu().numpy(), ls[i, :, j], ltol[i, :, j], "f32", f"lse of token {j} of {i}")

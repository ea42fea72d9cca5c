"""The token decoder example: its gradients against automatic differentiation of the same
network in float64 on the CPU, and that training lowers the loss."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import layer_refs as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("token_decoder", os.path.join(ROOT, "examples", "token_decoder.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_gradients_of_the_whole_step(example):
    model = example.TokenDecoder(codes=40, width=32, hidden=24, out=16, groups=4, dropout=0.2, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(5)
    codes = torch.randint(0, 40, (2, 6, 5), generator=gen, device="cuda")
    y, saved = model.forward(codes, step=7)
    dy = torch.randn((2, 24, 20, 16), generator=gen, device="cuda").half().movedim(-1, 1)
    grads = model.backward(dy, saved)
    torch.cuda.synchronize()

    book = model.codebook.half().double().cpu().requires_grad_()
    ga, be = (p.double().cpu().requires_grad_() for p in (model.gamma, model.beta))
    w1, w2 = model.w1.double().cpu(), model.w2.double().cpu()
    h = torch.nn.functional.conv_transpose2d(book[codes.cpu()].movedim(-1, 1), w1, stride=2, padding=1)
    a = torch.nn.functional.silu(torch.nn.functional.group_norm(h, 4, ga, be, 1e-5))
    keep = R.keep_mask(a.numel(), 0.2, 3, 7).reshape(a.movedim(1, -1).shape)
    a = a * torch.from_numpy(keep).movedim(-1, 1) * (65536 / (65536 - R.threshold(0.2)))
    want = torch.nn.functional.conv_transpose2d(a, w2, stride=2, padding=1)
    # float16 holds the activations between the operators: a few roundings of 2^-11, summed
    # over the taps as independent errors
    err = lambda got, ref: float((got.double().cpu() - ref).norm() / ref.norm())  # noqa: E731
    assert err(y, want.detach()) <= 4 * 2.0 ** -11
    want.backward(dy.double().cpu())
    for name, got, ref in zip(("codebook", "gamma", "beta"), grads, (book.grad, ga.grad, be.grad)):
        assert got.dtype == torch.float32 and err(got, ref) <= 6 * 2.0 ** -11, name


def test_training_lowers_the_loss(example):
    losses = example.train(steps=12)
    assert np.isfinite(losses).all() and losses[-1] < 0.9 * losses[0], losses

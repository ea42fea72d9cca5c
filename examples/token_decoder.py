"""Training a small token decoder with the library's operators, end to end on the GPU.

An image arrives as a grid of codes.  The decoder looks them up in a codebook
(``embedding_nd``), doubles the resolution twice with transposed convolutions
(``convtranspose_nd``, channels-last), and after the first of them normalises, applies SiLU
and drops out in one call (``group_norm_nd``).  The backward pass goes the same way back: the
convolutions' input gradients are ``convolution_nd`` with the same weights (the adjoint),
the norm's ``group_norm_backward_nd`` draws the same dropout mask again instead of loading
one, and the codebook's gradient sums the tokens of each code (``embedding_backward_nd``).
The codebook and the norm's parameters are trained; the convolutions keep their weights.

    python examples/token_decoder.py [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import transposed_convolution_amd as T  # noqa: E402


class TokenDecoder:
    """codes (N, H, W) -> images (N, out, 4H, 4W), float16 activations, float32 parameters."""

    ATTRS = dict(strides=[2, 2], pads=[1, 1, 1, 1])

    def __init__(self, codes=512, width=64, hidden=48, out=16, groups=8, dropout=0.1, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        randn = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
        self.groups, self.dropout, self.seed = groups, dropout, seed
        self.codebook = randn(codes, width)
        self.gamma, self.beta = torch.ones(hidden, device=device), torch.zeros(hidden, device=device)
        self.w1 = (randn(width, hidden, 4, 4) / (4 * width) ** 0.5).half()
        self.w2 = (randn(hidden, out, 4, 4) / (4 * hidden) ** 0.5).half()

    def norm_options(self, step):
        # one seed for the run, one offset a step: every step draws another mask
        return dict(activation="silu", dropout_p=self.dropout, seed=self.seed, offset=step)

    def forward(self, codes, step):
        x = T.embedding_nd(codes, self.codebook.half()).movedim(-1, 1)  # channels-last (N, width, H, W)
        h = T.convtranspose_nd(x, self.w1, channels_last=True, **self.ATTRS)
        a, mean, rstd = T.group_norm_nd(h, self.groups, self.gamma, self.beta, **self.norm_options(step))
        y = T.convtranspose_nd(a, self.w2, channels_last=True, **self.ATTRS)
        return y, (codes, h, mean, rstd, step)

    def backward(self, dy, saved):
        """Gradients of (codebook, gamma, beta) from the gradient of the images."""
        codes, h, mean, rstd, step = saved
        da = T.convolution_nd(dy, self.w2, channels_last=True, **self.ATTRS)
        dh, dgamma, dbeta = T.group_norm_backward_nd(da, h, mean, rstd, self.groups, self.gamma, self.beta,
                                                     **self.norm_options(step))
        dx = T.convolution_nd(dh, self.w1, channels_last=True, **self.ATTRS)
        dcodebook = T.embedding_backward_nd(dx.movedim(1, -1), codes, self.codebook.shape[0], grad_dtype=torch.float32)
        return dcodebook, dgamma, dbeta

    def parameters(self):
        return self.codebook, self.gamma, self.beta


def train(steps=20, images=4, grid=16, lr=0.3, seed=1, model=None):
    """Fits random targets; the mean squared error of each step."""
    model = model or TokenDecoder()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, model.codebook.shape[0], (images, grid, grid), generator=gen, device="cuda")
    shape = (images, 4 * grid, 4 * grid, model.w2.shape[1])
    target = torch.randn(shape, generator=gen, device="cuda").movedim(-1, 1)
    losses = []
    for step in range(steps):
        y, saved = model.forward(codes, step)
        diff = y.float() - target
        losses.append(diff.square().mean())
        # the gradient of the sum of squares over each position's channels: of order one, well
        # inside float16's range; the step size takes up the rest
        grads = model.backward((2.0 * diff / diff.shape[1]).half(), saved)
        for p, g in zip(model.parameters(), grads):
            p -= lr / (images * grid) * g
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args()
    for step, loss in enumerate(train(args.steps)):
        print(f"step {step:3d}  mean squared error {loss:.4f}", flush=True)


if __name__ == "__main__":
    main()

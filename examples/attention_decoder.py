"""Training a token decoder with an attention layer, with the library's operators alone.

A grid of codes is looked up in a codebook (``embedding_nd``) and normalised (``group_norm_nd``); a 1 x 1
convolution makes queries, keys and values side by side (``convolution_nd``, channels-last, so a
position's heads are one row of memory); the queries and keys turn by their row and column (``rotary_nd``,
in place) and the positions look at each other (``attention_nd``, two query heads a key head).  A second
1 x 1 convolution brings the result back beside the lookup, and a transposed convolution doubles the
resolution.  The gradient goes the same way back: the convolutions' are each other's, the rotary turn's is
the inverse turn, attention's computes its probabilities again.  The codebook and the norm's parameters take AdamW steps
(``adamw_nd``), which also write the float16 codebook of the next lookup; the convolutions keep their weights.

    python examples/attention_decoder.py [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import transposed_convolution_amd as T  # noqa: E402


class AttentionDecoder:
    """codes (N, H, W) -> images (N, out, 2H, 2W), float16 activations, float32 parameters."""

    UP = dict(strides=[2, 2], pads=[1, 1, 1, 1])

    def __init__(self, codes=256, width=64, heads=4, kv_heads=2, head=32, out=16, groups=8, state_bits=32, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        randn = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
        self.heads, self.kv_heads, self.head, self.groups = heads, kv_heads, head, groups
        self.sections = (head // 4, head // 4)
        self.codebook = randn(codes, width)
        self.lookup = self.codebook.half()
        self.gamma, self.beta = torch.ones(width, device=device), torch.zeros(width, device=device)
        self.w_qkv = (randn((heads + 2 * kv_heads) * head, width, 1, 1) / width ** 0.5).half()
        self.w_back = (randn(width, heads * head, 1, 1) / (heads * head) ** 0.5).half()
        self.w_up = (randn(width, out, 4, 4) / (4 * width) ** 0.5).half()
        # AdamW's states
        state = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        make = lambda: [torch.zeros(p.shape, dtype=state, device=device) for p in self.parameters()]  # noqa: E731
        scales = lambda: [torch.zeros((p.numel() + 255) // 256, device=device) for p in self.parameters()]  # noqa: E731
        self.m, self.v = make(), make()
        self.scales = {} if state_bits == 32 else dict(m_scales=scales(), v_scales=scales())
        self.betas = (0.9, 0.999 if state_bits == 32 else 0.95)  # what 8 bits can follow
        self.steps = torch.zeros(1, dtype=torch.int64, device=device)

    def parameters(self):
        return self.codebook, self.gamma, self.beta

    def positions(self, codes):
        n, h, w = codes.shape
        grid = torch.cartesian_prod(torch.arange(h, device=codes.device), torch.arange(w, device=codes.device)).reshape(1, h * w, 2)
        return grid.to(torch.int32).expand(n, -1, -1)

    def split(self, packed):
        """Queries, keys and values of a projection (N, T, heads, head)."""
        h, hk = self.heads, self.kv_heads
        return packed[:, :, :h], packed[:, :, h:h + hk], packed[:, :, h + hk:]

    def forward(self, codes):
        n, gh, gw = codes.shape
        x = T.embedding_nd(codes, self.lookup).movedim(-1, 1)  # channels-last (N, width, H, W)
        y, mean, rstd = T.group_norm_nd(x, self.groups, self.gamma, self.beta)
        p = T.convolution_nd(y, self.w_qkv, channels_last=True)
        packed = p.movedim(1, -1).reshape(n, gh * gw, -1, self.head)
        places = self.positions(codes)
        turning = packed[:, :, :self.heads + self.kv_heads]
        T.rotary_nd(turning, places, self.sections, out=turning)
        q, k, v = self.split(packed)
        a, lse = T.attention_nd(q, k, v)
        z = T.convolution_nd(a.reshape(n, gh, gw, -1).movedim(-1, 1), self.w_back, channels_last=True)
        z += x
        image = T.convtranspose_nd(z, self.w_up, channels_last=True, **self.UP)
        return image, (codes, x, mean, rstd, packed, places, a, lse)

    def backward(self, dimage, saved):
        """Gradients of (codebook, gamma, beta) from the gradient of the images."""
        codes, x, mean, rstd, packed, places, a, lse = saved
        n, gh, gw = codes.shape
        dz = T.convolution_nd(dimage, self.w_up, channels_last=True, **self.UP)
        da = T.convtranspose_nd(dz, self.w_back, channels_last=True).movedim(1, -1).reshape(a.shape)
        q, k, v = self.split(packed)
        dq, dk, dv = T.attention_backward_nd(da, q, k, v, a, lse)
        dpacked = torch.empty_like(packed)
        for part, whole in zip((dq, dk), self.split(dpacked)):
            T.rotary_nd(part, places, self.sections, inverse=True, out=whole)
        self.split(dpacked)[2].copy_(dv)
        dy = T.convtranspose_nd(dpacked.reshape(n, gh, gw, -1).movedim(-1, 1), self.w_qkv, channels_last=True)
        dx, dgamma, dbeta = T.group_norm_backward_nd(dy, x, mean, rstd, self.groups, self.gamma, self.beta)
        dx += dz
        dcodebook = T.embedding_backward_nd(dx.movedim(1, -1), codes, self.codebook.shape[0], grad_dtype=torch.float32)
        return dcodebook, dgamma, dbeta

    def update(self, grads, lr):
        self.steps += 1
        T.adamw_nd(self.parameters(), grads, self.m, self.v, lr=lr, step=self.steps, betas=self.betas, weight_decay=(0.01, 0.0, 0.0),
                   copies=(self.lookup, None, None), **self.scales)


def train(steps=20, images=4, grid=16, lr=0.02, seed=1, model=None):
    """Fits random targets; the mean squared error of each step."""
    model = model or AttentionDecoder()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, model.codebook.shape[0], (images, grid, grid), generator=gen, device="cuda")
    target = torch.randn((images, 2 * grid, 2 * grid, model.w_up.shape[1]), generator=gen, device="cuda").movedim(-1, 1)
    losses = []
    for _ in range(steps):
        y, saved = model.forward(codes)
        diff = y.float() - target
        losses.append(diff.square().mean())
        # the gradient of the sum of squares over each position's channels: of order one
        model.update(model.backward((2.0 * diff / diff.shape[1]).half(), saved), lr)
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args()
    for step, loss in enumerate(train(args.steps)):
        print(f"step {step:3d}  mean squared error {loss:.4f}", flush=True)


if __name__ == "__main__":
    main()

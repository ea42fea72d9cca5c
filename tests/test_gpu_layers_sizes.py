"""Group norm of very many small images on the GPU, against the plain 64-bit forms."""
import numpy as np
import pytest
import torch

import layer_refs as R
from test_gpu_layers import T, host, norm_inputs, rows_of  # noqa: F401

pytestmark = pytest.mark.gpu


def test_two_million_images(T):
    """Values of every image, and parameter gradients summed over all of them."""
    n, c, dims = (1 << 21) + 5, 2, (2,)
    print(f"[case] group norm {(n, c, dims)} f16", flush=True)
    x, xv, dy, dyv, ga, gav, be, bev = norm_inputs(n, c, dims, "f16", "f32", 1)
    y, mean, rstd = T.group_norm_nd(x, 1, ga, be, activation="silu")
    want, tol = R.group_norm(xv, 1, gav, bev, 1e-5, "silu")
    for name, got, w, t, dtype in (("y", rows_of(y), want[0], tol[0], "f16"), ("mean", host(mean), want[1], tol[1], "f32"),
                                   ("rstd", host(rstd), want[2], tol[2], "f32")):
        R.assert_close(got, w, t, dtype, name)
    grads = T.group_norm_backward_nd(dy, x, mean, rstd, 1, ga, be, activation="silu")
    want, tol = R.group_norm_grad(dyv, xv, host(mean), host(rstd), 1, gav, bev, "silu")
    R.assert_close(rows_of(grads[0]), want[0], tol[0], "f16", "dx")
    R.assert_close(host(grads[1]), want[1], tol[1], "f32", "dgamma")
    R.assert_close(host(grads[2]), want[2], tol[2], "f32", "dbeta")


def test_sixteen_million_groups(T):
    """Images times groups beyond 2^24: the first, the last and some others of the images."""
    n, c, groups = (1 << 19) + 1, 64, 32
    print(f"[case] group norm {(n, c, 1)} in {groups} f16", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, dy = (torch.randn((n, 1, c), generator=gen, device="cuda").half().movedim(-1, 1) for _ in range(2))
    ga, be = torch.rand(c, generator=gen, device="cuda") + 0.5, torch.randn(c, generator=gen, device="cuda")
    y, mean, rstd = T.group_norm_nd(x, groups, ga, be, activation="silu")
    dx, _, _ = T.group_norm_backward_nd(dy, x, mean, rstd, groups, ga, be, activation="silu")
    some = torch.cat([torch.arange(500), torch.randint(0, n, (500,)), torch.arange(n - 500, n)]).cuda()
    xv, dyv = rows_of(x[some]), rows_of(dy[some])
    want, tol = R.group_norm(xv, groups, host(ga), host(be), 1e-5, "silu")
    R.assert_close(rows_of(y[some]), want[0], tol[0], "f16", "y")
    R.assert_close(host(mean[some]), want[1], tol[1], "f32", "mean")
    R.assert_close(host(rstd[some]), want[2], tol[2], "f32", "rstd")
    want, tol = R.group_norm_grad(dyv, xv, host(mean[some]), host(rstd[some]), groups, host(ga), host(be), "silu")
    R.assert_close(rows_of(dx[some]), want[0], tol[0], "f16", "dx")

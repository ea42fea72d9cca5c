"""Group norm where float32 arithmetic can go wrong: values that are not finite, under every
activation."""
import pytest
import torch

from test_gpu_layers import ACTS, T, norm_inputs, path  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("kind,params", ACTS)
def test_a_diverged_group_is_seen(T, path, kind, params, bad):
    """One value that is not finite leaves its group without statistics: every output of the group
    is NaN under every activation, and so are its gradients, but dbeta of the identity, whose
    derivative depends on nothing.  The other groups and images keep their bits."""
    x, _, dy, _, ga, _, be, _ = norm_inputs(2, 32, (6, 5), "f16", "f32", 3)
    kw = dict(activation=kind, act_params=params)
    clean = T.group_norm_nd(x, 4, ga, be, **kw)
    grads = T.group_norm_backward_nd(dy, x, clean[1], clean[2], 4, ga, be, **kw)
    x = x.clone(memory_format=torch.preserve_format)
    x[1, 9, 2, 2] = float(bad)
    y, mean, rstd = T.group_norm_nd(x, 4, ga, be, **kw)
    dx, dgamma, dbeta = T.group_norm_backward_nd(dy, x, mean, rstd, 4, ga, be, **kw)
    assert torch.isnan(y[1, 8:16]).all()
    assert torch.isnan(dx[1, 8:16]).all() and torch.isnan(dgamma[8:16]).all()
    assert torch.equal(dbeta, grads[2]) if kind == "identity" else torch.isnan(dbeta[8:16]).all()
    for got, want in ((y, clean[0]), (dx, grads[0])):
        assert torch.equal(got[0], want[0])
        for part in (slice(0, 8), slice(16, 32)):
            assert torch.equal(got[1, part], want[1, part])
    for got, want in ((dgamma, grads[1]), (dbeta, grads[2])):
        for part in (slice(0, 8), slice(16, 32)):
            assert torch.equal(got[part], want[part])

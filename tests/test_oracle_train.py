"""The float64 references of the training-side operators, pinned against
PyTorch's float64 autograd and against central differences."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import train


def rng(seed):
    return np.random.default_rng(seed)


def gn_torch(x, groups, gamma, beta, eps, silu, t_isolated):
    n, d, h, w, c = x.shape
    z = x.reshape(n * d, h, w, c).permute(0, 3, 1, 2) if t_isolated else x.permute(0, 4, 1, 2, 3)
    y = F.group_norm(z, groups, gamma, beta, eps)
    y = F.silu(y) if silu else y
    return (y.permute(0, 2, 3, 1) if t_isolated else y.permute(0, 2, 3, 4, 1)).reshape(x.shape)


@pytest.mark.parametrize("t_isolated", [True, False])
@pytest.mark.parametrize("silu", [True, False])
def test_group_norm_matches_autograd(silu, t_isolated):
    r = rng(1)
    x = torch.tensor(r.standard_normal((2, 3, 4, 5, 12)) + 0.5, requires_grad=True)
    gamma = torch.tensor(r.uniform(0.5, 1.5, 12), requires_grad=True)
    beta = torch.tensor(r.standard_normal(12), requires_grad=True)
    dy = r.standard_normal(tuple(x.shape))
    y = gn_torch(x, 4, gamma, beta, 1e-5, silu, t_isolated)
    y.backward(torch.tensor(dy))
    args = (x.detach().numpy(), 4, gamma.detach().numpy(), beta.detach().numpy())
    got, stats, _ = train.group_norm_fwd(*args, eps=1e-5, silu=silu, t_isolated=t_isolated)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    (dx, dg, db), _ = train.group_norm_bwd(dy, *args, stats, silu=silu, t_isolated=t_isolated)
    for mine, theirs in ((dx, x.grad), (dg, gamma.grad), (db, beta.grad)):
        np.testing.assert_allclose(mine, theirs.numpy(), rtol=1e-10, atol=1e-11)


def test_group_norm_gradient_against_differences():
    r = rng(2)
    x, v = r.standard_normal((1, 2, 3, 3, 6)), r.standard_normal((1, 2, 3, 3, 6))
    gamma, beta = r.uniform(0.5, 1.5, 6), r.standard_normal(6)
    dy = r.standard_normal(x.shape)
    kw = dict(silu=True, t_isolated=True)

    def f(z):
        return (train.group_norm_fwd(z, 3, gamma, beta, eps=1e-5, **kw)[0] * dy).sum()

    stats = train.group_norm_fwd(x, 3, gamma, beta, eps=1e-5, **kw)[1]
    (dx, _, _), _ = train.group_norm_bwd(dy, x, 3, gamma, beta, stats, **kw)
    e = 1e-5
    assert abs((f(x + e * v) - f(x - e * v)) / (2 * e) - (dx * v).sum()) < 1e-7


def test_norm_silu_matches_autograd_and_differences():
    r = rng(3)
    v = torch.tensor(r.standard_normal((1, 2, 3, 4, 16)), requires_grad=True)
    gamma = torch.tensor(r.uniform(0.5, 1.5, 16), requires_grad=True)
    dy, dskip = r.standard_normal(tuple(v.shape)), r.standard_normal(tuple(v.shape))
    den = torch.clamp(v.norm(dim=-1, keepdim=True), min=1e-12)
    y = F.silu(v / den * 4.0 * gamma)
    np.testing.assert_allclose(train.norm_silu_fwd(v.detach().numpy(), gamma.detach().numpy()),
                               y.detach().numpy(), rtol=1e-12)
    ((y * torch.tensor(dy)).sum() + (v * torch.tensor(dskip)).sum()).backward()
    (dv, dg, db), _ = train.norm_silu_bwd(v.detach().numpy(), dy, gamma.detach().numpy(), dskip)
    np.testing.assert_allclose(dv, v.grad.numpy(), rtol=1e-10, atol=1e-11)
    np.testing.assert_allclose(dg, gamma.grad.numpy(), rtol=1e-10, atol=1e-11)
    np.testing.assert_allclose(db, v.grad.numpy().reshape(-1, 16).sum(0), rtol=1e-9, atol=1e-10)
    z, e, g = v.detach().numpy(), 1e-5, gamma.detach().numpy()
    w = r.standard_normal(z.shape)

    def f(t):
        return (train.norm_silu_fwd(t, g) * dy).sum()

    diff = (f(z + e * w) - f(z - e * w)) / (2 * e)
    assert abs(diff - ((dv - dskip) * w).sum()) < 1e-6


def test_norm_silu_below_the_clamp_has_no_projection():
    """|value| <= 1e-12: the denominator is the constant 1e-12."""
    v = np.zeros((1, 1, 1, 1, 8))
    dy = np.ones_like(v)
    (dv, dg, _), _ = train.norm_silu_bwd(v, dy, np.full(8, 0.5))
    # sigmoid(0) = 1/2, so da = 1/2
    np.testing.assert_allclose(dv, 0.5 * 0.5 * np.sqrt(8.0) * 1e12)
    assert np.all(dg == 0)

"""Training GroupNorm on groups that are constant, or nearly so, far from zero.

rstd reaches 1 / sqrt(eps) there, some 316, so whatever a difference from the
mean loses appears in the result 316 times as large. In a constant group every
difference from the mean is 0: h is 0, y is beta and dgamma is 0, whatever the
constant; the variance is 0 and rstd 1 / sqrt(eps), rounded to fp32 (half a
step; a step where the fp64 root and quotient fall on the other side).
"""
import numpy as np
import pytest
import torch

from convolution_video_vae_amd.layer import GroupNormTrain
from oracle import train
from test_gpu_train_norms import EPS, check, draw, np64, params

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]
# one work-group per range; units of several pieces; pieces with four rows per
# thread and fewer; one group of several channels per vector; statistics per clip
SHAPES = [((1, 2, 6, 6, 16), 4, True), ((1, 2, 64, 65, 128), 32, True),
          ((1, 1, 61, 67, 96), 32, True), ((2, 2, 20, 24, 64), 4, False)]


def dense(t):
    return t.cuda()


def odd(t):
    """The same as channels 1 and up of a wider tensor: no whole vectors."""
    wide = torch.full((*t.shape[:4], t.shape[4] + 3), 7.0, dtype=t.dtype, device="cuda")
    view = wide[..., 1:1 + t.shape[4]]
    view.copy_(t)
    return view


def constant(shape, groups, dtype, value):
    """Two groups of one value among normal ones, and that value in dtype."""
    x = draw(shape, dtype, 1)
    x[..., :2 * (shape[4] // groups)] = value
    return x, float(x.flatten()[0])


def nearly_constant(shape, dtype, value):
    """A value to which one in four adds a step of its type (fp32: 16 steps)."""
    g = torch.Generator().manual_seed(4)
    step = value * {torch.bfloat16: 2.0 ** -7, torch.float16: 2.0 ** -10,
                    torch.float32: 2.0 ** -20}[dtype]
    return (value + step * (torch.rand(shape, generator=g) < 0.25)).to(dtype)


def forward(x, groups, t_iso, silu, place):
    print(f"[gn_train] {tuple(x.shape)} g={groups} {x.dtype} {place.__name__}", flush=True)
    gamma, beta = params(x.shape[4], 3)
    op = GroupNormTrain(x.shape, groups, eps=EPS, silu=silu, t_isolated=t_iso, dtype=x.dtype)
    xd = place(x)
    y, stats = op.forward(xd, gamma.cuda(), beta.cuda())
    return op, xd, gamma, beta, y, stats


PLACES = pytest.mark.parametrize("place", [dense, odd], ids=["dense", "odd"])
DTYPES = pytest.mark.parametrize("dtype", TYPES, ids=str)
SHAPED = pytest.mark.parametrize("shape,groups,t_iso", SHAPES)


@PLACES
@pytest.mark.parametrize("value", [0.625, -10.0, 1000.0, 30000.0])
@DTYPES
@SHAPED
def test_statistics_of_constant_groups(shape, groups, t_iso, dtype, value, place):
    x, const = constant(shape, groups, dtype, value)
    stats = forward(x, groups, t_iso, False, place)[-1]
    assert torch.all(stats[:, :2, 0] == const)
    want = 1.0 / np.sqrt(float(np.float32(EPS)))
    assert np.all(np.abs(np64(stats)[:, :2, 1] - want) <= 2 * EPS32 * want)


@PLACES
@pytest.mark.parametrize("value", [10.0, 1000.0, 30000.0])
@DTYPES
@SHAPED
def test_statistics_of_nearly_constant_groups(shape, groups, t_iso, dtype, value, place):
    """The mean is rounded to fp32 once, and off by at most 128 roundings of
    twice the spread; the variance by 128 of four times its square."""
    x = nearly_constant(shape, dtype, value)
    got = np64(forward(x, groups, t_iso, True, place)[-1])
    none = np.zeros(shape[4])
    _, ref, _ = train.group_norm_fwd(np64(x), groups, none, none, eps=float(np.float32(EPS)),
                                     silu=False, t_isolated=t_iso)
    spread = float(x.double().max() - x.double().min())
    assert np.all(np.abs(got[..., 0] - ref[..., 0])
                  <= EPS32 * (np.abs(ref[..., 0]) + 256 * spread))
    rel = EPS32 * (4 + 512 * (spread * ref[..., 1]) ** 2)
    assert np.all(np.abs(got[..., 1] - ref[..., 1]) <= rel * ref[..., 1])


@PLACES
@pytest.mark.parametrize("value", [0.625, -10.0, 1000.0, 30000.0])
@DTYPES
@SHAPED
def test_constant_groups(shape, groups, t_iso, dtype, value, place):
    n = 2 * (shape[4] // groups)
    x, _ = constant(shape, groups, dtype, value)
    dy = draw(shape, dtype, 2, 0.1)
    op, xd, gamma, beta, y, stats = forward(x, groups, t_iso, False, place)
    assert torch.equal(y[..., :n].cpu(), beta[:n].to(dtype).expand(*shape[:4], -1))
    dx, dg, db = op.backward(place(dy), xd, gamma.cuda(), beta.cuda(), stats)
    assert torch.all(dg[:n] == 0)
    (rx, rg, rb), (tx, tg, tb) = train.group_norm_bwd(
        np64(dy), np64(x), groups, np64(gamma), np64(beta), np64(stats), silu=False, t_isolated=t_iso)
    check(dx, rx, tx, "dx")
    check(dg, rg, tg, "dgamma")
    check(db, rb, tb, "dbeta")


@PLACES
@pytest.mark.parametrize("value", [10.0, 1000.0, 30000.0])
@DTYPES
@SHAPED
def test_nearly_constant_groups(shape, groups, t_iso, dtype, value, place):
    x = nearly_constant(shape, dtype, value)
    dy = draw(shape, dtype, 5, 0.1)
    op, xd, gamma, beta, y, stats = forward(x, groups, t_iso, True, place)
    kw = dict(silu=True, t_isolated=t_iso)
    ry, _, ty = train.group_norm_fwd(np64(x), groups, np64(gamma), np64(beta),
                                     eps=float(np.float32(EPS)), **kw)
    check(y, ry, ty, "y")
    dx, dg, db = op.backward(place(dy), xd, gamma.cuda(), beta.cuda(), stats)
    (rx, rg, rb), (tx, tg, tb) = train.group_norm_bwd(
        np64(dy), np64(x), groups, np64(gamma), np64(beta), np64(stats), **kw)
    check(dx, rx, tx, "dx")
    check(dg, rg, tg, "dgamma")
    check(db, rb, tb, "dbeta")

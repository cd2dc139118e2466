"""Training-side norms at the sizes where a work-group loops: rows of the
channel norm's backward pass beyond one pass of the grid, and GroupNorm over
units of two passes whose results are stored past the caches. The float64
references are formed on the GPU or by oracle/train.py."""
import numpy as np
import pytest
import torch

from convolution_video_vae_amd.layer import GroupNormTrain, NormSiluBackward
from oracle import train
from test_gpu_train_norms import EPS, HALF, check, draw, np64, params

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24


def lanes(c):
    g = 1
    while g < 64 and 3 * g < c // 8:
        g *= 2
    return g


# channels of every (lanes of a row, vectors of a lane), an odd number of rows
# that the grid's 1024 work-groups pass over two or three times, the last
# pass short
@pytest.mark.parametrize("c,skip,bias,passes", [
    (8, True, True, 2), (16, False, False, 2), (24, True, False, 2), (32, False, True, 2),
    (48, True, True, 2), (56, False, True, 2), (96, True, True, 3), (128, False, True, 2),
    (192, True, False, 2), (256, True, True, 2), (384, False, False, 2), (512, True, True, 2),
    (640, False, True, 2), (776, True, True, 2), (1288, False, True, 2), (2048, True, True, 2)])
def test_norm_silu_bwd_over_several_rows(c, skip, bias, passes):
    per = 256 // lanes(c)                       # rows of a work-group's pass
    rows = 1024 * per * (passes - 1) + 337 * per + 1
    shape = (1, 1, 1, rows, c)
    print(f"[ns_bwd] {shape} skip={skip} bias={bias}", flush=True)
    v, dy = draw(shape, torch.bfloat16, c), draw(shape, torch.bfloat16, c + 1, 0.1)
    sk = draw(shape, torch.bfloat16, c + 2, 0.1) if skip else None
    gamma = params(c, c + 3)[0].bfloat16()
    dv, dg, db = NormSiluBackward(shape, bias=bias)(v.cuda(), dy.cuda(), gamma.cuda(),
                                                    dskip=None if sk is None else sk.cuda())
    torch.cuda.synchronize()
    # a thread adds `passes` rows, one thread adds a work-group's `per` of these
    k = passes + per + 8
    (rv, rg, rb), (tv, tg, tb) = train.norm_silu_bwd(np64(v), np64(dy), np64(gamma),
                                                     None if sk is None else np64(sk), k=k)
    check(dv, rv, tv, "dvalue")
    check(dg, rg, tg, "dgamma")
    if bias:
        check(db, rb, tb, "dbias")


def close(got, ref, tol, what):
    half = HALF[got.dtype]
    bad = ~((got.double() - ref).abs() <= tol + half * (ref.abs() + tol) + 2.0 ** -126)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("shape,groups", [((1, 9, 250, 251, 128), 32), ((2, 9, 191, 193, 192), 48)])
def test_two_pass_results_past_the_caches(shape, groups, dtype):
    """More than 128 MB of results over statistics units of more pieces than
    exchange sums. The bounds are those of oracle/train.py, on the GPU."""
    n, c = shape[0], shape[4]
    assert np.prod(shape) * dtype.itemsize > 128 << 20
    print(f"[gn_train] {shape} g={groups} {dtype}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(c)
    x = (torch.randn(shape, generator=g, device="cuda") + 0.5).to(dtype)
    dy = (torch.randn(shape, generator=g, device="cuda") * 0.1).to(dtype)
    gamma, beta = (p.cuda() for p in params(c, 98))
    op = GroupNormTrain(shape, groups, silu=True, t_isolated=False, dtype=dtype)
    y, stats = op.forward(x, gamma, beta)
    dx, dg, db = op.backward(dy, x, gamma, beta, stats)
    k, eps = 128, float(np.float32(EPS))
    dgamma = torch.zeros(c, dtype=torch.float64, device="cuda")
    dbeta, t_dg, t_db = (torch.zeros_like(dgamma) for _ in range(3))
    for i in range(n):
        shaped = (-1, groups, c // groups)
        xg, dg_, g4, b4 = (t.double().reshape(shaped) for t in (x[i], dy[i], gamma, beta))
        var, mean = torch.var_mean(xg, dim=(0, 2), correction=0, keepdim=True)
        rstd = 1.0 / torch.sqrt(var + eps)
        assert torch.all((stats[i, :, 0].double() - mean.view(-1)).abs()
                         <= EPS32 * (mean.view(-1).abs() + 2 * k * 6))
        h = (xg - mean) * rstd
        a = h * g4 + b4
        spread = (xg - mean).abs().amax(dim=(0, 2), keepdim=True)
        dm = k * EPS32 * 2 * spread + 2 * EPS32 * mean.abs()
        dr = k * EPS32 * 4 * spread ** 2 * rstd ** 2 + 4 * EPS32
        ref = a * torch.sigmoid(a)
        tol = 1.1 * (g4.abs() * (dm * rstd + h.abs() * (dr + 8 * EPS32)) + 4 * EPS32 * b4.abs())
        close(y[i].reshape(shaped), ref, tol + 8 * EPS32 * ref.abs(), "y")
        mean, rstd = (stats[i, :, j].double().view(1, groups, 1) for j in (0, 1))
        h = (xg - mean) * rstd
        a = h * g4 + b4
        s = torch.sigmoid(a)
        da = dg_ * (s + a * s * (1 - s))
        N = xg.shape[0] * (c // groups)
        db_, dgm = da.sum(dim=0, keepdim=True), (da * h).sum(dim=0, keepdim=True)
        c1 = (g4 * db_).sum(dim=2, keepdim=True) / N
        c2 = (g4 * dgm).sum(dim=2, keepdim=True) / N
        dh = 4 * EPS32 * h.abs()
        dda = dg_.abs() * (0.5 * (g4.abs() * dh + 4 * EPS32 * ((h * g4).abs() + b4.abs()))
                           + 16 * EPS32)
        e1 = (dda + k * EPS32 * da.abs()).sum(dim=0, keepdim=True)
        e2 = (dda * h.abs() + da.abs() * dh + k * EPS32 * (da * h).abs()).sum(dim=0, keepdim=True)
        m1 = (g4.abs() * e1).sum(dim=2, keepdim=True) / N + 2 * EPS32 * c1.abs()
        m2 = (g4.abs() * e2).sum(dim=2, keepdim=True) / N + 2 * EPS32 * c2.abs()
        ref = rstd * (g4 * da - c1 - h * c2)
        tol = rstd * (g4.abs() * dda + m1 + h.abs() * m2 + dh * c2.abs()
                      + 6 * EPS32 * ((g4 * da).abs() + c1.abs() + (h * c2).abs()))
        close(dx[i].reshape(shaped), ref, tol, "dx")
        dgamma += dgm.view(-1)
        dbeta += db_.view(-1)
        t_dg += e2.view(-1)
        t_db += e1.view(-1)
    close(dg, dgamma, t_dg + 2 * EPS32 * dgamma.abs(), "dgamma")
    close(db, dbeta, t_db + 2 * EPS32 * dbeta.abs(), "dbeta")

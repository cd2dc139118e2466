"""The training-side norms against the float64 references of oracle/train.py.

A result may differ from the reference by the reference's bound on fp32
arithmetic (at most `k` = 128 roundings on every summed term: a thread adds
fewer rows than that here) and by the rounding to its own type: half a step,
2^-8 of the value in bf16, 2^-11 in fp16 (2^-25 below its normal numbers),
2^-24 in fp32.
"""
import numpy as np
import pytest
import torch

import convolution_video_vae_amd as cv
from convolution_video_vae_amd.layer import Conv3d, GradClip, GroupNormTrain, NormSiluBackward
from guard import Guarded
from oracle import train

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
EPS = 1e-5


def np64(t):
    return t.detach().double().cpu().numpy()


def check(got, ref, tol, what):
    g = np64(got)
    assert g.shape == ref.shape, what
    half = HALF[got.dtype]
    t = tol + half * (np.abs(ref) + tol) + (2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -126)
    bad = ~(np.abs(g - ref) <= t)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst "
                           f"{np.nanmax(np.abs(g - ref) / t):.3g} of the tolerance")


def draw(shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


def params(c, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.rand(c, generator=g) + 0.5, torch.randn(c, generator=g) * 0.3


def gn_case(shape, groups, dtype, silu, t_iso, *, x=None, place=None, eps=EPS, seed=0, k=128):
    """Forward and backward of one case against the reference; `place` puts
    each activation somewhere on the GPU (default: its own dense tensor)."""
    print(f"[gn_train] {shape} g={groups} {dtype} silu={silu} per_frame={t_iso}", flush=True)
    place = place or (lambda t, what: t.cuda())
    x = draw(shape, dtype, seed) if x is None else x
    dy = draw(shape, dtype, seed + 1, 0.1)
    gamma, beta = params(shape[4], seed + 2)
    op = GroupNormTrain(shape, groups, eps=eps, silu=silu, t_isolated=t_iso, dtype=dtype)
    xd, dyd = place(x, "x"), place(dy, "dy")
    out = place(torch.full(shape, float("nan"), dtype=dtype), "y")
    y, stats = op.forward(xd, gamma.cuda(), beta.cuda(), y=out)
    dx, dg, db = op.backward(dyd, xd, gamma.cuda(), beta.cuda(), stats,
                             dx=place(torch.full(shape, float("nan"), dtype=dtype), "dx"))
    torch.cuda.synchronize()
    kw = dict(silu=silu, t_isolated=t_iso, k=k)
    e32 = float(np.float32(eps))
    ry, rs, ty = train.group_norm_fwd(np64(x), groups, np64(gamma), np64(beta), eps=e32, **kw)
    check(y, ry, ty, "y")
    # mean within its own spread's roundings, rstd relatively
    xs = np.abs(np64(x)).max() * 2 + 1e-30
    assert np.all(np.abs(np64(stats)[..., 0] - rs[..., 0]) <= (k + 2) * 2.0 ** -24 * xs)
    got_stats = np64(stats)
    (rx, rg, rb), (tx, tg, tb) = train.group_norm_bwd(np64(dy), np64(x), groups, np64(gamma),
                                                      np64(beta), got_stats, **kw)
    check(dx, rx, tx, "dx")
    check(dg, rg, tg, "dgamma")
    check(db, rb, tb, "dbeta")
    return y, stats, dx, dg, db


SHAPES = [
    # shape, groups, silu, per frame
    ((1, 1, 1, 1, 1), 1, True, True),            # one value
    ((1, 1, 1, 1, 8), 8, False, True),           # one value per group
    ((2, 3, 1, 1, 64), 32, True, True),          # one-pixel frames
    ((1, 2, 5, 7, 90), 30, False, True),         # no whole vectors per pixel
    ((2, 2, 9, 7, 45), 15, True, False),
    ((1, 3, 8, 8, 45), 15, True, True),          # rows of several pixels
    ((1, 2, 6, 4, 3), 1, True, False),
    ((1, 2, 6, 10, 2048), 256, True, True),
    ((1, 1, 4, 4, 2560), 32, True, True),        # more vectors than threads
    ((1, 1, 3, 5, 4099), 1, True, True),         # one group over many channel tiles
    ((1, 2, 61, 67, 128), 32, True, True),       # many chunks, the last one ragged
    ((2, 4, 6, 7, 64), 32, True, False),
    ((3, 1, 33, 1, 96), 32, False, False),
    ((1, 5, 16, 16, 1024), 32, True, True),
    ((1, 2, 32, 32, 512), 32, True, True),
    ((2, 1, 40, 52, 320), 32, True, True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("shape,groups,silu,t_iso", SHAPES)
def test_group_norm_train(shape, groups, silu, t_iso, dtype):
    gn_case(shape, groups, dtype, silu, t_iso, seed=sum(shape))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("wide,off", [(2, 0), (2, 1), (3, 8), (2, 5)])
def test_channel_slices(dtype, wide, off):
    """Every activation is a channel slice of its own wider tensor, at whole
    and odd vector offsets; what lies beside the slice stays."""
    shape, kept = (2, 2, 5, 6, 64), []

    def place(t, what):
        full = torch.full(shape[:4] + (64 * wide,), 7.0, dtype=dtype, device="cuda")
        view = full[..., off:off + 64]
        view.copy_(t)
        kept.append((full, off))
        return view

    gn_case(shape, 16, dtype, True, False, place=place, seed=5)
    for full, o in kept:
        assert torch.all(full[..., :o] == 7.0) and torch.all(full[..., o + 64:] == 7.0)


def test_y_beside_x_in_one_tensor():
    both = torch.zeros(1, 2, 7, 9, 128, dtype=torch.bfloat16, device="cuda")
    both[..., :64] = draw((1, 2, 7, 9, 64), torch.bfloat16, 3).cuda()
    gamma, beta = (p.cuda() for p in params(64, 4))
    op = GroupNormTrain((1, 2, 7, 9, 64), 32, silu=True)
    y, _ = op.forward(both[..., :64], gamma, beta, y=both[..., 64:])
    ref, _ = op.forward(both[..., :64].contiguous(), gamma, beta)
    assert torch.equal(y, ref)


def test_mean_far_above_spread_and_outliers():
    """Means of 1000 spreads, and groups whose first value is far outside."""
    shape = (1, 2, 40, 52, 64)
    x = draw(shape, torch.float32, 6, std=0.01, mean=10.0)
    gn_case(shape, 16, torch.float32, True, True, x=x, eps=1e-8)
    x = draw(shape, torch.float32, 7)
    x[:, :, 0, 0, ::4] = 300.0
    gn_case(shape, 16, torch.float32, True, True, x=x)


def test_constant_group_is_beta():
    shape = (1, 1, 6, 6, 16)
    x = draw(shape, torch.bfloat16, 8)
    x[..., :4] = 0.625
    y, stats, dx, _, _ = gn_case(shape, 4, torch.bfloat16, False, True, x=x, seed=20)
    _, beta = params(16, 22)
    assert torch.equal(y[..., :4].float().cpu(), beta[:4].bfloat16().float().expand(1, 1, 6, 6, 4))
    assert stats[0, 0, 0].item() == 0.625


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_values_stay_in_their_group(bad):
    shape = (2, 2, 5, 6, 64)
    x = draw(shape, torch.bfloat16, 9)
    gamma, beta = (p.cuda() for p in params(64, 10))
    dy = draw(shape, torch.bfloat16, 11).cuda()
    op = GroupNormTrain(shape, 16, silu=True)
    y0, s0 = op.forward(x.cuda(), gamma, beta)
    dx0, _, _ = op.backward(dy, x.cuda(), gamma, beta, s0)
    x[1, 0, 2, 3, 21] = bad                     # unit 2, group 5 (channels 20 to 23)
    y1, s1 = op.forward(x.cuda(), gamma, beta)
    dx1, dg, db = op.backward(dy, x.cuda(), gamma, beta, s1)
    hit = torch.zeros(shape, dtype=torch.bool, device="cuda")
    hit[1, 0, :, :, 20:24] = True
    for a, b in ((y0, y1), (dx0, dx1)):
        assert torch.isnan(b[hit]).all() and torch.equal(a[~hit], b[~hit])
    # the mean of values with an infinity is that infinity
    assert not torch.isfinite(s1[2, 5, 0]) and torch.isnan(s1[2, 5, 1])
    assert torch.isnan(dg[20:24]).all() and torch.isfinite(dg[:20]).all()
    assert torch.isnan(db[20:24]).all() and torch.isfinite(db[24:]).all()


def test_dx_in_place_of_dy_and_gradients_left_out():
    shape = (1, 3, 9, 11, 64)
    x, dy = draw(shape, torch.bfloat16, 12).cuda(), draw(shape, torch.bfloat16, 13).cuda()
    gamma, beta = (p.cuda() for p in params(64, 14))
    op = GroupNormTrain(shape, 32, silu=True)
    _, stats = op.forward(x, gamma, beta)
    dx, dg, db = op.backward(dy, x, gamma, beta, stats)
    only, a, b = op.backward(dy, x, gamma, beta, stats, need_params=False)
    assert a is None and b is None and torch.equal(only, dx)
    none, a, b = op.backward(dy, x, gamma, beta, stats, need_dx=False)
    assert none is None and torch.equal(a, dg) and torch.equal(b, db)
    same, a, _ = op.backward(dy, x, gamma, beta, stats, dx=dy)
    assert same is dy and torch.equal(dy, dx) and torch.equal(a, dg)


def test_dx_in_place_of_dy_in_units_of_several_pieces():
    shape = (1, 2, 64, 65, 128)
    x, dy = draw(shape, torch.bfloat16, 93), draw(shape, torch.bfloat16, 94)
    gamma, beta = params(128, 95)
    op = GroupNormTrain(shape, 32, silu=True)
    _, stats = op.forward(x.cuda(), gamma.cuda(), beta.cuda())
    dyd = dy.cuda()
    dx, dg, db = op.backward(dyd, x.cuda(), gamma.cuda(), beta.cuda(), stats, dx=dyd)
    (rx, rg, rb), (tx, tg, tb) = train.group_norm_bwd(np64(dy), np64(x), 32, np64(gamma),
                                                      np64(beta), np64(stats), silu=True,
                                                      t_isolated=True)
    check(dx, rx, tx, "dx")
    check(dg, rg, tg, "dgamma")
    check(db, rb, tb, "dbeta")


@pytest.mark.parametrize("shape", [(1, 2, 7, 5, 40), (1, 1, 67, 61, 64)])
def test_nothing_outside_the_outputs_is_written(shape):
    c = shape[4]
    bufs = {k: Guarded(shape) for k in ("y", "dx")}
    small = {k: Guarded((c,), torch.float32) for k in ("dg", "db")}
    stats = Guarded((shape[1], 8, 2), torch.float32)
    x, dy = draw(shape, torch.bfloat16, 15).cuda(), draw(shape, torch.bfloat16, 16).cuda()
    gamma, beta = (p.cuda() for p in params(c, 17))
    d = cv.make_group_norm_train_desc(shape, 8, silu=True)
    n = [cv.conv3d_group_norm_train_workspace_bytes(d, b) for b in (False, True)]
    ws = [Guarded((v // 2,), torch.int16) for v in n]
    cv.conv3d_group_norm_train_fwd(d, x, gamma, beta, bufs["y"].t, stats.t, ws[0].t, n[0])
    cv.conv3d_group_norm_train_bwd(d, dy, x, gamma, beta, stats.t, bufs["dx"].t, small["dg"].t,
                                   small["db"].t, ws[1].t, n[1])
    torch.cuda.synchronize()
    for k, v in {**bufs, **small, "stats": stats, "ws0": ws[0], "ws1": ws[1]}.items():
        v.assert_intact(k)
    for v in (*bufs.values(), *small.values(), stats):
        assert torch.isfinite(v.t.float()).all()


def test_gradient_against_differences():
    """The kernel's dx along a direction against central differences of the
    kernel's own fp32 forward pass: a step e leaves an error of order e^2 and
    a rounding of 2^-24 |f| / e, about 1e-3 of the slope at e = 1e-2."""
    shape = (1, 2, 6, 6, 24)
    x, v = (draw(shape, torch.float32, s).cuda() for s in (18, 19))
    dy = draw(shape, torch.float32, 20).cuda()
    gamma, beta = (p.cuda() for p in params(24, 21))
    op = GroupNormTrain(shape, 6, silu=True, dtype=torch.float32)
    _, stats = op.forward(x, gamma, beta)
    dx, _, _ = op.backward(dy, x, gamma, beta, stats)
    e = 1e-2
    up, dn = (op.forward(x + s * e * v, gamma, beta)[0].double() for s in (1, -1))
    slope = float(((up - dn) * dy.double()).sum()) / (2 * e)
    mine = float((dx.double() * v.double()).sum())
    scale = float((dx.double() * v.double()).abs().sum())
    assert abs(slope - mine) < 1e-3 * scale


def test_full_size_activation():
    """[1,17,256,256,128] bf16, whose results are stored past the caches: the
    first and last frames against the reference, the parameters' gradients
    against the sum of the frames' own."""
    shape = (1, 17, 256, 256, 128)
    g = torch.Generator(device="cuda").manual_seed(96)
    x = torch.randn(shape, generator=g, device="cuda").bfloat16()
    dy = (torch.randn(shape, generator=g, device="cuda") * 0.1).bfloat16()
    gamma, beta = params(128, 97)
    op = GroupNormTrain(shape, 32, silu=True)
    one = GroupNormTrain((1, 1) + shape[2:], 32, silu=True)
    y, stats = op.forward(x, gamma.cuda(), beta.cuda())
    dx, dg, db = op.backward(dy, x, gamma.cuda(), beta.cuda(), stats)
    kw = dict(silu=True, t_isolated=True)
    for f in (0, 16):
        at = slice(f, f + 1)
        ry, _, ty = train.group_norm_fwd(np64(x[:, at]), 32, np64(gamma), np64(beta),
                                         eps=float(np.float32(EPS)), **kw)
        check(y[:, at], ry, ty, f"y of frame {f}")
        (rx, _, _), (tx, _, _) = train.group_norm_bwd(np64(dy[:, at]), np64(x[:, at]), 32,
                                                      np64(gamma), np64(beta), np64(stats[at]), **kw)
        check(dx[:, at], rx, tx, f"dx of frame {f}")
    each = [one.backward(dy[:, f:f + 1], x[:, f:f + 1], gamma.cuda(), beta.cuda(), stats[f:f + 1],
                         need_dx=False) for f in range(17)]
    # both sides: at most 128 roundings on terms of |da|(|h| + 1) < 0.2 on
    # average, over 17 * 65536 pixels
    tol = 2 * 130 * 2.0 ** -24 * 0.2 * 17 * 65536
    assert (sum(e[1].double() for e in each) - dg.double()).abs().max() < tol
    assert (sum(e[2].double() for e in each) - db.double()).abs().max() < tol


def test_more_than_2_to_32_bytes():
    """5.4 GB of activations: the last frame's results are those of a call on
    that frame alone, up to the roundings of another chunking."""
    shape = (1, 10, 1024, 1024, 256)
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_()
    gamma, beta = (p.cuda() for p in params(256, 23))
    op = GroupNormTrain(shape, 32, silu=True)
    one = GroupNormTrain((1, 1) + shape[2:], 32, silu=True)
    y, stats = op.forward(x, gamma, beta)
    y1, s1 = one.forward(x[:, 9:], gamma, beta)
    # both means are off by at most k 2^-24 of the spread (5 of a normal
    # draw's 10), k = 2^20 pixels / 1024 chunks / 8 lanes = 128 here
    assert torch.allclose(stats[9], s1[0], rtol=0, atol=2 * 130 * 2.0 ** -24 * 10)
    diff = (y[:, 9:].float() - y1.float()).abs()
    assert torch.all(diff <= 2 * 2.0 ** -8 * (y1.float().abs() + 1e-3))
    dx, dg, db = op.backward(y, x, gamma, beta, stats)
    dx1, _, _ = one.backward(y[:, 9:], x[:, 9:], gamma, beta, stats[9:])
    diff = (dx[:, 9:].float() - dx1.float()).abs()
    assert torch.all(diff <= 2 * 2.0 ** -8 * (dx1.float().abs() + 1e-3))
    assert torch.isfinite(dg).all() and torch.isfinite(db).all()


def replay_check(run, inputs, refill):
    """Captures run() and replays it, with eager work and synchronisations
    between, against eager results on the same inputs."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run()
    for i in range(3):
        refill(i)
        want = [o.clone() for o in run()]
        torch.cuda.synchronize()
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), f"replay {i}"


@pytest.mark.parametrize("shape", [(1, 3, 24, 20, 128), (1, 2, 64, 65, 128), (1, 2, 61, 67, 45)])
def test_graph_replays(shape):
    c = shape[4]
    x, dy = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gamma, beta = (p.cuda() for p in params(c, 24))
    op = GroupNormTrain(shape, 32 if c == 128 else 15, silu=True)
    ns = NormSiluBackward(shape, bias=True) if c % 8 == 0 else None

    def run():
        y, stats = op.forward(x, gamma, beta)
        outs = [y, stats, *op.backward(dy, x, gamma, beta, stats)]
        return outs + (list(ns(x, dy, gamma.bfloat16())) if ns else [])

    def refill(i):
        x.copy_(draw(shape, torch.bfloat16, 30 + i))
        dy.copy_(draw(shape, torch.bfloat16, 40 + i))

    refill(9)
    replay_check(run, (x, dy), refill)


def test_two_graphs_side_by_side():
    """Two graphs captured from one object, replayed on two streams at once:
    each has its scratch memory in its own pool."""
    shape = (1, 4, 96, 96, 128)
    op = GroupNormTrain(shape, 32, silu=True)
    gamma, beta = (p.cuda() for p in params(128, 27))
    xs = [draw(shape, torch.bfloat16, 60 + i).cuda() for i in range(2)]
    want = []
    for x in xs:
        y, st = op.forward(x, gamma, beta)
        want.append((y, st, *op.backward(x, x, gamma, beta, st)))
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y, st = op.forward(x, gamma, beta)
            outs.append((y, st, *op.backward(x, x, gamma, beta, st)))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_two_streams_at_once():
    shape = (1, 4, 96, 96, 128)
    op = GroupNormTrain(shape, 32, silu=True)
    gamma, beta = (p.cuda() for p in params(128, 25))
    xs = [draw(shape, torch.bfloat16, 50 + i).cuda() for i in range(2)]
    want = [op.forward(x, gamma, beta) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for _ in range(4):
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                y, st = op.forward(x, gamma, beta)
                got.append((y, st, op.backward(x, x, gamma, beta, st)))
    torch.cuda.synchronize()
    ref = [op.backward(x, x, gamma, beta, w[1]) for x, w in zip(xs, want)]
    for i, (y, st, b) in enumerate(got):
        assert torch.equal(y, want[i % 2][0]) and torch.equal(st, want[i % 2][1])
        assert all(torch.equal(p, q) for p, q in zip(b, ref[i % 2]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("shape,groups", [((1, 2, 64, 65, 128), 32), ((1, 1, 61, 67, 96), 32),
                                          ((2, 1, 48, 50, 320), 32), ((1, 1, 40, 41, 64), 1),
                                          ((1, 2, 33, 31, 512), 16)])
def test_pieces_that_help_themselves_agree_bit_for_bit(shape, groups, dtype, monkeypatch):
    """Units of several pieces: with a bound of no polls at all every
    work-group forms its unit's sums alone, and nothing changes."""
    x, dy = (draw(shape, dtype, 90 + i).cuda() for i in range(2))
    gamma, beta = (p.cuda() for p in params(shape[4], 92))
    op = GroupNormTrain(shape, groups, silu=True, dtype=dtype)
    y, stats = op.forward(x, gamma, beta)
    want = (y, stats, *op.backward(dy, x, gamma, beta, stats))
    torch.cuda.synchronize()
    monkeypatch.setenv("CONV3D_GN_SPIN", "0")
    y, stats = op.forward(x, gamma, beta)
    got = (y, stats, *op.backward(dy, x, gamma, beta, stats))
    torch.cuda.synchronize()
    for a, b, what in zip(got, want, ("y", "stats", "dx", "dgamma", "dbeta")):
        assert torch.equal(a, b), what


BIG_SHAPES = [
    # units of several pieces (exchanged), and units too large for that
    ((1, 2, 128, 130, 128), 32, True, True), ((1, 1, 96, 100, 256), 32, False, True),
    ((2, 3, 32, 40, 64), 8, True, False), ((1, 1, 100, 90, 96), 32, True, True),
    ((1, 1, 64, 64, 480), 30, True, True), ((1, 1, 700, 720, 16), 4, True, True),
    ((1, 1, 50, 60, 1024), 4, True, True),
    # groups of 64 and 128 channels
    ((1, 2, 30, 31, 256), 2, True, True), ((1, 1, 50, 60, 512), 4, False, True),
    ((1, 1, 30, 40, 192), 3, True, False), ((2, 1, 3, 5, 256), 4, True, True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("shape,groups,silu,t_iso", BIG_SHAPES)
def test_group_norm_train_in_pieces(shape, groups, silu, t_iso, dtype):
    """k: a thread adds at most 16 rows of a piece, or, in two passes, its
    share of 504000 pixels in 2048 chunks."""
    gn_case(shape, groups, dtype, silu, t_iso, seed=sum(shape))


# ------------------------------------------------------- channel norm + SiLU

def ns_case(shape, *, skip=False, bias=True, value=None, seed=0):
    print(f"[ns_bwd] {shape} skip={skip}", flush=True)
    v = draw(shape, torch.bfloat16, seed) if value is None else value
    dy = draw(shape, torch.bfloat16, seed + 1, 0.1)
    sk = draw(shape, torch.bfloat16, seed + 2, 0.1) if skip else None
    gamma = params(shape[4], seed + 3)[0].bfloat16()
    dv, dg, db = NormSiluBackward(shape, bias=bias)(v.cuda(), dy.cuda(), gamma.cuda(),
                                                    dskip=None if sk is None else sk.cuda())
    torch.cuda.synchronize()
    (rv, rg, rb), (tv, tg, tb) = train.norm_silu_bwd(np64(v), np64(dy), np64(gamma),
                                                     None if sk is None else np64(sk))
    check(dv, rv, tv, "dvalue")
    check(dg, rg, tg, "dgamma")
    if bias:
        check(db, rb, tb, "dbias")
    else:
        assert db is None


@pytest.mark.parametrize("c", [8, 16, 24, 40, 64, 96, 128, 160, 200, 256, 320, 384, 512, 640, 1024,
                               1288, 2048])
def test_norm_silu_bwd(c):
    ns_case((1, 2, 5, 7, c), skip=c % 3 == 0, seed=c)


@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 8), (1, 1, 1, 1, 2048), (2, 3, 1, 1, 96),
                                   (1, 5, 16, 30, 640), (3, 1, 67, 61, 96)])
def test_norm_silu_bwd_rows(shape):
    ns_case(shape, skip=True, bias=shape[4] != 96, seed=7)


def test_norm_silu_bwd_zero_tiny_and_non_finite_rows():
    shape = (1, 1, 4, 4, 64)
    v = draw(shape, torch.bfloat16, 60)
    v[0, 0, 0, 0] = 0.0
    v[0, 0, 0, 1] = 1e-14                       # below the clamp
    v[0, 0, 0, 2] *= 1e6
    ns_case(shape, value=v, seed=61)
    dy = draw(shape, torch.bfloat16, 62)
    gamma = params(64, 63)[0].bfloat16().cuda()
    op = NormSiluBackward(shape, bias=True)
    clean, _, _ = op(v.cuda(), dy.cuda(), gamma)
    v[0, 0, 2, 1, 5] = float("nan")
    got, dg, db = op(v.cuda(), dy.cuda(), gamma)
    assert torch.isnan(got[0, 0, 2, 1]).all() and torch.isnan(dg).all() and torch.isnan(db).all()
    got[0, 0, 2, 1] = clean[0, 0, 2, 1]
    assert torch.equal(got, clean)


def test_norm_silu_bwd_in_place_and_guarded():
    shape = (1, 2, 9, 13, 160)
    v, dy, sk = (draw(shape, torch.bfloat16, 70 + i).cuda() for i in range(3))
    gamma = params(160, 73)[0].bfloat16().cuda()
    op = NormSiluBackward(shape, bias=True)
    dv, dg, db = op(v, dy, gamma, dskip=sk)
    no, a, b = NormSiluBackward(shape, gamma=False)(v, dy, gamma, dskip=sk)
    assert a is None and b is None and torch.equal(no, dv)
    for k in ("dy", "sk"):
        t = {"dy": dy.clone(), "sk": sk.clone()}
        got, a, b = op(v, t["dy"], gamma, dskip=t["sk"], dvalue=t[k])
        assert torch.equal(got, dv) and torch.equal(a, dg) and torch.equal(b, db)
    out = Guarded(shape)
    small = [Guarded((160,), torch.float32) for _ in range(2)]
    n = cv.conv3d_norm_silu_bwd_workspace_bytes(*shape)
    ws = Guarded((n // 2,), torch.int16)
    cv.conv3d_norm_silu_bwd(v, dy, sk, *shape, gamma, out.t, small[0].t, small[1].t, ws.t, n)
    torch.cuda.synchronize()
    for g in (out, ws, *small):
        g.assert_intact("norm_silu_bwd")
    assert torch.equal(out.t, dv) and torch.equal(small[0].t, dg) and torch.equal(small[1].t, db)


def test_norm_silu_bwd_more_than_2_to_32_bytes():
    shape = (1, 9, 1024, 1024, 256)
    v = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_()
    gamma = params(256, 74)[0].bfloat16().cuda()
    dv, dg, _ = NormSiluBackward(shape)(v, v, gamma)
    last, _, _ = NormSiluBackward((1, 1) + shape[2:])(v[:, 8:], v[:, 8:], gamma)
    assert torch.equal(dv[:, 8:], last) and torch.isfinite(dg).all()


# ------------------------------------------------------------------ together

def test_conv_norm_backward_clip_chain():
    """conv -> GroupNorm + SiLU (statistics kept) -> channel norm + SiLU, its
    gradients back to the conv's output, then all parameter gradients clipped
    by their global norm: each step against the reference on the values that
    the step before it produced."""
    shape = (1, 3, 10, 12, 64)
    w = draw((64, 64, 3, 3, 3), torch.bfloat16, 80, 0.03).cuda()
    x = draw(shape, torch.bfloat16, 81).cuda()
    gamma, beta = params(64, 82)
    g2 = params(64, 83)[0].bfloat16()
    dy = draw(shape, torch.bfloat16, 84, 0.1)
    conv = Conv3d(w, shape, pad_lo=(2, 1, 1), pad_hi=(0, 1, 1))
    op = GroupNormTrain(shape, 32, silu=True)
    a = conv(x)
    b, stats = op.forward(a, gamma.cuda(), beta.cuda())
    db_, dg2, dbias = NormSiluBackward(shape, bias=True)(b, dy.cuda(), g2.cuda())
    da, dgamma, dbeta = op.backward(db_, a, gamma.cuda(), beta.cuda(), stats)
    grads = [da, dgamma, dbeta, dg2, dbias]
    before = [np64(t) for t in grads]
    norm = GradClip(grads).clip(0.5)
    torch.cuda.synchronize()
    ry, _, ty = train.group_norm_fwd(np64(a), 32, np64(gamma), np64(beta), eps=float(np.float32(EPS)),
                                     silu=True, t_isolated=True)
    check(b, ry, ty, "b")
    (rv, rg2, rbias), (tv, tg2, tbias) = train.norm_silu_bwd(np64(b), np64(dy), np64(g2))
    check(db_, rv, tv, "db")
    (ra, rg, rb), (ta, tg, tb) = train.group_norm_bwd(np64(db_), np64(a), 32, np64(gamma),
                                                      np64(beta), np64(stats), silu=True,
                                                      t_isolated=True)
    total = np.sqrt(sum((t ** 2).sum() for t in before))
    coef = min(1.0, 0.5 / (total + 1e-6))
    assert coef < 1 and abs(norm.item() - total) <= 2.0 ** -23 * total
    for t, pre, ref, tol, what in zip(grads, before, (ra, rg, rb, rg2, rbias),
                                      (ta, tg, tb, tg2, tbias),
                                      ("dx", "dgamma", "dbeta", "dgamma2", "dbias")):
        half = 2.0 ** -8 if t.dtype == torch.bfloat16 else 2.0 ** -24
        assert np.all(np.abs(pre - ref) <= tol + half * (np.abs(ref) + tol)), what
        # coef in fp32, the product in fp32, the result in its own type
        assert np.all(np.abs(np64(t) - pre * coef) <= (half + 2.0 ** -22) * np.abs(pre * coef)), what

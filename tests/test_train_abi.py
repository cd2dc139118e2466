"""Refusals of the training-side entry points: every check runs on the host,
so fake (aligned, never dereferenced) addresses are enough."""
import ctypes

import pytest
import torch

import convolution_video_vae_amd as cv
from convolution_video_vae_amd import layer


def at(k):
    return (k + 1) << 34          # far apart, 16-byte aligned


NULL, SHAPE, ALIGN, OVERLAP, WORKSPACE, UNSUPPORTED = 1, 2, 3, 4, 5, 6


def status(f, *args, **kw):
    with pytest.raises(cv.Conv3dError) as e:
        f(*args, **kw)
    return e.value.status


def gn(shape=(1, 2, 4, 4, 64), groups=32, **kw):
    return cv.make_group_norm_train_desc(shape, groups, **kw)


def fwd(d, x=at(0), gamma=at(1), beta=at(2), y=at(3), stats=at(4), ws=at(5), n=1 << 30):
    cv.conv3d_group_norm_train_fwd(d, x, gamma, beta, y, stats, ws, n, stream=0)


def bwd(d, dy=at(6), x=at(0), gamma=at(1), beta=at(2), stats=at(4), dx=at(3), dgamma=at(7),
        dbeta=at(8), ws=at(5), n=1 << 30):
    cv.conv3d_group_norm_train_bwd(d, dy, x, gamma, beta, stats, dx, dgamma, dbeta, ws, n, stream=0)


def test_structs_match_the_header():
    assert ctypes.sizeof(cv.conv3d_group_norm_train_desc) == 10 * 4 + 3 * 8
    assert ctypes.sizeof(cv.conv3d_grad) == 2 * 8 + 8 + 2 * 4


@pytest.mark.parametrize("kw,want", [
    (dict(shape=(0, 2, 4, 4, 64)), SHAPE), (dict(shape=(1, 2, 4, 4, 0)), SHAPE),
    (dict(groups=0), SHAPE), (dict(groups=31), SHAPE), (dict(eps=0.0), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
    (dict(x_pitch=63), SHAPE), (dict(y_pitch=1), SHAPE), (dict(dx_pitch=-64), SHAPE),
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED),
    (dict(shape=(1, 1, 1, 1, 65537), groups=1), UNSUPPORTED),
    (dict(shape=(1 << 15, 1 << 15, 1 << 15, 1 << 15, 64)), UNSUPPORTED),
    (dict(shape=(1 << 20, 1, 1, 1, 32), groups=32), UNSUPPORTED),
    (dict(x_pitch=1 << 50), UNSUPPORTED),
])
def test_group_norm_train_descriptors_refused(kw, want):
    d = gn(**kw)
    assert status(fwd, d) == want
    assert status(bwd, d) == want
    for back in (False, True):
        assert status(cv.conv3d_group_norm_train_workspace_bytes, d, back) == want


def test_group_norm_train_pointers_refused():
    d = gn()
    for k in ("x", "gamma", "beta", "y", "stats"):
        assert status(fwd, d, **{k: None}) == NULL
    for k in ("dy", "x", "gamma", "beta", "stats"):
        assert status(bwd, d, **{k: None}) == NULL
    assert status(bwd, d, dx=None, dgamma=None, dbeta=None) == NULL
    assert status(fwd, d, x=at(0) + 1) == ALIGN
    assert status(fwd, gn(dtype=cv.ELT_FP32), y=at(3) + 2) == ALIGN
    assert status(fwd, d, stats=at(4) + 2) == ALIGN
    assert status(bwd, d, dgamma=at(7) + 1) == ALIGN
    for f, back in ((fwd, False), (bwd, True)):
        need = cv.conv3d_group_norm_train_workspace_bytes(d, back)
        assert status(f, d, n=need - 1) == WORKSPACE
        assert status(f, d, ws=None) == WORKSPACE
        assert status(f, d, ws=at(5) + 8) == ALIGN


def test_group_norm_train_overlaps_refused():
    d, size = gn(), 2 * 4 * 4 * 64 * 2
    assert status(fwd, d, y=at(0)) == OVERLAP                 # y may not be x
    assert status(fwd, d, y=at(0) + size - 2) == OVERLAP
    assert status(fwd, d, stats=at(0) + 16) == OVERLAP
    assert status(fwd, d, ws=at(3) + 16) == OVERLAP
    assert status(fwd, d, y=at(1)) == OVERLAP
    assert status(bwd, d, dx=at(0)) == OVERLAP                # dx may be dy, not x
    assert status(bwd, d, dx=at(6) + 16) == OVERLAP
    assert status(bwd, gn(dx_pitch=128), dx=at(6)) == OVERLAP  # dy's place, another pitch
    assert status(bwd, d, dbeta=at(7)) == OVERLAP
    assert status(bwd, d, dgamma=at(4)) == OVERLAP
    assert status(bwd, d, dx=at(4)) == OVERLAP
    # channels of one wide tensor: 64 of 128, and one element too near
    wide = gn(x_pitch=128, y_pitch=128)
    assert status(fwd, wide, y=at(0) + 126) == OVERLAP
    assert status(fwd, wide, y=at(0) + 130) == OVERLAP
    assert status(fwd, wide, y=at(0) + 128, n=0) == WORKSPACE     # told apart
    assert status(fwd, wide, x=at(0) + 128, y=at(0), gamma=at(0) + 256) == OVERLAP


def ns(shape=(1, 2, 4, 4, 64), value=at(0), dy=at(1), dskip=None, gamma=at(2), dvalue=at(3),
       dgamma=at(4), dbias=at(5), ws=at(6), n=1 << 30):
    cv.conv3d_norm_silu_bwd(value, dy, dskip, *shape, gamma, dvalue, dgamma, dbias, ws, n, stream=0)


def test_norm_silu_bwd_refusals():
    for k in ("value", "dy", "gamma", "dvalue"):
        assert status(ns, **{k: None}) == NULL
    assert status(ns, shape=(1, 0, 4, 4, 64)) == SHAPE
    assert status(ns, shape=(1, 2, 4, 4, 60)) == ALIGN
    assert status(ns, shape=(1, 2, 4, 4, 2056)) == UNSUPPORTED
    assert status(ns, shape=(1 << 15, 1 << 15, 1 << 15, 1, 64)) == UNSUPPORTED
    for k in ("value", "dy", "dskip", "gamma", "dvalue", "ws"):
        assert status(ns, **{k: at(9) + 8}) == ALIGN
    assert status(ns, dbias=at(5) + 2) == ALIGN
    need = cv.conv3d_norm_silu_bwd_workspace_bytes(1, 2, 4, 4, 64)
    assert status(ns, n=need - 1) == WORKSPACE
    assert status(ns, ws=None, dbias=None) == WORKSPACE
    assert status(ns, dvalue=at(0)) == OVERLAP
    assert status(ns, dvalue=at(1) + 16) == OVERLAP
    assert status(ns, dgamma=at(0)) == OVERLAP
    assert status(ns, dbias=at(4)) == OVERLAP
    assert status(ns, ws=at(3)) == OVERLAP
    assert status(ns, dskip=at(4)) == OVERLAP


def grads(*entries):
    return cv.make_grads([(g, o, n, dt, odt) for g, o, n, dt, odt in entries])


def clip(table, norm=at(20), ws=at(21), n=1 << 30, kind=0, max_norm=1.0):
    cv.conv3d_grad_clip(table, kind, max_norm, norm, ws, n, stream=0)


B, H, F = cv.ELT_BF16, cv.ELT_FP16, cv.ELT_FP32


def test_grad_refusals():
    ok = (at(0), None, 1000, B, B)
    for f in (clip, lambda t, **kw: cv.conv3d_grad_norm(
            t, kw.get("kind", 0), kw.get("norm", at(20)), kw.get("ws", at(21)),
            kw.get("n", 1 << 30), stream=0)):
        assert status(f, grads((None, None, 10, B, B))) == NULL
        assert status(f, grads(ok), norm=None) == NULL
        assert status(f, grads((at(0), None, -1, B, B))) == SHAPE
        assert status(f, grads((at(0), None, 10, 7, B))) == UNSUPPORTED
        assert status(f, grads((at(0), None, 10, B, 7))) == UNSUPPORTED
        assert status(f, grads((at(0), None, (1 << 40) + 1, B, B))) == UNSUPPORTED
        assert status(f, grads(ok), kind=2) == UNSUPPORTED
        assert status(f, grads((at(0) + 1, None, 10, B, B))) == ALIGN
        assert status(f, grads(ok), norm=at(20) + 2) == ALIGN
        assert status(f, grads(ok), ws=None) == WORKSPACE
        assert status(f, grads(ok), n=7) == WORKSPACE
        assert status(f, grads(ok), ws=at(21) + 4) == ALIGN
        assert status(f, grads(ok), norm=at(0) + 4) == OVERLAP
        assert status(f, grads(ok), norm=at(21)) == OVERLAP
        assert status(f, grads(ok), ws=at(0)) == OVERLAP
    for bad in (-1.0, float("nan"), float("inf")):
        assert status(clip, grads(ok), max_norm=bad) == SHAPE
    assert status(clip, grads(ok, ok)) == OVERLAP                       # twice, in place
    assert status(clip, grads(ok, (at(0) + 1998, None, 10, B, B))) == OVERLAP
    assert status(clip, grads((at(0), at(0), 10, B, F))) == OVERLAP     # in place, another type
    assert status(clip, grads((at(0), None, 10, B, F))) == OVERLAP
    assert status(clip, grads((at(0), at(0) + 2, 10, B, B))) == OVERLAP
    assert status(clip, grads((at(0), at(1), 10, B, B), (at(2), at(1), 10, B, B))) == OVERLAP
    assert status(clip, grads((at(0), at(1) + 2, 10, B, F))) == ALIGN
    # the same gradient into two outs is only read twice: it passes to the next check
    assert status(clip, grads((at(0), at(1), 10, B, B), (at(0), at(2), 10, B, B)), n=0) == WORKSPACE


def test_grad_workspace_holds_one_partial_per_work_group():
    one = cv.conv3d_grad_workspace_bytes(grads((at(0), None, 1, B, B)))
    big = cv.conv3d_grad_workspace_bytes(grads((at(0), None, 1 << 30, B, B)))
    assert one == 256 and 1024 * 8 < big <= 2048 * 8
    assert cv.conv3d_grad_workspace_bytes(grads((at(0), None, 0, B, B))) == 256


def test_layer_checks_refuse_host_and_odd_tensors():
    with pytest.raises(ValueError, match="dtype"):
        layer.GroupNormTrain((1, 1, 2, 2, 8), 2, dtype=torch.float64)
    g = layer.GroupNormTrain((1, 1, 2, 2, 8), 2)
    x = torch.zeros(1, 1, 2, 2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        g.forward(x, torch.ones(8), torch.ones(8))
    with pytest.raises(ValueError, match="GPU"):
        layer.NormSiluBackward((1, 1, 2, 2, 8))(x, x, torch.ones(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="no gradients"):
        layer.GradClip([])
    with pytest.raises(ValueError, match="dense"):
        layer.GradClip([torch.zeros(4)])
    with pytest.raises(ValueError, match="norm must be"):
        layer.GradClip([torch.zeros(4)], norm="l1")
    with pytest.raises(ValueError, match="outs"):
        layer.GradClip([torch.zeros(4)], [])


def test_pixel_pitch():
    t = torch.zeros(2, 3, 4, 5, 16)
    assert layer._pixel_pitch(t) == 16
    assert layer._pixel_pitch(t[..., 3:11]) == 16
    assert layer._pixel_pitch(t[:, :, :, :, ::2]) == 0            # channels apart
    assert layer._pixel_pitch(t[:, :, :, 1:, :]) == 0             # rows apart
    assert layer._pixel_pitch(t[:, :, :, :1, :8]) == 5 * 16
    assert layer._pixel_pitch(t[:1, :1, :1, :1, :8]) == 8         # a single pixel
    assert layer._pixel_pitch(torch.zeros(()).expand(2, 3, 4, 5, 16)) == 0
    assert layer._pixel_pitch(t.permute(0, 1, 2, 4, 3)) == 0


def test_dense_tensors():
    t = torch.zeros(4, 6, 8)
    assert layer._dense(t) and layer._dense(t.permute(2, 0, 1)) and layer._dense(t[1])
    assert not layer._dense(t[:, :3]) and not layer._dense(t[0].expand(4, 6, 8))
    assert layer._dense(torch.zeros(())) and layer._dense(torch.zeros(0))


class FakeTensor:
    """What the binding asks of a GPU tensor, on the host."""

    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_bindings_check_tensors():
    """Short buffers and other types are refused before the library is called
    (addresses of host memory would be accepted by it)."""
    def z(*shape, dtype=torch.float32):
        return FakeTensor(torch.zeros(*shape, dtype=dtype))

    d = cv.make_group_norm_train_desc((1, 2, 3, 4, 16), 4, dtype=cv.ELT_BF16, x_pitch=32)
    b16 = torch.bfloat16
    x, y, v, stats = z(24 * 32 - 16, dtype=b16), z(24, 16, dtype=b16), z(16), z(2, 4, 2)
    ws = z(8, dtype=torch.uint8)
    good = dict(x=x, gamma=v, beta=v, y=y, stats=stats)
    bad = [("x", z(24 * 32 - 17, dtype=b16)), ("x", z(24, 32)), ("y", z(24, 15, dtype=b16)),
           ("gamma", z(15)), ("beta", z(16, dtype=b16)), ("stats", z(15)),
           ("y", torch.zeros(24, 16, dtype=b16))]
    for what, t in bad:
        with pytest.raises(ValueError, match=what):
            cv.conv3d_group_norm_train_fwd(d, workspace=ws, workspace_bytes=8, stream=0,
                                           **{**good, what: t})
        if what != "y":
            args = {**good, what: t}
            args["dy"] = args.pop("y")
            with pytest.raises(ValueError, match=what):
                cv.conv3d_group_norm_train_bwd(d, dx=None, dgamma=v, dbeta=None, workspace=ws,
                                               workspace_bytes=8, stream=0, **args)
    with pytest.raises(ValueError, match="workspace"):
        cv.conv3d_group_norm_train_fwd(d, workspace=ws, workspace_bytes=9, stream=0, **good)
    a = z(2, 16, dtype=b16)
    for what, t in (("dy", z(31, dtype=b16)), ("gamma", z(16)), ("dgamma", z(15)),
                    ("dvalue", z(2, 16))):
        args = {**dict(value=a, dy=a, dskip=None, gamma=z(16, dtype=b16), dvalue=a, dgamma=v,
                       dbias=None), what: t}
        with pytest.raises(ValueError, match=what):
            cv.conv3d_norm_silu_bwd(n=1, d=1, h=1, w=2, c=16, workspace=ws, workspace_bytes=8,
                                    stream=0, **args)
    for t, elt in ((z(9), cv.ELT_FP32), (z(10), cv.ELT_FP16)):
        with pytest.raises(ValueError, match="gradient"):
            cv.make_grads([(t, None, 10, elt, elt)])
    table = cv.make_grads([(z(10), None, 10, cv.ELT_FP32, cv.ELT_FP32)])
    for f in (lambda **kw: cv.conv3d_grad_clip(table, 0, 1.0, stream=0, **kw),
              lambda **kw: cv.conv3d_grad_norm(table, 0, stream=0, **kw)):
        with pytest.raises(ValueError, match="norm"):
            f(norm=z(1, dtype=b16), workspace=ws, workspace_bytes=8)
        with pytest.raises(ValueError, match="workspace"):
            f(norm=z(1), workspace=ws, workspace_bytes=9)

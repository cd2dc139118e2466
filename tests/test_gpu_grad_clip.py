"""Gradient norm and clipping against float64 (the squares of up to 2^24
products summed exactly enough there: 2^-53 each).

The norm is an fp64 sum rounded to fp32 once: it may differ by one fp32 step.
A clipped value is g * coef with coef rounded to fp32 (half a step), the
product in fp32 (half a step) and the result in its own type (half a step)."""
import math

import numpy as np
import pytest
import torch

import convolution_video_vae_amd as cv
from convolution_video_vae_amd.layer import GradClip, clip_grads
from guard import Guarded

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def draw(n, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, generator=g) * std).to(dtype)


def np64(t):
    return t.detach().double().cpu().numpy()


def norm_of(ts, kind):
    if kind == "inf":
        return max((float(np.abs(t).max()) for t in ts if t.size), default=0.0)
    return math.sqrt(math.fsum(float(np.dot(t.ravel(), t.ravel())) for t in ts))


def check(got, src, coef, what):
    ref = np64(src) * coef
    tol = (HALF[got.dtype] + 2.0 ** -22) * np.abs(ref)
    tol += {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[got.dtype]
    assert np.all(np.abs(np64(got) - ref) <= tol), what


SIZES = [[1], [7], [0, 5, 0], [4096], [4097, 1, 8191], [100003, 3, 17], [1 << 20, 12345, 0, 9],
         [64] * 300, [1000003, 77] * 130]


@pytest.mark.parametrize("kind", ["l2", "inf"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_norm_and_clip_in_place(sizes, kind):
    ts = [draw(n, TYPES[i % 3], i) for i, n in enumerate(sizes)]
    print(f"[clip] {len(sizes)} tensors up to {max(sizes)} {kind}", flush=True)
    dev = [t.cuda() for t in ts]
    want = norm_of([np64(t) for t in ts], kind)
    op = GradClip(dev, norm=kind)
    assert abs(op.norm().item() - want) <= 2.0 ** -23 * want
    assert all(torch.equal(a.cpu(), b) for a, b in zip(dev, ts))       # the norm changes nothing
    limit = want / 3
    got = op.clip(limit)
    assert abs(got.item() - want) <= 2.0 ** -23 * want
    coef = min(1.0, float(np.float32(limit)) / (want + 1e-6))
    for i, (a, b) in enumerate(zip(dev, ts)):
        check(a, b, coef, f"tensor {i}")


def test_below_the_limit_nothing_changes():
    ts = [draw(n, TYPES[i % 3], i, 1e-3) for i, n in enumerate([5000, 77, 12288])]
    dev = [t.cuda() for t in ts]
    clip_grads(dev, 1e6)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(dev, ts))
    outs = [torch.full_like(t, 7.0) for t in dev]
    GradClip(dev, outs).clip(1e6)                     # but copies are written
    assert all(torch.equal(a, b) for a, b in zip(dev, outs))


@pytest.mark.parametrize("src", TYPES, ids=str)
@pytest.mark.parametrize("dst", TYPES, ids=str)
def test_into_other_tensors(src, dst):
    ts = [draw(n, src, i) for i, n in enumerate([1, 9, 4095, 70001])]
    dev = [t.cuda() for t in ts]
    outs = [torch.full(t.shape, 7.0, dtype=dst, device="cuda") for t in ts]
    norm = GradClip(dev, outs).clip(2.0).item()
    want = norm_of([np64(t) for t in ts], "l2")
    assert abs(norm - want) <= 2.0 ** -23 * want
    for a, b, c in zip(outs, ts, dev):
        check(a, b, 2.0 / (want + 1e-6), "out")
        assert torch.equal(c.cpu(), b)


@pytest.mark.parametrize("off", [1, 2, 3, 5, 8])
def test_tensors_at_odd_addresses_and_nothing_beside_them(off):
    """Back to back in one buffer after `off` elements; the buffer's other
    elements stay."""
    for dtype in TYPES:
        sizes = [1, 30, 4099, 3, 20000]
        flat = torch.full((off + sum(sizes) + 9,), 7.0, dtype=dtype, device="cuda")
        views, at = [], off
        for i, n in enumerate(sizes):
            flat[at:at + n] = draw(n, dtype, i).cuda()
            views.append(flat[at:at + n])
            at += n
        src = [v.cpu() for v in views]
        clip_grads(views, 0.25)
        want = norm_of([np64(t) for t in src], "l2")
        for a, b in zip(views, src):
            check(a, b, 0.25 / (want + 1e-6), "view")
        assert torch.all(flat[:off] == 7.0) and torch.all(flat[at:] == 7.0)


def test_dense_layouts_of_any_order():
    t = draw(2 * 3 * 4 * 5, torch.float32, 3).view(2, 3, 4, 5)
    cl = t.cuda().permute(0, 2, 3, 1)
    out = torch.empty(2, 3, 4, 5, device="cuda").permute(0, 2, 3, 1)
    GradClip([cl], [out]).clip(0.5)
    want = norm_of([np64(t)], "l2")
    check(out.permute(0, 3, 1, 2), t, 0.5 / (want + 1e-6), "permuted")
    with pytest.raises(ValueError, match="strides"):
        GradClip([cl], [torch.empty(2, 4, 5, 3, device="cuda")])
    with pytest.raises(ValueError, match="dense"):
        GradClip([torch.empty(4, 6, device="cuda")[:, :3]])


@pytest.mark.parametrize("kind", ["l2", "inf"])
def test_extreme_and_non_finite_values(kind):
    def run(values, dtype=torch.float32, limit=1.0):
        t = torch.tensor(values, dtype=dtype, device="cuda")
        return clip_grads([t], limit, norm=kind).item(), t

    for v in (3e30, 3e-30):                       # the squares leave fp32's range
        n, t = run([v, -v])
        want = norm_of([np.array([v, -v], np.float32).astype(np.float64)], kind)
        assert abs(n - want) <= 2.0 ** -23 * want
        assert torch.all(torch.isfinite(t))
    n, t = run([1.0, float("nan"), 2.0])
    assert math.isnan(n) and torch.isnan(t).all()
    n, t = run([1.0, float("inf"), -2.0])         # coef is 0: inf * 0 is NaN
    assert math.isinf(n) and torch.isnan(t[1]) and t[0] == 0 and t[2] == 0
    n, t = run([0.0] * 5)
    assert n == 0.0 and torch.all(t == 0)
    n, t = run([3.0, 4.0], limit=0.0)
    assert torch.all(t == 0)


@pytest.mark.parametrize("src,dst", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16),
                                     (torch.float16, torch.float16), (torch.float32, None)])
@pytest.mark.parametrize("kind", ["l2", "inf"])
def test_results_larger_than_the_cache_share(src, dst, kind):
    """More than 128 MB of results (stored past the caches), at odd addresses."""
    n = (1 << 26) + 4099
    g = torch.Generator(device="cuda").manual_seed(4)
    buf = torch.randn(n + 1, generator=g, device="cuda").to(src)
    t = buf[1:]
    before = t.clone()
    out = None if dst is None else torch.full((n + 3,), 7.0, dtype=dst, device="cuda")
    limit = 1.0
    norm = GradClip([t[:5], t[5:]], None if dst is None else [out[1:6], out[6:n + 1]],
                    norm=kind).clip(limit).double()
    want = before.double().abs().max() if kind == "inf" else before.double().square().sum().sqrt()
    assert abs(norm - want) <= 2.0 ** -23 * want
    got = t if dst is None else out[1:n + 1]
    ref = before.double() * (limit / (want + 1e-6))
    tol = (HALF[got.dtype] + 2.0 ** -22) * ref.abs() + (2.0 ** -25 if dst == torch.float16 else 0)
    assert torch.all((got.double() - ref).abs() <= tol)
    if dst is not None:
        assert out[0] == 7.0 and torch.all(out[n + 1:] == 7.0) and torch.equal(t, before)


def test_moved_tensors_are_looked_up_again():
    t = draw(5000, torch.float32, 1).cuda()
    op = GradClip([t])
    first = op.norm().item()
    keep = t.data
    t.data = (draw(5000, torch.float32, 2) * 2).cuda()
    want = norm_of([np64(t)], "l2")
    assert abs(op.norm().item() - want) <= 2.0 ** -23 * want and first != want
    assert keep is not None


def test_moved_to_a_smaller_size():
    """The old memory is not handed out again while its address stands for the
    old size."""
    t = torch.full((4096,), 2.0, device="cuda")
    op = GradClip([t])
    assert op.norm().item() == 128.0  # sqrt(4096 * 4)
    before = t.data_ptr()
    t.data = torch.empty(0, device="cuda")
    t.data = torch.ones(1024, device="cuda")
    assert t.data_ptr() != before
    assert op.norm().item() == 32.0


def test_more_than_2_to_32_elements():
    n = (1 << 32) + 4099
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[-3:] = 2.0
    t[5] = 1.0
    norm = clip_grads([t], 1.0)
    assert abs(norm.item() - math.sqrt(13.0)) <= 2.0 ** -23 * 4
    want = torch.tensor(2.0 / (math.sqrt(13.0) + 1e-6)).bfloat16()
    assert torch.all(t[-3:].cpu() == want) and t[6:-3].count_nonzero() == 0


def test_guarded_workspace_and_norm():
    ts = [draw(n, torch.bfloat16, i).cuda() for i, n in enumerate([100000, 33, 4096])]
    table = cv.make_grads([(t, None, t.numel(), cv.ELT_BF16, cv.ELT_BF16) for t in ts])
    n = cv.conv3d_grad_workspace_bytes(table)
    ws, norm = Guarded((n // 2,), torch.int16), Guarded((1,), torch.float32)
    cv.conv3d_grad_norm(table, 0, norm.t, ws.t, n)
    a = norm.t.item()
    cv.conv3d_grad_clip(table, 0, 1.0, norm.t, ws.t, n)
    torch.cuda.synchronize()
    ws.assert_intact("workspace")
    norm.assert_intact("norm")
    assert norm.t.item() == a


def test_graph_replays_and_repeats_bit_for_bit():
    src = [torch.zeros(n, dtype=TYPES[i % 3], device="cuda") for i, n in enumerate([70001, 33, 9000])]
    outs = [torch.zeros(t.shape, device="cuda") for t in src]
    op = GradClip(src, outs)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        op.clip(1.0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm = op.clip(1.0)
    for i in range(3):
        for k, t in enumerate(src):
            t.copy_(draw(t.numel(), t.dtype, 10 * i + k))
        want = op.clip(1.0).clone()
        copies = [o.clone() for o in outs]
        torch.cuda.synchronize()
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want)
        assert all(torch.equal(a, b) for a, b in zip(outs, copies))


@pytest.mark.parametrize("calls", [0, 1, 3])
def test_shortened_and_retyped_tensors_at_their_old_address(calls):
    """What lies behind a tensor cut short is neither summed nor scaled, and
    its bytes are read as the type they now have."""
    whole = draw(4096, torch.float32, 3).cuda()
    before = whole.cpu()
    t, other = whole.view(-1), draw(70, torch.bfloat16, 4).cuda()
    op = GradClip([other, t])
    for _ in range(calls):
        op.norm()
    t.data = t.data[:1000]
    kept = [np64(other), np64(t)]
    want = norm_of(kept, "l2")
    assert abs(op.norm().item() - want) <= 2.0 ** -23 * want
    op.clip(1.0)
    check(whole[:1000], before[:1000], 1.0 / (want + 1e-6), "in front")
    assert torch.equal(whole[1000:].cpu(), before[1000:])
    bits = whole[:500].cpu().view(torch.bfloat16)
    other.data = torch.zeros(1, dtype=torch.bfloat16, device="cuda")
    whole[:500] = torch.ones(1000, dtype=torch.bfloat16).view(torch.float32).cuda()
    t.data = whole[:500].view(torch.bfloat16)
    assert bits.numel() == t.numel() == 1000
    assert abs(op.norm().item() - math.sqrt(1000.0)) <= 2.0 ** -23 * 32


def test_a_storage_cut_short_is_refused():
    t = torch.full((4096,), 2.0, device="cuda")
    op = GradClip([t])
    assert op.norm().item() == 128.0
    t.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="storage"):
        op.norm()
    t.untyped_storage().resize_(1024)
    with pytest.raises(ValueError, match="storage"):
        op.clip(1.0)


@pytest.mark.parametrize("kind", ["l2", "inf"])
@pytest.mark.parametrize("count", [2560, 2561, 9000])
def test_many_tensors(count, kind):
    """Lists on both sides of the number of partials that the clip pass's
    work-groups add by themselves; the norm is the norm call's, bit for bit."""
    g = torch.Generator().manual_seed(count)
    flat = torch.randn(count * 24, generator=g)
    if kind == "inf":
        flat[count * 11] = 77.0
    dev = flat.cuda()
    op = GradClip(list(dev.split(24)), norm=kind)
    want = norm_of([np64(flat)], kind)
    first = op.norm()
    got = op.clip(want / 4)
    assert torch.equal(first, got) and abs(got.item() - want) <= 2.0 ** -23 * want
    check(dev, flat, float(np.float32(want / 4)) / (want + 1e-6), "gradients")
    dev[5] = float("nan")
    assert math.isnan(op.clip(1.0).item()) and torch.isnan(dev).all()

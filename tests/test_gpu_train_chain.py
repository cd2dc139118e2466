"""The channel norm's backward pass on what the forward pass left: the fused
conv epilogue's residual_out, or the conv's output that conv3d_norm_silu
normalised."""
import numpy as np
import pytest
import torch

import convolution_video_vae_amd as cv
from convolution_video_vae_amd.layer import Conv3d, NormSiluBackward, clip_grads
from oracle import train
from test_gpu_train_norms import check, draw, np64, params

pytestmark = pytest.mark.gpu


def forward_bound(value, gamma):
    """(silu(norm) of value, what bf16 roundings of the normalised, the scaled
    and the final value, of half a step each, may change in it). The slope of
    SiLU is below 1.1; fp32 arithmetic adds 2^-16 at most."""
    y = train.norm_silu_fwd(value, gamma)
    c = value.shape[-1]
    norm = np.maximum(np.sqrt((value ** 2).sum(axis=-1, keepdims=True)), 1e-12)
    a = np.abs(value / norm * np.sqrt(c) * gamma)
    return y, 1.1 * (4 * 2.0 ** -8) * a + 2 * 2.0 ** -8 * np.abs(y) + 2.0 ** -16


@pytest.mark.parametrize("fused", [True, False], ids=["residual_out", "conv output"])
@pytest.mark.parametrize("c", [96, 160])
def test_saved_value_through_the_backward_pass_and_the_clip(c, fused):
    shape = (1, 3, 10, 12, c)
    print(f"[chain] {shape} fused={fused}", flush=True)
    w = draw((c, c, 3, 3, 3), torch.bfloat16, 1, 0.03).cuda()
    x, res = (draw(shape, torch.bfloat16, 2 + i).cuda() for i in range(2))
    bias, gamma = draw((c,), torch.float32, 4, 0.2), params(c, 5)[0].bfloat16()
    pads = dict(pad_lo=(2, 1, 1), pad_hi=(0, 1, 1))
    if fused:
        conv = Conv3d(w, shape, bias=bias.cuda(), gamma=gamma.cuda(), norm_silu=True,
                      residual=True, residual_out=True, **pads)
        value = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        y = conv(x, residual=res, residual_out=value)
        plain = Conv3d(w, shape, bias=bias.cuda(), residual=True, **pads)(x, residual=res)
        assert torch.equal(value, plain)
    else:
        value = Conv3d(w, shape, bias=bias.cuda(), **pads)(x)
        y = torch.empty_like(value)
        cv.conv3d_norm_silu(value, *shape, cv.make_epilogue(gamma=gamma.cuda(), norm_silu=True),
                            None, None, y)
    ref, tol = forward_bound(np64(value), np64(gamma))
    assert np.all(np.abs(np64(y) - ref) <= tol)
    dy, dskip = (draw(shape, torch.bfloat16, 6 + i, 0.1) for i in range(2))
    dv, dg, db = NormSiluBackward(shape, bias=True)(value, dy.cuda(), gamma.cuda(),
                                                    dskip=dskip.cuda())
    (rv, rg, rb), (tv, tg, tb) = train.norm_silu_bwd(np64(value), np64(dy), np64(gamma),
                                                     np64(dskip))
    check(dv, rv, tv, "dvalue")
    check(dg, rg, tg, "dgamma")
    check(db, rb, tb, "dbias")
    before = [np64(t) for t in (dg, db)]
    norm = clip_grads([dg, db], 0.01).item()
    total = np.sqrt(sum((t ** 2).sum() for t in before))
    assert abs(norm - total) <= 2.0 ** -23 * total
    for t, b in zip((dg, db), before):
        want = b * 0.01 / (total + 1e-6)
        assert np.all(np.abs(np64(t) - want) <= (2.0 ** -24 + 2.0 ** -22) * np.abs(want))

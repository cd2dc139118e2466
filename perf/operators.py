"""The training-side operators of the norms between the convs, as measured work.

Four operators, each in its plain form (elementary torch operations in
32 bits, rounded once) and as the library's call:

  gn_fwd   channels-last GroupNorm (+ SiLU) that keeps its statistics
  gn_bwd   its backward pass: dx, dgamma, dbeta
  ns_bwd   the backward pass of the channel L2 norm x sqrt(C) x gamma -> SiLU
           (conv3d_norm_silu): dvalue, dgamma, dbias
  clip     the global gradient norm over many tensors, and clipping

Activation shapes are the encoder levels of the library's workloads; the
gradient lists are the parameters of such encoders.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # the deepest encoder level, one clip: 1024 channels on 16x16 frames, where latency counts
        dict(name="gn_fwd_1024_16x16", op="gn_fwd", n=1, d=5, h=16, w=16, c=1024, groups=32,
             per_frame=True, silu=True, dtype="bf16", wide=1),
        # full resolution, the largest activation an encoder normalises
        dict(name="gn_fwd_128_256x256", op="gn_fwd", n=1, d=17, h=256, w=256, c=128, groups=32,
             per_frame=True, silu=True, dtype="bf16", wide=1),
        # a batch in fp32 with channels that fill no 16-byte vector, statistics over whole clips
        dict(name="gn_fwd_odd_fp32", op="gn_fwd", n=2, d=3, h=61, w=67, c=90, groups=30,
             per_frame=False, silu=False, dtype="fp32", wide=1),
        dict(name="gn_bwd_1024_16x16", op="gn_bwd", n=1, d=5, h=16, w=16, c=1024, groups=32,
             per_frame=True, silu=True, dtype="bf16", wide=1),
        # half resolution in fp16
        dict(name="gn_bwd_256_128x128_fp16", op="gn_bwd", n=1, d=17, h=128, w=128, c=256,
             groups=32, per_frame=True, silu=True, dtype="fp16", wide=1),
        dict(name="gn_bwd_128_256x256", op="gn_bwd", n=1, d=17, h=256, w=256, c=128, groups=32,
             per_frame=True, silu=True, dtype="bf16", wide=1),
        # x and its gradient are the first half of the channels of a concatenated skip connection
        dict(name="gn_bwd_512_slice", op="gn_bwd", n=2, d=5, h=32, w=32, c=512, groups=32,
             per_frame=False, silu=True, dtype="bf16", wide=2),
        # the standalone post-operations above the fused tile, a quarter of the 64 x 120 level
        dict(name="ns_bwd_640_16x30", op="ns_bwd", n=1, d=5, h=16, w=30, c=640, skip=True,
             bias=True),
        # full-resolution 96-channel level
        dict(name="ns_bwd_96_352x640", op="ns_bwd", n=1, d=4, h=352, w=640, c=96, skip=False,
             bias=False),
        # the norms' gammas and betas alone (a fine-tune of the norms): many tiny tensors
        dict(name="clip_norm_params", op="clip", ch=128, mult="1,2,2,4,4,8", blocks=2,
             convs=False, weights="fp32", out="fp32", packed=False, kind="l2", std=1e-2),
        # a whole encoder's bf16 gradients clipped into the optimizer's fp32 gradients
        dict(name="clip_encoder_128", op="clip", ch=128, mult="1,2,2,4,4,8", blocks=2,
             convs=True, weights="bf16", out="fp32", packed=False, kind="l2", std=1e-3),
        # a step that needs no clipping, in place, in buckets without gaps (tensors at odd addresses)
        dict(name="clip_encoder_96_quiet", op="clip", ch=96, mult="1,2,4,4", blocks=2,
             convs=True, weights="bf16", out="", packed=True, kind="l2", std=1e-5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gn_fwd", "gn_bwd", "ns_bwd", "clip"])
    if op == "clip":
        out = rng.choice(["same", "fp32", ""])
        weights = rng.choice(["bf16", "fp16", "fp32"])
        levels = rng.randint(1, 4)
        return dict(op=op, ch=8 * _log(rng, 2, 12), blocks=rng.randint(1, 3),
                    mult=",".join(str(rng.choice([1, 2, 4, 5])) for _ in range(levels)),
                    convs=rng.random() < 0.8, weights=weights,
                    out=weights if out == "same" else out, packed=rng.random() < 0.5,
                    kind=rng.choice(["l2", "l2", "inf"]),
                    std=1e-5 if out == "" else rng.choice([1e-3, 1.0]))
    if op == "ns_bwd":
        c, cap = 8 * _log(rng, 1, 256), 60_000_000
    else:
        cpg = rng.choice([1, 2, 3, 4, 8, 16, 32])
        groups = rng.choice([1, 4, 8, 16, 30, 32])
        c, cap = cpg * groups, 60_000_000
    d, n = rng.randint(1, 6), rng.randint(1, 3)
    area = _log(rng, 16, max(16, min(cap // (n * d * c), 300_000)))
    w = max(1, int(math.sqrt(area) * rng.uniform(0.6, 1.6)))
    h = max(1, area // w)
    if op == "ns_bwd":
        return dict(op=op, n=n, d=d, h=h, w=w, c=c, skip=rng.random() < 0.5,
                    bias=rng.random() < 0.5)
    return dict(op=op, n=n, d=d, h=h, w=w, c=c, groups=groups, per_frame=rng.random() < 0.5,
                silu=rng.random() < 0.7, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                wide=rng.choice([1, 1, 2]))


# ------------------------------------------------------------------- inputs

def _grad_sizes(case):
    """Element counts of an encoder's gradients: conv tensors (weights, in the
    working type) and the fp32 ones (norm gammas and betas, biases)."""
    ch, blocks = case["ch"], case["blocks"]
    weights, vectors, cin = [27 * 12 * ch], [ch], ch
    for m in (int(v) for v in case["mult"].split(",")):
        cout = ch * m
        for _ in range(blocks):
            weights += [27 * cin * cout, 27 * cout * cout]
            vectors += [cin, cin, cout, cout, cout, cout]   # norm, bias, norm, bias
            if cin != cout:
                weights.append(cin * cout)
            cin = cout
    return (weights if case["convs"] else []), vectors


def _places(sizes, packed):
    """Offsets (elements) in one flat buffer, and its length: back to back
    after a first odd element, or at 64-element boundaries."""
    at, off = 1 if packed else 0, []
    for s in sizes:
        off.append(at)
        at += s if packed else (s + 63) // 64 * 64
    return off, at


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case=case)
    if case["op"] == "clip":
        s["flat"], s["out"], s["grads"], s["outs"] = [], [], [], []
        for sizes, dt in zip(_grad_sizes(case), (case["weights"], "fp32")):
            if not sizes:
                continue
            off, total = _places(sizes, case["packed"])
            flat = torch.zeros(total, dtype=DTYPES[dt], device="cuda")
            out = flat
            if case["out"]:
                out = torch.zeros(total, dtype=DTYPES[case["out"] if dt != "fp32" else "fp32"],
                                  device="cuda")
            for o, k in zip(off, sizes):
                flat[o:o + k] = normal(k, case["std"], DTYPES[dt])
                s["grads"].append(flat[o:o + k])
                s["outs"].append(out[o:o + k])
            s["flat"].append(flat)
            s["out"].append(out)
        return s
    n, d, h, w, c = (case[k] for k in "ndhwc")
    shape = (n, d, h, w, c)
    if case["op"] == "ns_bwd":
        s["value"] = normal(shape, 1.0, torch.bfloat16)
        s["dy"] = normal(shape, 1e-2, torch.bfloat16)
        s["gamma"] = (torch.rand(c, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
        s["dskip"] = normal(shape, 1e-2, torch.bfloat16) if case["skip"] else None
        return s
    dt = DTYPES[case["dtype"]]
    wide = normal((n, d, h, w, c * case["wide"]))
    wide[..., :c] += normal(c, 0.5)                 # a conv's output with its bias
    s["x"] = wide.to(dt)[..., :c]
    s["gamma"] = torch.rand(c, generator=g, device="cuda") + 0.5
    s["beta"] = normal(c, 0.1)
    if case["op"] == "gn_bwd":
        s["dy"] = normal(shape, 1e-2, dt)
        # the forward pass's statistics, kept for this call
        u, p, k = _units(case)
        x = s["x"].reshape(u, p, case["groups"], k)
        mean = x.mean(dim=(1, 3), dtype=torch.float64) if dt == torch.float32 else \
            x.float().mean(dim=(1, 3))
        var = (x.float() - mean.float()[:, None, :, None]).square().mean(dim=(1, 3))
        s["stats"] = torch.stack([mean.float(), 1.0 / torch.sqrt(var + EPS)], dim=-1)
        if case["wide"] > 1:
            s["dx"] = torch.empty((n, d, h, w, c * case["wide"]), dtype=dt,
                                  device="cuda")[..., :c]
    return s


def _units(case):
    """(statistics units, pixels of one, channels per group)."""
    n, d, p = case["n"], case["d"], case["h"] * case["w"]
    u, p = (n * d, p) if case["per_frame"] else (n, d * p)
    return u, p, case["c"] // case["groups"]


# ---------------------------------------------------------------------- run

def run(s):
    return globals()["_" + s["case"]["op"]](s)


def _gn_layer(s):
    """The layer object a program builds once per shape."""
    if "layer" not in s:
        from convolution_video_vae_amd.layer import GroupNormTrain
        c = s["case"]
        s["layer"] = GroupNormTrain((c["n"], c["d"], c["h"], c["w"], c["c"]), c["groups"],
                                    eps=EPS, silu=c["silu"], t_isolated=c["per_frame"],
                                    dtype=DTYPES[c["dtype"]])
    return s["layer"]


def _gn_fwd(s):
    c = s["case"]
    if own:
        return _gn_layer(s).forward(s["x"], s["gamma"], s["beta"])
    u, p, k = _units(c)
    x = s["x"].float().reshape(u, p, c["groups"], k)
    mean = x.mean(dim=(1, 3), keepdim=True)
    x = x - mean
    rstd = 1.0 / torch.sqrt(x.square().mean(dim=(1, 3), keepdim=True) + EPS)
    a = x * rstd * s["gamma"].view(1, 1, c["groups"], k) + s["beta"].view(1, 1, c["groups"], k)
    if c["silu"]:
        a = a / (1.0 + torch.exp(-a))
    stats = torch.stack([mean.view(u, c["groups"]), rstd.view(u, c["groups"])], dim=-1)
    return a.to(s["x"].dtype).view(s["x"].shape), stats


def _gn_bwd(s):
    c = s["case"]
    if own:
        return _gn_layer(s).backward(s["dy"], s["x"], s["gamma"], s["beta"], s["stats"],
                                     dx=s.get("dx"))
    u, p, k = _units(c)
    shape = (u, p, c["groups"], k)
    mean, rstd = (s["stats"][..., i].view(u, 1, c["groups"], 1) for i in (0, 1))
    gamma = s["gamma"].view(1, 1, c["groups"], k)
    xhat = (s["x"].float().reshape(shape) - mean) * rstd
    da = s["dy"].float().view(shape)
    if c["silu"]:
        a = xhat * gamma + s["beta"].view(1, 1, c["groups"], k)
        sig = 1.0 / (1.0 + torch.exp(-a))
        da = da * (sig * (1.0 + a * (1.0 - sig)))
    db, dg = da.sum(dim=1, keepdim=True), (da * xhat).sum(dim=1, keepdim=True)
    c1 = (db * gamma).sum(dim=3, keepdim=True) / (p * k)
    c2 = (dg * gamma).sum(dim=3, keepdim=True) / (p * k)
    dx = rstd * (gamma * da - c1 - xhat * c2)
    return (dx.to(s["x"].dtype).view(s["dy"].shape), dg.sum(dim=0).reshape(-1),
            db.sum(dim=0).reshape(-1))


def _ns_bwd(s):
    c = s["case"]
    if own:
        if "layer" not in s:
            from convolution_video_vae_amd.layer import NormSiluBackward
            s["layer"] = NormSiluBackward(tuple(s["value"].shape), bias=c["bias"])
        return s["layer"](s["value"], s["dy"], s["gamma"], dskip=s["dskip"])
    v, gamma = s["value"].float().view(-1, c["c"]), s["gamma"].float()
    root = math.sqrt(c["c"])
    norm = torch.sqrt(v.square().sum(dim=1, keepdim=True))
    den = torch.clamp(norm, min=1e-12)
    unit = v / den
    a = unit * root * gamma
    sig = 1.0 / (1.0 + torch.exp(-a))
    da = s["dy"].float().view(-1, c["c"]) * (sig * (1.0 + a * (1.0 - sig)))
    dgamma = (da * unit).sum(dim=0) * root
    dunit = da * gamma * root
    dot = torch.where(norm > 1e-12, (dunit * unit).sum(dim=1, keepdim=True), 0.0)
    dv = (dunit - unit * dot) / den
    if s["dskip"] is not None:
        dv = dv + s["dskip"].float().view(-1, c["c"])
    return (dv.to(torch.bfloat16).view(s["value"].shape), dgamma,
            dv.sum(dim=0) if c["bias"] else None)


def _clip(s):
    c = s["case"]
    if own:
        if "clip" not in s:
            from convolution_video_vae_amd.layer import GradClip
            s["clip"] = GradClip(s["grads"], s["outs"] if c["out"] else None, norm=c["kind"])
        return [s["clip"].clip(1.0)] + s["out"]
    flat = [f.float() for f in s["flat"]]
    if c["kind"] == "inf":
        norm = torch.stack([f.abs().max() for f in flat]).max()
    else:
        norm = torch.sqrt(torch.stack([f.square().sum(dtype=torch.float64) for f in flat])
                          .sum()).float()
    coef = torch.clamp(1.0 / (norm + 1e-6), max=1.0)
    return [norm] + [(f * coef).to(o.dtype) for f, o in zip(flat, s["out"])]


# --------------------------------------------------------------------- work

def work(case):
    if case["op"] == "clip":
        weights, vectors = (sum(v) for v in _grad_sizes(case))
        wb = DTYPES[case["weights"]].itemsize
        read = weights * wb + 4 * vectors
        write = 4 * vectors + weights * DTYPES[case["out"]].itemsize if case["out"] else 0
        return {"bytes": read + write, "flops": 3 * (weights + vectors)}
    e = case["n"] * case["d"] * case["h"] * case["w"] * case["c"]
    if case["op"] == "ns_bwd":
        return {"bytes": 2 * e * (4 if case["skip"] else 3), "flops": 30 * e}
    size = DTYPES[case["dtype"]].itemsize
    return {"bytes": e * size * (2 if case["op"] == "gn_fwd" else 3),
            "flops": e * (12 if case["op"] == "gn_fwd" else 30)}


# -------------------------------------------------------------------- exact

def _silu_slope(a):
    """d/da of a / (1 + e^-a), as 1/(1 + e^-a) + a e^-a / (1 + e^-a)^2 with e^-|a| alone."""
    t = torch.exp(-a.abs())
    q = 1.0 / (1.0 + t)
    return torch.where(a >= 0, q, t * q) + a * t * q * q


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        every = [g.double() for g in s["grads"]]
        if case["kind"] == "inf":
            norm = max(float(g.abs().max()) for g in every)
        else:
            norm = math.sqrt(math.fsum(float(torch.dot(g, g)) for g in every))
        coef = min(1.0, 1.0 / (norm + 1e-6))
        return [torch.tensor(norm, dtype=torch.float64)] + [f.double() * coef for f in s["flat"]]
    c = case["c"]
    if case["op"] == "ns_bwd":
        dgamma = torch.zeros(c, dtype=torch.float64, device="cuda")
        dbias, gamma, dvs = dgamma.clone(), s["gamma"].double(), []
        for i in range(case["n"]):
            for f in range(case["d"]):
                v, dy = s["value"][i, f].double(), s["dy"][i, f].double()
                norm = torch.linalg.vector_norm(v, dim=-1, keepdim=True)
                scale = math.sqrt(c) / norm.clamp(min=1e-12)
                da = dy * _silu_slope(v * scale * gamma)
                dgamma += (da * v * scale).sum(dim=(0, 1))
                dn = da * gamma * scale
                # d(v / |v|) is (I - v v^T / |v|^2) / |v|; below the clamp it is I / 1e-12
                part = (dn * v).sum(dim=-1, keepdim=True) / (norm * norm)
                dv = dn - v * torch.where(norm > 1e-12, part, torch.zeros_like(part))
                if s["dskip"] is not None:
                    dv = dv + s["dskip"][i, f].double()
                dbias += dv.sum(dim=(0, 1))
                dvs.append(dv)
        return (torch.stack(dvs).view(s["value"].shape), dgamma, dbias if case["bias"] else None)
    u, p, k = _units(case)
    x = s["x"].reshape(u, p, c)
    if case["op"] == "gn_fwd":
        ys, stats = [], torch.empty(u, case["groups"], 2, dtype=torch.float64, device="cuda")
        for i in range(u):
            xi = x[i].double().view(p, case["groups"], k)
            var, mean = torch.var_mean(xi, dim=(0, 2), correction=0, keepdim=True)
            a = ((xi - mean) * torch.rsqrt(var + EPS)).view(p, c) * s["gamma"].double() \
                + s["beta"].double()
            ys.append(a * torch.sigmoid(a) if case["silu"] else a)
            stats[i, :, 0] = mean.view(-1)
            stats[i, :, 1] = torch.rsqrt(var + EPS).view(-1)
        return torch.stack(ys).view(s["x"].shape), stats
    dy, gamma = s["dy"].reshape(u, p, c), s["gamma"].double()
    dgamma = torch.zeros(c, dtype=torch.float64, device="cuda")
    dbeta, dxs = dgamma.clone(), []
    for i in range(u):
        mean, rstd = (s["stats"][i, :, j].double().repeat_interleave(k) for j in (0, 1))
        xhat, da = (x[i].double() - mean) * rstd, dy[i].double()
        if case["silu"]:
            da = da * _silu_slope(xhat * gamma + s["beta"].double())
        dgamma += (da * xhat).sum(dim=0)
        dbeta += da.sum(dim=0)
        dh = (da * gamma).view(p, case["groups"], k)
        xh = xhat.view(p, case["groups"], k)
        m1 = dh.mean(dim=(0, 2), keepdim=True)
        m2 = (dh * xh).mean(dim=(0, 2), keepdim=True)
        dxs.append((dh - m1 - xh * m2).view(p, c) * rstd)
    return torch.stack(dxs).view(s["dy"].shape), dgamma, dbeta

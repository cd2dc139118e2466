"""Pack-once / execute-many wrapper around the C entry points.

The cuDNN page ("Requirements", "Weight Packing") describes the usage this
mirrors: pack a checkpoint weight once, keep the packed copy, and execute
with preallocated buffers on the caller's stream. PyTorch only allocates
the device buffers here; every step runs in the library's kernels.
"""
from __future__ import annotations

import operator
from typing import Optional, Sequence

import torch

from . import (ELT_BF16, ELT_FP16, ELT_FP32, GRAD_NORM_INF, GRAD_NORM_L2, NCDHW, NDHWC,
               conv3d_fwd, conv3d_fwd_padded, conv3d_grad_clip, conv3d_grad_norm, conv3d_grad_workspace_bytes,
               conv3d_group_norm, conv3d_group_norm_train_bwd, conv3d_group_norm_train_fwd,
               conv3d_group_norm_train_workspace_bytes, conv3d_group_norm_workspace_bytes,
               conv3d_norm_silu_bwd, conv3d_norm_silu_bwd_workspace_bytes, conv3d_output_dims,
               conv3d_pack_weight, conv3d_pack_weight_2d, conv3d_pack_weight_fp8,
               conv3d_packed_weight_bytes, conv3d_packed_weight_bytes_fp8,
               conv3d_padded_workspace_bytes, conv3d_stream_pack_input, conv3d_workspace_bytes,
               make_desc, make_epilogue, make_grads, make_group_norm_desc,
               make_group_norm_train_desc, make_out_pad)


def _expect(t: Optional[torch.Tensor], shape, what: str) -> None:
    """An output or operand tensor of the layer: bf16, contiguous, on a GPU,
    of exactly the layer's shape (the library sizes every access from the
    layer's descriptor)."""
    if t is None:
        return
    if (tuple(t.shape) != tuple(shape) or t.dtype != torch.bfloat16 or not t.is_contiguous()
            or not t.is_cuda):
        raise ValueError(f"{what} must be a contiguous bf16 GPU tensor of shape {tuple(shape)}, "
                         f"got {tuple(t.shape)} {t.dtype} on {t.device}"
                         f"{'' if t.is_contiguous() else ' (not contiguous)'}")


def pack_weight(w_oidhw: torch.Tensor, stream=None) -> torch.Tensor:
    """OIDHW bf16 [Cout][Cin][3][3][3] on the GPU -> packed weight buffer.
    A 4-D [Cout][Cin][3][3] weight is packed as the last temporal slice of a
    3x3x3 weight (for 2D and 1x3x3 layers run on single frames); an
    float8_e4m3fn 5-D weight is packed for the fp8 conv."""
    if w_oidhw.dtype == torch.float8_e4m3fn and w_oidhw.is_cuda and w_oidhw.dim() == 5:
        cout, cin = w_oidhw.shape[:2]
        w = w_oidhw.contiguous()
        out = torch.empty(conv3d_packed_weight_bytes_fp8(cout, cin), dtype=torch.uint8,
                          device=w.device)
        conv3d_pack_weight_fp8(w, out, cout, cin, stream)
        return out
    if w_oidhw.dtype != torch.bfloat16 or not w_oidhw.is_cuda or w_oidhw.dim() not in (4, 5):
        raise ValueError("weight must be a 4-D or 5-D bf16 CUDA tensor")
    cout, cin = w_oidhw.shape[:2]
    w = w_oidhw.contiguous()
    out = torch.empty(conv3d_packed_weight_bytes(cout, cin) // 2, dtype=torch.bfloat16,
                      device=w.device)
    if w.dim() == 4:
        conv3d_pack_weight_2d(w, out, cout, cin, stream)
    else:
        conv3d_pack_weight(w, out, cout, cin, stream)
    return out


class Conv3d:
    """One 3x3x3 bf16 conv layer with a packed weight and fixed shapes."""

    def __init__(self, weight: torch.Tensor, x_shape: Sequence[int], *, stride=(1, 1, 1),
                 pad_lo=(0, 0, 0), pad_hi=(0, 0, 0), layout: int = NDHWC,
                 out_layout: Optional[int] = None, split_k: int = 0,
                 bias: Optional[torch.Tensor] = None, gamma: Optional[torch.Tensor] = None,
                 norm_silu: bool = False, residual: bool = False, residual_out: bool = False,
                 out_pad_lo=None, out_pad_hi=(0, 0, 0), history_frames: int = 0,
                 cache_frames: int = 0, pad_mode: int = 0):
        """out_pad_lo / out_pad_hi: write the output into the interior of a
        zero-bordered buffer (the history_frames planes before it are the
        caller's); cache_frames > 0: also keep the last output frames in a
        cache passed to each call."""
        self.cout, self.cin = int(weight.shape[0]), int(weight.shape[1])
        self.layout = layout
        self.out_layout = layout if out_layout is None else out_layout
        self.x_shape = tuple(int(v) for v in x_shape)
        self.fp8 = weight.dtype == torch.float8_e4m3fn
        self.in_dtype = torch.float8_e4m3fn if self.fp8 else torch.bfloat16
        self.desc = make_desc(self.x_shape, self.cout, stride=stride, pad_lo=pad_lo, pad_hi=pad_hi,
                              layout=layout, out_layout=self.out_layout, split_k=split_k,
                              pad_mode=pad_mode, dtype=1 if self.fp8 else 0)
        self.out_dhw = conv3d_output_dims(self.desc)
        n = self.x_shape[0]
        if self.out_layout == NDHWC:
            self.out_shape = (n,) + self.out_dhw + (self.cout,)
        else:
            self.out_shape = (n, self.cout) + self.out_dhw
        self.padded = out_pad_lo is not None or cache_frames > 0
        self.out_pad_lo = tuple(out_pad_lo or (0, 0, 0))
        self.out_pad_hi = tuple(out_pad_hi)
        self.history_frames = history_frames
        self.cache_frames = cache_frames
        if self.padded:
            self.out_shape = (n,) + tuple(o + a + b for o, a, b in zip(
                self.out_dhw, self.out_pad_lo, self.out_pad_hi)) + (self.cout,)
            self.cache_shape = (n, cache_frames) + self.out_dhw[1:] + (self.cout,)
        self.device = weight.device
        self.w_packed = pack_weight(weight)
        self.bias = None if bias is None else bias.to(device=self.device, dtype=torch.float32).contiguous()
        self.gamma = None if gamma is None else gamma.to(device=self.device, dtype=torch.bfloat16).contiguous()
        self.norm_silu = norm_silu
        self.has_residual = residual
        self.has_residual_out = residual_out
        probe = make_epilogue(bias=self.bias, gamma=self.gamma, norm_silu=norm_silu)
        probe.flags |= (2 if residual else 0) | (8 if residual_out else 0)
        if self.padded:
            self.workspace_bytes = conv3d_padded_workspace_bytes(self.desc, probe,
                                                                 self._out_pad(None))
        else:
            self.workspace_bytes = conv3d_workspace_bytes(self.desc, probe)
        self.workspace = (torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.device)
                          if self.workspace_bytes else None)

    def _out_pad(self, cache):
        # the probe for the workspace size only needs a non-null cache address
        c = cache if cache is not None else (16 if self.cache_frames else None)
        return make_out_pad(self.out_pad_lo, self.out_pad_hi, self.history_frames, c,
                            self.cache_frames)

    def new_output(self) -> torch.Tensor:
        return torch.empty(self.out_shape, dtype=torch.bfloat16, device=self.device)

    def __call__(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                 y: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None,
                 stream=None, cache: Optional[torch.Tensor] = None) -> torch.Tensor:
        if (tuple(x.shape) != self.x_shape or x.dtype != self.in_dtype or not x.is_contiguous()
                or not x.is_cuda):
            raise ValueError(f"x must be a contiguous {self.in_dtype} GPU tensor of shape "
                             f"{self.x_shape}")
        if self.has_residual != (residual is not None):
            raise ValueError("residual presence differs from construction")
        if self.has_residual_out != (residual_out is not None):
            raise ValueError("residual_out presence differs from construction")
        n = self.x_shape[0]
        plain = ((n,) + self.out_dhw + (self.cout,) if self.out_layout == NDHWC
                 else (n, self.cout) + self.out_dhw)
        _expect(residual, plain, "residual")
        _expect(residual_out, plain, "residual_out")
        _expect(y, self.out_shape, "y")
        if self.padded:
            _expect(cache, self.cache_shape, "cache")
        if y is None:
            y = self.new_output()
        epi = make_epilogue(bias=self.bias, residual=residual, gamma=self.gamma,
                            residual_out=residual_out, norm_silu=self.norm_silu)
        if self.padded:
            if (cache is not None) != (self.cache_frames > 0):
                raise ValueError("cache presence differs from construction")
            conv3d_fwd_padded(self.desc, x, self.w_packed, epi if epi.flags else None,
                              self._out_pad(cache), y, self.workspace, self.workspace_bytes, stream)
        else:
            conv3d_fwd(self.desc, x, self.w_packed, epi if epi.flags else None, y, self.workspace,
                       self.workspace_bytes, stream)
        return y


def stream_pack_input(chunk: torch.Tensor, history: Optional[torch.Tensor], c_pad: int,
                      padded: Optional[torch.Tensor] = None, cache: Optional[torch.Tensor] = None,
                      cache_frames: int = 2, stream=None):
    """First layer of a streaming causal encoder: chunk [N, C, T, H, W] (any
    strides) and history [N, P, H, W, C] -> (padded [N, T+2, H+2, W+2, c_pad],
    cache [N, min(cache_frames, T+P), H, W, C])."""
    n, c, t, h, w = (int(v) for v in chunk.shape)
    P = 0 if history is None else int(history.shape[1])
    cf = min(cache_frames, t + P)
    if padded is None:
        padded = torch.empty((n, t + 2, h + 2, w + 2, c_pad), dtype=torch.bfloat16,
                             device=chunk.device)
    if cache is None and cf > 0:
        cache = torch.empty((n, cf, h, w, c), dtype=torch.bfloat16, device=chunk.device)
    if history is not None:
        history = history.contiguous()
    conv3d_stream_pack_input(chunk, chunk.stride(), n, c, t, h, w, history, P, padded, c_pad,
                             cache, cf if cache is not None else 0, stream)
    return padded, cache


class GroupNorm:
    """Channels-last GroupNorm (+ SiLU) of one NDHWC activation shape, with
    its workspace allocated once; statistics per frame when t_isolated."""

    def __init__(self, x_shape: Sequence[int], groups: int, gamma: torch.Tensor,
                 beta: torch.Tensor, *, eps: float = 1e-5, silu: bool = False,
                 t_isolated: bool = True):
        self.x_shape = tuple(int(v) for v in x_shape)
        self.desc = make_group_norm_desc(self.x_shape, groups, eps=eps, silu=silu,
                                         t_isolated=t_isolated)
        self.device = gamma.device
        self.gamma = gamma.to(dtype=torch.float32).contiguous()
        self.beta = beta.to(device=self.device, dtype=torch.float32).contiguous()
        self.workspace_bytes = conv3d_group_norm_workspace_bytes(self.desc)
        self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.device)

    def __call__(self, x: torch.Tensor, y: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
        """y = GroupNorm(x); pass y=x to normalise in place."""
        if tuple(x.shape) != self.x_shape or x.dtype != torch.bfloat16 or not x.is_contiguous():
            raise ValueError(f"x must be a contiguous bf16 tensor of shape {self.x_shape}")
        if y is None:
            y = torch.empty_like(x)
        conv3d_group_norm(self.desc, x, self.gamma, self.beta, y, self.workspace,
                          self.workspace_bytes, stream)
        return y


# --------------------------------------------------------------------------- training
# The classes below run on the current stream of their tensors' device.
# Outputs and scratch memory that a call needs come from PyTorch's allocator
# on that stream (inside a graph capture, from the graph's own pool), so one
# object may serve several streams and graphs at once. Autograd does not record
# these calls: results carry no graph, whatever their inputs require.

# The current stream's handle without a Stream object around it (3 us less per call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_stream(index: int) -> int:
    if _raw_stream is not None:
        return _raw_stream(index)
    return torch.cuda.current_stream(index).cuda_stream


_ELT = {torch.bfloat16: ELT_BF16, torch.float16: ELT_FP16, torch.float32: ELT_FP32}


def _pixel_pitch(t: torch.Tensor) -> int:
    """Elements between consecutive pixels of an NDHWC tensor whose channels
    are contiguous; 0 if its pixels are not evenly spaced."""
    c = t.shape[4]
    if t.is_contiguous():
        return c
    if c > 1 and t.stride(4) != 1:
        return 0
    pitch, run = 0, 1
    for i in (3, 2, 1, 0):
        if t.shape[i] > 1:
            if pitch == 0:
                pitch = t.stride(i)
                if pitch < c:
                    return 0
            elif t.stride(i) != pitch * run:
                return 0
        run *= t.shape[i]
    return pitch or c


def _activation(t: torch.Tensor, shape, dtype, what: str) -> int:
    """Checks an NDHWC activation (a channel slice of a wider tensor counts)
    and returns its pixel pitch."""
    pitch = (_pixel_pitch(t) if t.is_cuda and t.dtype == dtype and tuple(t.shape) == shape else 0)
    if not pitch:
        raise ValueError(f"{what} must be a {dtype} GPU tensor of shape {shape} with contiguous "
                         f"channels and evenly spaced pixels, got {tuple(t.shape)} {t.dtype} "
                         f"strides {tuple(t.stride())} on {t.device}")
    return pitch


def _vector(t: torch.Tensor, numel: int, dtype, device, what: str) -> None:
    if t.dtype != dtype or t.numel() != numel or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of {numel} values on "
                         f"{device}, got {tuple(t.shape)} {t.dtype} on {t.device}")


def _same_device(device, **tensors) -> None:
    for what, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{what} is on {t.device}, x on {device}")


class GroupNormTrain:
    """Channels-last GroupNorm (+ SiLU) of one NDHWC activation shape with its
    backward pass: forward keeps the statistics that backward needs. Tensors
    may be channel slices of wider ones."""

    def __init__(self, x_shape: Sequence[int], groups: int, *, eps: float = 1e-5,
                 silu: bool = False, t_isolated: bool = True, dtype=torch.bfloat16):
        if dtype not in _ELT:
            raise ValueError(f"dtype must be one of {list(_ELT)}, got {dtype}")
        self.x_shape = tuple(int(v) for v in x_shape)
        self.dtype = dtype
        n, d, _, _, c = self.x_shape
        self.c = c
        self.stats_shape = (n * d if t_isolated else n, groups, 2)
        self._stats_numel = self.stats_shape[0] * groups * 2
        self._kw = dict(eps=eps, silu=silu, t_isolated=t_isolated, dtype=_ELT[dtype])
        self.groups = groups
        self._descs = {}
        self._ws = tuple(conv3d_group_norm_train_workspace_bytes(self._desc(c, c, c), b)
                         for b in (False, True))

    def _desc(self, x_pitch: int, y_pitch: int, dx_pitch: int):
        key = (x_pitch, y_pitch, dx_pitch)
        d = self._descs.get(key)
        if d is None:
            d = self._descs[key] = make_group_norm_train_desc(
                self.x_shape, self.groups, x_pitch=x_pitch, y_pitch=y_pitch, dx_pitch=dx_pitch,
                **self._kw)
        return d

    def forward(self, x: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor,
                y: Optional[torch.Tensor] = None, stats: Optional[torch.Tensor] = None):
        """(y, stats): the norm of x, and per unit and group the fp32 mean and
        1/sqrt(var + eps). gamma and beta are fp32 [c]."""
        dev = x.device
        xp = _activation(x, self.x_shape, self.dtype, "x")
        if dev.index != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return self.forward(x, gamma, beta, y, stats)
        _vector(gamma, self.c, torch.float32, dev, "gamma")
        _vector(beta, self.c, torch.float32, dev, "beta")
        if y is None:
            y, yp = torch.empty(self.x_shape, dtype=self.dtype, device=dev), self.c
        else:
            yp = _activation(y, self.x_shape, self.dtype, "y")
            _same_device(dev, y=y)
        if stats is None:
            stats = torch.empty(self.stats_shape, dtype=torch.float32, device=dev)
        else:
            _vector(stats, self._stats_numel, torch.float32, dev, "stats")
        ws = torch.empty(self._ws[0], dtype=torch.uint8, device=dev)
        conv3d_group_norm_train_fwd(self._desc(xp, yp, yp), x.data_ptr(), gamma, beta, y, stats, ws,
                                    self._ws[0], _current_stream(dev.index))
        return y, stats

    def backward(self, dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor,
                 beta: torch.Tensor, stats: torch.Tensor, dx: Optional[torch.Tensor] = None,
                 need_dx: bool = True, need_params: bool = True):
        """(dx, dgamma, dbeta) for the gradient dy of y; dx may be given (dy
        itself included), and is None without need_dx, dgamma and dbeta
        (fp32) without need_params."""
        dev = x.device
        xp = _activation(x, self.x_shape, self.dtype, "x")
        dp = _activation(dy, self.x_shape, self.dtype, "dy")
        if dev.index != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return self.backward(dy, x, gamma, beta, stats, dx, need_dx, need_params)
        _vector(gamma, self.c, torch.float32, dev, "gamma")
        _vector(beta, self.c, torch.float32, dev, "beta")
        _vector(stats, self._stats_numel, torch.float32, dev, "stats")
        op = self.c
        if dx is not None:
            if not need_dx:
                raise ValueError("dx is given but not wanted")
            op = _activation(dx, self.x_shape, self.dtype, "dx")
        elif need_dx:
            dx = torch.empty(self.x_shape, dtype=self.dtype, device=dev)
        _same_device(dev, dy=dy, dx=dx)
        dgamma = dbeta = None
        if need_params:
            dgamma = torch.empty(self.c, dtype=torch.float32, device=dev)
            dbeta = torch.empty(self.c, dtype=torch.float32, device=dev)
        ws = torch.empty(self._ws[1], dtype=torch.uint8, device=dev)
        conv3d_group_norm_train_bwd(self._desc(xp, dp, op), dy, x.data_ptr(), gamma, beta, stats, dx,
                                    dgamma, dbeta, ws, self._ws[1], _current_stream(dev.index))
        return dx, dgamma, dbeta


class NormSiluBackward:
    """Backward pass of the channel L2 norm x sqrt(C) x gamma -> SiLU (the
    conv's norm_silu epilogue, conv3d_norm_silu) on one NDHWC bf16 shape."""

    def __init__(self, x_shape: Sequence[int], *, bias: bool = False, gamma: bool = True):
        """bias, gamma: whether their gradients are wanted."""
        self.x_shape = tuple(int(v) for v in x_shape)
        self.want_bias, self.want_gamma = bias, gamma
        self._ws = conv3d_norm_silu_bwd_workspace_bytes(*self.x_shape)

    def __call__(self, value: torch.Tensor, dy: torch.Tensor, gamma: torch.Tensor,
                 dskip: Optional[torch.Tensor] = None, dvalue: Optional[torch.Tensor] = None):
        """(dvalue, dgamma, dbias): dvalue bf16 is the gradient of `value` (the
        pre-norm sum: of the conv's output and of the residual alike), dgamma
        and dbias fp32 (None where not wanted). dskip: the gradient that
        reaches value past the norm. dvalue may be given (dy or dskip
        included)."""
        dev = value.device
        _expect(value, self.x_shape, "value")
        _expect(dy, self.x_shape, "dy")
        _expect(dskip, self.x_shape, "dskip")
        _same_device(dev, dy=dy, dskip=dskip, dvalue=dvalue)
        if dev.index != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return self(value, dy, gamma, dskip, dvalue)
        n, d, h, w, c = self.x_shape
        _vector(gamma, c, torch.bfloat16, dev, "gamma")
        if dvalue is None:
            dvalue = torch.empty_like(value)
        else:
            _expect(dvalue, self.x_shape, "dvalue")
        dgamma = torch.empty(c, dtype=torch.float32, device=dev) if self.want_gamma else None
        dbias = torch.empty(c, dtype=torch.float32, device=dev) if self.want_bias else None
        ws = None
        if self.want_gamma or self.want_bias:
            ws = torch.empty(self._ws, dtype=torch.uint8, device=dev)
        conv3d_norm_silu_bwd(value.data_ptr(), dy, dskip, n, d, h, w, c, gamma, dvalue, dgamma, dbias,
                             ws, self._ws, _current_stream(dev.index))
        return dvalue, dgamma, dbias


def _dense(t: torch.Tensor) -> bool:
    """Whether t's elements fill one run of memory, each once, in any order."""
    if t.is_contiguous():
        return True
    run = 1
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if stride != run:
            return False
        run *= size
    return True


_dtype = operator.attrgetter("dtype")


def _plain_same_addresses(tensors, ptrs, indices) -> bool:
    return list(map(torch.Tensor.data_ptr, tensors)) == ptrs


_same_addresses = getattr(torch._C, "_tensors_data_ptrs_at_indices_equal", _plain_same_addresses)


class _Layouts:
    """Types, sizes and strides of tensors; check(*tensors): whether they are
    as they were."""

    def __init__(self, tensors: Sequence[torch.Tensor]):
        self._seen = self._of(tensors)

    @staticmethod
    def _of(tensors):
        return [(t.dtype, t.shape, t.stride()) for t in tensors]

    def check(self, *tensors: torch.Tensor) -> bool:
        return self._of(tensors) == self._seen


def _guards(tensors: Sequence[torch.Tensor]):
    return torch._C._dynamo.guards.TensorGuards(
        *tensors, dynamic_dims_sizes=[list(t.size()) for t in tensors],
        dynamic_dims_strides=[list(t.stride()) for t in tensors])


def _tells_apart(make) -> bool:
    """Whether make(tensors).check tells tensors apart that differ in one thing."""
    t = torch.zeros(4, 6)
    others = (torch.zeros(24), torch.zeros(4, 5), torch.zeros(6, 4).t(), torch.zeros(4, 8)[:, :6],
              torch.zeros(34).as_strided((6, 4), (6, 1)), torch.zeros(4, 6, dtype=torch.int32))
    pair = make([t, others[0]])
    return (pair.check(t, others[0]) and not pair.check(others[0], t)
            and not any(make([t]).check(u) for u in others))


_layouts_class = None


def _layouts(tensors: Sequence[torch.Tensor]):
    """_Layouts, or one call inside PyTorch for all tensors where this version
    has that and it does the same (146 tensors: 5 us instead of 18 or more)."""
    global _layouts_class
    if _layouts_class is None:
        try:
            _layouts_class = _guards if _tells_apart(_guards) else _Layouts
        except Exception:
            _layouts_class = _Layouts
    return _layouts_class(tensors)


class GradClip:
    """Global norm of many gradient tensors (bf16, fp16 or fp32, mixed), and
    clipping, in place or into `outs` (same shapes and strides, any of the
    types). The lists are kept, and so is the memory that the tensors had at
    the last call: a tensor whose address, type, size or strides have changed
    since (`t.data = ...`) is looked up again, and none moves to where another
    was. For gradients that stay the same tensors from step to step; where each
    step makes new ones (`zero_grad()` sets .grad to None), these here would be
    the old ones, still held: call clip_grads."""

    def __init__(self, grads: Sequence[torch.Tensor],
                 outs: Optional[Sequence[torch.Tensor]] = None, *, norm: str = "l2"):
        if norm not in ("l2", "inf"):
            raise ValueError(f"norm must be 'l2' or 'inf', got {norm!r}")
        self.grads = list(grads)
        self.outs = None if outs is None else list(outs)
        if not self.grads:
            raise ValueError("no gradients")
        if self.outs is not None and len(self.outs) != len(self.grads):
            raise ValueError(f"{len(self.grads)} gradients but {len(self.outs)} outs")
        self._norm_type = GRAD_NORM_INF if norm == "inf" else GRAD_NORM_L2
        self.device = self.grads[0].device
        self._all = self.grads + (self.outs or [])
        self._indices = list(range(len(self._all)))
        self._build()

    def _build(self) -> None:
        index = self.device.index if self.device.type == "cuda" else None
        dtypes = list(map(_dtype, self._all))
        kinds = list(map(_ELT.get, dtypes))
        dense = list(map(torch.Tensor.is_contiguous, self._all))
        for i, (t, kind, dev) in enumerate(zip(self._all, kinds,
                                               map(torch.Tensor.get_device, self._all))):
            if kind is None or dev != index or not (dense[i] or _dense(t)):
                raise ValueError(f"gradient {i % len(self.grads)} must be a dense bf16, fp16 or "
                                 f"fp32 tensor on {self.device}, got {tuple(t.shape)} {t.dtype} "
                                 f"strides {tuple(t.stride())} on {t.device}")
        n = len(self.grads)
        for i, o in enumerate(self.outs or []):
            g = self.grads[i]
            if g.shape != o.shape or (g.stride() != o.stride() and not (dense[i] and dense[n + i])):
                raise ValueError(f"out {i} differs from its gradient in shape or strides")
        # held, so that an address that has not changed is still the same memory
        # (and of that size; one storage may hold many of the tensors)
        held = list(map(torch.Tensor.untyped_storage, self._all))
        self._held = list(dict(zip(map(torch.UntypedStorage.data_ptr, held), held)).values())
        self._held_bytes = list(map(torch.UntypedStorage.nbytes, self._held))
        self._ptrs = list(map(torch.Tensor.data_ptr, self._all))
        numels = list(map(torch.Tensor.numel, self._all))
        self._seen = (numels, dtypes, dense)
        self._strided = [] if all(dense) else [(i, t.shape, t.stride())
                                               for i, t in enumerate(self._all) if not dense[i]]
        self._checks, self._layouts = 0, None
        self._table = make_grads(list(zip(self._ptrs, self._ptrs[n:] or [None] * n, numels, kinds,
                                          kinds[n:] or kinds)))
        self._ws = conv3d_grad_workspace_bytes(self._table)

    def _as_built(self) -> bool:
        """Whether the table still describes the tensors."""
        every = self._all
        if (not _same_addresses(every, self._ptrs, self._indices)
                or list(map(torch.UntypedStorage.nbytes, self._held)) != self._held_bytes):
            return False
        if self._layouts is not None:
            return self._layouts.check(*every)
        self._checks += 1
        if ((list(map(torch.Tensor.numel, every)), list(map(_dtype, every)),
             list(map(torch.Tensor.is_contiguous, every))) != self._seen
                or any((every[i].shape, every[i].stride()) != (shape, stride)
                       for i, shape, stride in self._strided)):
            return False
        if self._checks > 1:             # a list that is used again and again
            self._layouts = _layouts(every)
        return True

    def _rebuild(self) -> None:
        for i, t in enumerate(self._all):
            end = (t.storage_offset() + t.numel()) * t.element_size()
            if t.untyped_storage().nbytes() < end:
                raise ValueError(f"gradient {i % len(self.grads)} holds {t.numel()} elements of "
                                 f"{t.dtype}, its storage is shorter than that")
        self._build()

    def _call(self, run, fresh=False):
        if self.device.index != torch.cuda.current_device():
            with torch.cuda.device(self.device):
                return self._call(run, fresh)
        if not fresh and not self._as_built():
            self._rebuild()
        norm = torch.empty((), dtype=torch.float32, device=self.device)
        ws = torch.empty(self._ws, dtype=torch.uint8, device=self.device)
        run(norm.data_ptr(), ws.data_ptr(), _current_stream(self.device.index))
        return norm

    def norm(self) -> torch.Tensor:
        """The norm over all gradients (fp32, on the GPU); nothing is changed."""
        return self._call(lambda norm, ws, stream: conv3d_grad_norm(
            self._table, self._norm_type, norm, ws, self._ws, stream))

    def clip(self, max_norm: float) -> torch.Tensor:
        """Scales every gradient by min(1, max_norm / (norm + 1e-6)) and
        returns the norm before that (fp32, on the GPU)."""
        return self._clip(max_norm)

    def _clip(self, max_norm: float, fresh=False) -> torch.Tensor:
        return self._call(lambda norm, ws, stream: conv3d_grad_clip(
            self._table, self._norm_type, max_norm, norm, ws, self._ws, stream), fresh)


def clip_grads(grads: Sequence[torch.Tensor], max_norm: float, *, norm: str = "l2") -> torch.Tensor:
    """Clips gradients in place by their global norm and returns it; nothing is
    kept of the list."""
    return GradClip(grads, norm=norm)._clip(max_norm, fresh=True)

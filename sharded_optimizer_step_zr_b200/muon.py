"""The matrix optimizer: orthogonalised momentum updates.

    o = orthogonalize(x)                       # a matrix or a batch [..., m, n] -> bf16

    plan = ZrPlan(shapes, W, rank, ZR_PARTITION_WHOLE_TENSOR)
    muon = ZrMuon(plan, lr=3e-4)               # next to plan.step, for a plan of matrices
    muon.step(grads, master, momentum, param_out)

The work is done by libzr.so's kernels (zr_orthogonalize, zr_muon_*); torch
supplies device memory and streams.
"""
from __future__ import annotations

import contextlib
import functools

from . import (ZR_DTYPE_BF16, ZR_DTYPE_F16, ZR_DTYPE_F32, ZR_MOMENTUM_F32, ZR_MOMENTUM_INT8, ZR_MUON_SCALE_RMS,
               ZR_MUON_SCALE_SPECTRAL, zr_muon_check_result, zr_muon_create, zr_muon_dequantize_momentum,
               zr_muon_destroy, zr_muon_quantize_momentum, zr_muon_scales, zr_muon_set_params,
               zr_muon_set_workspace, zr_muon_step, zr_muon_workspace_bytes, zr_orthogonalize,
               zr_orthogonalize_workspace_bytes, _stream)
from .plan import _require_all

MUON_COEFFS = (3.4445, -4.7750, 2.0315)
_SCALES = {"spectral": ZR_MUON_SCALE_SPECTRAL, "rms": ZR_MUON_SCALE_RMS}
_FORMATS = {"f32": ZR_MOMENTUM_F32, "int8": ZR_MOMENTUM_INT8}
_nothing = contextlib.nullcontext()
_workspace_bytes = functools.lru_cache(maxsize=1024)(zr_orthogonalize_workspace_bytes)     # of the sizes alone


@functools.cache
def _dtypes():
    import torch
    return {torch.float32: ZR_DTYPE_F32, torch.bfloat16: ZR_DTYPE_BF16, torch.float16: ZR_DTYPE_F16}


def _torch_stream(stream, device):
    """A stream argument (a torch stream, or a cudaStream_t as an integer) as a torch stream of `device`."""
    import torch
    if not isinstance(stream, int):
        return stream
    if stream in (0, 1):                   # the null stream, by either of its handles
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(stream, device=device)


def orthogonalize(x, steps=5, coeffs=MUON_COEFFS, eps=1e-7, out=None, workspace=None, stream=None, status=None):
    """Newton-Schulz orthogonalisation of x's matrices (its last two extents;
    any leading ones are a batch), as bf16.

    x: fp32, bf16 or fp16 on a CUDA device, its rows or its columns contiguous
    (a transposed view is orthogonalised through its transpose).  out: a bf16
    tensor of x's shape laid out alike, which may be x itself but not overlap
    it in another way; by default a new one.  workspace: a
    uint8 tensor of at least zr_orthogonalize_workspace_bytes on x's device,
    for calls that must not allocate; calls that share one must be ordered.
    stream: a torch.cuda.Stream of x's device (or a cudaStream_t); by default
    that device's current one.  The call is ordered by that stream alone: the
    caller lets it wait for what writes x (and a given out or workspace), and
    readers of the result wait for it.  What the call allocates is allocated
    on that stream; a tensor of another stream may be dropped as soon as the
    call has returned.

    status: an int32 tensor of at least one element on x's device; the call's
    work sets its first element to 0, or to 1 if a wait inside a kernel ran
    out, in which case the result is not valid (the first 32-bit word of a
    given workspace says the same).  Not expected, and looked at nowhere else:
    a call that is not given one cannot tell.

    Not differentiable: a tensor that requires a gradient is refused where
    gradients are recorded."""
    import torch
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"x: expected a torch tensor, got {type(x).__name__}")
    dtype = _dtypes().get(x.dtype)
    if dtype is None:
        raise ValueError(f"x: dtype {x.dtype}, expected float32, bfloat16 or float16")
    device = x.device
    if device.type != "cuda":
        raise ValueError(f"x: must be on a CUDA device, is on {device}")
    if x.dim() < 2:
        raise ValueError(f"x: {x.dim()} dimensions, expected at least 2")
    if torch.is_grad_enabled() and (x.requires_grad or getattr(out, "requires_grad", False)):
        raise ValueError("x or out requires a gradient, which the result does not carry: detach it, or call under "
                         "torch.no_grad()")
    if stream is not None and not isinstance(stream, int) and stream.device != device:
        raise ValueError(f"stream: of {stream.device}, x is on {device}")
    side = None                            # the given stream, where it is not the current one
    if stream is not None:
        side = _torch_stream(stream, device)
        if side.cuda_stream == torch.cuda.current_stream(device).cuda_stream:
            side = None
    # A block of the current stream's memory may still be read or written by
    # what that stream has queued, which `side` does not wait for.
    allocating = torch.cuda.stream(side) if side is not None else _nothing
    given = [x] + [t for t in (out, workspace, status) if isinstance(t, torch.Tensor)] if side is not None else ()
    if out is None:
        by_columns = x.shape[-1] > 1 and x.stride(-1) != 1 and (x.stride(-2) == 1 or x.shape[-2] == 1)
        with allocating:
            out = torch.empty(x.mT.shape if by_columns else x.shape, dtype=torch.bfloat16, device=device)
        if by_columns:
            out = out.mT
    else:
        if not isinstance(out, torch.Tensor):
            raise TypeError(f"out: expected a torch tensor, got {type(out).__name__}")
        if out.dtype != torch.bfloat16 or out.shape != x.shape or out.device != device:
            raise ValueError(f"out: {out.dtype} {tuple(out.shape)} on {out.device}, expected torch.bfloat16 "
                             f"{tuple(x.shape)} on {device}")
    if status is not None:
        if not isinstance(status, torch.Tensor):
            raise TypeError(f"status: expected a torch tensor, got {type(status).__name__}")
        _require_all([(status, "status", torch.int32, 1, False)], device)
    result = out
    if x.numel() == 0:
        if status is not None:
            with torch.cuda.stream(side) if side is not None else _nothing:
                status.view(-1)[:1].zero_()
        return result

    def rows(t):         # columns contiguous
        return t.shape[-1] == 1 or t.stride(-1) == 1

    if not (rows(x) and rows(out)):
        if not (rows(x.mT) and rows(out.mT)):
            raise ValueError(f"x and out must both have contiguous rows or both contiguous columns, "
                             f"have strides {x.stride()} and {out.stride()}")
        x, out = x.mT, out.mT
    m, n = x.shape[-2:]

    def strides(t, what):
        """Batch and row stride, the leading extents as one batch."""
        if t.dim() > 3:
            try:
                t = t.view(-1, m, n)
            except RuntimeError as e:
                raise ValueError(f"{what}: its leading extents are not one stride apart") from e
        return (t.stride(0) if t.dim() == 3 and t.shape[0] > 1 else 0), (t.stride(-2) if m > 1 else n)

    batch = x.numel() // (m * n)
    x_batch, x_row = strides(x, "x")
    o_batch, o_row = strides(out, "out")
    need = _workspace_bytes(batch, m, n)
    with torch.cuda.device(device) if torch.cuda.current_device() != device.index else _nothing:
        if workspace is None:
            with allocating:               # freed when this call returns, to the stream's own memory
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
        else:
            _require_all([(workspace, "workspace", torch.uint8, need, False)], device)
        if side is not None:               # memory that is freed on one stream and used on another
            for t in given:
                t.record_stream(side)
            if not any(t is result for t in given):
                result.record_stream(torch.cuda.current_stream(device))
        zr_orthogonalize(x, dtype, batch, m, n, x_batch, x_row, out, o_batch, o_row, coeffs, eps, steps, workspace,
                         workspace.numel(), stream)
        if status is not None:
            with torch.cuda.stream(side) if side is not None else _nothing:
                status.view(-1)[:1].copy_(workspace[:4].view(torch.int32))
    return result


class ZrMuon:
    """The Muon step (zr_muon_step) on a ZrPlan of matrices that owns whole
    tensors, with a torch-allocated workspace.  momentum_format: "f32", or
    "int8" for codes with one fp32 scale per 256 elements; scale: "rms" (0.2
    sqrt(max(m, n))) or "spectral" (sqrt(max(1, m / n))).  The step follows
    the plan's gather targets and parameter layout; the plan is kept alive and
    must not be closed before this object.

    The workspace is allocated, and its tables are written, on `stream` (by
    default the current one); steps on other streams wait for that, and for
    one another, by the caller's means.  The object may be dropped while its
    calls still run, unless a graph captured them: it outlives the replays.
    A stream given by its handle outlives the object."""

    def __init__(self, plan, lr=3e-4, momentum=0.95, weight_decay=0.1, nesterov=True, ns_steps=5,
                 ns_coeffs=MUON_COEFFS, eps=1e-7, scale="rms", momentum_format="f32", stream=None):
        import torch
        if scale not in _SCALES:
            raise ValueError(f"scale is one of {sorted(_SCALES)}")
        if momentum_format not in _FORMATS:
            raise ValueError(f"momentum_format is one of {sorted(_FORMATS)}")
        self.handle = 0
        self.plan = plan
        self.momentum_format = momentum_format
        self.params = dict(lr=lr, momentum=momentum, weight_decay=weight_decay, nesterov=nesterov,
                           scale=_SCALES[scale], coeffs=tuple(ns_coeffs), eps=eps, steps=ns_steps)
        self.handle = zr_muon_create(plan.handle, momentum_format=_FORMATS[momentum_format], **self.params)
        self.n_scales = zr_muon_scales(self.handle)
        self.workspace_bytes = zr_muon_workspace_bytes(self.handle)
        self.workspace = None
        self._streams = set()                  # that both workspaces are known to be used on
        self._plan_workspace = None
        if plan.device is not None:
            with torch.cuda.device(plan.device):
                with torch.cuda.stream(_torch_stream(stream, plan.device)) if stream is not None else _nothing:
                    self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=plan.device)
                zr_muon_set_workspace(self.handle, self.workspace, self.workspace.numel(), self._use(stream))

    def _use(self, stream):
        """Before a call on `stream`: this workspace and the plan's (which
        holds the gather targets) are not handed out again before that stream
        is done with them.  Returns the stream's handle."""
        import torch
        if self.workspace is None:
            return stream
        device = self.plan.device
        if stream is None and torch.cuda.current_device() != device.index:
            return stream                      # refused by the library: nothing runs
        if getattr(stream, "device", device) != device:
            raise ValueError(f"stream: of {stream.device}, the plan is on {device}")
        if self._plan_workspace is not self.plan.workspace:
            self._plan_workspace = self.plan.workspace
            self._streams.clear()
        handle = _stream(stream)
        if handle not in self._streams:
            s = _torch_stream(handle, device)
            for t in (self.workspace, self._plan_workspace):
                t.record_stream(s)
            self._streams.add(handle)
        return handle

    def set_lr(self, lr):
        """The learning rate of the following steps."""
        self.params["lr"] = lr
        zr_muon_set_params(self.handle, **self.params)

    def empty_momentum(self):
        """A zero momentum state: an fp32 tensor, or (codes, scales)."""
        import torch
        n, dev = max(self.plan.owned_numel, 8), self.plan.device
        if self.momentum_format == "f32":
            return torch.zeros(n, dtype=torch.float32, device=dev)
        return (torch.zeros(n, dtype=torch.int8, device=dev),
                torch.zeros(max(self.n_scales, 4), dtype=torch.float32, device=dev))

    def _momentum(self, momentum):
        import torch
        n = self.plan.owned_numel
        if self.momentum_format == "f32":
            return momentum, None, [(momentum, "momentum", torch.float32, n, False)]
        codes, scales = momentum
        return codes, scales, [(codes, "momentum codes", torch.int8, n, False),
                               (scales, "momentum scales", torch.float32, self.n_scales, False)]

    def step(self, grads, master, momentum, param_out, stream=None):
        """zr_muon_step: W bf16 gradient buffers, fp32 master and the momentum
        state (an fp32 tensor, or the pair (codes, scales)), all in owned
        order; param_out as ZrPlan.step's (None with gather targets).
        Asynchronous on `stream`."""
        import torch
        plan, n = self.plan, self.plan.owned_numel
        first, scales, specs = self._momentum(momentum)
        if len(grads) != plan.world_size:
            raise ValueError(f"grads: {len(grads)} buffers, the plan has W = {plan.world_size}")
        if n:
            _require_all([(g, f"grads[{w}]", torch.bfloat16, n, False) for w, g in enumerate(grads)] +
                         [(master, "master", torch.float32, n, False)] + specs +
                         [(param_out, "param_out", torch.bfloat16, plan.param_out_numel, False)], plan.device)
        zr_muon_step(self.handle, grads, master, first, scales, param_out, self._use(stream))

    def quantize_momentum(self, momentum, codes, scales, stream=None):
        """zr_muon_quantize_momentum: an fp32 momentum into (codes, scales)."""
        self._check_conversion(momentum, codes, scales)
        zr_muon_quantize_momentum(self.handle, momentum, codes, scales, self._use(stream))

    def dequantize_momentum(self, codes, scales, momentum, stream=None):
        """zr_muon_dequantize_momentum: (codes, scales) into an fp32 momentum."""
        self._check_conversion(momentum, codes, scales)
        zr_muon_dequantize_momentum(self.handle, codes, scales, momentum, self._use(stream))

    def _check_conversion(self, momentum, codes, scales):
        import torch
        n = self.plan.owned_numel
        _require_all([(momentum, "momentum", torch.float32, n, False), (codes, "codes", torch.int8, n, False),
                      (scales, "scales", torch.float32, self.n_scales, False)], self.plan.device)

    def check_result(self, stream=None):
        """True if a wait inside a step's kernels ever ran out (synchronises)."""
        return zr_muon_check_result(self.handle, self._use(stream))

    def close(self):
        if self.handle:
            zr_muon_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

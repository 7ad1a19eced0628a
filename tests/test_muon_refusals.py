"""Calls of the matrix optimizer that would give wrong results and are refused
(no GPU: a call that is let through ends at the device check instead), and the
documented sizes of workspaces."""
import pytest
import torch

import sharded_optimizer_step_zr_b200 as zr
from test_muon_abi import P, ortho

F32, BF16, F16 = zr.ZR_DTYPE_F32, zr.ZR_DTYPE_BF16, zr.ZR_DTYPE_F16
SIZE = 2 * 8 * 16                # elements of ortho()'s default batch


def status(**kw):
    try:
        ortho(**kw)
    except zr.ZrError as e:
        return e.status
    return zr.ZR_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are no device's")
@pytest.mark.parametrize("kw,refused", [
    (dict(dtype=F32), True),                                     # bf16 over fp32 at the same address
    (dict(dtype=F32, batch=1), True),
    (dict(dtype=BF16), False),                                   # in place
    (dict(dtype=F16), False),
    (dict(dtype=BF16, xr=20, xb=160, orow=20, ob=160), False),
    (dict(dtype=BF16, xr=20, xb=160), True),                     # from the same address, other strides
    (dict(dtype=BF16, xb=0), True),
    (dict(dtype=BF16, batch=1, xb=5, ob=200), False),            # a batch of one: its stride is not looked at
    (dict(dtype=BF16, batch=1, m=1, xr=40, orow=16), False),
    (dict(dtype=BF16, out=P + 2), True),                         # dense, shifted
    (dict(dtype=BF16, out=P + 2 * SIZE - 2), True),
    (dict(dtype=BF16, out=P + 2 * SIZE), False),                 # behind it
    (dict(dtype=BF16, out=P - 2 * SIZE), False),
    (dict(dtype=BF16, out=P - 2 * SIZE + 2), True),
    (dict(dtype=F32, out=P + 4 * SIZE - 2), True),
    (dict(dtype=F32, out=P + 4 * SIZE), False),
    (dict(dtype=BF16, xr=32, xb=256, orow=32, ob=256, out=P + 32), False),   # the halves of one buffer's rows
])
def test_a_result_written_over_its_source_is_refused(kw, refused):
    got = status(**kw)
    assert (got == zr.ZR_ERR_INVALID_ARG) == refused, got
    assert got != zr.ZR_OK


class OnDevice(torch.Tensor):
    """A host tensor that says it is on a CUDA device: far enough for the checks of arguments."""
    device = torch.device("cuda", 0)


def test_a_tensor_that_requires_a_gradient_is_refused():
    from sharded_optimizer_step_zr_b200.muon import orthogonalize
    x = torch.zeros(0, 4).as_subclass(OnDevice)
    out = torch.zeros(0, 4, dtype=torch.bfloat16).as_subclass(OnDevice)
    leaf = torch.zeros(0, 4).requires_grad_().as_subclass(OnDevice)
    for bad in (leaf, leaf * 2):
        assert bad.requires_grad
        with pytest.raises(ValueError, match="gradient"):
            orthogonalize(bad, out=out)
        with torch.no_grad():
            assert orthogonalize(bad, out=out) is out
    assert orthogonalize(x, out=out) is out
    assert orthogonalize(leaf.detach().as_subclass(OnDevice), out=out) is out
    out.requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        orthogonalize(x, out=out)


def test_a_status_of_the_wrong_kind_is_refused():
    from sharded_optimizer_step_zr_b200.muon import orthogonalize
    x = torch.zeros(0, 4).as_subclass(OnDevice)
    out = torch.zeros(0, 4, dtype=torch.bfloat16).as_subclass(OnDevice)
    with pytest.raises(TypeError, match="status"):
        orthogonalize(x, out=out, status=0)
    for bad in (torch.zeros(1), torch.zeros(0, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)[::2],
                torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="status"):            # the last one: on the host
            orthogonalize(x, out=out, status=bad)


@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 640, 1), (1, 1, 640), (1, 4096, 3), (7, 130, 66), (24, 128, 4096), (3, 2048, 8192),
                                   (1, 1 << 24, 1), (1 << 20, 4, 4)])
def test_workspaces_take_the_documented_bytes(shape):
    """8 bytes per element of X and 4 per element of a Gram matrix, columns
    rounded up to 64; the diagonals, scales, counters and sums of squares; each
    of twelve regions on 256 bytes."""
    b, m, n = shape
    g = min(m, n)

    def up64(k):
        return -(-k // 64) * 64
    copies = 8 * b * m * up64(n) + 4 * b * g * up64(g)
    small = 8 * b * g + 16 * b + 8 * b * -(-m // 8) * -(-n // 1024)
    got = zr.zr_orthogonalize_workspace_bytes(b, m, n)
    assert copies <= got <= copies + small + 12 * 256
    if b * m * n <= 1 << 24:
        p = zr.zr_plan_create([(b, m, n)], 1, 0, zr.ZR_PARTITION_WHOLE_TENSOR, 25 << 20)
        u = zr.zr_muon_create(p, 3e-4, 0.95, 0.1, True, zr.ZR_MUON_SCALE_RMS, (3.4445, -4.775, 2.0315), 1e-7, 5,
                              zr.ZR_MOMENTUM_F32)
        tiles = b * -(-m * n // 2048)
        got = zr.zr_muon_workspace_bytes(u)
        maps = 16 * 128                              # of the one shape
        assert copies <= got <= copies + 8 * b * g + 32 * b + 40 * tiles + maps + 20 * 256
        zr.zr_muon_destroy(u)
        zr.zr_plan_destroy(p)


class Recorder:
    """A workspace that keeps the streams it is recorded on."""

    def __init__(self):
        self.streams = []

    def record_stream(self, s):
        self.streams.append(s)


def test_a_stream_of_another_device_is_refused_and_not_kept(monkeypatch):
    """An event on it, when the workspace is freed, would fail long after the call."""
    from types import SimpleNamespace
    from sharded_optimizer_step_zr_b200 import muon
    own, other = torch.device("cuda", 0), torch.device("cuda", 1)
    current = {"device": 1}
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current["device"])
    monkeypatch.setattr(muon, "_stream", lambda s: 40 if s is None else s if isinstance(s, int) else s.cuda_stream)
    monkeypatch.setattr(muon, "_torch_stream", lambda s, device: (s, device))
    m = muon.ZrMuon.__new__(muon.ZrMuon)
    m.handle, m._streams, m._plan_workspace = 0, set(), None
    m.workspace, m.plan = Recorder(), SimpleNamespace(device=own, workspace=Recorder())
    with pytest.raises(ValueError, match="stream"):
        m._use(SimpleNamespace(device=other, cuda_stream=48))
    assert m._use(None) is None                      # the current device is the other one
    assert m.workspace.streams == m.plan.workspace.streams == []
    current["device"] = 0
    for s in (None, None, 40, SimpleNamespace(device=own, cuda_stream=56), 56, SimpleNamespace(cuda_stream=64)):
        m._use(s)
    assert m.workspace.streams == m.plan.workspace.streams == [(40, own), (56, own), (64, own)]
    m.plan.workspace = Recorder()                    # bound again
    m._use(40)
    assert m.plan.workspace.streams == [(40, own)]

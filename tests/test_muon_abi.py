"""The matrix optimizer's C ABI without a GPU: argument checks, sizes and
table counts (nothing here launches)."""
import ctypes

import pytest

import sharded_optimizer_step_zr_b200 as zr
from sharded_optimizer_step_zr_b200.muon import MUON_COEFFS

P = 1 << 20          # a plausible address; no call here gets as far as using it


def ortho(dtype=zr.ZR_DTYPE_F32, batch=2, m=8, n=16, xb=None, xr=None, ob=None, orow=None, x=P, out=P, coeffs=MUON_COEFFS,
          eps=1e-7, steps=5, ws=P, ws_bytes=1 << 40):
    xr = n if xr is None else xr
    orow = n if orow is None else orow
    xb = m * xr if xb is None else xb
    ob = m * orow if ob is None else ob
    zr.zr_orthogonalize(x, dtype, batch, m, n, xb, xr, out, ob, orow, coeffs, eps, steps, ws, ws_bytes, 0)


def refused(status, **kw):
    with pytest.raises(zr.ZrError) as e:
        ortho(**kw)
    assert e.value.status == status, (kw, e.value)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(dtype=-1), dict(batch=-1), dict(m=-1), dict(n=-1), dict(x=0), dict(out=0),
    dict(steps=0), dict(steps=33), dict(eps=0.0), dict(eps=-1e-7), dict(eps=2.0), dict(eps=float("nan")),
    dict(coeffs=(float("nan"), 0, 0)), dict(coeffs=(1e6, 0, 0)), dict(coeffs=(3.4445, 4.775, 2.03)),
    dict(xr=-1), dict(xb=-1), dict(orow=15), dict(ob=8 * 16 - 1), dict(xr=1 << 50), dict(ob=1 << 60),
])
def test_orthogonalize_refuses_bad_arguments(kw):
    refused(zr.ZR_ERR_INVALID_ARG, **kw)


def test_orthogonalize_refuses_misaligned_and_small_workspaces():
    refused(zr.ZR_ERR_ALIGNMENT, x=P + 2)
    refused(zr.ZR_ERR_ALIGNMENT, dtype=zr.ZR_DTYPE_BF16, x=P + 1)
    refused(zr.ZR_ERR_ALIGNMENT, out=P + 1)
    refused(zr.ZR_ERR_ALIGNMENT, ws=P + 128)
    refused(zr.ZR_ERR_NO_WORKSPACE, ws=0)
    need = zr.zr_orthogonalize_workspace_bytes(2, 8, 16)
    refused(zr.ZR_ERR_NO_WORKSPACE, ws_bytes=need - 1)


@pytest.mark.parametrize("shape", [(1, 1 << 25, 4), (1, 4, 1 << 25), (1 << 25, 4, 4), (1, 1 << 18, 1 << 18),
                                   (1 << 24, 1 << 12, 1 << 12)])
def test_orthogonalize_refuses_shapes_beyond_its_indices(shape):
    with pytest.raises(zr.ZrError) as e:
        zr.zr_orthogonalize_workspace_bytes(*shape)
    assert e.value.status == zr.ZR_ERR_UNSUPPORTED
    b, m, n = shape
    refused(zr.ZR_ERR_UNSUPPORTED, batch=b, m=m, n=n, xb=0, xr=0, ob=m * n, orow=n)


@pytest.mark.parametrize("shape", [(0, 4, 4), (2, 0, 4), (2, 4, 0)])
def test_orthogonalize_of_nothing_does_nothing(shape):
    b, m, n = shape
    ortho(batch=b, m=m, n=n, x=0, out=0, ws=0, ws_bytes=0)
    assert zr.zr_orthogonalize_workspace_bytes(b, m, n) >= 0


def test_workspace_is_monotone_and_covers_the_copies():
    last = 0
    for b, m, n in [(1, 1, 1), (1, 16, 16), (3, 16, 16), (3, 100, 16), (3, 100, 700), (3, 2048, 2048)]:
        w = zr.zr_orthogonalize_workspace_bytes(b, m, n)
        assert w >= 8 * b * m * n + 4 * b * min(m, n) ** 2 and w >= last and w % 256 == 0
        last = w


def plan(shapes, W=2, rank=0, mode=zr.ZR_PARTITION_WHOLE_TENSOR, **kw):
    return zr.zr_plan_create(shapes, W, rank, mode, 25 << 20, **kw)


def create(p, lr=3e-4, momentum=0.95, weight_decay=0.1, nesterov=True, scale=zr.ZR_MUON_SCALE_RMS, coeffs=MUON_COEFFS,
           eps=1e-7, steps=5, momentum_format=zr.ZR_MOMENTUM_F32):
    return zr.zr_muon_create(p, lr, momentum, weight_decay, nesterov, scale, coeffs, eps, steps, momentum_format)


@pytest.mark.parametrize("kw", [dict(lr=-1.0), dict(lr=float("inf")), dict(momentum=1.0), dict(momentum=-0.1),
                                dict(momentum=float("nan")), dict(weight_decay=-1.0), dict(weight_decay=float("nan")),
                                dict(scale=2), dict(momentum_format=2), dict(steps=0), dict(eps=0.0),
                                dict(coeffs=(100.0, 0.0, 0.0))])
def test_muon_create_refuses_bad_parameters(kw):
    p = plan([(8, 8), (4, 8)])
    with pytest.raises(zr.ZrError) as e:
        create(p, **kw)
    assert e.value.status == zr.ZR_ERR_INVALID_ARG
    u = create(p)
    if "momentum_format" not in kw:
        full = dict(lr=3e-4, momentum=0.95, weight_decay=0.1, nesterov=True, scale=1, coeffs=MUON_COEFFS, eps=1e-7, steps=5)
        with pytest.raises(zr.ZrError):
            zr.zr_muon_set_params(u, **{**full, **kw})
    zr.zr_muon_destroy(u)
    zr.zr_plan_destroy(p)


@pytest.mark.parametrize("shapes,kw,status", [
    ([(8, 8), (8,)], {}, zr.ZR_ERR_INVALID_ARG),                       # a vector
    ([(8, 8), ()], {}, zr.ZR_ERR_INVALID_ARG),                         # a scalar
    ([(64, 64), (64, 64), (8,)], dict(rank=1), zr.ZR_ERR_INVALID_ARG),  # a vector on another rank
    ([(8, 8)], dict(mode=zr.ZR_PARTITION_FLAT), zr.ZR_ERR_UNSUPPORTED),
    ([(8, 8)], dict(max_grad_norm=1.0), zr.ZR_ERR_UNSUPPORTED),
    ([(1 << 18, 1 << 18)], {}, zr.ZR_ERR_UNSUPPORTED),
])
def test_muon_create_refuses_plans_it_cannot_step(shapes, kw, status):
    p = plan(shapes, **kw)
    with pytest.raises(zr.ZrError) as e:
        create(p)
    assert e.value.status == status
    zr.zr_plan_destroy(p)


@pytest.mark.parametrize("W,mode", [(1, zr.ZR_PARTITION_FLAT), (1, zr.ZR_PARTITION_WHOLE_TENSOR),
                                    (3, zr.ZR_PARTITION_WHOLE_TENSOR)])
def test_scales_count_blocks_of_256_per_matrix(W, mode):
    shapes = [(16, 16), (3, 5, 100), (0, 7), (257, 1), (1, 1), (2, 4, 128, 2)]
    total = 0
    for rank in range(W):
        p = plan(shapes, W=W, rank=rank, mode=mode)
        u = create(p, momentum_format=zr.ZR_MOMENTUM_INT8)
        own = {s["tensor"] for s in zr.zr_plan_segments(p) if s["owner"] == rank and s["length"] > 0}
        want = 0
        for t in own:
            *lead, m, n = shapes[t]
            count = 1
            for d in lead:
                count *= d
            want += count * -(-m * n // 256)
        assert zr.zr_muon_scales(u) == want
        assert zr.zr_muon_workspace_bytes(u) >= 256
        total += want
        zr.zr_muon_destroy(u)
        zr.zr_plan_destroy(p)
    assert total == 1 + 3 * 2 + 2 + 1 + 8


def test_calls_before_the_workspace_are_refused():
    p = plan([(8, 8)], W=1)
    u = create(p)
    for call in (lambda: zr.zr_muon_step(u, [P], P, P, None, P, 0),
                 lambda: zr.zr_muon_quantize_momentum(u, P, P, P, 0),
                 lambda: zr.zr_muon_dequantize_momentum(u, P, P, P, 0),
                 lambda: zr.zr_muon_check_result(u, 0),
                 lambda: zr.zr_muon_set_workspace(u, P, 1 << 40, 0)):      # the plan has none yet
        with pytest.raises(zr.ZrError) as e:
            call()
        assert e.value.status == zr.ZR_ERR_NO_WORKSPACE
    with pytest.raises(zr.ZrError) as e:
        zr.zr_muon_set_workspace(u, P + 8, 1 << 40, 0)
    assert e.value.status == zr.ZR_ERR_ALIGNMENT
    with pytest.raises(zr.ZrError) as e:
        zr.zr_muon_set_workspace(u, P, 16, 0)
    assert e.value.status == zr.ZR_ERR_NO_WORKSPACE
    zr.zr_muon_destroy(u)
    zr.zr_plan_destroy(p)


def test_null_handles_are_refused():
    lib = zr.lib_handle()
    out = ctypes.c_uint64()
    assert lib.zr_muon_create(None, None, 0, None) == zr.ZR_ERR_INVALID_ARG
    assert lib.zr_muon_workspace_bytes(None, ctypes.byref(out)) == zr.ZR_ERR_INVALID_ARG
    assert lib.zr_muon_step(None, None, None, None, None, None, None) == zr.ZR_ERR_INVALID_ARG
    assert lib.zr_orthogonalize_workspace_bytes(1, 1, 1, None) == zr.ZR_ERR_INVALID_ARG
    lib.zr_muon_destroy(None)


def test_python_checks_its_tensors():
    import torch
    from sharded_optimizer_step_zr_b200.muon import orthogonalize
    with pytest.raises(TypeError):
        orthogonalize([[1.0]])
    with pytest.raises(ValueError, match="dtype"):
        orthogonalize(torch.zeros(4, 4, dtype=torch.float64))
    with pytest.raises(ValueError, match="CUDA"):
        orthogonalize(torch.zeros(4, 4))

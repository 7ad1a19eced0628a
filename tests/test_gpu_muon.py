"""Orthogonalisation and the Muon step against plain implementations in 64
bits (or, where every operation is one fp32 rounding, bit for bit).

Tolerances.  Orthogonalisation: the norm of the error over the norm of the
result.  The result's own rounding to bf16 is off by at most half a step,
2^-8 of each value.  A step of the iteration rounds X, A and B to fp16; what
is rounded without a correction (A and B off their diagonals) enters with half
a step, 2^-11, of a product that is no larger than the iterate itself.  So
2^-8 + steps * 2^-11.  Matrices of the Muon step add lr * s * ||O|| * steps *
2^-11 to fp32 master weights, whose own three roundings are 2^-24 each.
"""
import math

import pytest
import torch

import sharded_optimizer_step_zr_b200 as zr
from sharded_optimizer_step_zr_b200.muon import MUON_COEFFS, ZrMuon, orthogonalize
from sharded_optimizer_step_zr_b200.plan import ZrPlan

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16_HALF, F16_HALF, F32_HALF = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24


def reference(x, steps=5, coeffs=MUON_COEFFS, eps=1e-7):
    x = x.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    a, b, c = coeffs
    for _ in range(steps):
        g = x @ x.mT
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.mT if tall else x


def assert_orthogonal(got, x, steps=5, **kw):
    want = reference(x, steps, **kw)
    assert got.dtype == torch.bfloat16 and got.shape == x.shape
    err = (got.double() - want).flatten(-2).norm(dim=-1)
    norm = want.flatten(-2).norm(dim=-1)
    tol = BF16_HALF + steps * F16_HALF
    assert torch.all(err <= tol * norm), (err / norm).max().item()


def randn(*shape, seed=0, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (7, 1), (2, 3), (16, 16), (63, 65), (65, 63), (64, 64), (127, 129),
                                   (128, 256), (256, 128), (129, 257), (257, 511), (1, 3000), (3000, 1), (5, 2049),
                                   (700, 900), (900, 700)])
def test_shapes_and_types(shape, dtype):
    x = randn(*shape, seed=shape[0] * 31 + shape[1], dtype=dtype)
    assert_orthogonal(orthogonalize(x), x)


@pytest.mark.parametrize("batch", [2, 5, 150])
def test_batches(batch):
    x = randn(batch, 40, 72, seed=batch)
    assert_orthogonal(orthogonalize(x), x)
    y = randn(2, batch, 33, 21, seed=batch)
    assert_orthogonal(orthogonalize(y), y)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 8])
def test_steps(steps):
    x = randn(2, 130, 200, seed=steps)
    assert_orthogonal(orthogonalize(x, steps=steps), x, steps)


def test_other_coefficients_and_eps():
    x = randn(96, 160)
    cubic = (1.5, -0.5, 0.0)
    assert_orthogonal(orthogonalize(x, steps=12, coeffs=cubic), x, 12, coeffs=cubic)
    small = x * 1e-4
    assert_orthogonal(orthogonalize(small, eps=0.5), small, eps=0.5)


def test_few_strong_directions_keep_the_weak_ones():
    """16 directions 400 times stronger than the rest: the weak ones are the
    small difference that a 16-bit X alone loses."""
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(512, 16, generator=g, device=DEV) @ torch.randn(16, 640, generator=g, device=DEV)
    x = x + 0.05 * torch.randn(512, 640, generator=g, device=DEV)
    assert_orthogonal(orthogonalize(x), x)


@pytest.mark.parametrize("scale", [1e-25, 1e-12, 1e12, 1e30])
def test_magnitudes(scale):
    x = randn(60, 100) * scale
    assert_orthogonal(orthogonalize(x, eps=1e-30), x, eps=1e-30)


def test_a_norm_far_below_eps_gives_next_to_nothing():
    """X_0's elements below 2^-46 are zero in the scratch; what the exact
    iteration makes of them is at most a^5 times as much."""
    x = randn(60, 100) * 1e-25
    assert orthogonalize(x).abs().max() <= 2.0 ** -46 * MUON_COEFFS[0] ** 5


def test_views():
    big = randn(4, 50, 96)
    for x in (big[:, :, 5:70], big[1:3, 3:, :64], big[::2], big[0, ::3, 1:], big.mT, big[:, :, 7:50].mT,
              big[1].unsqueeze(0).expand(3, 50, 96), randn(3, 1, 64).expand(3, 20, 64)):
        assert_orthogonal(orthogonalize(x), x)
    with pytest.raises(ValueError, match="contiguous"):
        orthogonalize(big[:, :, ::2])


def test_output_views_leave_their_surroundings():
    x = randn(3, 70, 45)
    whole = torch.full((3, 80, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    out = whole[:, 2:72, 3:48]
    assert orthogonalize(x, out=out) is out
    assert_orthogonal(out, x)
    rest = torch.ones_like(whole, dtype=torch.bool)
    rest[:, 2:72, 3:48] = False
    assert torch.all(whole[rest] == 7.0)


def test_in_place_and_given_workspace():
    x = randn(2, 130, 70, dtype=torch.bfloat16)
    want = orthogonalize(x)
    ws = torch.empty(zr.zr_orthogonalize_workspace_bytes(2, 130, 70), dtype=torch.uint8, device=DEV)
    y = x.clone()
    assert orthogonalize(y, out=y, workspace=ws) is y
    assert torch.equal(y, want)
    assert int(ws[:4].view(torch.int32).item()) == 0
    with pytest.raises(ValueError, match="workspace"):
        orthogonalize(x, workspace=ws[:-1])


@pytest.mark.parametrize("shape", [(0, 4, 5), (2, 0, 5), (2, 4, 0)])
def test_nothing(shape):
    x = torch.zeros(shape, device=DEV)
    assert orthogonalize(x).shape == shape


def test_zero_and_non_finite_matrices_touch_no_other():
    x = randn(6, 40, 70)
    clean = orthogonalize(x)
    x[1] = 0.0
    x[2, 3, 5] = float("nan")
    x[4, 0, 0] = float("inf")
    got = orthogonalize(x)
    for i in (0, 3, 5):
        assert torch.equal(got[i], clean[i])
    assert torch.all(got[1] == 0)
    assert torch.isnan(got[2]).all()
    assert torch.isnan(got[4]).any()


def test_same_bits_every_time_and_on_any_stream():
    x = randn(3, 300, 500)
    want = orthogonalize(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [orthogonalize(x, stream=side) for _ in range(4)]
    with torch.cuda.stream(side):
        outs.append(orthogonalize(x))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(o, want) for o in outs)


def test_graph_replays():
    x = randn(2, 100, 164)
    ws = torch.empty(zr.zr_orthogonalize_workspace_bytes(2, 100, 164), dtype=torch.uint8, device=DEV)
    out = torch.empty(2, 100, 164, dtype=torch.bfloat16, device=DEV)
    orthogonalize(x, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        orthogonalize(x, out=out, workspace=ws)
    for seed in (5, 6):
        x.copy_(randn(2, 100, 164, seed=seed))
        graph.replay()
        assert torch.equal(out, orthogonalize(x))


# ---------------------------------------------------------------------------
# the Muon step
# ---------------------------------------------------------------------------

SETS = {
    "aligned": [(64, 128), (128, 64), (64, 64), (2, 32, 64)],
    "odd": [(33, 17), (5, 130, 66), (1, 77), (77, 1), (1, 1), (50, 51)],
    "tiny": [(512, 512), (512, 1024), (1024, 512)],
}


class Job:
    """One rank's buffers, and the same step in plain torch: the momentum in
    fp32 with the kernels' operations, the rest in 64 bits."""

    def __init__(self, shapes, W, rank, fmt="f32", seed=0, layout=zr.ZR_PARAMS_OWNED, mode=zr.ZR_PARTITION_WHOLE_TENSOR, **kw):
        self.hp = dict(lr=0.01, momentum=0.9, weight_decay=0.1, nesterov=True, ns_steps=5, scale="rms")
        self.hp.update(kw)
        self.plan = ZrPlan(shapes, W, rank, mode, device=DEV)
        if layout != zr.ZR_PARAMS_GLOBAL:
            self.plan.set_param_layout(layout)
        self.muon = ZrMuon(self.plan, momentum_format=fmt, **self.hp)
        self.W, self.fmt, self.n = W, fmt, self.plan.owned_numel
        own = {s["tensor"] for s in self.plan.segments() if s["owner"] == rank and s["length"] > 0}
        self.shapes = [shapes[t] for t in sorted(own)]
        self.gen = torch.Generator(device=DEV).manual_seed(seed)
        self.master = self.rand(0.02)
        self.momentum = self.muon.empty_momentum()
        self.param = torch.full((max(self.plan.param_out_numel, 8),), 3.0, dtype=torch.bfloat16, device=DEV)
        self.ref_master = self.master.double()
        self.ref_momentum = torch.zeros(self.n, device=DEV)
        self.slack = torch.zeros((), dtype=torch.float64, device=DEV)

    def rand(self, sigma):
        t = torch.zeros(max(self.n, 8), device=DEV)
        t[:self.n] = torch.randn(self.n, generator=self.gen, device=DEV) * sigma
        return t

    def new_grads(self, sigma=1e-3):
        self.grads = [self.rand(sigma).to(torch.bfloat16) for _ in range(self.W)]

    def matrices(self, flat):
        at = 0
        for s in self.shapes:
            size = math.prod(s)
            yield flat[at:at + size].view(-1, s[-2], s[-1])
            at += size

    def step(self, **kw):
        self.muon.step(self.grads, self.master, self.momentum, self.param, **kw)

    def ref_step(self):
        g = self.grads[0][:self.n].float()
        for more in self.grads[1:]:
            g = g + more[:self.n].float()
        g = g / torch.full((), float(self.W), device=DEV)
        old = self.ref_momentum
        if self.fmt == "int8":
            old = read_back(*quantize(old, self.shapes), self.shapes)
        new = old * self.hp["momentum"] + g
        u = g + new * self.hp["momentum"] if self.hp["nesterov"] else new
        self.ref_momentum = new
        lr = self.hp["lr"]
        for um, pm in zip(self.matrices(u), self.matrices(self.ref_master)):
            m, n = um.shape[-2:]
            s = 0.2 * math.sqrt(max(m, n)) if self.hp["scale"] == "rms" else math.sqrt(max(1, m / n))
            o = reference(um, self.hp["ns_steps"])
            pm.mul_(1 - lr * self.hp["weight_decay"]).sub_(lr * s * o)
            self.slack = self.slack + (lr * s * o).norm() * self.hp["ns_steps"] * F16_HALF

    def check(self, steps=1):
        n = self.n
        got = self.master[:n].double()
        err = (got - self.ref_master[:n]).norm()
        # decay, step_size and the element's three operations: six half steps a step
        assert err <= self.slack + steps * 6 * F32_HALF * self.ref_master[:n].norm(), (err, self.slack)
        if self.fmt == "f32":
            assert torch.equal(self.momentum[:n], self.ref_momentum)
        else:
            codes, scales = quantize(self.ref_momentum, self.shapes)
            assert torch.equal(self.momentum[0][:n], codes)
            assert torch.equal(self.momentum[1][:self.muon.n_scales], scales)
        assert not self.muon.check_result()

    def check_param(self):
        if self.plan.param_layout == zr.ZR_PARAMS_OWNED:
            assert torch.equal(self.param[:self.n], self.master[:self.n].to(torch.bfloat16))
            return
        want = torch.full_like(self.param, 3.0)
        for owned, glob, length in self.plan.runs():
            want[glob:glob + length] = self.master[owned:owned + length].to(torch.bfloat16)
        assert torch.equal(self.param, want)


def block_sizes(shapes):
    for s in shapes:
        for _ in range(math.prod(s[:-2])):
            yield s[-2] * s[-1]


def quantize(flat, shapes):
    codes, scales, at = [], [], 0
    for size in block_sizes(shapes):
        for b in range(0, size, 256):
            x = flat[at + b:at + min(b + 256, size)]
            s = x.abs().max() / torch.full((), 127.0, device=DEV)
            q = torch.round(x / s).clamp(-127, 127) if bool(s > 0) and bool(torch.isfinite(s)) else torch.zeros_like(x)
            codes.append(q.to(torch.int8))
            scales.append(s)
        at += size
    return torch.cat(codes), torch.stack(scales)


def read_back(codes, scales, shapes):
    out, at, k = [], 0, 0
    for size in block_sizes(shapes):
        for b in range(0, size, 256):
            out.append(codes[at + b:at + min(b + 256, size)].float() * scales[k])
            k += 1
        at += size
    return torch.cat(out)


@pytest.mark.parametrize("fmt", ["f32", "int8"])
@pytest.mark.parametrize("name,W", [("aligned", 1), ("aligned", 2), ("odd", 1), ("odd", 3), ("odd", 7), ("aligned", 12),
                                    ("odd", 33), ("aligned", 65)])
def test_step(name, W, fmt):
    shapes = SETS[name]
    for rank in range(min(W, 3)):
        job = Job(shapes, W, rank, fmt, seed=W + rank)
        for step in range(3):
            job.new_grads()
            job.step()
            job.ref_step()
            job.check(step + 1)
        job.check_param()
        job.muon.close()


@pytest.mark.parametrize("kw", [dict(nesterov=False), dict(scale="spectral"), dict(momentum=0.0), dict(weight_decay=0.0),
                                dict(ns_steps=3), dict(lr=0.0)])
def test_parameters(kw):
    job = Job(SETS["odd"], 2, 0, seed=4, **kw)
    for _ in range(2):
        job.new_grads()
        job.step()
        job.ref_step()
    job.check(2)


def test_tiny_set_and_new_learning_rate():
    job = Job(SETS["tiny"], 2, 0, seed=8)
    job.new_grads()
    job.step()
    job.ref_step()
    job.muon.set_lr(0.002)
    job.hp["lr"] = 0.002
    job.new_grads()
    job.step()
    job.ref_step()
    job.check(2)


@pytest.mark.parametrize("fmt", ["f32", "int8"])
def test_global_layout_writes_only_the_ranks_positions(fmt):
    for rank in range(2):
        job = Job(SETS["odd"], 2, rank, fmt, seed=rank, layout=zr.ZR_PARAMS_GLOBAL)
        job.new_grads()
        job.step()
        job.ref_step()
        job.check()
        job.check_param()


def test_flat_partition_of_one_rank():
    job = Job(SETS["odd"], 1, 0, mode=zr.ZR_PARTITION_FLAT, layout=zr.ZR_PARAMS_GLOBAL)
    job.new_grads()
    job.step()
    job.ref_step()
    job.check()
    job.check_param()


def test_gather_targets():
    job = Job(SETS["odd"], 2, 1, seed=5, layout=zr.ZR_PARAMS_GLOBAL)
    targets = [torch.full_like(job.param, 3.0) for _ in range(2)]
    zr.zr_plan_set_gather_targets(job.plan.handle, targets)
    job.new_grads()
    job.muon.step(job.grads, job.master, job.momentum, None)
    job.ref_step()
    job.check()
    for t in targets:
        job.param = t
        job.check_param()


def test_more_shapes_than_one_launch_holds():
    shapes = [(8 + i, 40 + 3 * i) for i in range(37)]
    job = Job(shapes, 1, 0, seed=9)
    job.new_grads()
    job.step()
    job.ref_step()
    job.check()
    job.check_param()


def test_a_rank_that_owns_nothing():
    plan = ZrPlan([(8, 8)], 2, 1, zr.ZR_PARTITION_WHOLE_TENSOR, device=DEV)
    muon = ZrMuon(plan)
    muon.step([None, None], None, None, None)
    assert muon.n_scales == 0


def test_non_finite_gradients_stay_in_their_matrix():
    a, b = Job(SETS["aligned"], 1, 0, seed=6), Job(SETS["aligned"], 1, 0, seed=6)
    a.new_grads()
    b.new_grads()
    first = math.prod(SETS["aligned"][0])
    a.grads[0][5] = float("nan")
    a.step()
    b.step()
    assert torch.isnan(a.master[:first]).all()
    assert torch.equal(a.master[first:], b.master[first:])


@pytest.mark.parametrize("fmt", ["f32", "int8"])
def test_graph_replays_as_the_next_step(fmt):
    a, b = Job(SETS["odd"], 2, 0, fmt, seed=2), Job(SETS["odd"], 2, 0, fmt, seed=2)
    a.new_grads()
    b.new_grads()
    a.step()
    b.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    for _ in range(3):
        a.gen.manual_seed(11)
        b.gen.manual_seed(11)
        fresh = [b.rand(1e-3).to(torch.bfloat16) for _ in range(2)]
        for g, h, f in zip(a.grads, b.grads, fresh):
            g.copy_(f)
            h.copy_(f)
        graph.replay()
        b.step()
        assert torch.equal(a.master, b.master) and torch.equal(a.param, b.param)
        for x, y in zip(a.momentum if fmt == "int8" else [a.momentum], b.momentum if fmt == "int8" else [b.momentum]):
            assert torch.equal(x, y)


def test_side_stream():
    a, b = Job(SETS["odd"], 3, 1, seed=2), Job(SETS["odd"], 3, 1, seed=2)
    a.new_grads()
    b.new_grads()
    a.step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.step(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a.master, b.master) and torch.equal(a.param, b.param)


@pytest.mark.parametrize("name", ["aligned", "odd"])
def test_conversions(name):
    job = Job(SETS[name], 1, 0, "int8")
    m = job.rand(1e-2)
    m[3] = 40.0                                  # one strong value: the rest of its block loses its codes
    m[256 * 2:256 * 3] = 0.0                     # an empty block
    m[256 * 4:256 * 5] *= 1e-42                  # a subnormal scale
    codes = torch.full((job.n + 5,), 99, dtype=torch.int8, device=DEV)
    scales = torch.full((job.muon.n_scales + 4,), 99.0, device=DEV)
    job.muon.quantize_momentum(m, codes, scales)
    want_codes, want_scales = quantize(m[:job.n], job.shapes)
    assert torch.equal(codes[:job.n], want_codes) and torch.equal(scales[:job.muon.n_scales], want_scales)
    assert torch.all(codes[job.n:] == 99) and torch.all(scales[job.muon.n_scales:] == 99.0)
    back = torch.full((job.n + 8,), 99.0, device=DEV)
    job.muon.dequantize_momentum(codes, scales, back)
    assert torch.equal(back[:job.n], read_back(want_codes, want_scales, job.shapes))
    assert torch.all(back[job.n:] == 99.0)


def test_a_block_with_a_non_finite_value_reads_back_as_nan():
    job = Job([(4, 256)], 1, 0, "int8")
    m = job.rand(1.0)
    m[10] = float("inf")
    m[300] = float("nan")
    codes, scales = job.muon.empty_momentum()
    job.muon.quantize_momentum(m, codes, scales)
    back = torch.zeros_like(m)
    job.muon.dequantize_momentum(codes, scales, back)
    assert torch.isnan(back[:512]).all() and torch.isfinite(back[512:]).all()


def test_refusals():
    job = Job(SETS["aligned"], 2, 0, "int8")
    job.new_grads()
    codes, scales = job.momentum
    for grads, master, momentum, param in (
            (job.grads[:1], job.master, job.momentum, job.param),
            (job.grads, job.master.double(), job.momentum, job.param),
            (job.grads, job.master, (codes.float(), scales), job.param),
            (job.grads, job.master, (codes, scales[:1]), job.param),
            (job.grads, job.master, job.momentum, job.param[:4])):
        with pytest.raises(ValueError):
            job.muon.step(grads, master, momentum, param)
    for args, status in (((job.grads, job.master, codes, None, job.param), zr.ZR_ERR_INVALID_ARG),
                         ((job.grads, job.master, codes, scales, None), zr.ZR_ERR_INVALID_ARG),
                         ((job.grads, job.master.data_ptr() + 4, codes, scales, job.param), zr.ZR_ERR_ALIGNMENT),
                         ((job.grads, job.master, codes.data_ptr() + 1, scales, job.param), zr.ZR_ERR_ALIGNMENT)):
        with pytest.raises(zr.ZrError) as e:
            zr.zr_muon_step(job.muon.handle, *args)
        assert e.value.status == status

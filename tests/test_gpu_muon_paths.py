"""Both kernels behind orthogonalisation and the Muon step, at the sizes where
one takes over from the other and where tiles, clusters and launches change:
matrices kept on the chip (smaller extent up to 128, larger one up to 4096, in
clusters of 1 to 16 CTAs), and the persistent kernel for all others.

Tolerances as in test_gpu_muon.py: half a bf16 step of the result, and half an
fp16 step of each iterate.
"""
import pytest
import torch

import sharded_optimizer_step_zr_b200 as zr
from sharded_optimizer_step_zr_b200.muon import ZrMuon, orthogonalize
from sharded_optimizer_step_zr_b200.plan import ZrPlan
from test_gpu_muon import DEV, Job, assert_orthogonal, quantize, randn, read_back

pytestmark = pytest.mark.gpu

EDGES = [(128, 128), (128, 129), (129, 128), (129, 129), (128, 256), (128, 257), (100, 320), (128, 512), (513, 128),
         (64, 1024), (1025, 77), (128, 2048), (2049, 128), (128, 4096), (4096, 128), (128, 4097), (4097, 128),
         (1, 4096), (4097, 1), (3, 260)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", EDGES)
def test_where_the_kernels_meet(shape, dtype):
    x = randn(*shape, seed=shape[0] + shape[1], dtype=dtype)
    assert_orthogonal(orthogonalize(x), x)


@pytest.mark.parametrize("shape", [(255, 256), (256, 257), (257, 700), (1500, 2100), (2100, 1500), (2305, 2305),
                                   (160, 9000), (9000, 160)])
def test_tiles_of_the_persistent_kernel(shape):
    x = randn(*shape, seed=shape[0])
    assert_orthogonal(orthogonalize(x), x)


@pytest.mark.parametrize("shape", [(300, 20, 700), (40, 128, 1100), (17, 100, 3000), (20, 200, 300), (90, 140, 130),
                                   (3, 1000, 1100)])
def test_batches_wider_than_the_device(shape):
    x = randn(*shape, seed=shape[0])
    assert_orthogonal(orthogonalize(x), x)


@pytest.mark.parametrize("steps", [1, 2, 7])
@pytest.mark.parametrize("shape", [(90, 600), (600, 90), (300, 400), (400, 300)])
def test_steps_of_both(shape, steps):
    x = randn(*shape, seed=steps)
    assert_orthogonal(orthogonalize(x, steps=steps), x, steps)


@pytest.mark.parametrize("shape", [(2, 200, 333), (2, 333, 200), (2, 100, 333), (2, 333, 100)])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_unaligned_output_leaves_its_surroundings(shape, offset):
    b, m, n = shape
    x = randn(*shape)
    whole = torch.full((b, m + 3, n + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    out = whole[:, 2:m + 2, offset:n + offset]
    orthogonalize(x, out=out)
    assert_orthogonal(out, x)
    rest = torch.ones_like(whole, dtype=torch.bool)
    rest[:, 2:m + 2, offset:n + offset] = False
    assert torch.all(whole[rest] == 7.0)


def test_in_place_and_transposed_views():
    for shape in ((2, 300, 200), (2, 90, 700)):
        x = randn(*shape, dtype=torch.bfloat16)
        want = orthogonalize(x)
        y = x.clone()
        assert orthogonalize(y, out=y) is y
        assert torch.equal(y, want)
        assert_orthogonal(orthogonalize(x.mT), x.mT)
        assert_orthogonal(orthogonalize(x[:, ::2, 3:-4]), x[:, ::2, 3:-4])


@pytest.mark.parametrize("shape", [(5, 200, 300), (5, 90, 700)])
def test_non_finite_matrices_touch_no_other(shape):
    x = randn(*shape)
    clean = orthogonalize(x)
    x[1] = 0.0
    x[2, 3, 5] = float("nan")
    x[4, 0, 0] = float("-inf")
    got = orthogonalize(x)
    for i in (0, 3):
        assert torch.equal(got[i], clean[i])
    assert torch.all(got[1] == 0)
    assert torch.isnan(got[2]).all()
    assert torch.isnan(got[4]).any()


def test_two_streams_at_once():
    """Two persistent kernels and a small one, each on its own stream: each
    needs every SM or a whole cluster at once, and all must end."""
    xs = [randn(700, 900, seed=1), randn(2, 600, 500, seed=2), randn(3, 128, 2000, seed=3)]
    want = [orthogonalize(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [[] for _ in xs]
    for _ in range(20):
        for x, s, o in zip(xs, streams, outs):
            o.append(orthogonalize(x, stream=s))
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, y) for y in o)


def test_two_captured_graphs_share_a_workspace_in_order():
    x, y = randn(300, 260, seed=1), randn(260, 300, seed=2)
    need = max(zr.zr_orthogonalize_workspace_bytes(1, 300, 260), zr.zr_orthogonalize_workspace_bytes(1, 260, 300))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    for t in (x, y):
        out = torch.empty(t.shape, dtype=torch.bfloat16, device=DEV)
        orthogonalize(t, out=out, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            orthogonalize(t, out=out, workspace=ws)
        graphs.append(g)
        outs.append(out)
    want = [orthogonalize(x), orthogonalize(y)]
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


# ---------------------------------------------------------------------------
# the Muon step
# ---------------------------------------------------------------------------

PATHS = {
    "small": [(100, 60), (60, 100), (3, 128, 128), (90, 600), (1, 2000), (640, 1)],
    "large": [(333, 517), (200, 140), (2, 150, 260), (513, 300)],
    "mixed": [(333, 517), (1001, 77), (5, 130, 66), (1, 2000), (640, 1)],
}


@pytest.mark.parametrize("fmt", ["f32", "int8"])
@pytest.mark.parametrize("name", list(PATHS))
def test_step_on_each_path(name, fmt):
    for W, rank in ((1, 0), (3, 1)):
        job = Job(PATHS[name], W, rank, fmt, seed=W, layout=zr.ZR_PARAMS_GLOBAL)
        for step in range(2):
            job.new_grads()
            job.step()
            job.ref_step()
            job.check(step + 1)
        job.check_param()


@pytest.mark.parametrize("least", [8, 129])
def test_more_shapes_than_a_launch_holds(least):
    job = Job([(least + i, least + 20 + 2 * i) for i in range(37)], 1, 0, seed=9)
    job.new_grads()
    job.step()
    job.ref_step()
    job.check()
    job.check_param()


@pytest.mark.parametrize("name", ["small", "large"])
def test_gather_targets_on_each_path(name):
    job = Job(PATHS[name], 3, 1, seed=5, layout=zr.ZR_PARAMS_GLOBAL)
    targets = [torch.full_like(job.param, 3.0) for _ in range(3)]          # one per rank
    zr.zr_plan_set_gather_targets(job.plan.handle, targets)
    job.new_grads()
    job.muon.step(job.grads, job.master, job.momentum, None)
    job.ref_step()
    job.check()
    for t in targets:
        job.param = t
        job.check_param()


def test_a_job_that_resumes_into_8_bits_and_saves_back():
    """An fp32 job's momentum taken into 8 bits, two steps from there, and the
    state read back: the operators as one run uses them, on both paths."""
    first = Job(PATHS["mixed"], 2, 0, "f32", seed=7)
    first.new_grads()
    first.step()
    first.ref_step()
    first.check()
    job = Job(PATHS["mixed"], 2, 0, "int8", seed=7)
    job.muon.quantize_momentum(first.momentum, *job.momentum)
    job.master.copy_(first.master)
    job.ref_master = job.master.double()
    job.ref_momentum = first.ref_momentum
    for step in range(2):
        job.new_grads()
        job.step()
        job.ref_step()
        job.check(step + 1)
    job.check_param()
    back = torch.zeros(max(job.n, 8), device=DEV)
    job.muon.dequantize_momentum(*job.momentum, back)
    assert torch.equal(back[:job.n], read_back(*quantize(job.ref_momentum, job.shapes), job.shapes))


def test_two_optimizers_on_two_streams():
    """Two jobs' steps at once (their own plans and workspaces) end as they do alone."""
    alone = [Job(PATHS["large"], 2, 0, seed=3), Job(PATHS["mixed"], 2, 1, seed=4)]
    both = [Job(PATHS["large"], 2, 0, seed=3), Job(PATHS["mixed"], 2, 1, seed=4)]
    for j in alone + both:
        j.new_grads()
    for j in alone:
        for _ in range(5):
            j.step()
    streams = [torch.cuda.Stream() for _ in both]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for j, s in zip(both, streams):
            j.step(stream=s)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert torch.equal(a.master, b.master) and torch.equal(a.param, b.param) and torch.equal(a.momentum, b.momentum)
        assert not b.muon.check_result()


# ---------------------------------------------------------------------------
# offsets past 32 bits
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("shape", [(36000, 60000), (60000, 36000)])
def test_more_than_2_to_31_elements(shape):
    """Zero but for blocks on the diagonal, one in the last corner: the
    polynomial acts on each block alone, with the whole matrix's norm."""
    m, n = shape
    x = torch.zeros(m, n, dtype=torch.bfloat16, device=DEV)
    blocks = [(0, 0, 40, 60), (17001, 20003, 130, 70), (m - 90, n - 50, 90, 50)]
    for i, (r, c, h, w) in enumerate(blocks):
        x[r:r + h, c:c + w] = randn(h, w, seed=i, dtype=torch.bfloat16)
    norm = sum(x[r:r + h, c:c + w].double().square().sum() for r, c, h, w in blocks).sqrt()
    steps = 2
    out = orthogonalize(x, steps=steps)
    a, b, c2 = 3.4445, -4.7750, 2.0315
    for r, c, h, w in blocks:
        want = x[r:r + h, c:c + w].double() / (norm + 1e-7)
        for _ in range(steps):
            g = want @ want.mT
            want = a * want + (b * g + c2 * (g @ g)) @ want
        got = out[r:r + h, c:c + w].double()
        assert (got - want).norm() <= (2.0 ** -8 + steps * 2.0 ** -11) * want.norm()
        out[r:r + h, c:c + w] = 0
    assert not out.any()


def test_master_weights_past_2_to_31_elements():
    """A plan of more than 2^31 owned elements: the last matrix's step, its
    8-bit codes and its scales, against the same matrix in a plan of its own."""
    big, tail = (2 ** 17, 16640), (300, 200)
    whole = ZrPlan([big, tail], 1, 0, zr.ZR_PARTITION_WHOLE_TENSOR, device=DEV)
    alone = ZrPlan([tail], 1, 0, zr.ZR_PARTITION_WHOLE_TENSOR, device=DEV)
    size, at = tail[0] * tail[1], big[0] * big[1]
    assert at > 2 ** 31
    got = []
    for plan, offset in ((whole, at), (alone, 0)):
        muon = ZrMuon(plan, lr=0.01, momentum_format="int8", ns_steps=1)
        n = plan.owned_numel
        grad = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
        master = torch.zeros(n, device=DEV)
        grad[offset:offset + size] = randn(size, seed=1, dtype=torch.bfloat16)
        master[offset:offset + size] = randn(size, seed=2)
        codes, scales = muon.empty_momentum()
        param = torch.zeros(plan.param_out_numel, dtype=torch.bfloat16, device=DEV)
        muon.step([grad], master, (codes, scales), param)
        assert not muon.check_result()
        blocks = muon.n_scales - (size + 255) // 256
        got.append((master[offset:offset + size].clone(), codes[offset:offset + size].clone(),
                    scales[blocks:muon.n_scales].clone(), param[offset:offset + size].clone()))
        if offset:
            assert not master[:offset].any() and not codes[:offset].any() and not param[:offset].any()
        muon.close()
        del muon, grad, master, codes, scales, param
    assert all(torch.equal(x, y) for x, y in zip(*got))

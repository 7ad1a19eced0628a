"""What orders the matrix optimizer's work: tensor maps that replace others in
the same memory, counters and flags between the roles of a kernel, streams and
the lifetime of workspaces.  Each test's outputs have to be the same bits
however the calls are arranged.
"""
import pytest
import torch

import sharded_optimizer_step_zr_b200 as zr
from sharded_optimizer_step_zr_b200.muon import ZrMuon, orthogonalize
from test_gpu_muon import DEV, Job, randn

pytestmark = pytest.mark.gpu

ONE = [(200, 140), (2, 150, 260), (333, 517)]              # several shapes: their tensor maps are in the workspace
OTHER = [(260, 330), (513, 300), (140, 150), (2, 180, 200)]


def bind(job, workspace):
    """The job's step on `workspace` (of any plan's size) from here on."""
    zr.zr_muon_set_workspace(job.muon.handle, workspace, workspace.numel())


def test_plans_take_turns_in_one_workspace():
    """Every binding writes other tensor maps to the same addresses."""
    alone = [Job(ONE, 1, 0, seed=1), Job(OTHER, 1, 0, seed=2)]
    turns = [Job(ONE, 1, 0, seed=1), Job(OTHER, 1, 0, seed=2)]
    shared = torch.empty(max(j.muon.workspace_bytes for j in turns), dtype=torch.uint8, device=DEV)
    for j in alone + turns:
        j.new_grads()
    for _ in range(20):
        for a, t in zip(alone, turns):
            bind(t, shared)
            t.step()
            a.step()
    for a, t in zip(alone, turns):
        assert torch.equal(a.master, t.master) and torch.equal(a.momentum, t.momentum) and torch.equal(a.param, t.param)
        assert not a.muon.check_result()
    assert not turns[-1].muon.check_result()
    assert torch.isfinite(alone[0].master).all()


@pytest.mark.parametrize("shapes", [ONE, [(777, 1025)] * 3, [(512, 512), (512, 1024), (1024, 512)]])
def test_a_step_repeats_itself_to_the_bit(shapes):
    """Diagonals and tiles cross from block to block many times a step; one
    that is read before it is written shows as other bits."""
    job = Job(shapes, 1, 0, seed=3)
    job.new_grads()
    start = job.master.clone()
    job.step()
    want = job.master.clone()
    for _ in range(100):
        job.momentum.zero_()
        job.master.copy_(start)
        job.step()
        assert torch.equal(job.master, want)
    assert not job.muon.check_result()


@pytest.mark.parametrize("shape", [(6, 777, 1025), (300, 257), (128, 128), (100, 3000), (3, 1100, 900)])
def test_a_call_repeats_itself_to_the_bit(shape):
    x = randn(*shape, seed=5)
    want = orthogonalize(x)
    for _ in range(50):
        assert torch.equal(orthogonalize(x), want)


def test_a_binding_is_not_captured():
    """A replay would read the host's tables when they are gone.  The refused
    call leaves the graph and the binding that was there as they are."""
    a, b = Job(ONE, 1, 0, seed=4), Job(ONE, 1, 0, seed=4)
    for j in (a, b):
        j.new_grads()
        j.step()
    other = torch.empty(a.muon.workspace_bytes, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(zr.ZrError) as e:
            bind(a, other)
        assert e.value.status == zr.ZR_ERR_UNSUPPORTED
        a.step()
    for _ in range(2):
        graph.replay()
        b.step()
    assert torch.equal(a.master, b.master) and torch.equal(a.momentum, b.momentum)


# ---------------------------------------------------------------------------
# streams and the lifetime of memory
# ---------------------------------------------------------------------------

BUSY = 200_000_000           # cycles: some 0.1 s in which the calls of a test are queued


def place(t):
    return t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()


def assert_not_handed_out(first, end):
    """Memory of [first, end) that a running call uses is not what the current
    stream's next allocations get (they are not written: the call goes on)."""
    got = [torch.empty(end - first, dtype=torch.uint8, device=DEV) for _ in range(3)]
    assert all(a >= end or b <= first for a, b in map(place, got))


def handles(side):
    return [side, side.cuda_stream]        # a stream is given as an object or as its handle


@pytest.mark.parametrize("shape", [(100, 300), (300, 400)])
def test_a_given_stream_takes_no_memory_that_the_current_one_still_reads(shape):
    x = randn(*shape)
    want = orthogonalize(x)
    sizes = (2 * x.numel(), zr.zr_orthogonalize_workspace_bytes(1, *shape))
    side = torch.cuda.Stream()
    for stream in handles(side):
        temporaries = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in sizes]
        copies = [torch.zeros_like(t) for t in temporaries]
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        for c, t in zip(copies, temporaries):
            c.copy_(t)
        del temporaries, t
        out = orthogonalize(x, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.all(c == 7) for c in copies)
        assert torch.equal(out, want)


@pytest.mark.parametrize("shape", [(100, 300), (300, 400)])
def test_tensors_may_be_dropped_while_the_given_stream_works(shape):
    x = randn(*shape)
    want = orthogonalize(x)
    n = zr.zr_orthogonalize_workspace_bytes(1, *shape)
    side = torch.cuda.Stream()
    for stream in handles(side):
        y, ws = x.clone(), torch.empty(n, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(BUSY)
        out = orthogonalize(y, workspace=ws, stream=stream)
        orthogonalize(y, stream=stream)                    # a result that nobody keeps
        del y, ws
        fresh = [torch.full_like(x, 5.0), torch.full((n,), 5, dtype=torch.uint8, device=DEV), torch.full_like(want, 5.0)]
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all(torch.all(f == 5) for f in fresh)


def test_the_null_stream_by_its_handle():
    x = randn(300, 400)
    want = orthogonalize(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = [orthogonalize(x, stream=0), orthogonalize(x, stream=torch.cuda.default_stream())]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("shapes", [ONE, [(100, 60), (90, 600)]])
def test_an_optimizer_may_be_dropped_while_its_step_runs(shapes):
    alone = Job(shapes, 1, 0, seed=6)
    alone.new_grads()
    alone.step()
    side = torch.cuda.Stream()
    for given in handles(side) + [None]:                   # None: the side stream is the current one
        job = Job(shapes, 1, 0, seed=6)
        job.new_grads()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(BUSY)
            if given is None:
                job.step()
        if given is not None:
            job.step(stream=given)
        used = place(job.muon.workspace)
        del job.muon
        assert_not_handed_out(*used)
        torch.cuda.synchronize()
        assert torch.equal(job.master, alone.master) and torch.equal(job.momentum, alone.momentum)


def test_an_optimizer_and_its_plan_may_be_dropped_while_the_step_writes_gather_targets():
    """The targets' addresses are read from the plan's workspace."""
    alone, job = (Job(ONE, 2, 0, seed=9, layout=zr.ZR_PARAMS_GLOBAL) for _ in range(2))
    targets = [[torch.zeros_like(j.param) for _ in range(2)] for j in (alone, job)]
    for j, t in zip((alone, job), targets):
        zr.zr_plan_set_gather_targets(j.plan.handle, t)
        j.new_grads()
    alone.muon.step(alone.grads, alone.master, alone.momentum, None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    job.muon.step(job.grads, job.master, job.momentum, None, stream=side)
    used = [place(job.muon.workspace), place(job.plan.workspace)]
    del job.muon, job.plan
    for u in used:
        assert_not_handed_out(*u)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*targets))


def test_conversions_may_outlive_their_handle():
    job = Job(ONE, 1, 0, "int8", seed=7)
    m = job.rand(1e-2)
    want = job.muon.empty_momentum()
    job.muon.quantize_momentum(m, *want)
    side = torch.cuda.Stream()
    codes, scales = job.muon.empty_momentum()
    back, want_back = torch.zeros_like(m), torch.zeros_like(m)
    job.muon.dequantize_momentum(*want, want_back)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    job.muon.quantize_momentum(m, codes, scales, stream=side)
    job.muon.dequantize_momentum(codes, scales, back, stream=side)
    used = place(job.muon.workspace)
    del job.muon
    assert_not_handed_out(*used)
    torch.cuda.synchronize()
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1]) and torch.equal(back, want_back)


def test_an_optimizer_made_on_a_given_stream_takes_no_memory_in_use():
    plan = Job(ONE, 1, 0, seed=8).plan
    n = ZrMuon(plan).workspace_bytes
    side = torch.cuda.Stream()
    for stream in handles(side):
        torch.cuda.synchronize()
        temporary = torch.full((n,), 7, dtype=torch.uint8, device=DEV)
        copy = torch.zeros_like(temporary)
        torch.cuda._sleep(BUSY)
        copy.copy_(temporary)
        del temporary
        muon = ZrMuon(plan, stream=stream)
        torch.cuda.synchronize()
        assert torch.all(copy == 7)
        assert not muon.check_result()

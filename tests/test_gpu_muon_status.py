"""A wait that ran out inside a call shows in the caller's status tensor."""
import pytest
import torch

import sharded_optimizer_step_zr_b200 as zr
from sharded_optimizer_step_zr_b200 import muon
from sharded_optimizer_step_zr_b200.muon import orthogonalize
from test_gpu_muon import DEV, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(100, 60), (300, 260), (0, 5)])
def test_status_of_a_sound_call_is_zero(shape):
    x = randn(*shape)
    side = torch.cuda.Stream()
    workspace = torch.full((zr.zr_orthogonalize_workspace_bytes(1, *shape),), 255, dtype=torch.uint8, device=DEV)
    for stream in (None, side, side.cuda_stream):
        for ws in (None, workspace):
            status = torch.full((2,), 7, dtype=torch.int32, device=DEV)
            torch.cuda.synchronize()
            orthogonalize(x, workspace=ws, stream=stream, status=status)
            torch.cuda.synchronize()
            assert status.tolist() == [0, 7]


def test_status_follows_the_workspaces_word(monkeypatch):
    """The library's call replaced by one that leaves the word as a wait that ran out does."""
    def gives_up(*args):
        args[13][:4].view(torch.int32).fill_(1)

    monkeypatch.setattr(muon, "zr_orthogonalize", gives_up)
    status = torch.full((1,), 7, dtype=torch.int32, device=DEV)
    orthogonalize(randn(30, 40), status=status)
    assert status.item() == 1
    graph_status = torch.zeros(1, dtype=torch.int32, device=DEV)
    x = randn(30, 40)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        orthogonalize(x, status=graph_status)
    graph_status.zero_()
    graph.replay()
    assert graph_status.item() == 1

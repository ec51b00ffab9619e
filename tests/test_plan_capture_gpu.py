"""A plan is not made while its stream is captured: a replay would read a host buffer that is gone."""
import pytest
import torch

from shared_prefix_grouped_gb300 import _lib, api, rollout
from shared_prefix_grouped_gb300.build import build

pytestmark = pytest.mark.gpu


def test_plan_is_refused_while_capturing():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    x = torch.zeros(8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(_lib.PgError, match="captured"):
            api.plan_decode([40], [2], 4, 2, 128, 16, 1)
        with pytest.raises(_lib.PgError, match="captured"):
            rollout.Rollout([40], [2], 4, 2, 128, 16)
        x += 1
    graph.replay()                       # the capture went on
    torch.cuda.synchronize()
    assert bool((x == 1).all())
    assert api.plan_decode([40], [2], 4, 2, 128, 16, 1).num_seqs == 2

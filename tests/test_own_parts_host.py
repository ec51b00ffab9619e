"""The plan's workspaces: the step over the plan's own type does not pay for what the step over 8 bits takes."""
import pytest
import torch

from shared_prefix_grouped_gb300 import api


def rows(st):
    return st.num_seqs * st.heads_q * (st.head_dim + 1) * 4


@pytest.mark.parametrize("responses", [1, 40, 256, 1024])
@pytest.mark.parametrize("keys", [64, 1024, 4096, 16384, 1 << 20])
@pytest.mark.parametrize("prefix", [0, 5000])
def test_workspaces(responses, keys, prefix):
    st, _ = api.plan_decode_host([prefix], [responses], 32, 8, 128, 64, keys // 64)
    assert st.own_slots <= st.own_slots_e4m3 <= max(st.own_slots, 4)
    for nbytes, own in ((st.workspace_bytes, st.own_slots), (st.workspace_bytes_e4m3, st.own_slots_e4m3)):
        need = max(st.simt_splits, st.prefix_slots + own) * rows(st)
        assert need <= nbytes < need + 512
    # enough responses to fill the GPU: one part each, whatever the room
    if responses >= 256:
        assert st.own_slots == 1


def test_of_a_plan_in_fp32():
    st, _ = api.plan_decode_host([5000], [4], 32, 8, 128, 64, 256, torch.float32)
    assert st.workspace_bytes == st.workspace_bytes_e4m3 and st.own_slots == st.own_slots_e4m3 == 0

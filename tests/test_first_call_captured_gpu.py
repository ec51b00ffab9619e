"""The first call that a process makes of an operator may be a captured one: what a launch asks of the device (attributes,
how many clusters run at once) is asked there."""
import os
import subprocess
import sys

import pytest
import torch

from shared_prefix_grouped_gb300.build import build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

POLICY = """
R, V, dt = {shape}
x = torch.randn((R, V), device="cuda").to(dt)
d = torch.empty_like(x)
tok = torch.randint(0, V, (R,), dtype=torch.int32, device="cuda")
adv = torch.randn(R, device="cuda")

def call():
    r = api.policy_loss(x, tok, advantages=adv, dlogits=d)
    return r.loss, r.logprobs, r.dlogits, *api.token_logprobs(x, tok)
"""
CACHE = """
k = torch.randn((600, 2, 128), device="cuda").to(torch.bfloat16)
q = torch.randn((2, 8, 128), device="cuda").to(torch.bfloat16)
ints = lambda *a: torch.arange(*a, dtype=torch.int32, device="cuda")
pp, op, pos, rows, first = ints(10).view(1, 10), ints(10, 12).view(2, 1), ints(600), 0 * ints(600), 0 * ints(2)
kv = [api.scaled_cache(12, 64, 2, 128) for _ in range(2)]
plan = api.plan_decode([600], [2], 8, 2, 128, 64, 1)
ws = api.decode_workspace(plan)

def call():
    api.cache_append_e4m3(k, k, *kv, pp, pos, page_rows=rows, rope_theta=1e4)
    api.cache_append_e4m3(k[:2], k[:2], *kv, op, first)
    return (*api.cache_read_e4m3(*kv, pp, pos, page_rows=rows),
            *api.decode_attn_e4m3(plan, q, *kv, pp, op, first + 1, workspace=ws))
"""
PROGRAM = """
import torch
from shared_prefix_grouped_gb300 import api
torch.manual_seed(0)
{setup}
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = call()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in out]
want = call()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and api.device_status() == 0
"""
SETUPS = {"policy_clusters": POLICY.format(shape="64, 70001, torch.float32"),
          "policy_streamed": POLICY.format(shape="160, 32000, torch.bfloat16"),
          "policy_registers": POLICY.format(shape="6, 60001, torch.bfloat16"), "cache_and_step": CACHE}


@pytest.mark.parametrize("name", SETUPS)
def test_first_call_captured(name):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    out = subprocess.run([sys.executable, "-c", PROGRAM.format(setup=SETUPS[name])], cwd=ROOT, capture_output=True,
                         text=True)
    assert out.returncode == 0, out.stderr[-2000:]

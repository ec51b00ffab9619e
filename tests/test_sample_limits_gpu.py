"""Sampling at the limits of its definition, against the sorted-list oracle: filters that leave the first
token of the order only, the border between a list of candidates and a long nucleus, and slices larger
than shared memory.  Tokens equal, log-probabilities as in test_sample_gpu.py: half a step of fp32 (2^-24
relative) plus 4e-9 (the sum's weights carry about 2^-30 each)."""
import math

import pytest
import torch

from oracle import rollout_oracle as ro
from shared_prefix_grouped_gb300 import api
from shared_prefix_grouped_gb300.build import build

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()


def compare(logits, u, **kw):
    tok, lp = api.sample(logits.cuda(), u.cuda(), **{n: t.cuda() for n, t in kw.items()})
    wt, wl = ro.sample(logits, u, **kw)
    assert torch.equal(tok.cpu(), wt), (tok.tolist(), wt.tolist())
    assert bool(((lp.cpu().double() - wl).abs() <= 2.0 ** -24 * wl.abs() + 4e-9).all())
    return tok.cpu()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [900, 40000])
@pytest.mark.parametrize("name,value", [("min_p", 1.5), ("min_p", INF), ("min_p", NAN), ("top_p", NAN)])
def test_filters_that_leave_the_first_token(name, value, V, dtype):
    # ties at the maximum, also of +inf, and of a whole row: the lowest index, whatever u is
    g = torch.Generator().manual_seed(V)
    x = torch.randn((6, V), generator=g)
    x[0, [40, V - 200]] = 9.0
    x[1, [5, 6, V - 100]] = INF
    x[2] = 0.0
    x[3, 100:] = 8.0
    x[4, [3, V - 1]] = 20.0
    x, u = x.to(dtype), torch.tensor([0.9, 0.9, 0.7, 0.8, 0.999, 0.5])
    row = lambda v, t=torch.float32: torch.full((6,), v, dtype=t)
    for kw in ({}, dict(temperature=row(0.7)), dict(top_k=row(5, torch.int32)),
               dict(top_k=row(600, torch.int32), min_p=row(0.01)), dict(top_p=row(0.9))):
        tok = compare(x, u, **{**kw, name: row(value)})
        assert tok[:5].tolist() == [40, 5, 0, 100, 3]
    # min_p of 1 itself keeps every token tied at the maximum
    tok = compare(x, u, min_p=row(1.0))
    assert tok[[0, 1, 4]].tolist() == [V - 200, V - 100, V - 1]

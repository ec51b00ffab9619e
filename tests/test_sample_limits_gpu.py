"""Sampling at the limits of its definition, against the sorted-list oracle: filters that leave the first
token of the order only, the border between a list of candidates and a long nucleus, and slices larger
than shared memory.  Tokens equal, log-probabilities as in test_sample_gpu.py: half a step of fp32 (2^-24
relative) plus 4e-9 (the sum's weights carry about 2^-30 each)."""
import math
import os
import re

import pytest
import torch

from oracle import rollout_oracle as ro
from shared_prefix_grouped_gb300 import api
from shared_prefix_grouped_gb300.build import build

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan
SOURCE = os.path.join(os.path.dirname(__file__), "..", "shared_prefix_grouped_gb300", "csrc", "pg_sample.cu")
LIST = int(re.search(r"constexpr int kList = (\d+);", open(SOURCE).read()).group(1))
KEPT = int(re.search(r"const int cap = std::min\(slice, (\d+)\);", open(SOURCE).read()).group(1))


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
@pytest.mark.parametrize("V", [900, 17000])
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [700, 17000])
def test_infinite_and_large_temperatures_with_masks(V, dtype):
    # Masks of the type's lowest value are finite: at T = inf they weigh 1 like every other logit, -inf 0.
    g = torch.Generator().manual_seed(V)
    low = torch.finfo(dtype).min
    x = torch.randn((5, V), generator=g).to(dtype)
    x[0, ::2] = low
    x[1, 5:] = -INF
    x[2] = low
    x[2, 3] = 1.0
    x[3, 1::2] = low / 2
    x[4, ::3] = INF
    u = torch.tensor([0.9, 0.5, 0.3, 0.77, 0.6])
    row = lambda v, t=torch.float32: torch.full((5,), v, dtype=t)
    for T in (INF, 1e38, 1e30):
        for kw in ({}, dict(top_p=row(0.8)), dict(top_k=row(300, torch.int32)),
                   dict(top_k=row(300, torch.int32), top_p=row(0.8), min_p=row(0.5))):
            compare(x, u, temperature=row(T), **kw)


@pytest.mark.parametrize("V", [3000, 17000], ids=["one_cta", "cluster"])
@pytest.mark.parametrize("n", [LIST - 1, LIST, LIST + 1, LIST + 44])
def test_candidates_around_the_length_of_the_list(n, V):
    # n logits above the rest: equal ones, different ones, and both kinds spread over all slices
    g = torch.Generator().manual_seed(n + V)
    x = torch.randn((4, V), generator=g)
    x[0, torch.randperm(V, generator=g)[:n]] = 30.0
    x[1, torch.randperm(V, generator=g)[:n]] = 30.0 + torch.rand(n, generator=g)
    x[2, torch.arange(n) * (V // n)] = 30.0 + torch.arange(n) % 7 / 4
    x[3, torch.randperm(V, generator=g)[:n]] = 30.0 + 3 * torch.rand(n, generator=g)
    u = torch.tensor([0.37, 0.81, 0.05, 0.999])
    row = lambda v, t=torch.float32: torch.full((4,), v, dtype=t)
    for k in (n - 1, n, n + 1):
        compare(x, u, top_k=row(k, torch.int32))
        compare(x, u, top_k=row(k, torch.int32), top_p=row(0.93), min_p=row(0.4))
    for p in (0.4, 0.999999):
        compare(x, u, top_p=row(p))
    compare(x.to(torch.bfloat16), u, top_k=row(n, torch.int32), top_p=row(0.9))
    compare(x.to(torch.bfloat16), u, top_p=row(0.97), temperature=row(1.3))


def definition(x, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """Tokens and log-probabilities in fp64 on the GPU (the list oracle would take minutes)."""
    S, V = x.shape
    col = lambda t, v: torch.full((S, 1), v, dtype=torch.float64, device=x.device) if t is None \
        else t.double()[:, None]
    X, T, p = x.double(), col(temperature, 1.0), col(top_p, 1.0)
    k = torch.zeros((S, 1), device=x.device, dtype=torch.long) if top_k is None else top_k.long()[:, None]
    greedy = T == 0
    w = torch.exp((X - X.amax(-1, keepdim=True)) / torch.where(greedy, torch.ones_like(T), T))
    order = torch.sort(X, dim=-1, descending=True, stable=True).indices
    ws, rank = w.gather(1, order), torch.arange(V, device=x.device)[None]
    keep = (rank < k) | (k <= 0)
    wk = ws * keep
    keep &= (torch.cumsum(wk, -1) - wk < p * wk.sum(-1, keepdim=True)) | (p >= 1)
    keep &= ws >= col(min_p, 0.0)
    keep = torch.where(greedy, rank == 0, keep | (rank == 0))
    kept = torch.zeros_like(w).scatter_(1, order, ws * keep)
    target = u.double()[:, None] * kept.sum(-1, keepdim=True)
    tok = (torch.cumsum(kept, -1) <= target).sum(-1)
    return tok, torch.log(w.gather(1, tok[:, None]) / w.sum(-1, keepdim=True))[:, 0], keep.sum(-1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_slices_larger_than_shared_memory(dtype):
    # Rows whose eight slices do not fit: every path of the sampler reads their ends from memory.
    S, V = 5, 8 * KEPT + 206785
    slice_ = (V + 7) // 8
    g = torch.Generator(device="cuda").manual_seed(17)
    x = torch.randn((S, V), generator=g, device="cuda") * 2
    x[1] *= 0.05                                            # flat: nuclei and top-k of many thousands
    x[2] = torch.randint(-3, 4, (V,), generator=g, device="cuda").float()        # few distinct logits
    x[3, ::3] = -INF
    x[4] = -8.0
    for c in range(1, 8):                                   # ties on both sides of every slice's border
        x[4, c * slice_ - 150:c * slice_ + 150] = 5.0
    x, u = x.to(dtype), torch.tensor([0.7, 0.31, 0.93, 0.5, 0.66], device="cuda")
    row = lambda v, t=torch.float32: torch.full((S,), v, dtype=t, device="cuda")
    few = False
    for kw, most in [({}, None), (dict(temperature=row(0.0)), 1), (dict(temperature=row(1.7)), None),
                     (dict(top_k=row(5000, torch.int32)), 5000), (dict(top_k=row(40, torch.int32)), 40),
                     (dict(top_k=row(1000, torch.int32), top_p=row(0.6)), 1000),
                     (dict(top_k=row(300000, torch.int32), top_p=row(0.5)), None),
                     (dict(top_p=row(0.9)), None), (dict(top_p=row(0.3), temperature=row(0.5)), None),
                     (dict(min_p=row(0.2)), None),
                     (dict(top_k=row(90000, torch.int32), top_p=row(0.8), min_p=row(0.05),
                           temperature=row(1.2)), 90000)]:
        tok, lp = api.sample(x, u, **kw)
        want, wl, n = definition(x, u, **kw)
        assert torch.equal(tok.long(), want), (tok.tolist(), want.tolist(), n.tolist())
        assert bool(((lp.double() - wl).abs() <= 2.0 ** -24 * wl.abs() + 4e-9).all())
        assert most is None or int(n.max()) <= most
        few |= bool((n > LIST).any()) and bool((n < V).all())
    assert few                                               # long nuclei were among them

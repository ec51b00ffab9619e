"""GPU sampling against the sorted-list oracle: tokens equal, log-probabilities within half a step of
fp32 (2^-24 relative) plus 4e-9 (the sum's weights carry about 2^-30 each)."""
import math

import pytest
import torch

from oracle import rollout_oracle as ro
from shared_prefix_grouped_gb300 import api
from shared_prefix_grouped_gb300.build import build

pytestmark = pytest.mark.gpu
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()


def compare(logits, u, **kw):
    dev = {n: t.cuda() for n, t in kw.items()}
    tok, lp = api.sample(logits.cuda(), u.cuda(), **dev)
    wt, wl = ro.sample(logits, u, **kw)
    assert torch.equal(tok.cpu(), wt), (tok.cpu() != wt).nonzero().flatten().tolist()
    lp = lp.cpu().double()
    fin = torch.isfinite(wl)
    assert torch.equal(torch.isfinite(lp), fin) and bool((lp[~fin] == wl[~fin]).all())
    assert bool(((lp - wl)[fin].abs() <= 2.0 ** -24 * wl[fin].abs() + 4e-9).all())
    return tok.cpu()


def draw(S, V, dtype=torch.float32, seed=0, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((S, V), generator=g) * spread
    x[torch.rand((S, V), generator=g) < 10.0 / V] += 7
    par = dict(temperature=0.3 + 1.2 * torch.rand(S, generator=g),
               top_k=torch.randint(0, max(V // 2, 2), (S,), generator=g, dtype=torch.int32),
               top_p=0.2 + 0.9 * torch.rand(S, generator=g), min_p=0.2 * torch.rand(S, generator=g))
    return x.to(dtype), torch.rand(S, generator=g), par


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 512, 2049, 10007])
def test_every_filter(V, dtype):
    S = 24
    x, u, par = draw(S, V, dtype, seed=V)
    compare(x, u)
    for names in (["temperature"], ["top_k"], ["top_p"], ["min_p"], ["top_k", "top_p"],
                  ["temperature", "top_k", "top_p", "min_p"]):
        compare(x, u, **{n: par[n] for n in names})


@pytest.mark.parametrize("S,V", [(1, 40000), (2, 131072), (40, 70001), (200, 33000), (1, 600000)])
def test_cluster_sizes_and_large_vocabularies(S, V):
    # One row on eight CTAs, rows shared by fewer, one CTA per row, and a slice larger than shared
    # memory keeps.  The definition in fp64 on the GPU (the list oracle would take minutes).
    x, u, par = draw(S, V, seed=S + V)
    par["top_k"][::3] = 0
    d = {n: t.cuda() for n, t in par.items()}
    xd, ud = x.cuda(), u.cuda()
    tok, lp = api.sample(xd, ud, **d)
    X = xd.double()
    w = torch.exp((X - X.amax(-1, keepdim=True)) / d["temperature"].double()[:, None])
    order = torch.sort(X, dim=-1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    rank = torch.arange(V, device="cuda")[None]
    k = d["top_k"].long()[:, None]
    keep = (rank < k) | (k <= 0)
    wk = ws * keep
    p = d["top_p"].double()[:, None]
    keep &= (torch.cumsum(wk, -1) - wk < p * wk.sum(-1, keepdim=True)) | (p >= 1)
    keep &= ws >= d["min_p"].double()[:, None]
    kept = torch.zeros_like(w).scatter_(1, order, ws * keep)
    cum = torch.cumsum(kept, -1)
    want = (cum <= ud.double()[:, None] * kept.sum(-1, keepdim=True)).sum(-1)
    assert torch.equal(tok.long(), want)
    wl = torch.log(w.gather(1, want[:, None]) / w.sum(-1, keepdim=True))[:, 0]
    assert bool(((lp.double() - wl).abs() <= 2.0 ** -24 * wl.abs() + 4e-9).all())


def test_ties_go_to_the_lower_index():
    V = 3000
    x = torch.zeros((8, V))
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 0.999, 0.1, 0.3, 0.9])
    compare(x, u)                                                # u V falls on borders exactly
    compare(x, u, top_k=torch.tensor([1, 2, 7, 100, 2999, 3000, 5000, 0], dtype=torch.int32))
    compare(x, u, top_p=torch.tensor([0.0, 1e-9, 0.25, 0.5, 1 / 3, 0.999, 1.0, 2.0]))
    compare(x, u, top_k=torch.full((8,), 10, dtype=torch.int32), top_p=torch.full((8,), 0.5))
    x[:, 1500:] = -0.0                                            # equal to 0
    compare(x, u, top_k=torch.full((8,), 1600, dtype=torch.int32))
    x = torch.randint(-3, 3, (8, V), generator=torch.Generator().manual_seed(1)).float()
    compare(x.to(torch.bfloat16), u, top_k=torch.full((8,), 700, dtype=torch.int32),
            top_p=torch.full((8,), 0.7), temperature=torch.full((8,), 2.0))


def test_masked_rows_infinities_and_nan():
    V = 700
    x, u, par = draw(8, V, seed=3)
    x[0] = -INF
    x[1] = -INF
    x[1, 650] = -2.0
    x[2, 10:] = -INF
    x[3, 5] = INF
    x[4, 5] = INF
    x[4, 600] = INF
    x[5, ::2] = float("nan")
    x[6] = float("nan")
    x[7] = torch.finfo(torch.float32).min
    for kw in ({}, par, dict(top_k=par["top_k"]), dict(top_p=par["top_p"])):
        tok = compare(x, u, **kw)
        assert tok[0] == -1 and tok[6] == -1 and tok[1] == 650
    compare(x, u, top_k=torch.full((8,), 600, dtype=torch.int32))


def test_top_k_that_cuts_nothing_leaves_the_nucleus_to_top_p():
    # 60 allowed tokens, top_k 100: the nucleus is of the 60.
    x, u, _ = draw(12, 5000, seed=31)
    x[:, 60:] = -INF
    compare(x, u, top_k=torch.full((12,), 100, dtype=torch.int32), top_p=torch.full((12,), 0.6))
    # and with more candidates than a list holds
    x, u, _ = draw(12, 5000, seed=32, spread=0.3)
    x[:, 2000:] = -INF
    compare(x, u, top_k=torch.full((12,), 3500, dtype=torch.int32), top_p=torch.full((12,), 0.8))


@pytest.mark.parametrize("n", [511, 512, 513, 700])
def test_candidate_counts_around_the_list(n):
    # n equal largest logits ahead of the rest, and n different ones
    g = torch.Generator().manual_seed(n)
    x = torch.randn((4, 6000), generator=g)
    x[0, torch.randperm(6000, generator=g)[:n]] = 30.0
    x[1, torch.randperm(6000, generator=g)[:n]] = 30.0 + torch.rand(n, generator=g)
    x[2] = x[1]
    u = torch.tensor([0.37, 0.81, 0.05, 0.5])
    for k in (n - 1, n, n + 1):
        compare(x, u, top_k=torch.full((4,), k, dtype=torch.int32))
        compare(x, u, top_k=torch.full((4,), k, dtype=torch.int32), top_p=torch.full((4,), 0.93),
                min_p=torch.full((4,), 0.4))
    compare(x, u, top_p=torch.full((4,), 0.999999))
    compare(x.to(torch.bfloat16), u, top_k=torch.full((4,), n, dtype=torch.int32),
            top_p=torch.full((4,), 0.9))


def test_greedy_and_extreme_temperatures():
    x, u, par = draw(9, 5000, seed=4)
    x[0, 17] = x[0, 4000] = 99.0
    t = torch.tensor([0.0, -1.0, float("nan"), 1e-30, 1e-3, 1e4, INF, 1e-42, 1e30])
    tok = compare(x, u, temperature=t)
    assert tok[0] == 17 and tok[3] == int(x[3].argmax())
    compare(x, u, **{**par, "temperature": t})


def test_random_numbers_at_their_ends():
    x, _, par = draw(6, 900, seed=5)
    u = torch.tensor([0.0, 2.0 ** -149, 1 - 2.0 ** -24, 2.0 ** -24, 0.5, 1e-30])
    compare(x, u)
    compare(x, u, **par)
    # outside [0, 1) and NaN: the last and the first kept token
    v = torch.tensor([1.0, 7.0, -0.5, float("nan"), INF, -INF])
    tok, _ = api.sample(x.cuda(), v.cuda())
    assert tok.tolist() == [899, 899, 0, 0, 899, 0]


def test_filters_at_their_ends():
    x, u, _ = draw(6, 1000, seed=6)
    compare(x, u, top_k=torch.tensor([-5, 0, 1, 1000, 999, 2 ** 31 - 1], dtype=torch.int32))
    compare(x, u, top_p=torch.tensor([-1.0, 0.0, 1e-20, 1.0, 0.9999999, 5.0]))
    compare(x, u, min_p=torch.tensor([-1.0, 0.0, 1e-30, 1.0, 0.999, 3.0]))


def test_strides_alignment_and_none_outputs():
    x, u, par = draw(7, 1003, torch.bfloat16, seed=7)
    buf = torch.full((7, 1100), 50.0, dtype=torch.bfloat16)      # the padding would win
    buf[:, 3:1006] = x
    d = {n: t.cuda() for n, t in par.items()}
    tok, lp = api.sample(buf.cuda()[:, 3:1006], u.cuda(), **d)
    want = compare(x, u, **par)
    assert torch.equal(tok.cpu(), want)
    guard = torch.full((9,), 77, dtype=torch.int32, device="cuda")
    t2, l2 = api.sample(x.cuda(), u.cuda(), **d, tokens=guard[1:8])
    assert torch.equal(t2.cpu(), want) and guard[0] == 77 and guard[8] == 77
    assert torch.equal(l2, lp)


def test_reproducible_in_a_graph():
    x, u, par = draw(64, 20011, seed=8)
    xd, ud, d = x.cuda(), u.cuda(), {n: t.cuda() for n, t in par.items()}
    want = api.sample(xd, ud, **d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = api.sample(xd, ud, **d)
    for _ in range(3):
        got[0].fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ud.copy_(1 - ud)
    graph.replay()
    torch.cuda.synchronize()
    again = api.sample(xd, ud, **d)
    assert torch.equal(got[0], again[0])


def test_frequencies_follow_the_weights():
    # 20000 equally spaced u over one row: each kept token's share within two spacings of its weight.
    V, n = 50, 20000
    x = torch.randn(V, generator=torch.Generator().manual_seed(2)).expand(n, V).contiguous()
    u = (torch.arange(n) + 0.5) / n
    tok, _ = api.sample(x.cuda(), u.float().cuda())
    share = torch.bincount(tok.cpu().long(), minlength=V).double() / n
    assert float((share - torch.softmax(x[0].double(), 0)).abs().max()) <= 2.0 / n


def test_binding_refusals():
    x, u, par = draw(3, 40, seed=9)
    d = {n: t.cuda() for n, t in par.items()}
    for bad in [dict(u=u.cuda()[:2]), dict(u=u.cuda().double()), dict(top_k=d["top_k"].long()),
                dict(temperature=d["temperature"][:1]), dict(logits=x.cuda().half()),
                dict(logits=x.cuda().t()), dict(top_p=par["top_p"])]:
        a = dict(logits=x.cuda(), u=u.cuda(), **d)
        a.update(bad)
        with pytest.raises(ValueError):
            api.sample(a.pop("logits"), a.pop("u"), **a)

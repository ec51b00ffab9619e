"""The policy loss where rows stream: 8 MB of logits and more, without a gradient 12 MB of rows from 128 KB on, in
every shape of the streaming kernel (with a gradient rows below 48 KB, below 100 KB and above; without one below 128 KB
and above), with the tolerances of tests/test_policy_gpu.py."""
import math

import pytest
import torch

import test_policy_gpu as base
from oracle import policy_oracle as po
from shared_prefix_grouped_gb300 import api
from test_policy_gpu import built  # noqa: F401  (the build, before anything here)

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


CASES = [   # targets of each row, vocabulary, padding, elements before the first, dtype
    ([1] * 480, 9001, 0, 1, BF16), ([2, 0, 1] * 96, 8003, 5, 0, F32), ([1, 0, 3] * 60, 32000, 0, 0, BF16),
    ([1, 2, 0, 1] * 24, 50001, 47, 3, BF16), ([1, 0, 5] * 40, 20001, 1, 1, F32), ([1] * 132, 32003, 0, 0, BF16),
    ([1, 1, 0] * 30, 25000, 0, 0, F32),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"r{len(c[0])}_v{c[1]}_{str(c[4])[6:]}")
def test_parity_in_place_and_alignment(case):
    assert len(case[0]) * case[1] * case[4].itemsize >= 8 << 20
    base.test_many_long_rows(case)


SHAPES = [(240, 10007, F32), (140, 32000, BF16), (105, 20001, F32), (65, 100001, BF16), (40, 131072, F32)]
IDS = ["f32_40KB", "bf16_64KB", "f32_80KB", "bf16_200KB", "f32_524KB"]


@pytest.mark.parametrize("several", [False, True], ids=["one", "several"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_masked_rows_rows_of_nothing_and_nan_among_many(shape, several):
    R, V, dtype = shape
    counts = [1, 2, 1, 3, 0] * (R // 5) if several else [1] * R
    p = base.problem(counts, V, dtype, seed=V + several)
    rows = po.rows_of(p["starts"], R)
    p["w"][:] = 0.75
    x = base.logits_of(p, "cpu").clone()
    low = torch.finfo(dtype).min
    g = torch.Generator().manual_seed(V)
    nothing, lowest, bad, unweighed = (5, 20), 10, (15, 26, R - 4), 31
    for r in nothing:
        x[r] = -math.inf
    x[lowest] = low
    masked = (0, 6, 11, 36, R - 5)
    for r in masked:                        # nine of ten logits masked, not those of its tokens
        keep = [int(p["tok"][n]) for n in range(len(rows)) if rows[n] == r]
        off = torch.rand(V, generator=g) < 0.9
        off[keep] = False
        x[r, off] = -math.inf if r % 2 else low
    x[bad[0], 100], x[bad[1], V - 1], x[bad[2], 0] = math.nan, math.inf, math.nan
    for n, r in enumerate(rows):
        if r == unweighed:
            p["w"][n] = 0
    fwd, step = base.run(p, logits=x.cuda()), base.run(p, logits=x.cuda(), grad=True)
    inplace = x.cuda()
    again = base.run(p, logits=inplace, dlogits=inplace)
    y = torch.where(x == low, torch.full_like(x, -math.inf), x)
    y[lowest] = 0                           # (uniform, whatever the value)
    good = [r for r in range(R) if r not in bad]
    for r in bad:
        y[r] = 0
    want = po.loss(y, p["tok"], advantages=p["adv"], old=p["old"], ref=p["ref"], weights=p["w"],
                   row_starts=p["starts"], clip_low=base.LO, clip_high=base.HI, kl_coef=0.1)
    dl, dp, dloss, dgrad, tol = base.bounds(p, y, want, 0.1)
    ok = torch.tensor([r not in bad for r in rows])
    lse = want[4].clone()
    lse[lowest] = low
    for r in (fwd, step, again):
        base.within(r.lse.cpu()[good], lse[good], dl[good])
        base.within(r.logprobs.cpu()[ok], want[1][ok], dp[ok])
        base.within(r.token_loss.cpu()[ok], want[2][ok], dloss[ok])
        base.within(r.token_grad.cpu()[ok], want[3][ok], dgrad[ok])
        assert bool(r.logprobs.cpu()[~ok].isnan().all()) and bool(r.token_grad.cpu()[~ok].isnan().all())
        assert all(math.isnan(float(r.lse[b])) for b in bad) and math.isnan(float(r.loss))
        assert all(float(r.lse[b]) == -math.inf for b in nothing)
        if r.dlogits is not None:
            base.within(r.dlogits.cpu()[good], want[5][good], tol[good])
            assert all(bool(r.dlogits[b].isnan().all()) for b in bad)
            assert not r.dlogits[unweighed].any() and not any(bool(r.dlogits[b].any()) for b in nothing)
    # (the forward's CTAs may be of another shape than the step's, so their sums are not equal bit by bit)
    assert same([t.nan_to_num(nan=3.0) for t in step[:5]], [t.nan_to_num(nan=3.0) for t in again[:5]])


def tensors(p):
    return {n: p[n].cuda() for n in ("tok", "starts", "old", "ref", "adv", "w")}


def call(x, t, **kw):
    return api.policy_loss(x, t["tok"], advantages=t["adv"], old_logprobs=t["old"], ref_logprobs=t["ref"],
                           weights=t["w"], row_starts=t["starts"], clip_low=base.LO, clip_high=base.HI,
                           kl_coef=0.1, **kw)


def same(a, b):
    return all(x is None and y is None or torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_captured_replayed_and_reproducible(shape):
    R, V, dtype = shape
    counts = [1, 0, 4, 1, 1] * (R // 5)
    ps = [base.problem(counts, V, dtype, seed=s) for s in (11, 12)]
    want = [(base.run(p, grad=True), base.run(p)) for p in ps]
    assert same(want[0][0], base.run(ps[0], grad=True))
    base.check(ps[0], want[0][0])
    t, x = tensors(ps[0]), base.logits_of(ps[0]).contiguous()
    d = torch.empty_like(x)

    def both():
        return call(x, t, dlogits=d), call(x, t)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for k in (1, 0, 1):
        x.copy_(base.logits_of(ps[k]))
        for n in t:
            t[n].copy_(ps[k][n])
        d.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert same(got[0], want[k][0]) and same(got[1], want[k][1])
    assert api.device_status() == 0


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_two_streams_at_once(shape):
    R, V, dtype = shape
    ps = [base.problem([1, 2, 0, 1, 1] * (R // 5), V, dtype, seed=s) for s in (13, 14)]
    want = [(base.run(p, grad=True), base.run(p)) for p in ps]
    args = [(base.logits_of(p), tensors(p)) for p in ps]
    torch.cuda.synchronize()
    outs = []
    for k, s in enumerate((torch.cuda.Stream(), torch.cuda.Stream())):
        with torch.cuda.stream(s):
            outs += [(k, g, call(*args[k], grad=g == 0)) for _ in range(4) for g in (0, 1)]
    torch.cuda.synchronize()
    assert all(same(r, want[k][g]) for k, g, r in outs)
    assert api.device_status() == 0


@pytest.mark.parametrize("V,dtype", [(131072, BF16), (32000, BF16)])
def test_offsets_past_32_bits(V, dtype):
    # the last rows begin more than 2^31 elements into the logits; rows between without a token
    few = 40
    p = base.problem([1, 0, 2, 1] * 10, V, dtype, seed=15)
    R = (1 << 31) // V + few + 9
    x = torch.zeros((R, V), dtype=dtype, device="cuda")
    x[-few:] = base.logits_of(p)
    starts = torch.zeros(R + 1, dtype=torch.int32)
    starts[-few - 1:] = p["starts"]
    t = tensors(dict(p, starts=starts))
    fwd = call(x, t)
    step = call(x, t, dlogits=x)
    torch.cuda.synchronize()
    for r in (fwd, step):
        assert not r.lse[:-few].any()
        base.check(p, r._replace(lse=r.lse[-few:], dlogits=None if r.dlogits is None else r.dlogits[-few:]))
    assert not x[:-few].any() and api.device_status() == 0

"""CPU checks of the policy loss: the oracle against autograd and finite differences, the rows of a packed
layout against a plain listing, and every refusal of the C entry points and of the binding."""
import math

import pytest
import torch

from oracle import policy_oracle as po
from shared_prefix_grouped_gb300 import _lib, api
from shared_prefix_grouped_gb300.build import build

BAD = _lib.PG_ERR_INVALID_ARG


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


# ------------------------------------------------------------------------------------- the oracle --

def problem(seed=0, R=5, V=11, starts=(0, 3, 3, 4, 6, 7)):
    g = torch.Generator().manual_seed(seed)
    N = starts[-1]
    x = torch.randn((R, V), generator=g, dtype=torch.float64)
    return dict(x=x, starts=torch.tensor(starts), tok=torch.randint(0, V, (N,), generator=g),
                adv=torch.randn(N, generator=g, dtype=torch.float64),
                old=-2 + 0.3 * torch.randn(N, generator=g, dtype=torch.float64),
                ref=-2 + 0.3 * torch.randn(N, generator=g, dtype=torch.float64),
                w=torch.rand(N, generator=g, dtype=torch.float64))


def torch_loss(p, x, T, kl):
    """The same loss from torch's own log-softmax."""
    row = torch.tensor(po.rows_of(p["starts"], x.shape[0]))
    lp = torch.log_softmax(x / T, -1)[row, p["tok"]]
    ratio = torch.exp(lp - p["old"])
    sur = torch.minimum(ratio * p["adv"], torch.clamp(ratio, 0.8, 1.3) * p["adv"])
    gap = p["ref"] - lp
    return (p["w"] * (-sur + kl * (torch.exp(gap) - gap - 1))).sum()


@pytest.mark.parametrize("T,kl", [(1.0, 0.0), (0.7, 0.1), (1.5, 0.04)])
def test_oracle_gradient_is_autograds(T, kl):
    for seed in range(4):
        p = problem(seed)
        x = p["x"].clone().requires_grad_()
        L = torch_loss(p, x, T, kl)
        L.backward()
        total, _, _, _, _, d, _ = po.loss(p["x"], p["tok"], advantages=p["adv"], old=p["old"], ref=p["ref"],
                                          weights=p["w"], row_starts=p["starts"], clip_high=0.3, kl_coef=kl,
                                          temperature=T)
        assert abs(total - float(L)) < 1e-12 and torch.allclose(d, x.grad, atol=1e-12)


def test_oracle_gradient_matches_central_differences():
    p, h = problem(7), 1e-6      # truncation h^2, rounding 1e-16 / h ~ 1e-10
    kw = dict(advantages=p["adv"], old=p["old"], ref=p["ref"], weights=p["w"], row_starts=p["starts"],
              kl_coef=0.1, temperature=0.9)
    d = po.loss(p["x"], p["tok"], **kw)[5]
    for r, i in [(0, int(p["tok"][0])), (0, 3), (1, 2), (2, 5), (4, int(p["tok"][6]))]:
        e = torch.zeros_like(p["x"])
        e[r, i] = h
        num = (po.loss(p["x"] + e, p["tok"], **kw)[0] - po.loss(p["x"] - e, p["tok"], **kw)[0]) / (2 * h)
        assert abs(num - float(d[r, i])) < 1e-8


def test_oracle_by_hand():
    ln = math.log
    x = torch.tensor([[ln(1), ln(3)]], dtype=torch.float64)              # probabilities 1/4, 3/4
    tok = torch.tensor([1])

    def run(A, old, **kw):
        L, lp, _, g, lse, d, _ = po.loss(x, tok, advantages=torch.tensor([A]), old=torch.tensor(
            [old], dtype=torch.float64), **kw)
        return L, float(g), d[0].tolist()

    assert run(2.0, ln(0.75)) == (pytest.approx(-2), pytest.approx(-2), pytest.approx([0.5, -0.5]))
    assert run(2.0, ln(0.5))[:2] == (pytest.approx(-2.4), 0.0)           # ratio 1.5, clipped at 1.2
    assert run(-2.0, ln(0.5))[:2] == (pytest.approx(3.0), pytest.approx(3.0))
    assert run(-2.0, ln(0.75 / 0.7))[:2] == (pytest.approx(1.6), 0.0)    # ratio 0.7, clipped at 0.8
    L, g, _ = run(0.0, ln(0.75), ref=torch.tensor([ln(0.375)], dtype=torch.float64), kl_coef=0.5)
    assert L == pytest.approx(0.5 * (0.5 + ln(2) - 1)) and g == pytest.approx(0.25)


# --------------------------------------------------------------------------------- the packed rows --

@pytest.mark.parametrize("plens,gs,rs", [
    ([3, 0, 2], [2, 2, 1], [2, 1, 3, 0, 2]), ([5], [0], []), ([1], [3], [0, 0, 0]), ([4, 4], [1, 2], [1, 1, 1]),
    ([0], [2], [1, 2]), ([7, 1], [4, 3], [9, 0, 1, 2, 5, 5, 1]),
])
def test_packed_rows(plens, gs, rs):
    starts, index = api.policy_rows(plens, gs, rs, device="cpu")
    want = po.packed_rows(plens, gs, rs)
    assert starts.dtype == torch.int32 and starts.numel() == sum(plens) + sum(rs) + 1 and starts[0] == 0
    got = [index[starts[r]:starts[r + 1]].tolist() for r in range(len(want))]
    assert got == want
    # every response token of a group with a prefix is somebody's target, once
    assert len(set(index.tolist())) == index.numel()


def test_packed_rows_refusals():
    for args in ([[3], [2], [1]], [[3, 1], [2], [1, 1]], [[-1], [1], [1]], [[1], [1], [-1]]):
        with pytest.raises(ValueError):
            api.policy_rows(*args, device="cpu")


# --------------------------------------------------------------------------------------- refusals --

def c_args(**kw):
    buf = torch.zeros(64)
    p = buf.data_ptr()
    a = dict(dtype=_lib.PG_F32, rows=2, vocab=4, logits=p, ld=4, n=2, starts=None, tokens=p, old=p, ref=p,
             adv=p, w=p, opts=_lib.PgPolicyOpts(1.0, 0.2, 0.2, 0.1), lse=p, lp=p, tl=p, tg=p, loss=p, dl=p,
             ldd=4, stream=None)
    a.update(kw)
    return a, buf


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(dtype=-1), dict(rows=0), dict(rows=-1), dict(rows=(1 << 27) + 1, starts=64),
    dict(vocab=0), dict(vocab=1 << 30, ld=1 << 30), dict(ld=3), dict(n=3), dict(n=-1, starts=64),
    dict(n=1 << 31, starts=64), dict(logits=None), dict(tokens=None), dict(logits=66), dict(dl=66),
    dict(ldd=3), dict(ldd=8), dict(opts=None), dict(lse=None), dict(lp=None), dict(tl=None), dict(tg=None),
    dict(loss=None), dict(adv=None), dict(old=65), dict(tokens=66), dict(starts=66),
    dict(opts=_lib.PgPolicyOpts(0.0, 0.2, 0.2, 0.1)), dict(opts=_lib.PgPolicyOpts(-1.0, 0.2, 0.2, 0.1)),
    dict(opts=_lib.PgPolicyOpts(math.inf, 0.2, 0.2, 0.1)), dict(opts=_lib.PgPolicyOpts(math.nan, 0.2, 0.2, 0.1)),
    dict(opts=_lib.PgPolicyOpts(1e-39, 0.2, 0.2, 0.1)),
    dict(opts=_lib.PgPolicyOpts(1.0, -0.1, 0.2, 0.1)), dict(opts=_lib.PgPolicyOpts(1.0, 0.2, math.nan, 0.1)),
    dict(opts=_lib.PgPolicyOpts(1.0, 0.2, 0.2, -1.0)), dict(opts=_lib.PgPolicyOpts(1.0, 0.2, 0.2, math.inf)),
], ids=lambda kw: "-".join(kw))
def test_loss_refusals(kw):
    # (checked on the host before anything is launched: no GPU is needed, or touched)
    a, buf = c_args(**kw)
    assert _lib.lib().pg_policy_loss(*a.values()) == BAD


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(rows=0), dict(vocab=0), dict(ld=3), dict(n=1), dict(logits=None), dict(tokens=None),
    dict(T=0.0), dict(T=math.nan), dict(lse=None), dict(tg=None), dict(go=66), dict(dl=None), dict(dl=66),
    dict(ldd=2), dict(ldd=8),
], ids=lambda kw: "-".join(kw))
def test_backward_refusals(kw):
    buf = torch.zeros(64)
    p = buf.data_ptr()
    a = dict(dtype=_lib.PG_F32, rows=2, vocab=4, logits=p, ld=4, n=2, starts=None, tokens=p, T=1.0, lse=p, tg=p,
             go=None, dl=p, ldd=4, stream=None)
    a.update(kw)
    assert _lib.lib().pg_policy_loss_bwd(*a.values()) == BAD


def test_binding_refuses_host_tensors():
    x, t = torch.zeros((2, 4)), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.policy_loss(x, t, advantages=torch.zeros(2))
    with pytest.raises(ValueError):
        api.token_logprobs(x, t)
    with pytest.raises(ValueError):
        api.policy_loss_bwd(x, t, torch.zeros(2), torch.zeros(2))

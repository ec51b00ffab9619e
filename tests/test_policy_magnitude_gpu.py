"""The policy loss on logits that are large beside their differences, where rows stream (8 MB of logits and
more, without a gradient 12 MB of rows from 128 KB on).

Nothing in a row depends on what all its logits have in common but the stored lse, so the oracle gets the logits less
their row's largest (exact in 64 bits), and the tolerances, with E = 2^-24, know only differences: D is 64
plus what a row's tokens lie below its largest logit, over T.  An exponent c (x - m) is off by its product's and
c's rounding, 2 E each of its size, and a thread's factor against the rounding of c m by 8 E; a thread adds
at most 128 terms a piece in two chains (64 E), a CTA's and a cluster's pairs 32 more (7 E each), and a sum is of
positive terms.  So ln sum is off by E (10 D + 300), the stored lse by 4 E |lse| more, a log-probability by
E (6 D + 4 |lp|) more, and loss and gradient as their formulas pass that on; dlogits are rounded once."""
import math

import pytest
import torch

from oracle import policy_oracle as po
from shared_prefix_grouped_gb300 import api
from shared_prefix_grouped_gb300.build import build

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
HALF = {torch.float32: E, torch.bfloat16: 2.0 ** -8}
LO, HI, KL = 0.2, 0.3, 0.1


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()


def targets(x, counts, T, seed):
    """Tokens of every row and what belongs to them, no ratio within 1e-3 of a border of the clipping."""
    g = torch.Generator().manual_seed(seed)
    starts = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    rows = torch.tensor(po.rows_of(starts, len(counts)), dtype=torch.long)
    tok = torch.randint(0, x.shape[1], (len(rows),), generator=g, dtype=torch.int32)
    return dict(starts=starts, rows=rows, tok=tok, T=T, g=g)


def finish(p, x):
    """The old and reference log-probabilities, advantages and weights, near the log-probabilities of x."""
    g, T = p["g"], p["T"]
    top = x.double().amax(1, keepdim=True)
    p["shifted"] = x.double() - top
    p["top"] = top[:, 0]
    lp = torch.log_softmax(p["shifted"] / T, 1)[p["rows"], p["tok"].long()]
    off = 0.5 * torch.randn(len(lp), generator=g, dtype=torch.float64)
    for border in (math.log(1 - LO), math.log(1 + HI)):
        off = torch.where((off - border).abs() < 1e-3, off + 0.01, off)
    p["old"], p["ref"] = (lp - off).float(), (lp + 0.4 * torch.randn(len(lp), generator=g)).float()
    p["adv"], p["w"] = torch.randn(len(lp), generator=g), torch.rand(len(lp), generator=g) + 0.1
    return p


def run(p, x, **kw):
    r = api.policy_loss(x, p["tok"].cuda(), advantages=p["adv"].cuda(), old_logprobs=p["old"].cuda(),
                        ref_logprobs=p["ref"].cuda(), weights=p["w"].cuda(), row_starts=p["starts"].cuda(),
                        clip_low=LO, clip_high=HI, kl_coef=KL, temperature=p["T"], **kw)
    torch.cuda.synchronize()
    assert api.device_status() == 0
    return r


def within(name, got, want, tol):
    off = (got.cpu().double() - want).abs() - tol
    assert bool((off <= 0).all()), (name, float(off.max()), int((~(off <= 0)).sum()))


def check(p, dtype, *results):
    T, rows = p["T"], p["rows"]
    y = p["shifted"]
    _, lp, tl, tg, lse, d, ratio = po.loss(y, p["tok"], advantages=p["adv"], old=p["old"], ref=p["ref"],
                                           weights=p["w"], row_starts=p["starts"], clip_low=LO, clip_high=HI,
                                           kl_coef=KL, temperature=T)
    R = y.shape[0]
    below = torch.zeros(R, dtype=torch.float64)
    for n, r in enumerate(rows.tolist()):
        below[r] = max(float(below[r]), -float(y[r, int(p["tok"][n])]))
    D = 64 + below / T
    ds = E * (10 * D + 300)
    whole = torch.where(torch.bincount(rows, minlength=R) > 0, lse + p["top"] / T, torch.zeros_like(lse))
    dp = ds[rows] + E * (6 * D[rows] + 4 * lp.abs())
    A, w = p["adv"].double().abs(), p["w"].double()
    dr = ratio * (dp + 4 * E + E * (lp - p["old"].double()).abs())
    gap = p["ref"].double() - lp
    em1 = torch.expm1(gap).abs()
    dg = dp + E * gap.abs()
    dloss = w * (A * (dr + 2 * E * (ratio + 2)) + KL * (em1 * dg + 4 * E * (em1 + gap.abs()))) + 2 * E * tl.abs()
    dgrad = w * (A * (dr + 2 * E * ratio) + KL * ((em1 + 1) * dg + 4 * E * em1)) + 2 * E * tg.abs()
    k = torch.bincount(rows, minlength=R).double()
    g_abs = torch.zeros(R, dtype=torch.float64).index_add_(0, rows, tg.abs())
    g_err = torch.zeros(R, dtype=torch.float64).index_add_(0, rows, dgrad)
    prob = torch.exp(y / T - lse[:, None]) * (k > 0)[:, None]
    rel = (ds + E * (6 * D + 12 + k))[:, None] - 6 * E * y / T
    tol = prob * (g_abs[:, None] * rel + g_err[:, None]) / T
    for n, r in enumerate(rows.tolist()):
        tol[r, int(p["tok"][n])] += float((dgrad[n] + 4 * E * g_abs[r]) / T)
    tol = tol * (1 + 2.0 ** -8) + HALF[dtype] * d.abs() + 2.0 ** -126 * (1 + g_abs[:, None] / T)
    for r in results:
        within("lse", r.lse, whole, ds + 4 * E * whole.abs())
        within("logprobs", r.logprobs, lp, dp)
        within("token_loss", r.token_loss, tl, dloss)
        within("token_grad", r.token_grad, tg, dgrad)
        if r.dlogits is not None:
            within("dlogits", r.dlogits, d, tol)


# Rows and targets, vocabulary, type, rows of 40, 64, 200 and 262 KB: 8.5 MB and more, of the longer two 12 MB.
SHAPES = [([1, 0, 2] * 72, 10007, torch.float32), ([1, 1, 0, 1, 3] * 28, 32000, torch.bfloat16),
          ([1, 1, 4] * 22, 50001, torch.float32), ([1, 1, 1, 2] * 13, 131072, torch.bfloat16)]
IDS = ["f32_40KB", "bf16_64KB", "f32_200KB", "bf16_262KB"]


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("common", [300.0, 1e4, -1e6, 1e9, -1e9, 1e10, -3e9])
def test_a_common_offset(shape, common):
    counts, V, dtype = shape
    g = torch.Generator().manual_seed(V)
    x = (common + 2.5 * torch.randn((len(counts), V), generator=g)).to(dtype)
    p = finish(targets(x, counts, 1.0, V + 1), x)
    xd = x.cuda()
    fwd, step = run(p, xd), run(p, xd, grad=True)
    check(p, dtype, fwd, step)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_a_low_temperature(shape):
    counts, V, dtype = shape
    g = torch.Generator().manual_seed(V + 2)
    x = (2.5 * torch.randn((len(counts), V), generator=g)).to(dtype)
    p = targets(x, counts, 0.01, V + 3)
    # the tokens are the largest logits' neighbours, as what was sampled at this temperature is
    p["tok"] = x.float().topk(8, 1).indices[p["rows"], torch.arange(len(p["rows"])) % 8].to(torch.int32)
    p = finish(p, x)
    check(p, dtype, run(p, x.cuda()), run(p, x.cuda(), grad=True))


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("value", [-1e9, 1e9, -3e9, 1e10])
def test_rows_of_one_value(shape, value):
    counts, V, dtype = shape
    x = torch.full((len(counts), V), value).to(dtype)
    p = finish(targets(x, counts, 1.0, V + 4), x)
    fwd, step = run(p, x.cuda()), run(p, x.cuda(), grad=True)
    check(p, dtype, fwd, step)
    assert bool(((step.logprobs.cpu() + math.log(V)).abs() < 1e-4).all())


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("common", [0.0, -2e5])
def test_tokens_far_below_the_largest(shape, common):
    # more than 2^100 below: the sum against the token's logit starts over with a maximum of its own, in the row's
    # first chunk or (where the peak stands at its end) in its last
    counts, V, dtype = shape
    g = torch.Generator().manual_seed(V + 5)
    x = 2.5 * torch.randn((len(counts), V), generator=g)
    p = targets(x, counts, 1.0, V + 6)
    for n, r in enumerate(p["rows"].tolist()):
        peak = (7, V - 3, V // 2)[r % 3]
        if int(p["tok"][n]) == peak:
            p["tok"][n] -= 1
        x[r, peak] = 90.0 if r % 2 else 10.0
    x = (common + x).to(dtype)
    # (in bf16 at the second offset the peak stands in a row of few values)
    p = finish(p, x)
    check(p, dtype, run(p, x.cuda()), run(p, x.cuda(), grad=True))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("common", [0.0, 1e6])
def test_a_row_scores_the_same_in_small_and_large_calls(dtype, common):
    # below 8 MB rows lie in registers, above they stream: either is off by no more than the tolerance above
    V = 20001
    g = torch.Generator().manual_seed(9)
    x = (common + 2.5 * torch.randn((320, V), generator=g)).to(dtype).cuda()
    tok = torch.randint(0, V, (320,), generator=g, dtype=torch.int32).cuda()
    many, _ = api.token_logprobs(x, tok)
    few, _ = api.token_logprobs(x[:8], tok[:8])
    y = x[:8].double()
    lp = torch.log_softmax(y - y.amax(1, keepdim=True), 1).gather(1, tok[:8, None].long())[:, 0]
    below = (y.amax(1) - y.gather(1, tok[:8, None].long())[:, 0])
    tol = E * (16 * (64 + below) + 300 + 4 * lp.abs())
    assert bool(((many[:8] - lp).abs() <= tol).all()) and bool(((few - lp).abs() <= tol).all())

"""GPU parity of the policy loss and its gradient against the fp64 oracle.

Tolerances, with E = 2^-24, Z = the largest |x| / T of a row whose logits are finite, L = log2 of the
number of vectors plus the pieces of a long row.  An exponent c (x - m) of the sum is off by the roundings of
x - m, of c and its own, E |x - m| / T <= 2 E Z each; 2^x by 4 E; a thread adds at most 128 terms a piece, one after another,
two chains, 64 E; joining two (maximum, sum) pairs costs 7 E each, at most 16 of them and one per piece.
The logarithm, its product with ln 2 and the stored value add 4 E (|lse| + Z).  So
|lse - ref| <= E (10 Z + 4 |lse| + 180 + 7 pieces) =: dl, and a log-probability, which shares the sum and
adds its own exponent's error, is off by dl + E (6 Z + 4 |lp|) =: dp.  A ratio is off by the factor
dp + 4 E + E |lp - old|, and the loss and its derivative as their formulas pass that on.  A probability is off by
the factor dl + E (6 Z + 8), and a gradient then by the sums over its tokens (k E each) and half a step of its
type."""
import math

import pytest
import torch

from oracle import policy_oracle as po
from shared_prefix_grouped_gb300 import _lib, api
from shared_prefix_grouped_gb300.build import build

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
HALF = {torch.float32: E, torch.bfloat16: 2.0 ** -8}
LO, HI = 0.2, 0.3


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()


def problem(counts, V, dtype, T=1.0, seed=0, pad=0, scale=2.5, offset=0):
    """Rows with counts[r] targets; no ratio within 1e-3 of a border of the clipping."""
    g = torch.Generator().manual_seed(seed)
    R, N = len(counts), sum(counts)
    flat = (scale * torch.randn(offset + R * (V + pad), generator=g)).to(dtype)
    x = flat[offset:].view(R, V + pad)
    starts = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    rows = po.rows_of(starts, R)
    tok = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    lp = torch.tensor([float(torch.log_softmax(x[r, :V].double() / T, 0)[int(t)])
                       for r, t in zip(rows, tok)]) if N else torch.zeros(0)
    off = 0.5 * torch.randn(N, generator=g)
    for border in (math.log(1 - LO), math.log(1 + HI)):
        off = torch.where((off - border).abs() < 1e-3, off + 0.01, off)
    w = torch.rand(N, generator=g)
    w[torch.rand(N, generator=g) < 0.15] = 0
    return dict(flat=flat, offset=offset, R=R, V=V, pad=pad, T=T, tok=tok,
                starts=None if all(c == 1 for c in counts) else starts, old=(lp - off).float(),
                ref=(lp + 0.4 * torch.randn(N, generator=g)).float(), adv=torch.randn(N, generator=g), w=w)


def logits_of(p, device="cuda"):
    flat = p["flat"].to(device)
    return flat[p["offset"]:].view(p["R"], p["V"] + p["pad"])[:, :p["V"]]


def dev(t):
    return None if t is None else t.cuda()


def run(p, kl=0.1, logits=None, **kw):
    r = api.policy_loss(logits_of(p) if logits is None else logits, p["tok"].cuda(), advantages=p["adv"].cuda(),
                        old_logprobs=dev(p["old"]), ref_logprobs=dev(p["ref"]), weights=dev(p["w"]),
                        row_starts=dev(p["starts"]), clip_low=LO, clip_high=HI, kl_coef=kl, temperature=p["T"], **kw)
    torch.cuda.synchronize()
    assert api.device_status() == 0
    return r


def bounds(p, x, ref, kl):
    """(lse, logprobs, token_loss, token_grad, dlogits): the tolerances above."""
    _, lp, _, tg, lse, d, ratio = ref
    V, T, R = p["V"], p["T"], p["R"]
    xd = x.double()
    fin = torch.where(torch.isfinite(xd), xd, torch.zeros_like(xd))
    Z = fin.abs().amax(1) / T
    pieces = 1 + V * x.element_size() // 262144
    dl = E * (10 * Z + 4 * lse.abs().nan_to_num(posinf=0, neginf=0) + 180 + 7 * pieces)
    rows = torch.tensor(po.rows_of(p["starts"], R), dtype=torch.long)
    lpf = lp.nan_to_num(neginf=0)
    dp = dl[rows] + E * (6 * Z[rows] + 4 * lpf.abs())
    w = torch.ones_like(lp) if p["w"] is None else p["w"].double()
    A = p["adv"].double().abs()
    old = lpf if p["old"] is None else p["old"].double()
    dr = ratio * (dp + 4 * E + E * (lpf - old).abs()) if p["old"] is not None else torch.zeros_like(lp)
    dloss, dgrad = w * A * (dr + 2 * E * (ratio + 2)), w * A * (dr + 2 * E * ratio)
    if p["ref"] is not None and kl > 0:
        gap = p["ref"].double() - lpf
        em1 = torch.expm1(gap).abs()
        dg = dp + E * gap.abs()
        dloss = dloss + w * kl * (em1 * dg + 4 * E * (em1 + gap.abs()))
        dgrad = dgrad + w * kl * ((em1 + 1) * dg + 4 * E * em1)
    prob = torch.zeros_like(d)
    for r in range(R):
        if float(lse[r]) > -math.inf:
            prob[r] = torch.exp(xd[r] / T - lse[r])
    k = torch.zeros(R, dtype=torch.float64).index_add_(0, rows, torch.ones_like(lp))
    g_abs = torch.zeros(R, dtype=torch.float64).index_add_(0, rows, tg.abs())
    g_err = torch.zeros(R, dtype=torch.float64).index_add_(0, rows, dgrad)
    rel = dl + E * (6 * Z + 12 + k)
    tol = prob * ((g_abs * rel + g_err) / T)[:, None]
    for n, r in enumerate(rows.tolist()):
        tol[r, int(p["tok"][n])] += float((dgrad[n] + 4 * E * g_abs[r]) / T)
    tol = tol * (1 + 2.0 ** -8) + HALF[x.dtype] * d.abs() + 2.0 ** -126 * (1 + g_abs[:, None] / T)
    return dl, dp, dloss + 2 * E * ref[2].abs(), dgrad + 2 * E * tg.abs(), tol


def within(got, ref, tol):
    got = got.cpu().double()
    same = (got == ref) | (got.isnan() & ref.isnan())
    off = torch.where(same, torch.zeros_like(ref), (got - ref).abs() - tol)
    assert bool((off <= 0).all()), (float(off.max()), int((off > 0).sum()))


def check(p, r, kl=0.1, x=None):
    x = logits_of(p, "cpu") if x is None else x
    ref = po.loss(x, p["tok"], advantages=p["adv"], old=p["old"], ref=p["ref"], weights=p["w"],
                  row_starts=p["starts"], clip_low=LO, clip_high=HI, kl_coef=kl, temperature=p["T"])
    dl, dp, dloss, dgrad, tol = bounds(p, x, ref, kl)
    within(r.lse, ref[4], dl)
    within(r.logprobs, ref[1], dp)
    within(r.token_loss, ref[2], dloss)
    within(r.token_grad, ref[3], dgrad)
    within(r.loss, torch.tensor([ref[0]], dtype=torch.float64), dloss.sum() + E * abs(ref[0]))
    if r.dlogits is not None:
        within(r.dlogits, ref[5], tol)
    return ref


SHAPES = [   # targets of each row, vocabulary, padding of a row, elements before the first
    ([1], 1, 0, 0), ([1, 1], 2, 0, 0), ([1] * 5, 7, 0, 0), ([1] * 3, 8, 8, 0), ([1] * 3, 1000, 0, 0),
    ([1] * 4, 2047, 3, 1), ([1] * 2, 2049, 0, 3), ([3, 0, 1, 2, 0, 1, 7], 501, 5, 0), ([0], 64, 0, 0),
    ([0, 0, 5], 33, 0, 1), ([300, 1], 129, 0, 0), ([1] * 2, 8193, 0, 0), ([1, 2], 50001, 47, 0),
    ([1, 0, 4], 32000, 0, 0), ([1, 1], 65537, 0, 5), ([2, 1], 131072, 0, 0), ([1], 140001, 0, 0),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"r{len(s[0])}_n{sum(s[0])}_v{s[1]}_pad{s[2]}_at{s[3]}")
def test_parity(shape, dtype):
    counts, V, pad, at = shape
    for T, kl in ((1.0, 0.1), (0.7, 0.0)):
        p = problem(counts, V, dtype, T, seed=V + len(counts), pad=pad, offset=at)
        check(p, run(p, kl, grad=True), kl)
        check(p, run(p, kl), kl)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_a_row_longer_than_the_registers_of_a_cluster(dtype):
    # more than 512 KB a row: several pieces, read again for the gradient, also in place
    V = 300001 if dtype == torch.bfloat16 else 150003
    p = problem([1, 2, 0], V, dtype, 0.9, seed=3, pad=1)
    check(p, run(p, grad=True))
    x = logits_of(p)
    check(p, run(p, logits=x, dlogits=x))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES[2:15:2], ids=lambda s: f"r{len(s[0])}_n{sum(s[0])}_v{s[1]}")
def test_forward_then_backward_and_in_place(shape, dtype):
    counts, V, pad, at = shape
    p = problem(counts, V, dtype, 0.8, seed=V, pad=pad, offset=at)
    step = run(p, grad=True)
    fwd = run(p)
    # what a call returns besides the gradient does not depend on whether that is asked for
    assert all(torch.equal(getattr(step, n), getattr(fwd, n)) for n in ("lse", "logprobs", "token_loss",
                                                                         "token_grad", "loss"))
    x, ref = logits_of(p, "cpu"), check(p, fwd)
    tol = bounds(p, x, ref, 0.1)[4]
    tok, st = p["tok"].cuda(), dev(p["starts"])
    for go in (None, -0.5):
        d = api.policy_loss_bwd(logits_of(p), tok, fwd.lse, fwd.token_grad, row_starts=st, temperature=0.8,
                                grad_output=None if go is None else torch.tensor([go], device="cuda"))
        s = 1.0 if go is None else go
        # (the stored lse is rounded once more: E |lse|, inside the 4 E |lse| of the bound)
        within(d, ref[5] * s, tol)
    # in place: the padding of a row and the elements around stay
    for bwd in (False, True):
        flat = p["flat"].cuda()
        v = flat[at:].view(p["R"], V + pad)[:, :V]
        if bwd:
            api.policy_loss_bwd(v, tok, fwd.lse, fwd.token_grad, row_starts=st, temperature=0.8, dlogits=v)
            within(v, ref[5], tol)
        else:
            r = run(p, logits=v, dlogits=v)
            assert r.dlogits.data_ptr() == v.data_ptr() and torch.equal(r.dlogits, step.dlogits)
            assert torch.equal(r.logprobs, fwd.logprobs) and torch.equal(r.loss, fwd.loss)
        back = flat.cpu()
        assert torch.equal(back[:at], p["flat"][:at])
        assert torch.equal(back[at:].view(p["R"], -1)[:, V:], p["flat"][at:].view(p["R"], -1)[:, V:])


STREAMED = [   # many long rows: targets of each, vocabulary, padding, elements before the first, dtype
    ([1] * 310, 9001, 0, 1, torch.bfloat16), ([1] * 400, 16384, 0, 0, torch.bfloat16),
    ([1, 0, 3, 1, 2] * 65, 8209, 7, 0, torch.float32), ([0] * 200 + [1, 40, 0] * 40, 20001, 3, 2, torch.bfloat16),
    ([1, 2, 0, 1] * 42, 110001, 0, 0, torch.bfloat16), ([1] * 155, 131072, 0, 0, torch.bfloat16),
    ([1, 0, 5] * 55, 60003, 1, 3, torch.float32), ([2, 1] * 40, 131072, 0, 0, torch.float32),
    ([1, 3] * 39, 200001, 7, 0, torch.bfloat16),
]


@pytest.mark.parametrize("case", STREAMED, ids=lambda c: f"r{len(c[0])}_n{sum(c[0])}_v{c[1]}_{str(c[4])[6:]}")
def test_many_long_rows(case):
    counts, V, pad, at, dtype = case
    p = problem(counts, V, dtype, 0.9, seed=V, pad=pad, offset=at)
    fwd = run(p)
    check(p, fwd)
    flat = p["flat"].cuda()
    x = flat[at:].view(p["R"], V + pad)[:, :V]
    r = run(p, logits=x, dlogits=x)                  # in place
    check(p, r)
    back = flat.cpu()
    assert torch.equal(back[:at], p["flat"][:at])
    assert torch.equal(back[at:].view(p["R"], -1)[:, V:], p["flat"][at:].view(p["R"], -1)[:, V:])
    again = run(p, grad=True)
    assert torch.equal(again.dlogits, r.dlogits) and torch.equal(again.loss, r.loss)
    out = torch.full((p["R"], V + 3), 7.0, dtype=dtype, device="cuda")       # another alignment
    run(p, dlogits=out[:, 1:V + 1])
    assert torch.equal(out[:, 1:V + 1], r.dlogits) and bool((out[:, 0] == 7).all() & (out[:, V + 1:] == 7).all())


def test_nothing_but_masked_rows_among_many():
    p = problem([1] * 320, 9000, torch.bfloat16, seed=30)
    x = logits_of(p).clone()
    x[5] = -math.inf
    x[7, 100] = math.nan
    x[300, 8999] = math.inf
    x[9] = torch.finfo(torch.bfloat16).min
    p["w"][:] = 1.0
    p["w"][11] = 0
    r = run(p, logits=x, grad=True)
    assert float(r.lse[5]) == -math.inf and not r.dlogits[5].any() and float(r.token_loss[5]) == 0
    assert math.isnan(float(r.lse[7])) and math.isnan(float(r.lse[300])) and not r.dlogits[11].any()
    assert float(r.lse[9]) == torch.finfo(torch.bfloat16).min
    assert abs(float(r.logprobs[9]) + math.log(9000)) < 1e-4
    good = [i for i in range(320) if i not in (5, 7, 9, 300)]
    y = logits_of(p, "cpu")
    want = po.loss(y, p["tok"], advantages=p["adv"], old=p["old"], ref=p["ref"], weights=p["w"], clip_low=LO,
                   clip_high=HI, kl_coef=0.1)
    tol = bounds(p, y, want, 0.1)[4]
    within(r.dlogits[good], want[5][good], tol[good])


def test_gradient_matches_differences_of_the_loss():
    # fp32 logits, fp64 differences of the oracle's loss at the kernel's own inputs
    p = problem([1, 3, 1], 37, torch.float32, 0.9, seed=8)
    d = run(p, grad=True).dlogits.cpu()
    x, h = logits_of(p, "cpu").double(), 1e-6
    kw = dict(advantages=p["adv"], old=p["old"], ref=p["ref"], weights=p["w"], row_starts=p["starts"], clip_low=LO,
              clip_high=HI, kl_coef=0.1, temperature=0.9)
    for r, i in [(0, int(p["tok"][0])), (0, 5), (1, int(p["tok"][2])), (1, 30), (2, int(p["tok"][4]))]:
        e = torch.zeros_like(x)
        e[r, i] = h
        num = (po.loss(x + e, p["tok"], **kw)[0] - po.loss(x - e, p["tok"], **kw)[0]) / (2 * h)
        assert abs(num - float(d[r, i])) < 1e-6 + 1e-5 * abs(num)


def test_outputs_with_another_alignment_or_stride():
    p = problem([1, 2, 1], 1003, torch.bfloat16, seed=4, pad=5, offset=2)
    want = run(p, grad=True).dlogits
    for at, stride in ((0, 1003), (1, 1008), (3, 1100)):
        buf = torch.full((at + 3 * stride,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[at:].view(3, stride)[:, :1003]
        run(p, dlogits=out)
        assert torch.equal(out, want)
        assert bool((buf[:at] == 7).all()) and bool((buf[at:].view(3, stride)[:, 1003:] == 7).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_masked_logits_and_rows_of_nothing(dtype):
    p = problem([1, 1, 3, 1], 3001, dtype, seed=5)
    x = logits_of(p, "cpu").clone()
    g = torch.Generator().manual_seed(1)
    low = torch.finfo(dtype).min
    for fill in (-math.inf, low):
        y = x.clone()
        for r in range(3):
            y[r, torch.rand(3001, generator=g) < 0.9] = fill
        for n, r in enumerate(po.rows_of(p["starts"], 4)):
            y[r, int(p["tok"][n])] = 1.0 + n         # a token of its own is allowed
        if fill == low:      # products with log2 e overflow to -inf, whose weight is 0 as well
            check(p, run(p, logits=y.cuda(), grad=True), x=torch.where(y == low, torch.full_like(y, -math.inf), y))
        else:
            y[3] = -math.inf
            r = run(p, logits=y.cuda(), grad=True)
            check(p, r, x=y)
            assert float(r.lse[3]) == -math.inf and float(r.logprobs[5]) == -math.inf
            assert not r.dlogits[3].any() and float(r.token_loss[5]) == 0
            b = api.policy_loss_bwd(y.cuda(), p["tok"].cuda(), r.lse, r.token_grad, row_starts=dev(p["starts"]))
            assert not b[3].any() and bool(torch.isfinite(b.float()).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_a_row_of_the_lowest_value_is_uniform(dtype):
    low, V = torch.finfo(dtype).min, 5003
    x = torch.full((2, V), low, dtype=dtype, device="cuda")
    x[1, 77] = -1.0
    r = api.policy_loss(x, torch.tensor([3, 77], dtype=torch.int32, device="cuda"),
                        advantages=torch.ones(2, device="cuda"), grad=True)
    lnv = math.log(V)
    assert float(r.lse[0]) == low and abs(float(r.logprobs[0]) + lnv) <= E * (4 * lnv + 260)
    assert float(r.logprobs[1]) == 0 and float(r.lse[1]) == -1 and not r.dlogits[1].any()
    want = torch.full((V,), 1 / V, dtype=torch.float64)
    want[3] -= 1
    within(r.dlogits[0], want, (HALF[dtype] + 300 * E) * want.abs())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_nan_and_inf_stay_in_their_row(bad):
    p = problem([1, 2, 1], 5000, torch.float32, seed=6)
    p["w"] = torch.tensor([1.0, 1.0, 0.0, 1.0])
    want = run(p, grad=True)
    x = logits_of(p).clone()
    x[1, 4321] = bad
    r = run(p, logits=x, grad=True)
    assert math.isnan(float(r.lse[1])) and bool(r.logprobs[1:3].isnan().all())
    assert math.isnan(float(r.token_loss[1])) and float(r.token_loss[2]) == 0     # weight 0
    assert bool(r.dlogits[1].isnan().all()) and math.isnan(float(r.loss))
    for row in (0, 2):
        assert torch.equal(r.dlogits[row], want.dlogits[row]) and r.lse[row] == want.lse[row]
    # with no weight at all the row has no gradient
    p["w"][1] = 0
    r = run(p, logits=x, grad=True)
    assert not r.dlogits[1].any() and bool(torch.isfinite(r.loss).all())


def test_padding_tokens_and_bad_indices():
    p = problem([1, 3, 1], 700, torch.float32, seed=7)
    p["tok"][[0, 2]] = torch.tensor([-1, -100], dtype=torch.int32)
    r = run(p, grad=True)
    check(p, r)
    assert not r.dlogits[0].any() and float(r.logprobs[0]) == 0
    tok = p["tok"].clone()
    tok[0] = 700                                    # taken as padding, and recorded
    q = api.policy_loss(logits_of(p), tok.cuda(), advantages=p["adv"].cuda(), old_logprobs=p["old"].cuda(),
                        ref_logprobs=p["ref"].cuda(), weights=p["w"].cuda(), row_starts=p["starts"].cuda(),
                        clip_low=LO, clip_high=HI, kl_coef=0.1, grad=True)
    assert api.device_status() == _lib.PG_ERR_DEVICE and api.device_status() == 0
    assert torch.equal(q.dlogits, r.dlogits) and torch.equal(q.loss, r.loss)
    b = api.policy_loss_bwd(logits_of(p), tok.cuda(), r.lse, torch.ones(5, device="cuda"),
                            row_starts=p["starts"].cuda())
    assert api.device_status() == _lib.PG_ERR_DEVICE and not b[0].any()
    for starts in ([0, 1, 9, 5], [-3, 1, 4, 5], [0, 4, 1, 5]):
        api.policy_loss(logits_of(p), p["tok"].cuda(), advantages=p["adv"].cuda(), grad=True,
                        row_starts=torch.tensor(starts, dtype=torch.int32, device="cuda"))
        assert api.device_status() == _lib.PG_ERR_DEVICE


@pytest.mark.parametrize("V", [700, 140001])
def test_tokens_of_no_row_are_recorded(V):
    # (the second: rows that stream)
    R = 6 if V == 700 else 40
    p = problem([1] * R, V, torch.float32, seed=8)
    whole = torch.arange(R + 1, dtype=torch.int32)
    for first, last, code in ((0, R, 0), (1, R, _lib.PG_ERR_DEVICE), (0, R - 1, _lib.PG_ERR_DEVICE)):
        api.policy_loss(logits_of(p), p["tok"].cuda(), advantages=p["adv"].cuda(), grad=True,
                        row_starts=whole.clamp(min=first, max=last).cuda())
        assert api.device_status() == code, (first, last)


@pytest.mark.parametrize("case", [([1], 1 << 22, torch.float32), ([1, 2], 1 << 22, torch.bfloat16),
                                  ([1] * 24, 200001, torch.bfloat16), ([3, 0, 1] * 11, 131072, torch.bfloat16)],
                         ids=lambda c: f"r{len(c[0])}_v{c[1]}")
def test_few_very_long_rows(case):
    counts, V, dtype = case
    p = problem(counts, V, dtype, 0.9, seed=12)
    check(p, run(p))
    check(p, run(p, grad=True))


def test_the_same_token_many_times_in_a_row():
    p = problem([600], 50, torch.float32, seed=9)
    p["tok"][:400] = 7
    check(p, run(p, grad=True))


def test_without_old_reference_or_weights():
    p = problem([1] * 6, 300, torch.float32, seed=10)
    p["old"] = p["ref"] = p["w"] = None
    r = run(p, grad=True)
    check(p, r)
    assert torch.equal(r.token_loss.cpu(), -p["adv"])
    lp, lse = api.token_logprobs(logits_of(p), p["tok"].cuda())
    assert torch.equal(lp, r.logprobs) and torch.equal(lse, r.lse)


def test_no_tokens_at_all():
    x = torch.randn((3, 40), device="cuda")
    none, starts = torch.zeros(0, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    r = api.policy_loss(x, none.int(), advantages=none, old_logprobs=none, row_starts=starts, grad=True)
    assert float(r.loss) == 0 and not r.dlogits.any() and not r.lse.any() and r.logprobs.numel() == 0
    lp, lse = api.token_logprobs(x, none.int(), row_starts=starts)
    assert lp.numel() == 0 and not lse.any()
    assert not api.policy_loss_bwd(x, none.int(), lse, none, row_starts=starts).any()


@pytest.mark.parametrize("V", [513, 60001])
def test_captured_replayed_and_reproducible(V):
    p = problem([1, 0, 4, 1, 1], V, torch.bfloat16, seed=11)
    q = problem([1, 0, 4, 1, 1], V, torch.bfloat16, seed=12)
    want = [run(p, grad=True), run(q, grad=True)]
    again = run(p, grad=True)
    assert all(torch.equal(a, b) for a, b in zip(want[0], again))
    t = {n: p[n].cuda() for n in ("tok", "starts", "old", "ref", "adv", "w")}
    x = logits_of(p).contiguous()
    d = torch.empty_like(x)

    def call():
        r = api.policy_loss(x, t["tok"], advantages=t["adv"], old_logprobs=t["old"], ref_logprobs=t["ref"],
                            weights=t["w"], row_starts=t["starts"], clip_low=LO, clip_high=HI, kl_coef=0.1,
                            dlogits=d)
        return r, api.policy_loss_bwd(x, t["tok"], r.lse, r.token_grad, row_starts=t["starts"])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, b = call()
    for src, w in ((q, want[1]), (p, want[0]), (q, want[1])):
        x.copy_(logits_of(src))
        for n in t:
            t[n].copy_(src[n])
        d.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(r, w))
        assert bool(torch.isfinite(b.float()).all())


def test_two_streams_at_once():
    p = problem([1] * 40, 20001, torch.bfloat16, seed=13)
    want = run(p, grad=True)
    x, args = logits_of(p), [p[n].cuda() for n in ("tok", "adv", "old", "ref", "w")]
    torch.cuda.synchronize()
    outs = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            outs += [api.policy_loss(x, args[0], advantages=args[1], old_logprobs=args[2], ref_logprobs=args[3],
                                     weights=args[4], clip_low=LO, clip_high=HI, kl_coef=0.1, grad=True)
                     for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))


def test_offsets_past_32_bits():
    # the last rows begin more than 2^31 elements into the logits
    V, R = 1 << 20, 2100
    x = torch.zeros((R, V), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x[-2:] = torch.randn((2, V), generator=g, device="cuda").to(torch.bfloat16)
    starts = torch.zeros(R + 1, dtype=torch.int32, device="cuda")
    starts[-2], starts[-1] = 1, 3
    tok = torch.tensor([5, V - 1, 77], dtype=torch.int32, device="cuda")
    adv = torch.tensor([1.0, -1.0, 0.5], device="cuda")
    r = api.policy_loss(x, tok, advantages=adv, row_starts=starts, dlogits=x.clone())
    small = api.policy_loss(x[-2:], tok, advantages=adv, row_starts=starts[-3:].contiguous(), grad=True)
    assert torch.equal(r.dlogits[-2:], small.dlogits) and not r.dlogits[:-2].any()
    assert torch.equal(r.lse[-2:], small.lse) and torch.equal(r.logprobs, small.logprobs)
    z = x[-2:].double()
    assert bool(((torch.logsumexp(z, 1) - small.lse).abs() <= E * (10 * 6 + 4 * 20 + 180 + 7 * 9)).all())


def test_binding_refusals():
    p = problem([1, 1], 40, torch.float32)
    x, tok, adv = logits_of(p), p["tok"].cuda(), p["adv"].cuda()
    for kw in (dict(old_logprobs=adv[:1]), dict(ref_logprobs=adv.double()), dict(weights=adv.cpu()),
               dict(row_starts=torch.zeros(2, dtype=torch.int32, device="cuda")),
               dict(row_starts=torch.zeros(3, device="cuda")), dict(dlogits=x[:1]),
               dict(dlogits=x.to(torch.bfloat16)), dict(dlogits=x.t()), dict(advantages=None)):
        with pytest.raises(ValueError):
            api.policy_loss(x, tok, **{**dict(advantages=adv), **kw})
    for args in ((x.t(), tok), (x, tok[:1]), (x, tok.long()), (x[0], tok), (x.half(), tok)):
        with pytest.raises(ValueError):
            api.policy_loss(*args, advantages=adv)
    with pytest.raises(_lib.PgError):
        api.policy_loss(x, tok, advantages=adv, temperature=0.0)
    for grad in (False, True):                      # one row for all
        with pytest.raises(_lib.PgError):
            api.policy_loss(x[:1].expand(2, 40), tok, advantages=adv, grad=grad)
    with pytest.raises(_lib.PgError):
        api.policy_loss(x, tok, advantages=adv, clip_low=-0.1)
    with pytest.raises(ValueError):
        api.policy_loss_bwd(x, tok, adv, adv[:1])
    with pytest.raises(ValueError):
        api.policy_loss_bwd(x, tok, adv, adv, grad_output=adv)

"""Rows with many targets: a CTA lists those of a row up to a number (512; where rows stream 256, 512 or 1024) and
adds them once, beyond it they are looked up at every vector.  Tolerances of tests/test_policy_gpu.py (a sum over k
targets is off by k E of their absolute values)."""
import pytest
import torch

import test_policy_gpu as base
from shared_prefix_grouped_gb300 import _lib, api
from test_policy_gpu import built  # noqa: F401  (the build, before anything here)

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

FEW = [   # rows that lie in registers
    ([2, 511, 0, 512], 700, 3, 1, F32), ([513, 1, 2], 5003, 0, 0, BF16), ([64, 1, 512], 50001, 47, 3, BF16),
    ([300, 2], 131072, 0, 0, BF16), ([2, 1500], 200001, 1, 1, F32), ([512, 2], 300001, 0, 0, BF16),
]
MANY = [   # rows that stream, of every shape, with as many targets as the list holds and one more
    ([1, 2, 0] * 70 + [255, 256, 257, 2], 10007, 5, 3, F32), ([1, 3] * 65 + [512, 64, 513], 32000, 0, 0, BF16),
    ([1, 0, 2] * 15 + [1023, 1024, 1025, 64], 50001, 1, 1, F32), ([1, 3] * 20 + [256, 64], 131072, 0, 0, BF16),
    ([2, 1] * 80 + [700], 100001, 1, 5, BF16),
]


def case_id(c):
    return f"n{sum(c[0])}_v{c[1]}_{str(c[4])[6:]}"


@pytest.mark.parametrize("case", FEW + MANY, ids=case_id)
@pytest.mark.parametrize("repeated", [False, True], ids=["spread", "repeated"])
def test_parity(case, repeated):
    counts, V, pad, at, dtype = case
    p = base.problem(counts, V, dtype, 0.9, seed=V, pad=pad, offset=at)
    if repeated:                            # first tokens of responses are often the same few, at the ends too
        few = torch.tensor([0, V - 1, V // 2, 7, V - 2, 1, V // 3], dtype=torch.int32)
        x = base.logits_of(p, "cpu")
        starts = torch.tensor([0] + counts).cumsum(0).tolist()
        for r, k in enumerate(counts):
            for j in range(k if k > 2 else 0):
                n, y = starts[r] + j, int(few[(j * j + r) % 7])
                p["tok"][n] = y
                p["old"][n] = float(torch.log_softmax(x[r].double() / 0.9, 0)[y]) - 0.1 if j < 9 else p["old"][n - 7]
        p["ref"] = p["old"] + 0.3
    fwd, step = base.run(p), base.run(p, grad=True)
    ref = base.check(p, step)
    base.check(p, fwd)
    flat = p["flat"].cuda()
    x = flat[at:].view(p["R"], V + pad)[:, :V]
    r = base.run(p, logits=x, dlogits=x)
    assert torch.equal(r.dlogits, step.dlogits)
    tol = base.bounds(p, base.logits_of(p, "cpu"), ref, 0.1)[4]
    tok, st = p["tok"].cuda(), base.dev(p["starts"])
    d = api.policy_loss_bwd(base.logits_of(p), tok, fwd.lse, fwd.token_grad, row_starts=st, temperature=0.9)
    base.within(d, ref[5], tol)
    flat = p["flat"].cuda()
    x = flat[at:].view(p["R"], V + pad)[:, :V]
    api.policy_loss_bwd(x, tok, fwd.lse, fwd.token_grad, row_starts=st, temperature=0.9, dlogits=x)
    assert torch.equal(x, d)


@pytest.mark.parametrize("counts,V", [([40, 3, 513], 900), ([40, 3, 300] + [1] * 230, 10007)], ids=["few", "many"])
def test_padding_and_bad_tokens_among_many(counts, V):
    p = base.problem(counts, V, F32, seed=4)
    p["tok"][::3] = -1
    p["tok"][1::7] = -5
    base.check(p, base.run(p, grad=True))
    tok = p["tok"].clone()
    tok[45] = V                             # taken as padding, and recorded
    p["tok"][45] = -1
    want = base.run(p, grad=True)
    q = api.policy_loss(base.logits_of(p), tok.cuda(), advantages=p["adv"].cuda(), old_logprobs=p["old"].cuda(),
                        ref_logprobs=p["ref"].cuda(), weights=p["w"].cuda(), row_starts=p["starts"].cuda(),
                        clip_low=base.LO, clip_high=base.HI, kl_coef=0.1, grad=True)
    assert api.device_status() == _lib.PG_ERR_DEVICE
    assert torch.equal(q.dlogits, want.dlogits) and torch.equal(q.loss, want.loss)


@pytest.mark.parametrize("rows", [3, 440], ids=["few", "many"])
def test_twenty_thousand_targets(rows):
    p = base.problem([1] * (rows - 1) + [20000], 5003, F32, seed=5)
    base.check(p, base.run(p, grad=True))


def microseconds(fn):
    for _ in range(3):
        fn()
    times = []
    for _ in range(15):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        fn()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    return sorted(times)[7]


@pytest.mark.parametrize("V,dtype", [(131072, BF16), (32000, BF16), (10007, F32)])
def test_a_group_s_targets_cost_little_more_than_one(V, dtype):
    # 256 responses' first tokens in one row of many: beside a hundred microseconds of rows, at most half as long again
    # (at every vector they took several times as long)
    R = (96 << 20) // (V * dtype.itemsize)
    x = torch.randn((R, V), device="cuda").to(dtype)
    d = torch.empty_like(x)

    def call(k):
        counts = torch.ones(R, dtype=torch.int64)
        counts[R // 2] = k
        starts = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).int().cuda()
        n = int(counts.sum())
        tok = torch.randint(0, V, (n,), dtype=torch.int32, device="cuda")
        adv = torch.randn(n, device="cuda")
        return lambda: api.policy_loss(x, tok, advantages=adv, row_starts=starts, dlogits=d)

    one, many = microseconds(call(1)), microseconds(call(256))
    assert many < 1.5 * one + 10, (one, many)

"""GPU parity of the one-token attention over a cache in 8 bits, against the fp64 oracle on the values that the
codes and scales stand for.

Tolerances as in tests/test_decode_gpu.py (E = 2^-24, A the largest sum of |q k|, M the mass, K the keys),
with what the 8-bit products add on the tensor cores: the query is off by 2^-17 of its row's largest element,
a score by 2^-17 W (W: scale max|q| sum|k|); its factor is a product of four (4 E A more).  A weight of a prefix
key is off by 2^-7 of it and by the least steps that the oracle sums up, a weight of an own key by 2^-11.  So
|o - ref| <= (2 (d E A + 4 E A + 2^-17 W) + (K / 8 + 64) E + weight) M + least + half |ref|."""
import math

import pytest
import torch

from oracle import rollout_oracle as ro
from shared_prefix_grouped_gb300 import _lib, api
from shared_prefix_grouped_gb300.build import build

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
HALF = {torch.float32: E, torch.bfloat16: 2.0 ** -8}
SIMT = _lib.PG_FLAG_SIMT
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()


def problem(plens, gsizes, olens, hq, hk, d, ps, dtype, own_pages=None, seed=0, qscale=1.0, spread=2.0,
            vscale=1.0):
    """Pages in random order; blocks with scales of their own; a slot that holds no key holds NaN, and a
    block without one has a NaN scale."""
    g = torch.Generator().manual_seed(seed)
    S, B = sum(gsizes), len(plens)
    wp = max((max(plens) + ps - 1) // ps, 1)
    wo = max((max(olens) + ps - 1) // ps, 0) if own_pages is None else own_pages
    total = B * wp + S * wo + 1
    perm = torch.randperm(total, generator=g).to(torch.int32)
    pp, op = perm[:B * wp].view(B, wp).contiguous(), perm[B * wp:B * wp + S * wo].view(S, wo).contiguous()
    live = torch.zeros((total, ps), dtype=torch.bool)
    for pages, n in [(pp[b], plens[b]) for b in range(B)] + [(op[s], olens[s]) for s in range(S)]:
        for i in range(0, n, ps):
            live[int(pages[i // ps]), :min(ps, n - i)] = True
    codes, scales = [], []
    for mult in (1.0, vscale):
        x = mult * torch.randn((total, ps // 16, 16, hk, d), generator=g, dtype=torch.float64)
        x *= torch.exp2(spread * (torch.rand((total, ps // 16, 1, hk, 1), generator=g, dtype=torch.float64) - 0.5))
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 4)) / 448)))
        c = ro.e4m3_round((x / s[:, :, None, :, None]).clamp(-448, 448)).view(total, ps, hk, d)
        c[~live] = float("nan")
        s[~live.view(total, ps // 16, 16).any(-1)] = float("nan")
        codes.append(c)
        scales.append(s)
    q = (qscale * torch.randn((S, hq, d), generator=g)).to(dtype)
    return dict(q=q, codes=codes, scales=scales, plens=plens, gsizes=gsizes, pp=pp, op=op,
                olens=torch.tensor(olens, dtype=torch.int32), ps=ps, wo=wo)


def caches(p):
    return [api.ScaledCache(c.float().to(F8).cuda(), s.float().cuda())
            for c, s in zip(p["codes"], p["scales"])]


def plan_of(p):
    q = p["q"]
    return api.plan_decode(p["plens"], p["gsizes"], q.shape[1], p["codes"][0].shape[2], q.shape[2], p["ps"],
                           p["wo"], q.dtype)


def run(p, flags=0, scale=0.0, plan=None, **kw):
    plan = plan_of(p) if plan is None else plan
    ws = api.decode_workspace(plan)
    ws.fill_(255)         # NaN bit patterns: nothing may be read that this call did not write
    o, lse = api.decode_attn_e4m3(plan, p["q"].cuda(), *caches(p), p["pp"].cuda() if max(p["plens"]) else None,
                                  p["op"].cuda() if p["wo"] else None, p["olens"].cuda() if p["wo"] else None,
                                  softmax_scale=scale, flags=flags, workspace=ws, **kw)
    torch.cuda.synchronize()
    return o, lse


def check(p, o, lse, tensor_cores, scale=None):
    q = p["q"]
    d = q.shape[2]
    ref, rl, mass, least, A, W = ro.decode_e4m3(q, p["codes"], p["scales"], p["plens"], p["gsizes"], p["pp"],
                                                p["op"], p["olens"] if p["wo"] else None, scale)
    K = max(p["plens"]) + int(p["olens"].max()) + 1
    sums = (K / 8 + 64) * E
    score = (d + 4) * E * A + (2.0 ** -17 * W if tensor_cores else 0)
    weight = 0 if not tensor_cores else (2.0 ** -7 if max(p["plens"]) else 2.0 ** -11)
    o, lse = o.cpu().double(), lse.cpu().double()
    tol = (2 * score + sums + weight) * mass + HALF[q.dtype] * ref.abs()
    if weight == 2.0 ** -7:
        tol = tol + least
    assert bool(((o - ref).abs() <= tol).all()), float(((o - ref).abs() - tol).max())
    empty = torch.isinf(rl)
    assert torch.equal(torch.isneginf(lse), empty)
    dl = (lse - rl)[~empty].abs()
    assert bool((dl <= score + sums + 4 * E * rl[~empty].abs()).all()), float(dl.max())
    assert api.device_status() == 0


CASES = [
    # prefix_lens, group_sizes, own_lens, Hq, Hkv, page_size
    ([0], [1], [1], 1, 1, 16),
    ([16], [1], [0], 1, 1, 16),
    ([1], [2], [0, 1], 2, 1, 16),
    ([100], [3], [5, 0, 64], 8, 2, 32),
    ([128], [1], [128], 4, 4, 128),
    ([0], [4], [15, 16, 17, 300], 12, 3, 16),
    ([129, 0, 257], [2, 3, 1], [1, 0, 127, 128, 129, 200], 6, 2, 64),
    ([700], [5], [33, 7, 250, 16, 17], 32, 8, 16),
    ([1000, 50], [40, 2], [(7 * i) % 90 for i in range(42)], 8, 2, 256),
    ([300], [33], [i for i in range(33)], 5, 1, 32),
    ([260, 9], [3, 0], [3, 2, 1], 32, 1, 64),
    ([513], [2], [2, 90], 64, 1, 16),
    ([2100], [2], [1025, 3], 4, 1, 128),
    ([70], [2], [40, 0], 160, 1, 32),        # more query heads per key/value head than a tile has rows
    ([200], [3], [30, 5, 17], 128, 1, 64),   # and just as many
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["f32", "bf16_simt", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "p%s_g%s_h%dx%d_page%d" % (
    "-".join(map(str, c[0])), "-".join(map(str, c[1])), c[3], c[4], c[5]))
def test_parity(case, kind, d):
    plens, gs, olens, hq, hk, ps = case
    dtype = torch.float32 if kind == "f32" else torch.bfloat16
    p = problem(plens, gs, olens, hq, hk, d, ps, dtype, seed=len(olens) + hq)
    o, lse = run(p, SIMT if kind == "bf16_simt" else 0)
    check(p, o, lse, kind == "bf16" and hq // hk <= 128)


def test_every_length_around_a_tile_and_number_of_responses():
    for n in (1, 31, 32, 33, 65):
        p = problem([140], [n], [(50 * i) % 131 for i in range(n)], 4, 1, 128, 16, torch.bfloat16, seed=n)
        check(p, *run(p), True)
    for lp in (15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 255, 256, 385):
        p = problem([lp], [2], [lp, lp + 1], 4, 1, 128, 16, torch.bfloat16, seed=lp)
        check(p, *run(p), True)


def test_no_own_pages_and_no_keys():
    p = problem([200], [4], [0] * 4, 8, 2, 128, 32, torch.bfloat16, own_pages=0)
    check(p, *run(p), True)
    p = problem([0, 64], [2, 2], [0, 3, 0, 0], 8, 2, 128, 32, torch.bfloat16)
    o, lse = run(p)
    check(p, o, lse, True)
    assert not o[0].any() and bool(torch.isneginf(lse[:, 0]).all())
    p = problem([0], [3], [0] * 3, 4, 2, 128, 32, torch.bfloat16, own_pages=0)
    o, lse = run(p)
    assert not o.any() and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("flags", [0, SIMT], ids=["tensor_cores", "simt"])
def test_large_scores_and_small_and_large_values(flags):
    for kw in (dict(qscale=40.0), dict(qscale=2.0 ** -40), dict(vscale=2.0 ** 60), dict(vscale=2.0 ** -70),
               dict(spread=24.0), dict(qscale=8.0, spread=16.0)):
        p = problem([900], [4], [70, 1, 0, 300], 8, 2, 128, 64, torch.bfloat16, seed=12, **kw)
        check(p, *run(p, flags), flags == 0)
    p = problem([900], [4], [70, 1, 0, 300], 8, 2, 128, 64, torch.bfloat16, seed=13)
    check(p, *run(p, flags, scale=0.7), flags == 0, scale=0.7)


def test_blocks_of_zeros():
    # a block of zeros has the least scale; its keys take part in the softmax all the same
    p = problem([600], [3], [70, 33, 0], 4, 2, 128, 16, torch.bfloat16, seed=14)
    least = 2.0 ** -126
    for pages in (p["pp"][0, :10], p["pp"][0, 20:22], p["op"][0, :2], p["op"][1, 1:3]):
        for x in pages.tolist():
            for c, s in zip(p["codes"], p["scales"]):
                c[x] = torch.where(c[x].isnan(), c[x], torch.zeros_like(c[x]))
                s[x] = least
    check(p, *run(p), True)
    for c, s in zip(p["codes"], p["scales"]):        # nothing but zeros
        c[~c.isnan()] = 0
        s[~s.isnan()] = least
    o, lse = run(p)
    assert not o.any()
    want = torch.log(torch.tensor([670.0, 633.0, 600.0]))
    assert bool(((lse.cpu() - want).abs() <= 64 * E * want).all())


def test_one_key_that_outweighs_many():
    # a first key with half the weight, and thousands that share the rest: none of those may be lost
    n = 4000
    p = problem([n], [2], [0, 700], 4, 1, 128, 64, torch.bfloat16, seed=15, qscale=0.02, spread=0.0)
    p["q"][:, :, 0] = 4.0
    for pages, n in ((p["pp"][0], n), (p["op"][1], 700)):
        page = int(pages[0])
        p["codes"][0][page, 0, 0] = 0
        p["scales"][0][page, 0, 0] = 2.0 ** -8 * 4
        p["codes"][0][page, 0, 0, 0] = 416.0 if n == 4000 else 320.0
        v = p["codes"][1]
        for i in range(n):       # values of one sign, so that what is lost shows
            v[int(pages[i // 64]), i % 64, 0] = v[int(pages[i // 64]), i % 64, 0].abs()
    o, lse = run(p)
    check(p, o, lse, True)


def test_one_plan_serves_a_growing_rollout():
    full = [60, 3, 200]
    p = problem([300], [3], full, 8, 2, 128, 32, torch.bfloat16)
    for c, s in zip(p["codes"], p["scales"]):
        c[c.isnan()] = 1.0
        s[s.isnan()] = 0.5
    plan = plan_of(p)
    q, pp, op, kv = p["q"].cuda(), p["pp"].cuda(), p["op"].cuda(), caches(p)
    lens, ws = torch.zeros(3, dtype=torch.int32, device="cuda"), api.decode_workspace(plan)
    o, lse = torch.empty_like(q), torch.empty((8, 3), device="cuda")
    api.decode_attn_e4m3(plan, q, *kv, pp, op, lens, out=o, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.decode_attn_e4m3(plan, q, *kv, pp, op, lens, out=o, lse=lse, workspace=ws)
    for step in ([0, 0, 0], [1, 3, 128], [60, 0, 200], [33, 2, 129]):
        lens.copy_(torch.tensor(step, dtype=torch.int32))
        o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        p["olens"] = torch.tensor(step, dtype=torch.int32)
        check(p, o, lse, True)


def test_calls_one_after_another_and_on_two_streams():
    ps = [problem([260], [5], [(29 * i + 50 * k) % 140 for i in range(5)], 8, 2, 128, 32, torch.bfloat16,
                  own_pages=5, seed=40 + k) for k in range(4)]
    plan = plan_of(ps[0])
    want = [run(p, plan=plan) for p in ps]
    args = [(p["q"].cuda(), *caches(p), *[p[n].cuda() for n in ("pp", "op", "olens")]) for p in ps]
    ws = api.decode_workspace(plan)
    torch.cuda.synchronize()
    got = [api.decode_attn_e4m3(plan, *args[i % 4], workspace=ws) for i in range(12)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % 4][0]) and torch.equal(l, want[i % 4][1]) for i, (o, l) in enumerate(got))
    outs = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            outs += [api.decode_attn_e4m3(plan, *args[i]) for i in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % 4][0]) and torch.equal(l, want[i % 4][1]) for i, (o, l) in enumerate(outs))


def test_inputs_written_just_before_the_call():
    p = problem([1000], [8], [60 + i for i in range(8)], 8, 2, 128, 32, torch.bfloat16, seed=50)
    want = run(p)
    plan, kv = plan_of(p), caches(p)
    flat = [p["q"].cuda()] + [t.view(torch.uint8) if t.dtype is F8 else t for c in kv for t in c] + \
        [p[n].cuda() for n in ("pp", "op", "olens")]
    big = torch.randn(64 << 20, device="cuda")
    for _ in range(5):
        dst = [torch.zeros_like(t) for t in flat]
        big.mul_(1.0001)                     # keeps the stream busy while the calls queue up
        for d, s in zip(dst, flat):
            d.copy_(s)
        k, v = api.ScaledCache(dst[1].view(F8), dst[2]), api.ScaledCache(dst[3].view(F8), dst[4])
        o, lse = api.decode_attn_e4m3(plan, dst[0], k, v, *dst[5:])
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_rows_do_not_leak_and_what_lies_behind_stays():
    p = problem([1500], [9], [(37 * i) % 200 for i in range(9)], 8, 2, 128, 32, torch.bfloat16, seed=3)
    big = torch.full((11, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    a, la = run(p, out=big[:9])
    assert bool((big[9:] == 7).all())
    s = 4
    p["q"][s] += 1
    for page in p["op"][s].tolist():
        p["scales"][0][page] *= 2
        p["codes"][1][page] = 1.0
    c, lc = run(p)
    keep = [i for i in range(9) if i != s]
    assert torch.equal(a[keep], c[keep]) and torch.equal(la[:, keep], lc[:, keep])
    assert not torch.equal(a[s], c[s])


@pytest.mark.parametrize("flags", [0, SIMT], ids=["tensor_cores", "simt"])
def test_bad_pages_and_lengths_are_reported(flags):
    p = problem([100], [2], [20, 40], 4, 2, 128, 16, torch.bfloat16, seed=7)
    keep = int(p["op"][1, 1])
    p["op"][1, 1] = p["codes"][0].shape[0] + 5
    o, lse = run(p, flags)
    assert api.device_status() == _lib.PG_ERR_DEVICE and api.device_status() == 0
    # the page reads as zero keys and values
    p["op"][1, 1] = keep
    p["codes"][0][keep], p["codes"][1][keep] = 0, 0
    check(p, o, lse, flags == 0)
    pre = int(p["pp"][0, 2])
    p["pp"][0, 2] = -1
    o, lse = run(p, flags)
    assert api.device_status() == _lib.PG_ERR_DEVICE
    p["pp"][0, 2] = pre
    p["codes"][0][pre], p["codes"][1][pre] = 0, 0
    check(p, o, lse, flags == 0)
    p = problem([100], [2], [48, 40], 4, 2, 128, 16, torch.bfloat16, seed=8)
    want = run(p, flags)
    p["olens"][0] = 49        # one more than its three pages hold: cut to them
    o, lse = run(p, flags)
    assert api.device_status() == _lib.PG_ERR_DEVICE
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("flags", [0, SIMT], ids=["tensor_cores", "simt"])
def test_nan_shows_in_its_rows_only(flags):
    p = problem([70], [3], [10, 20, 30], 4, 2, 128, 16, torch.bfloat16, seed=9)
    p["codes"][0][int(p["op"][1, 0]), 3, 0, 7] = float("nan")       # response 1, key/value head 0
    p["q"][2, 3, 5] = float("nan")
    o, lse = run(p, flags)
    assert bool(torch.isnan(o[1, :2]).all()) and bool(torch.isnan(lse[:2, 1]).all())
    assert bool(torch.isnan(o[2, 3]).all()) and bool(torch.isnan(lse[3, 2]))
    assert bool(torch.isfinite(o[0].float()).all()) and bool(torch.isfinite(o[1, 2:].float()).all())
    assert bool(torch.isfinite(o[2, :3].float()).all())


@pytest.mark.parametrize("flags", [0, SIMT], ids=["tensor_cores", "simt"])
def test_slots_past_32_bits(flags):
    # the prefix and the own keys lie more than 2^31 bytes into the caches
    num, few = (2 ** 31) // (256 * 128) + 8, 4
    p = problem([300], [2], [200, 33], 4, 1, 128, 256, torch.bfloat16, seed=16)
    assert p["codes"][0].shape[0] == few + 1
    kv = []
    for c, s in zip(p["codes"], p["scales"]):
        big = torch.zeros((num, 256, 1, 128), dtype=torch.uint8, device="cuda")
        big[-few - 1:] = c.float().to(F8).view(torch.uint8).cuda()
        sc = torch.zeros((num, 16, 1), device="cuda")
        sc[-few - 1:] = s.float().cuda()
        kv.append(api.ScaledCache(big.view(F8), sc))
    shift = num - few - 1
    o, lse = api.decode_attn_e4m3(plan_of(p), p["q"].cuda(), *kv, p["pp"].cuda() + shift, p["op"].cuda() + shift,
                                  p["olens"].cuda(), flags=flags)
    torch.cuda.synchronize()
    check(p, o, lse, flags == 0)


def test_binding_refusals():
    p = problem([40], [2], [4, 2], 4, 2, 128, 16, torch.bfloat16)
    plan, (k, v) = plan_of(p), caches(p)
    a = dict(q=p["q"].cuda(), k=k, v=v, pp=p["pp"].cuda(), op=p["op"].cuda(), ol=p["olens"].cuda())
    short = api.ScaledCache(k.codes, k.scales[:2].contiguous())
    wide = api.ScaledCache(k.codes, k.scales.double())
    for name, bad in [("q", a["q"][:1]), ("q", a["q"].float()), ("k", k.codes), ("k", short), ("v", wide),
                      ("v", api.ScaledCache(v.codes.view(torch.uint8), v.scales)), ("pp", a["pp"][:, :2]),
                      ("op", a["op"][:1]), ("ol", a["ol"].long())]:
        with pytest.raises(ValueError):
            api.decode_attn_e4m3(plan, *{**a, name: bad}.values())
    with pytest.raises(_lib.PgError):
        api.decode_attn_e4m3(plan, a["q"], k, v, None, a["op"], a["ol"])
    with pytest.raises(_lib.PgError):
        api.decode_attn_e4m3(plan, *a.values(), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))

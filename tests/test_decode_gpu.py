"""GPU parity of the one-token attention over a shared prefix and own pages, against the fp64 oracle.

Tolerances, with E = 2^-24 and M = sum_j p_j |v_j| of the element.  A score is a sum of d products of
up to A = max scale sum |q k|: its error is at most d E A, in log2 units too, so p_j is off by a factor
of 1 + 2 d E A (numerator and denominator) and the sums of K terms, at most K / 8 + 64 additions deep,
add (K / 8 + 64) E.  The tensor-core kernels also round p_j to bf16 (2^-8, numerator only).  Then one
rounding to the output type.  So |o - ref| <= (2 d E A + (K / 8 + 64) E + [2^-8]) M + half |ref| and
|lse - ref| <= d E A + (K / 8 + 64) E + 4 E |ref|."""
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


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()


def problem(plens, gsizes, olens, hq, hk, d, ps, dtype, own_pages=None, seed=0, junk=float("nan"),
            qscale=1.0):
    """Pages in random order; every slot that holds no key holds `junk`."""
    g = torch.Generator().manual_seed(seed)
    S, B = sum(gsizes), len(plens)
    wp = max((max(plens) + ps - 1) // ps, 1)
    wo = max((max(olens) + ps - 1) // ps, 0) if own_pages is None else own_pages
    total = B * wp + S * wo + 1
    perm = torch.randperm(total, generator=g).to(torch.int32)
    pp, op = perm[:B * wp].view(B, wp).contiguous(), perm[B * wp:B * wp + S * wo].view(S, wo).contiguous()
    kc, vc = (torch.full((total, ps, hk, d), junk, dtype=dtype) for _ in range(2))

    def fill(pages, n):
        for i in range(n):
            kc[int(pages[i // ps]), i % ps] = torch.randn((hk, d), generator=g).to(dtype)
            vc[int(pages[i // ps]), i % ps] = torch.randn((hk, d), generator=g).to(dtype)

    for b in range(B):
        fill(pp[b], plens[b])
    for s in range(S):
        fill(op[s], olens[s])
    q = (qscale * torch.randn((S, hq, d), generator=g)).to(dtype)
    return dict(q=q, kc=kc, vc=vc, plens=plens, gsizes=gsizes, pp=pp, op=op,
                olens=torch.tensor(olens, dtype=torch.int32), ps=ps, wo=wo)


def run(p, flags=0, scale=0.0, plan=None, **kw):
    q = p["q"].cuda()
    if plan is None:
        plan = api.plan_decode(p["plens"], p["gsizes"], q.shape[1], p["kc"].shape[2], q.shape[2],
                               p["ps"], p["wo"], q.dtype)
    ws = kw.pop("workspace", None)
    if ws is None:
        ws = api.decode_workspace(plan)
        ws.fill_(255)         # NaN bit patterns: nothing may be read that this call did not write
    o, lse = api.decode_attn(plan, q, p["kc"].cuda(), p["vc"].cuda(),
                             p["pp"].cuda() if max(p["plens"]) else None,
                             p["op"].cuda() if p["wo"] else None,
                             p["olens"].cuda() if p["wo"] else None, softmax_scale=scale, flags=flags,
                             workspace=ws, **kw)
    torch.cuda.synchronize()
    return o, lse


def check(p, o, lse, tensor_cores, scale=None):
    q = p["q"]
    d = q.shape[2]
    ref, rl, mass, A = ro.decode(q, p["kc"], p["vc"], p["plens"], p["gsizes"], p["pp"], p["op"],
                                 p["olens"] if p["wo"] else None, scale)
    K = max(p["plens"]) + int(p["olens"].max()) + 1
    sums = (K / 8 + 64) * E
    o, lse = o.cpu().double(), lse.cpu().double()
    tol = (2 * d * E * A + sums + (2.0 ** -8 if tensor_cores else 0)) * mass + HALF[q.dtype] * ref.abs()
    assert bool(((o - ref).abs() <= tol).all()), float(((o - ref).abs() - tol).max())
    empty = torch.isinf(rl)
    assert torch.equal(torch.isneginf(lse), empty)
    dl = (lse - rl)[~empty].abs()
    assert bool((dl <= d * E * A + sums + 4 * E * rl[~empty].abs()).all())
    assert api.device_status() == 0


CASES = [
    # prefix_lens, group_sizes, own_lens, Hq, Hkv, page_size
    ([0], [1], [1], 1, 1, 16),
    ([1], [2], [0, 1], 2, 1, 16),
    ([100], [3], [5, 0, 64], 8, 2, 32),
    ([128], [1], [128], 4, 4, 128),
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
@pytest.mark.parametrize("kind", ["f32", "bf16", "bf16_simt"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "p%s_g%s_h%dx%d_page%d" % (
    "-".join(map(str, c[0])), "-".join(map(str, c[1])), c[3], c[4], c[5]))
def test_parity(case, kind, d):
    plens, gs, olens, hq, hk, ps = case
    dtype = torch.float32 if kind == "f32" else torch.bfloat16
    p = problem(plens, gs, olens, hq, hk, d, ps, dtype, seed=len(olens) + hq)
    o, lse = run(p, SIMT if kind == "bf16_simt" else 0)
    check(p, o, lse, kind == "bf16")


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
    p["olens"], p["wo"] = torch.tensor([-4, 0, -1], dtype=torch.int32), 1
    p["op"] = torch.zeros((3, 1), dtype=torch.int32)
    o, lse = run(p)
    assert not o.any() and bool(torch.isneginf(lse).all()) and api.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_large_scores(dtype):
    # Scores of hundreds: the running maximum moves and single keys win.
    p = problem([900], [4], [70, 1, 0, 300], 8, 2, 128, 64, dtype, seed=12, qscale=40.0)
    check(p, *run(p), dtype == torch.bfloat16)
    p = problem([900], [4], [70, 1, 0, 300], 8, 2, 128, 64, dtype, seed=13)
    check(p, *run(p, scale=0.7), dtype == torch.bfloat16, scale=0.7)


def test_every_number_of_responses_and_lengths_around_a_tile():
    for n in (1, 31, 32, 33, 65):
        p = problem([140], [n], [(50 * i) % 131 for i in range(n)], 4, 1, 128, 16, torch.bfloat16, seed=n)
        check(p, *run(p), True)
    for lp in (15, 16, 17, 63, 64, 65, 127, 255, 256):
        p = problem([lp], [2], [lp, lp + 1], 4, 1, 128, 16, torch.bfloat16, seed=lp)
        check(p, *run(p), True)


def test_one_plan_serves_a_growing_rollout():
    # own_lens is read on the device: the same captured graph, replayed as the responses grow.
    full = [60, 3, 200]
    p = problem([300], [3], full, 8, 2, 128, 32, torch.bfloat16, junk=0.5)
    plan = api.plan_decode([300], [3], 8, 2, 128, 32, p["wo"])
    q, kc, vc, pp, op = (p[n].cuda() for n in ("q", "kc", "vc", "pp", "op"))
    lens, ws = torch.zeros(3, dtype=torch.int32, device="cuda"), api.decode_workspace(plan)
    o, lse = torch.empty_like(q), torch.empty((8, 3), device="cuda")
    api.decode_attn(plan, q, kc, vc, pp, op, lens, out=o, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.decode_attn(plan, q, kc, vc, pp, op, lens, out=o, lse=lse, workspace=ws)
    for step in ([0, 0, 0], [1, 3, 128], [60, 0, 200], [33, 2, 129]):
        lens.copy_(torch.tensor(step, dtype=torch.int32))
        o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        p["olens"] = torch.tensor(step, dtype=torch.int32)
        check(p, o, lse, True)


def test_results_are_reproducible_and_rows_do_not_leak():
    p = problem([1500], [9], [(37 * i) % 200 for i in range(9)], 8, 2, 128, 32, torch.bfloat16, seed=3)
    a, la = run(p)
    b, lb = run(p)
    assert torch.equal(a, b) and torch.equal(la, lb)
    # another response's query and own keys change: every other row bit for bit the same
    s = 4
    p["q"][s] += 1
    for page in p["op"][s]:
        p["kc"][int(page)] = 3.0
        p["vc"][int(page)] = -2.0
    c, lc = run(p)
    keep = [i for i in range(9) if i != s]
    assert torch.equal(a[keep], c[keep]) and torch.equal(la[:, keep], lc[:, keep])
    assert not torch.equal(a[s], c[s])


def test_calls_one_after_another_share_a_workspace():
    # Different problems of one plan, back to back on one stream: nothing of a call is left to the next.
    plan, args, want = None, [], []
    for seed in range(4):
        p = problem([260], [5], [(29 * i + 50 * seed) % 140 for i in range(5)], 8, 2, 128, 32,
                    torch.bfloat16, own_pages=5, seed=40 + seed)
        plan = plan or api.plan_decode([260], [5], 8, 2, 128, 32, 5)
        args.append([p[n].cuda() for n in ("q", "kc", "vc", "pp", "op", "olens")])
        want.append(run(p))
    ws = api.decode_workspace(plan)
    torch.cuda.synchronize()
    got = [api.decode_attn(plan, *args[i % 4], workspace=ws) for i in range(12)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % 4][0]) and torch.equal(l, want[i % 4][1])
               for i, (o, l) in enumerate(got))


def test_inputs_written_just_before_the_call():
    # The kernels of a call begin while the one before them ends: they must not read too early.
    p = problem([1000], [8], [60 + i for i in range(8)], 8, 2, 128, 32, torch.bfloat16, seed=50)
    want = run(p)
    plan = api.plan_decode(p["plens"], p["gsizes"], 8, 2, 128, 32, p["wo"])
    src = [p[n].cuda() for n in ("q", "kc", "vc", "pp", "op", "olens")]
    big = torch.randn(64 << 20, device="cuda")
    for _ in range(5):
        dst = [torch.zeros_like(t) for t in src]
        big.mul_(1.0001)                     # keeps the stream busy while the calls queue up
        for d, s in zip(dst, src):
            d.copy_(s)
        dst[0].mul_(1.0)                     # a kernel right before: q is its output
        o, lse = api.decode_attn(plan, *dst)
        o2 = o + 0                           # and one right after
        torch.cuda.synchronize()
        assert torch.equal(o2, want[0]) and torch.equal(lse, want[1])


def test_rows_behind_the_last_response_stay():
    p = problem([90], [3], [4, 0, 50], 4, 2, 128, 16, torch.bfloat16, seed=5)
    big = torch.full((5, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4 * 3 + 8,), 7.0, device="cuda")
    o, l = run(p, out=big[:3], lse=lse[:12].view(4, 3))
    check(p, o, l, True)
    assert bool((big[3:] == 7).all()) and bool((lse[12:] == 7).all())


def test_shared_pages_between_groups():
    # Two groups whose page tables name the same pages (one context, two batches of responses).
    p = problem([150, 150], [2, 2], [9, 1, 0, 20], 8, 2, 128, 32, torch.bfloat16, seed=6)
    p["pp"][1] = p["pp"][0]
    check(p, *run(p), True)


@pytest.mark.parametrize("flags", [0, SIMT], ids=["tensor_cores", "simt"])
def test_bad_pages_and_lengths_are_reported(flags):
    p = problem([100], [2], [20, 40], 4, 2, 128, 16, torch.bfloat16, seed=7, junk=0.25)
    assert api.device_status() == 0
    keep = int(p["op"][1, 1])
    p["op"][1, 1] = p["kc"].shape[0] + 5
    o, lse = run(p, flags)
    assert api.device_status() == _lib.PG_ERR_DEVICE and api.device_status() == 0
    assert bool(torch.isfinite(o.float()).all())
    # the page reads as zero keys and values
    p["op"][1, 1] = keep
    p["kc"][keep], p["vc"][keep] = 0, 0
    check(p, o, lse, flags == 0)
    p["pp"][0, 2] = -1
    run(p, flags)
    assert api.device_status() == _lib.PG_ERR_DEVICE
    p = problem([100], [2], [48, 40], 4, 2, 128, 16, torch.bfloat16, seed=8)
    want = run(p, flags)
    p["olens"][0] = 49        # one more than its three pages hold: cut to them
    o, lse = run(p, flags)
    assert api.device_status() == _lib.PG_ERR_DEVICE
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_nan_key_shows_in_its_rows_only():
    p = problem([70], [3], [10, 20, 30], 4, 2, 128, 16, torch.bfloat16, seed=9)
    p["kc"][int(p["op"][1, 0]), 3, 0, 7] = float("nan")       # response 1, key/value head 0
    o, lse = run(p)
    assert bool(torch.isnan(o[1, :2]).all()) and bool(torch.isnan(lse[:2, 1]).all())
    assert bool(torch.isfinite(o[[0, 2]].float()).all()) and bool(torch.isfinite(o[1, 2:].float()).all())


def test_long_prefix_and_long_own_keys():
    # 20000 prefix keys and 3000 own ones against fp64 attention on the GPU.
    g = torch.Generator(device="cuda").manual_seed(1)
    ps, S, hq, hk, d, lp = 64, 6, 8, 2, 128, 20001
    lens = [3000, 0, 1, 2999, 64, 1500]
    wp, wo = (lp + ps - 1) // ps, 47
    total = wp + S * wo
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    kc, vc = (torch.randn((total, ps, hk, d), generator=g, device="cuda").to(torch.bfloat16)
              for _ in range(2))
    q = torch.randn((S, hq, d), generator=g, device="cuda").to(torch.bfloat16)
    pp, op = perm[:wp].view(1, wp).contiguous(), perm[wp:].view(S, wo).contiguous()
    ol = torch.tensor(lens, dtype=torch.int32, device="cuda")
    plan = api.plan_decode([lp], [S], hq, hk, d, ps, wo)
    o, lse = api.decode_attn(plan, q, kc, vc, pp, op, ol)
    for s in range(S):
        k = torch.cat([kc[pp[0].long()].view(-1, hk, d)[:lp], kc[op[s].long()].view(-1, hk, d)[:lens[s]]])
        v = torch.cat([vc[pp[0].long()].view(-1, hk, d)[:lp], vc[op[s].long()].view(-1, hk, d)[:lens[s]]])
        x = torch.einsum("hed,khd->hek", q[s].double().view(hk, 4, d), k.double()) * d ** -0.5
        z = torch.logsumexp(x, -1)
        pr = torch.exp(x - z[..., None])
        ref = torch.einsum("hek,khd->hed", pr, v.double()).view(hq, d)
        mass = torch.einsum("hek,khd->hed", pr, v.double().abs()).view(hq, d)
        A, K = 40.0, 23001       # |q||k| / sqrt(d) < 40 for normal draws
        tol = (2 * d * E * A + (K / 8 + 64) * E + 2.0 ** -8) * mass + 2.0 ** -8 * ref.abs()
        assert bool(((o[s].double() - ref).abs() <= tol).all())
        assert bool(((lse[:, s].double() - z.view(-1)).abs() <= d * E * A + (K / 8 + 64) * E).all())


@pytest.mark.parametrize("flags", [0, SIMT], ids=["tensor_cores", "simt"])
def test_slots_past_32_bits(flags):
    # The prefix and the own keys lie more than 2^31 elements (4 GB) into the caches.
    num = (2 ** 31) // (256 * 128) + 8
    g = torch.Generator(device="cuda").manual_seed(2)
    kc, vc = (torch.zeros((num, 256, 1, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    last = num - 4
    for c in (kc, vc):
        c[last:] = torch.randn((4, 256, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn((2, 4, 128), generator=g, device="cuda").to(torch.bfloat16)
    pp = torch.tensor([[last + 2, last]], dtype=torch.int32, device="cuda")
    op = torch.tensor([[last + 3], [last + 1]], dtype=torch.int32, device="cuda")
    ol = torch.tensor([200, 33], dtype=torch.int32, device="cuda")
    plan = api.plan_decode([300], [2], 4, 1, 128, 256, 1)
    o, lse = api.decode_attn(plan, q, kc, vc, pp, op, ol, flags=flags)
    p = dict(q=q.cpu(), kc=kc[last:].cpu(), vc=vc[last:].cpu(), plens=[300], gsizes=[2], pp=pp.cpu() - last,
             op=op.cpu() - last, olens=ol.cpu(), wo=1)
    check(p, o, lse, flags == 0)


def test_two_streams_with_their_own_workspaces():
    p = problem([800], [6], [30, 0, 7, 100, 64, 1], 8, 2, 128, 32, torch.bfloat16, seed=21)
    want = run(p)
    plan = api.plan_decode(p["plens"], p["gsizes"], 8, 2, 128, 32, p["wo"])
    args = [p[n].cuda() for n in ("q", "kc", "vc", "pp", "op", "olens")]
    torch.cuda.synchronize()
    outs = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            outs.append([api.decode_attn(plan, *args) for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for r in outs for o, l in r)


def test_binding_refusals():
    p = problem([40], [2], [4, 2], 4, 2, 128, 16, torch.bfloat16)
    plan = api.plan_decode([40], [2], 4, 2, 128, 16, 1)
    a = dict(q=p["q"].cuda(), kc=p["kc"].cuda(), vc=p["vc"].cuda(), pp=p["pp"].cuda(),
             op=p["op"].cuda(), ol=p["olens"].cuda())
    for name, bad in [("q", a["q"][:1]), ("q", a["q"].float()), ("q", a["q"].cpu()),
                      ("kc", a["kc"][:, :8].contiguous()), ("vc", a["vc"][:1]),
                      ("pp", a["pp"][:, :2]), ("pp", a["pp"].long()), ("op", a["op"][:1]),
                      ("ol", a["ol"].long()), ("ol", a["ol"][:1])]:
        with pytest.raises(ValueError):
            api.decode_attn(plan, *{**a, name: bad}.values())
    with pytest.raises(_lib.PgError):
        api.decode_attn(plan, a["q"], a["kc"], a["vc"], None, a["op"], a["ol"])
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1 << 20, device="cuda")):
        with pytest.raises(ValueError):
            api.decode_attn(plan, *a.values(), workspace=ws)
    with pytest.raises(_lib.PgError):
        api.decode_attn(plan, *a.values(), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))

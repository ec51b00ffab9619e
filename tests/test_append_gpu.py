"""GPU parity of the append to the paged cache against the fp64 oracle.

Values pass through unchanged; rotated ones carry two products and an addition in fp32 with cos / sin
within 5 x 2^-24 and one rounding: 8 x 2^-24 (|a| + |b|) of the pair plus half a step of the type (bf16
2^-8, fp32 2^-24) of the value."""
import pytest
import torch

from oracle import rollout_oracle as ro
from shared_prefix_grouped_gb300 import _lib, api
from shared_prefix_grouped_gb300.build import build

pytestmark = pytest.mark.gpu
E32 = 2.0 ** -24
HALF = {torch.float32: E32, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()


def problem(seqs, per, hq, hk, d, ps, dtype, base=0, fused=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    N = seqs * per
    x = torch.randn((N, hq + 2 * hk, d), generator=g).to(dtype)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    width = (base + per + ps - 1) // ps
    total = seqs * width + 2
    pages = torch.randperm(total, generator=g)[:seqs * width].view(seqs, width).to(torch.int32)
    cache_pos = (base + torch.arange(N) % per).to(torch.int32)
    rows = (torch.arange(N) // per).to(torch.int32)
    kc, vc = (torch.randn((total, ps, hk, d), generator=g).to(dtype) for _ in range(2))
    return dict(q=q, k=k, v=v, kc=kc, vc=vc, pages=pages, cache_pos=cache_pos, rows=rows,
                positions=cache_pos + 1234, x=x, fused=fused)


def run(p, theta, rows=True, positions=True, **kw):
    hq, hk = p["q"].shape[1], p["k"].shape[1]
    if p["fused"]:
        x = p["x"].cuda()
        q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    else:
        q, k, v = (p[n].cuda() for n in ("q", "k", "v"))
    kc, vc = p["kc"].cuda(), p["vc"].cuda()
    qo = api.cache_append(k, v, kc, vc, p["pages"].cuda(), p["cache_pos"].cuda(),
                          page_rows=p["rows"].cuda() if rows else None, q=q if hq else None,
                          positions=p["positions"].cuda() if positions else None, rope_theta=theta,
                          **kw)
    torch.cuda.synchronize()
    return kc.cpu(), vc.cpu(), None if qo is None else qo.cpu()


def pair_sum(x):
    h = x.shape[-1] // 2
    s = x[..., :h].abs() + x[..., h:].abs()
    return torch.cat([s, s], -1)


CASES = [(1, 1, 1, 1, 128, 16, 0), (5, 1, 8, 2, 64, 32, 31), (16, 1, 32, 8, 128, 64, 700),
         (3, 77, 0, 3, 128, 16, 5), (2, 300, 6, 2, 64, 256, 0), (1, 1025, 0, 8, 128, 128, 0),
         (400, 1, 4, 1, 64, 16, 3)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("theta", [0.0, 1e4], ids=["norope", "rope"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "s%dx%d_h%dx%d_d%d_page%d_at%d" % c)
def test_append(case, theta, dtype):
    seqs, per, hq, hk, d, ps, base = case
    p = problem(seqs, per, hq, hk, d, ps, dtype, base, fused=seqs % 2 == 1, seed=seqs + per)
    kc, vc, qo = run(p, theta, rows=per > 1, positions=per % 2 == 1)
    pos = p["positions"] if per % 2 == 1 else None
    want_k, want_v = ro.append(p["k"], p["v"], p["kc"], p["vc"], p["pages"], p["cache_pos"],
                               p["rows"], pos, theta)
    assert torch.equal(vc.double(), want_v)          # and every other slot as it was
    tol = HALF[dtype] * want_k.abs() + (8 * E32 * pair_sum(want_k) if theta else 0)
    assert bool(((kc.double() - want_k).abs() <= tol).all())
    if hq:
        want = ro.rotate(p["q"], p["cache_pos"] if pos is None else pos, theta)
        assert bool(((qo.double() - want).abs()
                     <= HALF[dtype] * want.abs() + 8 * E32 * pair_sum(want)).all())
    assert api.device_status() == 0


def test_padding_rows_store_nothing_and_foreign_slots_stay():
    p = problem(6, 1, 2, 2, 64, 16, torch.bfloat16, base=9, seed=2)
    p["cache_pos"][2] = -1
    p["cache_pos"][5] = -7
    kc, vc, qo = run(p, 1e4, rows=False)
    want_k, want_v = ro.append(p["k"], p["v"], p["kc"], p["vc"], p["pages"], p["cache_pos"], None,
                               p["positions"], 1e4)
    assert torch.equal(vc.double(), want_v)
    assert int((kc != p["kc"]).any(-1).any(-1).sum()) == 4
    assert bool(torch.isfinite(qo.float()).all()) and api.device_status() == 0


@pytest.mark.parametrize("fault", ["page", "negative_page", "position", "row", "negative_row"])
def test_out_of_range_tokens_are_reported_and_not_stored(fault):
    p = problem(4, 1, 2, 2, 128, 16, torch.float32, base=3, seed=8)
    if fault == "page":
        p["pages"][1, 0] = p["kc"].shape[0]
    elif fault == "negative_page":
        p["pages"][1, 0] = -1
    elif fault == "position":
        p["cache_pos"][1] = 16
    elif fault == "row":
        p["rows"][1] = 4
    else:
        p["rows"][1] = -3
    assert api.device_status() == 0
    kc, vc, _ = run(p, 1e4)
    assert api.device_status() == _lib.PG_ERR_DEVICE and api.device_status() == 0
    keep = [0, 2, 3]
    want_k, want_v = ro.append(p["k"][keep], p["v"][keep], p["kc"], p["vc"], p["pages"],
                               p["cache_pos"][keep], p["rows"][keep], p["positions"][keep], 1e4)
    assert torch.equal(vc.double(), want_v)
    assert bool(((kc.double() - want_k).abs() <= E32 * want_k.abs() + 8 * E32 * pair_sum(want_k)).all())


def test_nan_values_are_stored_as_they_are():
    p = problem(3, 1, 0, 1, 64, 16, torch.bfloat16, seed=3)
    p["v"][1, 0, 5] = float("nan")
    p["v"][2, 0, 6] = float("inf")
    kc, vc, _ = run(p, 0.0)
    s = p["pages"][:, 0].long()
    assert torch.isnan(vc[s[1], 0, 0, 5]) and torch.isinf(vc[s[2], 0, 0, 6])
    assert int(torch.isnan(vc).sum()) == 1


def test_far_positions_rotate_exactly():
    # positions near 2^31: angles are reduced in 64-bit fixed point; the frequency itself is rounded
    # to 2^-53 of its value, 2^31 x 2^-53 x 2 pi = 1.5e-6 radians at most
    p = problem(4, 1, 2, 1, 128, 16, torch.float32, seed=4)
    p["positions"] = torch.tensor([2 ** 31 - 1, 2 ** 30 + 12345, 2 ** 24 + 1, 0], dtype=torch.int32)
    _, _, qo = run(p, 5e5)
    want = ro.rotate(p["q"], p["positions"], 5e5)
    assert bool(((qo.double() - want).abs() <= 4e-6 * pair_sum(want)).all())


def test_slots_past_32_bits():
    # A cache whose last pages lie more than 2^31 elements from its start: 65536 pages of 256 slots.
    num = (2 ** 31) // (256 * 128) + 64
    kc = torch.zeros((num, 256, 1, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    x = torch.randn((2, 1, 128), device="cuda").to(torch.bfloat16)
    pages = torch.tensor([[num - 1], [3]], dtype=torch.int32, device="cuda")
    api.cache_append(x, x, kc, vc, pages, torch.tensor([255, 0], dtype=torch.int32, device="cuda"))
    assert torch.equal(vc[num - 1, 255], x[0]) and torch.equal(kc[num - 1, 255], x[0])
    assert torch.equal(vc[3, 0], x[1])
    assert int((vc != 0).any(-1).sum()) == 2 and api.device_status() == 0


def test_q_rotated_in_place_and_in_a_graph():
    p = problem(8, 1, 4, 2, 128, 32, torch.bfloat16, base=40, seed=5)
    want = run(p, 1e4)
    q, k, v = (p[n].cuda() for n in ("q", "k", "v"))
    kc, vc, pages = p["kc"].cuda(), p["vc"].cuda(), p["pages"].cuda()
    cp, pos = p["cache_pos"].cuda(), p["positions"].cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = api.cache_append(k, v, kc, vc, pages, cp, q=q, positions=pos, rope_theta=1e4, q_out=q)
    assert out is q
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])
    assert torch.equal(q.cpu(), want[2])


def test_binding_refusals():
    p = problem(4, 1, 2, 2, 64, 16, torch.bfloat16)
    a = {n: p[n].cuda() for n in ("k", "v", "kc", "vc", "pages", "cache_pos")}
    for name, bad in [("v", a["v"][:3]), ("v", a["v"].float()), ("kc", a["kc"][:, :, :1]),
                      ("vc", a["vc"][:1]), ("kc", a["kc"].transpose(0, 1)), ("pages", a["pages"].long()),
                      ("pages", a["pages"][0]), ("cache_pos", a["cache_pos"][:2]),
                      ("cache_pos", a["cache_pos"].cpu())]:
        b = {**a, name: bad}
        with pytest.raises(ValueError):
            api.cache_append(b["k"], b["v"], b["kc"], b["vc"], b["pages"], b["cache_pos"])

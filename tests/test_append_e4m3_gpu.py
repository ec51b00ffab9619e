"""GPU parity of the append to the cache in 8 bits, and of reading it back, against the fp64 oracle.

What is stored without a rotation is exact: the same codes and scales, bit for bit.  A rotated key is off by
up to 8 x 2^-24 (|a| + |b|) of its pair before it is rounded (tests/test_append_gpu.py), so its code stands
for a number within half a step of e4m3 and that much of the key; a scale is the oracle's unless the
largest value is that near to a border, which none of these inputs is."""
import pytest
import torch

from oracle import rollout_oracle as ro
from shared_prefix_grouped_gb300 import _lib, api
from shared_prefix_grouped_gb300.build import build

pytestmark = pytest.mark.gpu
E32 = 2.0 ** -24
HALF = {torch.float32: E32, torch.bfloat16: 2.0 ** -8}
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()


class Cache:
    """A cache on the GPU and the oracle's beside it; slots that were never written hold NaN codes."""

    def __init__(self, total, ps, hk, d):
        self.ps, self.hk, self.d = ps, hk, d
        self.k, self.v = (api.scaled_cache(total, ps, hk, d) for _ in range(2))
        for c in (self.k, self.v):
            c.codes.view(torch.uint8).fill_(0x7f)
        self.codes = [torch.full((total, ps, hk, d), float("nan"), dtype=torch.float64) for _ in range(2)]
        self.scales = [torch.zeros((total, ps // 16, hk), dtype=torch.float64) for _ in range(2)]

    def append(self, k, v, pages, pos, rows=None, positions=None, theta=0.0, q=None, fused=False):
        a = [k.cuda(), v.cuda()]
        if fused:       # heads of a token as slices of one projection's rows
            x = torch.cat([k[:, :1], k, v], 1).cuda()
            a = [x[:, 1:1 + self.hk], x[:, 1 + self.hk:]]
        dev = [None if t is None else t.cuda() for t in (rows, q, positions)]
        out = api.cache_append_e4m3(*a, self.k, self.v, pages.cuda(), pos.cuda(), page_rows=dev[0], q=dev[1],
                                    positions=dev[2], rope_theta=theta)
        torch.cuda.synchronize()
        ro.append_e4m3(k, v, self.codes, self.scales, pages, pos, rows, positions, theta)
        return out

    def check(self, err_k=None):
        """err_k: how far a key may be off before it is rounded (None: not at all)."""
        assert api.device_status() == 0
        for got, codes, scales, err in ((self.k, self.codes[0], self.scales[0], err_k),
                                        (self.v, self.codes[1], self.scales[1], None)):
            assert torch.equal(got.scales.cpu().double(), scales)
            c = got.codes.cpu().float().double()
            if err is None:
                wrong = (c != codes) & ~(c.isnan() & codes.isnan())
                first = [(i, float(c[tuple(i)]), float(codes[tuple(i)])) for i in wrong.nonzero()[:4].tolist()]
                assert not first, first
            else:
                s = scales.repeat_interleave(16, 1)[..., None]
                step = (c - codes).abs()
                near = 2 * ro.e4m3_round(codes).abs().clamp(min=2.0 ** -6) * 2.0 ** -3
                assert torch.equal(c.isnan(), codes.isnan())
                # another code is the next one, and only where the key is that near to the middle
                other = (step > 0) & ~codes.isnan()
                assert bool((step[other] <= near[other]).all())
                assert float(other.double().mean()) <= err


def tokens(n, hk, d, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(scale * torch.randn((n, hk, d), generator=g)).to(dtype) for _ in range(2)]


def table(seqs, width, seed, extra=2):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(seqs * width + extra, generator=g)[:seqs * width].view(seqs, width).to(torch.int32)


CASES = [   # sequences, tokens each, first index, Hkv, page_size
    (1, 1, 0, 1, 16), (3, 16, 0, 2, 16), (2, 17, 0, 8, 32), (5, 33, 0, 3, 64), (2, 100, 0, 4, 128),
    (1, 300, 0, 2, 256), (40, 3, 0, 2, 16), (1, 15, 0, 5, 16), (17, 1, 0, 1, 32),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "s%d_n%d_at%d_h%d_page%d" % c)
def test_prompts_then_steps(case, d, dtype):
    # a prompt per sequence, then its continuation in pieces of 1, 5 and 16 tokens: blocks that begin, go on
    # and end inside a call, with scales that grow
    S, n, _, hk, ps = case
    width = (n + 40 + ps - 1) // ps
    pages, c = table(S, width, n), Cache(S * width + 2, ps, hk, d)
    at = 0
    for i, per in enumerate((n, 1, 1, 5, 16, 1)):
        k, v = tokens(S * per, hk, d, dtype, 100 + i, scale=2.0 ** (i - 1) if i % 2 else 0.3)
        pos = (at + torch.arange(S * per) % per).to(torch.int32)
        rows = (torch.arange(S * per) // per).to(torch.int32)
        c.append(k, v, pages, pos, None if per == 1 and i == 1 else rows, fused=i == 2)
        at += per
        c.check()
    # read back: every token, and a negative index in between
    pos = torch.arange(-1, at, dtype=torch.int32).repeat(S)
    rows = torch.arange(S, dtype=torch.int32).repeat_interleave(at + 1)
    vals = [ro.cache_values(x, s) for x, s in zip(c.codes, c.scales)]
    for dt in (torch.float32, torch.bfloat16):
        got = api.cache_read_e4m3(c.k, c.v, pages.cuda(), pos.cuda(), page_rows=rows.cuda(), dtype=dt)
        for g, val in zip(got, vals):
            want = torch.stack([val[int(pages[r, p // ps]), p % ps] if p >= 0 else torch.zeros_like(val[0, 0])
                                for r, p in zip(rows.tolist(), pos.tolist())])
            assert torch.equal(g.cpu().double(), want)      # (a code times a power of two is exact in both)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_rotated_keys_and_queries(d, dtype):
    S, n, hk, hq, ps, theta = 3, 45, 2, 6, 32, 5e5
    pages, c = table(S, 3, 1), Cache(11, ps, hk, d)
    g = torch.Generator().manual_seed(5)
    for at, per in ((0, n), (n, 1)):
        k, v = tokens(S * per, hk, d, dtype, per)
        q = torch.randn((S * per, hq, d), generator=g).to(dtype)
        pos = (at + torch.arange(S * per) % per).to(torch.int32)
        rows = (torch.arange(S * per) // per).to(torch.int32)
        positions = (pos + 40000).to(torch.int32)
        out = c.append(k, v, pages, pos, rows, positions, theta, q=q)
        # a key within 8 E (|a| + |b|) <= 2^-19 of a middle between codes 2^-3 apart: one in 2^14 at most
        c.check(err_k=2.0 ** -13)
        ref = ro.rotate(q, positions, theta)
        h = d // 2
        mag = q[..., :h].double().abs() + q[..., h:].double().abs()
        tol = 8 * E32 * torch.cat([mag, mag], -1) + HALF[dtype] * ref.abs()
        assert bool(((out.cpu().double() - ref).abs() <= tol).all())
    # the oracle may have chosen the neighbour of a code: go on from what the GPU holds
    got = ro.cache_values(c.k.codes.cpu().float(), c.k.scales.cpu())
    kr = ro.rotate(k, positions, theta)
    for s in range(S):
        x = got[int(pages[s, n // ps]), n % ps]
        scale = c.k.scales.cpu().double()[int(pages[s, n // ps]), n % ps // 16][:, None]
        half = scale * 2.0 ** (torch.floor(torch.log2((kr[s] / scale).abs().clamp(min=2.0 ** -6))) - 4)
        assert bool(((x - kr[s]).abs() <= half * (1 + 2.0 ** -10) + 16 * E32 * kr[s].abs().max()).all())


def test_padded_batch_and_rows_apart():
    # a padded batch: right padding is -1; the blocks of the others are theirs alone
    S, n, hk, d, ps = 4, 21, 2, 128, 16
    lens = [21, 0, 7, 16]
    pages, c = table(S, 2, 3), Cache(12, ps, hk, d)
    k, v = tokens(S * n, hk, d, torch.bfloat16, 7)
    pos = torch.tensor([[i if i < m else -1 for i in range(n)] for m in lens], dtype=torch.int32).view(-1)
    rows = (torch.arange(S * n) // n).to(torch.int32)
    c.append(k, v, pages, pos, rows)
    c.check()
    # left padding, and sequences in another order
    c2 = Cache(12, ps, hk, d)
    pos = torch.tensor([[i - (n - m) if i >= n - m else -5 for i in range(n)] for m in lens],
                       dtype=torch.int32).view(-1)
    c2.append(k, v, pages, pos, rows.flip(0))
    c2.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_extremes(dtype):
    # zeros, the largest and the smallest numbers, infinities and NaN; then growth over the whole range
    d, hk, ps = 64, 3, 16
    pages, c = torch.zeros((1, 1), dtype=torch.int32), Cache(1, ps, hk, d)
    k = torch.zeros((16, hk, d), dtype=dtype)
    k[1:, 0] = torch.tensor([2.0 ** (8 * i - 60) for i in range(15)], dtype=dtype)[:, None]
    k[:, 1, ::2] = torch.finfo(dtype).max
    k[3, 1, 0], k[5, 1, 1], k[6, 1, 2] = float("nan"), float("inf"), float("-inf")
    k[0, 2] = 2.0 ** -130
    v = -k.flip(0)
    for step in range(16):
        c.append(k[step:step + 1], v[step:step + 1], pages, torch.tensor([step], dtype=torch.int32))
        c.check()
    assert bool(c.k.codes.cpu().float()[0, [3, 5, 6], 1, [0, 1, 2]].isnan().all())
    # all at once gives the scale of the largest
    c = Cache(1, ps, hk, d)
    c.append(k, v, pages, torch.arange(16, dtype=torch.int32), torch.zeros(16, dtype=torch.int32))
    c.check()
    assert float(c.k.scales.cpu()[0, 0, 1]) == 2.0 ** 120


def test_borders_of_the_scale():
    # 448 * 2^e itself takes e, the next number above takes e + 1
    d, ps = 64, 16
    for e in (-126, -20, 0, 7, 119):
        top = 448.0 * 2.0 ** e
        for val, want in ((top, e), (float(torch.nextafter(torch.tensor(top), torch.tensor(float("inf")))), e + 1)):
            c = Cache(1, ps, 1, d)
            k = torch.zeros((1, 1, d))
            k[0, 0, 9] = val
            c.append(k, -k, torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
            c.check()
            assert float(c.k.scales.cpu()) == 2.0 ** want


def test_a_step_taken_back_and_again():
    d, hk, ps = 128, 2, 32
    pages, c = table(2, 1, 8), Cache(4, ps, hk, d)
    k, v = tokens(2 * 20, hk, d, torch.bfloat16, 8)
    pos = (torch.arange(40) % 20).to(torch.int32)
    rows = (torch.arange(40) // 20).to(torch.int32)
    c.append(k, v, pages, pos, rows)
    for scale in (30.0, 0.01):
        k1, v1 = tokens(2, hk, d, torch.bfloat16, 9, scale)
        for at in (18, 18, 19):
            c.append(k1, v1, pages, torch.tensor([at, at], dtype=torch.int32))
            c.check()


@pytest.mark.parametrize("kind", ["page", "row", "index"])
def test_bad_tokens_are_reported_and_not_stored(kind):
    d, hk, ps = 64, 2, 16
    pages, c = table(3, 2, 2), Cache(8, ps, hk, d)
    k, v = tokens(3 * 4, hk, d, torch.float32, 1)
    pos = (14 + torch.arange(12) % 4).to(torch.int32)
    start = (torch.arange(42) % 14).to(torch.int32)
    k0, v0 = tokens(42, hk, d, torch.float32, 3)
    c.append(k0, v0, pages, start, (torch.arange(42) // 14).to(torch.int32))
    c.check()
    rows = (torch.arange(12) // 4).to(torch.int32)
    bad_pages, bad_rows, bad_pos = pages.clone(), rows.clone(), pos.clone()
    if kind == "page":
        bad_pages[1] = torch.tensor([8, -3])
    elif kind == "row":
        bad_rows[4:8] = torch.tensor([3, -1, 77, 3])
    else:
        bad_pos[4:8] = torch.tensor([32, 33, 34, 100000])
    api.cache_append_e4m3(k.cuda(), v.cuda(), c.k, c.v, bad_pages.cuda(), bad_pos.cuda(), page_rows=bad_rows.cuda())
    assert api.device_status() == _lib.PG_ERR_DEVICE and api.device_status() == 0
    keep = [0, 1, 2, 3, 8, 9, 10, 11]
    ro.append_e4m3(k[keep], v[keep], c.codes, c.scales, pages, pos[keep], rows[keep], None, 0.0)
    c.check()
    got = api.cache_read_e4m3(c.k, c.v, bad_pages.cuda(), bad_pos.cuda(), page_rows=bad_rows.cuda())
    assert api.device_status() == _lib.PG_ERR_DEVICE
    assert not got[0][4:8].any() and bool(got[0][:4].any())


def test_slots_past_32_bits():
    num, ps, d = (2 ** 31) // (256 * 128) + 4, 256, 128
    c = [api.ScaledCache(torch.zeros((num, ps, 1, d), dtype=torch.uint8, device="cuda").view(F8),
                         torch.zeros((num, 16, 1), device="cuda")) for _ in range(2)]
    small = Cache(2, ps, 1, d)
    k, v = tokens(300, 1, d, torch.bfloat16, 4)
    pos = torch.arange(300, dtype=torch.int32)
    rows = torch.zeros(300, dtype=torch.int32)
    small.append(k, v, torch.tensor([[0, 1]], dtype=torch.int32), pos, rows)
    pages = torch.tensor([[num - 2, num - 1]], dtype=torch.int32, device="cuda")
    api.cache_append_e4m3(k.cuda(), v.cuda(), *c, pages, pos.cuda(), page_rows=rows.cuda())
    for big, few in zip(c, (small.k, small.v)):
        a, b = big.codes[-2:].view(-1, d)[:300], few.codes.view(-1, d)[:300]
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(big.scales[-2:], few.scales) and not big.codes[:-2].view(torch.uint8).any()
    got = api.cache_read_e4m3(*c, pages, pos.cuda(), page_rows=rows.cuda())
    want = api.cache_read_e4m3(small.k, small.v, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"),
                               pos.cuda(), page_rows=rows.cuda())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_and_replayed():
    # the append of a step, its index advanced on the device, as one graph
    S, hk, d, ps = 5, 2, 128, 32
    pages, c = table(S, 2, 6), Cache(S * 2 + 2, ps, hk, d)
    k = torch.zeros((S, hk, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    pos, pg = torch.zeros(S, dtype=torch.int32, device="cuda"), pages.cuda()
    warm = Cache(S * 2 + 2, ps, hk, d)
    api.cache_append_e4m3(k, v, warm.k, warm.v, pg, pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.cache_append_e4m3(k, v, c.k, c.v, pg, pos)
        pos += 1
    for step in range(35):
        ks, vs = tokens(S, hk, d, torch.bfloat16, step, scale=1 + step % 7)
        k.copy_(ks)
        v.copy_(vs)
        graph.replay()
        torch.cuda.synchronize()
        ro.append_e4m3(ks, vs, c.codes, c.scales, pages, torch.full((S,), step), None, None, 0.0)
    c.check()
    assert pos.tolist() == [35] * S


def test_binding_refusals():
    c = Cache(4, 32, 2, 64)
    k, v = (t.cuda() for t in tokens(3, 2, 64, torch.bfloat16, 1))
    pages, pos = table(3, 1, 1).cuda(), torch.zeros(3, dtype=torch.int32, device="cuda")
    scales = api.ScaledCache(c.k.codes, c.k.scales[:, :1].contiguous())
    plain = api.ScaledCache(c.k.codes.view(torch.uint8), c.k.scales)
    for args in ((k, v[:2], c.k, c.v, pages, pos), (k, v.float(), c.k, c.v, pages, pos),
                 (k, v, c.k.codes, c.v, pages, pos), (k, v, scales, c.v, pages, pos), (k, v, plain, c.v, pages, pos),
                 (k, v, c.k, c.v, pages.long(), pos), (k, v, c.k, c.v, pages, pos[:2]),
                 (k[:, :1], v[:, :1], c.k, c.v, pages, pos), (k, v, c.k, Cache(3, 32, 2, 64).v, pages, pos)):
        with pytest.raises(ValueError):
            api.cache_append_e4m3(*args)
    for args in ((c.k, c.v, pages, pos.long()), (c.k.codes, c.v, pages, pos), (c.k, scales, pages, pos)):
        with pytest.raises(ValueError):
            api.cache_read_e4m3(*args)
    with pytest.raises(ValueError):
        api.cache_read_e4m3(c.k, c.v, pages, pos, dtype=torch.float16)
    with pytest.raises(_lib.PgError):
        api.cache_append_e4m3(k, v, c.k, c.v, pages[:2], pos)

"""Codes of rotated keys: each is the nearest e4m3 number of some value within 8 x 2^-24 (|a| + |b|) of its pair from
the key that 64 bits give, over the block's scale.  So a code that differs from the oracle's is the next one, and its key
lies that near to the middle between them."""
import pytest
import torch

import test_append_e4m3_gpu as base
from oracle import rollout_oracle as ro
from test_append_e4m3_gpu import built  # noqa: F401  (the build, before anything here)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("first,theta", [(0, 1e4), (40000, 5e5), (1 << 20, 1e6), ((1 << 30) - 99, 1e4)])
def test_every_code_is_a_nearest_one(first, theta, d, dtype):
    S, n, hk, ps = 4, 83, 3, 32
    pages, c = base.table(S, 3, 1), base.Cache(S * 3 + 2, ps, hk, d)
    at = 0
    for i, per in enumerate((n, 1)):
        k, v = base.tokens(S * per, hk, d, dtype, 7 * i + d, scale=0.5)
        pos = (at + torch.arange(S * per) % per).to(torch.int32)
        rows = (torch.arange(S * per) // per).to(torch.int32)
        positions = (pos + first).to(torch.int32)
        before = c.k.codes.cpu().float().double()
        c.append(k, v, pages, pos, rows, positions, theta)
        exact = ro.rotate(k, positions, theta)
        a = k.double().abs()
        pair = a + a.roll(d // 2, -1)
        got, scales = c.k.codes.cpu().float().double(), c.k.scales.cpu().double()
        assert torch.equal(scales, c.scales[0])
        for t in range(S * per):
            page, slot = int(pages[int(rows[t]), int(pos[t]) // ps]), int(pos[t]) % ps
            s = scales[page, slot // 16][:, None]
            err = 8 * base.E32 * pair[t] / s
            low, high = ro.e4m3_round(exact[t] / s - err), ro.e4m3_round(exact[t] / s + err)
            mine = got[page, slot]
            assert bool(((mine >= low) & (mine <= high)).all()), (t, float((mine - exact[t] / s).abs().max()))
            before[page, slot] = mine
        if per == n:                 # nothing else was written
            assert torch.equal(before.nan_to_num(nan=1e9), got.nan_to_num(nan=1e9))
        c.codes[0] = got.clone()     # (the next call's earlier codes are these)
        at += per

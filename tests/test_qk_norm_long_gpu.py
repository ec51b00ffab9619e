"""Gain gradients of a long training batch against fp64 sums.

A lane adds the rows of its warp's tokens one after another: 304 blocks of 8 warps share the tokens, a
warp takes 256 / d rows at once, so its chain is L = ceil(T / 2432) ceil(H / (256 / d)) additions deep;
warps, blocks and the final sum add fewer than 32.  Each term is within 32 x 2^-24 of e |xhat|, e = |a|
+ |b| for dy = a cos + b sin (see test_qk_norm_gpu.py), so the sum is within (L + 64) 2^-24 of the sum of
those magnitudes, and the last rounding adds half a step of fp32."""
import math

import pytest
import torch

from shared_prefix_grouped_gb300 import api
from shared_prefix_grouped_gb300.build import build

pytestmark = pytest.mark.gpu
E32, EPS, THETA = 2.0 ** -24, 1e-5, 5e5


def exact(x, dout, pos):
    """(dgain, sum of magnitudes) in fp64, piece by piece."""
    T, H, d = x.shape
    h = d // 2
    freq = THETA ** (-2.0 * torch.arange(h, device="cuda", dtype=torch.float64) / d)
    dg, mag = (torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(2))
    for t in range(0, T, 8192):
        X, D = x[t:t + 8192].double(), dout[t:t + 8192].double()
        ang = (pos[t:t + 8192].double()[:, None] * freq)[:, None]
        a, b = D[..., :h], D[..., h:]
        dy = torch.cat([a * ang.cos() + b * ang.sin(), b * ang.cos() - a * ang.sin()], -1)
        xh = X * (X.square().mean(-1, keepdim=True) + EPS) ** -0.5
        e = a.abs() + b.abs()
        dg += (dy * xh).sum((0, 1))
        mag += (torch.cat([e, e], -1) * xh.abs()).sum((0, 1))
    return dg, mag


@pytest.mark.parametrize("dtype,hq,hk,d", [(torch.bfloat16, 24, 2, 128), (torch.float32, 40, 1, 64)],
                         ids=["bf16", "f32"])
@pytest.mark.parametrize("same_sign", [False, True], ids=["mixed", "same_sign"])
def test_gain_gradients_of_many_tokens(dtype, hq, hk, d, same_sign):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    T = 131077
    g = torch.Generator(device="cuda").manual_seed(d)
    draw = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)
    q, k, dq, dk = draw(T, hq, d), draw(T, hk, d), draw(T, hq, d), draw(T, hk, d)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    if same_sign:      # every term of the sums positive: positions 0, dout along x
        pos.zero_()
        dq, dk = q.clone(), k.clone()
    gain = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dtype)
    grads = api.qk_norm_rope_bwd(q, k, gain, gain, EPS, dq, dk, pos, rope_theta=THETA)
    for x, do, got in ((q, dq, grads[2]), (k, dk, grads[3])):
        want, mag = exact(x, do, pos)
        L = math.ceil(T / 2432) * math.ceil(x.shape[1] / (256 // d))
        assert bool(((got.double() - want).abs() <= (L + 64) * E32 * mag + E32 * want.abs()).all())
        if same_sign:
            assert bool((want > 0).all())
    again = api.qk_norm_rope_bwd(q, k, gain, gain, EPS, dq, dk, pos, rope_theta=THETA)
    assert torch.equal(grads[2], again[2]) and torch.equal(grads[3], again[3])

"""GPU parity of the per-head q / k norm with rotation, forward and backward, against the fp64 oracle.

Tolerances.  u = half a step of the output type (bf16 2^-8, fp32 2^-24), relative to the value.
Forward: y = x r g takes a sum of D squares (12 additions deep), a square root and two products, then
two products and an addition of the rotation with cos / sin within 5 x 2^-24: under 32 x 2^-24 of the
row's largest |y|, so 32 x 2^-24 max|y| + u |y|.  Backward: two such rows of sums, 64 x 2^-24 of the
magnitudes r max(g e) + r max|xhat| mean(|xhat g| e), e = |a| + |b| for dy = a cos + b sin: the two
parts of a rotated gradient may cancel, and its error is relative to the parts.  Gain gradients:
each term 32 x 2^-24 of e |xhat|, then sums at most 512 additions deep in one lane and 32 across:
576 x 2^-24 of the sum of magnitudes."""
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


def make(T, hq, hk, d, dtype, seed=0, fused=False):
    g = torch.Generator().manual_seed(seed)
    if fused:
        x = torch.randn((T, hq + 2 * hk, d), generator=g).to(dtype)
        q, k = x[:, :hq], x[:, hq:hq + hk]
    else:
        q = (3 * torch.randn((T, hq, d), generator=g)).to(dtype)
        k = (0.01 * torch.randn((T, hk, d), generator=g)).to(dtype)
    gq, gk = ((1 + 0.3 * torch.randn(d, generator=g)).to(dtype) for _ in range(2))
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    dq, dk = (torch.randn((T, h, d), generator=g).to(dtype) for h in (hq, hk))
    return q, k, gq, gk, pos, dq, dk


def close(got, want, atol, rel):
    got = got.cpu().double()
    assert bool(torch.isfinite(got).all())
    over = (got - want).abs() - (atol + rel * want.abs())
    assert float(over.max()) <= 0, float(over.max())


def device_views(q, k):
    """q and k on the GPU with the strides they have here (slices of one buffer stay slices)."""
    if q.untyped_storage().data_ptr() == k.untyped_storage().data_ptr():
        base = torch.as_strided(q, (q.shape[0], q.stride(0)), (q.stride(0), 1), 0).cuda()
        return (torch.as_strided(base, t.shape, t.stride(), t.storage_offset()) for t in (q, k))
    return q.cuda(), k.cuda()


CASES = [(1, 1, 1, 128), (3, 5, 1, 64), (17, 8, 2, 128), (130, 7, 7, 64), (257, 32, 8, 128),
         (1000, 3, 1, 128), (5001, 2, 1, 64)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("theta", [0.0, 5e5], ids=["norope", "rope"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "t%d_h%dx%d_d%d" % c)
def test_forward_and_backward(case, theta, dtype):
    T, hq, hk, d = case
    q, k, gq, gk, pos, dq, dk = make(*case, dtype, seed=T, fused=T % 2 == 1)
    eps = 1e-5
    dev = [t.cuda() for t in (gq, gk, pos, dq, dk)]
    qd, kd = device_views(q, k)
    qo, ko = api.qk_norm_rope_fwd(qd, kd, dev[0], dev[1], eps, dev[2], rope_theta=theta)
    grads = api.qk_norm_rope_bwd(qd, kd, dev[0], dev[1], eps, dev[3], dev[4], dev[2],
                                 rope_theta=theta)
    torch.cuda.synchronize()
    for x, g, do, out, dx, dg in ((q, gq, dq, qo, grads[0], grads[2]),
                                  (k, gk, dk, ko, grads[1], grads[3])):
        want = ro.norm_rope(x, g, eps, pos, theta)
        close(out, want, 32 * E32 * want.abs().amax(-1, keepdim=True), HALF[dtype])
        wx, wg, (row, mag) = ro.norm_rope_bwd(x, g, eps, do, pos, theta)
        close(dx, wx, 64 * E32 * row, HALF[dtype])
        close(dg, wg, 576 * E32 * mag, E32)


def test_gradients_match_differences_of_the_kernel():
    # fp32, loss = sum(w y) in fp64: step 2^-6 along a direction; the forward's rounding 2^-23 |y|
    # sums to about 2^-23 sqrt(n) |w y| / step = 1e-3, the third derivative's share is below 1e-3.
    q, k, gq, gk, pos, dq, dk = (t.cuda() for t in make(40, 4, 2, 128, torch.float32, seed=9))
    k = k * 100
    g = torch.Generator().manual_seed(4)
    vq, vk = (torch.randn(t.shape, generator=g).cuda() for t in (q, k))
    vgq, vgk = (torch.randn(128, generator=g).cuda() for _ in range(2))

    def loss(h):
        a, b = api.qk_norm_rope_fwd(q + h * vq, k + h * vk, gq + h * vgq, gk + h * vgk, 1e-5, pos,
                                    rope_theta=1e4)
        return float((a.double() * dq.double()).sum() + (b.double() * dk.double()).sum())

    gr = api.qk_norm_rope_bwd(q, k, gq, gk, 1e-5, dq, dk, pos, rope_theta=1e4)
    want = sum(float((a.double() * v.double()).sum()) for a, v in zip(gr, (vq, vk, vgq, vgk)))
    h = 2.0 ** -6
    num = (8 * (loss(h) - loss(-h)) - (loss(2 * h) - loss(-2 * h))) / (12 * h)
    assert abs(num - want) <= 2e-3 * abs(want) + 2e-2, (num, want)


def test_in_place_and_outputs_given():
    q, k, gq, gk, pos, dq, dk = (t.cuda() for t in make(65, 4, 2, 128, torch.bfloat16, seed=3))
    a, b = api.qk_norm_rope_fwd(q, k, gq, gk, 1e-6, pos, rope_theta=1e4)
    q2, k2 = q.clone(), k.clone()
    r = api.qk_norm_rope_fwd(q2, k2, gq, gk, 1e-6, pos, rope_theta=1e4, q_out=q2, k_out=k2)
    assert r[0] is q2 and torch.equal(q2, a) and torch.equal(k2, b)


def test_one_tensor_without_heads():
    q, k, gq, gk, pos, dq, dk = (t.cuda() for t in make(37, 3, 2, 64, torch.float32, seed=11))
    none = q[:, :0]
    a = api.qk_norm_rope_fwd(q, k, gq, gk, 1e-5, pos, rope_theta=1e4)
    b = api.qk_norm_rope_fwd(none, k, gq, gk, 1e-5, pos, rope_theta=1e4)
    assert b[0].numel() == 0 and torch.equal(a[1], b[1])
    ga = api.qk_norm_rope_bwd(q, k, gq, gk, 1e-5, dq, dk, pos, rope_theta=1e4)
    gb = api.qk_norm_rope_bwd(none, k, gq, gk, 1e-5, dq[:, :0], dk, pos, rope_theta=1e4)
    assert torch.equal(ga[1], gb[1]) and not gb[2].any()
    assert torch.allclose(ga[3], gb[3], rtol=1e-5, atol=1e-4)      # summed over other warps


def test_backward_in_place():
    # dq may be dq_out, dk may be dk_out (the C entry point)
    q, k, gq, gk, pos, dq, dk = (t.cuda() for t in make(301, 7, 2, 128, torch.bfloat16, seed=12))
    want = api.qk_norm_rope_bwd(q, k, gq, gk, 1e-5, dq, dk, pos, rope_theta=1e4)
    L, dg = _lib.lib(), [torch.empty(128, device="cuda") for _ in range(2)]
    n = L.pg_qk_norm_rope_bwd_workspace(301, 7, 2, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert L.pg_qk_norm_rope_bwd(
        _lib.PG_BF16, 301, 7, 2, 128, q.data_ptr(), 7 * 128, k.data_ptr(), 2 * 128, gq.data_ptr(),
        gk.data_ptr(), 1e-5, dq.data_ptr(), dk.data_ptr(), pos.data_ptr(), 1e4, dq.data_ptr(),
        dk.data_ptr(), dg[0].data_ptr(), dg[1].data_ptr(), ws.data_ptr(), n,
        torch.cuda.current_stream().cuda_stream) == _lib.PG_OK
    assert torch.equal(dq, want[0]) and torch.equal(dk, want[1])
    assert torch.equal(dg[0], want[2]) and torch.equal(dg[1], want[3])


def test_rows_of_zeros_and_extreme_values():
    q = torch.zeros((2, 2, 64), device="cuda")
    q[1] = 1e-18
    k = torch.full((2, 1, 64), 1e17, device="cuda")
    g = torch.ones(64, device="cuda")
    qo, ko = api.qk_norm_rope_fwd(q, k, g, g, 1e-5)
    assert not qo[0].any()
    assert torch.allclose(qo[1], torch.full_like(qo[1], 1e-18 * 1e5 ** 0.5), rtol=1e-5, atol=0)
    assert torch.allclose(ko, torch.ones_like(ko), rtol=1e-5)


def test_gain_gradients_are_reproducible_and_the_workspace_carries_nothing():
    q, k, gq, gk, pos, dq, dk = (t.cuda() for t in make(3000, 8, 2, 128, torch.bfloat16, seed=5))
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")     # NaN bit patterns
    a = api.qk_norm_rope_bwd(q, k, gq, gk, 1e-5, dq, dk, pos, rope_theta=1e4, workspace=ws)
    b = api.qk_norm_rope_bwd(q, k, gq, gk, 1e-5, dq, dk, pos, rope_theta=1e4, workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_side_stream_and_graph():
    q, k, gq, gk, pos, dq, dk = (t.cuda() for t in make(100, 8, 2, 128, torch.bfloat16, seed=6))
    want = api.qk_norm_rope_bwd(q, k, gq, gk, 1e-5, dq, dk, pos, rope_theta=1e4)
    want += api.qk_norm_rope_fwd(q, k, gq, gk, 1e-5, pos, rope_theta=1e4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = api.qk_norm_rope_bwd(q, k, gq, gk, 1e-5, dq, dk, pos, rope_theta=1e4)
            got += api.qk_norm_rope_fwd(q, k, gq, gk, 1e-5, pos, rope_theta=1e4)
        for t in got:
            t.zero_()
        graph.replay()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_binding_refusals():
    q, k, gq, gk, pos, dq, dk = (t.cuda() for t in make(4, 2, 1, 128, torch.bfloat16))
    for bad in [(q[:, :, :64], k, gq, gk, pos), (q[:3], k, gq, gk, pos), (q.float(), k, gq, gk, pos),
                (q, k, gq[:64], gk, pos), (q, k, gq, gk, pos.long()), (q, k, gq, gk, pos[:3]),
                (q.transpose(0, 1), k, gq, gk, pos), (q.cpu(), k, gq, gk, pos)]:
        with pytest.raises(ValueError):
            api.qk_norm_rope_fwd(*bad[:4], 1e-5, bad[4], rope_theta=1e4)
    with pytest.raises(ValueError):
        api.qk_norm_rope_bwd(q, k, gq, gk, 1e-5, dq.float(), dk, pos, rope_theta=1e4)

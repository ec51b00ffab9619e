"""The end of a rollout: a parked response costs and changes nothing any more, and a step past the room
that a response has is recorded."""
import pytest
import torch

from shared_prefix_grouped_gb300 import _lib, api, rollout, workloads
from shared_prefix_grouped_gb300.build import build

pytestmark = pytest.mark.gpu
PARKED = -2 ** 30


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()


class Generation:
    def __init__(self, plens, gs, max_new):
        w = workloads.small_layer(heads_q=4, heads_kv=2)
        prob = workloads.make_layer_problem(w, prefix_lens=plens, group_sizes=gs, suffix_lens=[1] * sum(gs),
                                            seed=3)
        self.W = [t.cuda() for t in (prob.w_qkv, prob.w_o, prob.w_gu, prob.w_d, prob.g1, prob.g2)]
        self.kw = dict(rope_theta=w.rope_theta, eps=w.rms_eps)
        self.r = rollout.Rollout(plens, gs, w.heads_q, w.heads_kv, w.head_dim, max_new, page_size=16)
        self.cache = self.r.cache()
        for c in self.cache:
            c.zero_()
        g = torch.Generator(device="cuda").manual_seed(1)
        draw = lambda n: torch.randn((n, w.hidden), generator=g, device="cuda").to(torch.bfloat16)
        rollout.layer_prefill(self.r, self.r.prefix_layout(), draw(sum(plens)), *self.W, *self.cache, **self.kw)
        self.x = [draw(sum(gs)) for _ in range(40)]

    def step(self, t):
        y = rollout.layer_decode(self.r, self.x[t], *self.W, *self.cache, **self.kw)
        self.r.advance()
        return y


def test_parked_response():
    plens, gs = [70, 20], [3, 2]
    a, b = Generation(plens, gs, 32), Generation(plens, gs, 32)
    keep = [0, 2, 3, 4]
    for t in range(24):
        if t == 9:
            b.r.cache_pos[1] = b.r.own_lens[1] = PARKED
            own = b.cache[0][b.r.own_pages[1].long()].clone()
        ya, yb = a.step(t), b.step(t)
        assert torch.equal(ya[keep], yb[keep])
        assert t < 9 or bool(torch.isfinite(yb[1].float()).all())
    assert torch.equal(b.cache[0][b.r.own_pages[1].long()], own)
    assert int(b.r.cache_pos[1]) < 0 and int(b.r.own_lens[1]) < 0
    for s in keep:
        p = a.r.own_pages[s].long()
        assert torch.equal(a.cache[0][p], b.cache[0][p]) and torch.equal(a.cache[1][p], b.cache[1][p])
    assert api.device_status() == _lib.PG_OK


def test_step_past_the_room_is_recorded():
    a = Generation([70, 20], [3, 2], 20)          # two pages of 16: room for 32
    for t in range(32):
        a.step(t)
    assert api.device_status() == _lib.PG_OK
    before = [c.clone() for c in a.cache]
    y = a.step(32)
    assert api.device_status() == _lib.PG_ERR_DEVICE and api.device_status() == _lib.PG_OK
    assert all(torch.equal(c, d) for c, d in zip(a.cache, before))
    assert bool(torch.isfinite(y.float()).all())

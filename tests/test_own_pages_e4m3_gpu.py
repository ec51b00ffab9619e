"""How the attention step over a cache in 8 bits shares its own keys: by their present number and not by the room for
them, and parts with more pages than are read at a time (32).  Tolerances of tests/test_decode_e4m3_gpu.py."""
import pytest
import torch

import test_decode_e4m3_gpu as base
from shared_prefix_grouped_gb300 import api, rollout
from test_decode_e4m3_gpu import built  # noqa: F401  (the build, before anything here)

pytestmark = pytest.mark.gpu


def test_many_responses_with_many_small_pages():
    # as many responses and heads as fill the GPU: parts of up to 1000 keys in pages of 16
    olens = [0, 1, 511, 512, 513, 1000, 1023, 1025, 2000, 2016]
    p = base.problem([40], [180], [olens[i % 10] if i < 170 else 33 * i % 2016 for i in range(180)], 8, 8, 64, 16,
                     torch.bfloat16, seed=1)
    base.check(p, *base.run(p), True)


@pytest.mark.parametrize("d", [64, 128])
def test_few_long_responses_with_small_pages(d):
    # more than 64 pages a part: the pages read ahead move on twice
    p = base.problem([0], [2], [17000, 16391], 2, 1, d, 16, torch.bfloat16, seed=2)
    base.check(p, *base.run(p), True)


LENS = [0, 1, 31, 32, 33, 255, 256, 257, 511, 512, 513, 767, 768, 769, 1023, 1024, 1025, 1500, 4000]


def wide(p, pages):
    """The same problem with room for `pages` pages of own keys (the new ones out of range, as none is read)."""
    more = torch.full((p["op"].shape[0], pages - p["wo"]), -1, dtype=torch.int32)
    return dict(p, op=torch.cat([p["op"], more], 1), wo=pages)


def test_parts_around_their_borders():
    n = len(LENS)
    p = base.problem([300, 0], [171, 9], [LENS[i % n] if i < 3 * n else 29 * i % 300 for i in range(180)], 8, 8, 64, 64,
                     torch.bfloat16, seed=3)
    plan = base.plan_of(p)
    assert plan.struct.own_slots == 1 and plan.struct.own_slots_e4m3 == 4
    o, lse = base.run(p, plan=plan)
    base.check(p, o, lse, True)
    # the room for more changes nothing
    p2 = wide(p, 1024)
    o2, lse2 = base.run(p2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_a_workspace_without_room_for_all_parts():
    p = base.problem([100], [180], [LENS[i % len(LENS)] if i < 60 else 7 for i in range(180)], 8, 8, 64, 64,
                     torch.bfloat16, seed=4)
    plan = base.plan_of(p)
    st = plan.struct
    args = (p["q"].cuda(), *base.caches(p), *[p[n].cuda() for n in ("pp", "op", "olens")])
    for nbytes in (st.workspace_bytes, (st.workspace_bytes + st.workspace_bytes_e4m3) // 2, st.workspace_bytes_e4m3):
        ws = torch.full((nbytes + 64,), 255, dtype=torch.uint8, device="cuda")
        o, lse = api.decode_attn_e4m3(plan, *args, workspace=ws[:nbytes])
        torch.cuda.synchronize()
        base.check(p, o, lse, True)
        assert bool((ws[nbytes:] == 255).all())


def test_a_rollout_allocates_for_the_cache_it_has():
    kw = dict(heads_q=8, heads_kv=8, head_dim=64, max_new=8192, page_size=64)
    a = rollout.Rollout([100], [180], **kw)
    b = rollout.Rollout([100], [180], cache_dtype=torch.float8_e4m3fn, **kw)
    assert a.workspace.numel() == a.plan.struct.workspace_bytes < a.plan.struct.workspace_bytes_e4m3
    assert b.workspace.numel() == b.plan.struct.workspace_bytes_e4m3


def test_time_goes_by_the_present_lengths():
    # 256 responses with 32 keys each: room for 16384 costs little beside room for 1536 (once four times the time)
    def step(room):
        S, hk, d, ps = 256, 8, 128, 64
        plan = api.plan_decode([0], [S], 4 * hk, hk, d, ps, room // ps)
        kv = [api.scaled_cache(S, ps, hk, d) for _ in range(2)]
        for c in kv:
            c.codes.view(torch.uint8).zero_()
        op = torch.arange(S, dtype=torch.int32, device="cuda")[:, None].expand(S, room // ps).contiguous()
        q, lens = torch.randn((S, 4 * hk, d), device="cuda").to(torch.bfloat16), torch.full((S,), 32, device="cuda")
        ws, o = api.decode_workspace(plan), torch.empty_like(q)
        lens = lens.to(torch.int32)
        times = []
        for _ in range(20):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda._sleep(200000)         # the host is ahead of the GPU
            a.record()
            api.decode_attn_e4m3(plan, q, *kv, None, op, lens, out=o, workspace=ws)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 1e3)
        return sorted(times)[5]

    short, long = step(1536), step(16384)
    assert long < 1.5 * short + 5, (short, long)

"""The rollout operators as a program runs them together: the decoder layer with per-head q / k norms
(forward, every gradient) and generation step by step, against the fp64 layer and against the
training forward over the packed [P; R1; ...; RG], normwise 2e-2 as every bf16 layer test (each path
rounds its activations to bf16 some ten times, 2^-8 each)."""
import pytest
import torch

from oracle import prefix_grouper_oracle as orc
from oracle import rollout_oracle as ro
from shared_prefix_grouped_gb300 import api, layer, rollout, workloads
from shared_prefix_grouped_gb300.build import build

pytestmark = pytest.mark.gpu
TOL = 2e-2


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()


def problem(plens, gs, rs, seed=0, gains=True, **kw):
    w = workloads.small_layer(heads_q=4, heads_kv=2, **kw)
    prob = workloads.make_layer_problem(w, prefix_lens=plens, group_sizes=gs, suffix_lens=rs, seed=seed)
    g = torch.Generator().manual_seed(seed + 77)
    gq, gk = ((1 + 0.3 * torch.randn(w.head_dim, generator=g)).to(torch.bfloat16) for _ in range(2))
    W = (prob.w_qkv, prob.w_o, prob.w_gu, prob.w_d, prob.g1, prob.g2)
    return w, prob, W, (gq, gk) if gains else (None, None)


def dims(w):
    return dict(heads_q=w.heads_q, heads_kv=w.heads_kv, head_dim=w.head_dim)


@pytest.mark.parametrize("fused_rope", [True, False], ids=["rope_with_norm", "rope_in_attn"])
def test_layer_with_qk_norms_matches_autograd(fused_rope):
    plens, gs, rs = [150, 40], [3, 2], [70, 1, 129, 30, 64]
    w, prob, W, (gq, gk) = problem(plens, gs, rs)
    lay = orc.pack_layout(plens, gs, rs)
    leaves = [t.double().requires_grad_() for t in (prob.x, *W, gq, gk)]
    ref = ro.layer(leaves[0], orc.visibility_mask(lay), lay.position_ids, leaves[1:7], **dims(w),
                   theta=w.rope_theta, eps=w.rms_eps, g_q=leaves[7], g_k=leaves[8])
    ref.backward(prob.dy.double())
    dev = torch.device("cuda")
    L = api.pack(plens, gs, rs, dev)
    Wd, x, dy, gqd, gkd = [t.cuda() for t in W], prob.x.cuda(), prob.dy.cuda(), gq.cuda(), gk.cuda()
    kw = dict(**dims(w), rope_theta=w.rope_theta, eps=w.rms_eps, g_q=gqd, g_k=gkd)
    y, saved = layer.layer_fwd(L, x, *Wd, fused_rope=fused_rope, **kw)
    g = layer.layer_bwd(L, x, *Wd, saved, dy, **kw)
    torch.cuda.synchronize()
    assert api.device_status() == 0
    got = (g.dx, g.w_qkv, g.w_o, g.w_gu, g.w_d, g.g1, g.g2, g.g_q, g.g_k)
    errs = {"y": orc.normwise_error(y.float().cpu(), ref.detach())}
    for n, a, b in zip(("dx", "qkv", "o", "gu", "d", "g1", "g2", "g_q", "g_k"), got, leaves):
        errs[n] = orc.normwise_error(a.float().cpu(), b.grad)
    assert all(e <= TOL for e in errs.values()), errs


def generate(w, prob, W, gains, plens, gs, rs, graph):
    """The responses' rows of y, token by token, with the rows of x as the tokens' inputs."""
    steps, S = max(rs), sum(gs)
    r = rollout.Rollout(plens, gs, w.heads_q, w.heads_kv, w.head_dim, steps, page_size=16)
    Wd, x = [t.cuda() for t in W], prob.x.cuda()
    gq, gk = (None if t is None else t.cuda() for t in gains)
    kc, vc = r.cache()
    kc.fill_(float("nan"))
    vc.fill_(float("nan"))
    kw = dict(rope_theta=w.rope_theta, eps=w.rms_eps, g_q=gq, g_k=gk)
    pre, res, t0 = [], [], 0
    for lp, G in zip(plens, gs):
        pre += range(t0, t0 + lp)
        t0 += lp
        for i in range(G):
            n = rs[len(res)]
            res.append(range(t0, t0 + n))
            t0 += n
    lay = r.prefix_layout()
    y_pre = rollout.layer_prefill(r, lay, x[pre].contiguous(), *Wd, kc, vc, **kw)
    xin = torch.zeros((S, w.hidden), dtype=torch.bfloat16, device="cuda")
    state = [t.clone() for t in (r.cache_pos, r.own_lens, r.positions)]
    if graph:
        rollout.layer_decode(r, xin, *Wd, kc, vc, **kw)     # warm-up; its key is written again below
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = rollout.layer_decode(r, xin, *Wd, kc, vc, **kw)
            r.advance()
        for t, v in zip((r.cache_pos, r.own_lens, r.positions), state):
            t.copy_(v)
    out = torch.full((x.shape[0], w.hidden), float("nan"), device="cuda")
    out[pre] = y_pre.float()
    for t in range(steps):
        # a response that has ended goes on with zeros, which nobody reads
        xin.copy_(torch.stack([x[s[t]] if t < len(s) else torch.zeros_like(x[0]) for s in res]))
        if graph:
            g.replay()
        else:
            y = rollout.layer_decode(r, xin, *Wd, kc, vc, **kw)
            r.advance()
        for i, s in enumerate(res):
            if t < len(s):
                out[s[t]] = y[i].float()
    torch.cuda.synchronize()
    assert api.device_status() == 0
    return out.cpu()


@pytest.mark.parametrize("gains", [True, False], ids=["qk_norm", "plain"])
@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_generation_equals_the_training_forward(gains, graph):
    plens, gs, rs = [150, 33], [3, 2], [20, 1, 37, 18, 33]
    w, prob, W, gn = problem(plens, gs, rs, seed=5, gains=gains)
    got = generate(w, prob, W, gn, plens, gs, rs, graph)
    lay = orc.pack_layout(plens, gs, rs)
    ref = ro.layer(prob.x.double(), orc.visibility_mask(lay), lay.position_ids,
                   [t.double() for t in W], **dims(w), theta=w.rope_theta, eps=w.rms_eps,
                   g_q=None if gn[0] is None else gn[0].double(),
                   g_k=None if gn[1] is None else gn[1].double())
    assert orc.normwise_error(got, ref) <= TOL
    dev = torch.device("cuda")
    y, _ = layer.layer_fwd(api.pack(plens, gs, rs, dev), prob.x.cuda(), *[t.cuda() for t in W], **dims(w),
                           rope_theta=w.rope_theta, eps=w.rms_eps,
                           g_q=None if gn[0] is None else gn[0].cuda(),
                           g_k=None if gn[1] is None else gn[1].cuda())
    assert orc.normwise_error(got, y.float().cpu().double()) <= TOL


def test_two_layers_a_head_and_sampled_tokens():
    # Tokens generated through two layers, an embedding and a head: every sampled token is the one that
    # the definition gives for the logits of its step, and its log-probability is the head's.
    plens, gs, steps, V = [90, 20], [2, 3], 12, 517
    w, prob, W, (gq, gk) = problem(plens, gs, [1] * 5, seed=9)
    g = torch.Generator(device="cuda").manual_seed(3)
    emb = torch.randn((V, w.hidden), generator=g, device="cuda").to(torch.bfloat16)
    head = (0.2 * torch.randn((V, w.hidden), generator=g, device="cuda")).to(torch.bfloat16)
    Wd, gains = [t.cuda() for t in W], dict(g_q=gq.cuda(), g_k=gk.cuda())
    kw = dict(rope_theta=w.rope_theta, eps=w.rms_eps, **gains)
    r = rollout.Rollout(plens, gs, w.heads_q, w.heads_kv, w.head_dim, steps, page_size=16)
    caches = [r.cache(), r.cache()]
    lay = r.prefix_layout()
    x = emb[torch.randint(0, V, (sum(plens),), generator=g, device="cuda")]
    for c in caches:
        x = rollout.layer_prefill(r, lay, x, *Wd, *c, **kw)
    tok = torch.randint(0, V, (5,), generator=g, device="cuda", dtype=torch.int32)
    temp, top_p = torch.full((5,), 0.8, device="cuda"), torch.full((5,), 0.9, device="cuda")
    top_k = torch.full((5,), 40, dtype=torch.int32, device="cuda")
    seen = []
    for _ in range(steps):
        x = emb[tok.long()]
        for c in caches:
            x = rollout.layer_decode(r, x, *Wd, *c, **kw)
        h, _, _ = api.rmsnorm_fwd(x, Wd[5], w.rms_eps)
        logits = api.gemm_bf16(h, head)
        u = torch.rand(5, generator=g, device="cuda")
        tok, lp = api.sample(logits, u, temperature=temp, top_k=top_k, top_p=top_p)
        r.advance()
        wt, wl = ro.sample(logits.cpu(), u.cpu(), temp.cpu(), top_k.cpu(), top_p.cpu())
        assert torch.equal(tok.cpu(), wt)
        assert bool(((lp.cpu().double() - wl).abs() <= 2.0 ** -24 * wl.abs() + 4e-9).all())
        seen.append(tok.cpu())
    assert torch.stack(seen).unique().numel() > 10 and api.device_status() == 0

"""The rollout over a cache in 8 bits and the policy loss on what it generated, as a program runs them
together.

A key or value element is rounded to e4m3 by at most 2^-4 of itself, 2^-4 / sqrt 3 = 0.036 in the root mean
square.  Keys: a score is off by scale |q| 0.036 rms(k), which for the normalised queries and keys of these layers
is about 0.04, so a weight is off by 4 % of itself at random; values: 3.6 %.  Attention averages both over
the keys as it does the values themselves, so its output is off by sqrt(0.036^2 + 0.04^2) = 0.054 < 2^-4 normwise,
the layer's (a sum of its input, attention and the rest) by less.  With the 2e-2 that every bf16 layer test
has: 2e-2 + 2^-4."""
import pytest
import torch

from oracle import policy_oracle as po
from oracle import prefix_grouper_oracle as orc
from oracle import rollout_oracle as ro
from shared_prefix_grouped_gb300 import _lib, api, layer, rollout, workloads
from shared_prefix_grouped_gb300.build import build

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
TOL = 2e-2
PARKED = -2 ** 30


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()


def problem(plens, gs, rs, seed=0, gains=True):
    w = workloads.small_layer(heads_q=4, heads_kv=2)
    prob = workloads.make_layer_problem(w, prefix_lens=plens, group_sizes=gs, suffix_lens=rs, seed=seed)
    g = torch.Generator().manual_seed(seed + 77)
    gq, gk = ((1 + 0.3 * torch.randn(w.head_dim, generator=g)).to(BF16) for _ in range(2))
    W = (prob.w_qkv, prob.w_o, prob.w_gu, prob.w_d, prob.g1, prob.g2)
    return w, prob, W, (gq, gk) if gains else (None, None)


def fill(cache, byte):
    for c in cache:
        c.codes.view(torch.uint8).fill_(byte)


def packed_rows(plens, gs, rs):
    """(rows of the prefixes, rows of each response) of the packed layout."""
    pre, res, t0 = [], [], 0
    for lp, G in zip(plens, gs):
        pre += range(t0, t0 + lp)
        t0 += lp
        for _ in range(G):
            n = rs[len(res)]
            res.append(range(t0, t0 + n))
            t0 += n
    return pre, res


def test_the_cache_is_the_one_asked_for():
    for kw, dt in ((dict(), BF16), (dict(cache_dtype=BF16), BF16)):
        r = rollout.Rollout([20], [2], 4, 2, 64, 8, page_size=16, **kw)
        assert [c.dtype for c in r.cache()] == [dt, dt]
    r = rollout.Rollout([20], [2], 4, 2, 64, 8, page_size=16, cache_dtype=E4M3)
    k, v = r.cache()
    assert k.codes.dtype is E4M3 and k.codes.shape == (r.num_pages, 16, 2, 64)
    assert k.scales.shape == (r.num_pages, 1, 2) and k.codes.data_ptr() != v.codes.data_ptr()


@pytest.mark.parametrize("gains", [True, False], ids=["qk_norm", "plain"])
@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_generation_is_near_the_training_forward(gains, graph):
    plens, gs, rs = [150, 33], [3, 2], [20, 1, 37, 18, 33]
    w, prob, W, (gq, gk) = problem(plens, gs, rs, seed=5, gains=gains)
    steps, S = max(rs), sum(gs)
    r = rollout.Rollout(plens, gs, w.heads_q, w.heads_kv, w.head_dim, steps, page_size=16, cache_dtype=E4M3)
    Wd, x = [t.cuda() for t in W], prob.x.cuda()
    kw = dict(rope_theta=w.rope_theta, eps=w.rms_eps, g_q=None if gq is None else gq.cuda(),
              g_k=None if gk is None else gk.cuda())
    kc, vc = r.cache()
    fill((kc, vc), 0x7f)                                    # NaN
    pre, res = packed_rows(plens, gs, rs)
    out = torch.full((x.shape[0], w.hidden), float("nan"), device="cuda")
    out[pre] = rollout.layer_prefill(r, r.prefix_layout(), x[pre].contiguous(), *Wd, kc, vc, **kw).float()
    xin = torch.zeros((S, w.hidden), dtype=BF16, device="cuda")
    counters = (r.cache_pos, r.own_lens, r.positions)
    if graph:
        state = [t.clone() for t in counters]
        rollout.layer_decode(r, xin, *Wd, kc, vc, **kw)     # warm-up; its key is written again below
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = rollout.layer_decode(r, xin, *Wd, kc, vc, **kw)
            r.advance()
        for t, s in zip(counters, state):
            t.copy_(s)
    for t in range(steps):
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
    lay = orc.pack_layout(plens, gs, rs)
    ref = ro.layer(prob.x.double(), orc.visibility_mask(lay), lay.position_ids, [t.double() for t in W],
                   heads_q=w.heads_q, heads_kv=w.heads_kv, head_dim=w.head_dim, theta=w.rope_theta, eps=w.rms_eps,
                   g_q=None if gq is None else gq.double(), g_k=None if gk is None else gk.double())
    assert orc.normwise_error(out.cpu(), ref) <= TOL + 2.0 ** -4


def test_a_parked_response():
    plens, gs, keep = [70, 20], [3, 2], [0, 2, 3, 4]
    w, prob, W, _ = problem(plens, gs, [1] * 5, seed=3, gains=False)
    Wd, kw = [t.cuda() for t in W], dict(rope_theta=w.rope_theta, eps=w.rms_eps)
    g = torch.Generator(device="cuda").manual_seed(1)
    x_pre, *xs = (torch.randn((n, w.hidden), generator=g, device="cuda").to(BF16) for n in [90] + [5] * 24)
    r = [rollout.Rollout(plens, gs, 4, 2, w.head_dim, 32, page_size=16, cache_dtype=E4M3) for _ in range(2)]
    caches = [x.cache() for x in r]
    for a, c in zip(r, caches):
        fill(c, 0)
        rollout.layer_prefill(a, a.prefix_layout(), x_pre, *Wd, *c, **kw)
    own = r[1].own_pages[1].long()
    for t, x in enumerate(xs):
        if t == 9:
            r[1].cache_pos[1] = r[1].own_lens[1] = PARKED
            held = [u[own].clone().view(torch.uint8) for c in caches[1] for u in c]
        ya, yb = (rollout.layer_decode(a, x, *Wd, *c, **kw) for a, c in zip(r, caches))
        for a in r:
            a.advance()
        assert torch.equal(ya[keep], yb[keep]) and bool(torch.isfinite(yb[1].float()).all())
    assert all(torch.equal(u[own].view(torch.uint8), h) for u, h in
               zip([u for c in caches[1] for u in c], held))
    assert api.device_status() == _lib.PG_OK


def test_step_past_the_room_is_recorded():
    r = rollout.Rollout([20], [2], 4, 2, 64, 10, page_size=16, cache_dtype=E4M3)     # room for 16
    kc, vc = r.cache()
    fill((kc, vc), 0)
    k = torch.randn((2, 2, 64), device="cuda").to(BF16)
    for t in range(16):
        r.append(k, k, kc, vc, r.own_pages, r.cache_pos)
        r.advance()
    assert api.device_status() == _lib.PG_OK
    before = [t.clone().view(torch.uint8) for c in (kc, vc) for t in c]
    r.append(k, k, kc, vc, r.own_pages, r.cache_pos)
    assert api.device_status() == _lib.PG_ERR_DEVICE and api.device_status() == _lib.PG_OK
    assert all(torch.equal(t.view(torch.uint8), b) for t, b in zip((t for c in (kc, vc) for t in c), before))


@pytest.mark.parametrize("dtype", [BF16, torch.float32], ids=["bf16", "f32"])
def test_generate_sample_and_learn(dtype):
    # Responses are sampled through two layers over 8-bit caches, the first token of each from its group's
    # prefix; the packed [P; R1; ...; RG] then gives logits, the loss and the gradient of the head and of what
    # it reads, against the fp64 gradient from the same logits.  The vocabulary is padded to the 8 that the
    # products take: its rows of the head are zero, and so is what the loss leaves of the gradient's columns.
    plens, gs, rs, V, VP, T = [90, 20], [2, 3], [12, 5, 1, 9, 12], 517, 520, 0.8
    w, prob, W, (gq, gk) = problem(plens, gs, rs, seed=9)
    g = torch.Generator(device="cuda").manual_seed(3)
    emb = torch.randn((V, w.hidden), generator=g, device="cuda").to(BF16)
    head = (0.1 * torch.randn((VP, w.hidden), generator=g, device="cuda")).to(BF16)
    head[V:] = 0
    Wd, dims = [t.cuda() for t in W], dict(heads_q=w.heads_q, heads_kv=w.heads_kv, head_dim=w.head_dim)
    kw = dict(rope_theta=w.rope_theta, eps=w.rms_eps, g_q=gq.cuda(), g_k=gk.cuda())
    S, pre_rows = sum(gs), packed_rows(plens, gs, rs)
    temp = torch.full((S,), T, device="cuda")

    def logits_of(x):
        h, _, _ = api.rmsnorm_fwd(x, Wd[5], w.rms_eps)
        return h, api.gemm_bf16(h, head, out_dtype=dtype)[:, :V]

    r = rollout.Rollout(plens, gs, w.heads_q, w.heads_kv, w.head_dim, max(rs), page_size=16, cache_dtype=E4M3)
    caches = [r.cache(), r.cache()]
    prompt = torch.randint(0, V, (sum(plens),), generator=g, device="cuda")
    x = emb[prompt]
    for c in caches:
        x = rollout.layer_prefill(r, r.prefix_layout(), x, *Wd, *c, **kw)
    ends = torch.tensor(plens).cumsum(0) - 1
    _, first = logits_of(x)
    logits = first[torch.repeat_interleave(ends, torch.tensor(gs)).cuda()]
    toks, lps = [], []
    for t in range(max(rs)):
        tok, lp = api.sample(logits, torch.rand(S, generator=g, device="cuda"), temperature=temp)
        toks.append(tok.clone())
        lps.append(lp.clone())
        x = emb[tok.long()]
        for c in caches:
            x = rollout.layer_decode(r, x, *Wd, *c, **kw)
        r.advance()
        _, logits = logits_of(x)
    torch.cuda.synchronize()
    assert api.device_status() == 0

    toks, lps = torch.stack(toks).cpu(), torch.stack(lps).cpu()
    lay = orc.pack_layout(plens, gs, rs)
    pre, res = pre_rows
    packed, old = torch.zeros(lay.total_tokens, dtype=torch.int32), torch.zeros(lay.total_tokens)
    packed[pre] = prompt.cpu().int()
    for s, rows in enumerate(res):
        packed[list(rows)], old[list(rows)] = toks[:len(rows), s], lps[:len(rows), s]
    adv = torch.randn(S, generator=torch.Generator().manual_seed(1))
    A = torch.zeros(lay.total_tokens)
    for s, rows in enumerate(res):
        A[list(rows)] = adv[s]
    starts, index = api.policy_rows(plens, gs, rs)
    assert index.numel() == sum(rs)                       # every generated token, from the first on
    at = index.cpu()
    L = api.pack(plens, gs, rs, torch.device("cuda"))
    x = emb[packed.cuda().long()]
    for _ in caches:
        x, _ = layer.layer_fwd(L, x, *Wd, **dims, **kw)
    h, logits = logits_of(x)
    tokens, weights = packed[at], torch.full((len(at),), 1.0 / len(at))
    args = dict(advantages=A[at].cuda(), old_logprobs=old[at].cuda(), ref_logprobs=(old[at] - 0.1).cuda(),
                weights=weights.cuda(), row_starts=starts, clip_low=0.4, clip_high=0.5, kl_coef=0.05, temperature=T)
    whole = torch.zeros((lay.total_tokens, VP), dtype=dtype, device="cuda")
    out = api.policy_loss(logits, tokens.cuda(), dlogits=whole[:, :V], **args)
    two = api.policy_loss(logits, tokens.cuda(), **args)
    back = api.policy_loss_bwd(logits, tokens.cuda(), two.lse, two.token_grad, row_starts=starts, temperature=T)
    dz = whole.to(BF16)
    dh = api.gemm_bf16(dz, head, b_mn=True, out_dtype=BF16)
    dhead = api.gemm_bf16(dz, h, a_mn=True, b_mn=True)
    torch.cuda.synchronize()
    assert api.device_status() == 0

    want = po.loss(logits.cpu(), tokens, advantages=A[at], old=old[at], ref=old[at] - 0.1, weights=weights,
                   row_starts=starts.cpu(), clip_low=0.4, clip_high=0.5, kl_coef=0.05, temperature=T)
    # A log-probability is off by a few hundred 2^-24 (below 1e-4), and its loss by that times the derivative.
    assert abs(float(out.loss) - want[0]) <= 1e-4 * float(want[2].abs().sum() + want[3].abs().sum())
    # The gradient's own error is a thousandth; bf16 adds 2^-8 of an element, the products 2^-8 again.
    d = want[5]
    hf, headf = h.cpu().double(), head[:V].cpu().double()
    for name, got, ref in (("dlogits", out.dlogits, d), ("bwd", back, d), ("dh", dh, d @ headf),
                           ("dhead", dhead[:V], d.t() @ hf)):
        assert orc.normwise_error(got.float().cpu(), ref) <= 2.0 ** -6, name
    assert float(whole[:, V:].abs().max()) == 0.0
    # rows that predict nothing: the prefixes but for their last, each response's last
    empty = (starts[1:] == starts[:-1]).cpu()
    assert int((~empty).sum()) == sum(n - 1 for n in rs) + len(plens)
    assert float(out.dlogits[empty.cuda()].abs().max()) == 0.0
    assert torch.equal(two.loss, out.loss) and torch.equal(two.logprobs, out.logprobs)

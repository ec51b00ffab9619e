"""Measured cases of the operators around a rollout of shared-prefix groups: the per-head query / key
norm with the position rotation (forward and backward), the append to a paged K/V cache with the
rotation on the way, the attention of one new token per response over the shared prefix and its own
pages, and the sampling of the next token from given random numbers.

``own`` False: plain torch operations, in 32 bits (64 for angles and for the sampling weights, whose
borders decide a whole number).  ``own`` True: the calls a program makes of the framework.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
THETA = 5e5


# ------------------------------------------------------------------------------------- the cases --

def listed():
    return [
        # --- query / key norm with rotation ---
        # One decode step of a small batch: a launch whose latency counts.
        dict(name="qk_norm_fwd_t16", op="qk_norm", direction="fwd", dtype="bf16", tokens=16,
             heads_q=32, heads_kv=8, head_dim=128, padded_rows=True),
        # The decoder-layer training step's forward: 2 groups of 8192 + 8 x 1024 tokens.
        dict(name="qk_norm_fwd_t32768", op="qk_norm", direction="fwd", dtype="bf16", tokens=32768,
             heads_q=32, heads_kv=8, head_dim=128, padded_rows=False),
        # The backward of a training step over one long-prefix group (odd token count).
        dict(name="qk_norm_bwd_t26601", op="qk_norm", direction="bwd", dtype="bf16", tokens=26601,
             heads_q=32, heads_kv=8, head_dim=128, padded_rows=False),
        # --- append to the paged cache ---
        # One step of 16 responses: one token each, q rotated in the same call, strided projections.
        dict(name="append_step_s16", op="append", dtype="bf16", seqs=16, tokens_per_seq=1,
             heads_q=32, heads_kv=8, head_dim=128, page_size=64, base_len=700, fused_qkv=True,
             capacity=1024),
        # Eight prompts of 2048 tokens written after their prefill, pages of 32.
        dict(name="append_prefill_b8_p2048", op="append", dtype="bf16", seqs=8, tokens_per_seq=2048,
             heads_q=0, heads_kv=8, head_dim=128, page_size=32, base_len=0, fused_qkv=False,
             capacity=2560),
        # --- attention of one new token per response ---
        # A few short responses at the start of a rollout, exact fp32, 64-wide heads.
        dict(name="decode_f32_g4_p256", op="decode", dtype="f32", groups=1, group_size=4,
             prefix_lo=256, prefix_hi=256, own_lo=1, own_hi=48, heads_q=2, heads_kv=2, head_dim=64,
             page_size=16, own_pages=8),
        # 16 responses of a 16384-token prefix, up to 1024 tokens into their answers.
        dict(name="decode_g16_p16384", op="decode", dtype="bf16", groups=1, group_size=16,
             prefix_lo=16384, prefix_hi=16384, own_lo=256, own_hi=1024, heads_q=32, heads_kv=8,
             head_dim=128, page_size=64, own_pages=16),
        # Eight ragged groups of 16: many medium prefixes, every response at its own length.
        dict(name="decode_b8_g16_p2048", op="decode", dtype="bf16", groups=8, group_size=16,
             prefix_lo=1601, prefix_hi=2495, own_lo=0, own_hi=512, heads_q=32, heads_kv=8,
             head_dim=128, page_size=32, own_pages=20),
        # 64 responses for each of four 32768-token contexts: several row blocks read one prefix.
        dict(name="decode_b4_g64_p32768", op="decode", dtype="bf16", groups=4, group_size=64,
             prefix_lo=32768, prefix_hi=32768, own_lo=1, own_hi=1537, heads_q=32, heads_kv=8,
             head_dim=128, page_size=128, own_pages=16),
        # --- sampling ---
        # 16 responses of one group, temperature only.
        dict(name="sample_s16_v32000", op="sample", dtype="f32", rows=16, vocab=32000, row_pad=0,
             filters="temperature", masked=0.0),
        # 64 rows of a padded, odd vocabulary in bf16 (many equal logits), nucleus sampling with a
        # tenth of the tokens ruled out.
        dict(name="sample_s64_v50001_bf16", op="sample", dtype="bf16", rows=64, vocab=50001,
             row_pad=47, filters="top_p", masked=0.1),
        # 256 rows of a large vocabulary, every filter, other settings in every row.
        dict(name="sample_s256_v131072", op="sample", dtype="f32", rows=256, vocab=131072, row_pad=0,
             filters="all", masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_norm", "append", "decode", "decode", "sample", "sample"])
    hkv = rng.choice([1, 2, 4, 8])
    hp = rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "qk_norm":
        hq = min(hp * hkv, 32)
        return dict(op=op, direction=rng.choice(["fwd", "bwd"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    tokens=_log_int(rng, 1, 16384), heads_q=hq, heads_kv=hkv,
                    head_dim=rng.choice([64, 128]), padded_rows=rng.random() < 0.5)
    if op == "append":
        step = rng.random() < 0.5
        base = _log_int(rng, 1, 2000) if step else rng.choice([0, 0, _log_int(rng, 1, 500)])
        per = 1 if step else _log_int(rng, 2, 1600)
        page = rng.choice([16, 32, 64, 128, 256])
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    seqs=_log_int(rng, 1, 128) if step else rng.randint(1, 6), tokens_per_seq=per,
                    heads_q=rng.choice([0, min(hp * hkv, 32)]), heads_kv=hkv,
                    head_dim=rng.choice([64, 128]), page_size=page, base_len=base,
                    fused_qkv=rng.random() < 0.5, capacity=base + per + rng.randint(0, 300))
    if op == "decode":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        groups = rng.randint(1, 5)
        plo = rng.choice([0, 1, _log_int(rng, 1, 4000), _log_int(rng, 100, 16000)])
        phi = min(plo + rng.choice([0, rng.randint(0, 900)]), 16384)
        page = rng.choice([16, 32, 64, 128, 256])
        olo = rng.choice([0, 1, rng.randint(0, 300)])
        ohi = olo + _log_int(rng, 1, 900)
        if dtype == "f32":
            plo, phi, olo, ohi = plo // 8, phi // 8, olo // 4, max(ohi // 4, olo // 4)
        ohi = max(ohi, 1)
        return dict(op=op, dtype=dtype, groups=groups, group_size=_log_int(rng, 1, 33),
                    prefix_lo=plo, prefix_hi=phi, own_lo=olo, own_hi=ohi,
                    heads_q=min(hp, 32 // hkv) * hkv, heads_kv=hkv,
                    head_dim=rng.choice([64, 128, 128]), page_size=page,
                    own_pages=(ohi + page - 1) // page + rng.randint(0, 2))
    dtype = rng.choice(["f32", "bf16"])
    vocab = _log_int(rng, 2, 131072)
    return dict(op=op, dtype=dtype, rows=_log_int(rng, 1, 200), vocab=vocab,
                row_pad=rng.choice([0, 0, rng.randint(1, 63)]),
                filters=rng.choice(["temperature", "top_k", "top_p", "min_p", "all"]),
                masked=rng.choice([0.0, 0.0, 0.1, 0.5]))


# ----------------------------------------------------------------------------------------- inputs --

def _spaced(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]."""
    return [lo + (i * (hi - lo)) // max(n - 1, 1) for i in range(n)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _prefix_lens(case):
    return _spaced(case["prefix_lo"], case["prefix_hi"], case["groups"])


def _own_lens(case):
    return _spaced(case["own_lo"], case["own_hi"], case["groups"] * case["group_size"])


def _inputs(case, seed):
    """The tensors a program holds before the call, from the seed alone."""
    g = _gen(seed)
    dev = "cuda"
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)

    if case["op"] == "qk_norm":
        T, hq, hk, d = case["tokens"], case["heads_q"], case["heads_kv"], case["head_dim"]
        if case["padded_rows"]:     # views of one fused projection's rows [q | k | v]
            x = normal(T, hq + 2 * hk, d, scale=1.5)
            q, k = x[:, :hq], x[:, hq:hq + hk]
        else:
            q, k = normal(T, hq, d, scale=1.5), normal(T, hk, d, scale=0.5)
        s = dict(q=q, k=k, gain_q=(1 + normal(d, scale=0.2, dtype=torch.float32)).to(dt),
                 gain_k=(1 + normal(d, scale=0.2, dtype=torch.float32)).to(dt),
                 positions=torch.randint(0, 40000, (T,), generator=g, device=dev, dtype=torch.int32))
        if case["direction"] == "bwd":
            s["dq_out"], s["dk_out"] = normal(T, hq, d), normal(T, hk, d)
        return s
    if case["op"] == "append":
        S, n, hq, hk, d = (case[x] for x in ("seqs", "tokens_per_seq", "heads_q", "heads_kv",
                                             "head_dim"))
        ps, N = case["page_size"], case["seqs"] * case["tokens_per_seq"]
        per_seq = (case["capacity"] + ps - 1) // ps
        total = S * per_seq + 3
        if case["fused_qkv"]:
            x = normal(N, hq + 2 * hk, d)
            q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        else:
            q, k, v = normal(N, hq, d), normal(N, hk, d), normal(N, hk, d)
        pages = torch.randperm(total, generator=g, device=dev)[:S * per_seq]
        idx = torch.arange(N, device=dev, dtype=torch.int32)
        cache_pos = case["base_len"] + idx % n
        return dict(q=q if hq else None, k=k, v=v, k_cache=normal(total, ps, hk, d),
                    v_cache=normal(total, ps, hk, d),
                    pages=pages.view(S, per_seq).to(torch.int32).contiguous(),
                    page_rows=(idx // n).to(torch.int32), cache_pos=cache_pos.to(torch.int32),
                    # the tokens sit behind a shared prefix that has pages of its own
                    positions=(cache_pos + 5000).to(torch.int32))
    if case["op"] == "decode":
        B, G, hq, hk, d, ps = (case[x] for x in ("groups", "group_size", "heads_q", "heads_kv",
                                                 "head_dim", "page_size"))
        S = B * G
        plens, olens = _prefix_lens(case), torch.tensor(_own_lens(case), dtype=torch.int32)
        olens = olens.to(dev)[torch.randperm(S, generator=g, device=dev)]
        per_prefix, per_own = max((max(plens) + ps - 1) // ps, 1), case["own_pages"]
        total = B * per_prefix + S * per_own
        perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        return dict(q=normal(S, hq, d), k_cache=normal(total, ps, hk, d),
                    v_cache=normal(total, ps, hk, d), prefix_lens=plens, group_sizes=[G] * B,
                    prefix_pages=perm[:B * per_prefix].view(B, per_prefix).contiguous(),
                    own_pages=perm[B * per_prefix:].view(S, per_own).contiguous(), own_lens=olens)
    S, V = case["rows"], case["vocab"]
    x = torch.randn((S, V + case["row_pad"]), generator=g, device=dev) * 2.5
    # a language model's head: a few tokens stand out of the bulk
    out = torch.rand(x.shape, generator=g, device=dev) < 24.0 / V
    x += out * (6 + 3 * torch.rand(x.shape, generator=g, device=dev))
    if case["masked"] > 0:
        x[torch.rand(x.shape, generator=g, device=dev) < case["masked"]] = float("-inf")
        x[:, 0] = 0.0      # the token that ends a text is always allowed
    f = case["filters"]

    def uniform(lo, hi):
        return lo + (hi - lo) * torch.rand(S, generator=g, device=dev)

    s = dict(logits=x.to(dt)[:, :V], u=torch.rand(S, generator=g, device=dev),
             temperature=uniform(0.6, 1.2), top_k=None, top_p=None, min_p=None)
    if f in ("top_k", "all"):
        s["top_k"] = torch.randint(1, 200, (S,), generator=g, device=dev, dtype=torch.int32)
    if f in ("top_p", "all"):
        s["top_p"] = uniform(0.5, 0.99)
    if f in ("min_p", "all"):
        s["min_p"] = uniform(0.0, 0.1)
    if f == "all":
        # every fourth row without top-k, every fifth without a nucleus, a few greedy
        row = torch.arange(S, device=dev)
        s["top_k"][row % 4 == 1] = 0
        s["top_p"][row % 5 == 2] = 1.0
        s["temperature"][row % 16 == 7] = 0.0
    return s


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if own and case["op"] == "decode":
        from shared_prefix_grouped_gb300 import api
        # Kept for a whole rollout: the plan and its workspace.
        state["plan"] = api.plan_decode(state["prefix_lens"], state["group_sizes"], case["heads_q"],
                                        case["heads_kv"], case["head_dim"], case["page_size"],
                                        case["own_pages"], DTYPES[case["dtype"]], device="cuda")
        state["workspace"] = api.decode_workspace(state["plan"])
    return state


# --------------------------------------------------------------------------------- the plain forms --

def _cos_sin(positions, d):
    k = torch.arange(d // 2, device=positions.device, dtype=torch.float64)
    a = positions.double()[:, None] * THETA ** (-2.0 * k / d)
    return a.cos().float()[:, None, :], a.sin().float()[:, None, :]


def _rotate(x, c, s):
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return torch.cat([a * c - b * s, b * c + a * s], dim=-1)


def _plain_qk_norm(st):
    c, s = _cos_sin(st["positions"], st["q"].shape[-1])
    outs, gains = [], []
    for name in ("q", "k"):
        x, g = st[name].float(), st["gain_" + name].float()
        r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        if st["case"]["direction"] == "fwd":
            outs.append(_rotate(x * r * g, c, s).to(st[name].dtype))
            continue
        dy = _rotate(st["d" + name + "_out"].float(), c, -s)
        xhat = x * r
        dx = r * (g * dy - xhat * (xhat * g * dy).mean(-1, keepdim=True))
        outs.append(dx.to(st[name].dtype))
        gains.append((dy * xhat).double().sum((0, 1)).float())
    return tuple(outs + gains)


def _plain_append(st):
    c, s = _cos_sin(st["positions"], st["k"].shape[-1])
    ps = st["k_cache"].shape[1]
    cp = st["cache_pos"].long()
    page = st["pages"][st["page_rows"].long(), cp // ps].long()
    st["k_cache"][page, cp % ps] = _rotate(st["k"].float(), c, s).to(st["k_cache"].dtype)
    st["v_cache"][page, cp % ps] = st["v"]
    out = [st["k_cache"], st["v_cache"]]
    if st["q"] is not None:
        out.append(_rotate(st["q"].float(), c, s).to(st["q"].dtype))
    return tuple(out)


def _plain_decode(st):
    q, kc, vc = st["q"].float(), st["k_cache"], st["v_cache"]
    S, hq, d = q.shape
    ps, hk = kc.shape[1], kc.shape[2]
    hp, scale = hq // hk, d ** -0.5
    o, lse = torch.empty_like(q), torch.empty((hq, S), device=q.device)
    s0 = 0
    for b, G in enumerate(st["group_sizes"]):
        n = st["prefix_lens"][b]
        used = (n + ps - 1) // ps
        pp = st["prefix_pages"][b, :used].long()
        kp = kc[pp].reshape(-1, hk, d)[:n].float()              # [n, hk, d]
        vp = vc[pp].reshape(-1, hk, d)[:n].float()
        op = st["own_pages"][s0:s0 + G].long()
        ko = kc[op].reshape(G, -1, hk, d).float()               # [G, L, hk, d]
        vo = vc[op].reshape(G, -1, hk, d).float()
        ol = st["own_lens"][s0:s0 + G]
        qg = q[s0:s0 + G].view(G, hk, hp, d)
        sp = torch.matmul(qg.permute(1, 0, 2, 3).reshape(hk, G * hp, d), kp.permute(1, 2, 0))
        sp = sp.view(hk, G, hp, n).transpose(0, 1) * scale      # [G, hk, hp, n]
        so = torch.matmul(qg, ko.permute(0, 2, 3, 1)) * scale   # [G, hk, hp, L]
        seen = torch.arange(ko.shape[1], device=q.device)[None, :] < ol[:, None]
        so = so.masked_fill(~seen[:, None, None, :], float("-inf"))
        sc = torch.cat([sp, so], -1)
        m = sc.amax(-1, keepdim=True)
        m0 = torch.where(m == float("-inf"), torch.zeros_like(m), m)
        p = torch.exp(sc - m0)
        l = p.sum(-1, keepdim=True)
        pn = p / torch.where(l == 0, torch.ones_like(l), l)
        vo = vo.masked_fill(~seen[:, :, None, None], 0.0)
        acc = torch.matmul(pn[..., :n].transpose(0, 1).reshape(hk, G * hp, n), vp.transpose(0, 1))
        acc = acc.view(hk, G, hp, d).transpose(0, 1) + torch.matmul(pn[..., n:], vo.transpose(1, 2))
        o[s0:s0 + G] = acc.reshape(G, hq, d)
        lse[:, s0:s0 + G] = (m0 + torch.log(l)).reshape(G, hq).t()
        s0 += G
    return o.to(st["q"].dtype), lse


def _plain_sample(st):
    x = st["logits"].double()
    S, V = x.shape
    t = st["temperature"].double()[:, None]
    greedy = t == 0
    t = torch.where(greedy, torch.ones_like(t), t)
    w = torch.exp((x - x.amax(-1, keepdim=True)) / t)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    rank = torch.arange(V, device=x.device)[None, :]
    keep = torch.ones_like(ws, dtype=torch.bool)
    if st["top_k"] is not None:
        k = st["top_k"].long()[:, None]
        keep = rank < torch.where(k <= 0, torch.full_like(k, V), k)
    if st["top_p"] is not None:
        p = st["top_p"].double()[:, None]
        wk = ws * keep
        before = torch.cumsum(wk, -1) - wk
        keep = keep & ((before < p * wk.sum(-1, keepdim=True)) | (p >= 1))
    if st["min_p"] is not None:
        keep = keep & (ws >= st["min_p"].double()[:, None])
    keep = torch.where(greedy, rank == 0, keep | (rank == 0))
    kept = torch.zeros_like(w).scatter_(1, order, ws * keep)
    cum = torch.cumsum(kept, -1)
    target = st["u"].double()[:, None] * kept.sum(-1, keepdim=True)
    token = (cum <= target).sum(-1).clamp_(max=V - 1)
    logprob = torch.log(w.gather(1, token[:, None]) / w.sum(-1, keepdim=True))[:, 0]
    return token.to(torch.int32), logprob.float()


# ---------------------------------------------------------------------------------------- the calls --

def run(state):
    op = state["case"]["op"]
    if not own:
        return {"qk_norm": _plain_qk_norm, "append": _plain_append, "decode": _plain_decode,
                "sample": _plain_sample}[op](state)
    from shared_prefix_grouped_gb300 import api
    st = state
    if op == "qk_norm":
        if st["case"]["direction"] == "fwd":
            return api.qk_norm_rope_fwd(st["q"], st["k"], st["gain_q"], st["gain_k"], EPS,
                                        st["positions"], rope_theta=THETA)
        return api.qk_norm_rope_bwd(st["q"], st["k"], st["gain_q"], st["gain_k"], EPS,
                                    st["dq_out"], st["dk_out"], st["positions"], rope_theta=THETA)
    if op == "append":
        q = api.cache_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["pages"],
                             st["cache_pos"], page_rows=st["page_rows"], q=st["q"],
                             positions=st["positions"], rope_theta=THETA)
        return (st["k_cache"], st["v_cache"]) + (() if q is None else (q,))
    if op == "decode":
        return api.decode_attn(st["plan"], st["q"], st["k_cache"], st["v_cache"], st["prefix_pages"],
                               st["own_pages"], st["own_lens"], workspace=st["workspace"])
    return api.sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"],
                      top_p=st["top_p"], min_p=st["min_p"])


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "qk_norm":
        n = case["tokens"] * (case["heads_q"] + case["heads_kv"]) * case["head_dim"]
        fwd = case["direction"] == "fwd"
        return {"bytes": n * e * (2 if fwd else 3) + 4 * case["tokens"], "flops": n * (8 if fwd else 18)}
    if case["op"] == "append":
        n = case["seqs"] * case["tokens_per_seq"]
        rows = n * case["head_dim"]
        return {"bytes": 2 * rows * e * (case["heads_q"] + 2 * case["heads_kv"]) + 16 * n,
                "flops": 3 * rows * (case["heads_q"] + case["heads_kv"])}
    if case["op"] == "decode":
        S, G = case["groups"] * case["group_size"], case["group_size"]
        plens, olens = _prefix_lens(case), _own_lens(case)
        keys = sum(plens) + sum(olens)
        pairs = G * sum(plens) + sum(olens)
        row = case["head_dim"] * e
        return {"bytes": 2 * keys * case["heads_kv"] * row + S * case["heads_q"] * (2 * row + 4),
                "flops": 4 * pairs * case["heads_q"] * case["head_dim"]}
    return {"bytes": case["rows"] * (case["vocab"] * e + 28), "flops": 4 * case["rows"] * case["vocab"]}


# ------------------------------------------------------------------------------- the definitions --

def _exact_turn(x, positions):
    """Pairs (j, j + d/2) as complex numbers, multiplied by exp(i pos theta^(-2j/d)), in 64 bits."""
    d = x.shape[-1]
    z = torch.complex(x[..., :d // 2], x[..., d // 2:])
    freq = torch.tensor([THETA ** (-2.0 * j / d) for j in range(d // 2)], dtype=torch.float64,
                        device=x.device)
    ang = torch.outer(positions.double(), freq)
    z = z * torch.polar(torch.ones_like(ang), ang)[:, None, :]
    return torch.cat([z.real, z.imag], -1)


def _exact_qk_norm(case, st):
    outs, gains = [], []
    for name in ("q", "k"):
        x = st[name].double()
        g = st["gain_" + name].double()
        d = x.shape[-1]
        norm = torch.sqrt(x.square().sum(-1) / d + EPS)
        if case["direction"] == "fwd":
            outs.append(_exact_turn(x / norm[..., None] * g, st["positions"]))
        else:
            up = _exact_turn(st["d" + name + "_out"].double(), -st["positions"].long())
            gains.append(torch.einsum("thj,thj,th->j", up, x, 1 / norm))
            gu = g * up
            dot = (gu * x).sum(-1)
            outs.append(gu / norm[..., None] - x * (dot / (d * norm ** 3))[..., None])
    return tuple(outs + gains)


def _exact_append(case, st):
    ps, hk, d = st["k_cache"].shape[1:]
    kc, vc = st["k_cache"].double().view(-1, hk, d), st["v_cache"].double().view(-1, hk, d)
    cp = st["cache_pos"].long()
    row = st["pages"].long()[st["page_rows"].long()]
    slot = row.gather(1, (cp // ps)[:, None])[:, 0] * ps + cp % ps
    kc.index_copy_(0, slot, _exact_turn(st["k"].double(), st["positions"]))
    vc.index_copy_(0, slot, st["v"].double())
    out = [kc.view(-1, ps, hk, d), vc.view(-1, ps, hk, d)]
    if st["q"] is not None:
        out.append(_exact_turn(st["q"].double(), st["positions"]))
    return tuple(out)


def _exact_decode(case, st):
    hq, hk, d, ps = (case[x] for x in ("heads_q", "heads_kv", "head_dim", "page_size"))
    S = case["groups"] * case["group_size"]
    k, v = st["k_cache"].view(-1, hk, d), st["v_cache"].view(-1, hk, d)
    dev = k.device
    offs = torch.arange(ps, device=dev)
    o = torch.zeros((S, hq, d), dtype=torch.float64, device=dev)
    lse = torch.full((hq, S), float("-inf"), dtype=torch.float64, device=dev)
    lens = st["own_lens"].tolist()
    for b in range(case["groups"]):
        slots = (st["prefix_pages"][b].long()[:, None] * ps + offs).reshape(-1)
        slots = slots[:st["prefix_lens"][b]]
        pk, pv = k[slots].double().transpose(0, 1), v[slots].double().transpose(0, 1)
        for s in range(b * case["group_size"], (b + 1) * case["group_size"]):
            mine = (st["own_pages"][s].long()[:, None] * ps + offs).reshape(-1)[:lens[s]]
            if len(slots) + len(mine) == 0:
                continue
            q = st["q"][s].double().view(hk, hq // hk, d)
            ok, ov = k[mine].double().transpose(0, 1), v[mine].double().transpose(0, 1)
            sc = torch.cat([q @ pk.mT, q @ ok.mT], -1) / math.sqrt(d)
            z = torch.logsumexp(sc, -1)
            p = torch.exp(sc - z[..., None])
            o[s] = (p[..., :len(slots)] @ pv + p[..., len(slots):] @ ov).view(hq, d)
            lse[:, s] = z.view(hq)
    return o, lse


def _exact_sample(case, st):
    x = st["logits"].double().cpu().numpy()
    S, V = x.shape
    par = {n: None if st[n] is None else st[n].double().cpu().numpy()
           for n in ("u", "temperature", "top_k", "top_p", "min_p")}
    tokens, logprobs = np.empty(S, np.int32), np.empty(S, np.float64)
    for r in range(S):
        best = int(np.argmax(x[r]))
        temp = par["temperature"][r]
        with np.errstate(under="ignore"):
            w = np.exp((x[r] - x[r, best]) / (temp if temp > 0 else 1.0))
        full = math.fsum(w)
        if temp == 0:
            tok = best
        else:
            order = np.argsort(-x[r], kind="stable")
            n = V
            if par["top_k"] is not None and par["top_k"][r] > 0:
                n = min(V, int(par["top_k"][r]))
            order = order[:n]
            if par["top_p"] is not None and par["top_p"][r] < 1:
                c = np.cumsum(w[order])
                # the first prefix of the order that reaches the share
                order = order[:int(np.searchsorted(c, par["top_p"][r] * c[-1], side="left")) + 1]
            if par["min_p"] is not None:
                ok = w[order] >= par["min_p"][r]
                order = order[ok] if ok.any() else order[:1]
            idx = np.sort(order)
            c = np.cumsum(w[idx])
            tok = idx[min(int(np.searchsorted(c, par["u"][r] * c[-1], side="right")), len(idx) - 1)]
        tokens[r], logprobs[r] = tok, math.log(w[tok] / full)
    return torch.from_numpy(tokens).cuda(), torch.from_numpy(logprobs).cuda()


def exact(case, seed):
    st = _inputs(case, seed)
    return {"qk_norm": _exact_qk_norm, "append": _exact_append, "decode": _exact_decode,
            "sample": _exact_sample}[case["op"]](case, st)

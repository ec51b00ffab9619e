"""Measured cases of the operators around a rollout whose cache is held in 8 bits and of the policy's
loss on what was rolled out: the append to a paged e4m3 cache with a scale for each block of 16 tokens
and head (with the rotation on the way) and its reading back, the attention of one new token per response
over such a cache, and the clipped policy loss with a KL term from the logits, with its gradient.

``own`` False: plain torch operations, in 32 bits (64 for angles and for sums over all tokens).  ``own``
True: the calls a program makes of the framework.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
BLOCK = 16           # tokens that share a scale
THETA = 5e5


# ------------------------------------------------------------------------------------- the cases --

def listed():
    return [
        # --- append to the 8-bit cache, and what its blocks then hold ---
        # One step of 16 responses in the middle of their answers: one token each joins a block that
        # holds twelve already, q rotated in the same call, strided projections.
        dict(name="append8_step_s16", op="append8", dtype="bf16", seqs=16, tokens_per_seq=1,
             heads_q=32, heads_kv=8, head_dim=128, page_size=64, base_len=700, fused_qkv=True,
             capacity=1024),
        # Eight prompts of 2048 tokens written after their prefill, pages of 32.
        dict(name="append8_prefill_b8_p2048", op="append8", dtype="bf16", seqs=8, tokens_per_seq=2048,
             heads_q=0, heads_kv=8, head_dim=128, page_size=32, base_len=0, fused_qkv=False,
             capacity=2560),
        # --- attention of one new token per response ---
        # A few short responses at the start of a rollout, 64-wide heads.
        dict(name="decode8_g4_p256", op="decode8", dtype="bf16", groups=1, group_size=4,
             prefix_lo=256, prefix_hi=256, own_lo=1, own_hi=48, heads_q=2, heads_kv=2, head_dim=64,
             page_size=16, own_pages=8),
        # 16 responses of a 16384-token prefix, up to 1024 tokens into their answers.
        dict(name="decode8_g16_p16384", op="decode8", dtype="bf16", groups=1, group_size=16,
             prefix_lo=16384, prefix_hi=16384, own_lo=256, own_hi=1024, heads_q=32, heads_kv=8,
             head_dim=128, page_size=64, own_pages=16),
        # Eight ragged groups of 16: many medium prefixes, every response at its own length.
        dict(name="decode8_b8_g16_p2048", op="decode8", dtype="bf16", groups=8, group_size=16,
             prefix_lo=1601, prefix_hi=2495, own_lo=0, own_hi=512, heads_q=32, heads_kv=8,
             head_dim=128, page_size=32, own_pages=20),
        # 64 responses for each of four 32768-token contexts: several row blocks read one prefix.
        dict(name="decode8_b4_g64_p32768", op="decode8", dtype="bf16", groups=4, group_size=64,
             prefix_lo=32768, prefix_hi=32768, own_lo=1, own_hi=1537, heads_q=32, heads_kv=8,
             head_dim=128, page_size=128, own_pages=16),
        # --- policy loss ---
        # The log-probabilities of one step's 16 tokens: a launch whose latency counts.
        dict(name="policy_fwd_r16_v32000", op="policy", direction="fwd", dtype="f32", rows=16,
             vocab=32000, row_pad=0, shared=0, kl=True, temperature=1.0),
        # The reference policy's scores of the responses of a few groups.
        dict(name="policy_fwd_r5120_v131072", op="policy", direction="fwd", dtype="bf16", rows=5120,
             vocab=131072, row_pad=0, shared=0, kl=False, temperature=1.0),
        # A training step in fp32, the last prefix row shared by the group's first tokens.
        dict(name="policy_step_r1024_v32000", op="policy", direction="step", dtype="f32", rows=1024,
             vocab=32000, row_pad=0, shared=8, kl=True, temperature=1.0),
        # A padded, odd vocabulary in bf16, sampled at a temperature.
        dict(name="policy_step_r2045_v50001", op="policy", direction="step", dtype="bf16", rows=2045,
             vocab=50001, row_pad=47, shared=16, kl=True, temperature=0.8),
        # 16 responses of 512 tokens over a large vocabulary: loss and gradient of a whole group.
        dict(name="policy_step_r8192_v131072", op="policy", direction="step", dtype="bf16", rows=8192,
             vocab=131072, row_pad=0, shared=16, kl=True, temperature=1.0),
        # The backward alone, from the saved normaliser, as when the loss is part of a larger one.
        dict(name="policy_bwd_r4096_v131072", op="policy", direction="bwd", dtype="bf16", rows=4096,
             vocab=131072, row_pad=0, shared=16, kl=True, temperature=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append8", "decode8", "decode8", "policy", "policy"])
    hkv = rng.choice([1, 2, 4, 8])
    hp = rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "append8":
        step = rng.random() < 0.5
        base = _log_int(rng, 1, 2000) if step else rng.choice([0, 0, _log_int(rng, 1, 500)])
        per = 1 if step else _log_int(rng, 2, 1600)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    seqs=_log_int(rng, 1, 128) if step else rng.randint(1, 6), tokens_per_seq=per,
                    heads_q=rng.choice([0, min(hp * hkv, 32)]), heads_kv=hkv,
                    head_dim=rng.choice([64, 128]), page_size=rng.choice([16, 32, 64, 128, 256]),
                    base_len=base, fused_qkv=rng.random() < 0.5,
                    capacity=base + per + rng.randint(0, 300))
    if op == "decode8":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        plo = rng.choice([0, 1, _log_int(rng, 1, 4000), _log_int(rng, 100, 16000)])
        phi = min(plo + rng.choice([0, rng.randint(0, 900)]), 16384)
        page = rng.choice([16, 32, 64, 128, 256])
        olo = rng.choice([0, 1, rng.randint(0, 300)])
        ohi = olo + _log_int(rng, 1, 900)
        if dtype == "f32":
            plo, phi, olo, ohi = plo // 8, phi // 8, olo // 4, max(ohi // 4, olo // 4)
        ohi = max(ohi, 1)
        return dict(op=op, dtype=dtype, groups=rng.randint(1, 5), group_size=_log_int(rng, 1, 33),
                    prefix_lo=plo, prefix_hi=phi, own_lo=olo, own_hi=ohi,
                    heads_q=min(hp, 32 // hkv) * hkv, heads_kv=hkv,
                    head_dim=rng.choice([64, 128, 128]), page_size=page,
                    own_pages=(ohi + page - 1) // page + rng.randint(0, 2))
    return dict(op=op, direction=rng.choice(["fwd", "step", "step", "bwd"]),
                dtype=rng.choice(["bf16", "bf16", "f32"]), rows=_log_int(rng, 1, 4000),
                vocab=_log_int(rng, 2, 131072), row_pad=rng.choice([0, 0, rng.randint(1, 63)]),
                shared=rng.choice([0, 0, rng.randint(2, 40)]), kl=rng.random() < 0.7,
                temperature=rng.choice([1.0, 1.0, round(rng.uniform(0.6, 1.3), 2)]))


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


def _block_scale(amax):
    """The least power of two 2^e, e >= -126, with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)
    e = (torch.where(m <= 0.875, e - 9, e - 8)).clamp_(min=-126)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, torch.full_like(e, -126)))


def _held_cache(g, pages, ps, hk, d):
    """A cache [pages, ps, hk, d] whose blocks were all written before: (codes, scales)."""
    x = torch.randn((pages, ps // BLOCK, BLOCK, hk, d), generator=g, device="cuda")
    x *= torch.exp2(torch.rand((pages, ps // BLOCK, 1, hk, 1), generator=g, device="cuda") * 2 - 1)
    s = _block_scale(x.abs().amax((2, 4)))
    return (x / s[:, :, None, :, None]).to(F8).view(pages, ps, hk, d), s


def _row_counts(rows, shared):
    """Targets of each row: with `shared`, a row before a group's responses has the first tokens of all
    of them and a row at the end of a response has none."""
    if not shared:
        return [1] * rows
    return [shared if r % 97 == 0 else (0 if r % 97 in (31, 66) else 1) for r in range(rows)]


def _inputs(case, seed):
    """The tensors a program holds before the call, from the seed alone."""
    g = _gen(seed)
    dev = "cuda"
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)

    if case["op"] == "append8":
        S, n, hq, hk, d = (case[x] for x in ("seqs", "tokens_per_seq", "heads_q", "heads_kv",
                                             "head_dim"))
        ps, N, base = case["page_size"], case["seqs"] * case["tokens_per_seq"], case["base_len"]
        per_seq = (case["capacity"] + ps - 1) // ps
        total = S * per_seq + 3
        if case["fused_qkv"]:
            x = normal(N, hq + 2 * hk, d)
            q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        else:
            q, k, v = normal(N, hq, d), normal(N, hk, d), normal(N, hk, d)
        pages = torch.randperm(total, generator=g, device=dev)[:S * per_seq]
        idx = torch.arange(N, device=dev, dtype=torch.int32)
        cache_pos = base + idx % n
        k_codes, k_scales = _held_cache(g, total, ps, hk, d)
        v_codes, v_scales = _held_cache(g, total, ps, hk, d)
        # Everything the call may change: the blocks it touches, from their first token on.
        first = base // BLOCK * BLOCK
        held = torch.arange(first, base + n, device=dev, dtype=torch.int32)
        return dict(q=q if hq else None, k=k, v=v, k_codes=k_codes, k_scales=k_scales, v_codes=v_codes,
                    v_scales=v_scales, pages=pages.view(S, per_seq).to(torch.int32).contiguous(),
                    page_rows=(idx // n).to(torch.int32), cache_pos=cache_pos.to(torch.int32),
                    # the tokens sit behind a shared prefix that has pages of its own
                    positions=(cache_pos + 5000).to(torch.int32),
                    read_rows=torch.arange(S, device=dev, dtype=torch.int32).repeat_interleave(len(held)),
                    read_pos=held.repeat(S))
    if case["op"] == "decode8":
        B, G, hq, hk, d, ps = (case[x] for x in ("groups", "group_size", "heads_q", "heads_kv",
                                                 "head_dim", "page_size"))
        S = B * G
        plens, olens = _prefix_lens(case), torch.tensor(_own_lens(case), dtype=torch.int32)
        olens = olens.to(dev)[torch.randperm(S, generator=g, device=dev)]
        per_prefix, per_own = max((max(plens) + ps - 1) // ps, 1), case["own_pages"]
        total = B * per_prefix + S * per_own
        perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        k_codes, k_scales = _held_cache(g, total, ps, hk, d)
        v_codes, v_scales = _held_cache(g, total, ps, hk, d)
        return dict(q=normal(S, hq, d), k_codes=k_codes, k_scales=k_scales, v_codes=v_codes,
                    v_scales=v_scales, prefix_lens=plens, group_sizes=[G] * B,
                    prefix_pages=perm[:B * per_prefix].view(B, per_prefix).contiguous(),
                    own_pages=perm[B * per_prefix:].view(S, per_own).contiguous(), own_lens=olens)
    R, V, T = case["rows"], case["vocab"], case["temperature"]
    x = torch.randn((R, V + case["row_pad"]), generator=g, device=dev, dtype=dt)
    x *= 2.5
    # a language model's head: a few tokens stand out of the bulk
    n_hot = min(24, V)
    each = V // n_hot
    hot = torch.arange(n_hot, device=dev) * each + torch.randint(0, each, (R, n_hot), generator=g, device=dev)
    x.scatter_(1, hot, normal(R, n_hot, scale=1.5) + 9)
    logits = x[:, :V]
    counts = torch.tensor(_row_counts(R, case["shared"]), device=dev)
    starts = torch.zeros(R + 1, dtype=torch.int32, device=dev)
    starts[1:] = counts.cumsum(0).to(torch.int32)
    row = torch.arange(R, device=dev).repeat_interleave(counts)
    N = row.numel()
    # tokens that the policy itself might have drawn, from 64 candidates and the ones that stand out
    cand = torch.cat([torch.randint(0, V, (N, 64), generator=g, device=dev), hot[row]], 1)
    u = torch.rand(cand.shape, generator=g, device=dev).clamp_(1e-6, 1 - 1e-6)
    z = logits[row[:, None], cand].float() / T - torch.log(-torch.log(u))
    tokens = cand.gather(1, z.argmax(1, keepdim=True))[:, 0].to(torch.int32)
    lse = torch.cat([torch.logsumexp(c.float() / T, 1) for c in logits.split(512)])
    lp = logits[row, tokens.long()].float() / T - lse[row]
    seq = torch.arange(N, device=dev) // 37       # responses: an advantage for all tokens of one
    weights = torch.full((N,), 1.0 / max(N, 1), device=dev)
    weights[torch.rand(N, generator=g, device=dev) < 0.05] = 0.0      # tokens that are not trained on
    s = dict(logits=logits, tokens=tokens, row=row, live=counts > 0, row_starts=starts if case["shared"] else None,
             temperature=T, clip_low=0.2, clip_high=0.28, kl_coef=0.04 if case["kl"] else 0.0,
             old_logprobs=lp + 0.15 * normal(N, dtype=torch.float32),
             ref_logprobs=lp + 0.2 * normal(N, dtype=torch.float32) if case["kl"] else None,
             advantages=normal(N // 37 + 1, dtype=torch.float32)[seq], weights=weights)
    if case["direction"] == "bwd":
        s["lse"] = lse
        s["token_grad"] = weights * normal(N, dtype=torch.float32)
        s["grad_output"] = torch.full((1,), 0.5, device=dev)
    return s


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if own and case["op"] in ("append8", "decode8"):
        from shared_prefix_grouped_gb300 import api
        for n in ("k", "v"):
            state[n + "_cache"] = api.ScaledCache(state[n + "_codes"], state[n + "_scales"])
        if case["op"] == "decode8":
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


def _plain_append8(st):
    c, s = _cos_sin(st["positions"], st["k"].shape[-1])
    ps, hk, d = st["k_codes"].shape[1:]
    cp = st["cache_pos"].long()
    page = st["pages"][st["page_rows"].long(), cp // ps].long()
    block = page * (ps // BLOCK) + cp % ps // BLOCK
    inside = cp % BLOCK
    blocks, which = torch.unique(block, return_inverse=True)
    # a block that gets its first token in this call holds nothing from before
    begun = torch.zeros(blocks.numel(), dtype=torch.bool, device=cp.device)
    begun[which[inside == 0]] = True
    out = []
    for name, x in (("k", _rotate(st["k"].float(), c, s)), ("v", st["v"].float())):
        codes, scales = st[name + "_codes"], st[name + "_scales"]
        need = torch.zeros((blocks.numel(), hk), device=cp.device)
        need.scatter_reduce_(0, which[:, None].expand(-1, hk), x.abs().amax(-1), "amax")
        held = scales.view(-1, hk)[blocks]
        old = torch.where(begun[:, None], torch.zeros_like(held), held)
        new = torch.maximum(_block_scale(need), old)
        in_block = codes.view(-1, BLOCK, hk, d)
        kept = in_block.view(torch.uint8)[blocks].view(F8).float() * (old / new)[:, None, :, None]
        kept[which, inside] = x / new[which][:, :, None]
        in_block.view(torch.uint8)[blocks] = kept.to(F8).view(torch.uint8)
        scales.view(-1, hk)[blocks] = new
        rp = st["read_pos"].long()
        rpage = st["pages"][st["read_rows"].long(), rp // ps].long()
        got = codes.view(torch.uint8)[rpage, rp % ps].view(F8).float()
        out.append((got * scales[rpage, rp % ps // BLOCK][:, :, None]).to(st["k"].dtype))
    if st["q"] is not None:
        out.append(_rotate(st["q"].float(), c, s).to(st["q"].dtype))
    return tuple(out)


def _plain_decode8(st):
    q = st["q"].float()
    S, hq, d = q.shape
    ps, hk = st["k_codes"].shape[1:3]
    hp, scale = hq // hk, d ** -0.5

    def read(name, pages):                                       # [.., pages] -> [.., keys, hk, d]
        x = st[name + "_codes"].view(torch.uint8)[pages].view(F8).float()
        x = x.view(*pages.shape, ps // BLOCK, BLOCK, hk, d)
        x = x * st[name + "_scales"][pages][..., None, :, None]
        return x.reshape(*pages.shape[:-1], -1, hk, d)

    o, lse = torch.empty_like(q), torch.empty((hq, S), device=q.device)
    s0 = 0
    for b, G in enumerate(st["group_sizes"]):
        n = st["prefix_lens"][b]
        pp = st["prefix_pages"][b, :(n + ps - 1) // ps].long()
        kp, vp = read("k", pp)[:n], read("v", pp)[:n]           # [n, hk, d]
        op = st["own_pages"][s0:s0 + G].long()
        ko, vo = read("k", op), read("v", op)                   # [G, L, hk, d]
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


def _plain_gradient(st, p, token_grad):
    """Gradient of the logits from the probabilities p (overwritten) and the tokens' gradients."""
    g = token_grad / st["temperature"]
    total = torch.zeros(p.shape[0], device=p.device).index_add_(0, st["row"], g)
    p *= -total[:, None]
    p.index_put_((st["row"], st["tokens"].long()), g, accumulate=True)
    return p.to(st["logits"].dtype)


def _plain_policy(st):
    x = st["logits"].float() / st["temperature"]
    row, tok = st["row"], st["tokens"].long()
    if st["case"]["direction"] == "bwd":
        p = torch.exp(x.sub_(st["lse"][:, None]))
        return _plain_gradient(st, p, st["token_grad"] * st["grad_output"])
    m = x.amax(-1, keepdim=True)
    picked = x[row, tok] - m[row, 0]
    p = torch.exp(x.sub_(m))
    total = p.sum(-1, keepdim=True)
    log_total = torch.log(total)[:, 0]
    lp = picked - log_total[row]
    ratio = torch.exp(lp - st["old_logprobs"])
    adv, w = st["advantages"], st["weights"]
    free = ratio * adv
    clipped = torch.clamp(ratio, 1 - st["clip_low"], 1 + st["clip_high"]) * adv
    loss = -torch.minimum(free, clipped)
    grad = torch.where(free <= clipped, -free, torch.zeros_like(free))
    if st["ref_logprobs"] is not None:
        gap = st["ref_logprobs"] - lp
        loss = loss + st["kl_coef"] * (torch.expm1(gap) - gap)
        grad = grad - st["kl_coef"] * torch.expm1(gap)
    loss, grad = loss * w, grad * w
    # a row without targets has no normaliser
    lse = torch.where(st["live"], m[:, 0] + log_total, torch.zeros_like(log_total))
    out = [loss.double().sum().float().reshape(1), lp, loss, grad, lse]
    if st["case"]["direction"] == "step":
        out.append(_plain_gradient(st, p.div_(total), grad))
    return tuple(out)


# ---------------------------------------------------------------------------------------- the calls --

def run(state):
    op = state["case"]["op"]
    if not own:
        return {"append8": _plain_append8, "decode8": _plain_decode8, "policy": _plain_policy}[op](state)
    from shared_prefix_grouped_gb300 import api
    st = state
    if op == "append8":
        q = api.cache_append_e4m3(st["k"], st["v"], st["k_cache"], st["v_cache"], st["pages"],
                                  st["cache_pos"], page_rows=st["page_rows"], q=st["q"],
                                  positions=st["positions"], rope_theta=THETA)
        out = api.cache_read_e4m3(st["k_cache"], st["v_cache"], st["pages"], st["read_pos"],
                                  page_rows=st["read_rows"], dtype=st["k"].dtype)
        return out + (() if q is None else (q,))
    if op == "decode8":
        return api.decode_attn_e4m3(st["plan"], st["q"], st["k_cache"], st["v_cache"],
                                    st["prefix_pages"], st["own_pages"], st["own_lens"],
                                    workspace=st["workspace"])
    if st["case"]["direction"] == "bwd":
        return api.policy_loss_bwd(st["logits"], st["tokens"], st["lse"], st["token_grad"],
                                   row_starts=st["row_starts"], temperature=st["temperature"],
                                   grad_output=st["grad_output"])
    r = api.policy_loss(st["logits"], st["tokens"], old_logprobs=st["old_logprobs"],
                        advantages=st["advantages"], weights=st["weights"],
                        ref_logprobs=st["ref_logprobs"], row_starts=st["row_starts"],
                        clip_low=st["clip_low"], clip_high=st["clip_high"], kl_coef=st["kl_coef"],
                        temperature=st["temperature"], grad=st["case"]["direction"] == "step")
    out = (r.loss, r.logprobs, r.token_loss, r.token_grad, r.lse)
    return out if r.dlogits is None else out + (r.dlogits,)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append8":
        S, n, hq, hk, d = (case[x] for x in ("seqs", "tokens_per_seq", "heads_q", "heads_kv",
                                             "head_dim"))
        N, held = S * n, S * (case["base_len"] % BLOCK + n)
        # q read and written; k, v read; codes written, then read back with the tokens before them in
        # their blocks and given out as values; a scale per 16 tokens
        return {"bytes": N * d * e * (2 * hq + 2 * hk) + 2 * N * hk * d + 2 * held * hk * d * (1 + e) +
                         held * hk + 16 * N + 8 * held,
                "flops": 3 * N * d * (hq + hk) + 4 * held * hk * d}
    if case["op"] == "decode8":
        S, G = case["groups"] * case["group_size"], case["group_size"]
        plens, olens = _prefix_lens(case), _own_lens(case)
        keys = sum(plens) + sum(olens)
        pairs = G * sum(plens) + sum(olens)
        row = case["head_dim"]
        return {"bytes": keys * case["heads_kv"] * (2 * row + 8 / BLOCK) +
                         S * case["heads_q"] * (2 * row * e + 4),
                "flops": 4 * pairs * case["heads_q"] * row}
    R, V = case["rows"], case["vocab"]
    counts = _row_counts(R, case["shared"])
    live, N = sum(c > 0 for c in counts), sum(counts)
    fwd, step = case["direction"] == "fwd", case["direction"] == "step"
    # rows without targets need not be read; their gradient is written
    return {"bytes": live * V * e + (0 if fwd else R * V * e) + 4 * R + 32 * N,
            "flops": live * V * (8 if step else 4)}


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


def _to_e4m3(x):
    """x, at most 448 in magnitude, to the nearest of the numbers with three fraction bits and exponents
    from -6 on (below: multiples of 2^-9), ties to the even one; in 64 bits."""
    e = torch.frexp(x.abs())[1].double() - 1
    step = torch.exp2(e.clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_append8(case, st):
    ps, hk, d = st["k_codes"].shape[1:]
    S, n, base = case["seqs"], case["tokens_per_seq"], case["base_len"]
    lo = base // BLOCK * BLOCK
    count = base + n - lo
    # the sequences' keys from the first block that changes: [S, blocks, 16, hk, d], behind the end zero
    nb = (count + BLOCK - 1) // BLOCK
    pos = torch.arange(lo, lo + nb * BLOCK, device=st["k"].device)
    page = st["pages"].long()[:, (pos // ps).clamp(max=st["pages"].shape[1] - 1)]
    new = (pos >= base) & (pos < base + n)
    before = pos < base
    out = []
    for name, x in (("k", _exact_turn(st["k"].double(), st["positions"])), ("v", st["v"].double())):
        fresh = torch.zeros((S, nb * BLOCK, hk, d), dtype=torch.float64, device=pos.device)
        fresh[:, new] = x.view(S, n, hk, d)
        sc = st[name + "_scales"].double()[page, pos % ps // BLOCK]                 # [S, keys, hk]
        old = st[name + "_codes"].float().double()[page, pos % ps] * sc[..., None]
        old[:, ~before] = 0
        fresh, old = (t.view(S, nb, BLOCK, hk, d) for t in (fresh, old))
        top = fresh.abs().amax((2, 4))                                              # [S, nb, hk]
        e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0))
        e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
        e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp(min=-126)
        scale = torch.exp2(e)
        if base > lo:       # the first block goes on with at least the scale it has
            scale[:, 0] = torch.maximum(scale[:, 0], sc.view(S, nb, BLOCK, hk)[:, 0, 0])
        scale = scale[:, :, None, :, None]
        val = (_to_e4m3((fresh + old) / scale) * scale).view(S, nb * BLOCK, hk, d)
        out.append(val[:, :count].reshape(-1, hk, d))
    if st["q"] is not None:
        out.append(_exact_turn(st["q"].double(), st["positions"]))
    return tuple(out)


def _exact_decode8(case, st):
    hq, hk, d, ps = (case[x] for x in ("heads_q", "heads_kv", "head_dim", "page_size"))
    S = case["groups"] * case["group_size"]
    dev = st["q"].device
    offs = torch.arange(ps, device=dev)
    o = torch.zeros((S, hq, d), dtype=torch.float64, device=dev)
    lse = torch.full((hq, S), float("-inf"), dtype=torch.float64, device=dev)

    def keys(pages, n):
        slot = (pages.long()[:, None] * ps + offs).reshape(-1)[:n]
        got = []
        for name in ("k", "v"):
            c = st[name + "_codes"].view(torch.uint8).view(-1, hk, d)[slot].view(F8).float().double()
            got.append((c * st[name + "_scales"].view(-1, hk)[slot // BLOCK].double()[..., None]
                        ).transpose(0, 1))
        return got

    lens = st["own_lens"].tolist()
    for b in range(case["groups"]):
        pk, pv = keys(st["prefix_pages"][b], st["prefix_lens"][b])
        for s in range(b * case["group_size"], (b + 1) * case["group_size"]):
            if st["prefix_lens"][b] + lens[s] == 0:
                continue
            ok, ov = keys(st["own_pages"][s], lens[s])
            q = st["q"][s].double().view(hk, hq // hk, d)
            sc = torch.cat([q @ pk.mT, q @ ok.mT], -1) / math.sqrt(d)
            z = torch.logsumexp(sc, -1)
            p = torch.exp(sc - z[..., None])
            n = pk.shape[1]
            o[s] = (p[..., :n] @ pv + p[..., n:] @ ov).view(hq, d)
            lse[:, s] = z.view(hq)
    return o, lse


def _exact_policy(case, st):
    R, T = case["rows"], st["temperature"]
    row, tok = st["row"], st["tokens"].long()
    bwd = case["direction"] == "bwd"
    if bwd:
        lse = st["lse"].double()
    else:
        lse = torch.cat([torch.logsumexp(c.double() / T, 1) for c in st["logits"].split(256)])
    at = st["logits"][row, tok].double() / T
    lp = at - lse[row]
    if bwd:
        g = st["token_grad"].double() * st["grad_output"].double()
    else:
        lo, hi = 1 - st["clip_low"], 1 + st["clip_high"]
        r = torch.exp(lp - st["old_logprobs"].double())
        A, w = st["advantages"].double(), st["weights"].double()
        # the smaller of r A and clip(r) A: r counts up to hi where A > 0, from lo on where A < 0
        moves = torch.where(A >= 0, r <= hi, r >= lo)
        loss = -w * A * torch.where(moves, r, torch.where(A >= 0, hi, lo))
        g = torch.where(moves, -w * A * r, torch.zeros_like(r))
        if st["ref_logprobs"] is not None:
            x = st["ref_logprobs"].double() - lp
            loss = loss + w * st["kl_coef"] * (x.exp() - x - 1)
            g = g + w * st["kl_coef"] * (1 - x.exp())
        out = [loss.sum().reshape(1), lp, loss, g, lse * st["live"]]
        if case["direction"] == "fwd":
            return tuple(out)
    d = torch.empty(st["logits"].shape, dtype=torch.float64, device=lse.device)
    for r0 in range(0, R, 256):
        d[r0:r0 + 256] = torch.exp(st["logits"][r0:r0 + 256].double() / T - lse[r0:r0 + 256, None])
    d *= -torch.bincount(row, weights=g, minlength=R)[:, None] / T
    d.index_put_((row, tok), g / T, accumulate=True)
    return d if bwd else tuple(out) + (d,)


def exact(case, seed):
    st = _inputs(case, seed)
    return {"append8": _exact_append8, "decode8": _exact_decode8, "policy": _exact_policy}[
        case["op"]](case, st)

"""CPU oracle of the rollout operators, fp64: per-head norm with rotation (forward, backward), append
to a paged cache, attention of one token per response over a shared prefix and its own keys, and
token sampling.  Plain loops and textbook formulas; shares no code with the CUDA path.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def rotate(x: torch.Tensor, positions: torch.Tensor, theta: float, inverse: bool = False):
    """Rotate-half RoPE of x [T, H, d] at positions [T]: pair (j, j + d/2) by pos * theta^(-2j/d)."""
    x = x.to(F64)
    if theta <= 0:
        return x.clone()
    d = x.shape[-1]
    j = torch.arange(d // 2, dtype=F64)
    ang = positions.to(F64)[:, None, None] * theta ** (-2 * j / d)
    if inverse:
        ang = -ang
    a, b = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)


def norm_rope(x, gain, eps, positions, theta):
    x = x.to(F64)
    r = (x.square().mean(-1, keepdim=True) + eps) ** -0.5
    return rotate(x * r * gain.to(F64), positions, theta)


def norm_rope_bwd(x, gain, eps, dout, positions, theta):
    """(dx, dgain, scales): scales are the magnitudes that rounding errors are relative to.  An element
    of dy is a sum a cos + b sin that may cancel, so its error is relative to e = |a| + |b|:
    r max(g e) + r max|xhat| mean(|xhat g| e) for a row of dx, sum of e |xhat| for a gain gradient."""
    x, g = x.to(F64), gain.to(F64)
    r = (x.square().mean(-1, keepdim=True) + eps) ** -0.5
    xh = x * r
    dy = rotate(dout, positions, theta, inverse=True)
    dx = r * (g * dy - xh * (xh * g * dy).mean(-1, keepdim=True))
    h = dout.shape[-1] // 2
    e = dout[..., :h].to(F64).abs() + dout[..., h:].to(F64).abs()
    e = torch.cat([e, e], -1)
    row = r * ((g.abs() * e).amax(-1, keepdim=True)
               + xh.abs().amax(-1, keepdim=True) * ((xh * g).abs() * e).mean(-1, keepdim=True))
    return dx, (dy * xh).sum((0, 1)), (row, (e * xh.abs()).sum((0, 1)))


def append(k, v, k_cache, v_cache, pages, cache_pos, page_rows, positions, theta):
    """The caches after the append (fp64 copies), token by token."""
    kc, vc = k_cache.to(F64).clone(), v_cache.to(F64).clone()
    ps = kc.shape[1]
    kr = rotate(k, cache_pos if positions is None else positions, theta)
    for n in range(k.shape[0]):
        c = int(cache_pos[n])
        if c < 0:
            continue
        page = int(pages[n if page_rows is None else int(page_rows[n]), c // ps])
        kc[page, c % ps] = kr[n]
        vc[page, c % ps] = v[n].to(F64)
    return kc, vc


def gather(cache, pages, n):
    """The first n rows [n, Hkv, d] of a sequence whose pages are `pages`."""
    ps = cache.shape[1]
    idx = [(int(pages[i // ps]), i % ps) for i in range(n)]
    if not idx:
        return cache.new_zeros((0,) + tuple(cache.shape[2:])).to(F64)
    p, o = zip(*idx)
    return cache[list(p), list(o)].to(F64)


def decode(q, k_cache, v_cache, prefix_lens, group_sizes, prefix_pages, own_pages, own_lens, scale=None):
    """(o [S, Hq, d], lse [Hq, S], mass [S, Hq, d] = sum_j p_j |v_j|, dots: max_j scale sum |q k_j|)."""
    S, Hq, d = q.shape
    Hkv = k_cache.shape[2]
    hp = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    o, mass = torch.zeros((S, Hq, d), dtype=F64), torch.zeros((S, Hq, d), dtype=F64)
    lse = torch.full((Hq, S), -math.inf, dtype=F64)
    dots, s = 0.0, 0
    for b, G in enumerate(group_sizes):
        if G == 0:
            continue
        pk = gather(k_cache, prefix_pages[b] if prefix_lens[b] else [], prefix_lens[b])
        pv = gather(v_cache, prefix_pages[b] if prefix_lens[b] else [], prefix_lens[b])
        for _ in range(G):
            n = max(int(own_lens[s]), 0) if own_lens is not None else 0
            k = torch.cat([pk, gather(k_cache, own_pages[s], n)]) if n else pk
            v = torch.cat([pv, gather(v_cache, own_pages[s], n)]) if n else pv
            if k.shape[0]:
                for h in range(Hq):
                    x = scale * (k[:, h // hp] @ q[s, h].to(F64))
                    lse[h, s] = torch.logsumexp(x, 0)
                    p = torch.exp(x - lse[h, s])
                    o[s, h] = p @ v[:, h // hp]
                    mass[s, h] = p @ v[:, h // hp].abs()
                    dots = max(dots, scale * float((k[:, h // hp].abs() @ q[s, h].to(F64).abs()).max()))
            s += 1
    return o, lse, mass, dots


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """(tokens, logprobs): one row after another, from the sorted list of tokens."""
    S, V = logits.shape
    tokens, logprobs = [], []
    for r in range(S):
        x = logits[r].to(F64)
        x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x)
        order = sorted(range(V), key=lambda i: (-float(x[i]), i))
        m = float(x[order[0]])
        if m == -math.inf:
            tokens.append(-1)
            logprobs.append(-math.inf)
            continue
        T = 1.0 if temperature is None else float(temperature[r])
        greedy = not T > 0
        if greedy:
            T = 1.0
        if m == math.inf:
            w = [1.0 if float(v) == math.inf else 0.0 for v in x]
        else:
            w = [math.exp((float(v) - m) / T) if float(v) > -math.inf else 0.0 for v in x]
        total = math.fsum(w)
        keep = list(order)
        if greedy:
            keep = order[:1]
        else:
            if top_k is not None and int(top_k[r]) > 0:
                keep = keep[:int(top_k[r])]
            if top_p is not None and not float(top_p[r]) >= 1:      # NaN: the first token only
                part, out, mass = 0.0, [], math.fsum(w[i] for i in keep)
                for i in keep:
                    if out and not part < float(top_p[r]) * mass:
                        break
                    out.append(i)
                    part += w[i]
                keep = out
            if min_p is not None:
                keep = [i for i in keep if w[i] >= float(min_p[r])] or keep[:1]
        keep.sort()
        target = float(u[r]) * math.fsum(w[i] for i in keep)
        run, tok = 0.0, keep[-1]
        for i in keep:
            run += w[i]
            if run > target:
                tok = i
                break
        tokens.append(tok)
        logprobs.append(math.log(w[tok] / total))
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(logprobs, dtype=F64)


def layer(x, mask, positions, weights, *, heads_q, heads_kv, head_dim, theta, eps, g_q=None, g_k=None):
    """A Llama-style decoder layer over rows x [T, hidden] of which row t sees the rows mask[t], in fp64
    torch operations (so its gradients are autograd's); g_q and g_k: per-head norm gains of q and k."""
    w_qkv, w_o, w_gu, w_d, g1, g2 = weights
    T, Hq, Hkv, d = x.shape[0], heads_q, heads_kv, head_dim

    def rms(v, g):
        return v * (v.square().mean(-1, keepdim=True) + eps) ** -0.5 * g

    qkv = (rms(x, g1) @ w_qkv.t()).view(T, Hq + 2 * Hkv, d)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if g_q is not None:
        q, k = rms(q, g_q), rms(k, g_k)
    q, k = rotate(q, positions, theta), rotate(k, positions, theta)
    k, v = (t.repeat_interleave(Hq // Hkv, 1) for t in (k, v))
    sc = torch.einsum("thd,shd->hts", q, k) * d ** -0.5
    p = torch.softmax(sc.masked_fill(~mask, -math.inf), -1)
    x2 = x + torch.einsum("hts,shd->thd", p, v).reshape(T, Hq * d) @ w_o.t()
    gu = rms(x2, g2) @ w_gu.t()
    n = gu.shape[1] // 2
    return x2 + (torch.nn.functional.silu(gu[:, :n]) * gu[:, n:]) @ w_d.t()

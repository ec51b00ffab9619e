"""CPU oracle of the policy loss, fp64: token after token from the textbook formulas; shares no code with
the CUDA path.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def rows_of(row_starts, n_rows):
    """The row of every token."""
    if row_starts is None:
        return list(range(n_rows))
    return [r for r in range(n_rows) for _ in range(int(row_starts[r + 1]) - int(row_starts[r]))]


def loss(logits, tokens, *, advantages=None, old=None, ref=None, weights=None, row_starts=None,
         clip_low=0.2, clip_high=0.2, kl_coef=0.0, temperature=1.0):
    """(loss, logprobs [N], token_loss [N], token_grad [N], lse [R], dlogits [R, V], ratio [N])."""
    R, V = logits.shape
    z = logits.to(F64) / temperature
    owner = rows_of(row_starts, R)
    has = [False] * R
    for r in owner:
        has[r] = True
    lse = torch.tensor([float(torch.logsumexp(z[r], 0)) if has[r] else 0.0 for r in range(R)], dtype=F64)
    N = len(owner)
    lps, losses, grads, ratios = (torch.zeros(N, dtype=F64) for _ in range(4))
    d = torch.zeros((R, V), dtype=F64)
    for n, r in enumerate(owner):
        y = int(tokens[n])
        if not 0 <= y < V:
            continue
        dead = bool((z[r] == -math.inf).all())
        lp = -math.inf if dead else float(z[r, y] - lse[r])
        lps[n] = lp
        w = 1.0 if weights is None else float(weights[n])
        if advantages is None or w == 0.0 or dead:
            continue
        A = float(advantages[n])
        ratio = 1.0 if old is None else math.exp(lp - float(old[n]))
        ratios[n] = ratio
        clipped = min(max(ratio, 1 - clip_low), 1 + clip_high)
        losses[n] = -min(ratio * A, clipped * A)
        grads[n] = -ratio * A if ratio * A <= clipped * A else 0.0
        if ref is not None and kl_coef > 0:
            gap = float(ref[n]) - lp
            losses[n] += kl_coef * (math.exp(gap) - gap - 1)
            grads[n] += kl_coef * (1 - math.exp(gap))
        losses[n] *= w
        grads[n] *= w
    d = gradient(logits, tokens, lse, grads, row_starts, temperature)
    return float(losses.sum()), lps, losses, grads, lse, d, ratios


def gradient(logits, tokens, lse, token_grad, row_starts=None, temperature=1.0):
    """dlogits [R, V] from the tokens' gradients."""
    R, V = logits.shape
    d = torch.zeros((R, V), dtype=F64)
    for n, r in enumerate(rows_of(row_starts, R)):
        g, y = float(token_grad[n]), int(tokens[n])
        if g == 0.0 or not 0 <= y < V:
            continue
        if float(lse[r]) > -math.inf:
            d[r] -= g / temperature * torch.exp(logits[r].to(F64) / temperature - float(lse[r]))
        d[r, y] += g / temperature
    return d


def packed_rows(prefix_lens, group_sizes, suffix_lens):
    """For every row of the packed sequences, the packed tokens it predicts."""
    rows, t, s = [], 0, 0
    for lp, G in zip(prefix_lens, group_sizes):
        lens = suffix_lens[s:s + G]
        s += G
        begin, at = [], t + lp
        for n in lens:
            begin.append(at)
            at += n
        rows += [[] for _ in range(lp)]
        if lp:
            rows[-1] = [b for b, n in zip(begin, lens) if n]
        for b, n in zip(begin, lens):
            rows += [[b + j + 1] if j + 1 < n else [] for j in range(n)]
        t = at
    return rows

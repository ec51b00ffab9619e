"""CPU checks of the rollout operators and the q / k norm: the oracle against closed forms and finite
differences, the attention step's plan, and every refusal of the C entry points (host checks that
return before anything is launched) and of the binding."""
import ctypes as C
import math
import os
import shutil
import subprocess

import pytest
import torch

from oracle import rollout_oracle as ro
from shared_prefix_grouped_gb300 import _lib, api
from shared_prefix_grouped_gb300.build import build

BAD = _lib.PG_ERR_INVALID_ARG
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


# ------------------------------------------------------------------------------------- the oracle --

@pytest.mark.parametrize("theta", [0.0, 100.0])
def test_norm_rope_backward_matches_central_differences(theta):
    g = torch.Generator().manual_seed(1)
    T, H, d, eps = 3, 2, 64, 1e-3
    x = torch.randn((T, H, d), generator=g, dtype=torch.float64)
    gain = 1 + 0.3 * torch.randn(d, generator=g, dtype=torch.float64)
    w = torch.randn((T, H, d), generator=g, dtype=torch.float64)
    pos = torch.tensor([0, 5, 1000])
    dx, dg, _ = ro.norm_rope_bwd(x, gain, eps, w, pos, theta)
    h = 1e-5      # truncation h^2 ~ 1e-10, rounding 1e-16 |loss| / h ~ 1e-9

    def loss(x, gain):
        return float((w * ro.norm_rope(x, gain, eps, pos, theta)).sum())

    for idx in [(0, 0, 0), (1, 1, 31), (2, 0, 63), (2, 1, 40)]:
        e = torch.zeros_like(x)
        e[idx] = h
        num = (loss(x + e, gain) - loss(x - e, gain)) / (2 * h)
        assert abs(num - float(dx[idx])) < 1e-6
    for j in [0, 33, 63]:
        e = torch.zeros_like(gain)
        e[j] = h
        assert abs((loss(x, gain + e) - loss(x, gain - e)) / (2 * h) - float(dg[j])) < 1e-6


def test_rotation_is_a_rotation():
    x = torch.randn((4, 2, 64), dtype=torch.float64, generator=torch.Generator().manual_seed(2))
    pos = torch.tensor([0, 1, 77, 2 ** 20])
    y = ro.rotate(x, pos, 1e4)
    assert torch.equal(y[0], x[0])
    assert torch.allclose(y.square().sum(-1), x.square().sum(-1), atol=1e-12)
    assert torch.allclose(ro.rotate(y, pos, 1e4, inverse=True), x, atol=1e-12)
    z = torch.complex(x[..., :32], x[..., 32:])[1] * torch.exp(
        1j * 1e4 ** (-2 * torch.arange(32, dtype=torch.float64) / 64))
    assert torch.allclose(torch.cat([z.real, z.imag], -1), y[1], atol=1e-12)


def test_decode_oracle_is_causal_attention_of_the_last_token():
    # One response with prefix P and own keys R: the last row of softmax attention over [P; R].
    g = torch.Generator().manual_seed(3)
    Hq, Hkv, d, ps = 4, 2, 64, 16
    kc, vc = (torch.randn((8, ps, Hkv, d), generator=g, dtype=torch.float64) for _ in range(2))
    q = torch.randn((1, Hq, d), generator=g, dtype=torch.float64)
    pp, op = torch.tensor([[3, 0]]), torch.tensor([[7, 1]])
    o, lse, _, _ = ro.decode(q, kc, vc, [21], [1], pp, op, torch.tensor([18]))
    k = torch.cat([kc[3], kc[0][:5], kc[7], kc[1][:2]])
    v = torch.cat([vc[3], vc[0][:5], vc[7], vc[1][:2]])
    ref = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), k.repeat_interleave(2, 1).transpose(0, 1),
        v.repeat_interleave(2, 1).transpose(0, 1))
    assert torch.allclose(o.transpose(0, 1), ref, atol=1e-12)
    o0, l0, _, _ = ro.decode(q, kc, vc, [0], [1], None, op, torch.tensor([0]))
    assert not o0.any() and bool((l0 == -math.inf).all())


def test_sample_oracle_by_hand():
    ln = math.log
    x = torch.tensor([[ln(1), ln(4), ln(2), ln(4), ln(1)]], dtype=torch.float64)   # weights /12

    def draw(u, **kw):
        kw = {n: torch.tensor([v]) for n, v in kw.items()}
        t, lp = ro.sample(x, torch.tensor([u]), **kw)
        return int(t), float(lp)

    assert [draw(u)[0] for u in (0.0, 0.08, 0.09, 0.4, 0.42, 0.57, 0.59, 0.91, 0.92)] == \
        [0, 0, 1, 1, 2, 2, 3, 3, 4]
    assert draw(0.5)[1] == pytest.approx(ln(2 / 12))
    assert [draw(u, top_k=2)[0] for u in (0.0, 0.49, 0.51)] == [1, 1, 3]
    assert [draw(u, top_k=1)[0] for u in (0.0, 0.99)] == [1, 1]          # the tie goes to the lower index
    assert [draw(u, top_p=0.33)[0] for u in (0.0, 0.99)] == [1, 1]       # 4/12 reaches it
    assert [draw(u, top_p=0.34)[0] for u in (0.0, 0.99)] == [1, 3]
    assert [draw(u, min_p=0.5)[0] for u in (0.0, 0.99)] == [1, 3]
    assert [draw(u, min_p=0.49)[0] for u in (0.3, 0.5, 0.99)] == [1, 2, 3]
    assert draw(0.99, temperature=0.0) == (1, pytest.approx(ln(4 / 12)))
    assert ro.sample(torch.full((1, 3), -math.inf), torch.tensor([0.5]))[0].tolist() == [-1]


# --------------------------------------------------------------------------------------- the plan --

def test_plan_tables_list_every_response_with_its_group():
    st, tab = api.plan_decode_host([300, 0, 17], [3, 2, 1], 8, 2, 128, 32, 4)
    assert (st.num_groups, st.num_seqs, st.max_prefix) == (3, 6, 300)
    raw = tab.numpy().tobytes()
    seqs = torch.frombuffer(bytearray(raw[st.off_seqs: st.off_seqs + 16 * 6]),
                            dtype=torch.int32).view(6, 4)
    assert seqs[:, 0].tolist() == [0, 0, 0, 1, 1, 2]
    assert seqs[:, 1].tolist() == [300, 300, 300, 0, 0, 17]
    slots = max(st.simt_splits, st.prefix_slots + st.own_slots)
    assert st.workspace_bytes >= slots * 6 * 8 * (128 + 1) * 4
    # a group without responses needs no pages
    st, _ = api.plan_decode_host([10, 5000], [2, 0], 2, 2, 64, 16, 1, torch.float32)
    assert st.max_prefix == 10


@pytest.mark.parametrize("kw", [
    dict(prefix_lens=[], group_sizes=[]), dict(prefix_lens=[-1]), dict(group_sizes=[-1]),
    dict(group_sizes=[0]), dict(prefix_lens=[1 << 30]), dict(group_sizes=[1 << 20]),
    dict(heads_q=3), dict(heads_kv=0), dict(head_dim=96), dict(page_size=24), dict(page_size=512),
    dict(own_pages=-1), dict(own_pages=1 << 26),
])
def test_plan_refusals(kw):
    args = dict(prefix_lens=[100], group_sizes=[2], heads_q=4, heads_kv=2, head_dim=128,
                page_size=16, own_pages=4)
    api.plan_decode_host(**args)
    with pytest.raises(_lib.PgError) as e:
        api.plan_decode_host(**{**args, **kw})
    assert e.value.status == BAD


def test_plan_refuses_a_short_table():
    L, nb = _lib.lib(), C.c_int64()
    args = api._plan_args([100], [2], 4, 2, 128, 16, 4, torch.bfloat16)
    assert L.pg_plan_decode_size(*args, C.byref(nb)) == _lib.PG_OK
    buf, st = torch.empty(nb.value, dtype=torch.uint8), _lib.PgDecodePlan()
    assert L.pg_plan_decode_host(*args, C.c_void_p(buf.data_ptr()), nb.value - 1, C.byref(st)) == BAD
    assert L.pg_plan_decode_host(*args, None, nb.value, C.byref(st)) == BAD
    assert L.pg_plan_decode_size(*args, None) == BAD
    with pytest.raises(ValueError):
        api.plan_decode_host([100, 5], [2], 4, 2, 128, 16, 4)


C_PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include "pg_rollout.h"
int main(void) {
  const int32_t lens[2] = {300, 17}, sizes[2] = {3, 1};
  int64_t bytes = 0;
  pg_decode_plan plan;
  void* tables;
  if (pg_plan_decode_size(2, lens, sizes, PG_BF16, 8, 2, 128, 32, 4, &bytes) != PG_OK) return 1;
  tables = malloc((size_t)bytes);
  if (pg_plan_decode_host(2, lens, sizes, PG_BF16, 8, 2, 128, 32, 4, tables, bytes, &plan) != PG_OK)
    return 2;
  printf("%d %d %ld %lu %d", plan.num_seqs, plan.n_items, (long)bytes, (unsigned long)plan.workspace_bytes,
         (int)pg_sample(PG_F32, 0, 5, 0, 5, 0, 0, 0, 0, 0, 0, 0, 0));
  free(tables);
  return 0;
}
"""


def test_header_and_plan_from_c(tmp_path):
    # The headers are C99; a plan made from C is the binding's.
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    src, exe, libdir = tmp_path / "p.c", tmp_path / "p", os.path.dirname(_lib.LIB_PATH)
    src.write_text(C_PROGRAM)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                    os.path.join(ROOT, "include"), str(src), "-L", libdir, "-lpg_gb300",
                    f"-Wl,-rpath,{libdir}", "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    st, tab = api.plan_decode_host([300, 17], [3, 1], 8, 2, 128, 32, 4)
    assert [int(x) for x in out] == [st.num_seqs, st.n_items, tab.numel(), st.workspace_bytes, BAD]


def test_plan_items_cover_every_response_and_key_once():
    # Each (response, prefix key) pair belongs to exactly one item, whose part is the response's.
    for plens, gs, hq, hkv in [([300], [40], 8, 2), ([5000, 0, 129], [33, 2, 1], 32, 8),
                               ([128, 64], [1, 70], 6, 1), ([40000], [1], 4, 4)]:
        st, tab = api.plan_decode_host(plens, gs, hq, hkv, 128, 16, 3)
        raw = tab.numpy().tobytes()
        seqs = torch.frombuffer(bytearray(raw[st.off_seqs:]), dtype=torch.int32)[:4 * st.num_seqs]
        items = torch.frombuffer(bytearray(raw[st.off_items:]), dtype=torch.int32)[:8 * st.n_items]
        seen = {s: [] for s in range(st.num_seqs)}
        for group, s0, n, lo, hi, slot, _, _ in items.view(-1, 8).tolist():
            assert lo % 128 == 0 and lo < hi and 1 <= n <= st.seqs_per_item
            assert n * (hq // hkv) <= 128
            for s in range(s0, s0 + n):
                assert seqs[4 * s] == group and slot < seqs[4 * s + 2] <= st.prefix_slots
                seen[s].append((slot, lo, hi))
        for s, parts in seen.items():
            parts.sort()
            assert [p[0] for p in parts] == list(range(int(seqs[4 * s + 2])))
            ends = [0] + [p[2] for p in parts]
            assert [p[1] for p in parts] == ends[:-1] and ends[-1] == int(seqs[4 * s + 1])


# --------------------------------------------------------------------- refusals of the entry points --

def pointers():
    buf = torch.zeros(1 << 16, dtype=torch.uint8)
    base = (buf.data_ptr() + 255) // 256 * 256
    return buf, C.c_void_p(base), C.c_void_p(base + 4)


def refused(fn, args, **change):
    """Calls fn with the named arguments of `args` after `change` and expects a refusal."""
    assert set(change) <= set(args)
    assert fn(*{**args, **change}.values()) == BAD, change
    assert _lib.lib().pg_last_error_message()


def test_qk_norm_refusals():
    buf, p, odd = pointers()
    L = _lib.lib()
    fwd = dict(dtype=_lib.PG_BF16, T=4, hq=2, hkv=1, d=128, q=p, ldq=256, k=p, ldk=128, gq=p, gk=p,
               eps=1e-5, pos=p, theta=1e4, qo=p, ko=p, stream=None)
    for ch in [dict(dtype=2), dict(T=0), dict(T=1 << 31), dict(hq=-1), dict(hq=0, hkv=0), dict(d=96),
               dict(q=None), dict(k=odd), dict(gq=None), dict(gk=odd), dict(ldq=255), dict(ldq=128),
               dict(ldk=120), dict(eps=-1.0), dict(eps=math.nan), dict(theta=-1.0), dict(pos=None),
               dict(qo=None), dict(ko=odd)]:
        refused(L.pg_qk_norm_rope_fwd, fwd, **ch)
    need = L.pg_qk_norm_rope_bwd_workspace(4, 2, 1, 128)
    bwd = dict(dtype=_lib.PG_BF16, T=4, hq=2, hkv=1, d=128, q=p, ldq=256, k=p, ldk=128, gq=p, gk=p,
               eps=1e-5, dqo=p, dko=p, pos=p, theta=1e4, dq=p, dk=p, dgq=p, dgk=p, ws=p, nws=need,
               stream=None)
    for ch in [dict(dtype=-1), dict(d=32), dict(dqo=None), dict(dko=odd), dict(dq=odd), dict(dk=None),
               dict(dgq=None), dict(dgk=None), dict(ws=None), dict(ws=odd), dict(nws=need - 1),
               dict(pos=None)]:
        refused(L.pg_qk_norm_rope_bwd, bwd, **ch)


def test_append_refusals():
    buf, p, odd = pointers()
    ok = dict(dtype=_lib.PG_F32, n=3, hq=2, hkv=1, d=64, q=p, ldq=128, qo=p, k=p, ldk=64, v=p, ldv=64,
              positions=p, theta=1e4, kc=p, vc=p, num_pages=4, page_size=16, pages=p, rows=3,
              per_row=2, stride=2, page_rows=None, cache_pos=p, stream=None)
    for ch in [dict(dtype=7), dict(n=0), dict(hq=-1), dict(hkv=0), dict(d=80), dict(theta=-1.0),
               dict(theta=math.nan), dict(page_size=8), dict(page_size=48), dict(num_pages=0),
               dict(rows=0), dict(rows=2), dict(per_row=0), dict(stride=1), dict(k=None), dict(k=odd),
               dict(v=odd), dict(ldk=60), dict(ldk=66), dict(ldv=0), dict(kc=None), dict(vc=odd),
               dict(pages=None), dict(cache_pos=None), dict(q=None), dict(qo=None), dict(q=odd),
               dict(ldq=124), dict(ldq=64)]:
        refused(_lib.lib().pg_cache_append, ok, **ch)


def test_decode_refusals():
    buf, p, odd = pointers()
    st, tab = api.plan_decode_host([40], [2], 4, 2, 128, 16, 2)
    opts = lambda *a: C.byref(_lib.PgOpts(*a))
    ok = dict(plan=C.byref(st), q=p, kc=p, vc=p, num_pages=8, pp=p, pstride=3, op=p, ostride=2, lens=p,
              o=p, lse=p, opts=opts(0.0, 0.0, 0, 0), ws=p, nws=st.workspace_bytes, stream=None)
    empty = _lib.PgDecodePlan()
    for ch in [dict(plan=None), dict(plan=C.byref(empty)), dict(q=None), dict(kc=odd), dict(vc=None),
               dict(num_pages=0), dict(num_pages=-1), dict(num_pages=1 << 27), dict(pp=None),
               dict(pstride=2), dict(op=None), dict(ostride=1), dict(lens=None), dict(o=odd),
               dict(lse=None), dict(opts=opts(-1.0, 0.0, 0, 0)), dict(opts=opts(0.0, 1e4, 0, 0)),
               dict(opts=opts(0.0, 0.0, _lib.PG_FLAG_RESPONSES_ONLY, 0)),
               dict(opts=opts(0.0, 0.0, 0, 1)), dict(ws=None), dict(ws=odd),
               dict(nws=st.workspace_bytes - 1)]:
        refused(_lib.lib().pg_decode_attn, ok, **ch)


def test_sample_refusals():
    buf, p, odd = pointers()
    off = C.c_void_p(p.value + 1)
    ok = dict(dtype=_lib.PG_BF16, rows=2, vocab=10, logits=p, ld=10, u=p, t=p, k=p, tp=p, mp=p, tok=p,
              lp=p, stream=None)
    for ch in [dict(dtype=3), dict(rows=0), dict(rows=(1 << 24) + 1), dict(vocab=0),
               dict(vocab=(1 << 20) + 1), dict(ld=9), dict(logits=None), dict(logits=off), dict(u=None),
               dict(tok=None), dict(tok=off), dict(u=off), dict(k=off), dict(lp=off)]:
        refused(_lib.lib().pg_sample, ok, **ch)
    refused(_lib.lib().pg_sample, ok, dtype=_lib.PG_F32, logits=C.c_void_p(p.value + 2))


def test_binding_refuses_host_tensors():
    x = torch.zeros((2, 2, 64))
    idx = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.qk_norm_rope_fwd(x, x, x[0, 0], x[0, 0], 1e-5, idx)
    with pytest.raises(ValueError):
        api.cache_append(x, x, torch.zeros(2, 16, 2, 64), torch.zeros(2, 16, 2, 64), idx[:, None], idx)
    with pytest.raises(ValueError):
        api.sample(torch.zeros(2, 5), torch.zeros(2))

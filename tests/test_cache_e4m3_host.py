"""CPU checks of the cache in 8 bits: the oracle against torch's own e4m3 type, definitions and hand-made
blocks, the attention plan's share for it, and every refusal of the C entry points (host checks that return
before anything is launched) and of the binding."""
import ctypes as C
import math
import os
import shutil
import subprocess

import pytest
import torch

from oracle import rollout_oracle as ro
from shared_prefix_grouped_gb300 import _lib, api, rollout
from shared_prefix_grouped_gb300.build import build

BAD = _lib.PG_ERR_INVALID_ARG
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


# ------------------------------------------------------------------------------------- the oracle --

def test_rounding_is_the_types():
    # all codes, the midpoints of neighbours (ties to even) and what lies just beside them
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = (codes[1:] + codes[:-1]) / 2
    x = torch.cat([codes, mid, mid * (1 + 1e-5), mid * (1 - 1e-5)])
    x = torch.cat([x, -x])
    assert torch.equal(ro.e4m3_round(x), x.float().to(torch.float8_e4m3fn).double())
    assert bool(ro.e4m3_round(torch.tensor([math.inf, -math.inf, math.nan])).isnan().all())


def test_block_exponent():
    for e in (-126, -125, -3, 0, 5, 119):
        top = math.ldexp(448.0, e)
        assert ro.block_exponent(top) == e
        assert ro.block_exponent(top * (1 + 2 ** -23)) == e + 1
    assert ro.block_exponent(0.0) == -126 and ro.block_exponent(torch.finfo(torch.float32).max) == 120


def test_append_oracle_by_hand():
    codes = [torch.zeros((2, 16, 1, 64), dtype=torch.float64) for _ in range(2)]
    scales = [torch.zeros((2, 1, 1), dtype=torch.float64) for _ in range(2)]

    def step(value, cp):
        x = torch.zeros((1, 1, 64))
        x[..., 0] = value
        ro.append_e4m3(x, -x, codes, scales, torch.tensor([[1]]), torch.tensor([cp]), None, None, 0.0)

    step(440.0, 0)                       # below 448: scale 1; 440 is a tie of 416 and 448, 448 has the even code
    assert float(scales[0][1, 0, 0]) == 1 and codes[0][1, :2, 0, 0].tolist() == [448, 0]
    step(449.0, 1)                       # past it: scale 2, the earlier code halved
    assert float(scales[0][1, 0, 0]) == 2 and codes[0][1, :3, 0, 0].tolist() == [224, 224, 0]
    step(3.0, 2)                         # a scale stays
    assert float(scales[1][1, 0, 0]) == 2 and codes[1][1, :3, 0, 0].tolist() == [-224, -224, -1.5]
    assert float(scales[0][0].abs().max()) == 0 and float(codes[0][0].abs().max()) == 0
    step(1.0, 0)                         # a block is begun anew from its first slot on
    assert float(scales[0][1, 0, 0]) == 2.0 ** ro.block_exponent(1.0) == 2.0 ** -8
    assert float(codes[0][1, 0, 0, 0]) == 256


def test_attention_oracle_is_attention_over_the_values():
    g = torch.Generator().manual_seed(3)
    codes = [ro.e4m3_round(100 * torch.randn((6, 16, 2, 64), generator=g)) for _ in range(2)]
    scales = [2.0 ** torch.randint(-12, -4, (6, 1, 2), generator=g).double() for _ in range(2)]
    q = torch.randn((3, 4, 64), generator=g)
    pp, op = torch.tensor([[0, 1], [2, 0]]), torch.tensor([[3], [4], [5]])
    lens = torch.tensor([5, 0, 16])
    a = ro.decode_e4m3(q, codes, scales, [20, 0], [2, 1], pp, op, lens)
    k, v = (ro.cache_values(c, s) for c, s in zip(codes, scales))
    b = ro.decode(q, k, v, [20, 0], [2, 1], pp, op, lens)
    assert torch.allclose(a[0], b[0], atol=1e-12) and torch.allclose(a[1], b[1], atol=1e-12)
    assert bool((a[0].abs() <= a[2] * (1 + 1e-12)).all()) and bool((a[3] <= a[2] / 8 * (1 + 1e-12)).all())


# -------------------------------------------------------------------------------------- the plan --

@pytest.mark.parametrize("own_pages,page", [(1, 16), (64, 16), (65, 16), (100, 64), (64, 256), (4096, 16)])
def test_plan_gives_each_cta_few_own_keys(own_pages, page):
    st, _ = api.plan_decode_host([300, 17], [3, 1], 8, 2, 128, page, own_pages)
    keys = own_pages * page
    assert st.own_slots_e4m3 == min(max(st.own_slots, math.ceil(keys / 1024)), 16)
    # the workspace holds either form's partial results: an output row and its lse, fp32
    slots = st.prefix_slots + max(st.own_slots, st.own_slots_e4m3)
    assert st.workspace_bytes >= slots * st.num_seqs * st.heads_q * (128 + 1) * 4


C_PROGRAM = r"""
#include <stdio.h>
#include "pg_policy.h"
#include "pg_rollout.h"
int main(void) {
  pg_policy_opts o = {1.0f, 0.2f, 0.2f, 0.0f};
  printf("%d %d %d %d %d\n",
         pg_policy_loss(PG_BF16, 0, 8, 0, 8, 0, 0, 0, 0, 0, 0, 0, &o, 0, 0, 0, 0, 0, 0, 0, 0),
         pg_policy_loss_bwd(PG_BF16, 0, 8, 0, 8, 0, 0, 0, 1.0f, 0, 0, 0, 0, 0, 0),
         pg_cache_append_e4m3(PG_BF16, 0, 0, 1, 64, 0, 0, 0, 0, 64, 0, 64, 0, 0.0f, 0, 0, 0, 0, 1, 16, 0, 1, 1,
                              1, 0, 0, 0),
         pg_cache_read_e4m3(PG_BF16, 0, 1, 64, 0, 0, 0, 0, 1, 16, 0, 1, 1, 1, 0, 0, 0, 0, 0),
         pg_decode_attn_e4m3(0, 0, 0, 0, 0, 0, 1, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0));
  return 0;
}
"""


def test_headers_from_c(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    src, exe, libdir = tmp_path / "p.c", tmp_path / "p", os.path.dirname(_lib.LIB_PATH)
    src.write_text(C_PROGRAM)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                    os.path.join(ROOT, "include"), str(src), "-L", libdir, "-lpg_gb300",
                    f"-Wl,-rpath,{libdir}", "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in out] == [BAD] * 5


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


def test_append_refusals():
    buf, p, odd = pointers()
    ok = dict(dtype=_lib.PG_BF16, n=3, hq=2, hkv=1, d=64, q=p, ldq=128, qo=p, k=p, ldk=64, v=p, ldv=64,
              positions=p, theta=1e4, kc=p, vc=p, ks=p, vs=p, num_pages=4, page_size=16, pages=p, rows=3,
              per_row=2, stride=2, page_rows=None, cache_pos=p, stream=None)
    for ch in [dict(dtype=7), dict(n=0), dict(n=1 << 27), dict(hq=-1), dict(hkv=0), dict(hkv=65537), dict(d=80),
               dict(d=256), dict(theta=-1.0), dict(theta=math.nan), dict(page_size=8), dict(page_size=48),
               dict(page_size=512), dict(num_pages=0), dict(rows=0), dict(rows=2), dict(per_row=0),
               dict(stride=1), dict(k=None), dict(k=odd), dict(v=odd), dict(ldk=60), dict(ldk=66),
               dict(ldv=0), dict(kc=None), dict(kc=odd), dict(vc=odd), dict(ks=None), dict(ks=odd),
               dict(vs=None), dict(vs=odd), dict(pages=None), dict(cache_pos=None), dict(q=None),
               dict(qo=None), dict(q=odd), dict(qo=odd), dict(ldq=124), dict(ldq=64)]:
        refused(_lib.lib().pg_cache_append_e4m3, ok, **ch)


def test_read_refusals():
    buf, p, odd = pointers()
    ok = dict(dtype=_lib.PG_F32, n=3, hkv=1, d=64, kc=p, vc=p, ks=p, vs=p, num_pages=4, page_size=16, pages=p,
              rows=3, per_row=2, stride=2, page_rows=None, cache_pos=p, k=p, v=p, stream=None)
    for ch in [dict(dtype=2), dict(n=0), dict(n=1 << 27), dict(hkv=0), dict(d=32), dict(kc=None), dict(vc=odd),
               dict(ks=odd), dict(vs=None), dict(num_pages=0), dict(page_size=24), dict(pages=None),
               dict(rows=2), dict(per_row=0), dict(stride=1), dict(cache_pos=None), dict(k=None), dict(k=odd),
               dict(v=None), dict(v=odd)]:
        refused(_lib.lib().pg_cache_read_e4m3, ok, **ch)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_refusals(dtype):
    buf, p, odd = pointers()
    st, tab = api.plan_decode_host([40], [2], 4, 2, 128, 16, 2, dtype)
    opts = lambda *a: C.byref(_lib.PgOpts(*a))
    ok = dict(plan=C.byref(st), q=p, kc=p, vc=p, ks=p, vs=p, num_pages=8, pp=p, pstride=3, op=p, ostride=2,
              lens=p, o=p, lse=p, opts=opts(0.0, 0.0, 0, 0), ws=p, nws=st.workspace_bytes, stream=None)
    empty = _lib.PgDecodePlan()
    for ch in [dict(plan=None), dict(plan=C.byref(empty)), dict(q=None), dict(q=odd), dict(kc=odd),
               dict(vc=None), dict(ks=None), dict(ks=odd), dict(vs=None), dict(vs=odd), dict(num_pages=0),
               dict(num_pages=-1), dict(num_pages=1 << 27), dict(pp=None), dict(pstride=2), dict(op=None),
               dict(ostride=1), dict(lens=None), dict(o=odd), dict(lse=None),
               dict(opts=opts(-1.0, 0.0, 0, 0)), dict(opts=opts(0.0, 1e4, 0, 0)),
               dict(opts=opts(0.0, 0.0, _lib.PG_FLAG_RESPONSES_ONLY, 0)), dict(opts=opts(0.0, 0.0, 0, 1)),
               dict(ws=None), dict(ws=odd), dict(nws=st.workspace_bytes - 1)]:
        refused(_lib.lib().pg_decode_attn_e4m3, ok, **ch)


def test_binding_refuses_host_tensors():
    x = torch.zeros((2, 2, 64))
    idx = torch.zeros(2, dtype=torch.int32)
    c = api.scaled_cache(2, 16, 2, 64, device="cpu")
    assert c.codes.shape == (2, 16, 2, 64) and c.scales.shape == (2, 1, 2)
    with pytest.raises(ValueError):
        api.cache_append_e4m3(x, x, c, c, idx[:, None], idx)
    with pytest.raises(ValueError):
        api.cache_read_e4m3(c, c, idx[:, None], idx)


def test_rollout_refusals():
    # (refused before anything is allocated)
    for kw in (dict(cache_dtype=torch.float16), dict(cache_dtype=torch.float32),
               dict(cache_dtype=torch.float8_e5m2), dict(cache_dtype=torch.float8_e4m3fn, page_size=8)):
        with pytest.raises(ValueError):
            rollout.Rollout([16], [1], 2, 1, 64, 8, device="cpu", **kw)

"""The attention step reads what the append right before it wrote: thousands of tokens appended, the
step called at once, compared bit for bit with the same calls a synchronise apart; and how the step's
launches are ordered in a captured graph."""
import ctypes

import pytest
import torch

from shared_prefix_grouped_gb300 import _lib, api
from shared_prefix_grouped_gb300.build import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()


class Step:
    """An append of every prefix key, every own key and the step's own token (whose q it rotates), then
    the attention step over them.  `data` is read by the append; `load` puts other data there."""

    def __init__(self, plens, gsizes, own, hq, hk, d, ps):
        S, B = sum(gsizes), len(plens)
        wp, wo = (max(plens) + ps - 1) // ps, (own + ps - 1) // ps
        rows = max(wp, wo, 1)
        g = torch.Generator().manual_seed(1)
        perm = torch.randperm(B * wp + S * wo + 1, generator=g).to(torch.int32)
        # one table whose rows are the prefixes', then the responses'
        table = torch.zeros((B + S, rows), dtype=torch.int32)
        table[:B, :wp] = perm[:B * wp].view(B, wp)
        if wo:
            table[B:, :wo] = perm[B * wp:B * wp + S * wo].view(S, wo)
        lens = list(plens) + [own] * S
        row = [r for r, n in enumerate(lens) for _ in range(n)]
        pos = [i for n in lens for i in range(n)]
        # one token per response at the end: stored nowhere (a padding row), its q rotated
        row += [0] * S
        pos += [-1] * S
        cu = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        self.S, self.N, self.hq, self.hk, self.d = S, len(row), hq, hk, d
        self.rows, self.cache_pos = cu(row), cu(pos)
        self.positions = torch.where(self.cache_pos < 0, cu([max(plens) + own] * len(row)), self.cache_pos)
        self.table = table.cuda()
        self.pp = self.table[:B] if wp else None
        self.op = self.table[B:, :wo] if wo else None
        self.own_lens = cu([own] * S) if wo else None
        shape = (len(perm), ps, hk, d)
        self.kc, self.vc = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.x = torch.zeros((self.N, hq + 2 * hk, d), dtype=torch.bfloat16, device="cuda")
        self.q = torch.zeros((self.N, hq, d), dtype=torch.bfloat16, device="cuda")
        self.plan = api.plan_decode(plens, gsizes, hq, hk, d, ps, wo)
        self.ws = api.decode_workspace(self.plan)
        self.o = torch.zeros((S, hq, d), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.zeros((hq, S), device="cuda")

    def data(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return torch.randn(self.x.shape, generator=g, device="cuda").to(torch.bfloat16)

    def append(self):
        x, hq, hk = self.x, self.hq, self.hk
        api.cache_append(x[:, hq:hq + hk], x[:, hq + hk:], self.kc, self.vc, self.table, self.cache_pos,
                         page_rows=self.rows, q=x[:, :hq], positions=self.positions, rope_theta=1e4,
                         q_out=self.q)

    def attend(self):
        api.decode_attn(self.plan, self.q[-self.S:], self.kc, self.vc, self.pp, self.op, self.own_lens,
                        out=self.o, lse=self.lse, workspace=self.ws)


CASES = {
    "prefix_and_own": dict(plens=[2000, 1500], gsizes=[16, 9], own=130, hq=8, hk=2, d=128, ps=32),
    "d64": dict(plens=[3000], gsizes=[20], own=200, hq=8, hk=4, d=64, ps=64),
    "own_only": dict(plens=[0, 0], gsizes=[30, 10], own=150, hq=8, hk=2, d=128, ps=16),
    "prefix_only": dict(plens=[4000, 700], gsizes=[33, 2], own=0, hq=8, hk=2, d=128, ps=128),
}


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("case", CASES)
def test_append_then_step_at_once(case, graph):
    st = Step(**CASES[case])
    data = [st.data(s) for s in range(4)]
    want = []
    for x in data:
        st.x.copy_(x)
        torch.cuda.synchronize()
        st.append()
        torch.cuda.synchronize()
        st.attend()
        torch.cuda.synchronize()
        want.append((st.o.clone(), st.lse.clone()))
    assert not torch.equal(want[0][0], want[1][0])
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            st.append()
            st.attend()
    got = []
    for i in range(24):
        st.x.copy_(data[i % 4])
        if graph:
            g.replay()
        else:
            st.append()
            st.attend()
        got.append((st.o.clone(), st.lse.clone()))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 4][0]) and torch.equal(lse, want[i % 4][1]), i
    assert api.device_status() == _lib.PG_OK


class EdgeData(ctypes.Structure):
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte), ("type", ctypes.c_ubyte),
                ("reserved", ctypes.c_ubyte * 5)]


def edges(graph):
    """[(from, to, programmatic)] of a kept captured graph."""
    cu = ctypes.CDLL("libcuda.so.1")
    h, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetEdges_v2(h, None, None, None, ctypes.byref(n)) == 0
    src, dst, data = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (EdgeData * n.value)()
    assert cu.cuGraphGetEdges_v2(h, src, dst, data, ctypes.byref(n)) == 0
    return [(src[i], dst[i], data[i].type != 0) for i in range(n.value)]


@pytest.mark.parametrize("case,kernels,early", [("prefix_and_own", 4, [2, 3]), ("own_only", 3, [2]),
                                                ("prefix_only", 3, [2])])
def test_order_of_the_launches(case, kernels, early):
    # Append, then the step's kernels: the first one that reads what the append wrote starts after its
    # end, and so the append's writes are complete for every later one too; only the step's later kernels
    # may start beside the one before them.
    st = Step(**CASES[case])
    st.append()
    st.attend()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        st.append()
        st.attend()
    es = edges(g)
    after = {a: (b, p) for a, b, p in es}
    assert len(after) == len(es) == kernels - 1          # a chain
    node, got = (set(after) - {b for _, b, _ in es}).pop(), []
    while node in after:
        node, programmatic = after[node]
        got.append(programmatic)
    assert [i + 1 for i, p in enumerate(got) if p] == early

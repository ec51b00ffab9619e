"""Python binding of the grouped-attention C ABI.  Torch supplies device memory and streams only;
every step of the computation runs in the library's CUDA kernels.

    layout = pack(prefix_lens, group_sizes, suffix_lens)          # pg_pack
    o, lse = grouped_attn_fwd(layout, q, k, v, rope_theta=1e4)     # pg_grouped_attn_fwd
    dq, dk, dv = grouped_attn_bwd(layout, q, k, v, o, lse, do)    # pg_grouped_attn_bwd

Generating a group's responses (pg_rollout.h), one token per response and step:

    plan = plan_decode(prefix_lens, group_sizes, Hq, Hkv, d, page_size, own_pages, dtype)
    q = cache_append(k, v, k_cache, v_cache, own_pages, cache_pos, q=q, positions=pos, rope_theta=1e4)
    o, lse = decode_attn(plan, q, k_cache, v_cache, prefix_pages, own_pages, own_lens)
    tokens, logprobs = sample(logits, u, temperature=t, top_p=p)
"""
from __future__ import annotations

import ctypes as C
from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import PgDecodePlan, PgLayout, PgOpts, check, int_array

_DT = {torch.float32: _lib.PG_F32, torch.bfloat16: _lib.PG_BF16}


def _stream_ptr(device: torch.device) -> C.c_void_p:
    return C.c_void_p(torch.cuda.current_stream(device).cuda_stream)


class Layout:
    """A packed batch: the C layout struct plus the device buffers it points into."""

    def __init__(self, prefix_lens, group_sizes, suffix_lens, struct: PgLayout,
                 position_ids: torch.Tensor, tables: torch.Tensor):
        self.prefix_lens = list(prefix_lens)
        self.group_sizes = list(group_sizes)
        self.suffix_lens = list(suffix_lens)
        self.struct = struct
        self.position_ids = position_ids
        self.tables = tables

    @property
    def total_tokens(self) -> int:
        return int(self.struct.total_tokens)

    @property
    def pairs(self) -> int:
        return int(self.struct.pairs)


def pack_size(prefix_lens, group_sizes, suffix_lens):
    T, nb = C.c_int64(), C.c_int64()
    check("pg_pack_size", _lib.lib().pg_pack_size(
        len(prefix_lens), int_array(prefix_lens), int_array(group_sizes), int_array(suffix_lens),
        C.byref(T), C.byref(nb)))
    return T.value, nb.value


def pack_host(prefix_lens: Sequence[int], group_sizes: Sequence[int], suffix_lens: Sequence[int]):
    """Host-only packing (no CUDA): returns (position_ids int32 tensor, tables uint8 tensor, struct)."""
    T, nb = pack_size(prefix_lens, group_sizes, suffix_lens)
    pos = torch.empty(T, dtype=torch.int32)
    tab = torch.empty(nb, dtype=torch.uint8)
    st = PgLayout()
    check("pg_pack_host", _lib.lib().pg_pack_host(
        len(prefix_lens), int_array(prefix_lens), int_array(group_sizes), int_array(suffix_lens),
        C.cast(pos.data_ptr(), _lib.I32P), C.c_void_p(tab.data_ptr()), nb, C.byref(st)))
    return pos, tab, st


def pack(prefix_lens: Sequence[int], group_sizes: Sequence[int], suffix_lens: Sequence[int],
         device="cuda") -> Layout:
    device = torch.device(device)
    T, nb = pack_size(prefix_lens, group_sizes, suffix_lens)
    pos = torch.empty(T, dtype=torch.int32, device=device)
    tab = torch.empty(nb, dtype=torch.uint8, device=device)
    st = PgLayout()
    with torch.cuda.device(device):
        check("pg_pack", _lib.lib().pg_pack(
            len(prefix_lens), int_array(prefix_lens), int_array(group_sizes),
            int_array(suffix_lens), C.c_void_p(pos.data_ptr()), C.c_void_p(tab.data_ptr()), nb,
            C.byref(st), _stream_ptr(device)))
    return Layout(prefix_lens, group_sizes, suffix_lens, st, pos, tab)


def pack_tree_size(parent: Sequence[int], seg_lens: Sequence[int]):
    T, nb = C.c_int64(), C.c_int64()
    check("pg_pack_tree_size", _lib.lib().pg_pack_tree_size(
        len(parent), int_array(parent), int_array(seg_lens), C.byref(T), C.byref(nb)))
    return T.value, nb.value


def pack_tree_host(parent: Sequence[int], seg_lens: Sequence[int]):
    """Host-only packing of nested prefixes: (position_ids, tables, struct), as pack_host."""
    T, nb = pack_tree_size(parent, seg_lens)
    pos = torch.empty(T, dtype=torch.int32)
    tab = torch.empty(nb, dtype=torch.uint8)
    st = PgLayout()
    check("pg_pack_tree_host", _lib.lib().pg_pack_tree_host(
        len(parent), int_array(parent), int_array(seg_lens), C.cast(pos.data_ptr(), _lib.I32P),
        C.c_void_p(tab.data_ptr()), nb, C.byref(st)))
    return pos, tab, st


def pack_tree(parent: Sequence[int], seg_lens: Sequence[int], device="cuda") -> Layout:
    """Layout of nested prefixes: segments in depth-first preorder, parent[i] = -1 for a root."""
    device = torch.device(device)
    T, nb = pack_tree_size(parent, seg_lens)
    pos = torch.empty(T, dtype=torch.int32, device=device)
    tab = torch.empty(nb, dtype=torch.uint8, device=device)
    st = PgLayout()
    with torch.cuda.device(device):
        check("pg_pack_tree", _lib.lib().pg_pack_tree(
            len(parent), int_array(parent), int_array(seg_lens), C.c_void_p(pos.data_ptr()),
            C.c_void_p(tab.data_ptr()), nb, C.byref(st), _stream_ptr(device)))
    lay = Layout([], [], [], st, pos, tab)
    lay.tree = (list(parent), list(seg_lens))
    return lay


def _padded_args(num_groups, prefix_len, group_size, max_response_len, response_lens):
    assert len(response_lens) == num_groups * group_size
    return (int(num_groups), int(prefix_len), int(group_size), int(max_response_len),
            int_array(response_lens))


def pack_padded_size(num_groups: int, prefix_len: int, group_size: int, max_response_len: int,
                     response_lens: Sequence[int]):
    T, nb = C.c_int64(), C.c_int64()
    check("pg_pack_padded_size", _lib.lib().pg_pack_padded_size(
        *_padded_args(num_groups, prefix_len, group_size, max_response_len, response_lens),
        C.byref(T), C.byref(nb)))
    return T.value, nb.value


def pack_padded_host(num_groups: int, prefix_len: int, group_size: int, max_response_len: int,
                     response_lens: Sequence[int]):
    """Host-only padded packing: (position_ids, tables, struct), as pack_host."""
    T, nb = pack_padded_size(num_groups, prefix_len, group_size, max_response_len, response_lens)
    pos = torch.empty(T, dtype=torch.int32)
    tab = torch.empty(nb, dtype=torch.uint8)
    st = PgLayout()
    check("pg_pack_padded_host", _lib.lib().pg_pack_padded_host(
        *_padded_args(num_groups, prefix_len, group_size, max_response_len, response_lens),
        C.cast(pos.data_ptr(), _lib.I32P), C.c_void_p(tab.data_ptr()), nb, C.byref(st)))
    return pos, tab, st


def pack_padded(num_groups: int, prefix_len: int, group_size: int, max_response_len: int,
                response_lens: Sequence[int], device="cuda") -> Layout:
    """Layout of a padded batch [P; slot_1; ...; slot_G] per group (slots of max_response_len
    tokens, response i in the first response_lens[i] of its slot); attention calls on it write
    zeros (and lse = +inf) on the padding rows."""
    device = torch.device(device)
    T, nb = pack_padded_size(num_groups, prefix_len, group_size, max_response_len, response_lens)
    pos = torch.empty(T, dtype=torch.int32, device=device)
    tab = torch.empty(nb, dtype=torch.uint8, device=device)
    st = PgLayout()
    with torch.cuda.device(device):
        check("pg_pack_padded", _lib.lib().pg_pack_padded(
            *_padded_args(num_groups, prefix_len, group_size, max_response_len, response_lens),
            C.c_void_p(pos.data_ptr()), C.c_void_p(tab.data_ptr()), nb, C.byref(st),
            _stream_ptr(device)))
    return Layout([prefix_len] * num_groups, [group_size] * num_groups,
                  [max_response_len] * (num_groups * group_size), st, pos, tab)


def make_opts(rope_theta: float = 0.0, softmax_scale: float = 0.0, flags: int = 0,
              debug: int = 0) -> PgOpts:
    return PgOpts(float(softmax_scale), float(rope_theta), int(flags), int(debug))


def _dims(q: torch.Tensor, k: torch.Tensor):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [T, Hq, d] and k, v [T, Hkv, d]")
    return q.shape[1], k.shape[1], q.shape[2]


def _ptr(t: Optional[torch.Tensor]) -> C.c_void_p:
    return C.c_void_p(t.data_ptr() if t is not None else 0)


def _contig(*ts):
    for t in ts:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")


def workspace_size(layout: Layout, dtype: torch.dtype, Hq: int, Hkv: int, d: int, opts: PgOpts,
                   phase: int) -> int:
    n = C.c_size_t()
    check("pg_workspace_size", _lib.lib().pg_workspace_size(
        C.byref(layout.struct), _DT[dtype], Hq, Hkv, d, C.byref(opts), phase, C.byref(n)))
    return n.value


def _workspace(n: int, device) -> torch.Tensor:
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def grouped_attn_fwd(layout: Layout, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
                     rope_theta: float = 0.0, softmax_scale: float = 0.0, flags: int = 0,
                     debug: int = 0, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    Hq, Hkv, d = _dims(q, k)
    _contig(q, k, v)
    opts = make_opts(rope_theta, softmax_scale, flags, debug)
    T = layout.total_tokens
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = _workspace(workspace_size(layout, q.dtype, Hq, Hkv, d, opts, 0), q.device)
    with torch.cuda.device(q.device):
        check("pg_grouped_attn_fwd", _lib.lib().pg_grouped_attn_fwd(
            C.byref(layout.struct), _DT[q.dtype], Hq, Hkv, d, _ptr(q), _ptr(k), _ptr(v),
            _ptr(out), _ptr(lse), C.byref(opts), _ptr(workspace), workspace.numel(),
            _stream_ptr(q.device)))
    return out, lse


def grouped_attn_bwd(layout: Layout, q, k, v, o, lse, do, *, rope_theta: float = 0.0,
                     softmax_scale: float = 0.0, flags: int = 0, debug: int = 0,
                     dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                     dv: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None):
    Hq, Hkv, d = _dims(q, k)
    _contig(q, k, v, o, lse, do)
    opts = make_opts(rope_theta, softmax_scale, flags, debug)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = _workspace(workspace_size(layout, q.dtype, Hq, Hkv, d, opts, 1), q.device)
    with torch.cuda.device(q.device):
        check("pg_grouped_attn_bwd", _lib.lib().pg_grouped_attn_bwd(
            C.byref(layout.struct), _DT[q.dtype], Hq, Hkv, d, _ptr(q), _ptr(k), _ptr(v), _ptr(o),
            _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv), C.byref(opts), _ptr(workspace),
            workspace.numel(), _stream_ptr(q.device)))
    return dq, dk, dv


def rope_table(layout: Layout, dtype: torch.dtype, Hq: int, Hkv: int, d: int,
               workspace: torch.Tensor, *, rope_theta: float, flags: int) -> int:
    """Writes the cos/sin table of PG_FLAG_PRE_ROTATED into `workspace` (pg_rope_table) and
    returns its device address; flags must include PG_FLAG_PRE_ROTATED."""
    opts = make_opts(rope_theta, 0.0, flags)
    table = C.c_void_p()
    with torch.cuda.device(workspace.device):
        check("pg_rope_table", _lib.lib().pg_rope_table(
            C.byref(layout.struct), _DT[dtype], Hq, Hkv, d, C.byref(opts), _ptr(workspace),
            workspace.numel(), C.byref(table), _stream_ptr(workspace.device)))
    return int(table.value)


def gemm_bf16_rope(a: torch.Tensor, b: torch.Tensor, table: int, table_rows: int, head_dim: int,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bf16 [M, N] = a [M, K] @ b [N, K]^T with every head_dim-wide column block RoPE-rotated in
    the epilogue by the rows' (cos, sin) from `table` (pg_gemm_bf16_rope)."""
    if a.dtype != torch.bfloat16 or b.dtype != torch.bfloat16:
        raise ValueError("gemm_bf16_rope takes bf16 operands")
    _contig(a, b)
    M, K = a.shape
    N, Kb = b.shape
    if K != Kb:
        raise ValueError("inner dimensions differ")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    if out.dtype != torch.bfloat16 or out.dim() != 2 or out.stride(1) != 1 or out.shape != (M, N):
        raise ValueError("out must be a bf16 [M, N] matrix with unit column stride")
    with torch.cuda.device(a.device):
        check("pg_gemm_bf16_rope", _lib.lib().pg_gemm_bf16_rope(
            M, N, K, _ptr(a), a.shape[1], _ptr(b), b.shape[1], _ptr(out), out.stride(0), head_dim,
            C.c_void_p(table), table_rows, _stream_ptr(a.device)))
    return out


def device_status(clear: bool = True) -> int:
    """The kernels' status word (0 = ok); synchronous."""
    return int(_lib.lib().pg_device_status(1 if clear else 0))


def gemm_bf16(a: torch.Tensor, b: torch.Tensor, *, a_mn: bool = False, b_mn: bool = False,
              out_dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
              accumulate: bool = False):
    """C[m, n] = sum_k A(m, k) B(n, k) on the tensor cores (pg_gemm_bf16).

    a is [M, K] (a_mn False) or [K, M] (a_mn True); b is [N, K] (b_mn False) or [K, N] (True).
    """
    if a.dtype != torch.bfloat16 or b.dtype != torch.bfloat16:
        raise ValueError("gemm_bf16 takes bf16 operands")
    _contig(a, b)
    M, K = (a.shape[1], a.shape[0]) if a_mn else (a.shape[0], a.shape[1])
    N, Kb = (b.shape[1], b.shape[0]) if b_mn else (b.shape[0], b.shape[1])
    if K != Kb:
        raise ValueError("inner dimensions differ")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    if out.dim() != 2 or out.stride(1) != 1 or not out.is_cuda or out.shape != (M, N):
        raise ValueError("out must be a [M, N] CUDA matrix with unit column stride")
    with torch.cuda.device(a.device):
        check("pg_gemm_bf16", _lib.lib().pg_gemm_bf16(
            M, N, K, _ptr(a), int(a_mn), a.shape[1], _ptr(b), int(b_mn), b.shape[1], _ptr(out),
            _DT[out.dtype], out.stride(0), int(accumulate), _stream_ptr(a.device)))
    return out


def rmsnorm_fwd(x: torch.Tensor, gamma: torch.Tensor, eps: float, residual=None):
    """out = rmsnorm(x [+ residual]) * gamma; returns (out, y, rstd) with y the normalised input."""
    _contig(x, gamma)
    T, H = x.shape
    out = torch.empty_like(x)
    y = torch.empty_like(x) if residual is not None else x
    rstd = torch.empty(T, dtype=torch.float32, device=x.device)
    with torch.cuda.device(x.device):
        check("pg_rmsnorm_fwd", _lib.lib().pg_rmsnorm_fwd(
            T, H, _ptr(x), _ptr(residual), _ptr(gamma), float(eps), _ptr(out),
            _ptr(y if residual is not None else None), _ptr(rstd), _stream_ptr(x.device)))
    return out, y, rstd


def rmsnorm_bwd(y, gamma, rstd, dout, dres=None, dx_dtype=torch.bfloat16):
    """Returns (dx, dgamma)."""
    T, H = y.shape
    dx = torch.empty((T, H), dtype=dx_dtype, device=y.device)
    dgamma = torch.empty(H, dtype=torch.float32, device=y.device)
    L = _lib.lib()
    nws = L.pg_rmsnorm_bwd_workspace(T, H)
    ws = _workspace(nws, y.device)
    with torch.cuda.device(y.device):
        check("pg_rmsnorm_bwd", L.pg_rmsnorm_bwd(
            T, H, _ptr(y), _ptr(gamma), _ptr(rstd), _ptr(dout), _DT[dout.dtype], _ptr(dres),
            _ptr(dx), _DT[dx_dtype], _ptr(dgamma), _ptr(ws), ws.numel(), _stream_ptr(y.device)))
    return dx, dgamma


def swiglu_fwd(gate_up: torch.Tensor):
    T, I2 = gate_up.shape
    out = torch.empty((T, I2 // 2), dtype=gate_up.dtype, device=gate_up.device)
    with torch.cuda.device(gate_up.device):
        check("pg_swiglu_fwd", _lib.lib().pg_swiglu_fwd(T, I2 // 2, _ptr(gate_up), _ptr(out),
                                                         _stream_ptr(gate_up.device)))
    return out


def swiglu_bwd(gate_up: torch.Tensor, dout: torch.Tensor):
    T, I2 = gate_up.shape
    dgu = torch.empty_like(gate_up)
    with torch.cuda.device(gate_up.device):
        check("pg_swiglu_bwd", _lib.lib().pg_swiglu_bwd(T, I2 // 2, _ptr(gate_up), _ptr(dout),
                                                         _ptr(dgu), _stream_ptr(gate_up.device)))
    return dgu


# The calls from here on are made once per generated token: their checks are written to cost little when
# they pass, and addresses go to ctypes as plain numbers.

def _like(name: str, t: torch.Tensor, device, dtype, shape) -> None:
    """A contiguous tensor of exactly this device, dtype and shape."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    raise ValueError(f"{name} must be contiguous {dtype} {list(shape)} on {device}, got {t.dtype} "
                     f"{list(t.shape)} with strides {t.stride()} on {t.device}")


def _addr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _launch(where: str, device: torch.device, fn, *args) -> None:
    """fn(*args, stream) with `device` current and its current stream."""
    index = device.index
    stream = torch._C._cuda_getCurrentRawStream(index)    # current_stream(device).cuda_stream, 2 us less
    if torch.cuda.current_device() == index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status != _lib.PG_OK:
        check(where, status)


def _output(name: str, t: Optional[torch.Tensor], shape, dtype, device) -> torch.Tensor:
    """The given output, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _like(name, t, device, dtype, shape)
    return t


def _scratch(workspace: torch.Tensor, device) -> torch.Tensor:
    if workspace.dtype is not torch.uint8 or workspace.device != device or \
            not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    return workspace


def _token_rows(name: str, t: torch.Tensor):
    """[tokens, heads, d] with the heads of a token contiguous (a slice of a fused projection's
    output will do): returns its shape and the stride from token to token."""
    if t.dim() != 3 or not t.is_cuda or t.dtype not in _DT:
        raise ValueError(f"{name} must be a [tokens, heads, head_dim] f32 or bf16 CUDA tensor")
    shape = t.shape
    n, h, d = shape
    sn, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return shape, sn if n > 1 else h * d


def _index(name: str, t: Optional[torch.Tensor], device, n: int) -> Optional[int]:
    """The address of an int32 [n] tensor, or None."""
    if t is None:
        return None
    _like(name, t, device, torch.int32, (n,))
    return t.data_ptr()


def _qk(q: torch.Tensor, k: torch.Tensor, gain_q, gain_k):
    """q's shape, k's shape, their dtype and device, and the call's arguments up to the gains."""
    qs, ldq = _token_rows("q", q)
    ks, ldk = _token_rows("k", k)
    dt, dev, d = q.dtype, q.device, qs[2]
    if ks[0] != qs[0] or ks[2] != d or k.dtype is not dt or k.device != dev:
        raise ValueError("q and k must agree in tokens, head_dim, dtype and device")
    _like("gain_q", gain_q, dev, dt, (d,))
    _like("gain_k", gain_k, dev, dt, (d,))
    return qs, ks, dt, dev, (_DT[dt], qs[0], qs[1], ks[1], d, q.data_ptr(), ldq, k.data_ptr(), ldk,
                             gain_q.data_ptr(), gain_k.data_ptr())


def qk_norm_rope_fwd(q: torch.Tensor, k: torch.Tensor, gain_q: torch.Tensor, gain_k: torch.Tensor,
                     eps: float, positions: Optional[torch.Tensor] = None, *,
                     rope_theta: float = 0.0, q_out: Optional[torch.Tensor] = None,
                     k_out: Optional[torch.Tensor] = None):
    """RMSNorm of every head of q [T, Hq, d] and k [T, Hkv, d] with its gain, and the rotation at
    `positions` (int32 [T], e.g. Layout.position_ids), in one pass: returns (q_out, k_out)."""
    qs, ks, dt, dev, args = _qk(q, k, gain_q, gain_k)
    pos = _index("positions", positions, dev, qs[0])
    q_out = _output("q_out", q_out, qs, dt, dev)
    k_out = _output("k_out", k_out, ks, dt, dev)
    _launch("pg_qk_norm_rope_fwd", dev, _lib.lib().pg_qk_norm_rope_fwd, *args, float(eps), pos,
            float(rope_theta), q_out.data_ptr(), k_out.data_ptr())
    return q_out, k_out


def qk_norm_rope_bwd(q: torch.Tensor, k: torch.Tensor, gain_q: torch.Tensor, gain_k: torch.Tensor,
                     eps: float, dq_out: torch.Tensor, dk_out: torch.Tensor,
                     positions: Optional[torch.Tensor] = None, *, rope_theta: float = 0.0,
                     workspace: Optional[torch.Tensor] = None):
    """Returns (dq, dk, dgain_q, dgain_k), the gains' gradients in fp32; dq_out and dk_out are the
    gradients of the forward's outputs (with rope_theta 0: already rotated back)."""
    qs, ks, dt, dev, args = _qk(q, k, gain_q, gain_k)
    T, Hq, d = qs
    pos = _index("positions", positions, dev, T)
    _like("dq_out", dq_out, dev, dt, qs)
    _like("dk_out", dk_out, dev, dt, ks)
    L = _lib.lib()
    dq = torch.empty(qs, dtype=dt, device=dev)
    dk = torch.empty(ks, dtype=dt, device=dev)
    # the call writes nothing for a tensor without heads
    dgq = (torch.empty if Hq else torch.zeros)(d, dtype=torch.float32, device=dev)
    dgk = (torch.empty if ks[1] else torch.zeros)(d, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _workspace(L.pg_qk_norm_rope_bwd_workspace(T, Hq, ks[1], d), dev)
    _launch("pg_qk_norm_rope_bwd", dev, L.pg_qk_norm_rope_bwd, *args, float(eps), dq_out.data_ptr(),
            dk_out.data_ptr(), pos, float(rope_theta), dq.data_ptr(), dk.data_ptr(), dgq.data_ptr(),
            dgk.data_ptr(), _scratch(workspace, dev).data_ptr(), workspace.numel())
    return dq, dk, dgq, dgk


def _cache(k_cache: torch.Tensor, v_cache: torch.Tensor, device, dtype, heads: int, d: int):
    """(pages, page_size) of a pair of caches [pages, page_size, heads, d]."""
    shape = k_cache.shape
    if len(shape) != 4 or shape[2] != heads or shape[3] != d:
        raise ValueError(f"k_cache must be [pages, page_size, {heads}, {d}], got {list(shape)}")
    _like("k_cache", k_cache, device, dtype, shape)
    _like("v_cache", v_cache, device, dtype, shape)
    return shape[0], shape[1]


def _page_table(name: str, t: torch.Tensor, device):
    """int32 [rows, pages] with unit column stride: returns its shape and row stride."""
    if t.dim() != 2 or t.dtype is not torch.int32 or t.device != device:
        raise ValueError(f"{name} must be an int32 [rows, pages] matrix on {device}")
    rows, width = t.shape
    sr, sc = t.stride()
    if sc != 1 and width > 1:
        raise ValueError(f"{name} must have unit column stride")
    return rows, width, sr if rows > 1 else max(width, 1)


def cache_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 pages: torch.Tensor, cache_pos: torch.Tensor, *,
                 page_rows: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                 positions: Optional[torch.Tensor] = None, rope_theta: float = 0.0,
                 q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Store k (rotated at `positions`, default `cache_pos`) and v [N, Hkv, d] at index cache_pos[n]
    of row page_rows[n] (default n) of `pages`; a negative cache_pos stores nothing.  Returns q
    [N, Hq, d] rotated at the same positions, if given."""
    ks, ldk = _token_rows("k", k)
    vs, ldv = _token_rows("v", v)
    N, Hkv, d = ks
    dt, dev = k.dtype, k.device
    if vs != ks or v.dtype is not dt or v.device != dev:
        raise ValueError("k and v must agree in shape, dtype and device")
    num_pages, page_size = _cache(k_cache, v_cache, dev, dt, Hkv, d)
    rows, width, stride = _page_table("pages", pages, dev)
    Hq, ldq, q_ptr, out_ptr = 0, 0, None, None
    if q is not None:
        qs, ldq = _token_rows("q", q)
        Hq = qs[1]
        if qs[0] != N or qs[2] != d or q.dtype is not dt or q.device != dev:
            raise ValueError("q and k must agree in tokens, head_dim, dtype and device")
        q_out = _output("q_out", q_out, qs, dt, dev)
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    _launch("pg_cache_append", dev, _lib.lib().pg_cache_append, _DT[dt], N, Hq, Hkv, d, q_ptr, ldq,
            out_ptr, k.data_ptr(), ldk, v.data_ptr(), ldv, _index("positions", positions, dev, N),
            float(rope_theta), k_cache.data_ptr(), v_cache.data_ptr(), num_pages, page_size,
            pages.data_ptr(), rows, width, stride, _index("page_rows", page_rows, dev, N),
            _index("cache_pos", cache_pos, dev, N))
    return q_out if q is not None else None


class DecodePlan:
    """The attention step of a rollout: the C plan plus the device buffer it points into."""

    def __init__(self, struct: PgDecodePlan, tables: torch.Tensor):
        self.struct = struct
        self.tables = tables
        self.dtype = torch.float32 if struct.dtype == _lib.PG_F32 else torch.bfloat16
        self.device = tables.device

    @property
    def num_seqs(self) -> int:
        return int(self.struct.num_seqs)


def _plan_args(prefix_lens, group_sizes, heads_q, heads_kv, head_dim, page_size, own_pages, dtype):
    if len(prefix_lens) != len(group_sizes):
        raise ValueError("prefix_lens and group_sizes must have one entry per group")
    if dtype not in _DT:
        raise ValueError("dtype must be torch.float32 or torch.bfloat16")
    return (len(prefix_lens), int_array(prefix_lens), int_array(group_sizes), _DT[dtype],
            int(heads_q), int(heads_kv), int(head_dim), int(page_size), int(own_pages))


def plan_decode_host(prefix_lens: Sequence[int], group_sizes: Sequence[int], heads_q: int,
                     heads_kv: int, head_dim: int, page_size: int, own_pages: int,
                     dtype: torch.dtype = torch.bfloat16):
    """Host-only plan (no CUDA): (struct, tables uint8 tensor)."""
    args = _plan_args(prefix_lens, group_sizes, heads_q, heads_kv, head_dim, page_size, own_pages,
                      dtype)
    nb = C.c_int64()
    check("pg_plan_decode_size", _lib.lib().pg_plan_decode_size(*args, C.byref(nb)))
    tab, st = torch.empty(nb.value, dtype=torch.uint8), PgDecodePlan()
    check("pg_plan_decode_host", _lib.lib().pg_plan_decode_host(
        *args, C.c_void_p(tab.data_ptr()), nb.value, C.byref(st)))
    return st, tab


def plan_decode(prefix_lens: Sequence[int], group_sizes: Sequence[int], heads_q: int,
                heads_kv: int, head_dim: int, page_size: int, own_pages: int,
                dtype: torch.dtype = torch.bfloat16, device="cuda") -> DecodePlan:
    """Plan of the attention steps of one rollout: group b's group_sizes[b] responses share a prefix
    of prefix_lens[b] keys; a response holds up to own_pages * page_size keys of its own."""
    device = torch.device(device)
    args = _plan_args(prefix_lens, group_sizes, heads_q, heads_kv, head_dim, page_size, own_pages,
                      dtype)
    nb = C.c_int64()
    check("pg_plan_decode_size", _lib.lib().pg_plan_decode_size(*args, C.byref(nb)))
    tab, st = torch.empty(nb.value, dtype=torch.uint8, device=device), PgDecodePlan()
    with torch.cuda.device(device):
        check("pg_plan_decode", _lib.lib().pg_plan_decode(
            *args, C.c_void_p(tab.data_ptr()), nb.value, C.byref(st), _stream_ptr(device)))
    return DecodePlan(st, tab)


def decode_workspace(plan: DecodePlan) -> torch.Tensor:
    """A workspace for decode_attn with this plan."""
    return _workspace(int(plan.struct.workspace_bytes), plan.device)


def decode_attn(plan: DecodePlan, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                prefix_pages: Optional[torch.Tensor], own_pages: Optional[torch.Tensor],
                own_lens: Optional[torch.Tensor], *, softmax_scale: float = 0.0, flags: int = 0,
                out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None):
    """Attention of one query token per response, q [S, Hq, d], over its group's prefix (row b of
    prefix_pages) and its own first own_lens[s] keys (row s of own_pages): returns (o [S, Hq, d],
    lse fp32 [Hq, S])."""
    st, dev, dt = plan.struct, plan.device, plan.dtype
    S, Hq, d = st.num_seqs, st.heads_q, st.head_dim
    _like("q", q, dev, dt, (S, Hq, d))
    num_pages, page_size = _cache(k_cache, v_cache, dev, dt, st.heads_kv, d)
    if page_size != st.page_size:
        raise ValueError(f"the plan is for pages of {st.page_size}, the cache has {page_size}")
    pstride = ostride = 0
    if prefix_pages is not None:
        rows, width, pstride = _page_table("prefix_pages", prefix_pages, dev)
        if rows < st.num_groups or width * page_size < st.max_prefix:
            raise ValueError("prefix_pages must have a row per group that covers its prefix")
    if own_pages is not None:
        rows, width, ostride = _page_table("own_pages", own_pages, dev)
        if rows < S or width < st.own_pages:
            raise ValueError("own_pages must have a row of the plan's own_pages per response")
    out = _output("out", out, (S, Hq, d), dt, dev)
    lse = _output("lse", lse, (Hq, S), torch.float32, dev)
    workspace = decode_workspace(plan) if workspace is None else _scratch(workspace, dev)
    opts = C.byref(make_opts(0.0, softmax_scale, flags)) if softmax_scale or flags else None
    _launch("pg_decode_attn", dev, _lib.lib().pg_decode_attn, C.byref(st), q.data_ptr(),
            k_cache.data_ptr(), v_cache.data_ptr(), num_pages, _addr(prefix_pages), pstride,
            _addr(own_pages), ostride, _index("own_lens", own_lens, dev, S), out.data_ptr(),
            lse.data_ptr(), opts, workspace.data_ptr(), workspace.numel())
    return out, lse


def sample(logits: torch.Tensor, u: torch.Tensor, *, temperature: Optional[torch.Tensor] = None,
           top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
           min_p: Optional[torch.Tensor] = None, tokens: Optional[torch.Tensor] = None,
           logprobs: Optional[torch.Tensor] = None):
    """One token per row of logits [S, V] (f32 or bf16, unit column stride) from the random numbers u
    in [0, 1); temperature, top_p, min_p fp32 [S], top_k int32 [S].  Returns (tokens int32 [S],
    log-probabilities fp32 [S] at the row's temperature, before the filters)."""
    if logits.dim() != 2 or not logits.is_cuda or logits.dtype not in _DT or \
            (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be an f32 or bf16 [rows, vocab] CUDA matrix with unit column "
                         "stride")
    S, V = logits.shape
    dev = logits.device

    def per_row(name, t):
        if t is None:
            return None
        _like(name, t, dev, torch.float32, (S,))
        return t.data_ptr()

    if u is None:
        raise ValueError("u, the rows' random numbers, is needed")
    tokens = _output("tokens", tokens, (S,), torch.int32, dev)
    logprobs = _output("logprobs", logprobs, (S,), torch.float32, dev)
    _launch("pg_sample", dev, _lib.lib().pg_sample, _DT[logits.dtype], S, V, logits.data_ptr(),
            logits.stride(0) if S > 1 else V, per_row("u", u), per_row("temperature", temperature),
            _index("top_k", top_k, dev, S), per_row("top_p", top_p), per_row("min_p", min_p),
            tokens.data_ptr(), logprobs.data_ptr())
    return tokens, logprobs

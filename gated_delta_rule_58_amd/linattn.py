"""ctypes binding of kda_linattn.h (same names as the C entry points, without
the kda_ prefix): linear attention with one decay per head, and layer norm."""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Tuple

import torch

from .binding import KDA_F32, _check, _dt, _i32, _i64, _ptr, _stream, _vp, lib

_int, _f32, _size = ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_SIGNATURES = {
    "kda_linattn_chunk_prefill": (_int, [
        _vp, _i64, _vp, _i64, _vp, _i64, _int, _vp, _i64, _vp, _vp, _i32, _vp, _vp, _int, _i64,
        _vp, _vp, _int, _i64, _i32, _i32, _i32, _i32, _f32, _vp, _size, _vp]),
    "kda_linattn_chunk_prefill_workspace_bytes": (_size, [_i64, _i32, _i32, _i32, _i32]),
    "kda_linattn_chunk_prefill_backward": (_int, [
        _vp, _i64, _vp, _i64, _vp, _i64, _int, _vp, _i64, _vp, _vp, _i32, _vp, _vp, _int, _vp,
        _vp, _vp, _vp, _int, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _f32, _vp, _size, _vp]),
    "kda_linattn_chunk_prefill_backward_workspace_bytes": (
        _size, [_i64, _i32, _i32, _i32, _i32, _i32]),
    "kda_linattn_recurrent_decode": (_int, [
        _vp, _i64, _vp, _i64, _vp, _i64, _int, _vp, _i64, _vp, _int, _i64, _vp, _vp, _int, _i32,
        _i32, _i32, _i32, _i32, _f32, _vp]),
    "kda_zero_rows_behind": (_int, [_vp, _i32, _i64, _vp, _vp, _i32, _vp]),
    "kda_layernorm": (_int, [_vp, _int, _vp, _vp, _i64, _vp, _int, _i64, _i32, _f32, _vp]),
    "kda_layernorm_backward": (_int, [_vp, _int, _vp, _int, _vp, _i64, _vp, _vp, _vp, _i64, _i32,
                                      _f32, _vp, _size, _vp]),
    "kda_layernorm_backward_workspace_bytes": (_size, [_i64, _i64, _i32]),
}
_FNS = {}


def _fn(name: str):
    """The library's entry point, its signature declared on first use."""
    f = _FNS.get(name)
    if f is None:
        f = getattr(lib(), name)
        f.restype, f.argtypes = _SIGNATURES[name]
        _FNS[name] = f
    return f


def _on(dev: torch.device):
    """Makes dev the current device for a call on its stream."""
    if dev.index is None or dev.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _same_device(dev: torch.device, **tensors):
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU (got %s)" % dev)
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError("%s is on %s, not on %s" % (name, t.device, dev))


def _shape(name: str, t: Optional[torch.Tensor], *shape):
    if t is not None and tuple(t.shape) != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))


def _dtype(name: str, t: Optional[torch.Tensor], *dtypes):
    if t is not None and t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (
            name, " or ".join(str(d).replace("torch.", "") for d in dtypes), t.dtype))


def _row_stride(name: str, t: torch.Tensor) -> int:
    """Elements between the rows of [rows, heads, dim], whose heads and channels are dense."""
    rows, h, d = t.shape
    if d > 1 and t.stride(2) != 1 or h > 1 and t.stride(1) != d:
        raise ValueError("%s: the heads and channels of a token must be dense" % name)
    return t.stride(0) if rows > 1 else h * d


def _inputs(q, k, v, g):
    """Checks what the three linear attention calls share; (rows, H, Hk, dk, dv)."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [tokens, heads, dim]")
    rows, Hk, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    _shape("k", k, rows, Hk, dk)
    _shape("v", v, rows, H, dv)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must have one dtype")
    _dtype("g", g, torch.float32)
    if tuple(g.shape) not in ((rows, H), (H,)):
        raise ValueError("g must be [%d, %d] or [%d], got %s" % (rows, H, H, list(g.shape)))
    return rows, H, Hk, dk, dv


def _sequences(rows, cu_seqlens, cu_seqlens_host, num_seqs):
    """(N, host pointer keeper): the packed batch's sequences."""
    if cu_seqlens is None:
        if cu_seqlens_host is not None:
            raise ValueError("cu_seqlens_host needs cu_seqlens")
        return num_seqs, None
    _dtype("cu_seqlens", cu_seqlens, torch.int32)
    N = cu_seqlens.numel() - 1
    if cu_seqlens_host is None:
        return N, None
    _dtype("cu_seqlens_host", cu_seqlens_host, torch.int32)
    if cu_seqlens_host.device.type != "cpu" or cu_seqlens_host.numel() != N + 1:
        raise ValueError("cu_seqlens_host must be cu_seqlens on the CPU")
    return N, cu_seqlens_host.contiguous()


def _host_ptr(t):
    return None if t is None else ctypes.cast(t.data_ptr(), _vp)


def zero_rows_behind(cu_seqlens: torch.Tensor, *tensors: torch.Tensor):
    """kda_zero_rows_behind: zeros the rows of up to four [T, ...] tensors that lie behind the
    last sequence (from cu_seqlens[N] on), without waiting for cu_seqlens on the host."""
    _dtype("cu_seqlens", cu_seqlens, torch.int32)
    if not tensors:
        return
    dev, T, n = cu_seqlens.device, tensors[0].shape[0], len(tensors)
    for t in tensors:
        _same_device(dev, tensor=t)
        if t.dim() < 1 or t.shape[0] != T:
            raise ValueError("the tensors must have the same number of rows")
    ptrs = (_vp * n)(*[_ptr(t) for t in tensors])
    sizes = (_i64 * n)(*[t.numel() // max(T, 1) * t.element_size() for t in tensors])
    with _on(dev):
        st = _fn("kda_zero_rows_behind")(_ptr(cu_seqlens), cu_seqlens.numel() - 1, T, ptrs, sizes,
                                         n, _stream(dev))
    _check(st)


def linattn_chunk_prefill_workspace_bytes(T_tot: int, N: int, H: int, dk: int = 128,
                                          dv: int = 128) -> int:
    """kda_linattn_chunk_prefill_workspace_bytes."""
    return int(_fn("kda_linattn_chunk_prefill_workspace_bytes")(T_tot, N, H, dk, dv))


def linattn_chunk_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                          cu_seqlens: Optional[torch.Tensor] = None,
                          initial_state: Optional[torch.Tensor] = None,
                          output_final_state: bool = True, scale: float = 1.0,
                          o_dtype: Optional[torch.dtype] = None,
                          out: Optional[torch.Tensor] = None,
                          final_state: Optional[torch.Tensor] = None,
                          cu_seqlens_host: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None,
                          state_indices: Optional[torch.Tensor] = None,
                          state_dtype: Optional[torch.dtype] = None, num_seqs: int = 1):
    """kda_linattn_chunk_prefill: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.

    q, k [T, Hk, dk], v [T, H, dv] (rows may be strided), g float32 [T, H] or [H].
    cu_seqlens int32 [N+1] on the device; None: num_seqs sequences of T / num_seqs
    tokens.  cu_seqlens_host (optional) is checked and sizes the work; nothing is
    copied or waited for when it is missing.  States are [N, H, dk, dv] float32 or
    bfloat16, or with state_indices (int32 [N] on the device) pools
    [num_slots, H, dk, dv], in which final_state (possibly initial_state itself) is
    written only when passed.  workspace: uint8; None allocates what the library asks for.
    Rows behind the last sequence (cu_seqlens[N] < T, which needs cu_seqlens_host to be
    missing) stay as they were in `out`, and are zeros when out is None.
    Returns (o [T, H, dv], final state or None)."""
    T, H, Hk, dk, dv = _inputs(q, k, v, g)
    dev = q.device
    _same_device(dev, k=k, v=v, g=g, cu_seqlens=cu_seqlens, initial_state=initial_state, out=out,
                 final_state=final_state, workspace=workspace, state_indices=state_indices)
    N, hp = _sequences(T, cu_seqlens, cu_seqlens_host, num_seqs)
    if state_dtype is None:
        state_dtype = initial_state.dtype if initial_state is not None else (
            final_state.dtype if final_state is not None else torch.float32)
    if state_indices is not None:
        _dtype("state_indices", state_indices, torch.int32)
        _shape("state_indices", state_indices, N)
        output_final_state = False  # a pool is written only when passed as final_state
    new_out = out is None
    if new_out:
        out = torch.empty((T, H, dv), dtype=o_dtype or q.dtype, device=dev)
    _shape("out", out, T, H, dv)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, dk, dv), dtype=state_dtype, device=dev)
    pools = [t for t in (initial_state, final_state) if t is not None]
    num_slots = pools[0].shape[0] if pools else N
    for t in pools:
        _dtype("a state", t, state_dtype)
        _shape("a state", t, num_slots, H, dk, dv)
    if workspace is None:
        nbytes = linattn_chunk_prefill_workspace_bytes(T, N, H, dk, dv)
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    with _on(dev):
        st = _fn("kda_linattn_chunk_prefill")(
            q.data_ptr(), _row_stride("q", q), k.data_ptr(), _row_stride("k", k), v.data_ptr(),
            _row_stride("v", v), _dt(q), _ptr(g), g.numel(), _ptr(cu_seqlens), _host_ptr(hp), N,
            _ptr(initial_state), _ptr(final_state),
            _dt(pools[0]) if pools else KDA_F32, num_slots, _ptr(state_indices), _ptr(out),
            _dt(out), T, H, Hk, dk, dv, float(scale), _ptr(workspace),
            workspace.numel() * workspace.element_size() if workspace is not None else 0,
            _stream(dev))
    _check(st)
    if new_out and cu_seqlens is not None and hp is None:
        zero_rows_behind(cu_seqlens, out)
    return out, final_state


def linattn_chunk_prefill_backward_workspace_bytes(T_tot: int, N: int, H: int, Hk: int,
                                                   dk: int = 128, dv: int = 128) -> int:
    """kda_linattn_chunk_prefill_backward_workspace_bytes."""
    return int(_fn("kda_linattn_chunk_prefill_backward_workspace_bytes")(T_tot, N, H, Hk, dk, dv))


def linattn_chunk_prefill_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                   g: torch.Tensor, d_o: Optional[torch.Tensor],
                                   cu_seqlens: Optional[torch.Tensor] = None,
                                   initial_state: Optional[torch.Tensor] = None,
                                   d_final_state: Optional[torch.Tensor] = None,
                                   scale: float = 1.0, want_d_initial_state: bool = True,
                                   grad_dtype: Optional[torch.dtype] = None,
                                   cu_seqlens_host: Optional[torch.Tensor] = None,
                                   workspace: Optional[torch.Tensor] = None, num_seqs: int = 1):
    """kda_linattn_chunk_prefill_backward: gradients of linattn_chunk_prefill's (o,
    final state) against d_o [T, H, dv] (None: zero) and d_final_state (None: zero).
    The gradients of rows behind the last sequence (cu_seqlens[N] < T, which needs
    cu_seqlens_host to be missing) are zeros.

    Returns (dq, dk [T, Hk, dk], dv [T, H, dv] in grad_dtype (default: q's), dg in g's
    shape, float32, d_initial_state [N, H, dk, dv] float32 or None)."""
    T, H, Hk, dk, dv = _inputs(q, k, v, g)
    dev = q.device
    _same_device(dev, k=k, v=v, g=g, d_o=d_o, cu_seqlens=cu_seqlens, initial_state=initial_state,
                 d_final_state=d_final_state, workspace=workspace)
    N, hp = _sequences(T, cu_seqlens, cu_seqlens_host, num_seqs)
    _shape("d_o", d_o, T, H, dv)
    for name, t in (("initial_state", initial_state), ("d_final_state", d_final_state)):
        _dtype(name, t, torch.float32)
        _shape(name, t, N, H, dk, dv)
    gdt = grad_dtype or q.dtype
    dq = torch.empty((T, Hk, dk), dtype=gdt, device=dev)
    dk_ = torch.empty((T, Hk, dk), dtype=gdt, device=dev)
    dv_ = torch.empty((T, H, dv), dtype=gdt, device=dev)
    dg = torch.empty(tuple(g.shape), dtype=torch.float32, device=dev)
    dS0 = (torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
           if want_d_initial_state else None)
    if workspace is None:
        nbytes = linattn_chunk_prefill_backward_workspace_bytes(T, N, H, Hk, dk, dv)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    with _on(dev):
        st = _fn("kda_linattn_chunk_prefill_backward")(
            q.data_ptr(), _row_stride("q", q), k.data_ptr(), _row_stride("k", k), v.data_ptr(),
            _row_stride("v", v), _dt(q), _ptr(g), g.numel(), _ptr(cu_seqlens), _host_ptr(hp), N,
            _ptr(initial_state), _ptr(d_o), _dt(d_o) if d_o is not None else _dt(q),
            _ptr(d_final_state), _ptr(dq), _ptr(dk_), _ptr(dv_), _dt(dq), _ptr(dg), _ptr(dS0), T,
            H, Hk, dk, dv, float(scale), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(dev))
    _check(st)
    if cu_seqlens is not None and hp is None:
        zero_rows_behind(cu_seqlens, dq, dk_, dv_, *([dg] if g.dim() == 2 else []))
    return dq, dk_, dv_, dg, dS0


def linattn_recurrent_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                             state: torch.Tensor, state_indices: Optional[torch.Tensor] = None,
                             scale: float = 1.0, o_dtype: Optional[torch.dtype] = None,
                             out: Optional[torch.Tensor] = None):
    """kda_linattn_recurrent_decode: q, k [N, Hk, dk], v [N, H, dv] (rows may be strided),
    g float32 [N, H] or [H]; state pool [num_slots, H, dk, dv] (float32 or bfloat16) updated
    in place; state_indices int32 [N] on the device (None: sequence n uses slot n).
    Returns o (zeros for sequences whose slot is outside the pool)."""
    N, H, Hk, dk, dv = _inputs(q, k, v, g)
    dev = q.device
    _same_device(dev, k=k, v=v, g=g, state=state, state_indices=state_indices, out=out)
    if state_indices is not None:
        _dtype("state_indices", state_indices, torch.int32)
        _shape("state_indices", state_indices, N)
    if state.dim() != 4 or tuple(state.shape[1:]) != (H, dk, dv):
        raise ValueError("state must be [num_slots, %d, %d, %d], got %s" % (H, dk, dv,
                                                                           list(state.shape)))
    if out is None:
        out = torch.empty((N, H, dv), dtype=o_dtype or q.dtype, device=dev)
    _shape("out", out, N, H, dv)
    with _on(dev):
        st = _fn("kda_linattn_recurrent_decode")(
            q.data_ptr(), _row_stride("q", q), k.data_ptr(), _row_stride("k", k), v.data_ptr(),
            _row_stride("v", v), _dt(q), _ptr(g), g.numel(), _ptr(state), _dt(state),
            state.shape[0], _ptr(state_indices), _ptr(out), _dt(out), N, H, Hk, dk, dv,
            float(scale), _stream(dev))
    _check(st)
    return out


def _norm_rows(x: torch.Tensor, weight, bias) -> Tuple[int, int, int]:
    """(rows, groups, d): weight [d], or [H, d] for x [..., H, d]."""
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    d = x.shape[-1]
    if d == 0:
        raise ValueError("x must have channels")
    groups = 1
    for name, t in (("weight", weight), ("bias", bias)):
        _dtype(name, t, torch.float32)
    w = weight if weight is not None else bias
    if w is not None and w.dim() == 2:
        if x.dim() < 2 or tuple(w.shape) != tuple(x.shape[-2:]):
            raise ValueError("weight must be [%d] or x's last two dimensions, got %s" % (
                d, list(w.shape)))
        groups = w.shape[0]
    elif w is not None:
        _shape("weight", w, d)
    if weight is not None and bias is not None:
        _shape("bias", bias, *weight.shape)
    return x.numel() // d, max(groups, 1), d


def layernorm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
              bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
              out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None):
    """kda_layernorm over the last dimension of x [..., d] (float32 or bfloat16); weight
    and bias float32 [d], or [H, d] for x [..., H, d] (every head its own), or None.
    out may be x (in place).  Returns the normalised tensor."""
    rows, groups, d = _norm_rows(x, weight, bias)
    dev = x.device
    _same_device(dev, weight=weight, bias=bias, out=out)
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=dev)
    _shape("out", out, *x.shape)
    with _on(dev):
        st = _fn("kda_layernorm")(_ptr(x), _dt(x), _ptr(weight), _ptr(bias), groups, _ptr(out),
                                  _dt(out), rows, d, float(eps), _stream(dev))
    _check(st)
    return out


def layernorm_backward_workspace_bytes(rows: int, groups: int, d: int) -> int:
    """kda_layernorm_backward_workspace_bytes."""
    return int(_fn("kda_layernorm_backward_workspace_bytes")(rows, groups, d))


def layernorm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                       eps: float = 1e-5, want_dbias: bool = True,
                       workspace: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None):
    """kda_layernorm_backward: gradients of layernorm(x, weight, bias, eps) against dy.
    bias: its values do not matter; without a weight it says that there is one, and
    dbias gets its shape.

    Returns (dx in x's dtype, dweight, dbias), the last two float32 in weight's (bias's)
    shape (dweight None without a weight, dbias without either or unless want_dbias)."""
    rows, groups, d = _norm_rows(x, weight, bias)
    dev = x.device
    _same_device(dev, dy=dy, weight=weight, bias=bias, workspace=workspace)
    _shape("dy", dy, *x.shape)
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    affine = weight if weight is not None else bias
    dw = None if weight is None else torch.empty(weight.shape, dtype=torch.float32, device=dev)
    db = (torch.empty(affine.shape, dtype=torch.float32, device=dev)
          if affine is not None and want_dbias else None)
    if workspace is None and (dw is not None or db is not None):
        nbytes = layernorm_backward_workspace_bytes(rows, groups, d)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    with _on(dev):
        st = _fn("kda_layernorm_backward")(
            _ptr(dy), _dt(dy), _ptr(x), _dt(x), _ptr(weight), groups, _ptr(dx), _ptr(dw),
            _ptr(db), rows, d, float(eps), _ptr(workspace),
            workspace.numel() * workspace.element_size() if workspace is not None else 0,
            _stream(dev))
    _check(st)
    return dx, dw, db

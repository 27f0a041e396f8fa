"""ctypes binding of kda_gatedrec.h (same names as the C entry points, without the kda_
prefix): gated linear recurrence, and RMS norm."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .binding import KDA_F32, _check, _dt, _i32, _i64, _ptr, _vp, lib
from .linattn import (_dtype, _host_ptr, _norm_rows, _on, _same_device, _sequences, _shape,
                      zero_rows_behind)

_int, _f32, _size = ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ROWS = [_vp, _i64, _vp, _i64, _vp, _i64, _int, _vp, _vp, _i32]  # x, r, i, dtype, the gate
_SIGNATURES = {
    "kda_gatedrec_scan": (_int, _ROWS + [
        _vp, _vp, _i32, _vp, _vp, _int, _i64, _vp, _vp, _int, _vp, _i64, _i32, _vp, _size, _vp]),
    "kda_gatedrec_scan_workspace_bytes": (_size, [_i64, _i32]),
    "kda_gatedrec_starts_bytes": (_size, [_i64, _i32]),
    "kda_gatedrec_scan_backward": (_int, _ROWS + [
        _vp, _vp, _i32, _vp, _vp, _vp, _int, _vp, _vp, _vp, _vp, _int, _vp, _vp, _vp, _i64, _i32,
        _vp, _size, _vp]),
    "kda_gatedrec_scan_backward_workspace_bytes": (_size, [_i64, _i32, _i32]),
    "kda_gatedrec_decode": (_int, _ROWS + [_vp, _int, _i64, _vp, _vp, _int, _i32, _i32, _vp]),
    "kda_rmsnorm": (_int, [_vp, _int, _i64, _vp, _vp, _int, _vp, _i64, _vp, _int, _i64, _i32, _f32,
                           _vp]),
    "kda_rmsnorm_e4m3": (_int, [_vp, _int, _i64, _vp, _vp, _int, _vp, _i64, _vp, _vp, _i32, _i64,
                                _i32, _f32, _vp]),
    "kda_rmsnorm_backward": (_int, [_vp, _int, _vp, _int, _i64, _vp, _i64, _vp, _vp, _vp, _i64,
                                    _i32, _f32, _vp, _size, _vp]),
    "kda_rmsnorm_backward_workspace_bytes": (_size, [_i64, _i64, _i32]),
}
_FNS = {}
_E4M3 = torch.float8_e4m3fn
STARTS_TOKENS = 32  # tokens between two states of `starts`


def _fn(name: str):
    """The library's entry point, its signature declared on first use."""
    f = _FNS.get(name)
    if f is None:
        f = getattr(lib(), name)
        f.restype, f.argtypes = _SIGNATURES[name]
        _FNS[name] = f
    return f


def _stream(dev: torch.device) -> int:
    """The current stream's handle, without a Stream object around it (0.1 us for 2)."""
    return torch._C._cuda_getCurrentRawStream(
        torch.cuda.current_device() if dev.index is None else dev.index)


def _inputs(x, r, i, A_log, dt_bias):
    """Checks what the recurrence's calls share; (rows, C)."""
    if x.dim() != 2:
        raise ValueError("x, r and i must be [tokens, channels]")
    rows, C = x.shape
    for name, t in (("r", r), ("i", i)):
        _shape(name, t, rows, C)
        if t is not None and t.dtype != x.dtype:
            raise TypeError("x, r and i must have one dtype")
    for name, t in (("A_log", A_log), ("dt_bias", dt_bias)):
        _dtype(name, t, torch.float32)
        _shape(name, t, C)
    return rows, C


def _rows(x, r, i, A_log, dt_bias, normalize):
    """The first arguments of the recurrence's calls."""
    out = []
    for name, t in (("x", x), ("r", r), ("i", i)):
        if t is None:
            out += [None, 0]
            continue
        rows, C = t.shape
        if C > 1 and t.stride(1) != 1:
            raise ValueError("%s: the channels of a token must be dense" % name)
        out += [t.data_ptr(), t.stride(0) if rows > 1 else C]
    return out + [_dt(x), _ptr(A_log), _ptr(dt_bias), 1 if normalize else 0]


def _new_rows(T, C, dtype, dev, behind):
    """A new [T, C] output; (tensor, whether its rows behind the last sequence still have to be
    cleared, which the library does for rows of whole 4 bytes)."""
    if behind and C * dtype.itemsize % 4:
        return torch.zeros((T, C), dtype=dtype, device=dev), False
    return torch.empty((T, C), dtype=dtype, device=dev), behind


def gatedrec_scan_workspace_bytes(T_tot: int, C: int) -> int:
    """kda_gatedrec_scan_workspace_bytes."""
    return int(_fn("kda_gatedrec_scan_workspace_bytes")(T_tot, C))


def gatedrec_scan(x: torch.Tensor, r: torch.Tensor, i: Optional[torch.Tensor] = None,
                  A_log: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
                  normalize: bool = False, cu_seqlens: Optional[torch.Tensor] = None,
                  initial_state: Optional[torch.Tensor] = None, output_final_state: bool = True,
                  output_starts: bool = False, h_dtype: Optional[torch.dtype] = None,
                  out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
                  starts: Optional[torch.Tensor] = None,
                  cu_seqlens_host: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None,
                  state_indices: Optional[torch.Tensor] = None,
                  state_dtype: Optional[torch.dtype] = None, num_seqs: int = 1):
    """kda_gatedrec_scan: h_t = exp(g_t) h_{t-1} + m_t sigmoid(i_t) x_t per channel, with
    g = -exp(A_log) softplus(r + dt_bias) (A_log None: g = r, which must not be above 0; where it
    is the kernels take 0, and KDA_DEBUG=1 refuses it) and m = sqrt(1 - exp(2 g)) if normalize,
    else 1.

    x, r and i [T, C] (float32 or bfloat16; rows may be strided; i None: no input gate),
    A_log and dt_bias float32 [C].  cu_seqlens int32 [N+1] on the device; None: num_seqs
    sequences of T / num_seqs tokens.  cu_seqlens_host (optional) is checked; nothing is
    copied or waited for when it is missing.  States are [N, C] float32 or bfloat16, or with
    state_indices (int32 [N] on the device) pools [num_slots, C], in which final_state
    (possibly initial_state itself) is written only when passed.  output_starts: also return
    the states that gatedrec_scan_backward wants (`starts`: a tensor for them, float32
    [ceil(T / 32), C]).  workspace:
    uint8; None allocates what the library asks for.  Rows behind the last sequence
    (cu_seqlens[N] < T, which needs cu_seqlens_host to be missing) stay as they were in
    `out`, and are zeros when out is None.
    Returns (h [T, C], final state or None, starts or None)."""
    T, C = _inputs(x, r, i, A_log, dt_bias)
    dev = x.device
    _same_device(dev, r=r, i=i, A_log=A_log, dt_bias=dt_bias, cu_seqlens=cu_seqlens,
                 initial_state=initial_state, out=out, final_state=final_state, starts=starts,
                 workspace=workspace, state_indices=state_indices)
    N, hp = _sequences(T, cu_seqlens, cu_seqlens_host, num_seqs)
    if state_dtype is None:
        state_dtype = initial_state.dtype if initial_state is not None else (
            final_state.dtype if final_state is not None else torch.float32)
    if state_indices is not None:
        _dtype("state_indices", state_indices, torch.int32)
        _shape("state_indices", state_indices, N)
        output_final_state = False  # a pool is written only when passed as final_state
    clear = False
    if out is None:
        out, clear = _new_rows(T, C, h_dtype or x.dtype, dev, cu_seqlens is not None and hp is None)
    _shape("out", out, T, C)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, C), dtype=state_dtype, device=dev)
    pools = [t for t in (initial_state, final_state) if t is not None]
    num_slots = pools[0].shape[0] if pools else N
    for t in pools:
        _dtype("a state", t, state_dtype)
        _shape("a state", t, num_slots, C)
    if starts is None and output_starts:
        starts = torch.empty((-(-T // STARTS_TOKENS), C), dtype=torch.float32, device=dev)
    _dtype("starts", starts, torch.float32)
    _shape("starts", starts, -(-T // STARTS_TOKENS), C)
    if workspace is None:
        nbytes = gatedrec_scan_workspace_bytes(T, C)
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    with _on(dev):
        st = _fn("kda_gatedrec_scan")(
            *_rows(x, r, i, A_log, dt_bias, normalize), _ptr(cu_seqlens), _host_ptr(hp), N,
            _ptr(initial_state), _ptr(final_state), _dt(pools[0]) if pools else KDA_F32, num_slots,
            _ptr(state_indices), _ptr(out), _dt(out), _ptr(starts), T, C, _ptr(workspace),
            workspace.numel() * workspace.element_size() if workspace is not None else 0,
            _stream(dev))
    _check(st)
    if clear:
        zero_rows_behind(cu_seqlens, out)
    return out, final_state, starts


def gatedrec_scan_backward_workspace_bytes(T_tot: int, C: int, has_starts: bool = True) -> int:
    """kda_gatedrec_scan_backward_workspace_bytes."""
    return int(_fn("kda_gatedrec_scan_backward_workspace_bytes")(T_tot, C, 1 if has_starts else 0))


def gatedrec_scan_backward(x: torch.Tensor, r: torch.Tensor, i: Optional[torch.Tensor],
                           dh: Optional[torch.Tensor], A_log: Optional[torch.Tensor] = None,
                           dt_bias: Optional[torch.Tensor] = None, normalize: bool = False,
                           cu_seqlens: Optional[torch.Tensor] = None,
                           initial_state: Optional[torch.Tensor] = None,
                           d_final_state: Optional[torch.Tensor] = None,
                           starts: Optional[torch.Tensor] = None,
                           want_d_initial_state: bool = True,
                           grad_dtype: Optional[torch.dtype] = None,
                           cu_seqlens_host: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, num_seqs: int = 1):
    """kda_gatedrec_scan_backward: gradients of gatedrec_scan's (h, final state) against dh
    [T, C] (None: zero) and d_final_state [N, C] (None: zero).  starts: what gatedrec_scan
    returned for the same inputs with output_starts; None forms those states again.  The
    gradients of rows behind the last sequence (cu_seqlens[N] < T, which needs cu_seqlens_host
    to be missing) are zeros.

    Returns (dx, dr, di [T, C] in grad_dtype (default: x's; di None without i), dA_log,
    ddt_bias float32 [C] (None without A_log, dt_bias), d_initial_state float32 [N, C] or
    None)."""
    T, C = _inputs(x, r, i, A_log, dt_bias)
    dev = x.device
    _same_device(dev, r=r, i=i, A_log=A_log, dt_bias=dt_bias, dh=dh, cu_seqlens=cu_seqlens,
                 initial_state=initial_state, d_final_state=d_final_state, starts=starts,
                 workspace=workspace)
    N, hp = _sequences(T, cu_seqlens, cu_seqlens_host, num_seqs)
    _shape("dh", dh, T, C)
    for name, t, rows in (("initial_state", initial_state, N), ("d_final_state", d_final_state, N),
                          ("starts", starts, -(-T // STARTS_TOKENS))):
        _dtype(name, t, torch.float32)
        _shape(name, t, rows, C)
    behind = cu_seqlens is not None and hp is None
    grads, clear = [], []
    for t in (x, r, i):
        g, c = (None, False) if t is None else _new_rows(T, C, grad_dtype or x.dtype, dev, behind)
        grads.append(g)
        clear += [g] if c else []
    dA = None if A_log is None else torch.empty(C, dtype=torch.float32, device=dev)
    db = None if dt_bias is None else torch.empty(C, dtype=torch.float32, device=dev)
    dS0 = torch.empty((N, C), dtype=torch.float32, device=dev) if want_d_initial_state else None
    if workspace is None:
        nbytes = gatedrec_scan_backward_workspace_bytes(T, C, starts is not None)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    with _on(dev):
        st = _fn("kda_gatedrec_scan_backward")(
            *_rows(x, r, i, A_log, dt_bias, normalize), _ptr(cu_seqlens), _host_ptr(hp), N,
            _ptr(initial_state), _ptr(starts), _ptr(dh), _dt(dh) if dh is not None else _dt(x),
            _ptr(d_final_state), _ptr(grads[0]), _ptr(grads[1]), _ptr(grads[2]), _dt(grads[0]),
            _ptr(dA), _ptr(db), _ptr(dS0), T, C, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(dev))
    _check(st)
    if clear:
        zero_rows_behind(cu_seqlens, *clear)
    return grads[0], grads[1], grads[2], dA, db, dS0


def gatedrec_decode(x: torch.Tensor, r: torch.Tensor, i: Optional[torch.Tensor],
                    state: torch.Tensor, A_log: Optional[torch.Tensor] = None,
                    dt_bias: Optional[torch.Tensor] = None, normalize: bool = False,
                    state_indices: Optional[torch.Tensor] = None,
                    h_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None):
    """kda_gatedrec_decode: one token per sequence, x, r and i [N, C] (rows may be strided),
    state pool [num_slots, C] (float32 or bfloat16) updated in place; state_indices int32 [N]
    on the device (None: sequence n uses slot n).
    Returns h [N, C] (zeros for sequences whose slot is outside the pool)."""
    N, C = _inputs(x, r, i, A_log, dt_bias)
    dev = x.device
    _same_device(dev, r=r, i=i, A_log=A_log, dt_bias=dt_bias, state=state,
                 state_indices=state_indices, out=out)
    if state_indices is not None:
        _dtype("state_indices", state_indices, torch.int32)
        _shape("state_indices", state_indices, N)
    if state.dim() != 2 or state.shape[1] != C:
        raise ValueError("state must be [num_slots, %d], got %s" % (C, list(state.shape)))
    if out is None:
        out = torch.empty((N, C), dtype=h_dtype or x.dtype, device=dev)
    _shape("out", out, N, C)
    with _on(dev):
        st = _fn("kda_gatedrec_decode")(
            *_rows(x, r, i, A_log, dt_bias, normalize), _ptr(state), _dt(state), state.shape[0],
            _ptr(state_indices), _ptr(out), _dt(out), N, C, _stream(dev))
    _check(st)
    return out


def _token_stride(name: str, x: torch.Tensor, groups: int, d: int) -> int:
    """Elements between the tokens of x, whose rows [groups, d] are dense."""
    if x.is_contiguous():
        return groups * d
    lead = x.dim() - (2 if groups > 1 else 1)  # dimensions of tokens
    if lead != 1 or (d > 1 and x.stride(-1) != 1) or (groups > 1 and x.stride(-2) != d):
        raise ValueError("%s must be contiguous, or [tokens, ...] with dense rows" % name)
    return x.stride(0) if x.shape[0] > 1 else groups * d


def _norm_inputs(x, weight, residual, residual_out):
    """(rows, groups, d, s): s is where x + residual goes (None without a residual)."""
    rows, groups, d = _norm_rows(x, weight, None)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
        return rows, groups, d, None
    _shape("residual", residual, *x.shape)
    _dtype("residual", residual, x.dtype, torch.float32)
    if residual_out is None:
        residual_out = torch.empty(x.shape, dtype=residual.dtype, device=x.device)
    _shape("residual_out", residual_out, *x.shape)
    _dtype("residual_out", residual_out, residual.dtype)
    return rows, groups, d, residual_out


def rmsnorm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
            residual: Optional[torch.Tensor] = None, eps: float = 1e-5,
            out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
            residual_out: Optional[torch.Tensor] = None):
    """kda_rmsnorm over the last dimension of s = x + residual (s = x without one): x [..., d]
    float32 or bfloat16, its tokens possibly strided; residual in x's dtype or float32;
    weight float32 [d], or [H, d] for x [..., H, d] (every head its own), or None.  out may
    be x, residual_out residual or x (in place).
    Returns (y, s as it is stored, in residual's dtype, or None without a residual)."""
    rows, groups, d, s = _norm_inputs(x, weight, residual, residual_out)
    dev = x.device
    _same_device(dev, weight=weight, residual=residual, out=out, residual_out=residual_out)
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=dev)
    _shape("out", out, *x.shape)
    with _on(dev):
        st = _fn("kda_rmsnorm")(x.data_ptr(), _dt(x), _token_stride("x", x, groups, d),
                                _ptr(residual), _ptr(s), _dt(residual) if s is not None else _dt(x),
                                _ptr(weight), groups, _ptr(out), _dt(out), rows, d, float(eps),
                                _stream(dev))
    _check(st)
    return out, s


def rmsnorm_e4m3(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                 residual: Optional[torch.Tensor] = None, eps: float = 1e-5,
                 scale_group: int = 128, out: Optional[torch.Tensor] = None,
                 scales: Optional[torch.Tensor] = None,
                 residual_out: Optional[torch.Tensor] = None):
    """kda_rmsnorm_e4m3: rmsnorm with y in 8 bits (torch.float8_e4m3fn) and a float32 scale for
    each 128 columns of a row (scale_group 128) or for the row (scale_group 0).
    Returns (y, scales [..., ceil(d / 128)] or [..., 1], s or None): y * scale is the norm."""
    rows, groups, d, s = _norm_inputs(x, weight, residual, residual_out)
    dev = x.device
    _same_device(dev, weight=weight, residual=residual, out=out, residual_out=residual_out,
                 scales=scales)
    if out is None:
        out = torch.empty(x.shape, dtype=_E4M3, device=dev)
    _dtype("out", out, _E4M3)
    _shape("out", out, *x.shape)
    per_row = 1 if scale_group == 0 else -(-d // 128)
    if scales is None:
        scales = torch.empty((*x.shape[:-1], per_row), dtype=torch.float32, device=dev)
    _dtype("scales", scales, torch.float32)
    _shape("scales", scales, *x.shape[:-1], per_row)
    with _on(dev):
        st = _fn("kda_rmsnorm_e4m3")(
            x.data_ptr(), _dt(x), _token_stride("x", x, groups, d), _ptr(residual), _ptr(s),
            _dt(residual) if s is not None else _dt(x), _ptr(weight), groups, _ptr(out),
            _ptr(scales), scale_group, rows, d, float(eps), _stream(dev))
    _check(st)
    return out, scales, s


def rmsnorm_backward_workspace_bytes(rows: int, groups: int, d: int) -> int:
    """kda_rmsnorm_backward_workspace_bytes."""
    return int(_fn("kda_rmsnorm_backward_workspace_bytes")(rows, groups, d))


def rmsnorm_backward(dy: torch.Tensor, s: torch.Tensor, weight: Optional[torch.Tensor] = None,
                     d_residual: Optional[torch.Tensor] = None, eps: float = 1e-5,
                     workspace: Optional[torch.Tensor] = None):
    """kda_rmsnorm_backward: gradients of rmsnorm against dy, from s (what rmsnorm returned with
    a residual, else x).  d_residual (s's dtype): the gradient that reaches s from where the
    residual stream goes on; it is added.

    Returns (dx in s's dtype, which is the gradient of x and of residual, dweight float32 in
    weight's shape or None)."""
    rows, groups, d = _norm_rows(s, weight, None)
    dev = s.device
    _same_device(dev, dy=dy, weight=weight, d_residual=d_residual, workspace=workspace)
    _shape("dy", dy, *s.shape)
    _shape("d_residual", d_residual, *s.shape)
    _dtype("d_residual", d_residual, s.dtype)
    dx = torch.empty(s.shape, dtype=s.dtype, device=dev)
    dw = None if weight is None else torch.empty(weight.shape, dtype=torch.float32, device=dev)
    if workspace is None and dw is not None:
        nbytes = rmsnorm_backward_workspace_bytes(rows, groups, d)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    with _on(dev):
        st = _fn("kda_rmsnorm_backward")(
            _ptr(dy), _dt(dy), s.data_ptr(), _dt(s), _token_stride("s", s, groups, d),
            _ptr(weight), groups, _ptr(d_residual), _ptr(dx), _ptr(dw), rows, d, float(eps),
            _ptr(workspace), workspace.numel() * workspace.element_size()
            if workspace is not None else 0, _stream(dev))
    _check(st)
    return dx, dw

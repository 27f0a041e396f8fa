"""ctypes binding of libkda.so (same names as the C entry points)."""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

KDA_F32 = 0
KDA_BF16 = 1
_STATUS = {0: "KDA_OK", 1: "KDA_ERR_INVALID_ARG", 2: "KDA_ERR_SHAPE", 3: "KDA_ERR_DTYPE",
           4: "KDA_ERR_UNSUPPORTED", 5: "KDA_ERR_ALIGNMENT", 6: "KDA_ERR_WORKSPACE",
           7: "KDA_ERR_LAUNCH", 8: "KDA_ERR_DOMAIN", 9: "KDA_ERR_NONFINITE"}
# default cap on the prefill workspace the binding allocates (the chunk axis is
# processed in passes when a batch needs more)
DEFAULT_WORKSPACE_BYTES = 1 << 30
CHUNK = 64
KDA_ACT_NONE = 0
KDA_ACT_SILU = 1

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64


class KdaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (_STATUS.get(status, str(status)), message))
        self.status = status


def lib_path() -> str:
    return os.path.join(_HERE, "libkda.so")


def lib():
    """Load libkda.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise ImportError("libkda.so not built: run __graft_entry__.build() or "
                              "python gated_delta_rule_58_amd/build.py")
        L = ctypes.CDLL(path)
        L.kda_last_error.restype = ctypes.c_char_p
        L.kda_last_error.argtypes = []
        L.kda_version.restype = ctypes.c_char_p
        L.kda_version.argtypes = []
        L.kda_gate.restype = ctypes.c_int
        L.kda_gate.argtypes = [_vp, ctypes.c_int, _vp, ctypes.c_int, _vp, _i64, _vp, _i64, _vp,
                               _vp, _i64, _i32, _i32, _vp]
        L.kda_chunk_prefill.restype = ctypes.c_int
        L.kda_chunk_prefill.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _vp, _i32,
                                        _vp, _vp, _vp, ctypes.c_int, _i64, _i32, _i32, _i32,
                                        ctypes.c_float, _vp, ctypes.c_size_t, _vp]
        L.kda_chunk_prefill_gated.restype = ctypes.c_int
        L.kda_chunk_prefill_gated.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, ctypes.c_int, _vp,
                                              ctypes.c_int, _vp, _i64, _vp, _i64, _vp, _vp, _i32,
                                              _vp, _vp, ctypes.c_int, _i64, _vp, _vp, ctypes.c_int,
                                              _i64, _i32, _i32, _i32, ctypes.c_float, _vp,
                                              ctypes.c_size_t, _vp]
        L.kda_chunk_prefill_gated_static.restype = ctypes.c_int
        L.kda_chunk_prefill_gated_static.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp,
                                                     ctypes.c_int, _vp, ctypes.c_int, _vp, _i64,
                                                     _vp, _i64, _vp, _vp, _i32, _vp, _vp,
                                                     ctypes.c_int, _i64, _vp, _vp, ctypes.c_int,
                                                     _i64, _i32, _i32, _i32, ctypes.c_float, _vp]
        L.kda_chunk_prefill_workspace_bytes.restype = ctypes.c_size_t
        L.kda_chunk_prefill_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32]
        L.kda_recurrent_decode_gated.restype = ctypes.c_int
        L.kda_recurrent_decode_gated.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, ctypes.c_int,
                                                 _vp, ctypes.c_int, _vp, _i64, _vp, _i64, _vp,
                                                 ctypes.c_int, _i64, _vp, _vp, ctypes.c_int,
                                                 _i32, _i32, _i32, _i32, ctypes.c_float, _vp]
        L.kda_shortconv_l2norm.restype = ctypes.c_int
        L.kda_shortconv_l2norm.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _i64,
                                           _i32, ctypes.c_float, _vp, _vp, _i32, _vp, _vp, _vp,
                                           _vp, _vp, ctypes.c_int, _i64, _i32, _i32, _vp]
        L.kda_gate_backward.restype = ctypes.c_int
        L.kda_gate_backward.argtypes = [_vp, ctypes.c_int, _vp, ctypes.c_int, _vp, _i64, _vp,
                                        _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32,
                                        _vp, ctypes.c_size_t, _vp]
        L.kda_gate_backward_workspace_bytes.restype = ctypes.c_size_t
        L.kda_gate_backward_workspace_bytes.argtypes = [_i64, _i32, _i32]
        L.kda_chunk_prefill_backward.restype = ctypes.c_int
        L.kda_chunk_prefill_backward.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _vp,
                                                 _i32, _vp, _vp, ctypes.c_int, _vp, _vp, _vp,
                                                 _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32,
                                                 ctypes.c_float, _vp, ctypes.c_size_t, _vp]
        L.kda_chunk_prefill_backward_workspace_bytes.restype = ctypes.c_size_t
        L.kda_chunk_prefill_backward_workspace_bytes.argtypes = [_i64, _i32, _i32, _i32, _i32]
        L.kda_recurrent_decode.restype = ctypes.c_int
        L.kda_recurrent_decode.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _vp,
                                           ctypes.c_int, _i32, _i32, _i32, _i32, ctypes.c_float,
                                           _vp]
        _LIB = L
    return _LIB


def exported_symbols():
    return ["kda_last_error", "kda_version", "kda_gate", "kda_chunk_prefill",
            "kda_chunk_prefill_gated", "kda_chunk_prefill_gated_static",
            "kda_chunk_prefill_workspace_bytes", "kda_recurrent_decode",
            "kda_recurrent_decode_gated", "kda_shortconv_l2norm", "kda_chunk_prefill_backward",
            "kda_chunk_prefill_backward_workspace_bytes", "kda_gate_backward",
            "kda_gate_backward_workspace_bytes", "kda_linattn_chunk_prefill",
            "kda_linattn_chunk_prefill_workspace_bytes", "kda_linattn_chunk_prefill_backward",
            "kda_linattn_chunk_prefill_backward_workspace_bytes", "kda_linattn_recurrent_decode",
            "kda_zero_rows_behind", "kda_layernorm", "kda_layernorm_backward", "kda_layernorm_backward_workspace_bytes",
            "kda_gatedrec_scan", "kda_gatedrec_scan_workspace_bytes", "kda_gatedrec_starts_bytes",
            "kda_gatedrec_scan_backward", "kda_gatedrec_scan_backward_workspace_bytes",
            "kda_gatedrec_decode", "kda_rmsnorm", "kda_rmsnorm_e4m3", "kda_rmsnorm_backward",
            "kda_rmsnorm_backward_workspace_bytes"]


def _check(status: int):
    if status != 0:
        raise KdaError(status, lib().kda_last_error().decode())


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return KDA_F32
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    raise TypeError("unsupported dtype %s (float32 or bfloat16)" % t.dtype)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _alog(A_log: torch.Tensor, H: int, d: int) -> torch.Tensor:
    """A_log as the library takes it: [H] per head, or [H, d] per (head, channel).
    A 2-D tensor of another shape is refused here (its flat length could pass
    for [H, d] with the axes swapped); 1-D lengths are checked by the library."""
    if A_log.dim() == 2 and tuple(A_log.shape) != (H, d):
        raise ValueError(f"A_log must be [H] or [H, d] = [{H}, {d}], got {tuple(A_log.shape)}")
    return A_log.contiguous()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def gate(x: torch.Tensor, b: torch.Tensor, A_log: torch.Tensor, dt_bias: torch.Tensor,
         g_out: Optional[torch.Tensor] = None, beta_out: Optional[torch.Tensor] = None
         ) -> Tuple[torch.Tensor, torch.Tensor]:
    """kda_gate: x [T,H,d], b [T,H], A_log [H] or [H,d], dt_bias [H,d]
    -> g [T,H,d] fp32, beta [T,H] fp32."""
    T, H, d = x.shape
    A_log = _alog(A_log, H, d)
    if g_out is None:
        g_out = torch.empty((T, H, d), dtype=torch.float32, device=x.device)
    if beta_out is None:
        beta_out = torch.empty((T, H), dtype=torch.float32, device=x.device)
    st = lib().kda_gate(_ptr(x), _dt(x), _ptr(b), _dt(b), _ptr(A_log), A_log.numel(),
                        _ptr(dt_bias), dt_bias.numel(), _ptr(g_out), _ptr(beta_out), T, H, d,
                        _stream(x.device))
    _check(st)
    return g_out, beta_out


def chunk_prefill_workspace_bytes(N: int, H: int, dk: int = 128, dv: int = 128,
                                  chunks_per_pass: int = 1) -> int:
    """kda_chunk_prefill_workspace_bytes."""
    return int(lib().kda_chunk_prefill_workspace_bytes(N, H, dk, dv, chunks_per_pass))


def _prefill_common(q, v, cu_seqlens, cu_seqlens_host, initial_state, output_final_state,
                    o_dtype, out, final_state, workspace, max_workspace_bytes,
                    state_dtype=torch.float32):
    T, H, dk = q.shape
    dv = v.shape[2]
    dev = q.device
    if cu_seqlens is None:
        cu_seqlens_host = torch.tensor([0, T], dtype=torch.int32)
        cu_seqlens = cu_seqlens_host.to(dev)
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    if cu_seqlens_host is None:
        cu_seqlens_host = cu_seqlens.cpu()
    N = cu_seqlens.numel() - 1
    o_dtype = o_dtype or q.dtype
    if out is None:
        out = torch.empty((T, H, dv), dtype=o_dtype, device=dev)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, dk, dv), dtype=state_dtype, device=dev)
    hp = cu_seqlens_host.contiguous()
    if workspace is None:
        lens = (hp[1:] - hp[:-1]).clamp(min=0)
        max_chunks = max(1, int((int(lens.max()) + CHUNK - 1) // CHUNK)) if N > 0 else 1
        one = chunk_prefill_workspace_bytes(N, H, dk, dv, 1)
        per = chunk_prefill_workspace_bytes(N, H, dk, dv, 2) - one
        fit = max(1, (max_workspace_bytes - (one - per)) // per) if per > 0 else 1
        nbytes = chunk_prefill_workspace_bytes(N, H, dk, dv, int(min(max_chunks, fit)))
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    return T, H, dk, dv, dev, cu_seqlens, hp, N, out, final_state, workspace


def chunk_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                  beta: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                  initial_state: Optional[torch.Tensor] = None, output_final_state: bool = True,
                  scale: float = 1.0, o_dtype: Optional[torch.dtype] = None,
                  out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
                  cu_seqlens_host: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None,
                  max_workspace_bytes: int = DEFAULT_WORKSPACE_BYTES):
    """kda_chunk_prefill on packed [T_tot, H, d] tensors.

    cu_seqlens: int32 [N+1] (device); None means one sequence of length T_tot.
    workspace: uint8 device tensor; None allocates one that covers the longest
    sequence in one pass, capped at max_workspace_bytes (at least the minimum).
    Returns (o [T_tot,H,dv], final_state [N,H,dk,dv] or None).
    """
    T, H, dk, dv, dev, cu_seqlens, hp, N, out, final_state, workspace = _prefill_common(
        q, v, cu_seqlens, cu_seqlens_host, initial_state, output_final_state, o_dtype, out,
        final_state, workspace, max_workspace_bytes)
    st = lib().kda_chunk_prefill(
        _ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
        ctypes.cast(hp.data_ptr(), _vp), N, _ptr(initial_state), _ptr(final_state), _ptr(out),
        _dt(out), T, H, dk, dv, float(scale), _ptr(workspace), workspace.numel(), _stream(dev))
    _check(st)
    return out, final_state


def chunk_prefill_gated(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, x: torch.Tensor,
                        b: torch.Tensor, A_log: torch.Tensor, dt_bias: torch.Tensor,
                        cu_seqlens: Optional[torch.Tensor] = None,
                        initial_state: Optional[torch.Tensor] = None,
                        output_final_state: bool = True, scale: float = 1.0,
                        o_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                        final_state: Optional[torch.Tensor] = None,
                        cu_seqlens_host: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None,
                        max_workspace_bytes: int = DEFAULT_WORKSPACE_BYTES,
                        state_indices: Optional[torch.Tensor] = None,
                        state_dtype: Optional[torch.dtype] = None):
    """kda_chunk_prefill_gated: the gate's raw inputs (x [T,H,dk] logits, b [T,H]
    beta logits, A_log [H] or [H,dk], dt_bias [H,dk]) instead of g and beta.

    States are float32 or bfloat16 (state_dtype; default: initial_state's dtype,
    else float32).  Without state_indices they are [N,H,dk,dv] per sequence and a
    final state is allocated when output_final_state is set and none is given.
    With state_indices ([N] int32 on the device) initial_state and final_state
    are pools [num_slots,H,dk,dv] (final_state may be initial_state: an in-place
    update; it is written only when passed), and sequence n uses slot
    state_indices[n]; a slot outside the pool starts from zeros and is not
    written."""
    if state_dtype is None:
        state_dtype = initial_state.dtype if initial_state is not None else (
            final_state.dtype if final_state is not None else torch.float32)
    if state_indices is not None:
        if state_indices.dtype != torch.int32:
            raise TypeError("state_indices must be int32")
        output_final_state = False  # a pool is written only when passed as final_state
    T, H, dk, dv, dev, cu_seqlens, hp, N, out, final_state, workspace = _prefill_common(
        q, v, cu_seqlens, cu_seqlens_host, initial_state, output_final_state, o_dtype, out,
        final_state, workspace, max_workspace_bytes, state_dtype)
    for t in (initial_state, final_state):
        if t is not None and t.dtype != state_dtype:
            raise TypeError("initial_state and final_state must both be %s" % state_dtype)
    pools = [t for t in (initial_state, final_state) if t is not None]
    num_slots = pools[0].shape[0] if pools else N
    if any(t.shape[0] != num_slots for t in pools):
        raise ValueError("initial_state and final_state must have the same number of slots")
    A_log = _alog(A_log, H, dk)
    dt_bias = dt_bias.contiguous()
    st = lib().kda_chunk_prefill_gated(
        _ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(x), _dt(x), _ptr(b), _dt(b), _ptr(A_log),
        A_log.numel(), _ptr(dt_bias), dt_bias.numel(), _ptr(cu_seqlens),
        ctypes.cast(hp.data_ptr(), _vp), N, _ptr(initial_state), _ptr(final_state),
        KDA_BF16 if state_dtype == torch.bfloat16 else KDA_F32, num_slots, _ptr(state_indices),
        _ptr(out), _dt(out), T, H, dk, dv, float(scale), _ptr(workspace), workspace.numel(),
        _stream(dev))
    _check(st)
    return out, final_state


def chunk_prefill_gated_static(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                               x: torch.Tensor, b: torch.Tensor, A_log: torch.Tensor,
                               dt_bias: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                               initial_state: Optional[torch.Tensor] = None,
                               final_state: Optional[torch.Tensor] = None,
                               out: Optional[torch.Tensor] = None, scale: float = 1.0,
                               cu_seqlens_host: Optional[torch.Tensor] = None,
                               state_indices: Optional[torch.Tensor] = None,
                               state_dtype: Optional[torch.dtype] = None):
    """kda_chunk_prefill_gated_static: chunk_prefill_gated over the library's own
    device scratch (no workspace).  The caller passes every output: o as `out`
    and, if wanted, final_state; nothing is allocated.  Returns (out, final_state)."""
    T, H, dk = q.shape
    dv = v.shape[2]
    if out is None:
        raise ValueError("chunk_prefill_gated_static allocates nothing: pass out")
    if cu_seqlens is None or cu_seqlens_host is None:
        raise ValueError("chunk_prefill_gated_static needs cu_seqlens and cu_seqlens_host")
    if cu_seqlens.dtype != torch.int32 or cu_seqlens_host.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    hp = cu_seqlens_host.contiguous()
    N = cu_seqlens.numel() - 1
    if state_dtype is None:
        state_dtype = initial_state.dtype if initial_state is not None else (
            final_state.dtype if final_state is not None else torch.float32)
    pools = [t for t in (initial_state, final_state) if t is not None]
    num_slots = pools[0].shape[0] if pools else N
    A_log = _alog(A_log, H, dk)
    st = lib().kda_chunk_prefill_gated_static(
        _ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(x), _dt(x), _ptr(b), _dt(b), _ptr(A_log),
        A_log.numel(), _ptr(dt_bias), dt_bias.numel(), _ptr(cu_seqlens),
        ctypes.cast(hp.data_ptr(), _vp), N, _ptr(initial_state), _ptr(final_state),
        KDA_BF16 if state_dtype == torch.bfloat16 else KDA_F32, num_slots, _ptr(state_indices),
        _ptr(out), _dt(out), T, H, dk, dv, float(scale), _stream(q.device))
    _check(st)
    return out, final_state


def gate_backward(x: torch.Tensor, b: torch.Tensor, A_log: torch.Tensor, dt_bias: torch.Tensor,
                  dg: torch.Tensor, dbeta: torch.Tensor):
    """kda_gate_backward: gradients of gate() against dg [T,H,d] and dbeta [T,H].

    Returns (dx [T,H,d], db [T,H], dA_log (A_log's shape), ddt_bias [H,d]), float32."""
    T, H, d = x.shape
    A_log = _alog(A_log, H, d)
    dev = x.device
    f32 = dict(dtype=torch.float32, device=dev)
    dx = torch.empty((T, H, d), **f32)
    db = torch.empty((T, H), **f32)
    dA = torch.empty(tuple(A_log.shape), **f32)
    ddt = torch.empty((H, d), **f32)
    nbytes = int(lib().kda_gate_backward_workspace_bytes(T, H, d))
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    st = lib().kda_gate_backward(_ptr(x), _dt(x), _ptr(b), _dt(b), _ptr(A_log), A_log.numel(),
                                 _ptr(dt_bias.contiguous()), dt_bias.numel(), _ptr(dg),
                                 _ptr(dbeta), _ptr(dx), _ptr(db), _ptr(dA), _ptr(ddt), T, H, d,
                                 _ptr(ws), ws.numel(), _stream(dev))
    _check(st)
    return dx, db, dA, ddt


def chunk_prefill_backward_workspace_bytes(T_tot: int, N: int, H: int, dk: int = 128,
                                           dv: int = 128) -> int:
    """kda_chunk_prefill_backward_workspace_bytes."""
    return int(lib().kda_chunk_prefill_backward_workspace_bytes(T_tot, N, H, dk, dv))


def chunk_prefill_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                           beta: torch.Tensor, d_o: Optional[torch.Tensor],
                           cu_seqlens: Optional[torch.Tensor] = None,
                           initial_state: Optional[torch.Tensor] = None,
                           d_final_state: Optional[torch.Tensor] = None, scale: float = 1.0,
                           want_d_initial_state: bool = True,
                           cu_seqlens_host: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None):
    """kda_chunk_prefill_backward: gradients of chunk_prefill's (o, final_state)
    against d_o [T,H,dv] (None: zero) and d_final_state [N,H,dk,dv] (None: zero).

    Returns (dq, dk, dv, dg, dbeta, d_initial_state) as float32 tensors
    (d_initial_state None unless want_d_initial_state)."""
    T, H, dk = q.shape
    dv = v.shape[2]
    dev = q.device
    if cu_seqlens is None:
        cu_seqlens_host = torch.tensor([0, T], dtype=torch.int32)
        cu_seqlens = cu_seqlens_host.to(dev)
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    if cu_seqlens_host is None:
        cu_seqlens_host = cu_seqlens.cpu()
    hp = cu_seqlens_host.contiguous()
    N = cu_seqlens.numel() - 1
    f32 = dict(dtype=torch.float32, device=dev)
    dq = torch.empty((T, H, dk), **f32)
    dk_ = torch.empty((T, H, dk), **f32)
    dv_ = torch.empty((T, H, dv), **f32)
    dg = torch.empty((T, H, dk), **f32)
    dbeta = torch.empty((T, H), **f32)
    dS0 = torch.empty((N, H, dk, dv), **f32) if want_d_initial_state else None
    if workspace is None:
        nbytes = chunk_prefill_backward_workspace_bytes(T, N, H, dk, dv)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    st = lib().kda_chunk_prefill_backward(
        _ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
        ctypes.cast(hp.data_ptr(), _vp), N, _ptr(initial_state), _ptr(d_o),
        _dt(d_o) if d_o is not None else KDA_F32, _ptr(d_final_state), _ptr(dq), _ptr(dk_),
        _ptr(dv_), _ptr(dg), _ptr(dbeta), _ptr(dS0), T, H, dk, dv, float(scale),
        _ptr(workspace), workspace.numel(), _stream(dev))
    _check(st)
    return dq, dk_, dv_, dg, dbeta, dS0


def recurrent_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                     beta: torch.Tensor, state: torch.Tensor, scale: float = 1.0,
                     o_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None):
    """kda_recurrent_decode: q/k/v [N,H,d], state [N,H,dk,dv] updated in place. Returns o."""
    N, H, dk = q.shape
    dv = v.shape[2]
    if out is None:
        out = torch.empty((N, H, dv), dtype=o_dtype or q.dtype, device=q.device)
    st = lib().kda_recurrent_decode(_ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(g), _ptr(beta),
                                    _ptr(state), _ptr(out), _dt(out), N, H, dk, dv, float(scale),
                                    _stream(q.device))
    _check(st)
    return out


def recurrent_decode_gated(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, x: torch.Tensor,
                           b: torch.Tensor, A_log: torch.Tensor, dt_bias: torch.Tensor,
                           state: torch.Tensor, state_indices: Optional[torch.Tensor] = None,
                           scale: float = 1.0, o_dtype: Optional[torch.dtype] = None,
                           out: Optional[torch.Tensor] = None):
    """kda_recurrent_decode_gated: q/k/v/x [N,H,d], b [N,H], A_log [H] or [H,d], dt_bias [H,d];
    state pool [num_slots,H,dk,dv] (float32 or bfloat16) updated in place;
    state_indices [N] int32 on the device (None: sequence n uses slot n).
    Returns o (zeros for sequences whose slot is outside the pool)."""
    N, H, dk = q.shape
    dv = v.shape[2]
    if state_indices is not None and state_indices.dtype != torch.int32:
        raise TypeError("state_indices must be int32")
    A_log = _alog(A_log, H, dk)
    if out is None:
        out = torch.empty((N, H, dv), dtype=o_dtype or q.dtype, device=q.device)
    st = lib().kda_recurrent_decode_gated(
        _ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(x), _dt(x), _ptr(b), _dt(b), _ptr(A_log),
        A_log.numel(), _ptr(dt_bias), dt_bias.numel(), _ptr(state), _dt(state), state.shape[0],
        _ptr(state_indices), _ptr(out), _dt(out), N, H, dk, dv, float(scale), _stream(q.device))
    _check(st)
    return out


def shortconv_l2norm(xq: torch.Tensor, xk: torch.Tensor, xv: torch.Tensor, wq: torch.Tensor,
                     wk: torch.Tensor, wv: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                     conv_state: Optional[torch.Tensor] = None, output_state: bool = True,
                     activation: Optional[str] = "silu", eps: float = 1e-6,
                     out_dtype: Optional[torch.dtype] = None,
                     cu_seqlens_host: Optional[torch.Tensor] = None,
                     state_out: Optional[torch.Tensor] = None):
    """kda_shortconv_l2norm: xq/xk/xv [T,H,d] projections, conv weights [H*d,4]
    (or the checkpoint's [H*d,1,4]) -> (yq, yk, yv, conv_state_out) with q and k
    L2-normalised.  conv_state [N,3,3,H*d] fp32 or None (zeros); state_out may
    be conv_state itself (in place) when no sequence exceeds 64 tokens."""
    T, H, d = xq.shape
    dev = xq.device
    if cu_seqlens is None:
        cu_seqlens = torch.tensor([0, T], dtype=torch.int32, device=dev)
    if cu_seqlens_host is None:
        cu_seqlens_host = cu_seqlens.detach().to("cpu", torch.int32)
    cu_h = cu_seqlens_host.contiguous()
    N = cu_h.numel() - 1
    odt = out_dtype or xq.dtype
    ys = [torch.empty((T, H, d), dtype=odt, device=dev) for _ in range(3)]
    if output_state and state_out is None:
        state_out = torch.empty((N, 3, 3, H * d), dtype=torch.float32, device=dev)
    act = {None: KDA_ACT_NONE, "silu": KDA_ACT_SILU}[activation]
    ws = [w.contiguous() for w in (wq, wk, wv)]
    st = lib().kda_shortconv_l2norm(
        _ptr(xq), _ptr(xk), _ptr(xv), _dt(xq), _ptr(ws[0]), _ptr(ws[1]), _ptr(ws[2]),
        ws[0].numel(), act, float(eps), _ptr(cu_seqlens.to(dev, torch.int32).contiguous()),
        cu_h.data_ptr(), N, _ptr(conv_state), _ptr(state_out if output_state else None),
        _ptr(ys[0]), _ptr(ys[1]), _ptr(ys[2]), _dt(ys[0]), T, H, d, _stream(dev))
    _check(st)
    return ys[0], ys[1], ys[2], (state_out if output_state else None)

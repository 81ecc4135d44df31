"""Gated linear recurrence over packed sequences: forward, backward and decode step.

    h_t = a_t h_{t-1} + b_t x_t,    y_t = h_t

per channel, with gates per channel or shared by a head's channels, on the packed batches and state pools of the
gated delta rule.  Like the package's other calls these marshal arguments for the C ABI (``include/gdn_linear.h``);
the work is done by the kernels of ``libgdn_prefill.so``.  :func:`gated_linear_recurrence` is differentiable.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import (DTYPE_F32, GdnError, _pow2_at_least, _ptr, _QKV_DTYPES, _STATE_DTYPES, lib)

__all__ = ["gated_linear_recurrence", "gated_linear_recurrence_backward", "gated_linear_recurrence_decode", "LinearDesc",
           "LinearArgs", "LINEAR_FLAGS", "LINEAR_TILE", "gdn_linear_plan", "gdn_linear_plan_destroy",
           "gdn_linear_forward_run", "gdn_linear_backward_run", "gdn_linear_decode_run"]

LINEAR_TILE = 64  # packed tokens a row of tile_states stands for
LINEAR_FLAGS = {"HAS_B": 1 << 0, "GATES_PER_HEAD": 1 << 1, "HAS_INITIAL_STATE": 1 << 2, "OUTPUT_FINAL_STATE": 1 << 3,
                "HAS_STATE_INDICES": 1 << 4, "CU_SEQLENS_I64": 1 << 5, "STATE_INDICES_I64": 1 << 6}
_HAS_B, _PER_HEAD, _HAS_INIT, _FINAL, _HAS_IDX, _CU_I64, _IDX_I64 = (1 << i for i in range(7))


class LinearDesc(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("gate_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32), ("max_total_tokens", ctypes.c_int64),
                ("max_num_seqs", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class LinearArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("x_stride", ctypes.c_int64), ("a_stride", ctypes.c_int64), ("b_stride", ctypes.c_int64),
                ("cu_seqlens", ctypes.c_void_p), ("num_seqs", ctypes.c_int32), ("total_tokens", ctypes.c_int64),
                ("initial_state", ctypes.c_void_p), ("output_state", ctypes.c_void_p), ("state_stride", ctypes.c_int64),
                ("state_indices", ctypes.c_void_p), ("n_pool", ctypes.c_int32), ("device_status", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("y_stride", ctypes.c_int64), ("tile_states", ctypes.c_void_p),
                ("dy", ctypes.c_void_p), ("dy_stride", ctypes.c_int64), ("d_final_state", ctypes.c_void_p),
                ("d_initial_state", ctypes.c_void_p), ("dx", ctypes.c_void_p), ("da", ctypes.c_void_p),
                ("db", ctypes.c_void_p), ("dx_stride", ctypes.c_int64), ("da_stride", ctypes.c_int64),
                ("db_stride", ctypes.c_int64)]


def _register(L):
    """Argument types of the entry points (called once, when the library is loaded)."""
    run = [ctypes.c_void_p, ctypes.POINTER(LinearArgs), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    L.gdn_linear_plan.argtypes = [ctypes.POINTER(LinearDesc), ctypes.POINTER(ctypes.c_void_p),
                                  ctypes.POINTER(ctypes.c_size_t)]
    L.gdn_linear_plan.restype = ctypes.c_int
    L.gdn_linear_plan_destroy.argtypes = [ctypes.c_void_p]
    L.gdn_linear_plan_destroy.restype = None
    for fn in (L.gdn_linear_forward_run, L.gdn_linear_backward_run):
        fn.argtypes = run
        fn.restype = ctypes.c_int
    L.gdn_linear_decode_run.argtypes = [ctypes.c_void_p, ctypes.POINTER(LinearArgs), ctypes.c_int32, ctypes.c_void_p]
    L.gdn_linear_decode_run.restype = ctypes.c_int


def gdn_linear_plan(desc: LinearDesc):
    """Returns (status, plan handle, workspace bytes)."""
    plan = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    st = lib().gdn_linear_plan(ctypes.byref(desc), ctypes.byref(plan), ctypes.byref(ws))
    return st, plan, ws.value


def gdn_linear_plan_destroy(plan) -> None:
    lib().gdn_linear_plan_destroy(plan)


def gdn_linear_forward_run(plan, args: LinearArgs, workspace_ptr, workspace_bytes: int, stream_ptr) -> int:
    return lib().gdn_linear_forward_run(plan, args, workspace_ptr, workspace_bytes, stream_ptr)


def gdn_linear_backward_run(plan, args: LinearArgs, workspace_ptr, workspace_bytes: int, stream_ptr) -> int:
    return lib().gdn_linear_backward_run(plan, args, workspace_ptr, workspace_bytes, stream_ptr)


def gdn_linear_decode_run(plan, args: LinearArgs, tokens_per_seq: int, stream_ptr) -> int:
    return lib().gdn_linear_decode_run(plan, args, tokens_per_seq, stream_ptr)


class _Plan:
    """A plan and its bounds.  Holds no device memory: every run takes its workspace from torch's allocator, on the
    stream that it runs on."""

    def __init__(self, desc):
        st, self.handle, self.workspace_bytes = gdn_linear_plan(desc)
        if st != 0:
            self.handle = None
            raise GdnError(st, "gdn_linear_plan")
        self.max_tokens, self.max_seqs = desc.max_total_tokens, desc.max_num_seqs

    def __del__(self):
        try:
            if self.handle:
                gdn_linear_plan_destroy(self.handle)
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass


_plans = {}
_plans_lock = threading.Lock()


def _get_plan(key, T, N):
    """key: (heads, dim, x dtype, gate dtype, state dtype, flags, power-of-two bound of the tokens)."""
    p = _plans.get(key)
    if p is None or p.max_seqs < N:
        with _plans_lock:
            p = _Plan(LinearDesc(*key[:5], key[6], _pow2_at_least(N), key[5]))
            _plans[key] = p
    return p


def _tokens(name, t, shape, dtype, device):
    """Checks a [T, ...] tensor; returns its token stride (0: dense)."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.is_contiguous():
        return 0
    row = 1
    for n, s in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if n > 1 and s != row:
            raise ValueError(f"{name} must be contiguous within a token")
        row *= n
    if t.stride(0) < row:
        raise ValueError(f"{name}'s tokens must not overlap")
    return t.stride(0)


def _inputs(x, a, b):
    """Checks x and the gates; returns T, H, D, flags and the token strides."""
    if x.dim() != 3:
        raise ValueError("x must be [total_tokens, heads, head_dim]")
    device = x.device
    if device.type != "cuda":
        raise ValueError("x must be a CUDA tensor: this library has no CPU path")
    T, H, D = shape = x.shape
    if x.dtype not in _QKV_DTYPES:
        raise ValueError(f"unsupported dtype {x.dtype}")
    if a.dtype != x.dtype and a.dtype != torch.float32:
        raise ValueError("the gates must be float32 or of x's dtype")
    flags = 0
    if a.dim() == 2:
        flags = _PER_HEAD
        gshape = shape[:2]
    else:
        gshape = shape
    xs = _tokens("x", x, shape, x.dtype, device)
    as_ = _tokens("a", a, gshape, a.dtype, device)
    bs = 0
    if b is not None:
        flags |= _HAS_B
        bs = _tokens("b", b, gshape, a.dtype, device)
    return T, H, D, flags, xs, as_, bs


def _sequences(cu_seqlens, device):
    """(N, flag) of cu_seqlens, or of one sequence without it."""
    if cu_seqlens is None:
        return 1, 0
    if cu_seqlens.device != device or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous() or cu_seqlens.numel() < 1:
        raise ValueError(f"cu_seqlens must be a contiguous vector of N + 1 entries on {device}")
    if cu_seqlens.dtype == torch.int32:
        return cu_seqlens.numel() - 1, 0
    if cu_seqlens.dtype == torch.int64:
        return cu_seqlens.numel() - 1, _CU_I64
    raise ValueError("cu_seqlens must be int32 or int64")


def _states(initial_state, output_state, state_indices, N, H, D, device):
    """Checks the states; returns (dtype code, row stride, pool rows, flags)."""
    dt, stride, n_pool, flags = DTYPE_F32, 0, 0, 0
    first = None
    for name, t in (("initial_state", initial_state), ("output_state", output_state)):
        if t is None:
            continue
        if t.device != device or t.dim() != 3 or t.shape[1] != H or t.shape[2] != D:
            raise ValueError(f"{name} must be [rows, {H}, {D}] on {device}")
        if (D > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != D) or (t.shape[0] > 1 and t.stride(0) < H * D):
            raise ValueError(f"{name} must have contiguous rows that do not overlap")
        if t.dtype not in _STATE_DTYPES:
            raise ValueError(f"unsupported state dtype {t.dtype}")
        if first is None:
            first, dt, stride = t, _STATE_DTYPES[t.dtype], t.stride(0) if t.shape[0] > 1 else 0
        elif t.dtype != first.dtype or t.shape != first.shape or (t.shape[0] > 1 and t.stride(0) != stride):
            raise ValueError("initial_state and output_state must share shape, dtype and strides")
    if state_indices is not None:
        if first is None:
            raise ValueError("state_indices needs a state pool (initial_state and/or output_state)")
        if state_indices.device != device or state_indices.shape != (N,) or not state_indices.is_contiguous():
            raise ValueError(f"state_indices must be a contiguous vector of {N} entries on {device}")
        flags = _HAS_IDX
        if state_indices.dtype == torch.int64:
            flags |= _IDX_I64
        elif state_indices.dtype != torch.int32:
            raise ValueError("state_indices must be int32 or int64")
        n_pool = first.shape[0]
    elif first is not None and first.shape[0] != N:
        raise ValueError(f"the states must have {N} rows")
    if initial_state is not None:
        flags |= _HAS_INIT
    if output_state is not None:
        flags |= _FINAL
    return dt, stride, n_pool, flags


def _status_ptr(device_status, device):
    if device_status is None:
        return None
    if device_status.dtype != torch.int32 or device_status.device != device:
        raise ValueError(f"device_status must be int32 on {device}")
    return device_status.data_ptr()


def _run(fn, name, key, T, N, args, device):
    p = _get_plan(key, T, N)
    with torch.cuda.device(device):
        ws = torch.empty(p.workspace_bytes, dtype=torch.uint8, device=device)
        st = fn(p.handle, args, ws.data_ptr(), p.workspace_bytes, torch.cuda.current_stream(device).cuda_stream)
    if st != 0:
        raise GdnError(st, name)


def _new_states(initial_state, N, H, D, device):
    if initial_state is None:
        return torch.empty(N, H, D, dtype=torch.float32, device=device)
    return torch.empty_strided(initial_state.shape, initial_state.stride(), dtype=initial_state.dtype, device=device)


def _forward(x, a, b, initial_state, output_state, cu_seqlens, output, state_indices, tile_states, device_status):
    T, H, D, flags, xs, as_, bs = _inputs(x, a, b)
    device = x.device
    N, f = _sequences(cu_seqlens, device)
    flags |= f
    sdt, sstride, n_pool, f = _states(initial_state, output_state, state_indices, N, H, D, device)
    flags |= f
    ys = 0
    if output is None:
        output = torch.empty(T, H, D, dtype=x.dtype, device=device)
    else:
        ys = _tokens("output", output, x.shape, x.dtype, device)
    if tile_states is not None and _tokens("tile_states", tile_states, (-(-T // LINEAR_TILE), H, D), torch.float32, device):
        raise ValueError("tile_states must be contiguous")
    key = (H, D, _QKV_DTYPES[x.dtype], _QKV_DTYPES[a.dtype], sdt, flags, _pow2_at_least(T, LINEAR_TILE))
    args = LinearArgs(x.data_ptr(), a.data_ptr(), _ptr(b), xs, as_, bs, _ptr(cu_seqlens), N, T, _ptr(initial_state),
                      _ptr(output_state), sstride, _ptr(state_indices), n_pool, _status_ptr(device_status, device),
                      output.data_ptr(), ys, _ptr(tile_states))
    _run(lib().gdn_linear_forward_run, "gdn_linear_forward_run", key, T, N, args, device)
    return output


class _Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, a, b, initial_state, cu_seqlens, output_final_state, device_status):
        T, H, D = x.shape
        N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
        final = _new_states(initial_state, N, H, D, x.device) if output_final_state else None
        tiles = torch.empty(-(-T // LINEAR_TILE), H, D, dtype=torch.float32, device=x.device)
        y = _forward(x, a, b, initial_state, final, cu_seqlens, None, None, tiles, device_status)
        ctx.save_for_backward(x, a, b, initial_state, cu_seqlens, tiles, device_status)
        return y, final

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, d_final):
        x, a, b, initial_state, cu_seqlens, tiles, status = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros_like(x)
        dx, da, db, d0 = gated_linear_recurrence_backward(
            dy.contiguous(), x, a, b, tile_states=tiles, initial_state=initial_state,
            d_final_state=None if d_final is None else d_final.float().contiguous(), cu_seqlens=cu_seqlens,
            device_status=status)
        if d0 is not None:
            d0 = d0.to(initial_state.dtype) if ctx.needs_input_grad[3] else None
        return dx, da, db, d0, None, None, None


def gated_linear_recurrence(x, a, b=None, initial_state=None, output_final_state=False, cu_seqlens=None, output=None,
                            output_state=None, state_indices=None, tile_states=None, device_status=None):
    """y_t = h_t = a_t h_{t-1} + b_t x_t over packed sequences (fp32 states, y rounded once to x's type).

    ``x`` [T, H, D] (bf16, fp16 or fp32); gates ``a`` and ``b`` (None: ones) [T, H, D], or [T, H] shared by a head's
    channels, both fp32 or x's type.  Tokens may be strided (slices of a projection's output).  ``cu_seqlens`` [N + 1]
    (int32 or int64) bounds the sequences (None: one sequence); ``initial_state`` and ``output_state`` are [N, H, D], or
    pools addressed by ``state_indices``, and may be one buffer.  ``tile_states`` [ceil(T / 64), H, D] fp32, when given,
    receives what :func:`gated_linear_recurrence_backward` needs.  ``device_status`` (int32) receives the error bits of
    device data.  Returns ``output`` or ``(output, final_state)``.

    Differentiable in x, a, b and initial_state when called without output, output_state, state_indices and
    tile_states.
    """
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, a, b, initial_state)):
        if output is not None or output_state is not None or state_indices is not None or tile_states is not None:
            raise ValueError("output, output_state, state_indices and tile_states cannot be differentiated through")
        y, final = _Recurrence.apply(x, a, b, initial_state, cu_seqlens, output_final_state, device_status)
        return (y, final) if output_final_state else y
    if not output_final_state:
        output_state = None
    elif output_state is None:
        if state_indices is not None:
            raise ValueError("output_final_state with state_indices requires the output_state pool")
        N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
        output_state = _new_states(initial_state, N, x.shape[-2], x.shape[-1], x.device)
    y = _forward(x, a, b, initial_state, output_state, cu_seqlens, output, state_indices, tile_states, device_status)
    return (y, output_state) if output_final_state else y


def gated_linear_recurrence_backward(dy, x, a, b=None, tile_states=None, initial_state=None, d_final_state=None,
                                     cu_seqlens=None, device_status=None):
    """Gradients of :func:`gated_linear_recurrence`: ``(dx, da, db, d_initial_state)``.

    ``dy`` is the gradient of y, ``d_final_state`` [N, H, D] fp32 that of the final states (None: zero), ``tile_states``
    what the forward run saved (not needed up to 64 tokens).  dx has x's type, da and db (None without b) the gates'
    type and shape; d_initial_state [N, H, D] is fp32 (None without initial_state).
    """
    T, H, D, flags, xs, as_, bs = _inputs(x, a, b)
    device = x.device
    N, f = _sequences(cu_seqlens, device)
    flags |= f
    sdt, sstride, _, f = _states(initial_state, None, None, N, H, D, device)
    flags |= f
    dys = _tokens("dy", dy, x.shape, x.dtype, device)
    if tile_states is not None:
        if _tokens("tile_states", tile_states, (-(-T // LINEAR_TILE), H, D), torch.float32, device):
            raise ValueError("tile_states must be contiguous")
    elif T > LINEAR_TILE:
        raise ValueError("tile_states of the forward run are needed")
    if d_final_state is not None and (d_final_state.shape != (N, H, D) or d_final_state.dtype != torch.float32 or
                                      d_final_state.device != device or not d_final_state.is_contiguous()):
        raise ValueError(f"d_final_state must be contiguous float32 [{N}, {H}, {D}] on {device}")
    dx = torch.empty(T, H, D, dtype=x.dtype, device=device)
    da = torch.empty(a.shape, dtype=a.dtype, device=device)
    db = torch.empty(a.shape, dtype=a.dtype, device=device) if b is not None else None
    d0 = torch.empty(N, H, D, dtype=torch.float32, device=device) if initial_state is not None else None
    key = (H, D, _QKV_DTYPES[x.dtype], _QKV_DTYPES[a.dtype], sdt, flags, _pow2_at_least(T, LINEAR_TILE))
    args = LinearArgs(x.data_ptr(), a.data_ptr(), _ptr(b), xs, as_, bs, _ptr(cu_seqlens), N, T, _ptr(initial_state),
                      None, sstride, None, 0, _status_ptr(device_status, device), None, 0, _ptr(tile_states),
                      dy.data_ptr(), dys, _ptr(d_final_state), _ptr(d0), dx.data_ptr(), da.data_ptr(), _ptr(db))
    _run(lib().gdn_linear_backward_run, "gdn_linear_backward_run", key, T, N, args, device)
    return dx, da, db, d0


def gated_linear_recurrence_decode(x, a, b=None, initial_state=None, state_indices=None, output_final_state=True,
                                   output_state=None, tokens_per_seq=1, output=None, device_status=None):
    """Decode step (or a short run of tokens) of :func:`gated_linear_recurrence`: N sequences of ``tokens_per_seq``
    tokens each, rows i * tokens_per_seq + j of x, a and b.  With ``state_indices`` the state is read from its pool row
    and written back in place (or to ``output_state``'s row).  Returns ``output`` or ``(output, final_state)``."""
    T, H, D, flags, xs, as_, bs = _inputs(x, a, b)
    device = x.device
    m = int(tokens_per_seq)
    if m < 1 or T % m:
        raise ValueError("x must have N * tokens_per_seq rows")
    N = T // m
    if not output_final_state:
        output_state = None
    elif output_state is None:
        if state_indices is not None:
            if initial_state is None:
                raise ValueError("state_indices needs the state pool as initial_state")
            output_state = initial_state
        else:
            output_state = _new_states(initial_state, N, H, D, device)
    sdt, sstride, n_pool, f = _states(initial_state, output_state, state_indices, N, H, D, device)
    flags |= f
    ys = 0
    if output is None:
        output = torch.empty(T, H, D, dtype=x.dtype, device=device)
    else:
        ys = _tokens("output", output, x.shape, x.dtype, device)
    p = _get_plan((H, D, _QKV_DTYPES[x.dtype], _QKV_DTYPES[a.dtype], sdt, flags, _pow2_at_least(T, LINEAR_TILE)), T, N)
    args = LinearArgs(x.data_ptr(), a.data_ptr(), _ptr(b), xs, as_, bs, None, N, T, _ptr(initial_state),
                      _ptr(output_state), sstride, _ptr(state_indices), n_pool, _status_ptr(device_status, device),
                      output.data_ptr(), ys)
    with torch.cuda.device(device):
        st = lib().gdn_linear_decode_run(p.handle, args, m, torch.cuda.current_stream(device).cuda_stream)
    if st != 0:
        raise GdnError(st, "gdn_linear_decode_run")
    return (output, output_state) if output_final_state else output

"""Gated linear recurrence over packed sequences: forward, backward and decode step.

    h_t = a_t h_{t-1} + b_t x_t,    y_t = h_t

per channel, with gates per channel or shared by a head's channels, on the packed batches and state pools of the
gated delta rule.  Like the package's other calls these marshal arguments for the C ABI (``include/gdn_linear.h``);
the work is done by the kernels of ``libgdn_prefill.so``.  :func:`gated_linear_recurrence` is differentiable.
"""
from __future__ import annotations

import ctypes
import struct
import threading

import torch
from torch.autograd.graph import increment_version

from . import DTYPE_F32, GdnError, _pow2_at_least, _QKV_DTYPES, _STATE_DTYPES, lib, on_device

__all__ = ["gated_linear_recurrence", "gated_linear_recurrence_backward", "gated_linear_recurrence_decode", "LinearDesc",
           "LinearArgs", "LINEAR_FLAGS", "LINEAR_TILE", "gdn_linear_plan", "gdn_linear_plan_destroy",
           "gdn_linear_run_workspace", "gdn_linear_forward_run", "gdn_linear_backward_run", "gdn_linear_decode_run"]

LINEAR_TILE = 64  # packed tokens a row of tile_states stands for
_MAX_TOKENS = 0x7fffffff - LINEAR_TILE  # of any plan
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


# The bytes of a LinearArgs, in C's alignment: the calls below pack their arguments in one go.
_pack = struct.Struct("@PPPqqqPiqPPqPiPPqPPqPPPPPqqq").pack


def _register(L):
    """Argument types of the entry points (called once, when the library is loaded)."""
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    L.gdn_linear_plan.argtypes = [ctypes.POINTER(LinearDesc), ctypes.POINTER(vp), ctypes.POINTER(sz)]
    L.gdn_linear_plan.restype = ctypes.c_int
    L.gdn_linear_plan_destroy.argtypes = [vp]
    L.gdn_linear_plan_destroy.restype = None
    L.gdn_linear_run_workspace.argtypes = [vp, vp, ctypes.c_int32]
    L.gdn_linear_run_workspace.restype = sz
    for fn in (L.gdn_linear_forward_run, L.gdn_linear_backward_run):
        fn.argtypes = [vp, vp, vp, sz, vp]
        fn.restype = ctypes.c_int
    L.gdn_linear_decode_run.argtypes = [vp, vp, ctypes.c_int32, vp]
    L.gdn_linear_decode_run.restype = ctypes.c_int


def gdn_linear_plan(desc: LinearDesc):
    """Returns (status, plan handle, workspace bytes)."""
    plan = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    st = lib().gdn_linear_plan(ctypes.byref(desc), ctypes.byref(plan), ctypes.byref(ws))
    return st, plan, ws.value


def gdn_linear_plan_destroy(plan) -> None:
    lib().gdn_linear_plan_destroy(plan)


def gdn_linear_run_workspace(plan, args: LinearArgs, backward: bool) -> int:
    """Bytes of workspace that a run of these arguments needs (at most the plan's)."""
    return lib().gdn_linear_run_workspace(plan, ctypes.byref(args), int(backward))


def gdn_linear_forward_run(plan, args: LinearArgs, workspace_ptr, workspace_bytes: int, stream_ptr) -> int:
    return lib().gdn_linear_forward_run(plan, ctypes.byref(args), workspace_ptr, workspace_bytes, stream_ptr)


def gdn_linear_backward_run(plan, args: LinearArgs, workspace_ptr, workspace_bytes: int, stream_ptr) -> int:
    return lib().gdn_linear_backward_run(plan, ctypes.byref(args), workspace_ptr, workspace_bytes, stream_ptr)


def gdn_linear_decode_run(plan, args: LinearArgs, tokens_per_seq: int, stream_ptr) -> int:
    return lib().gdn_linear_decode_run(plan, ctypes.byref(args), tokens_per_seq, stream_ptr)


class _Plan:
    """A plan and its bounds.  Holds no device memory: every run takes its workspace from torch's allocator, on the
    stream that it runs on."""

    def __init__(self, desc):
        st, self.handle, _ = gdn_linear_plan(desc)
        if st != 0:
            self.handle = None
            raise GdnError(st, "gdn_linear_plan")
        self.max_seqs = desc.max_num_seqs

    def __del__(self):
        try:
            if self.handle:
                gdn_linear_plan_destroy(self.handle)
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass


_plans = {}
_plans_lock = threading.Lock()


def _get_plan(H, D, x, a, state_dt, flags, T, N):
    key = (H, D, x.dtype, a.dtype, state_dt, flags, T.bit_length())
    p = _plans.get(key)
    if p is None or p.max_seqs < N:
        with _plans_lock:
            p = _Plan(LinearDesc(H, D, _QKV_DTYPES[x.dtype], _QKV_DTYPES[a.dtype], state_dt,
                                 min((1 << T.bit_length()) - 1, _MAX_TOKENS), _pow2_at_least(N), flags))
            _plans[key] = p
    return p


def _tokens(name, t, shape, dtype, device):
    """Checks a [T, ...] tensor; returns its token stride (0: dense)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        raise ValueError(f"{name} must be {dtype} {list(shape)} on cuda:{device}, not {t.dtype} {list(t.shape)} on {t.device}")
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
    """Checks x and the gates; returns the device, T, H, D, flags and the token strides."""
    shape = x.shape
    if len(shape) != 3:
        raise ValueError("x must be [total_tokens, heads, head_dim]")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor: this library has no CPU path")
    dtype, gdtype, device = x.dtype, a.dtype, x.get_device()
    if dtype not in _QKV_DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    if gdtype is not dtype and gdtype is not torch.float32:
        raise ValueError("the gates must be float32 or of x's dtype")
    T, H, D = shape
    flags, gshape = (_PER_HEAD, (T, H)) if a.dim() == 2 else (0, shape)
    xs = _tokens("x", x, shape, dtype, device)
    as_ = _tokens("a", a, gshape, gdtype, device)
    bs = 0
    if b is not None:
        flags |= _HAS_B
        bs = _tokens("b", b, gshape, gdtype, device)
    return device, T, H, D, flags, xs, as_, bs


def _sequences(cu_seqlens, device):
    """(N, flag) of cu_seqlens, or of one sequence without it."""
    if cu_seqlens is None:
        return 1, 0
    if cu_seqlens.dim() != 1 or cu_seqlens.get_device() != device or not cu_seqlens.is_contiguous() or not cu_seqlens.numel():
        raise ValueError(f"cu_seqlens must be a contiguous vector of N + 1 entries on cuda:{device}")
    if cu_seqlens.dtype is torch.int32:
        return cu_seqlens.numel() - 1, 0
    if cu_seqlens.dtype is torch.int64:
        return cu_seqlens.numel() - 1, _CU_I64
    raise ValueError("cu_seqlens must be int32 or int64")


def _state(name, t, H, D, device):
    """Checks a state; returns its row stride (0: dense)."""
    if t.dim() != 3 or t.shape[1] != H or t.shape[2] != D or t.get_device() != device:
        raise ValueError(f"{name} must be [rows, {H}, {D}] on cuda:{device}")
    if t.dtype not in _STATE_DTYPES:
        raise ValueError(f"unsupported state dtype {t.dtype}")
    if t.is_contiguous():
        return 0
    if (D > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != D) or (t.shape[0] > 1 and t.stride(0) < H * D):
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return t.stride(0) if t.shape[0] > 1 else 0


def _states(initial_state, output_state, state_indices, N, H, D, device):
    """Checks the states; returns (dtype code, row stride, pool rows, flags)."""
    flags, n_pool, first, stride = 0, 0, None, 0
    if initial_state is not None:
        flags, first = _HAS_INIT, initial_state
        stride = _state("initial_state", initial_state, H, D, device)
    if output_state is not None:
        flags |= _FINAL
        if first is None:
            first, stride = output_state, _state("output_state", output_state, H, D, device)
        elif output_state is not first and (_state("output_state", output_state, H, D, device) != stride or
                                            output_state.dtype is not first.dtype or output_state.shape != first.shape):
            raise ValueError("initial_state and output_state must share shape, dtype and strides")
    if state_indices is not None:
        if first is None:
            raise ValueError("state_indices needs a state pool (initial_state and/or output_state)")
        if state_indices.shape != (N,) or state_indices.get_device() != device or not state_indices.is_contiguous():
            raise ValueError(f"state_indices must be a contiguous vector of {N} entries on cuda:{device}")
        flags |= _HAS_IDX
        if state_indices.dtype is torch.int64:
            flags |= _IDX_I64
        elif state_indices.dtype is not torch.int32:
            raise ValueError("state_indices must be int32 or int64")
        n_pool = first.shape[0]
    elif first is not None and first.shape[0] != N:
        raise ValueError(f"the states must have {N} rows")
    return _STATE_DTYPES[first.dtype] if first is not None else DTYPE_F32, stride, n_pool, flags


def _status_ptr(device_status, device):
    if device_status is None:
        return 0
    if device_status.dtype is not torch.int32 or device_status.get_device() != device or not device_status.numel():
        raise ValueError(f"device_status must be int32 on cuda:{device}")
    return device_status.data_ptr()


def _written(*tensors):
    """Tells autograd what a kernel has changed in place (None: nothing), so that a backward pass that saved one of these tensors
    refuses to go on with other values."""
    increment_version([t for t in tensors if t is not None])


def _addr(t):
    return 0 if t is None else t.data_ptr()


def _run(backward, plan, x, args):
    """Runs an entry point on x's device and the caller's stream, with a workspace from torch's allocator."""
    L, handle, ws, at = lib(), plan.handle, None, 0
    with on_device(x.get_device()) as stream:
        n = L.gdn_linear_run_workspace(handle, args, backward)
        if n:
            ws = torch.empty(n, dtype=torch.uint8, device=x.device)
            at = ws.data_ptr()
        st = (L.gdn_linear_backward_run if backward else L.gdn_linear_forward_run)(handle, args, at, n, stream)
    if st != 0:
        raise GdnError(st, "gdn_linear_backward_run" if backward else "gdn_linear_forward_run")


def _new_states(initial_state, N, H, D, device):
    if initial_state is None:
        return torch.empty(N, H, D, dtype=torch.float32, device=device)
    if initial_state.is_contiguous():
        return torch.empty_like(initial_state)
    return torch.empty_strided(initial_state.shape, initial_state.stride(), dtype=initial_state.dtype, device=device)


def _forward(x, a, b, initial_state, output_state, cu_seqlens, output, state_indices, tile_states, device_status):
    device, T, H, D, flags, xs, as_, bs = _inputs(x, a, b)
    N, cf = _sequences(cu_seqlens, device)
    sdt, sstride, n_pool, sf = _states(initial_state, output_state, state_indices, N, H, D, device)
    ys = 0
    if output is None:
        output = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        ys = _tokens("output", output, x.shape, x.dtype, device)
    if tile_states is not None and _tokens("tile_states", tile_states, (-(-T // LINEAR_TILE), H, D), torch.float32, device):
        raise ValueError("tile_states must be contiguous")
    plan = _get_plan(H, D, x, a, sdt, flags | cf | sf, T, N)
    args = _pack(x.data_ptr(), a.data_ptr(), _addr(b), xs, as_, bs, _addr(cu_seqlens), N, T, _addr(initial_state),
                 _addr(output_state), sstride, _addr(state_indices), n_pool, _status_ptr(device_status, device),
                 output.data_ptr(), ys, _addr(tile_states), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    _run(0, plan, x, args)
    _written(output, output_state, tile_states)
    return output


class _Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, a, b, initial_state, cu_seqlens, output_final_state, device_status):
        T, H, D = x.shape
        N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
        final = _new_states(initial_state, N, H, D, x.device) if output_final_state else None
        tiles = torch.empty(-(-T // LINEAR_TILE), H, D, dtype=torch.float32, device=x.device)
        y = _forward(x, a, b, initial_state, final, cu_seqlens, None, None, tiles, device_status)
        ctx.save_for_backward(x, a, b, initial_state, cu_seqlens, tiles)
        ctx.device_status = device_status  # written to, never read: the caller may clear it in between
        ctx.set_materialize_grads(False)  # a final state that the loss does not use has no gradient to be read
        return y, final

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, d_final):
        x, a, b, initial_state, cu_seqlens, tiles = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros_like(x)
        dx, da, db, d0 = gated_linear_recurrence_backward(
            dy.contiguous(), x, a, b, tile_states=tiles, initial_state=initial_state,
            d_final_state=None if d_final is None else d_final.float().contiguous(), cu_seqlens=cu_seqlens,
            device_status=ctx.device_status)
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
    device data (``DEVICE_ERR``); without it such errors go unreported, and the outputs are unspecified where they occur.  (A
    wait inside a kernel that ran out, "TIMEOUT", leaves NaN in all that depends on it.)  Returns ``output`` or ``(output, final_state)``.

    Differentiable in x, a, b and initial_state when called without output, output_state, state_indices and
    tile_states.

    Fastest where tokens of x, a and b are multiples of 16 bytes at addresses that are, too.  Gates per head whose rows are not
    (12 heads in bf16, for one; in fp32 they are) take about twice as long in both directions.
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
    device, T, H, D, flags, xs, as_, bs = _inputs(x, a, b)
    N, cf = _sequences(cu_seqlens, device)
    sdt, sstride, _, sf = _states(initial_state, None, None, N, H, D, device)
    dys = _tokens("dy", dy, x.shape, x.dtype, device)
    if tile_states is not None:
        if _tokens("tile_states", tile_states, (-(-T // LINEAR_TILE), H, D), torch.float32, device):
            raise ValueError("tile_states must be contiguous")
    elif T > LINEAR_TILE:
        raise ValueError("tile_states of the forward run are needed")
    if d_final_state is not None and _tokens("d_final_state", d_final_state, (N, H, D), torch.float32, device):
        raise ValueError("d_final_state must be contiguous")
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    da = torch.empty(a.shape, dtype=a.dtype, device=x.device)
    db = torch.empty_like(da) if b is not None else None
    d0 = torch.empty(N, H, D, dtype=torch.float32, device=x.device) if initial_state is not None else None
    plan = _get_plan(H, D, x, a, sdt, flags | cf | sf, T, N)
    args = _pack(x.data_ptr(), a.data_ptr(), _addr(b), xs, as_, bs, _addr(cu_seqlens), N, T, _addr(initial_state), 0, sstride, 0, 0,
                 _status_ptr(device_status, device), 0, 0, _addr(tile_states), dy.data_ptr(), dys, _addr(d_final_state), _addr(d0),
                 dx.data_ptr(), da.data_ptr(), _addr(db), 0, 0, 0)
    _run(1, plan, x, args)
    return dx, da, db, d0


def gated_linear_recurrence_decode(x, a, b=None, initial_state=None, state_indices=None, output_final_state=True,
                                   output_state=None, tokens_per_seq=1, output=None, device_status=None):
    """Decode step (or a short run of tokens) of :func:`gated_linear_recurrence`: N sequences of ``tokens_per_seq``
    tokens each, rows i * tokens_per_seq + j of x, a and b.  With ``state_indices`` the state is read from its pool row
    and written back in place (or to ``output_state``'s row).  Returns ``output`` or ``(output, final_state)``.  A step of
    serving: not differentiable."""
    device, T, H, D, flags, xs, as_, bs = _inputs(x, a, b)
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
            output_state = _new_states(initial_state, N, H, D, x.device)
    sdt, sstride, n_pool, sf = _states(initial_state, output_state, state_indices, N, H, D, device)
    ys = 0
    if output is None:
        output = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        ys = _tokens("output", output, x.shape, x.dtype, device)
    plan = _get_plan(H, D, x, a, sdt, flags | sf, T, N)
    args = _pack(x.data_ptr(), a.data_ptr(), _addr(b), xs, as_, bs, 0, N, T, _addr(initial_state), _addr(output_state), sstride,
                 _addr(state_indices), n_pool, _status_ptr(device_status, device), output.data_ptr(), ys, 0, 0, 0, 0, 0, 0, 0, 0, 0,
                 0, 0)
    with on_device(device) as stream:
        st = lib().gdn_linear_decode_run(plan.handle, args, m, stream)
    if st != 0:
        raise GdnError(st, "gdn_linear_decode_run")
    _written(output, output_state)
    return (output, output_state) if output_final_state else output

"""Rotary positions, writing keys and values into a paged cache, and attention over that cache.

What the attention layers beside gated delta rule layers need, on the same packed batches and on the pages that
:func:`cache_reserve` and its siblings hand out: a step reserves pages, advances ``lengths``, and calls, layer by layer,
:func:`cache_append` and :func:`paged_attention`.  Prompts, chunks of prompts and single tokens go through the same calls, mixed in
any way.  Like the package's other calls these marshal arguments for the C ABI (``include/gdn_attention.h``); the work is done
by the kernels of ``libgdn_prefill.so``.  :func:`rotary_embedding` is differentiable.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch
from torch.autograd.graph import increment_version

from . import _QKV_DTYPES, GdnError, lib, on_device
from .linear import _addr, _sequences, _status_ptr, _tokens
from .pages import _int32

__all__ = ["rotary_frequencies", "rotary_embedding", "rotary_embedding_backward", "cache_append", "paged_attention", "KvBatch",
           "KvCache", "RotaryArgs", "AttentionArgs"]


class KvBatch(ctypes.Structure):
    _fields_ = [("cu_seqlens", ctypes.c_void_p), ("seqs", ctypes.c_void_p), ("table", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("total_tokens", ctypes.c_int64), ("num_seqs", ctypes.c_int32), ("tokens_per_seq", ctypes.c_int32),
                ("cu_i64", ctypes.c_int32), ("max_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("device_status", ctypes.c_void_p)]


class KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_page_stride", ctypes.c_int64), ("k_token_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("v_page_stride", ctypes.c_int64), ("v_token_stride", ctypes.c_int64),
                ("v_head_stride", ctypes.c_int64), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class RotaryArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64),
                ("k_out_stride", ctypes.c_int64), ("frequencies", ctypes.c_void_p), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("inverse", ctypes.c_int32), ("magnitude", ctypes.c_float),
                ("dtype", ctypes.c_int32)]


class AttentionArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("output", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                ("output_stride", ctypes.c_int64), ("heads", ctypes.c_int32), ("scale", ctypes.c_float), ("causal", ctypes.c_int32),
                ("window", ctypes.c_int32)]


# The bytes of the structures above, in C's alignment: the calls pack their arguments in one go.
_pack_batch = struct.Struct("@PPPPqiiiiiiiP").pack
_pack_cache = struct.Struct("@PPqqqqqqiii4x").pack
_pack_rotary = struct.Struct("@PPPPqqqqPiiiiiifi").pack
_pack_attention = struct.Struct("@PPPqqifii").pack


def _register(L):
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L.gdn_rotary_run.argtypes = [vp, vp, i32, vp, i32, i32, i64, vp]
    L.gdn_cache_append_run.argtypes = [vp, vp, vp, vp, i64, vp]
    L.gdn_attention_workspace.argtypes = [vp, vp, vp]
    L.gdn_attention_workspace.restype = sz
    L.gdn_attention_run.argtypes = [vp, vp, vp, vp, sz, vp]
    for fn in (L.gdn_rotary_run, L.gdn_cache_append_run, L.gdn_attention_run):
        fn.restype = ctypes.c_int


def rotary_frequencies(rotary_dim, base=10000.0, factor=1.0, original_length=None, slow_turns=1.0, fast_turns=32.0, device="cuda"):
    """Angles a token (radians, float64 [rotary_dim / 2]): ``base ** (-2 i / rotary_dim)``, slowed down for longer contexts.

    ``factor`` divides all of them; with ``original_length`` (the context that a model was trained on) only those that turn
    at most ``slow_turns`` times over that length are divided, those that turn ``fast_turns`` times or more stay, and in
    between the two are mixed in proportion to the number of turns.  (Models whose released code mixes in proportion to the channel's
    index between those two numbers of turns need frequencies of their own: any float64 vector will do.)"""
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even")
    if not (base > 0 and factor > 0):
        raise ValueError("base and factor must be positive")
    f = float(base) ** (-2.0 * torch.arange(rotary_dim // 2, dtype=torch.float64) / max(rotary_dim, 1))
    if original_length is None:
        f = f / factor
    else:
        if not fast_turns > slow_turns:
            raise ValueError("fast_turns must be above slow_turns")
        kept = ((original_length * f / (2 * math.pi) - slow_turns) / (fast_turns - slow_turns)).clamp(0, 1)
        f = f * (kept + (1 - kept) / factor)
    return f.to(device)


def _heads(name, t, T, D, dtype, device):
    """Checks [T, heads, D]; returns the heads and the token stride (0: dense)."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [total_tokens, heads, head_dim]")
    return t.shape[1], _tokens(name, t, (T, t.shape[1], D), dtype, device)


def _first(name, t):
    """(T, D, dtype, device) of a call's first tensor."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [total_tokens, heads, head_dim]")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor: this library has no CPU path")
    if t.dtype not in _QKV_DTYPES:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return t.shape[0], t.shape[2], t.dtype, t.get_device()


def _frequencies(f, D, device):
    """Checks the frequencies; returns the rotary dimension and their address."""
    if f is None:
        return 0, 0
    if f.dtype is not torch.float64 or f.dim() != 1 or f.get_device() != device or not f.is_contiguous():
        raise ValueError(f"frequencies must be a contiguous float64 vector on cuda:{device}")
    if 2 * f.numel() > D:
        raise ValueError(f"{f.numel()} frequencies turn more than the {D} channels of a head")
    return 2 * f.numel(), f.data_ptr()


def _out(name, out, like, T, D, dtype, device):
    """The output tensor (a new one without `out`) and its token stride."""
    if out is None:
        return torch.empty_like(like) if like.is_contiguous() else torch.empty(like.shape, dtype=dtype, device=like.device), 0
    return out, _tokens(name, out, like.shape, dtype, device)


def _rotary(q, k, frequencies, positions, cu_seqlens, interleaved, magnitude, q_out, k_out, inverse):
    T, D, dtype, device = _first("q", q) if q is not None else _first("k", k)
    R, f = _frequencies(frequencies, D, device)
    pos64, N, cf = 0, 0, 0
    if positions is not None:
        if cu_seqlens is not None:
            raise ValueError("give positions or cu_seqlens, not both")
        if positions.shape != (T,) or positions.get_device() != device or not positions.is_contiguous() or \
                positions.dtype not in (torch.int32, torch.int64):
            raise ValueError(f"positions must be contiguous int32 or int64 [{T}] on cuda:{device}")
        pos64 = int(positions.dtype is torch.int64)
    elif cu_seqlens is not None:
        N, cf = _sequences(cu_seqlens, device)
    Hq = Hk = qs = ks = qos = kos = 0
    if q is not None:
        Hq, qs = _heads("q", q, T, D, dtype, device)
        q_out, qos = _out("q_out", q_out, q, T, D, dtype, device)
    if k is not None:
        Hk, ks = _heads("k", k, T, D, dtype, device)
        k_out, kos = _out("k_out", k_out, k, T, D, dtype, device)
    args = _pack_rotary(_addr(q), _addr(k), _addr(q_out), _addr(k_out), qs, ks, qos, kos, f, Hq, Hk, D, R, int(bool(interleaved)),
                        inverse, float(magnitude), _QKV_DTYPES[dtype])
    with on_device(device) as stream:
        st = lib().gdn_rotary_run(args, _addr(positions), pos64, _addr(cu_seqlens), int(cf != 0), N, T, stream)
    if st != 0:
        raise GdnError(st, "gdn_rotary_run")
    return q_out, k_out


class _Serving(torch.autograd.Function):
    """A step of serving: what `run` returns, with a history that says that there is no gradient."""

    @staticmethod
    def forward(ctx, name, run, *inputs):
        ctx.name = name
        return run()

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name} is a step of serving and has no gradient; a loss through it needs the attention in other "
                           "operations, serving torch.no_grad()")


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, frequencies, positions, cu_seqlens, interleaved, magnitude):
        ctx.save_for_backward(frequencies, positions, cu_seqlens)
        ctx.how = interleaved, magnitude
        ctx.set_materialize_grads(False)
        return _rotary(q, k, frequencies, positions, cu_seqlens, interleaved, magnitude, None, None, 0)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk):
        if ctx.needs_input_grad[2]:
            raise RuntimeError("rotary_embedding has no gradient with respect to its frequencies")
        frequencies, positions, cu_seqlens = ctx.saved_tensors
        dq, dk = (d.contiguous() if d is not None and n else None for d, n in zip((dq, dk), ctx.needs_input_grad))
        if dq is not None or dk is not None:
            dq, dk = _rotary(dq, dk, frequencies, positions, cu_seqlens, *ctx.how, None, None, 1)
        return dq, dk, None, None, None, None, None


def rotary_embedding(q, k, frequencies, positions=None, cu_seqlens=None, interleaved=False, magnitude=1.0, q_out=None, k_out=None):
    """Turns pair i of every head of ``q`` [T, heads, D] and ``k`` [T, kv_heads, D] (either may be None) by position times
    ``frequencies[i]`` (float64, radians, see :func:`rotary_frequencies`) and multiplies it by ``magnitude``.  The pairs are
    channels (i, i + R / 2) of the first R = 2 * len(frequencies), or (2 i, 2 i + 1) when ``interleaved``; the channels behind
    R stay as they are.  Positions are ``positions`` [T] (int32 or int64, as far as 2^31), or count from 0 in each sequence of
    ``cu_seqlens`` (int32 or int64; rows past its end go on counting), or from 0 over all rows.  Tokens may be strided (slices of a
    projection's output).  ``q_out`` and ``k_out`` may be q and k themselves, or are apart from them and from each other.  Returns ``(q_out, k_out)``.

    Differentiable in q and k when called without q_out and k_out; not in the frequencies (a backward pass that would need their
    gradients raises an error)."""
    if q is None and k is None:
        raise ValueError("q or k must be given")
    if (q is None and q_out is not None) or (k is None and k_out is not None):
        raise ValueError("q_out needs q, and k_out needs k")
    if torch.is_grad_enabled() and ((q is not None and q.requires_grad) or (k is not None and k.requires_grad)):
        if q_out is not None or k_out is not None:
            raise ValueError("q_out and k_out cannot be differentiated through")
        return _Rotary.apply(q, k, frequencies, positions, cu_seqlens, interleaved, magnitude)
    if frequencies is not None and frequencies.requires_grad and torch.is_grad_enabled() and q_out is None and k_out is None:
        return _Rotary.apply(q, k, frequencies, positions, cu_seqlens, interleaved, magnitude)
    out = _rotary(q, k, frequencies, positions, cu_seqlens, interleaved, magnitude, q_out, k_out, 0)
    if q_out is not None or k_out is not None:
        increment_version([t for t in (q_out, k_out) if t is not None])
    return out


def rotary_embedding_backward(dq, dk, frequencies, positions=None, cu_seqlens=None, interleaved=False, magnitude=1.0):
    """Gradients of :func:`rotary_embedding` with respect to q and k, from those of its results: the turn the other way."""
    if dq is None and dk is None:
        raise ValueError("dq or dk must be given")
    return _rotary(dq, dk, frequencies, positions, cu_seqlens, interleaved, magnitude, None, None, 1)


def _cache(k_cache, v_cache, D, dtype, device):
    """Checks the caches; returns them packed, with pages, tokens a page and heads."""
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.shape[3] != D:
        raise ValueError(f"k_cache and v_cache must be [pages, page_tokens, kv_heads, {D}]")
    strides = []
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype is not dtype or t.get_device() != device:
            raise ValueError(f"{name} must be {dtype} on cuda:{device}")
        if D > 1 and t.stride(3) != 1:
            raise ValueError(f"{name} must have contiguous channels")
        strides += t.stride()[:3]
    P, pt, Hk, _ = k_cache.shape
    if max(P, pt) > 0x7fffffff:
        raise ValueError("pages and their tokens must fit 32 bits")
    return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), *strides, Hk, D, _QKV_DTYPES[dtype]), P, pt, Hk


def _batch(T, table, lengths, seqs, cu_seqlens, tokens_per_seq, P, pt, device_status, device):
    """Checks a step's sequences; returns them packed."""
    if table.dim() != 2:
        raise ValueError("table must be [sequences, max_pages]")
    S, M = table.shape
    N, m, cf = 1 if T else 0, max(T, 1), 0
    if cu_seqlens is not None:
        if tokens_per_seq is not None:
            raise ValueError("give cu_seqlens or tokens_per_seq, not both")
        N, cf = _sequences(cu_seqlens, device)
        m = 0
    elif tokens_per_seq is not None:
        m = int(tokens_per_seq)
        if m < 1 or T % m:
            raise ValueError("there must be N * tokens_per_seq rows")
        N = T // m
    if seqs is None and N > S:
        raise ValueError(f"{N} sequences need as many rows of table, not {S}")
    return _pack_batch(_addr(cu_seqlens), 0 if seqs is None else _int32("seqs", seqs, (N,), device), _int32("table", table, (S, M), device),
                       _int32("lengths", lengths, (S,), device), T, N, m, int(cf != 0), S, M, P, pt, _status_ptr(device_status, device))


def cache_append(k, v, k_cache, v_cache, table, lengths, seqs=None, cu_seqlens=None, tokens_per_seq=None, q=None, frequencies=None,
                 interleaved=False, magnitude=1.0, output=None, device_status=None):
    """Writes the new tokens' keys (turned as by :func:`rotary_embedding`, unless ``frequencies`` is None) and values [T,
    kv_heads, D] into their pages of ``k_cache`` and ``v_cache`` [pages, page_tokens, kv_heads, D] (any strides over contiguous
    channels).  The batch is packed by ``cu_seqlens`` [N + 1], or has ``tokens_per_seq`` tokens a sequence (decode), or is one
    sequence; sequence i is row ``seqs[i]`` (None: i) of ``table`` and ``lengths``, and ``lengths`` counts the new tokens already: new
    token j of n has position lengths - n + j.  ``q`` [T, heads, D], when given, is turned as well, to ``output`` (a new tensor
    without it; q itself is allowed, else apart from q, k and v) in the same launch.  Returns that, or None.

    No two entries of ``seqs`` may name one row.  Tokens without a page are not written (``device_status``, an int32 tensor, receives
    the bits of DEVICE_ERR and PAGES_ERR).  Rows past the last sequence are padding and stay as they are.  A step of serving: not
    differentiable (a backward pass through a new output raises an error; one through ``output`` or the caches ends there)."""
    if output is None and q is not None and torch.is_grad_enabled() and (q.requires_grad or (frequencies is not None and frequencies.requires_grad)):
        return _Serving.apply("cache_append", lambda: _append(k, v, k_cache, v_cache, table, lengths, seqs, cu_seqlens, tokens_per_seq, q, frequencies,
                                                              interleaved, magnitude, None, device_status), q, frequencies)
    return _append(k, v, k_cache, v_cache, table, lengths, seqs, cu_seqlens, tokens_per_seq, q, frequencies, interleaved, magnitude, output,
                   device_status)


def _append(k, v, k_cache, v_cache, table, lengths, seqs, cu_seqlens, tokens_per_seq, q, frequencies, interleaved, magnitude, output, device_status):
    T, D, dtype, device = _first("k", k)
    packed, P, pt, Hk = _cache(k_cache, v_cache, D, dtype, device)
    batch = _batch(T, table, lengths, seqs, cu_seqlens, tokens_per_seq, P, pt, device_status, device)
    R, f = _frequencies(frequencies, D, device)
    ks, vs = _tokens("k", k, (T, Hk, D), dtype, device), _tokens("v", v, (T, Hk, D), dtype, device)
    Hq = qs = os_ = 0
    given = output
    if q is not None:
        Hq, qs = _heads("q", q, T, D, dtype, device)
        output, os_ = _out("output", output, q, T, D, dtype, device)
    elif output is not None:
        raise ValueError("output needs q")
    args = _pack_rotary(_addr(q), k.data_ptr(), _addr(output), 0, qs, ks, os_, 0, f, Hq, Hk, D, R, int(bool(interleaved)), 0,
                        float(magnitude), _QKV_DTYPES[dtype])
    with on_device(device) as stream:
        st = lib().gdn_cache_append_run(batch, packed, args, v.data_ptr(), vs, stream)
    if st != 0:
        raise GdnError(st, "gdn_cache_append_run")
    increment_version((k_cache, v_cache) if given is None else (k_cache, v_cache, given))
    return output


def paged_attention(q, k_cache, v_cache, table, lengths, seqs=None, cu_seqlens=None, tokens_per_seq=None, scale=None, causal=True,
                    window=0, output=None, lse=None, device_status=None):
    """Attention of the new tokens ``q`` [T, heads, D] over their sequences in the cache (see :func:`cache_append` for the
    batch and the caches; the new tokens' own keys and values are there already).  Head h reads key head
    h // (heads // kv_heads).  New token j of n, at position p = lengths - n + j, sees the sequence's tokens up to p (all of them
    without ``causal``), and with ``window`` only those after p - window.  ``scale`` is 1 / sqrt(D) by default.  ``lse`` [T, heads]
    fp32, when given, receives the logarithm of the sum of the scores' exponentials.  Returns ``output`` [T, heads, D].

    A token that sees nothing gets zeros (lse: minus infinity; so does one that sees only scores of minus infinity); what a token
    does not see has no influence on it, whatever it holds.  A channel in which it sees an infinite value is infinite (NaN, where it
    sees both signs or NaN, or where the weight, rounded to q's type, vanishes).  Sums of weights times values are fp32: values past
    the largest fp32 divided by the number of keys may overflow.  ``output``, when given, has its rows apart from q's (slices of one
    tensor are allowed), and ``lse`` lies apart from both.  ``device_status`` (int32) receives the bits of DEVICE_ERR and PAGES_ERR;
    what has no page is not seen.  After "TIMEOUT", a wait inside the kernel that ran out, what depends on it is NaN.  Rows past the last sequence are padding and stay as they
    are.  D is at most 256.  A step of serving: not differentiable (a backward pass through a new output raises an error; one through
    ``output`` or ``lse`` ends there).

    Fastest in bf16 and fp16 where D is a multiple of 8, pages have a multiple of 8 tokens, and q's and the caches' strides and
    addresses are multiples of 16 bytes.  Other pages, strides and addresses take two to ten times as long.  On CUDA cores, at about a
    fortieth of the rate, are computed: fp32; rows (heads, strides or addresses of q and the caches) that are no multiples of 4 bytes;
    and few tokens of up to 124 channels (64, where rows are multiples of 8 bytes) in rows that are no multiples of 16 bytes."""
    if output is None and torch.is_grad_enabled() and (q.requires_grad or k_cache.requires_grad or v_cache.requires_grad):
        return _Serving.apply("paged_attention", lambda: _attend(q, k_cache, v_cache, table, lengths, seqs, cu_seqlens, tokens_per_seq, scale, causal,
                                                                 window, None, lse, device_status), q, k_cache, v_cache)
    return _attend(q, k_cache, v_cache, table, lengths, seqs, cu_seqlens, tokens_per_seq, scale, causal, window, output, lse, device_status)


def _attend(q, k_cache, v_cache, table, lengths, seqs, cu_seqlens, tokens_per_seq, scale, causal, window, output, lse, device_status):
    T, D, dtype, device = _first("q", q)
    packed, P, pt, Hk = _cache(k_cache, v_cache, D, dtype, device)
    Hq, qs = _heads("q", q, T, D, dtype, device)
    if Hk < 1 or Hq < 1 or Hq % Hk:
        raise ValueError(f"{Hq} heads cannot share {Hk} key heads")
    if window < 0:
        raise ValueError("window must not be negative")
    batch = _batch(T, table, lengths, seqs, cu_seqlens, tokens_per_seq, P, pt, device_status, device)
    given = output
    output, os_ = _out("output", output, q, T, D, dtype, device)
    if given is not None and T and given.data_ptr() == q.data_ptr():
        raise ValueError("output must be apart from q")
    if lse is not None and _tokens("lse", lse, (T, Hq), torch.float32, device):
        raise ValueError("lse must be contiguous")
    args = _pack_attention(q.data_ptr(), output.data_ptr(), _addr(lse), qs, os_, Hq,
                           1.0 / math.sqrt(D) if scale is None else float(scale), int(bool(causal)), min(int(window), 0x7fffffff))
    L = lib()
    with on_device(device) as stream:
        n = L.gdn_attention_workspace(batch, packed, args)
        ws = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
        st = L.gdn_attention_run(batch, packed, args, _addr(ws), n, stream)
    if st != 0:
        raise GdnError(st, "gdn_attention_run")
    if given is not None or lse is not None:
        increment_version([t for t in (given, lse) if t is not None])
    return output

"""Inputs, expected values and bounds of the tests of rotary positions, cache writes and attention over pages."""
import numpy as np
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from oracle import attention as ref

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = {**gdn.DEVICE_ERR, **gdn.PAGES_ERR}


def f64(t):
    return t.detach().double().cpu().numpy()


def half_step(want, dtype):
    """Half a unit in the last place, relative, and half the distance of subnormals."""
    info = torch.finfo(dtype)
    return np.abs(want) * info.eps / 2 + info.smallest_normal * info.eps / 2


def close(name, got, want, lim):
    got = f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    same = (got == want) | (np.isnan(got) & np.isnan(want))  # infinities, and what the definition has as NaN
    off = np.where(same, 0, np.abs(np.where(same, 0, got) - np.where(same, 0, want)))
    bad = ~same & ~(off <= lim)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size} off, worst {np.nanmax(off - lim):.3g} at {np.argwhere(bad)[0]}"


def close_rotary(name, got, want, size, dtype):
    """The angle is exact but for 2^-32 of a turn; its remainder, sine and cosine (2 units each), the magnitude's product and the two
    products and sum of the turn are fp32: fewer than 8 roundings of 2^-24 of |a| + |b|.  Then one rounding to the type."""
    lim = 8 * 2.0 ** -24 * size
    close(name, got, want, lim + np.where(size > 0, half_step(np.abs(want) + lim, dtype), 0))


def attention_bound(out, size, products, count, D, dtype):
    """Scores: D products and sums in fp32 (2^-23 each: the tensor cores cut instead of rounding), their scaling and the
    exponential: relative errors of a weight, once in the numerator and once in the sum.  A weight's rounding to a 16-bit type, which
    the sum of weights does not see.  The sums over the keys, the join's weights, the division: fp32.  Then one rounding."""
    score = (D + 8) * 2.0 ** -23 * products[..., None] + 2.0 ** -20
    weight = torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0
    lim = size * (2 * score * (1 + score) + weight + (count[..., None] + 16) * 2.0 ** -23)
    return lim + half_step(np.abs(out) + lim, dtype) + 2.0 ** -126


class Cache:
    """Sequences of given lengths (with the new tokens) in pages in random order; what belongs to nobody is NaN."""

    def __init__(self, lens, past, heads, kv_heads, D, page_tokens, dtype, seed=0, layout="token", spare=3, fill=float("nan")):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.dtype, self.D = list(lens), TYPES[dtype], D
        dt, N = self.dtype, len(lens)
        total = [p + n for p, n in zip(past, lens)]
        need = [-(-max(t, 0) // page_tokens) for t in total]
        S, P, M = N + spare, sum(need) + 2, max(need + [1])
        order = torch.randperm(P, generator=g).tolist()
        self.seqs = torch.randperm(S, generator=g)[:N].to(torch.int32)
        self.table = torch.full((S, M), -1, dtype=torch.int32)
        self.lengths = torch.zeros(S, dtype=torch.int32)
        shape = (P, page_tokens, kv_heads, D)
        self.k, self.v = torch.full(shape, fill), torch.full(shape, fill)
        for s, t, n in zip(self.seqs.tolist(), total, need):
            pages = [order.pop() for _ in range(n)]
            self.table[s, :n] = torch.tensor(pages, dtype=torch.int32)
            self.lengths[s] = t
            for i, p in enumerate(pages):
                m = min(page_tokens, t - i * page_tokens)
                self.k[p, :m] = torch.randn(m, kv_heads, D, generator=g)
                self.v[p, :m] = torch.randn(m, kv_heads, D, generator=g)
        self.q = (1.5 * torch.randn(sum(lens), heads, D, generator=g)).to(dt)
        self.k, self.v = self.k.to(dt), self.v.to(dt)
        self.cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)
        self.layout = layout

    def placed(self, t):
        """On the GPU, in one of four layouts: tokens before heads, heads before tokens, or rows wider than needed, by 8 channels or 1."""
        t = t.cuda()
        if self.layout == "head":
            return t.transpose(1, 2).contiguous().transpose(1, 2)
        if self.layout in ("wide", "odd"):
            P, pt, H, D = t.shape
            whole = torch.full((P, 2, pt, H, D + (8 if self.layout == "wide" else 1)), float("nan"), dtype=t.dtype, device="cuda")
            whole[:, 1, :, :, :D] = t
            return whole[:, 1, :, :, :D]
        return t

    def gpu(self):
        return dict(k_cache=self.placed(self.k), v_cache=self.placed(self.v), table=self.table.cuda(), lengths=self.lengths.cuda(),
                    seqs=self.seqs.cuda())

    def want(self, scale=None, causal=True, window=0):
        scale = self.D ** -0.5 if scale is None else scale
        return ref.attend(f64(self.q), f64(self.k), f64(self.v), self.table.numpy().astype(np.int64), self.lengths.tolist(),
                          self.seqs.tolist(), self.lens, scale, causal, window)

    def check(self, scale=None, causal=True, window=0, tokens=None, status=0, strided=False, **kw):
        """Runs the kernels and compares outputs and logarithms; returns the output."""
        T, H, D = self.q.shape
        out, lse, size, products, count = self.want(scale, causal, window)
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        got_lse = torch.full((T, H), float("nan"), device="cuda")
        q = self.q.cuda()
        if strided:
            whole = torch.full((T, H + 3, D), float("nan"), dtype=self.dtype, device="cuda")
            whole[:, 1: H + 1] = q
            q = whole[:, 1: H + 1]
        how = dict(tokens_per_seq=tokens) if tokens else dict(cu_seqlens=self.cu.cuda())
        got = gdn.paged_attention(q, **{**self.gpu(), **kw}, **how, scale=scale, causal=causal, window=window, lse=got_lse,
                                  device_status=word)
        assert int(word) == status, int(word)
        close("output", got, out, attention_bound(out, size, products, count, D, self.dtype))
        score = (D + 8) * 2.0 ** -23 * products + 2.0 ** -20
        close("lse", got_lse, lse, np.where(np.isfinite(lse), score + np.abs(np.where(np.isfinite(lse), lse, 0)) * 2.0 ** -22 +
                                            (count + 16) * 2.0 ** -23, 0))
        return got

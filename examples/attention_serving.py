"""An attention layer with rotary positions, served from pages of a key/value cache.

    python examples/attention_serving.py

Training: gradients through the rotary positions of a packed batch.  Serving: two prompts come in chunks, each is forked into several
answers (full pages are shared, the partly filled one is copied), the answers decode token by token, two are dropped, and what is left
moves to the front of the cache.  A step reserves pages, advances the lengths, writes the new keys and values and attends.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_chunked_device_gb300 as gdn  # noqa: E402


class Layer(torch.nn.Module):
    """hidden -> (queries, keys, values) -> attention -> out; `heads` share `kv_heads` keys, half of each head is turned."""

    def __init__(self, width, heads, kv_heads, dim, device="cuda", dtype=torch.bfloat16):
        super().__init__()
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.project = torch.nn.Linear(width, (heads + 2 * kv_heads) * dim, bias=False, device=device, dtype=dtype)
        self.out = torch.nn.Linear(heads * dim, width, bias=False, device=device, dtype=dtype)
        self.frequencies = gdn.rotary_frequencies(dim // 2, factor=4.0, original_length=256, device=device)

    def qkv(self, hidden):
        return self.project(hidden).view(-1, self.heads + 2 * self.kv_heads, self.dim).split([self.heads, self.kv_heads, self.kv_heads], dim=1)

    def forward(self, hidden, cu_seqlens):
        """A packed batch of whole sequences, differentiable (the attention itself in plain torch)."""
        q, k, v = self.qkv(hidden)
        q, k = gdn.rotary_embedding(q, k, self.frequencies, cu_seqlens=cu_seqlens)
        group, outs, bounds = self.heads // self.kv_heads, [], cu_seqlens.tolist()
        for a, b in zip(bounds, bounds[1:]):
            x, y, z = q[a:b].float(), k[a:b].float().repeat_interleave(group, 1), v[a:b].float().repeat_interleave(group, 1)
            s = torch.einsum("thd,shd->hts", x, y) / self.dim ** 0.5
            s = s.masked_fill(torch.ones(b - a, b - a, dtype=torch.bool, device=s.device).triu(1), float("-inf"))
            outs.append(torch.einsum("hts,shd->thd", s.softmax(-1), z))
        return self.out(torch.cat(outs).to(hidden.dtype).flatten(1))

    def step(self, hidden, cache, seqs, **batch):
        """New tokens of the sequences `seqs` of a cache whose lengths count them already."""
        q, k, v = self.qkv(hidden)
        pools = cache["k"], cache["v"]
        where = dict(seqs=seqs, device_status=cache["status"], **batch)
        q = gdn.cache_append(k, v, *pools, cache["table"], cache["lengths"], q=q, frequencies=self.frequencies, **where)
        return self.out(gdn.paged_attention(q, *pools, cache["table"], cache["lengths"], **where).flatten(1))


def ids(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def make_cache(layer, pages=64, page_tokens=16, seqs=16):
    dtype = layer.out.weight.dtype
    pools = [torch.empty(pages, page_tokens, layer.kv_heads, layer.dim, device="cuda", dtype=dtype) for _ in range(2)]
    z = dict(dtype=torch.int32, device="cuda")
    return dict(k=pools[0], v=pools[1], table=torch.full((seqs, pages // 2), -1, **z), refcounts=torch.zeros(pages, **z),
                lengths=torch.zeros(seqs, **z), status=torch.zeros(1, **z), page_tokens=page_tokens)


def advance(cache, seqs, new):
    """Counts the new tokens and gives their pages to the sequences."""
    cache["lengths"][seqs.long()] += new
    counts = (cache["lengths"][seqs.long()] + cache["page_tokens"] - 1) // cache["page_tokens"]
    gdn.cache_reserve(cache["table"], cache["refcounts"], seqs, counts.int(), device_status=cache["status"])


@torch.no_grad()
def serve(layer, width, generator):
    """Returns the prompts' and the answers' outputs with the hidden states that went in, and the cache."""
    dtype, cache = layer.out.weight.dtype, make_cache(layer)
    book = cache["table"], cache["refcounts"]

    def hidden(n):
        return torch.randn(n, width, generator=generator, device="cuda").to(dtype)

    prompts, seen = ids(0, 1), []
    for chunk in ((70, 37), (30, 0)):
        x, cu = hidden(sum(chunk)), ids(0, chunk[0], sum(chunk))
        advance(cache, prompts, ids(*chunk))
        seen.append((prompts.tolist(), chunk, x, layer.step(x, cache, prompts, cu_seqlens=cu)))

    answers = ids(2, 3, 4, 5, 6)  # three to the first prompt, two to the second
    gdn.cache_fork([cache["k"], cache["v"]], *book, ids(0, 0, 0, 1, 1), answers, page_tokens=cache["page_tokens"], lengths=cache["lengths"],
                   device_status=cache["status"])
    gdn.cache_free(*book, prompts, lengths=cache["lengths"], device_status=cache["status"])
    for step in range(40):
        if step == 20:  # two answers are done; what is left moves to the front
            gdn.cache_free(*book, ids(2, 5), lengths=cache["lengths"], device_status=cache["status"])
            gdn.cache_compact([cache["k"], cache["v"]], *book, device_status=cache["status"])
            answers = ids(3, 4, 6)
        x = hidden(answers.numel())
        advance(cache, answers, 1)
        seen.append((answers.tolist(), (1,) * answers.numel(), x, layer.step(x, cache, answers, tokens_per_seq=1)))
    assert int(cache["status"]) == 0, int(cache["status"])
    return seen, cache


def main():
    gdn.build()
    torch.manual_seed(0)
    g = torch.Generator(device="cuda").manual_seed(1)
    layer = Layer(256, 8, 2, 64)
    x = torch.randn(300, 256, generator=g, device="cuda").bfloat16()
    layer(x, ids(0, 170, 170, 300)).float().square().mean().backward()
    print("gradient of the projection:", float(layer.project.weight.grad.float().norm()))
    seen, cache = serve(layer, 256, g)
    print("tokens:", sum(x.shape[0] for _, _, x, _ in seen), "lengths:", cache["lengths"][cache["lengths"] > 0].tolist(),
          "live pages:", int((cache["refcounts"] > 0).sum()))


if __name__ == "__main__":
    main()

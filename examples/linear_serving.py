"""A layer with a gated linear recurrence, trained for a step and then served from a pool of states.

    python examples/linear_serving.py

Training: the gradients of one packed batch, through autograd.  Serving: pages (one state row a sequence) are reserved,
two prompts of different length prefill their states, each is forked into several answers, the answers decode token by
token in place, the shorter ones are dropped, and what is left moves to the front of the pool.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_chunked_device_gb300 as gdn  # noqa: E402


class Layer(torch.nn.Module):
    """x -> (values, decays, input gates) -> recurrence -> out, heads of `dim` channels, gates per channel."""

    def __init__(self, width, heads, dim, device="cuda", dtype=torch.bfloat16):
        super().__init__()
        self.heads, self.dim = heads, dim
        self.project = torch.nn.Linear(width, 3 * heads * dim, bias=False, device=device, dtype=dtype)
        self.out = torch.nn.Linear(heads * dim, width, bias=False, device=device, dtype=dtype)

    def gates(self, hidden):
        v, r, i = self.project(hidden).view(-1, 3, self.heads, self.dim).unbind(1)
        return v, torch.exp(-torch.nn.functional.softplus(r.float()) / 16), torch.sigmoid(i.float())

    def forward(self, hidden, cu_seqlens):
        v, a, b = self.gates(hidden)
        y = gdn.gated_linear_recurrence(v, a, b, cu_seqlens=cu_seqlens)
        return self.out(y.flatten(1))

    def prefill(self, hidden, cu_seqlens, pool, rows):
        v, a, b = self.gates(hidden)
        y, _ = gdn.gated_linear_recurrence(v, a, b, initial_state=pool, output_state=pool, state_indices=rows,
                                           output_final_state=True, cu_seqlens=cu_seqlens)
        return self.out(y.flatten(1))

    def decode(self, hidden, pool, rows):
        v, a, b = self.gates(hidden)
        y, _ = gdn.gated_linear_recurrence_decode(v, a, b, initial_state=pool, state_indices=rows)
        return self.out(y.flatten(1))


def ids(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def train(layer, width, generator):
    """One step: the loss falls."""
    lens = [700, 0, 1, 323]
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    x, target = (torch.randn(sum(lens), width, generator=generator, device="cuda").bfloat16() for _ in range(2))
    losses = []
    for _ in range(2):
        loss = (layer(x, cu).float() - target.float()).square().mean()
        losses.append(float(loss.detach()))
        layer.zero_grad()
        loss.backward()
        with torch.no_grad():
            for p in layer.parameters():
                p -= (0.05 / (1e-12 + p.grad.float().norm())) * p.grad
    return losses


@torch.no_grad()
def serve(layer, width, generator):
    """Returns the answers' outputs, step by step, and the pool's bookkeeping after the last one."""
    pages, seqs = 32, 16
    pool = torch.zeros(pages, layer.heads, layer.dim, device="cuda")
    table, refcounts = torch.full((seqs, 1), -1, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    book = dict(device_status=status)

    rows = gdn.cache_reserve(table, refcounts, ids(0, 1), ids(1, 1), **book).view(-1)
    prompts = torch.randn(300 + 41, width, generator=generator, device="cuda").bfloat16()
    layer.prefill(prompts, ids(0, 300, 341), pool, rows)

    answers = ids(2, 3, 4, 5, 6)  # three to the first prompt, two to the second
    rows = gdn.cache_fork(pool, table, refcounts, ids(0, 0, 0, 1, 1), answers, **book).view(-1)
    gdn.cache_free(table, refcounts, ids(0, 1), **book)
    outputs = []
    for step in range(6):
        if step == 3:  # two answers are done; the others move to the front of the pool
            gdn.cache_free(table, refcounts, ids(2, 5), **book)
            gdn.cache_compact(pool, table, refcounts, **book)
            answers = ids(3, 4, 6)
            rows = table[answers.long()].view(-1)
        token = torch.randn(answers.numel(), width, generator=generator, device="cuda").bfloat16()
        outputs.append(layer.decode(token, pool, rows))
    assert int(status) == 0, int(status)
    return outputs, pool, table, refcounts


def main():
    gdn.build()
    torch.manual_seed(0)
    g = torch.Generator(device="cuda").manual_seed(1)
    layer = Layer(256, 4, 64)
    print("loss before and after a step:", train(layer, 256, g))
    outputs, _, table, refcounts = serve(layer, 256, g)
    print("decoded", sum(o.shape[0] for o in outputs), "tokens; rows in use:", table[table >= 0].tolist(),
          "live pages:", int((refcounts > 0).sum()))


if __name__ == "__main__":
    main()

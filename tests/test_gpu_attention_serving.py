"""Rotary positions, cache writes, attention and the page operators as a program uses them together (examples/attention_serving.py)."""
import importlib.util
import os

import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_serving.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()
    spec = importlib.util.spec_from_file_location("attention_serving", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_answers_of_the_cache_are_those_of_whole_sequences(example, dtype):
    """Each sequence's outputs are those of its prompt and tokens as one sequence.  fp32: products over 128 inputs, 64 channels, at
    most 140 keys and 512 channels, fewer than 900 roundings of 2^-23 of sums whose terms' sizes add up to less than 20 times the
    largest output: 2^-9 of it.  bf16: the attention's result is off by a rounding of its weights (2^-8 of the values' mean size)
    and one or two of its own on either side, 4 * 2^-8 of the largest value; the output's weights carry that on, and it is rounded
    itself on either side."""
    torch.manual_seed(0)
    layer = example.Layer(128, 8, 2, 64, dtype=dtype)
    seen, cache = example.serve(layer, 128, torch.Generator(device="cuda").manual_seed(1))
    parent = {2: 0, 3: 0, 4: 0, 5: 1, 6: 1}
    inputs, outputs = {}, {}
    for seqs, counts, x, y in seen:
        at = 0
        for s, n in zip(seqs, counts):
            inputs.setdefault(s, []).append(x[at: at + n])
            outputs.setdefault(s, []).append(y[at: at + n])
            at += n
    order = sorted(parent)
    whole = [torch.cat(inputs[parent[s]] + inputs[s]) for s in order]
    bounds = torch.tensor([0] + [w.shape[0] for w in whole], device="cuda").cumsum(0)
    with torch.no_grad():
        want = layer(torch.cat(whole), bounds)
        v = layer.qkv(torch.cat(whole))[2]
        if dtype == torch.float32:
            lim = 2.0 ** -9 * want.abs().max()
        else:
            lim = layer.out.weight.float().abs().sum(1) * (4 * 2.0 ** -8 * v.float().abs().max()) + 2 * 2.0 ** -8 * want.float().abs()
    for i, s in enumerate(order):
        got = torch.cat(outputs[parent[s]] + outputs[s]).float()
        part = slice(int(bounds[i]), int(bounds[i + 1]))
        off = (got - want[part].float()).abs()
        assert bool((off <= (lim if dtype == torch.float32 else lim[part])).all()), (s, float(off.max()))
    live = [3, 4, 6]
    assert cache["lengths"].nonzero().view(-1).tolist() == live and cache["lengths"][live].tolist() == [140, 140, 77]


def test_gradients_pass_through(example):
    """The layer's gradients against those of the same layer with the turn in plain torch, in fp32: fewer than 1000 roundings."""
    torch.manual_seed(0)
    layer = example.Layer(64, 4, 2, 32, dtype=torch.float32)
    x = torch.randn(50, 64, device="cuda")
    cu = example.ids(0, 20, 20, 50)
    layer(x, cu).square().sum().backward()
    got = layer.project.weight.grad.clone()
    layer.zero_grad()
    turned = gdn.rotary_embedding

    def plain(q, k, f, cu_seqlens):
        pos = torch.cat([torch.arange(20), torch.arange(30)]).cuda()
        a = pos[:, None].double() * f
        c, s = a.cos().float()[:, None], a.sin().float()[:, None]

        def turn(t):
            n = f.numel()
            return torch.cat([t[..., :n] * c - t[..., n: 2 * n] * s, t[..., n: 2 * n] * c + t[..., :n] * s, t[..., 2 * n:]], -1)

        return turn(q), turn(k)

    gdn.rotary_embedding = plain
    try:
        layer(x, cu).square().sum().backward()
    finally:
        gdn.rotary_embedding = turned
    want = layer.project.weight.grad
    assert float((got - want).abs().max()) <= 1000 * 2.0 ** -23 * float(want.abs().max())

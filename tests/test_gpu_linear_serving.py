"""The recurrence and the page operators as a program uses them together (examples/linear_serving.py)."""
import importlib.util
import os

import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "linear_serving.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()
    spec = importlib.util.spec_from_file_location("linear_serving", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_a_step_of_training_lowers_the_loss(example):
    torch.manual_seed(0)
    g = torch.Generator(device="cuda").manual_seed(1)
    before, after = example.train(example.Layer(256, 4, 64), 256, g)
    assert after < before


def test_answers_of_the_pool_are_those_of_whole_sequences(example):
    """Each answer's state is that of its prompt and tokens as one sequence, from the same values, decays and gates: only the
    recurrence's fp32 rounding differs."""
    torch.manual_seed(0)
    layer = example.Layer(256, 4, 64)
    outputs, pool, table, refs = example.serve(layer, 256, torch.Generator(device="cuda").manual_seed(1))
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = torch.randn(341, 256, generator=g, device="cuda").bfloat16()
    tokens = [torch.randn(5 if s < 3 else 3, 256, generator=g, device="cuda").bfloat16() for s in range(6)]
    assert sorted(table[table >= 0].tolist()) == [0, 1, 2] and refs.tolist() == [1, 1, 1] + [0] * 29
    for answer, (first, second), prompt in ((3, (1, 0), prompts[:300]), (4, (2, 1), prompts[:300]), (6, (4, 2), prompts[300:])):
        with torch.no_grad():
            parts = [layer.gates(prompt)] + [tuple(t[first if s < 3 else second][None] for t in layer.gates(tokens[s]))
                                             for s in range(6)]
            v, a, b = (torch.cat(t) for t in zip(*parts))
            h = torch.zeros(4, 64, dtype=torch.float64, device="cuda")
            for t in range(v.shape[0]):
                h = a[t].double() * h + b[t].double() * v[t].double()
        got = pool[int(table[answer, 0])].double()
        # E_t <= a E_{t-1} + 4 u M_t and 16 u M_t, as in oracle/linear.py, with M the recurrence of absolute values
        with torch.no_grad():
            m = e = torch.zeros_like(h)
            for t in range(v.shape[0]):
                m = a[t].double() * m + (b[t].double() * v[t].double()).abs()
                e = a[t].double() * e + 4 * 2.0 ** -24 * m
        assert ((got - h).abs() <= e + 16 * 2.0 ** -24 * m).all()

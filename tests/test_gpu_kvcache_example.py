"""examples/paged_serving.py: rotary positions, page writes, chunked and
single-token attention and the block copy together."""
import importlib.util
import os

import pytest
import torch

import cache_reference as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("paged_serving", os.path.join(ROOT, "examples", "paged_serving.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
def test_pages_may_move(example, fmt, capsys):
    assert example.main(["--format", fmt, "--prompt", "300", "--chunk", "77", "--new", "3"]) == 0
    assert "the same bits" in capsys.readouterr().out


def test_against_the_definitions(example):
    """The 16-bit layer's outputs against rotary positions and attention of
    the whole sequence in 64 bits.  Queries and keys are rounded once after
    the turn, as the layer's are, so what may differ is the attention's own
    error, and the rounding of a turned value that lies within 2^-21 of a
    border (one in some thousands)."""
    torch.manual_seed(0)
    dev = torch.device("cuda:0")
    layer = example.Layer(12, "bf16", dev)
    n, parts = 70, []
    rows = [torch.randn(n, h, example.DIM).bfloat16() for h in (example.HEADS, example.KV_HEADS, example.KV_HEADS)]
    for a, b in ((0, 33), (33, 69), (69, 70)):
        parts.append(layer.step({5: [x[a:b].to(dev) for x in rows]})[5])
    got = torch.cat(parts).cpu().double()
    pos = torch.arange(n, dtype=torch.int32)
    freqs = layer.freqs.cpu()
    q, k = (R.rope(x, pos, freqs, False, 1.0, False)[0].bfloat16().double() for x in rows[:2])
    pages = [x.permute(1, 0, 2)[None] for x in (k, rows[2].double())]
    want, _, tol, _ = R.attention(q, pages[0], pages[1], torch.zeros(1, 1, dtype=torch.int32), n, [n], [n],
                                  example.HEADS // example.KV_HEADS, 0, example.DIM ** -0.5, torch.bfloat16,
                                  torch.bfloat16)
    # a border changes one of a score's 128 products by a step of at most 2^-7 of it; a score
    # off by d moves the output by at most 2 d of the largest value
    d = 2.0 ** -7 * (q.abs().amax() * k.abs().amax() * example.DIM ** -0.5).item()
    assert ((got - want).abs() <= tol + 2 * d * rows[2].double().abs().amax()).all()

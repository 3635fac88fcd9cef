"""The cache operators on the GPU at the ends of what they accept, against the
definitions in 64 bits (tests/cache_reference.py) or against a call that
differs in nothing that may matter."""
import math

import pytest
import torch

import cache_reference as R
import test_gpu_kvcache as base
from test_gpu_kvcache import C  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP, F8, I8, F32 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.int8, torch.float32


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30])
@pytest.mark.parametrize("q_lens,ctx,heads", [([4, 1], [1, 7], 4), ([50, 20], [30, 2], 2), ([300], [40], 4)])
def test_the_largest_windows_hide_nothing(C, window, q_lens, ctx, heads):
    """A window beyond every context is none, for rows before the first key
    too: the same bits as without."""
    c = base._case(q_lens=q_lens, ctx=ctx, heads=heads, kv=1, dtype=BF, kind=BF)
    a = base._attend(C, torch.Generator().manual_seed(3), **c)
    b = base._attend(C, torch.Generator().manual_seed(3), **dict(c, window=window))
    base._compare(a, **c)
    assert base._eq_bits(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])

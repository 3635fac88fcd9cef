"""How many bits of a softmax weight the second product of attention keeps:
what include/kvcache.h says, weight by weight, against the definitions in 64
bits.  tests/test_gpu_kvcache.py allows 2^-8 of every weight over bfloat16 and
8-bit pages and fp16's smallest step of every weight over float16 ones; here
a weight's own bits are counted, however small it is."""
import math

import pytest
import torch

import cache_reference as R
import test_gpu_kvcache as base
from test_gpu_kvcache import C  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
BF, FP, F8, I8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.int8


def bounds(r, c, unit):
    """(result, allowed error) for weights kept to `unit` of themselves: with
    it the sums' and scores' errors in 32 bits (as cache_reference.attention
    counts them) and the output's own rounding."""
    want, _, tol, _ = R.attention(r["q"], R.held(r["kp"], r["ks"]), R.held(r["vp"], r["vs"]), r["table"], c["page"],
                                  c["q_lens"], c["ctx"], c["heads"] // c["kv"], c["window"], c["dim"] ** -0.5,
                                  torch.float32, torch.float32)
    near, *_ = R.attention(r["q"], R.held(r["kp"], r["ks"]), R.held(r["vp"], r["vs"]).abs(), r["table"], c["page"],
                           c["q_lens"], c["ctx"], c["heads"] // c["kv"], c["window"], c["dim"] ** -0.5,
                           torch.float32, torch.float32)
    rest = tol + unit * near
    return want, rest + R.UNIT[c["dtype"]] * (want.abs() + rest) + R.TINY[c["dtype"]]


HEADS, DIM, PAGE = 4, 64, 16


def crafted(C, q_len, dtype, kind, keys, values, key_scales=None, value_scales=None):
    """Attention of q_len tokens, whose queries are 1 in column 0, over keys
    whose column 0 and values that are the same in every column are given."""
    ctx = len(keys)
    n = -(-ctx // PAGE)
    order = torch.randperm(n, generator=torch.Generator().manual_seed(ctx))

    def paged(x, width, kind):
        rows = torch.zeros(n * PAGE, width, dtype=torch.float64)
        rows[:ctx] = x
        pages = torch.empty(n, 1, PAGE, width, dtype=kind)
        pages[order] = rows.view(n, 1, PAGE, width).to(kind)
        assert torch.equal(pages[order].double().view(-1, width), rows)     # nothing is lost on the way
        return pages.to(base.DEV)

    k = torch.zeros(ctx, DIM, dtype=torch.float64)
    k[:, 0] = keys
    kp, vp = paged(k, DIM, kind), paged(values[:, None].expand(-1, DIM), DIM, kind)
    ks = vs = None
    if kind in (F8, I8):
        ks, vs = (paged(s[:, None], 1, torch.float32)[..., 0].contiguous() for s in (key_scales, value_scales))
    q = torch.zeros(q_len, HEADS, DIM, dtype=dtype)
    q[..., 0] = 1.0
    cache, table = C.PagedCache(kp, vp, ks, vs), order.to(torch.int32)[None]
    plan = C.AttentionPlan(cache, q_heads=HEADS, num_seqs=1, total_q=q_len, max_q_len=q_len, max_context=ctx, dtype=dtype)
    out = plan(q.to(base.DEV), table.to(base.DEV), torch.tensor([0, q_len], dtype=torch.int32, device=base.DEV),
               torch.tensor([ctx], dtype=torch.int32, device=base.DEV))
    case = dict(q_lens=[q_len], ctx=[ctx], heads=HEADS, kv=1, dim=DIM, page=PAGE, window=0, dtype=dtype)
    return dict(q=q, kp=kp, vp=vp, ks=ks, vs=vs, table=table), case, out.cpu().double()


def farthest(held):
    """Of exp(x / 8), x a negative bfloat16 value: the x whose weight lies
    farthest, relative to itself, from `held`'s nearest value, and that value."""
    x = -torch.arange(64, 512, dtype=torch.float64) / 128      # 8 bits at most, scores -0.06 .. -0.5
    x = x[x.to(BF).double() == x]
    w = (x * DIM ** -0.5).exp()
    off = (w.to(held).double() - w).abs() / w
    i = int(off.argmax())
    assert off[i] > 0.4 * R.UNIT[held]
    return x[i].item(), w[i].to(held).item()


@pytest.mark.parametrize("dtype,kind,q_len,unit", [
    (BF, BF, 1, 2.0 ** -16), (BF, F8, 1, 2.0 ** -16), (BF, I8, 4, 2.0 ** -16), (FP, F8, 1, 2.0 ** -16),
    (FP, I8, 1, 2.0 ** -16), (FP, FP, 1, 2.0 ** -22), (FP, FP, 4, 2.0 ** -22),
    (FP, F8, 40, 2.0 ** -16), (FP, I8, 40, 2.0 ** -16)])
def test_weights_in_two_parts(C, dtype, kind, q_len, unit):
    """Half the keys have weight 1 and a value equal to the other keys' weight
    rounded once, those have value -1: weights of one part give a sum of 0 where
    it is their rounding."""
    ctx = 150
    x, near = farthest(FP if kind == FP else BF)
    other = torch.arange(ctx) % 2 == 1
    one = torch.ones(ctx, dtype=torch.float64)
    if kind in (F8, I8):
        r, c, got = crafted(C, q_len, dtype, kind, torch.where(other, -1.0, 0.0).double(), torch.where(other, -one, one),
                            torch.where(other, -x * one, one), torch.where(other, one, near * one))
    else:
        r, c, got = crafted(C, q_len, dtype, kind, torch.where(other, x * one, 0.0 * one),
                            torch.where(other, -one, near * one))
    want, tol = bounds(r, c, unit)
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max()
    # and one part would not do
    rounded = want + (near - math.exp(x * DIM ** -0.5)) * other.sum() / (ctx / 2 * (1 + near)) * -1
    assert ((rounded - want).abs() > 2 * tol)[-1].all()


@pytest.mark.parametrize("q_len", [1, 40])
@pytest.mark.parametrize("ctx", [200, 3000])
def test_small_weights_over_float16_pages(C, q_len, ctx):
    """Keys of weight 1 with value 0, and keys of weights from 2^-19 to 2^-27
    with value 1,000, whose sum is the result: fp16's own smallest step is 2^-24.
    A weight is off by 2^-11 of itself, or by 2^-32 of the largest."""
    t = torch.arange(ctx)
    small = t % 16 != 3
    keys = torch.where(small, -105.0 - (t % 13).double() * 3.75, 0.0)
    r, c, got = crafted(C, q_len, FP, FP, keys.to(FP).double(), torch.where(small, 1000.0, 0.0).double())
    want, tol = bounds(r, c, 2.0 ** -11)
    # the largest weights are at least 1 / 16 of the keys a row sees
    seen = torch.tensor([ctx - q_len + i + 1 for i in range(q_len)], dtype=torch.float64)
    tol = tol + (2.0 ** -32 * 1000 * seen / (seen // 16))[:, None, None]
    assert (tol < want / 8).all() and (want > 1e-4).all()
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max()

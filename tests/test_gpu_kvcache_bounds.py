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


@pytest.mark.parametrize("kind", [BF, FP, F8, I8])
@pytest.mark.parametrize("q_len", [1, 40])
@pytest.mark.parametrize("ctx", [400, 6000])
def test_values_of_no_weight_that_read_as_nan(C, q_len, kind, ctx):
    """A NaN that a row sees reaches it where another key takes all the weight
    too, whichever splits the two lie in: few splits and many."""
    page, group = 16, 4

    def spoil(kp, vp, table, ks, vs):
        a, b = int(table[0][1]), int(table[0][(ctx - q_len) // page - 1])
        if ks is not None:
            ks[b, :, 3] = 1e4
            vs[a, :, 5] = math.nan
        else:
            kp[b, :, 3] *= 1e3
            vp[a, :, 5] = math.nan
    c = base._case(q_lens=[q_len], ctx=[ctx], heads=group, kv=1, dim=64, page=page, dtype=FP if kind == FP else BF,
                   kind=kind)
    r = base._attend(C, torch.Generator().manual_seed(5), edit=spoil, q_scale=20.0, **c)
    assert r["out"].isnan().all()
    splits = r["plan"].args.workspace_bytes // (q_len * group * (64 + 2) * 4)
    assert (splits > 8) == (ctx == 6000)
    # and an infinity does not leave as a number
    if kind in (BF, FP):
        def spoil_more(kp, vp, table, ks, vs):
            spoil(kp, vp, table, ks, vs)
            vp[int(table[0][1]), :, 5] = math.inf
        assert not base._attend(C, torch.Generator().manual_seed(5), edit=spoil_more, q_scale=20.0, **c)["out"].isfinite().any()


@pytest.mark.parametrize("dim", [128, 12])
@pytest.mark.parametrize("kind", [BF, F8, I8])
def test_slots_named_twice_spoil_no_other(C, kind, dim):
    """Padding tokens that share a slot: what the others wrote is as without."""
    g = torch.Generator().manual_seed(3)
    tokens, heads, page = 200, 2, 16
    k, v = (torch.randn(tokens, heads, dim, generator=g).to(BF).to(DEV) for _ in range(2))
    slots = torch.randperm(20 * page, generator=g)[:tokens]
    slots[slots == 0] = 20 * page       # slot 0 is the padding's
    slots[::3] = 0
    alone = torch.where(slots == 0, -1, slots)
    rows = []
    for s in (slots, alone):
        (kp, ks, kraw), (vp, vs, vraw) = (base._blank(21, heads, page, dim, kind, "hnd", 4) for _ in range(2))
        C.write(C.PagedCache(kp, vp, ks, vs), k, v, s.to(DEV))
        rows.append([x.reshape(21, heads, page, -1).transpose(1, 2).flatten(0, 1)[1:]
                     for x in (kraw, vraw, ks, vs) if x is not None])
    assert all(base._eq_bits(a, b) for a, b in zip(*rows))


@pytest.mark.parametrize("dim,rot", [(64, 64), (20, 12)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_float32_turns_keep_their_bits(C, dim, rot, interleaved):
    """Pairs (1, 0) come out as the cosine and the sine, to the last rounding:
    half a step (2^-24), and what an angle loses in 64 bits, of which it takes
    four roundings (the definition's product, the frequency in turns, its
    factor, the product)."""
    tokens = 700
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(-2 ** 20, 2 ** 20, (tokens,), generator=g).to(torch.int32)
    pos[:3] = torch.tensor([0, 1, 2 ** 31 - 1])
    freqs = C.rope_frequencies(rot)
    x = torch.zeros(tokens, 1, dim)
    i0 = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    i1 = i0 + 1 if interleaved else i0 + rot // 2
    x[..., i0] = 1.0
    angle = pos.double()[:, None] * freqs
    for factor in (1.0, 0.5, 1.2079441308975220):
        f = torch.tensor(factor).double()      # as 32 bits hold it
        y, _ = C.rope(pos.to(DEV), freqs.to(DEV), x.to(DEV), interleaved=interleaved, factor=factor)
        y = y[:, 0].cpu().double()
        for got, want in ((y[:, i0], angle.cos() * f), (y[:, i1], angle.sin() * f)):
            tol = want.abs() * 2.0 ** -24 * (1 + 2.0 ** -20) + angle.abs() * 4 * 2.0 ** -53 * f + 2.0 ** -150
            assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max()


@pytest.mark.parametrize("kind", [BF, I8])
def test_strides_of_one_token_head_or_page(C, kind):
    """One token (or head, page, place) of a tensor whose other strides are
    odd: what a slice of a wider buffer looks like."""
    g = torch.Generator().manual_seed(11)

    def odd(x, dim):
        """x with a stride along dim, of extent 1, that is no multiple of 8."""
        st = list(x.stride())
        st[dim] = 12345677
        return x.as_strided(x.shape, st)

    for tokens, heads, kv, page, ctx in ((1, 4, 2, 16, 40), (3, 1, 1, 16, 40), (1, 2, 1, 1, 5), (30, 4, 1, 64, 50)):
        c = base._case(q_lens=[tokens], ctx=[ctx], heads=heads, kv=kv, page=page, dtype=BF, kind=kind)
        r = base._attend(C, g, **c)
        q, *rest = r["args"]
        k, v, ks, vs = r["kp"], r["vp"], r["ks"], r["vs"]
        if kv == 1:
            k, v = odd(k, 1), odd(v, 1)
            if ks is not None:
                ks, vs = odd(ks, 1), odd(vs, 1)
        if page == 1:
            k, v = odd(k, 2), odd(v, 2)
        if heads == 1:
            q = odd(q, 1)
        out = torch.zeros_like(r["out"])
        if tokens == 1:
            q, out = odd(q, 0), odd(out, 0)
        cache = C.PagedCache(k, v, ks, vs)
        plan = C.AttentionPlan(cache, q_heads=heads, num_seqs=1, total_q=tokens, max_q_len=tokens, max_context=ctx)
        plan(q, *rest, out=out)
        assert base._eq_bits(out, r["out"])
        # the same rows through writes, reads and turns
        x = torch.randn(tokens, kv, 64, generator=g).to(BF).to(DEV)
        y = odd(x, 0) if tokens == 1 else odd(x, 1) if kv == 1 else x
        slots = torch.randperm(k.shape[0] * page, generator=g)[:tokens].to(DEV)
        C.write(cache, y, y, slots)
        got = [t.clone() for t in C.read(cache, slots)]
        plain = C.PagedCache(r["kp"], r["vp"], r["ks"], r["vs"])
        C.write(plain, x, x, slots)
        assert all(torch.equal(a, b) for a, b in zip(got, C.read(plain, slots)))
        pos, freqs = torch.arange(tokens, dtype=torch.int32, device=DEV), C.rope_frequencies(64, device=DEV)
        assert torch.equal(C.rope(pos, freqs, y)[0], C.rope(pos, freqs, x)[0])


def test_gradients_are_not_lost_silently(C):
    """What would need one is refused while gradients are on."""
    x = torch.ones(2, 4, 64, dtype=BF, device=DEV)
    y = x.clone().requires_grad_()
    pos, freqs = torch.arange(2, dtype=torch.int32, device=DEV), C.rope_frequencies(64, device=DEV)
    p, s = torch.zeros(3, 4, 16, 64, device=DEV), torch.zeros(3, 4, 16, device=DEV)
    for ask in (lambda: C.rope(pos, freqs, y), lambda: C.rope(pos, freqs, x, y), lambda: C.rope(pos, freqs, x, q_out=y),
                lambda: C.rope(pos, freqs, x, x, k_out=y),
                lambda: C.PagedCache(p.to(BF).requires_grad_(), p.to(BF)), lambda: C.PagedCache(p.to(BF), p.to(BF).requires_grad_()),
                lambda: C.PagedCache(p.to(I8), p.to(I8), s, s.clone().requires_grad_())):
        with pytest.raises(ValueError, match="gradient"):
            ask()
    with torch.no_grad():
        a, _ = C.rope(pos, freqs, y)
    assert torch.equal(a, C.rope(pos, freqs, x)[0]) and not a.requires_grad


@pytest.mark.parametrize("kind", [BF, F8])
@pytest.mark.parametrize("q_lens,ctx", [([1, 1, 1], [500, 333, 96]), ([40, 7, 20], [500, 333, 96])])
def test_sequences_that_share_pages(C, kind, q_lens, ctx):
    """A common prefix, held once."""
    def share(kp, vp, table, ks, vs):
        table[1, :5], table[2, :6] = table[0, :5], table[0, :6]
    c = base._case(q_lens=q_lens, ctx=ctx, heads=4, kv=2, dim=128, dtype=BF, kind=kind)
    r = base._attend(C, torch.Generator().manual_seed(2), edit=share, **c)
    assert len(set(r["table"][:, 0].tolist())) == 1
    base._compare(r, **c)


@pytest.mark.parametrize("dtype,kind", [(BF, BF), (FP, I8)])
@pytest.mark.parametrize("q_lens,bound", [([1, 1], 1), ([1, 1], 3), ([1, 1], 300), ([3, 2], 16), ([40, 23], 700)])
@pytest.mark.parametrize("window", [0, 50])
def test_bounds_beyond_the_lengths(C, dtype, kind, q_lens, bound, window):
    """max_q_len, max_context and a table for more than there is."""
    c = base._case(q_lens=q_lens, ctx=[333, 70], heads=4, kv=2, dtype=dtype, kind=kind, window=window)
    r = base._attend(C, torch.Generator().manual_seed(2), **c)
    q, table, starts, lens = r["args"]
    wide = torch.full((2, 400), -3, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    for most in (333, 334, 6400):
        plan = C.AttentionPlan(r["cache"], q_heads=4, num_seqs=2, total_q=sum(q_lens), max_q_len=bound, max_context=most,
                               window=window)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        lse = torch.empty(sum(q_lens), 4, device=DEV)
        out = plan(q, wide, starts, lens, lse=lse, status=status)
        assert status.item() == 0
        base._compare(dict(r, out=out, lse=lse), **c)

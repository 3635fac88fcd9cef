"""The cache operators on the GPU against plain definitions in 64 bits
(tests/cache_reference.py), at the sizes, layouts and values where they can go
wrong."""
import math
import random

import numpy as np
import pytest
import torch

import cache_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP, F8, I8, F32 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.int8, torch.float32


@pytest.fixture(scope="module")
def C():
    from block_copy_amd import kvcache
    return kvcache


def _pages(g, n, heads, page, dim, kind, order="hnd", pad=0):
    """A filled cache (pages, scales) with `pad` unused values behind each row."""
    shape = (n, heads, page, dim + pad) if order == "hnd" else (n, page, heads, dim + pad)
    x = torch.randn(shape, generator=g)
    if kind == I8:
        x = (x * 45).clamp(-127, 127).round().to(I8)
    elif kind == F8:
        x = (x * 150).clamp(-448, 448).to(F8)
    else:
        x = x.to(kind)
    x = x.to(DEV)
    if order == "nhd":
        x = x.transpose(1, 2)
    x = x[..., :dim]
    s = None
    if kind in (I8, F8):
        s = ((1 + torch.rand(n, heads, page, generator=g)) * 3 / R.Q[kind]).to(DEV)
    return x, s


def _eq_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,kv,dim,rot,factor", [
    (1, 32, 8, 128, 128, 1.0), (5, 3, 1, 64, 64, 1.25), (37, 7, 2, 80, 32, 1.0),
    (2, 1, 0, 20, 6, 1.0), (600, 4, 4, 96, 48, 0.75), (3, 2, 1, 256, 256, 1.0), (4, 1, 1, 512, 512, 1.0),
    (3, 2, 2, 64, 0, 1.0)])
def test_rope(C, dtype, interleaved, tokens, heads, kv, dim, rot, factor):
    g = torch.Generator().manual_seed(tokens * 7 + dim)
    base = torch.randn(tokens, heads + kv, dim, generator=g).to(dtype)
    pos = torch.randint(-5, 1 << 21, (tokens,), generator=g).to(torch.int32)
    freqs = C.rope_frequencies(rot) if rot else torch.zeros(0, dtype=torch.float64)
    d = base.to(DEV)
    q, k = d[:, :heads], d[:, heads:] if kv else None
    for inverse in (False, True):
        qo, ko = C.rope(pos.to(DEV), freqs.to(DEV), q, k, interleaved=interleaved, factor=factor, inverse=inverse)
        for got, x in ((qo, base[:, :heads]), (ko, base[:, heads:])):
            if got is None:
                continue
            want, tol = R.rope(x, pos, freqs, interleaved, factor, inverse)
            assert ((got.cpu().double() - want).abs() <= tol).all()
    # in place, and any alignment: a view that starts at an odd element
    q2, _ = C.rope(pos.to(DEV), freqs.to(DEV), d[:, :heads].clone(), interleaved=interleaved, factor=factor)
    w = d[:, :heads].clone()
    C.rope(pos.to(DEV), freqs.to(DEV), w, q_out=w, interleaved=interleaved, factor=factor)
    assert _eq_bits(w, q2)
    flat = torch.zeros(tokens * heads * dim + 1, dtype=dtype, device=DEV)
    odd = flat[1:].view(tokens, heads, dim)
    odd.copy_(d[:, :heads])
    q3, _ = C.rope(pos.to(DEV), freqs.to(DEV), odd, interleaved=interleaved, factor=factor)
    assert _eq_bits(q3, q2)


def test_rope_inverse_is_the_gradient(C):
    """Against central differences of the forward form (linear: exact but for
    rounding), and as the way back."""
    g = torch.Generator().manual_seed(3)
    t, h, d, rot, factor = 3, 2, 16, 12, 1.5
    x, up = torch.randn(t, h, d, generator=g), torch.randn(t, h, d, generator=g)
    pos = torch.tensor([0, 9, 70001], dtype=torch.int32).to(DEV)
    f = C.rope_frequencies(rot, device=DEV)
    for inter in (False, True):
        grad, _ = C.rope(pos, f, up.to(DEV), interleaved=inter, factor=factor, inverse=True)
        grad = grad.cpu().double()
        for i, j, e in ((0, 0, 3), (1, 1, 0), (2, 0, 7), (2, 1, 11), (1, 0, 15)):
            ys = []
            for step in (1.0, -1.0):
                y = x.clone()
                y[i, j, e] += step
                o, _ = C.rope(pos, f, y.to(DEV), interleaved=inter, factor=factor)
                ys.append((o.cpu().double() * up.double()).sum().item())
            # eight values of size below 2^3 change, each off by 2^-21 of that, twice
            assert abs((ys[0] - ys[1]) / 2 - grad[i, j, e].item()) <= 2.0 ** -13
        y, _ = C.rope(pos, f, x.to(DEV), interleaved=inter, factor=factor)
        z, _ = C.rope(pos, f, y, interleaved=inter, factor=1 / factor, inverse=True)
        # the turn and its reverse: each pair's size, off by 2^-21 twice, factors by 2^-23
        assert ((z[..., :rot].cpu() - x[..., :rot]).abs() <= 2.0 ** -18 * x.abs().max()).all()


# ---------------------------------------------------------------------------
# writing and reading
# ---------------------------------------------------------------------------

ROWS = [  # tokens, heads, page, dim, order, pad
    (1, 1, 16, 128, "hnd", 0), (19, 8, 16, 128, "hnd", 0), (33, 3, 7, 64, "nhd", 0), (21, 2, 1, 80, "hnd", 0),
    (5, 2, 100, 256, "nhd", 8), (9, 2, 24, 36, "hnd", 0), (11, 1, 16, 5, "nhd", 3), (4, 3, 16, 512, "hnd", 0),
    (300, 8, 16, 96, "nhd", 0)]


def _blank(n, heads, page, dim, kind, order, pad):
    shape = (n, heads, page, dim + pad) if order == "hnd" else (n, page, heads, dim + pad)
    raw = torch.full(shape, 0x35, dtype=torch.uint8, device=DEV) if kind in (F8, I8) else \
        torch.full(shape, 0.625, dtype=kind, device=DEV)
    x = raw.view(kind) if kind in (F8, I8) else raw
    x = x.transpose(1, 2) if order == "nhd" else x
    s = torch.full((n, heads, page), -7.0, device=DEV) if kind in (F8, I8) else None
    return x[..., :dim], s, raw


@pytest.mark.parametrize("tokens,heads,page,dim,order,pad", ROWS)
@pytest.mark.parametrize("dtype,kind", [(BF, F8), (FP, F8), (BF, I8), (FP, I8), (BF, BF), (FP, FP)])
def test_write_then_read(C, tokens, heads, page, dim, order, pad, dtype, kind):
    g = torch.Generator().manual_seed(tokens + dim)
    n = -(-tokens // page) + 2
    slots = torch.randperm(n * page, generator=g)[:tokens]
    if tokens > 4:
        slots[2] = -1
    k, v = (torch.randn(tokens, heads, dim, generator=g).to(dtype) for _ in range(2))
    k[0] = 0.0                                  # a row of zeros
    if tokens > 4:
        k[1] = (torch.randint(-8, 9, (heads, dim), generator=g).float() / 8).to(dtype)  # many borders
        v[3] *= 1e-7 if dtype == FP else 1e-38  # near the smallest values
        v[4, :, 0] = 65504.0 if dtype == FP else 3e38
    kp, ks, kraw = _blank(n, heads, page, dim, kind, order, pad)
    vp, vs, vraw = _blank(n, heads, page, dim, kind, order, pad)
    before = kraw.clone()
    cache = C.PagedCache(kp, vp, ks, vs)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    C.write(cache, k.to(DEV), v.to(DEV), slots.to(DEV), status=status)
    assert status.item() == 0
    untouched = torch.ones(n, page, dtype=torch.bool)
    for t in range(tokens):
        if slots[t] >= 0:
            untouched[slots[t] // page, slots[t] % page] = False
    for x, p, s in ((k, kp, ks), (v, vp, vs)):
        at, place = slots.clamp(min=0) // page, slots.clamp(min=0) % page
        live = slots >= 0
        got = p.cpu().float()[at, :, place][live]
        if kind in (F8, I8):
            want, scale = R.quantise(x, kind)
            assert np.array_equal(got.double().numpy(), want[live.numpy()])
            assert np.array_equal(s.cpu()[at, :, place][live].numpy(), scale[live.numpy()])
            assert (s.cpu().transpose(1, 2)[untouched] == -7.0).all()
        else:
            assert torch.equal(got, x.float()[live])
    # nothing else changed: other slots, padding
    raw = kraw.transpose(1, 2) if order == "hnd" else kraw
    old = before.transpose(1, 2) if order == "hnd" else before
    assert torch.equal(raw.cpu()[untouched], old.cpu()[untouched])
    assert torch.equal(raw[..., dim:], old[..., dim:])
    # and back, in each output type
    for out in (BF, FP, F32):
        ko, vo = C.read(cache, slots.to(DEV), dtype=out)
        for got, p, s in ((ko, kp, ks), (vo, vp, vs)):
            val = p.cpu().float()
            if s is not None:
                val = val * s.cpu()[..., None]
            val = val[slots.clamp(min=0) // page, :, slots.clamp(min=0) % page]
            val[slots < 0] = 0.0
            assert torch.equal(got.cpu(), val.to(out))


@pytest.mark.parametrize("dim", [64, 12])
@pytest.mark.parametrize("kind", [F8, I8])
def test_write_of_infinities_and_nan(C, kind, dim):
    x = torch.ones(4, 2, dim, dtype=BF)
    x[0, 0, 3], x[1, 1, 5], x[2, 0, 0] = math.inf, math.nan, -math.inf
    kp, ks, _ = _blank(1, 2, 4, dim, kind, "hnd", 0)
    vp, vs, _ = _blank(1, 2, 4, dim, kind, "hnd", 0)
    cache = C.PagedCache(kp, vp, ks, vs)
    slots = torch.arange(4, device=DEV)
    C.write(cache, x.to(DEV), x.to(DEV), slots)
    ko, vo = C.read(cache, slots, dtype=F32)
    bad = torch.zeros(4, 2, dtype=torch.bool)
    bad[0, 0] = bad[1, 1] = bad[2, 0] = True
    for o in (ko, vo):
        assert o.cpu()[bad].isnan().all() and torch.equal(o.cpu()[~bad], torch.ones(5, dim))
    assert (kp.cpu().float()[0].transpose(0, 1)[bad] == 0).all()


@pytest.mark.parametrize("dim", [64, 12])
def test_slots_beyond_the_pages(C, dim):
    kp, _, kraw = _blank(2, 1, 4, dim, BF, "hnd", 0)
    vp, _, _ = _blank(2, 1, 4, dim, BF, "hnd", 0)
    cache = C.PagedCache(kp, vp)
    x = torch.ones(4, 1, dim, dtype=BF, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    slots = torch.tensor([8, 1 << 40, -(1 << 40), 7], device=DEV)
    C.write(cache, x, x, slots, status=status)
    assert status.item() == C.BAD_SLOT
    assert (kraw[1, 0, 3] == 1).all() and (kraw.sum(-1) == 0.625 * dim).sum() == 7
    status.zero_()
    ko, vo = C.read(cache, slots, status=status)
    assert status.item() == C.BAD_SLOT
    assert (ko[:3] == 0).all() and (ko[3] == 1).all() and (vo[:3] == 0).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _attend(C, g, *, q_lens, ctx, heads, kv, dim, page, dtype, kind, window=0, order="hnd", pad=0, scale=None,
            edit=None, q_scale=1.5):
    """Runs a case and compares it; returns what a test looks at further."""
    n_seq, total = len(q_lens), sum(q_lens)
    per = [-(-c // page) for c in ctx]
    pool = sum(per) + 2
    kp, ks = _pages(g, pool, kv, page, dim, kind, order, pad)
    vp, vs = _pages(g, pool, kv, page, dim, kind, order, pad)
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    cols = max(per + [1])
    table = torch.full((n_seq, cols), -9, dtype=torch.int32)     # unused entries are not page numbers
    at = 0
    for s, p in enumerate(per):
        table[s, :p] = perm[at:at + p]
        at += p
    q = (torch.randn(total, heads, dim, generator=g) * q_scale).to(dtype)
    if edit:
        edit(kp, vp, table, ks, vs)
    cache = C.PagedCache(kp, vp, ks, vs)
    plan = C.AttentionPlan(cache, q_heads=heads, num_seqs=n_seq, total_q=total, max_q_len=max(q_lens + [1]),
                           max_context=max(ctx), window=window, dtype=dtype, scale=scale)
    starts = torch.tensor(np.cumsum([0] + list(q_lens)), dtype=torch.int32)
    out = torch.full((total, heads, dim + 8), 77.0, dtype=dtype, device=DEV)[..., :dim]
    lse = torch.full((total, 2 * heads), 77.0, device=DEV)[:, ::2]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    if plan.workspace is not None:
        plan.workspace.fill_(0xff)                                # NaN, if read before it is written
    args = (q.to(DEV), table.to(DEV), starts.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV))
    plan(*args, out=out, lse=lse, status=status)
    assert status.item() == 0
    return dict(cache=cache, plan=plan, args=args, out=out, lse=lse, q=q, table=table, ks=ks, vs=vs, kp=kp, vp=vp)


def _compare(r, *, q_lens, ctx, heads, kv, page, window, dtype, kind, scale=None, **_):
    dim = r["q"].shape[2]
    held = BF if kind in (F8, I8) else dtype
    want, lse, tol, ltol = R.attention(r["q"], R.held(r["kp"], r["ks"]), R.held(r["vp"], r["vs"]), r["table"], page,
                                       q_lens, ctx, heads // kv, window, dim ** -0.5 if scale is None else scale,
                                       held, dtype)
    got, glse = r["out"].cpu().double(), r["lse"].cpu().double()
    empty = torch.isinf(lse)
    assert torch.equal(torch.isinf(glse), empty) and (glse[empty] < 0).all()
    assert (got[empty] == 0).all()
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol.clamp(min=1e-30)).max()
    assert ((glse - lse).abs()[~empty] <= ltol[~empty]).all()


def _case(**kw):
    return dict(dict(heads=4, kv=2, dim=64, page=16, window=0, order="hnd", pad=0), **kw)


CASES = [
    _case(q_lens=[1], ctx=[1]),
    _case(q_lens=[1], ctx=[2], dim=128, page=1),
    _case(q_lens=[1, 1, 1, 1], ctx=[31, 32, 33, 129], heads=8, kv=1, dim=128),
    _case(q_lens=[1, 1, 0, 1], ctx=[0, 5, 7, 300], heads=7, kv=1, dim=96, page=7, order="nhd"),
    _case(q_lens=[1, 1], ctx=[2000, 900], heads=2, kv=2, dim=256, page=24),
    _case(q_lens=[1, 1], ctx=[1500, 3], heads=16, kv=1, dim=80, page=100, pad=8),
    _case(q_lens=[3, 5, 2], ctx=[40, 5, 700], heads=3, kv=1, dim=64, window=9),
    _case(q_lens=[4], ctx=[2], heads=4, kv=1),                      # rows before the first key
    _case(q_lens=[1, 1], ctx=[513, 1100], window=1, dim=24, page=8),
    _case(q_lens=[1], ctx=[1301], window=400, dim=8, heads=1, kv=1),
    _case(q_lens=[33], ctx=[33], heads=1, kv=1),
    _case(q_lens=[17, 0, 40], ctx=[17, 9, 111], heads=6, kv=2, dim=128, page=5),
    _case(q_lens=[65], ctx=[1400], heads=4, kv=1, dim=128, order="nhd"),   # split keys
    _case(q_lens=[40, 23], ctx=[600, 1203], heads=2, kv=2, dim=256, page=24, window=100),
    _case(q_lens=[130, 7], ctx=[130, 650], heads=4, kv=4, dim=96, page=100, window=64),
    _case(q_lens=[50, 20], ctx=[30, 20], heads=2, kv=1, dim=40, page=16),  # rows before the first key
    _case(q_lens=[20], ctx=[555], heads=32, kv=1, dim=64, page=64, window=1),
    _case(q_lens=[1], ctx=[700], heads=32, kv=1, dim=192, page=16),        # one token, many heads
    _case(q_lens=[1, 2], ctx=[333, 70], heads=4, kv=2, dim=128, pad=8),    # 8-bit rows 8 bytes apart from 16
    _case(q_lens=[40], ctx=[140], heads=4, kv=2, dim=64, pad=8),
]


@pytest.mark.parametrize("dtype,kind", [(BF, BF), (FP, FP), (BF, F8), (FP, F8), (BF, I8), (FP, I8)])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_attention(C, i, dtype, kind):
    c = dict(CASES[i], dtype=dtype, kind=kind)
    g = torch.Generator().manual_seed(100 + i)
    r = _attend(C, g, **c)
    _compare(r, **c)
    # the same call twice gives the same bits
    again = torch.empty_like(r["out"])
    r["plan"](*r["args"], out=again)
    assert _eq_bits(r["out"], again)


@pytest.mark.parametrize("kind", [BF, FP, F8, I8])
@pytest.mark.parametrize("q_lens,ctx,heads", [([1, 1], [70, 40], 4), ([3, 2], [70, 40], 4), ([40, 9], [90, 30], 4)])
def test_unseen_values_never_matter(C, kind, q_lens, ctx, heads):
    """Infinities and NaN in what no row sees, and in tokens that only some
    rows of a chunk see, reach just the rows that see them."""
    page, dtype, window = 16, FP if kind == FP else BF, 20
    c = _case(q_lens=q_lens, ctx=ctx, heads=heads, kv=1, dim=64, page=page, window=window, dtype=dtype, kind=kind)

    def spoil(kp, vp, table, ks, vs):
        for s, (n, m) in enumerate(zip(q_lens, ctx)):
            spots = [t for t in range(m, len(table[s][table[s] >= 0]) * page)]      # behind the context
            spots += [t for t in range(0, max(0, m - n - window + 1))]              # left of every window
            for t in spots:
                at, place = int(table[s][t // page]), t % page
                for x, sc in ((kp, ks), (vp, vs)):
                    if sc is not None:
                        sc[at, :, place] = math.nan if t % 2 else math.inf
                    else:
                        x[at, :, place] = math.nan if t % 3 == 0 else (-1) ** t * math.inf

    a = _attend(C, torch.Generator().manual_seed(5), **c)
    b = _attend(C, torch.Generator().manual_seed(5), edit=spoil, **c)
    assert _eq_bits(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    if max(q_lens) == 1:
        return

    # the last token of each sequence, which only its last row sees
    def last(kp, vp, table, ks, vs):
        for s, m in enumerate(ctx):
            at, place = int(table[s][(m - 1) // page]), (m - 1) % page
            if vs is not None:
                vs[at, :, place] = math.nan
            else:
                vp[at, :, place, :32] = math.nan
                vp[at, :, place, 32] = math.inf
                vp[at, :, place, 33] = -math.inf
    d = _attend(C, torch.Generator().manual_seed(5), edit=last, **c)
    ends = np.cumsum(q_lens) - 1
    others = torch.tensor([r for r in range(sum(q_lens)) if r not in set(ends)])
    assert _eq_bits(a["out"][others], d["out"][others])
    assert torch.equal(a["lse"], d["lse"])
    got = d["out"].cpu()[torch.tensor(ends)].float()
    if kind in (F8, I8):
        assert got.isnan().all()
    else:
        assert got[..., :32].isnan().all() and (got[..., 32] == math.inf).all() and (got[..., 33] == -math.inf).all()
        assert got[..., 34:].isfinite().all()


@pytest.mark.parametrize("kind", [BF, FP])
@pytest.mark.parametrize("q_len", [1, 40])
def test_seen_infinities(C, q_len, kind):
    """Infinities and NaN among values that every row sees, far from any edge."""
    def spoil(kp, vp, table, ks, vs):
        at = int(table[0][1])
        vp[at, :, 3, 5], vp[at, :, 4, 6], vp[at, :, 5, 7] = math.inf, -math.inf, math.nan
        vp[at, :, 6, 8], vp[at, :, 7, 8] = math.inf, -math.inf
    c = _case(q_lens=[q_len], ctx=[400], heads=4, kv=1, dim=64, page=16, dtype=kind, kind=kind)
    a = _attend(C, torch.Generator().manual_seed(5), **c)
    b = _attend(C, torch.Generator().manual_seed(5), edit=spoil, **c)
    keep = torch.ones(64, dtype=torch.bool)
    keep[5:9] = False
    assert _eq_bits(a["out"][..., keep], b["out"][..., keep])
    o = b["out"].float()
    assert (o[..., 5] == math.inf).all() and (o[..., 6] == -math.inf).all() and o[..., 7:9].isnan().all()


@pytest.mark.parametrize("kind", [F8, I8])
@pytest.mark.parametrize("q_len", [1, 40])
def test_seen_scales_of_nan(C, q_len, kind):
    """A value that reads as NaN reaches every row that sees it, however small
    its weight: here each row's weight for it is 0 or 1."""
    def spoil(kp, vp, table, ks, vs):
        at = int(table[0][1])
        ks[at, :, 3], vs[at, :, 3] = 1e4, math.nan
    c = _case(q_lens=[q_len], ctx=[400], heads=4, kv=1, dim=64, page=16, dtype=BF, kind=kind)
    assert _attend(C, torch.Generator().manual_seed(5), edit=spoil, **c)["out"].isnan().all()


@pytest.mark.parametrize("q_len", [1, 40])
def test_extreme_scores(C, q_len):
    """Large scores of both signs: the running maximum grows and shrinks."""
    c = _case(q_lens=[q_len], ctx=[900], heads=4, kv=1, dim=128, page=16, dtype=BF, kind=BF, scale=3.0)
    r = _attend(C, torch.Generator().manual_seed(8), q_scale=1.0, **c)
    _compare(r, **c)
    c["scale"] = 0.0
    _compare(_attend(C, torch.Generator().manual_seed(8), **c), **c)
    c["scale"] = -0.5
    _compare(_attend(C, torch.Generator().manual_seed(9), **c), **c)


@pytest.mark.parametrize("q_len", [1, 40])
@pytest.mark.parametrize("kind", [BF, I8])
def test_bad_pages_read_as_zeros(C, q_len, kind):
    page, ctx = 16, 90
    c = _case(q_lens=[q_len], ctx=[ctx], heads=4, kv=1, dim=64, page=page, dtype=BF, kind=kind)
    r = _attend(C, torch.Generator().manual_seed(4), **c)
    zero = _attend(C, torch.Generator().manual_seed(4), **c,
                   edit=lambda kp, vp, t, ks, vs: [x.view(torch.uint8)[int(t[0][j])].zero_() for x in (kp, vp) for j in (1, 3)]
                   + [x[int(t[0][j])].zero_() for x in (ks, vs) if x is not None for j in (1, 3)])
    q, table, starts, lens = r["args"]
    table = table.clone()
    table[0, 1], table[0, 3] = -1, r["cache"].num_pages
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = r["plan"](q, table, starts, lens, status=status)
    assert status.item() == C.BAD_PAGE
    assert _eq_bits(out, zero["out"])


def test_lengths_beyond_the_bounds_are_flagged(C):
    c = _case(q_lens=[3], ctx=[50], heads=2, kv=1, dtype=BF, kind=BF)
    r = _attend(C, torch.Generator().manual_seed(4), **c)
    q, table, starts, lens = r["args"]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for st, ln in (([0, 3], [51]), ([0, 4], [50]), ([-1, 3], [50]), ([2, 1], [50]), ([0, 3], [-4]),
                   ([0, 3], [2 ** 31 - 1])):
        status.zero_()
        r["plan"](q, table, torch.tensor(st, dtype=torch.int32, device=DEV),
                  torch.tensor(ln, dtype=torch.int32, device=DEV), status=status)
        assert status.item() & C.BAD_LENGTH, (st, ln)


# ---------------------------------------------------------------------------
# streams, graphs, far offsets, the operators together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("q_len", [1, 30])
def test_graph_replays(C, q_len):
    """Write and attention captured together, replayed with new contents and
    eager work between."""
    g = torch.Generator().manual_seed(1)
    heads, kv, dim, page, cap = 4, 2, 64, 16, 1200
    pool = cap // page + 1
    blank = [_blank(pool, kv, page, dim, I8, "hnd", 0) for _ in range(2)]
    cache = C.PagedCache(blank[0][0], blank[1][0], blank[0][1], blank[1][1])
    cache.k.zero_(), cache.v.zero_(), cache.k_scales.zero_(), cache.v_scales.zero_()
    plan = C.AttentionPlan(cache, q_heads=heads, num_seqs=1, total_q=q_len, max_q_len=q_len, max_context=cap)
    assert plan.workspace is not None
    table = torch.randperm(pool, generator=g).to(torch.int32)[None].to(DEV)
    starts = torch.tensor([0, q_len], dtype=torch.int32, device=DEV)
    q, k, v = (torch.zeros(q_len, h, dim, dtype=BF, device=DEV) for h in (heads, kv, kv))
    slots = torch.zeros(q_len, dtype=torch.int64, device=DEV)
    lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.zeros_like(q)

    def step():
        C.write(cache, k, v, slots)
        plan(q, table, starts, lens, out=out)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    at = 0
    for _ in range(5):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g).to(BF))
        t = torch.arange(at, at + q_len)
        slots.copy_(table[0].cpu().long()[t // page] * page + t % page)
        at += q_len
        lens.fill_(at)
        graph.replay()
        torch.cuda.synchronize()
        replayed = out.clone()
        out.zero_()
        step()
        torch.cuda.synchronize()
        assert _eq_bits(out, replayed) and (replayed != 0).any()


def test_side_streams(C):
    """Two plans on two streams at once give what they give alone."""
    c = _case(q_lens=[1] * 8, ctx=[3000] * 8, heads=8, kv=2, dim=128, dtype=BF, kind=F8)
    a = _attend(C, torch.Generator().manual_seed(1), **c)
    b = _attend(C, torch.Generator().manual_seed(2), **c)
    torch.cuda.synchronize()
    outs = []
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(6):
        r = (a, b)[i % 2]
        o = torch.zeros_like(r["out"])
        torch.cuda.synchronize()
        outs.append(o)
        if i < 2:
            r["plan"](*r["args"], out=o, stream=s[i % 2])
        else:
            with torch.cuda.stream(s[i % 2]):
                r["plan"](*r["args"], out=o)
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert _eq_bits(o, (a, b)[i % 2]["out"])


@pytest.mark.parametrize("kind", [BF, I8])
def test_offsets_beyond_32_bits(C, kind):
    """Pages that lie more than 2^32 bytes and elements apart."""
    page, heads, dim, far = 16, 1, 64, (1 << 32) + 4096
    row = heads * page * dim
    raw = [torch.zeros(far + row, dtype=torch.uint8 if kind == I8 else kind, device=DEV) for _ in range(2)]
    pages = [torch.as_strided(x, (2, heads, page, dim), (far, page * dim, dim, 1)).view(kind) for x in raw]
    scales = [torch.zeros(2, heads, page, device=DEV) for _ in range(2)] if kind == I8 else [None, None]
    cache = C.PagedCache(*pages, *scales)
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(20, heads, dim, generator=g).to(BF) for _ in range(2))
    table = torch.tensor([[1, 0]], dtype=torch.int32)
    t = torch.arange(20)
    slots = table[0].long()[t // page] * page + t % page
    C.write(cache, k.to(DEV), v.to(DEV), slots.to(DEV))
    ko, vo = C.read(cache, slots.to(DEV), dtype=F32)
    if kind == BF:
        assert torch.equal(ko.cpu(), k.float()) and torch.equal(vo.cpu(), v.float())
    for n in (1, 18):
        q = torch.randn(n, 2, dim, generator=g).to(BF)
        plan = C.AttentionPlan(cache, q_heads=2, num_seqs=1, total_q=n, max_q_len=n, max_context=20)
        lse = torch.zeros(n, 2, device=DEV)
        out = plan(q.to(DEV), table.to(DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV),
                   torch.tensor([20], dtype=torch.int32, device=DEV), lse=lse)
        r = dict(q=q, kp=ko[:16].cpu().transpose(0, 1)[None], out=out, lse=lse, ks=None, vs=None)
        both = lambda x: torch.cat([x, torch.zeros(12, heads, dim, device=DEV)]).view(2, page, heads, dim).transpose(1, 2)  # noqa: E731
        r["kp"], r["vp"], r["table"] = both(ko), both(vo), torch.tensor([[0, 1]])
        _compare(r, q_lens=[n], ctx=[20], heads=2, kv=1, page=page, window=0, dtype=BF, kind=kind)

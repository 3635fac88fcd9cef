"""Measured cases of the paged key/value cache operators: rotary positions,
writing new tokens into cache pages (as they are or in 8 bits), reading them
back, and attention of new tokens over the paged cache.

`run` computes an operator from elementary torch operations in 32 bits, or,
with `own` set, through block_copy_amd.kvcache.  `exact` computes the same
from the definitions in 64 bits.

Definitions shared by both:

  * Pages are indexed [page, head, place, dim].  Token t of a sequence lives
    in page table[t // page_size], place t % page_size; a slot is
    page * page_size + place, and a negative slot is a token to leave out.
  * An 8-bit row (one token, one head) holds codes and one float scale:
    scale = amax / Q and code = round_to_nearest_even(x * Q / amax), with
    Q = 448 for e4m3 and 127 for int8, amax the row's largest magnitude; a row
    of zeros has scale 0 and codes 0.  The value is code * scale.
  * Rotary positions turn pair i of the first rot values of a head by the
    angle position * freq[i] and multiply it by a constant; pair i is
    (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved.
  * Query r of a sequence with q new tokens and c tokens in the cache (the
    new ones among them) stands at position c - q + r and sees the keys at
    positions p with p <= position and, with a window w, p > position - w.
    Rows that see no key give 0, and -inf as their log-sum.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "fp8": torch.float8_e4m3fn, "int8": torch.int8}
QMAX = {"fp8": 448.0, "int8": 127.0}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one new token of one sequence: queries and keys of a layer turned before its attention
        dict(name="rope one token", op="rope", tokens=1, heads=32, kv_heads=8, dim=128, rot=128,
             dtype="bf16", interleaved=False, scaling="none", far=40000),
        # a long prompt's queries and keys at far positions, frequencies scaled for a long context
        dict(name="rope 16384 tokens", op="rope", tokens=16384, heads=32, kv_heads=8, dim=128,
             rot=128, dtype="bf16", interleaved=False, scaling="parts", far=1000000),
        # a decode step's new tokens into e4m3 pages
        dict(name="write 33 tokens fp8", op="write", tokens=33, kv_heads=8, dim=128, page=16,
             order="hnd", dtype="bf16", format="fp8", back=False),
        # a prompt's keys and values into e4m3 pages of 4 KiB blocks
        dict(name="write 32768 tokens fp8", op="write", tokens=32768, kv_heads=8, dim=128,
             page=32, order="hnd", dtype="bf16", format="fp8", back=False),
        # a chunk quantised to int8 as it is written, and read back by a connector
        dict(name="write, read 8191 int8", op="write", tokens=8191, kv_heads=8, dim=128, page=16,
             order="nhd", dtype="fp16", format="int8", back=True),
        # a few blocks read back for one short sequence
        dict(name="read 257 tokens fp8", op="read", tokens=257, kv_heads=8, dim=128, page=16,
             order="hnd", dtype="bf16", format="fp8"),
        # a long prefix read back for another process
        dict(name="read 65536 tokens int8", op="read", tokens=65536, kv_heads=8, dim=128, page=16,
             order="hnd", dtype="bf16", format="int8"),
        # single tokens: one short sequence, where latency counts
        dict(name="decode 1 x 1000", op="attention", seqs=1, q_len=1, context=1000, heads=32,
             kv_heads=8, dim=128, page=16, order="hnd", dtype="bf16", format="bf16", window=0,
             mix=1),
        # single tokens of a full batch with ragged contexts
        dict(name="decode 64 x 8192", op="attention", seqs=64, q_len=1, context=8192, heads=32,
             kv_heads=8, dim=128, page=16, order="hnd", dtype="bf16", format="bf16", window=0,
             mix=2),
        # single tokens over long e4m3 contexts
        dict(name="decode 12 x 40001 fp8", op="attention", seqs=12, q_len=1, context=40001,
             heads=32, kv_heads=8, dim=128, page=16, order="hnd", dtype="bf16", format="fp8",
             window=0, mix=3),
        # ragged chunks of several prompts, odd sizes, a sliding window, pages of 24 tokens
        dict(name="chunks 5 x 517 windowed", op="attention", seqs=5, q_len=517, context=5003,
             heads=14, kv_heads=2, dim=64, page=24, order="nhd", dtype="fp16", format="fp16",
             window=1500, mix=4),
        # a prompt's chunk over a long cached prefix
        dict(name="chunk 2048 of 18432", op="attention", seqs=1, q_len=2048, context=18432,
             heads=32, kv_heads=8, dim=128, page=16, order="hnd", dtype="bf16", format="bf16",
             window=0, mix=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attention", "attention"])
    dim = rng.choice([64, 64, 80, 96, 128, 128, 128, 256])
    page = rng.choice([1, 8, 16, 16, 16, 24, 32, 64, 100])
    kv = rng.choice([1, 2, 4, 8])
    order = rng.choice(["hnd", "nhd"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "rope":
        rot = rng.choice([dim, dim, dim // 2])
        return dict(op=op, tokens=_log(rng, 1, 8000), heads=kv * rng.choice([1, 4, 7, 8]),
                    kv_heads=kv, dim=dim, rot=rot, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "parts"]), far=_log(rng, 100, 2000000))
    if op in ("write", "read"):
        fmt = rng.choice([dtype, "fp8", "int8", "int8"])
        case = dict(op=op, tokens=_log(rng, 1, 16000), kv_heads=kv, dim=dim, page=page, order=order,
                    dtype=dtype, format=fmt)
        if op == "write":
            case["back"] = fmt == "int8"
        return case
    fmt = rng.choice([dtype, dtype, "fp8", "int8"])
    group = rng.choice([1, 2, 4, 7, 8, 16])
    kind = rng.choice(["decode", "decode", "few", "chunk"])
    if kind == "decode":
        seqs, q_len = _log(rng, 1, 48), 1
    elif kind == "few":
        seqs, q_len = _log(rng, 1, 16), rng.randint(2, 9)
    else:
        seqs, q_len = rng.randint(1, 4), _log(rng, 16, 1100)
    # keep a plain pass within what the largest listed case costs
    most = min(40000, int(6e8 / (seqs * max(q_len * kv * group, 8 * kv * dim // 16))))
    context = max(q_len, _log(rng, 64, max(128, most)))
    return dict(op=op, seqs=seqs, q_len=q_len, context=context, heads=kv * group, kv_heads=kv,
                dim=dim, page=page, order=order, dtype=dtype, format=fmt,
                window=rng.choice([0, 0, 0, _log(rng, 8, 5000)]), mix=rng.randint(10, 1 << 20))


def _lengths(case):
    """(new tokens, cached tokens) of each sequence: the first has the case's
    own, the others shorter ones."""
    r = random.Random(case["mix"])
    q, c = [case["q_len"]], [max(case["q_len"], case["context"])]
    for _ in range(case["seqs"] - 1):
        n = case["q_len"] if case["q_len"] <= 8 else r.randint(1, case["q_len"])
        q.append(n)
        c.append(n + int((case["context"] - n) * r.random() ** 0.5) if case["context"] > n else n)
    return q, c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    return g


def _pool(pages, case, fill):
    """Pages [page, head, place, dim] in the case's memory order, from `fill`
    of that shape in memory."""
    h, p, d = case["kv_heads"], case["page"], case["dim"]
    if case["order"] == "nhd":
        return fill((pages, p, h, d)).transpose(1, 2)
    return fill((pages, h, p, d))


def _random_pages(pages, case, g):
    """A filled cache: codes or values, and its scales."""
    fmt = case["format"]

    def fill(shape):
        x = torch.randn(shape, device="cuda", generator=g, dtype=torch.float32)
        if fmt == "int8":
            return (x * 40).clamp_(-127, 127).round_().to(torch.int8)
        if fmt == "fp8":
            return (x * 150).clamp_(-448, 448).to(torch.float8_e4m3fn)
        return x.to(DTYPES[fmt])

    out = _pool(pages, case, fill)
    if fmt not in QMAX:
        return out, None
    top = QMAX[fmt]
    s = torch.rand((pages, case["kv_heads"], case["page"]), device="cuda", generator=g)
    return out, (1.5 + 3.0 * s) / top


def _frequencies(case):
    """Radians per position of each pair, in 64 bits."""
    half = case["rot"] // 2
    i = torch.arange(half, dtype=torch.float64, device="cuda")
    freq = 10000.0 ** (-i / half) if case["scaling"] != "parts" else 500000.0 ** (-i / half)
    if case["scaling"] == "linear":
        freq = freq / 4.0
    elif case["scaling"] == "parts":
        # long waves slowed by 8, short ones kept, a ramp between
        turns = 8192.0 * freq / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        freq = freq * (keep + (1.0 - keep) / 8.0)
    return freq


def prepare(case, seed):
    g = _rng(seed)
    s = {"case": case}

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    if case["op"] == "rope":
        t, d, dt = case["tokens"], case["dim"], DTYPES[case["dtype"]]
        # queries and keys are slices of one projection's output, as they are in a model
        qkv = randn(t, case["heads"] + 2 * case["kv_heads"], d).to(dt)
        s["q"], s["k"] = qkv[:, :case["heads"]], qkv[:, case["heads"]:case["heads"] + case["kv_heads"]]
        start = torch.randint(0, case["far"], (1,), device="cuda", generator=g)
        s["positions"] = (start + torch.arange(t, device="cuda")).to(torch.int32)
        s["freqs"] = _frequencies(case)
        s["factor"] = 1.0 if case["scaling"] != "parts" else 0.1 * math.log(8.0) + 1.0
        s["q_out"] = torch.empty((t, case["heads"], d), device="cuda", dtype=dt)
        s["k_out"] = torch.empty((t, case["kv_heads"], d), device="cuda", dtype=dt)
        return s
    if case["op"] in ("write", "read"):
        t, h, d = case["tokens"], case["kv_heads"], case["dim"]
        pages = -(-t // case["page"]) + 3
        s["slots"] = torch.randperm(pages * case["page"], device="cuda", generator=g)[:t].contiguous()
        if case["op"] == "write" and t > 16:
            # whole pages in a shuffled order, as an allocator hands them out
            order = torch.randperm(pages, device="cuda", generator=g)
            at = torch.arange(t, device="cuda")
            s["slots"] = order[at // case["page"]] * case["page"] + at % case["page"]
            s["slots"][t // 2] = -1     # a padded token
    if case["op"] == "write":
        kv = randn(t, 2 * h, d).to(DTYPES[case["dtype"]])
        s["k"], s["v"] = kv[:, :h], kv[:, h:]
        dt = DTYPES[case["format"]]
        for n in ("k", "v"):
            s[n + "_pages"] = _pool(pages, case, lambda shape: torch.zeros(
                shape, device="cuda", dtype=torch.uint8 if dt.itemsize == 1 else dt)).view(dt)
            s[n + "_scales"] = torch.zeros((pages, h, case["page"]), device="cuda") \
                if case["format"] in QMAX else None
    elif case["op"] == "read":
        for n in ("k", "v"):
            s[n + "_pages"], s[n + "_scales"] = _random_pages(pages, case, g)
    if case["op"] == "read" or case.get("back"):
        for n in ("k", "v"):
            s[n + "_out"] = torch.empty((t, h, d), device="cuda", dtype=DTYPES[case["dtype"]])
    if case["op"] == "attention":
        q, c = _lengths(case)
        per = [-(-x // case["page"]) for x in c]
        pages = sum(per) + 2
        s["max_pages"], s["q_lens"], s["contexts"] = max(per), q, c
        order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
        starts = torch.tensor([0] + per, device="cuda").cumsum(0)
        at = starts[:-1, None] + torch.arange(max(per), device="cuda")[None, :]
        held = torch.arange(max(per), device="cuda")[None, :] < torch.tensor(per, device="cuda")[:, None]
        s["table"] = torch.where(held, order[at.clamp(max=pages - 1)], 0).to(torch.int32).contiguous()
        s["q_starts"] = torch.tensor([0] + q, device="cuda").cumsum(0).to(torch.int32)
        s["context_lens"] = torch.tensor(c, device="cuda", dtype=torch.int32)
        s["q"] = (randn(sum(q), case["heads"], case["dim"]) * 1.5).to(DTYPES[case["dtype"]])
        for n in ("k", "v"):
            s[n + "_pages"], s[n + "_scales"] = _random_pages(pages, case, g)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], device="cuda")
    if own and case["op"] != "rope":
        from block_copy_amd import kvcache
        s["cache"] = kvcache.PagedCache(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
        if case["op"] == "attention":
            s["plan"] = kvcache.AttentionPlan(
                s["cache"], q_heads=case["heads"], num_seqs=case["seqs"], total_q=sum(q),
                max_q_len=max(q), max_context=max(c), window=case["window"])
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    return {"rope": _rope, "write": _write, "read": _read, "attention": _attention}[case["op"]](case, state)


def _rope(case, s):
    if own:
        from block_copy_amd import kvcache
        kvcache.rope(s["positions"], s["freqs"], s["q"], s["k"], q_out=s["q_out"], k_out=s["k_out"],
                     interleaved=case["interleaved"], factor=s["factor"])
        return {"q": s["q_out"], "k": s["k_out"]}
    angle = s["positions"].double()[:, None, None] * s["freqs"]
    cos, sin = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()

    def turn(x):
        rot = case["rot"]
        y = x.float()
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if case["interleaved"] else (y[..., :rot // 2], y[..., rot // 2:rot])
        lo, hi = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack((lo, hi), -1).flatten(-2) if case["interleaved"] else torch.cat((lo, hi), -1)
        return torch.cat((turned, y[..., rot:]), -1).to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _quantise(x, fmt):
    """Codes and scales of rows of 16-bit values; quotients in 64 bits, since
    many of them lie on a border between two codes."""
    amax = x.abs().amax(-1).float()
    quotient = x.double() * QMAX[fmt] / torch.where(amax == 0, 1.0, amax).double()[..., None]
    codes = quotient.round().to(torch.int8) if fmt == "int8" else quotient.to(torch.float8_e4m3fn)
    return codes, amax / QMAX[fmt]


def _bytes(x):
    """The same memory as whole numbers, which torch indexes."""
    return x.view(torch.uint8) if x.element_size() == 1 else x


def _held(s, n, slots):
    """Float values of the rows at `slots`."""
    page = s["case"]["page"]
    pages, scales = s[n + "_pages"], s[n + "_scales"]
    at, place = slots // page, slots % page
    x = _bytes(pages)[at, :, place].view(pages.dtype).float()
    return x if scales is None else x * scales[at, :, place][..., None]


def _write(case, s):
    if own:
        from block_copy_amd import kvcache
        kvcache.write(s["cache"], s["k"], s["v"], s["slots"])
        if case["back"]:
            kvcache.read(s["cache"], s["slots"], s["k_out"], s["v_out"])
    else:
        # a token to leave out stands for the one before it, written twice with the same values
        at = torch.arange(case["tokens"], device="cuda")
        at = torch.where(s["slots"] < 0, at - 1, at)
        slots = s["slots"][at]
        page, place = slots // case["page"], slots % case["page"]
        for n in ("k", "v"):
            x = s[n][at]
            if case["format"] in QMAX:
                x, scale = _quantise(x, case["format"])
                s[n + "_scales"][page, :, place] = scale
            _bytes(s[n + "_pages"])[page, :, place] = _bytes(x)
        if case["back"]:
            _read(case, s)
    out = {"k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    if case["back"]:
        return dict(out, k=s["k_out"], v=s["v_out"])
    return dict(out, k=s["k_pages"], v=s["v_pages"])


def _read(case, s):
    if own:
        from block_copy_amd import kvcache
        kvcache.read(s["cache"], s["slots"], s["k_out"], s["v_out"])
    else:
        held = (s["slots"] >= 0)[:, None, None]
        for n in ("k", "v"):
            s[n + "_out"].copy_(torch.where(held, _held(s, n, s["slots"].clamp(min=0)), 0.0))
    return {"k": s["k_out"], "v": s["v_out"]}


def _attention(case, s):
    if own:
        s["plan"](s["q"], s["table"], s["q_starts"], s["context_lens"], out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    b, qm, cm = case["seqs"], max(s["q_lens"]), max(s["contexts"])
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    group = h // hk
    starts, ctx = s["q_starts"].long(), s["context_lens"].long()
    lens = starts[1:] - starts[:-1]
    r = torch.arange(qm, device="cuda")
    rows = (starts[:-1, None] + r).clamp(max=s["q"].shape[0] - 1)                      # [b, qm]
    q = s["q"].float()[rows].view(b, qm, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, group * qm, d)
    t = torch.arange(cm, device="cuda")
    slots = s["table"].long()[:, t // case["page"]] * case["page"] + t % case["page"]  # [b, cm]
    k, v = (_held(s, n, slots).permute(0, 2, 1, 3).contiguous() for n in ("k", "v"))
    pos = (ctx - lens)[:, None] + r                                                    # [b, qm]
    seen = (t <= pos[..., None]) & (t < ctx[:, None, None])
    if case["window"]:
        seen &= t > pos[..., None] - case["window"]
    seen = seen[:, None, None]                                                         # [b, 1, 1, qm, cm]
    score = torch.matmul(q, k.transpose(2, 3).contiguous()).view(b, hk, group, qm, cm) / math.sqrt(d)
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score.view(b, hk, group * qm, cm), v).view(b, hk, group, qm, d)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (total.log() + top).squeeze(-1)
    # back to one row a token
    tok = torch.arange(s["q"].shape[0], device="cuda")
    seq = (tok[:, None] >= starts[None, 1:]).sum(1)
    own_row = tok - starts[seq]
    out = out.permute(0, 3, 1, 2, 4).reshape(b, qm, h, d)[seq, own_row].to(s["q"].dtype)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(b, qm, h)[seq, own_row]}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "rope":
        values = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 2 * values * DTYPES[case["dtype"]].itemsize + 4 * case["tokens"] + 4 * case["rot"],
                "flops": 3 * values * case["rot"] / case["dim"]}
    size = DTYPES[case["dtype"]].itemsize
    held = DTYPES[case["format"]].itemsize
    row = held * case["dim"] + (4 if case["format"] in QMAX else 0)
    if case["op"] in ("write", "read"):
        rows = 2 * case["tokens"] * case["kv_heads"]
        passes = 2 if case.get("back") else 1
        return {"bytes": passes * (rows * (row + size * case["dim"]) + 8 * case["tokens"]),
                "flops": passes * 2 * rows * case["dim"]}
    keys = pairs = 0
    q, c = _lengths(case)
    for n, m in zip(q, c):
        w = case["window"] or m
        keys += min(m, n - 1 + w)
        # row r stands at m - n + r and sees min(position + 1, w) keys
        full = max(0, min(n, w - (m - n)))      # rows whose window reaches the start
        pairs += full * (m - n) + full * (full + 1) // 2 + (n - full) * w
    return {"bytes": 2 * keys * case["kv_heads"] * row + sum(q) * case["heads"] * (2 * size * case["dim"] + 4),
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "write": _exact_write, "read": _exact_read,
            "attention": _exact_attention}[case["op"]](case, s)


def _exact_rope(case, s):
    unit = torch.polar(torch.full_like(s["freqs"], s["factor"]).expand(case["tokens"], -1),
                       torch.outer(s["positions"].double(), s["freqs"]))[:, None, :]

    def turn(x):
        y = x.double().clone()
        half = case["rot"] // 2
        first = slice(0, case["rot"], 2) if case["interleaved"] else slice(0, half)
        second = slice(1, case["rot"], 2) if case["interleaved"] else slice(half, case["rot"])
        z = torch.complex(y[..., first], y[..., second]) * unit
        y[..., first], y[..., second] = z.real, z.imag
        return y

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _codes(x, fmt):
    """The nearest code of each value of rows x * Q / amax, ties to the even
    code, from the list of all codes."""
    if fmt == "int8":
        table = torch.arange(128, device="cuda", dtype=torch.float64)
    else:
        n = torch.arange(127, device="cuda")
        e, m = n // 8, n % 8
        table = torch.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e.double() - 7))
    top = x.abs().amax(-1, keepdim=True)
    y = x.abs() * QMAX[fmt] / torch.where(top == 0, 1.0, top)
    hi = torch.searchsorted(table, y).clamp(max=table.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = table[hi] - y, y - table[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.sign(x) * table[pick], top[..., 0] / QMAX[fmt]


def _exact_write(case, s):
    out = {}
    take = (s["slots"] >= 0).nonzero()[:, 0]
    slots = s["slots"][take]
    for n in ("k", "v"):
        x = s[n].double()
        pages = torch.zeros(s[n + "_pages"].shape, device="cuda", dtype=torch.float64)
        scales = None
        if case["format"] in QMAX:
            x, scale = _codes(x, case["format"])
            scales = torch.zeros(s[n + "_scales"].shape, device="cuda", dtype=torch.float64)
            scales[slots // case["page"], :, slots % case["page"]] = scale[take]
        pages[slots // case["page"], :, slots % case["page"]] = x[take]
        out[n + "_scales"] = scales
        if case["back"]:
            values = torch.zeros_like(x)
            values[take] = x[take] * scale[take][..., None]
            out[n] = values
        else:
            out[n] = pages
    return out


def _exact_read(case, s):
    out = {}
    for n in ("k", "v"):
        flat = s[n + "_pages"].double().transpose(1, 2).reshape(-1, case["kv_heads"], case["dim"])
        out[n] = flat[s["slots"]]
        if s[n + "_scales"] is not None:
            out[n] = out[n] * s[n + "_scales"].double().transpose(1, 2).reshape(-1, case["kv_heads"], 1)[s["slots"]]
    return out


def _exact_attention(case, s):
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.full(s["q"].shape[:2], -math.inf, device="cuda", dtype=torch.float64)
    group, at = case["heads"] // case["kv_heads"], 0
    for b, (n, m) in enumerate(zip(s["q_lens"], s["contexts"])):
        used = s["table"][b, :-(-m // case["page"])].long()
        pos = torch.arange(m - n, m, device="cuda")[:, None]
        t = torch.arange(m, device="cuda")[None, :]
        hidden = t > pos
        if case["window"]:
            hidden = hidden | (t <= pos - case["window"])
        for j in range(case["kv_heads"]):
            held = []
            for name in ("k", "v"):
                x = s[name + "_pages"][used, j].double()
                if s[name + "_scales"] is not None:
                    x = x * s[name + "_scales"][used, j].double()[..., None]
                held.append(x.reshape(-1, case["dim"])[:m])
            for i in range(j * group, (j + 1) * group):
                logits = s["q"][at:at + n, i].double() @ held[0].T / case["dim"] ** 0.5
                logits = logits.masked_fill(hidden, -math.inf)
                lse[at:at + n, i] = torch.logsumexp(logits, 1)
                out[at:at + n, i] = torch.softmax(logits, 1) @ held[1]
        at += n
    return {"out": out, "lse": lse}

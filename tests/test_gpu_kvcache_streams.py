"""The cache operators on streams other than torch's current one: what they
make themselves is theirs, whatever work is queued elsewhere, and calls on
several streams overlap without meeting."""
import pytest
import torch

import test_gpu_kvcache as base
from test_gpu_kvcache import C  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F8, I8 = torch.bfloat16, torch.float8_e4m3fn, torch.int8
LONG = 100_000_000     # cycles that a stream is kept busy for: some 50 ms


def _late_write(shapes, dtype):
    """Frees blocks of these sizes that work queued on the current stream will
    still write, as a program does that reuses its buffers."""
    late = [torch.empty(s, dtype=dtype, device=DEV) for s in shapes]
    torch.cuda._sleep(LONG)
    for x in late:
        x.view(torch.uint8).fill_(0x7f)


def _as(stream, kind):
    return stream if kind == "stream" else stream.cuda_stream


@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_outputs_made_for_another_stream(C, kind):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(64, 2, 64, generator=g).to(BF).to(DEV)
    pages = [torch.zeros(4, 2, 16, 64, dtype=BF, device=DEV) for _ in range(2)]
    cache, slots = C.PagedCache(*pages), torch.arange(64, device=DEV)
    C.write(cache, x, x, slots)
    pos, freqs = torch.arange(64, dtype=torch.int32, device=DEV), C.rope_frequencies(64, device=DEV)
    want_q, want_k = C.rope(pos, freqs, x, x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        _late_write([x.shape] * 2, BF)
        k, v = C.read(cache, slots, stream=_as(side, kind))
        side.synchronize()
        kept = k.cpu(), v.cpu()
        torch.cuda.synchronize()
        assert torch.equal(k, x) and torch.equal(v, x) and torch.equal(kept[0], x.cpu())
        del k, v
        _late_write([x.shape] * 2, BF)
        q, k = C.rope(pos, freqs, x, x, stream=_as(side, kind))
        torch.cuda.synchronize()
        assert torch.equal(q, want_q) and torch.equal(k, want_k)
        del q, k


@pytest.mark.parametrize("kind", ["stream", "handle"])
@pytest.mark.parametrize("q_len", [1, 30])
def test_plans_called_on_another_stream(C, kind, q_len):
    """The workspace: made while work on the current stream still writes the
    block it would get there, and dropped while the call still uses it."""
    c = base._case(q_lens=[q_len], ctx=[3000], heads=4, kv=1, dim=64, dtype=BF, kind=I8)
    r = base._attend(C, torch.Generator().manual_seed(4), **c)
    need, want = r["plan"].args.workspace_bytes, r["out"].cpu()
    assert need > 0
    del r["plan"]
    sizes = dict(q_heads=4, num_seqs=1, total_q=q_len, max_q_len=q_len, max_context=3000)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        _late_write([(need,)], torch.uint8)
        plan = C.AttentionPlan(r["cache"], **sizes)
        out = plan(*r["args"], stream=_as(side, kind))
        side.synchronize()
        assert base._eq_bits(out.cpu(), want)
        torch.cuda.synchronize()
        assert base._eq_bits(out.cpu(), want)
        with torch.cuda.stream(side):
            torch.cuda._sleep(LONG)
        out = plan(*r["args"], stream=_as(side, kind))
        del plan
        for _ in range(4):
            torch.empty(need, dtype=torch.uint8, device=DEV).fill_(0x7f)
        torch.cuda.current_stream().synchronize()
        side.synchronize()
        assert base._eq_bits(out.cpu(), want)


def test_the_default_stream_by_its_handle(C):
    """Handle 0 from within another stream's context."""
    x = torch.ones(4, 1, 64, dtype=BF, device=DEV)
    cache, slots = C.PagedCache(torch.zeros(1, 1, 4, 64, dtype=BF, device=DEV), torch.zeros(1, 1, 4, 64, dtype=BF, device=DEV)), \
        torch.arange(4, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        C.write(cache, x, x, slots, stream=0)
        k, v = C.read(cache, slots, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(k, x) and torch.equal(v, x)


@pytest.mark.parametrize("kind", [BF, F8])
@pytest.mark.parametrize("q_len", [1, 40])
def test_calls_that_overlap(C, kind, q_len):
    """Two caches, and one plan on two streams: nothing waits between the
    calls, and each gives what it gives alone."""
    c = base._case(q_lens=[q_len] * 4, ctx=[3000, 1700, 3000, 900], heads=8, kv=2, dim=128, dtype=BF, kind=kind)
    a, b = (base._attend(C, torch.Generator().manual_seed(s), **c) for s in (1, 2))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.zeros_like(a["out"]) for _ in range(24)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        r = (a, b)[i % 2]
        if i < 12:
            r["plan"](*r["args"], out=o, stream=streams[i % 2])
        else:      # a's plan on both streams
            a["plan"](*a["args"], out=o, stream=streams[i % 2])
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert base._eq_bits(o, (a, b)[i % 2 if i < 12 else 0]["out"]), i


def test_a_graph_after_an_eager_call(C):
    """A plan warmed up on one stream, captured on another, and called eagerly
    between replays: every result is the same."""
    c = base._case(q_lens=[1, 1], ctx=[2500, 800], heads=4, kv=1, dim=128, dtype=BF, kind=F8)
    r = base._attend(C, torch.Generator().manual_seed(7), **c)
    out, eager = torch.zeros_like(r["out"]), torch.zeros_like(r["out"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r["plan"](*r["args"], out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r["plan"](*r["args"], out=out)
    for _ in range(4):
        out.zero_()
        eager.zero_()
        graph.replay()
        r["plan"](*r["args"], out=eager)
        torch.cuda.synchronize()
        assert base._eq_bits(out, r["out"]) and base._eq_bits(eager, r["out"])

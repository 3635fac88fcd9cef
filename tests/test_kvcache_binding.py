"""What the torch binding of the cache operators hands to the library, seen on
the CPU: host tensors in place of the GPU's, and a recorder in place of the
call, so nothing is enqueued."""
import ctypes
import os
import subprocess
import types

import pytest
import torch

from block_copy_amd import kvcache as C

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000   # an address that no call gets as far as using


def host_cache(fmt=C.INT8, dim=64, kv=2, page=16, pages=300):
    """What AttentionPlan reads of a PagedCache."""
    coded = fmt in (C.FP8, C.INT8)
    p = C.Pages(ctypes.sizeof(C.Pages), fmt, A, A, A if coded else None, A if coded else None)
    p.k_stride[:] = p.v_stride[:] = (kv * page * dim, page * dim, dim)
    p.ks_stride[:] = p.vs_stride[:] = (kv * page, page, 1)
    p.num_pages, p.kv_heads, p.page_size, p.head_dim = pages, kv, page, dim
    dtype = {C.BF16: BF, C.FP16: FP, C.FP8: torch.float8_e4m3fn, C.INT8: torch.int8}[fmt]
    return types.SimpleNamespace(pages=p, _ref=ctypes.byref(p), coded=coded, dtype=dtype, page_size=page, head_dim=dim,
                                 kv_heads=kv, num_pages=pages, device=torch.device("cpu"))


@pytest.fixture
def calls(monkeypatch):
    """The types of every attention call that reaches the library."""
    seen = []
    monkeypatch.setattr(C, "_call", lambda fn, where, device, stream, pages, args: seen.append(args._obj.dtype))
    return seen


SIZES = dict(q_heads=4, num_seqs=1, total_q=2, max_q_len=2, max_context=40)


def attend(plan, dtype, **kw):
    q = torch.zeros(2, 4, 64, dtype=dtype)
    return plan(q, torch.zeros(1, 3, dtype=torch.int32), torch.tensor([0, 2], dtype=torch.int32),
                torch.tensor([40], dtype=torch.int32), **kw)


def test_a_plan_over_codes_takes_either_type_of_rows(calls):
    plan = C.AttentionPlan(host_cache(), **SIZES)
    for dt in (FP, BF, FP):
        assert attend(plan, dt).dtype == dt
    assert calls == [C.FP16, C.BF16, C.FP16]
    for q, out in ((F32, F32), (BF, FP)):
        with pytest.raises(ValueError):
            attend(plan, q, out=torch.zeros(2, 4, 64, dtype=out))
    assert len(calls) == 3


def test_a_plan_for_one_type_takes_that_type(calls):
    for plan, good, bad in ((C.AttentionPlan(host_cache(), dtype=FP, **SIZES), FP, BF),
                            (C.AttentionPlan(host_cache(C.BF16), **SIZES), BF, FP)):
        attend(plan, good)
        with pytest.raises(ValueError):
            attend(plan, bad)
    assert calls == [C.FP16, C.BF16]
    with pytest.raises(ValueError):
        C.AttentionPlan(host_cache(), dtype=F32, **SIZES)


def test_a_plan_has_a_workspace_for_each_stream(monkeypatch):
    """Memory made under one stream is never given to a call on another."""
    current, spaces, made = [7], [], []
    monkeypatch.setattr(C, "_raw_stream", lambda index: current[0])
    monkeypatch.setattr(C, "_call", lambda fn, where, device, stream, pages, args: spaces.append(args._obj.workspace))
    empty = C._empty
    monkeypatch.setattr(C, "_empty", lambda shape, dtype, device, stream: (
        made.append((C._handle(stream, None), tuple(shape))), empty(shape, dtype, device, None))[1])
    plan = C.AttentionPlan(host_cache(), **dict(SIZES, max_context=4000))
    need = plan.args.workspace_bytes
    assert need > 0 and made == [(7, (need,))]

    def attend(stream):
        plan(torch.zeros(2, 4, 64, dtype=BF), torch.zeros(1, 250, dtype=torch.int32),
             torch.tensor([0, 2], dtype=torch.int32), torch.tensor([4000], dtype=torch.int32), stream=stream)

    attend(None), attend(7), attend(9)
    current[0] = 9
    attend(None), attend(7)
    assert spaces[0] == spaces[1] == spaces[4] == plan.workspace.data_ptr()
    assert spaces[2] == spaces[3] != spaces[0]
    assert [m for m in made if m[1] == (need,)] == [(7, (need,)), (9, (need,))]
    # outputs that are not given are made for the stream that writes them
    assert [m[0] for m in made if m[1] != (need,)] == [7, 7, 9, 9, 7]


def test_windows_as_large_as_they_may_be(tmp_path):
    """tests/native/window_check.cpp, under sanitizers."""
    exe = tmp_path / "window"
    subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-fsanitize=undefined,address", "-fno-sanitize-recover=all",
                    "-I" + os.path.join(ROOT, "block_copy_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "window_check.cpp"), "-o", str(exe)],
                   check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


def test_gradients_are_not_lost_silently(calls):
    """What would need one is refused while gradients are on."""
    x = torch.zeros(2, 4, 64, dtype=BF)
    y = x.clone().requires_grad_()
    cache, plan = host_cache(kv=4), C.AttentionPlan(host_cache(), **SIZES)
    slots = torch.arange(2)
    table, starts, lens = torch.zeros(1, 3, dtype=torch.int32), torch.tensor([0, 2], dtype=torch.int32), \
        torch.tensor([40], dtype=torch.int32)
    asks = [lambda: C.write(cache, y, x, slots), lambda: C.write(cache, x, y, slots), lambda: C.read(cache, slots, y, x), lambda: C.read(cache, slots, x, y),
            lambda: plan(y, table, starts, lens), lambda: plan(x, table, starts, lens, out=y),
            lambda: plan(x, table, starts, lens, lse=torch.zeros(2, 4, requires_grad=True))]
    for ask in asks:
        with pytest.raises(ValueError, match="gradient"):
            ask()
    assert not calls
    for ready in (torch.no_grad(), torch.inference_mode()):
        with ready:
            plan(y, table, starts, lens)
    plan(y.detach(), table, starts, lens)
    assert len(calls) == 3


@pytest.mark.parametrize("kw", [
    dict(q_heads=3), dict(q_heads=0), dict(window=-1), dict(num_seqs=65536), dict(num_seqs=-1), dict(total_q=-2),
    dict(total_q=1 << 31), dict(max_q_len=1 << 31), dict(max_context=(1 << 31) - 1), dict(scale=float("nan")),
    # values that 32 bits would take for others
    dict(q_heads=(1 << 32) + 4), dict(num_seqs=(1 << 32) + 1), dict(total_q=(1 << 32) + 2), dict(max_q_len=(1 << 32) + 2),
    dict(max_context=(1 << 32) + 40), dict(window=1 << 32), dict(window=1 << 31), dict(max_q_len=2.5), dict(window=1.0)])
def test_plans_that_no_call_would_take(calls, kw):
    """Refused when they are made, not at their first call."""
    with pytest.raises((C.KvcopyError, ValueError, TypeError)):
        C.AttentionPlan(host_cache(), **dict(SIZES, **kw))


def test_plans_over_pages_that_no_call_would_take(calls):
    with pytest.raises(C.KvcopyError) as e:
        C.AttentionPlan(host_cache(C.BF16), dtype=FP, **SIZES)
    assert e.value.code == C.EINVAL
    for kw, code in ((dict(dim=60), C.EALIGN), (dict(dim=264), C.EINVAL)):
        with pytest.raises(C.KvcopyError) as e:
            C.AttentionPlan(host_cache(**kw), **SIZES)
        assert e.value.code == code
    odd = host_cache()
    odd.pages.k = A + 4
    with pytest.raises(C.KvcopyError) as e:
        C.AttentionPlan(odd, **SIZES)
    assert e.value.code == C.EALIGN
    # empty batches are plans
    for kw in (dict(num_seqs=0, total_q=0), dict(total_q=0), dict(max_q_len=0, total_q=0), dict(max_context=0)):
        C.AttentionPlan(host_cache(), **dict(SIZES, **kw))
    # and so are sizes at their limits: a launch of 2^23 workgroups is beyond the grid
    big = dict(q_heads=16, num_seqs=1, max_q_len=(1 << 28) - 8192, total_q=(1 << 28) - 8192)
    with pytest.raises(C.KvcopyError):
        C.AttentionPlan(host_cache(kv=2), **dict(SIZES, **dict(big, q_heads=14)))
    C.AttentionPlan(host_cache(kv=2), **dict(SIZES, **dict(big, max_q_len=(1 << 27) - 512, total_q=(1 << 27) - 512)))


@pytest.mark.parametrize("args", [(-8,), ((1 << 32) + 64,), (64, 1e4, "parts", 2.0, -1), (64, 1e4, "parts", 2.0, (1 << 32) + 1)])
def test_frequencies_of_sizes_beyond_32_bits(args):
    with pytest.raises((C.KvcopyError, ValueError)):
        C.rope_frequencies(*args)


def test_strides_of_one_do_not_matter():
    """A dimension of extent 1 is never stepped over, whatever its stride."""
    def check(**kw):
        pages = host_cache(C.INT8, kv=kw.get("kv_heads", 2), page=kw.get("page_size", 16), pages=kw.get("num_pages", 9)).pages
        for n, v in kw.items():
            if isinstance(v, dict):
                for i, stride in v.items():
                    getattr(pages, n)[i] = stride
        a = C.AttentionArgs(ctypes.sizeof(C.AttentionArgs), C.BF16)
        a.num_seqs = a.total_q = a.max_q_len = a.table_columns = 1
        a.q_heads, a.max_context, a.scale = 2, 1, 1.0
        return C.lib.kvcache_attention_check(ctypes.byref(pages), ctypes.byref(a))

    for n, i in (("num_pages", 0), ("kv_heads", 1), ("page_size", 2)):
        for name in ("k_stride", "v_stride"):
            for stride in (3, -5, 1 << 50):
                assert check(**{n: 1, name: {i: stride}}) == C.OK, (n, name, stride)
            assert check(**{n: 2, name: {i: 3}}) == C.EALIGN
    for name in ("ks_stride", "vs_stride"):
        assert check(num_pages=1, **{name: {0: -7}}) == C.OK and check(page_size=1, **{name: {2: 1 << 40}}) == C.OK
        assert check(num_pages=2, **{name: {0: -7}}) == C.EINVAL


def test_more_rows_than_the_join_of_splits_takes():
    """Refused before the first launch, not after it."""
    pages = host_cache().pages

    def check(**kw):
        a = C.AttentionArgs(ctypes.sizeof(C.AttentionArgs), C.BF16)
        a.num_seqs = a.max_q_len = 1
        a.q_heads, a.scale, a.max_context, a.table_columns = 16, 1.0, 4096, 256
        for n, v in kw.items():
            setattr(a, n, v)
        return C.lib.kvcache_attention_check(ctypes.byref(pages), ctypes.byref(a)), \
            C.lib.kvcache_attention_workspace_bytes(ctypes.byref(pages), ctypes.byref(a))
    for n in (1, 40):
        assert check(total_q=1 << 20, max_q_len=n)[0] == C.EINVAL
        rc, need = check(total_q=(1 << 20) - 1, max_q_len=n)
        assert rc == C.OK and need > 0
        rc, need = check(total_q=1 << 20, max_q_len=n, max_context=32)      # one split: nothing is joined
        assert rc == C.OK and need == 0

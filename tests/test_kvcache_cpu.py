"""The cache operators' host side, without a GPU: the binding against the
compiled header, refusals, frequencies, and the paging arithmetic."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kvcache.h")


@pytest.fixture(scope="module")
def C():
    from block_copy_amd import kvcache
    return kvcache


def test_header_symbols_are_exported(C):
    txt = open(HEADER).read()
    declared = sorted(set(re.findall(r"^(?:int|uint64_t) (kvcache_\w+)\(", txt, re.M)))
    assert declared == sorted(C.EXPORTS)
    from block_copy_amd.kvcopy import LIB_PATH
    out = subprocess.run(["nm", "-D", "--defined-only", LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert set(declared) <= set(re.findall(r"\bT (kvcache_\w+)", out))


def test_binding_matches_the_compiled_header(C, tmp_path):
    consts = {n: "KVCACHE_" + n for n in ("BF16", "FP16", "FP32", "FP8", "INT8", "BAD_PAGE", "BAD_SLOT", "BAD_LENGTH",
                                          "ROPE_INTERLEAVED", "ROPE_INVERSE", "MAX_HEAD_DIM",
                                          "MAX_ATTENTION_HEAD_DIM")}
    kinds = {"none": "PLAIN", "linear": "LINEAR", "base": "BASE", "parts": "PARTS"}
    structs = {"kvcache_rows_t": C.Rows, "kvcache_pages_t": C.Pages, "kvcache_rope_t": C.Rope,
               "kvcache_attention_t": C.AttentionArgs}
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "kvcache.h"', "int main(void) {"]
    src += [f'printf("{k} %lld\\n", (long long)({v}));' for k, v in consts.items()]
    src += [f'printf("kind_{k} %d\\n", (int)KVCACHE_ROPE_{v});' for k, v in kinds.items()]
    for name, cls in structs.items():
        src.append(f'printf("sizeof {name} %zu\\n", sizeof({name}));')
        src += [f'printf("offsetof {name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src += ["return 0;", "}"]
    c, exe = tmp_path / "c.c", tmp_path / "c"
    c.write_text("\n".join(src) + "\n")
    subprocess.run(["gcc", "-std=c11", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + os.path.join(ROOT, "include"), str(c), "-o", str(exe)], check=True, capture_output=True)
    got = dict(line.rsplit(" ", 1) for line in subprocess.run([str(exe)], check=True, capture_output=True,
                                                              text=True).stdout.splitlines())
    for n in consts:
        assert getattr(C, n) == int(got[n]), n
    # the packed form of kvcache_rope_t: the same bytes as the structure's
    rows = [(10 + i, 20 + i, 30 + i) for i in range(4)]
    flat = (C.ctypes.sizeof(C.Rope), 1, 2, 0.5, 77, 88, 9, 64, 32, 8, 2)
    a = C.Rope(*flat, *[C.Rows(*r) for r in rows])
    assert bytes(a) == C._PACK_ROPE(*flat, *[x for r in rows for x in r])
    for k in kinds:
        assert C.SCALINGS[k] == int(got["kind_" + k])
    for name, cls in structs.items():
        assert ctypes.sizeof(cls) == int(got[f"sizeof {name}"])
        for f, _ in cls._fields_:
            assert getattr(cls, f).offset == int(got[f"offsetof {name} {f}"]), (name, f)


def test_paging_arithmetic(tmp_path):
    """tests/native/paging_check.cpp against plain arithmetic, under sanitizers."""
    exe = tmp_path / "paging"
    subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-fsanitize=undefined,address", "-fno-sanitize-recover=all",
                    "-I" + os.path.join(ROOT, "block_copy_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "paging_check.cpp"), "-o", str(exe)],
                   check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


# ---------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------

def test_frequencies(C):
    near = lambda a, b: abs(a - b) <= 4e-15 * abs(b)  # noqa: E731  (a power and a product in 64 bits)
    f = C.rope_frequencies(128, 10000.0)
    assert f.dtype == torch.float64 and f.shape == (64,)
    for i in range(64):
        assert near(f[i].item(), math.exp(-2 * i / 128 * math.log(10000.0)))
    assert torch.equal(C.rope_frequencies(128, scaling="linear", factor=4.0), f / 4)
    b = C.rope_frequencies(64, scaling="base", factor=8.0)
    assert b[0] == 1.0 and near(b[-1].item(), 10000.0 ** (-62 / 64) / 8.0)
    p = C.rope_frequencies(64, 500000.0, "parts", 8.0, 8192, 1.0, 4.0)
    plain = C.rope_frequencies(64, 500000.0)
    seen = set()
    for i in range(32):
        turns = 8192 * plain[i].item() / (2 * math.pi)
        if turns >= 4.0:
            want, kind = plain[i].item(), "kept"
        elif turns <= 1.0:
            want, kind = plain[i].item() / 8, "slowed"
        else:
            keep, kind = (turns - 1) / 3, "between"
            want = plain[i].item() * (keep + (1 - keep) / 8)
        seen.add(kind)
        assert near(p[i].item(), want)
    assert seen == {"kept", "slowed", "between"}


@pytest.mark.parametrize("args", [
    (0,), (7,), (514,), (64, 1.0), (64, 0.5), (64, math.inf), (64, math.nan), (64, 1e4, "linear", 0.5),
    (64, 1e4, "linear", math.nan), (2, 1e4, "base", 2.0), (64, 1e4, "parts", 2.0, 0), (64, 1e4, "parts", 2.0, 100, -1.0, 4.0),
    (64, 1e4, "parts", 2.0, 100, 4.0, 4.0), (64, 1e308, "base", 1e10)])
def test_frequency_refusals(C, args):
    with pytest.raises(C.KvcopyError) as e:
        C.rope_frequencies(*args)
    assert e.value.code == C.EINVAL


# ---------------------------------------------------------------------------
# refusals of the C entries: nothing below reaches a GPU
# ---------------------------------------------------------------------------

A = 0x10000   # an address no call gets as far as using


def _pages(C, **kw):
    p = C.Pages(ctypes.sizeof(C.Pages), C.INT8, A, A, A, A)
    for n in ("k_stride", "v_stride"):
        setattr(p, n, (ctypes.c_int64 * 3)(2 * 16 * 64, 16 * 64, 64))
    for n in ("ks_stride", "vs_stride"):
        setattr(p, n, (ctypes.c_int64 * 3)(32, 16, 1))
    p.num_pages, p.kv_heads, p.page_size, p.head_dim = 10, 2, 16, 64
    for n, v in kw.items():
        setattr(p, n, (ctypes.c_int64 * 3)(*v) if n.endswith("stride") else v)
    return p


BAD_PAGES = [dict(struct_size=8), dict(format=2), dict(format=9), dict(k=None), dict(v=None), dict(k_scale=None),
             dict(v_scale=None), dict(num_pages=0), dict(kv_heads=0), dict(page_size=0), dict(head_dim=0),
             dict(head_dim=520), dict(kv_heads=1 << 17), dict(num_pages=1 << 27), dict(num_pages=1 << 40)]


def _row_call(C, f, pages, dtype=0, tokens=3, k=A, v=A, slots=A, status=None):
    r, w = C.Rows(k, 128, 64), C.Rows(v, 128, 64)
    return f(ctypes.byref(pages), dtype, ctypes.byref(r), ctypes.byref(w), slots, tokens, status, None)


@pytest.mark.parametrize("name", ["kvcache_write", "kvcache_read"])
def test_row_refusals(C, name):
    f = getattr(C.lib, name)
    for kw in BAD_PAGES:
        assert _row_call(C, f, _pages(C, **kw)) == C.EINVAL, kw
    p = _pages(C)
    for kw in (dict(dtype=3), dict(dtype=4), dict(k=None), dict(v=None), dict(slots=None), dict(tokens=1 << 31),
               dict(tokens=1 << 30)):
        assert _row_call(C, f, p, **kw) == C.EINVAL, kw
    for kw in (dict(k=A + 1), dict(v=A + 1), dict(slots=A + 4), dict(status=A + 2)):
        assert _row_call(C, f, p, **kw) == C.EALIGN, kw
    assert _row_call(C, f, _pages(C, k_scale=A + 2)) == C.EALIGN
    assert _row_call(C, f, _pages(C, format=0, k=A + 1)) == C.EALIGN
    assert f(None, 0, None, None, A, 3, None, None) == C.EINVAL
    assert f(ctypes.byref(p), 0, None, None, A, 3, None, None) == C.EINVAL
    assert _row_call(C, f, p, tokens=0, k=None, v=None, slots=None) == C.OK
    if name == "kvcache_write":
        assert _row_call(C, f, p, dtype=2) == C.EINVAL
        assert _row_call(C, f, _pages(C, format=1), dtype=0) == C.EINVAL


def test_rope_refusals(C):
    def call(**kw):
        a = C.Rope(ctypes.sizeof(C.Rope), 0, 0, 1.0, A, A, 4, 64, 64, 8, 2, C.Rows(A, 512, 64), C.Rows(A, 128, 64),
                   C.Rows(A, 512, 64), C.Rows(A, 128, 64))
        for n, v in kw.items():
            if "_data" in n:
                getattr(a, n[:-5]).data = v
            else:
                setattr(a, n, v)
        return C.lib.kvcache_rope(ctypes.byref(a), None)
    assert C.lib.kvcache_rope(None, None) == C.EINVAL
    for kw in (dict(struct_size=4), dict(dtype=3), dict(dtype=7), dict(flags=4), dict(factor=math.inf),
               dict(factor=math.nan), dict(head_dim=0), dict(head_dim=514), dict(rot_dim=7), dict(rot_dim=66),
               dict(q_heads=0), dict(q_heads=1 << 17), dict(k_heads=1 << 17), dict(k_heads=0), dict(tokens=1 << 31),
               dict(positions=None), dict(freq=None), dict(q_data=None), dict(q_out_data=None), dict(k_out_data=None)):
        assert call(**kw) == C.EINVAL, kw
    for kw in (dict(q_data=A + 1), dict(k_out_data=A + 1), dict(positions=A + 2), dict(freq=A + 4)):
        assert call(**kw) == C.EALIGN, kw
    assert call(tokens=0) == C.OK


def _attention(C, pages=None, **kw):
    a = C.AttentionArgs(ctypes.sizeof(C.AttentionArgs), 0, C.Rows(A, 512, 64), C.Rows(A, 512, 64), A, 8, 1, A, 8, A, A,
                        None, 0, None, 4, 8, 8, 4, 1, 128, 0, 0.125)
    for n, v in kw.items():
        if n.endswith("_rows"):
            setattr(a, n[:-5], C.Rows(*v))
        else:
            setattr(a, n, v)
    return pages if pages is not None else _pages(C), a


def test_attention_refusals(C):
    def call(pages=None, **kw):
        p, a = _attention(C, pages, **kw)
        return C.lib.kvcache_attention(ctypes.byref(p), ctypes.byref(a), None)
    for kw in BAD_PAGES + [dict(head_dim=264)]:
        assert call(_pages(C, **kw)) == C.EINVAL, kw
    p = _pages(C)
    assert C.lib.kvcache_attention(ctypes.byref(p), None, None) == C.EINVAL
    assert C.lib.kvcache_attention(None, None, None) == C.EINVAL
    for kw in (dict(struct_size=8), dict(dtype=2), dict(dtype=3), dict(q_heads=0), dict(q_heads=7),
               dict(q_heads=1 << 17), dict(num_seqs=65536), dict(total_q=(1 << 31) - 1), dict(max_q_len=(1 << 31) - 1),
               dict(max_context=(1 << 31) - 1), dict(max_context=129), dict(table_columns=7), dict(window=-1),
               dict(scale=math.nan), dict(scale=math.inf), dict(q_rows=(None, 512, 64)), dict(out_rows=(None, 512, 64)),
               dict(q_starts=None), dict(context_lens=None), dict(page_table=None)):
        assert call(**kw) == C.EINVAL, kw
    assert call(_pages(C, format=0), dtype=1) == C.EINVAL
    for kw in (dict(k_stride=(-2048, 1024, 64)), dict(v_stride=(2048, 1024, -64)), dict(k_stride=(1 << 35, 1024, 64)),
               dict(ks_stride=(1 << 32, 16, 1)), dict(vs_stride=(32, 16, -1))):
        assert call(_pages(C, **kw)) == C.EINVAL, kw
    # a workspace that is too small, or missing
    long = dict(num_seqs=1, max_context=4096, table_columns=256)
    pg, a = _attention(C, **long)
    need = C.lib.kvcache_attention_workspace_bytes(ctypes.byref(pg), ctypes.byref(a))
    assert need > 0
    assert call(**long, workspace=A, workspace_bytes=need - 1) == C.EINVAL
    assert call(**long, workspace=None, workspace_bytes=need) == C.EINVAL
    assert call(**long, workspace=A + 8, workspace_bytes=need) == C.EALIGN
    for kw in (dict(q_rows=(A + 2, 512, 64)), dict(q_rows=(A, 516, 64)), dict(q_rows=(A, 512, 68)),
               dict(out_rows=(A + 8, 512, 64)), dict(out_rows=(A, 512, 65)), dict(lse=A + 2), dict(status=A + 1),
               dict(page_table=A + 2), dict(q_starts=A + 1), dict(context_lens=A + 3)):
        assert call(**kw) == C.EALIGN, kw
    for kw in (dict(head_dim=60), dict(k=A + 4), dict(v_stride=(2048, 1024, 65)), dict(k_stride=(2049, 1024, 64))):
        assert call(_pages(C, **kw)) == C.EALIGN, kw
    for kw in (dict(num_seqs=0), dict(total_q=0), dict(max_q_len=0)):
        assert call(**kw) == C.OK


def test_workspace_depends_on_sizes_alone(C):
    pg, a = _attention(C, num_seqs=1, max_context=4096, table_columns=256)
    f = C.lib.kvcache_attention_workspace_bytes
    need = f(ctypes.byref(pg), ctypes.byref(a))
    a.q_starts = a.context_lens = a.page_table = None
    assert f(ctypes.byref(pg), ctypes.byref(a)) == need
    a.window = -1
    assert f(ctypes.byref(pg), ctypes.byref(a)) == 0


def test_tensors_on_the_wrong_device_or_of_the_wrong_kind(C):
    x = torch.zeros(2, 1, 16, 64)
    for t in (x.bfloat16(), x):
        with pytest.raises(ValueError):
            C.PagedCache(t, t)
    with pytest.raises(ValueError):
        C.rope(torch.zeros(1, dtype=torch.int32), torch.zeros(4, dtype=torch.float64), x[0])


@pytest.mark.parametrize("src", ["cache_kernels.hip", "attention.hip"])
def test_no_kernel_uses_packed_fp32(src):
    """The build keeps packed fp32 arithmetic out of the kernels."""
    from block_copy_amd import build as B
    out = os.path.join(ROOT, "_build", src + ".meta.s")
    os.makedirs(os.path.dirname(out), exist_ok=True)
    subprocess.run(["hipcc", *B.HIPCC_FLAGS, "--cuda-device-only", "-S", "-I" + os.path.join(ROOT, "include"),
                    "-I" + os.path.join(ROOT, "block_copy_amd", "csrc"),
                    os.path.join(ROOT, "block_copy_amd", "csrc", src), "-o", out], check=True, capture_output=True)
    assert not re.search(r"v_pk_(add|mul|fma)_f32", open(out).read())

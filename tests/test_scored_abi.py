"""Refusals of the scored-attention and page-move entry points (CPU only: nothing is launched) and
the layout of the score descriptor."""
import ctypes
import os
import shutil
import subprocess

import pytest

from paged_kv_cache_238_gb300 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists(
    os.path.join(ROOT, "paged_kv_cache_238_gb300", "libpa.so")), reason="needs nvcc to build libpa")

FAKE = 0x10000  # a 16-byte-aligned non-null address; never dereferenced by these calls


def score(**kw):
    d = B.ScoreDesc()
    for k, v in kw.items():
        setattr(d, k, v)
    return d


BAD_SHAPES = [
    (dict(Hq=6, Hkv=4), B.PA_ERR_INVALID_ARG),
    (dict(D=96), B.PA_ERR_UNSUPPORTED),
    (dict(D=0), B.PA_ERR_INVALID_ARG),
    (dict(dt=7), B.PA_ERR_INVALID_ARG),
    (dict(bs=48), B.PA_ERR_UNSUPPORTED),
    (dict(bs=0), B.PA_ERR_INVALID_ARG),
    (dict(max_len=65), B.PA_ERR_INVALID_ARG),             # beyond max_blocks * 16
    (dict(q=None), B.PA_ERR_INVALID_ARG),
    (dict(out=FAKE + 8), B.PA_ERR_INVALID_ARG),
    (dict(bt=FAKE + 2), B.PA_ERR_INVALID_ARG),
    (dict(S=-1), B.PA_ERR_INVALID_ARG),
    (dict(NB=1 << 27), B.PA_ERR_UNSUPPORTED),
    (dict(Hq=70000, Hkv=70000), B.PA_ERR_UNSUPPORTED),    # beyond the grid
    (dict(sc=score(softcap=-1.0)), B.PA_ERR_INVALID_ARG),
    (dict(sc=score(softcap=float("nan"))), B.PA_ERR_INVALID_ARG),
    (dict(sc=score(softcap=float("inf"))), B.PA_ERR_INVALID_ARG),
    (dict(sc=score(window=-1)), B.PA_ERR_INVALID_ARG),
    (dict(sc=score(alibi_slopes=FAKE + 2)), B.PA_ERR_INVALID_ARG),
    (dict(sc=score(key_start=FAKE + 1)), B.PA_ERR_INVALID_ARG),
    (dict(sc=score(prefix_len=FAKE + 3)), B.PA_ERR_INVALID_ARG),
    (dict(S=0, out=None, q=None), B.PA_OK),
]


def base(**kw):
    a = dict(out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, mb=4, lens=FAKE, qsl=FAKE, S=2, chunk=16, max_len=64, Hq=8,
             Hkv=2, D=128, NB=16, bs=16, dt=B.PA_BF16, sc=None)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,expect", BAD_SHAPES)
def test_decode_scored_refuses(kw, expect):
    a = base(**kw)
    assert B.load().pa_decode_scored(a["out"], a["q"], a["kc"], a["vc"], a["bt"], a["mb"], a["lens"], a["S"],
                                     a["max_len"], a["Hq"], a["Hkv"], a["D"], a["NB"], a["bs"], 0.1, a["sc"], a["dt"],
                                     FAKE, 1 << 30, None) == expect


@pytest.mark.parametrize("kw,expect", BAD_SHAPES + [
    (dict(qsl=None), B.PA_ERR_INVALID_ARG),
    (dict(qsl=FAKE + 2), B.PA_ERR_INVALID_ARG),
    (dict(chunk=65), B.PA_ERR_INVALID_ARG),
    (dict(chunk=-1), B.PA_ERR_INVALID_ARG),
    (dict(chunk=0, q=None), B.PA_OK),
    (dict(S=1 << 27, chunk=64), B.PA_ERR_UNSUPPORTED),
])
def test_prefill_scored_refuses(kw, expect):
    a = base(**kw)
    assert B.load().pa_prefill_scored(a["out"], a["q"], a["kc"], a["vc"], a["bt"], a["mb"], a["lens"], a["qsl"], a["S"],
                                      a["chunk"], a["max_len"], a["Hq"], a["Hkv"], a["D"], a["NB"], a["bs"], 0.1,
                                      a["sc"], a["dt"], FAKE, 1 << 30, None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), B.PA_ERR_INVALID_ARG),
    (dict(H=0), B.PA_ERR_INVALID_ARG),
    (dict(D=12), B.PA_ERR_UNSUPPORTED),                   # rows of 24 bytes
    (dict(bs=8), B.PA_ERR_UNSUPPORTED),
    (dict(dt=3), B.PA_ERR_INVALID_ARG),
    (dict(pools=[FAKE, 0]), B.PA_ERR_INVALID_ARG),        # a null pool
    (dict(pools=[FAKE, FAKE + 8]), B.PA_ERR_INVALID_ARG),  # a misaligned one
    (dict(pairs=None), B.PA_ERR_INVALID_ARG),
    (dict(pairs=FAKE + 4), B.PA_ERR_INVALID_ARG),         # pairs are read as 8 bytes
    (dict(tokens=FAKE + 2), B.PA_ERR_INVALID_ARG),
    (dict(table=FAKE, lens=None), B.PA_ERR_INVALID_ARG),  # a table without lengths
    (dict(table=FAKE, mb=0), B.PA_ERR_INVALID_ARG),
    (dict(table=FAKE, S=-1), B.PA_ERR_INVALID_ARG),
    (dict(n=0, pairs=None), B.PA_OK),
    (dict(pools=[]), B.PA_OK),
])
def test_move_blocks_refuses(kw, expect):
    a = dict(pools=[FAKE, FAKE], H=2, D=128, NB=16, bs=16, dt=B.PA_BF16, pairs=FAKE, n=3, tokens=None, table=None,
             mb=4, lens=FAKE, S=2)
    a.update(kw)
    ptrs = (ctypes.c_void_p * max(1, len(a["pools"])))(*a["pools"])
    assert B.load().pa_move_blocks(ptrs, len(a["pools"]), a["H"], a["D"], a["NB"], a["bs"], a["dt"], a["pairs"], a["n"],
                                   a["tokens"], a["table"], a["mb"], a["lens"], a["S"], None) == expect


def test_score_desc_layout_matches_the_header(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("needs gcc")
    names = [f[0] for f in B.ScoreDesc._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "pa.h"\nint main(void) {\n'
                   '  printf("%zu\\n", sizeof(pa_score));\n' +
                   "".join(f'  printf("%zu\\n", offsetof(pa_score, {n}));\n' for n in names) + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(B.ScoreDesc)] + [getattr(B.ScoreDesc, n).offset for n in names]


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    t = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    pool = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.pa_decode_scored(t, t, pool, pool, table, lens, 64, 0.1)
    with pytest.raises(ValueError):
        B.pa_prefill_scored(t, t, pool, pool, table, lens, lens, 1, 64, 0.1)
    with pytest.raises(ValueError):
        B.pa_move_blocks([pool], torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        B.PoolList([])
    with pytest.raises(TypeError):
        B.PoolList([pool.half()])

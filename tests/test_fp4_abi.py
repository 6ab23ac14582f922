"""Refusals of the rotation and 4-bit pool entry points (CPU only: nothing is launched), the layout of the rotation's
descriptor, and the 4-bit definition that the GPU tests compare with."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import fp4_reference as R
from paged_kv_cache_238_gb300 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists(
    os.path.join(ROOT, "paged_kv_cache_238_gb300", "libpa.so")), reason="needs nvcc to build libpa")

FAKE = 0x10000  # a 16-byte-aligned non-null address; never dereferenced by these calls
NAN, INF = float("nan"), float("inf")


def rotate(**kw):
    a = dict(q_out=FAKE, q=FAKE, k=FAKE, v=FAKE, q_out_stride=1024, q_stride=1024, k_stride=256, v_stride=256,
             positions=FAKE, cos_sin=FAKE, num_positions=100, rotary_dim=128, interleaved=0, k_cache=FAKE, v_cache=FAKE,
             slot_mapping=FAKE, num_tokens=2, num_q_heads=8, num_kv_heads=2, head_dim=128, num_blocks=16, block_size=16,
             dtype=B.PA_BF16, cache_dtype=B.PA_FP4, k_scale=1.0, v_scale=1.0)
    a.update(kw)
    d = B.RotateDesc()
    for k, v in a.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,expect", [
    (dict(num_tokens=-1), B.PA_ERR_INVALID_ARG),
    (dict(num_q_heads=-1), B.PA_ERR_INVALID_ARG),
    (dict(num_kv_heads=0), B.PA_ERR_INVALID_ARG),
    (dict(num_positions=-1), B.PA_ERR_INVALID_ARG),
    (dict(rotary_dim=0), B.PA_ERR_INVALID_ARG),
    (dict(rotary_dim=144), B.PA_ERR_INVALID_ARG),
    (dict(rotary_dim=24), B.PA_ERR_UNSUPPORTED),
    (dict(interleaved=2), B.PA_ERR_INVALID_ARG),
    (dict(head_dim=192), B.PA_ERR_UNSUPPORTED),
    (dict(block_size=8), B.PA_ERR_UNSUPPORTED),
    (dict(block_size=0), B.PA_ERR_INVALID_ARG),
    (dict(dtype=B.PA_FP4), B.PA_ERR_INVALID_ARG),
    (dict(cache_dtype=B.PA_F32), B.PA_ERR_INVALID_ARG),  # neither the call's type nor 4 bits
    (dict(k_scale=0.0), B.PA_ERR_INVALID_ARG),
    (dict(k_scale=3.0), B.PA_ERR_INVALID_ARG),
    (dict(v_scale=-1.0), B.PA_ERR_INVALID_ARG),
    (dict(v_scale=NAN), B.PA_ERR_INVALID_ARG),
    (dict(v_scale=INF), B.PA_ERR_INVALID_ARG),
    (dict(v_scale=2.0 ** 25), B.PA_ERR_INVALID_ARG),
    (dict(v_scale=2.0 ** -25), B.PA_ERR_INVALID_ARG),
    (dict(num_blocks=1 << 27), B.PA_ERR_UNSUPPORTED),
    (dict(num_tokens=1 << 26), B.PA_ERR_UNSUPPORTED),     # more items than 31 bits count
    (dict(k=None), B.PA_ERR_INVALID_ARG),
    (dict(q=None), B.PA_ERR_INVALID_ARG),
    (dict(q_out=FAKE + 8), B.PA_ERR_INVALID_ARG),
    (dict(v=FAKE + 2), B.PA_ERR_INVALID_ARG),
    (dict(cos_sin=None), B.PA_ERR_INVALID_ARG),
    (dict(cos_sin=FAKE + 4), B.PA_ERR_INVALID_ARG),
    (dict(positions=FAKE + 4), B.PA_ERR_INVALID_ARG),
    (dict(slot_mapping=FAKE + 4), B.PA_ERR_INVALID_ARG),
    (dict(k_stride=252), B.PA_ERR_INVALID_ARG),   # rows off the 16-byte grid
    (dict(k_stride=248), B.PA_ERR_INVALID_ARG),   # rows into one another
    (dict(q_stride=1016), B.PA_ERR_INVALID_ARG),
    (dict(q_out_stride=0), B.PA_ERR_INVALID_ARG),
    (dict(num_tokens=0, k=None, q=None), B.PA_OK),
])
def test_rotate_refuses(kw, expect):
    assert B.load().pa_rotate_and_cache(ctypes.byref(rotate(**kw)), None) == expect


def test_no_descriptor_is_refused():
    for call in ("pa_rotate_and_cache", "pa_decode_fp4", "pa_prefill_fp4", "pa_gather_fp4"):
        assert getattr(B.load(), call)(None, None) == B.PA_ERR_INVALID_ARG


SHAPES = [
    (dict(Hq=6, Hkv=4), B.PA_ERR_INVALID_ARG),
    (dict(D=96), B.PA_ERR_UNSUPPORTED),
    (dict(dt=B.PA_FP4), B.PA_ERR_INVALID_ARG),             # the pools are 4-bit, the queries are not
    (dict(bs=48), B.PA_ERR_UNSUPPORTED),
    (dict(max_len=65), B.PA_ERR_INVALID_ARG),
    (dict(q=None), B.PA_ERR_INVALID_ARG),
    (dict(kc=FAKE + 8), B.PA_ERR_INVALID_ARG),
    (dict(bt=FAKE + 2), B.PA_ERR_INVALID_ARG),
    (dict(S=-1), B.PA_ERR_INVALID_ARG),
    (dict(NB=1 << 27), B.PA_ERR_UNSUPPORTED),
    (dict(Hq=70000, Hkv=70000), B.PA_ERR_UNSUPPORTED),
    (dict(ks=1.5), B.PA_ERR_INVALID_ARG),
    (dict(vs=0.0), B.PA_ERR_INVALID_ARG),
    (dict(S=0, out=None, q=None), B.PA_OK),
]


def base(**kw):
    a = dict(out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, mb=4, lens=FAKE, qsl=FAKE, S=2, chunk=16, max_len=64, Hq=8,
             Hkv=2, D=128, NB=16, bs=16, dt=B.PA_BF16, ks=1.0, vs=1.0)
    a.update(kw)
    return a


def attention(**kw):
    a = base(**kw)
    d = B.Fp4AttentionDesc()
    for field, key in (("out", "out"), ("q", "q"), ("k_cache", "kc"), ("v_cache", "vc"), ("block_table", "bt"), ("seq_lens", "lens"),
                       ("query_start_loc", "qsl"), ("max_blocks_per_seq", "mb"), ("num_seqs", "S"), ("max_chunk_len", "chunk"),
                       ("max_seq_len", "max_len"), ("num_q_heads", "Hq"), ("num_kv_heads", "Hkv"), ("head_dim", "D"),
                       ("num_blocks", "NB"), ("block_size", "bs"), ("dtype", "dt"), ("k_scale", "ks"), ("v_scale", "vs")):
        setattr(d, field, a[key])
    d.scale, d.workspace, d.workspace_bytes = 0.1, FAKE, 1 << 30
    return ctypes.byref(d)


@pytest.mark.parametrize("kw,expect", SHAPES)
def test_decode_fp4_refuses(kw, expect):
    assert B.load().pa_decode_fp4(attention(**kw), None) == expect


@pytest.mark.parametrize("kw,expect", SHAPES + [
    (dict(qsl=None), B.PA_ERR_INVALID_ARG),
    (dict(chunk=65), B.PA_ERR_INVALID_ARG),
    (dict(chunk=0, q=None), B.PA_OK),
    (dict(S=1 << 27, chunk=64), B.PA_ERR_UNSUPPORTED),
])
def test_prefill_fp4_refuses(kw, expect):
    assert B.load().pa_prefill_fp4(attention(**kw), None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), B.PA_ERR_INVALID_ARG),
    (dict(H=0), B.PA_ERR_INVALID_ARG),
    (dict(D=80), B.PA_ERR_UNSUPPORTED),
    (dict(bs=24), B.PA_ERR_UNSUPPORTED),
    (dict(dt=B.PA_FP4), B.PA_ERR_INVALID_ARG),
    (dict(ks=0.3), B.PA_ERR_INVALID_ARG),
    (dict(k=FAKE + 8), B.PA_ERR_INVALID_ARG),
    (dict(vc=None), B.PA_ERR_INVALID_ARG),
    (dict(slots=FAKE + 4), B.PA_ERR_INVALID_ARG),
    (dict(NB=1 << 30), B.PA_ERR_UNSUPPORTED),
    (dict(n=0, k=None), B.PA_OK),
])
def test_gather_fp4_refuses(kw, expect):
    a = dict(k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, slots=FAKE, n=3, H=2, D=128, NB=16, bs=16, ks=1.0, vs=1.0, dt=B.PA_BF16)
    a.update(kw)
    d = B.Fp4RowsDesc()
    for field, key in (("k_out", "k"), ("v_out", "v"), ("k_cache", "kc"), ("v_cache", "vc"), ("slots", "slots"), ("num_slots", "n"),
                       ("num_kv_heads", "H"), ("head_dim", "D"), ("num_blocks", "NB"), ("block_size", "bs"), ("dtype", "dt"),
                       ("k_scale", "ks"), ("v_scale", "vs")):
        setattr(d, field, a[key])
    assert B.load().pa_gather_fp4(ctypes.byref(d), None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(tokens=FAKE), B.PA_ERR_UNSUPPORTED),  # codes and scales of a token lie apart
    (dict(D=96), B.PA_ERR_UNSUPPORTED),
    (dict(bs=24), B.PA_ERR_UNSUPPORTED),
    (dict(pools=FAKE + 8), B.PA_ERR_INVALID_ARG),
    (dict(n=0), B.PA_OK),
])
def test_move_blocks_of_4_bit_pools_refuses(kw, expect):
    a = dict(pools=FAKE, H=1, D=64, NB=16, bs=16, n=3, tokens=None)
    a.update(kw)
    ptrs = (ctypes.c_void_p * 1)(a["pools"])
    assert B.load().pa_move_blocks(ptrs, 1, a["H"], a["D"], a["NB"], a["bs"], B.PA_FP4, FAKE, a["n"], a["tokens"], None,
                                   0, None, 0, None) == expect


def test_pool_size_for_memory():
    per = 2 * 4 * 16 * 72  # a block of one layer: K and V, 4 kv heads, 16 rows of 72 bytes
    assert B.pa_bm_num_blocks_for_memory(100 * per + 1, 1.0, 1, 4, 128, B.PA_FP4) == 100
    assert B.pa_bm_num_blocks_for_memory(100 * per, 0.5, 5, 4, 128, B.PA_FP4, 32) == 5
    assert B.pa_bm_num_blocks_for_memory(1 << 30, 1.0, 1, 4, 72, B.PA_FP4) == -1


@pytest.mark.parametrize("name,desc,pack", [("pa_rotate", B.RotateDesc, B._pack_rotate),
                                            ("pa_fp4_attention", B.Fp4AttentionDesc, B._pack_attention),
                                            ("pa_fp4_rows", B.Fp4RowsDesc, B._pack_rows)])
def test_descriptors_match_the_header(tmp_path, name, desc, pack):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("needs gcc")
    names = [f[0] for f in desc._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "pa.h"\nint main(void) {\n'
                   f'  printf("%zu\\n", sizeof({name}));\n' +
                   "".join(f'  printf("%zu\\n", offsetof({name}, {n}));\n' for n in names) + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(desc)] + [getattr(desc, n).offset for n in names]
    # the packed form that the binding passes: every field in its place, the same size
    values = list(range(1, len(names) + 1))
    packed = pack(*values)
    assert len(packed) == ctypes.sizeof(desc)
    d = desc.from_buffer_copy(packed)
    assert [getattr(d, n) for n in names] == values


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    t = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    k = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    pool = torch.zeros(B.fp4_pool_shape(4, 2, 16, 128), dtype=torch.uint8)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    i64, cs = torch.zeros(2, dtype=torch.int64), torch.zeros(9, 128)
    with pytest.raises(ValueError):
        B.pa_rotate_and_cache(t, t, k, k, i64, cs, pool, pool, i64)
    for q_out, q in ((None, t), (t, None)):
        with pytest.raises(ValueError, match="go together"):
            B.pa_rotate_and_cache(q_out, q, k, k, i64, cs, pool, pool, i64)
    with pytest.raises(ValueError):
        B.pa_decode_fp4(t, t, pool, pool, table, lens, 64, 0.1)
    with pytest.raises(ValueError):
        B.pa_prefill_fp4(t, t, pool, pool, table, lens, lens, 1, 64, 0.1)
    with pytest.raises(ValueError):
        B.pa_gather_fp4(k, k, pool, pool, i64)
    with pytest.raises(ValueError):
        B.PoolList([pool])


def test_definition_of_the_codes():
    # every scale that e4m3 has comes back from its own value; ties go to the even one
    b = np.arange(127, dtype=np.uint8)
    v = R.e4m3_values(b)
    assert (R.e4m3_bytes(v) == b).all()
    mid = (v[:-1] + v[1:]) / 2
    assert (R.e4m3_bytes(mid) == np.where(b[:-1] % 2 == 0, b[:-1], b[1:])).all()
    assert R.e4m3_bytes(np.array([1e9]))[0] == 126
    # the 16 codes, and ties between them, in a group whose scale is 1
    x = np.array([6.0, -6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, 0.2, 0.3, 4.9, 5.1, 0.0])
    codes, scales = R.quantise(x[None])
    assert R.e4m3_values(scales)[0, 0] == 1.0
    assert codes[0].tolist() == [7, 15, 0, 2, 2, 4, 4, 6, 6, 8, 10, 0, 1, 6, 7, 0]
    # a pool's values are themselves when stored again
    x = np.random.default_rng(0).standard_normal((2, 3, 32, 64))
    pool = R.to_pool(x, 0.25)
    again = R.from_pool(pool, 0.25)
    assert np.abs(again - x).max() < 0.6
    assert (R.from_pool(R.to_pool(again, 0.25), 0.25) == again).all()

"""Attention over 4-bit pools in the forms that only large batches take: decode in several launches, prefill whose CTAs are
ordered sequence by sequence, prefill of more sequences than are ordered at all. Tolerances: fp4_reference.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import fp4_reference as R  # noqa: E402
from paged_kv_cache_238_gb300 import binding as B  # noqa: E402
from test_fp4_gpu import Device, check  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_errors_left():
    B.pa_get_device_errors()
    yield
    assert B.pa_get_device_errors() == 0


def ragged(seed, n, lo, hi):
    x = np.random.default_rng(seed).integers(lo, hi + 1, n)
    x[n // 2] = hi
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,H_q,H_kv,D,BS", [(1100, 4, 2, 64, 16),    # more sequences than a launch takes
                                             (600, 32, 32, 64, 32),   # more segments than it counts
                                             (1030, 20, 1, 128, 16)])
def test_decode_in_several_launches(dtype, S, H_q, H_kv, D, BS):
    """The launches share a workspace; a sequence of each is cut between CTAs. Equal bits when it is used again."""
    lens = ragged(70, S, 0, 40)
    lens[3], lens[-2] = 2500, 1300
    d = check(R.Case(71, lens, H_q, H_kv, D, BS, dtype, k_scale=0.5, v_scale=2.0))
    first = d.got()
    d.out.fill_(7.0)
    d.run()
    assert (d.got() == first).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,chunk,prior,H_q,H_kv,D", [(50, 60, 600, 32, 32, 64),    # bf16: one query tile a CTA
                                                      (50, 40, 500, 32, 32, 128),
                                                      (20, 260, 600, 32, 32, 64),   # two
                                                      (20, 260, 600, 32, 32, 128),
                                                      (80, 70, 500, 48, 16, 64)])
def test_prefill_sequence_by_sequence(dtype, S, chunk, prior, H_q, H_kv, D):
    """More CTAs than are ordered pair by pair; key lists longer than the rings of K and V; chunks of no and of one row."""
    chunks = ragged(72, S, 0, chunk)
    chunks[1], chunks[2] = 0, 1
    check(R.Case(73, chunks + ragged(74, S, 0, prior), H_q, H_kv, D, 16, dtype, chunks=chunks))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,chunk,prior,H_q,H_kv,D", [(300, 7, 40, 4, 2, 64), (300, 140, 300, 4, 1, 128), (257, 3, 900, 8, 1, 64)])
def test_prefill_of_many_sequences(dtype, S, chunk, prior, H_q, H_kv, D):
    chunks = ragged(75, S, 0, chunk)
    lens = chunks + ragged(76, S, 0, prior)
    chunks[5] = lens[5] = 0
    check(R.Case(77, lens, H_q, H_kv, D, 64, dtype, chunks=chunks))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("chunks", [True, False])
def test_more_sequences_than_a_grid_has_rows(dtype, chunks):
    """Sequences of one key or none: an output is the key's V, or zero (decode), or not there (prefill)."""
    n, block = np.arange(66000), 1 + np.arange(66000) % 97
    lens = (n % 3 != 0).astype(np.int32)
    c = R.Case(78, [16] * 97, 2, 2, 64, 16, dtype)  # 97 blocks of keys, which the sequences share
    held = c.values[1][:, :, 0]  # [block][head][64]: of each block's first key
    q = np.random.default_rng(79).standard_normal((len(n), 2, 64))
    rows = lens > 0
    c.lens, c.table, c.decode, c.chunks = lens, c.table[:, :1][block - 1], not chunks, lens
    c.qsl = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    if chunks:
        q = q[rows]
    c.q = R.W.f32_to_bf16_bits(q.astype(np.float32)) if dtype == "bf16" else q.astype(np.float32)
    d = Device(c)
    d.run()
    want = held[c.table[:, 0]] * lens[:, None, None]
    want = want[rows] if chunks else want
    # one weight over itself, as the tolerance has it for one key without an error of its score; 6 significant bits are bf16's own
    tol = (2.0 ** -20 + (4 * 17 + 1) * R.U) * np.abs(want) if dtype == "f32" else 0.0
    assert (np.abs(d.got() - want) <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_more_heads_than_a_tile_has_rows_on_long_contexts(dtype, D):
    """On the CUDA cores, with the keys in partitions."""
    check(R.Case(80, [3000, 700], 130, 1, D, 32, dtype, chunks=[1, 1], k_scale=0.25, v_scale=4.0))

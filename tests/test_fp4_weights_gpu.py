"""Attention over 4-bit pools where what is small next to a row's largest weight, or to a query's largest element, decides
the output. The bounds are those of fp4_reference.py for fp32 queries, whose halves lie within fp16's range in the same
way; bf16 queries add the rounding of the weights to fp16:

  * the largest weight is 2^7 at least, and fp16's numbers below 2^-14 are 2^-24 apart: a weight w of a sum l is off by
    max(2^-11 w, 2^-25), 2^-25 being 2^-32 l at most: 2^-11 A + n 2^-32 max |v|;
  * a query's largest magnitude lies in [2^14, 2^15): 8 bits fit above 2^-14, and an element below is off by 2^-25 at
    most, 2^-39 of the largest magnitude.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import fp4_reference as R  # noqa: E402
from paged_kv_cache_238_gb300 import binding as B  # noqa: E402
from test_fp4_gpu import Device  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_errors_left():
    B.pa_get_device_errors()
    yield
    assert B.pa_get_device_errors() == 0


def bits(x, dtype):
    x = np.ascontiguousarray(x, dtype=np.float32)
    return R.W.f32_to_bf16_bits(x) if dtype == "bf16" else x


def check(c):
    dtype, values = c.dtype, c.values
    c.dtype = "f32"
    ref, err = c.reference()
    if dtype == "bf16":
        c.values = [values[0], np.abs(values[1])]
        err = err + 2.0 ** -11 * c.reference()[0]
        err = err + 2.0 ** -8 * (np.abs(ref) + err)
    c.dtype, c.values = dtype, values
    d = Device(c)
    d.run()
    bad = np.abs(d.got() - ref) > err
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, worst {np.max(np.abs(d.got() - ref) / err):.2f} x"


def sinks(dtype, S, chunk, H, L=2000):
    """S sequences over the same L keys: the first scores 10 to 27 log2 units above the others, all alike, and its V is zero,
    so that an output is the others' mean times their share of the weights, 0.7 to 1.5e-5."""
    c = R.Case(40, [L], H, H, 64, 16, dtype, chunks=None if chunk is None else [chunk])
    rng, ids = np.random.default_rng(41), c.table[0]
    k, v = np.zeros((L // 16, H, 16, 64)), np.abs(rng.standard_normal((L // 16, H, 16, 64)))
    k[0, :, 0, :16], v[0, :, 0] = 6.0, 0.0
    for i, x in enumerate((k, v)):
        c.pools[i][ids] = R.to_pool(x)
        c.values[i] = R.from_pool(c.pools[i])
    rows = S * (1 if chunk is None else chunk)
    q = np.zeros((rows, H, 64))
    q[..., :16] = rng.permutation(np.linspace(10, 27, rows * H)).reshape(rows, H, 1) / (np.log2(np.e) * c.scale * 96)
    c.q = bits(q, dtype)
    c.lens, c.chunks = np.repeat(c.lens, S), np.repeat(c.chunks, S)
    c.qsl, c.table = np.concatenate([[0], np.cumsum(c.chunks)]).astype(np.int32), np.repeat(c.table, S, axis=0)
    whole = R.Case.keys

    class Shared(R.Case):
        def keys(self, s):  # every sequence's are the first one's
            if getattr(self, "of", None) is not self.values:
                self.of, self.held = self.values, whole(self, 0)
            return self.held

    c.__class__ = Shared
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,chunk,H", [(160, None, 16),  # a sequence's keys to a warp
                                       (170, 8, 1), (160, 130, 1)])  # one query tile and two, lists that are not split
def test_many_weights_far_below_the_largest(dtype, S, chunk, H):
    check(sinks(dtype, S, chunk, H))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("chunks", [None, [150, 40, 3]])
@pytest.mark.parametrize("D", [64, 128])
def test_elements_of_q_far_below_the_largest(dtype, chunks, D):
    """The largest element of each row meets keys that are 0 in its dim; the others, 2^-24 of it, decide the scores."""
    c = R.Case(42, [300, 40, 17], 8, 2, D, 16, dtype, chunks=chunks)
    for b in {int(x) for x in c.table.ravel()} - {0}:  # code 0 in dim 0 of every key
        c.pools[0][b].reshape(2, 9 * D)[:, :8 * D].reshape(2, 16, D // 2)[..., 0] &= 0xF0
    c.values[0] = R.from_pool(c.pools[0])
    q = R.W.as_f64(c.q) * 2.0 ** -24
    q[..., 0] = 1.5
    c.q = bits(q, dtype)
    c.scale *= 2.0 ** 24
    check(c)

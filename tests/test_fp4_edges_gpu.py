"""Attention over 4-bit pools at the ends of its arguments' ranges."""
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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale,k_scale", [(-0.0, 1.0), (-1e-38, 2.0 ** -24), (1e-38, 2.0 ** -24)])
@pytest.mark.parametrize("chunks", [None, [40, 3]])
def test_scales_that_vanish(dtype, scale, k_scale, chunks):
    """A scale of zero of either sign, given or left by the product with the pool's factor: uniform weights."""
    c = R.Case(50, [77, 9], 8, 2, 64, 16, dtype, chunks=chunks, k_scale=k_scale)
    c.scale = scale
    check(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H_q", [1, 8])
def test_the_largest_chunk_bound(dtype, H_q):
    """A bound of the chunk's length of 2^31 - 1, and a table for as many keys: the chunks themselves are short."""
    c = R.Case(51, [300], H_q, 1, 64, 128, dtype, chunks=[150])
    bound = 2 ** 31 - 1
    d = Device(c, max_len=bound, max_chunk=bound)
    wide = torch.zeros(1, 2 ** 24, dtype=torch.int32, device="cuda")
    wide[:, :d.table.shape[1]] = d.table
    d.table = wide
    d.run()
    ref, tol = c.reference()
    assert (np.abs(d.got() - ref) <= tol).all()


def test_numbers_that_no_field_holds():
    """Bounds past 32 bits and factors that are no numbers are refused as other bad arguments are."""
    for chunks in (None, [20, 3]):
        c = R.Case(52, [20, 5], 8, 2, 64, 16, chunks=chunks)
        d = Device(c)
        d.max_len = 2 ** 31
        with pytest.raises(ValueError):
            d.run()
        d.max_len, c.v_scale = 20, "1"
        with pytest.raises(ValueError):
            d.run()
        assert (d.got() == 7.0).all()
    rows, pool = torch.zeros(1, 2, 64, device="cuda"), torch.zeros(B.fp4_pool_shape(2, 2, 16, 64), dtype=torch.uint8, device="cuda")
    one = torch.zeros(1, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        B.pa_gather_fp4(rows, rows.clone(), pool, pool, one, k_scale=None)
    with pytest.raises(ValueError):
        B.pa_rotate_and_cache(None, None, rows, rows, one, torch.zeros(1, 64, device="cuda"), pool, pool.clone(), one, k_scale=None)

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

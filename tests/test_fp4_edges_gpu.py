"""Attention over 4-bit pools at the ends of its arguments' ranges."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import fp4_reference as R  # noqa: E402
from paged_kv_cache_238_gb300 import binding as B  # noqa: E402
from test_fp4_gpu import check  # noqa: E402

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

"""The bounded waits of attention over 4-bit pools, made to run out on purpose (pa_debug_set_wait_drill), as
test_wait_drill_gpu.py does for the other calls: one barrier phase waits for 16 bytes that nothing brings, and nothing that the
kernel would abandon is in flight. The wait gives up after the shortened limit, the call ends with
PA_DEVERR_WAIT_TIMEOUT, and the same call without the drill, its workspace zeroed, is right again."""
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import fp4_reference as R  # noqa: E402
from paged_kv_cache_238_gb300 import binding as B  # noqa: E402
from test_fp4_gpu import Device  # noqa: E402

pytestmark = pytest.mark.gpu

LIMIT_NS = 2_000_000  # 2 ms instead of 1 s while a drill is on


@pytest.fixture(autouse=True)
def drill_off_around_each_test():
    B.pa_debug_set_wait_drill(B.PA_DRILL_OFF)
    B.pa_get_device_errors(clear=True)
    yield
    B.pa_debug_set_wait_drill(B.PA_DRILL_OFF)
    assert B.pa_get_device_errors(clear=True) == 0


def drilled(kind, c):
    ref, tol = c.reference()
    d = Device(c)
    B.pa_debug_set_wait_drill(kind, LIMIT_NS)
    try:
        t0 = time.perf_counter()
        d.run()
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
    finally:
        B.pa_debug_set_wait_drill(B.PA_DRILL_OFF)
    errors = B.pa_get_device_errors(clear=True)
    assert errors == B.PA_DEVERR_WAIT_TIMEOUT, f"errors {errors:#x}"
    assert took < 0.5, f"the drilled call took {took:.3f} s: the shortened limit was not used"
    if d.ws is not None:
        d.ws.zero_()
    d.out.fill_(7.0)
    d.run()
    assert (np.abs(d.got() - ref) <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,H_q,H_kv,D", [([300, 17, 64, 1000, 5, 2048], 8, 2, 128),
                                             ([700], 16, 1, 64),         # more than 8 heads a segment
                                             ([3] * 40, 4, 4, 64)])      # segments of one page
def test_decode_wait_runs_out(dtype, lens, H_q, H_kv, D):
    drilled(B.PA_DRILL_DECODE_STAGE, R.Case(60, lens, H_q, H_kv, D, 16, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("chunks,lens,H_q,H_kv,D", [([100, 1, 257], [100, 300, 700], 8, 2, 128),
                                                    ([100, 1, 257], [100, 300, 1700], 4, 4, 64),
                                                    ([20], [20], 4, 4, 64),             # one key tile
                                                    ([9], [4000], 16, 2, 128),          # a list cut into runs
                                                    ([300] * 90, [300] * 90, 8, 8, 64)])  # sequence by sequence
def test_prefill_wait_runs_out(dtype, chunks, lens, H_q, H_kv, D):
    drilled(B.PA_DRILL_PREFILL_K_TILE, R.Case(61, lens, H_q, H_kv, D, 16, dtype, chunks=chunks))


def test_each_drill_leaves_the_other_call_alone():
    for kind, chunks in ((B.PA_DRILL_DECODE_STAGE, [100, 3]), (B.PA_DRILL_PREFILL_K_TILE, None)):
        c = R.Case(62, [300, 40], 8, 2, 128, 16, "bf16", chunks=chunks)
        ref, tol = c.reference()
        d = Device(c)
        B.pa_debug_set_wait_drill(kind, LIMIT_NS)
        d.run()
        assert (np.abs(d.got() - ref) <= tol).all()

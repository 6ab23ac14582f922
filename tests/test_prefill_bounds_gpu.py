"""Prefill calls whose chunk bound is the largest that the arguments allow: the number of query tiles that it gives fits 32
bits, and the short chunks under it come out right."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import oracle  # noqa: E402
from helpers import DeviceWorkload, assert_close, to_f64  # noqa: E402
from paged_kv_cache_238_gb300 import binding as B  # noqa: E402
from paged_kv_cache_238_gb300 import workloads as W  # noqa: E402

pytestmark = pytest.mark.gpu

BOUND = 2 ** 31 - 1


@pytest.mark.parametrize("call,dtype,D", [("chunk", "bf16", 128),   # tensor cores
                                          ("scored", "bf16", 64),
                                          ("scored", "f32", 64)])  # CUDA cores
def test_the_largest_chunk_bound(call, dtype, D):
    wl = W.build_mixed(78, prior_lens=[100], chunk_lens=[150], decode_lens=[], H_q=1, H_kv=1, D=D, num_blocks=20,
                       dtype=dtype, pad_multiple=64)
    dw = DeviceWorkload(wl)
    B.pa_reshape_and_cache(dw.k_new, dw.v_new, dw.k_cache, dw.v_cache, dw.slot_mapping)
    table = torch.zeros(1, 2 ** 27, dtype=torch.int32, device="cuda")
    table[:, :dw.block_table_prefill.shape[1]] = dw.block_table_prefill
    args = (dw.out_prefill, dw.q_prefill, dw.k_cache, dw.v_cache, table, dw.seq_lens_prefill, dw.query_start_loc, BOUND, BOUND,
            wl.scale)
    if call == "chunk":
        B.pa_prefill_chunk(*args)
    else:
        n = B.pa_prefill_scored_workspace_size(1, BOUND, 1, 1, D, BOUND, dw.tdtype)
        B.pa_prefill_scored(*args, None, torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None)
    torch.cuda.synchronize()
    assert B.pa_get_device_errors(clear=True) == 0
    kc, vc = dw.host_pool_after_writes()
    ref = oracle.attention(wl.q_prefill, kc, vc, wl.block_table_prefill, wl.seq_lens_prefill, wl.scale,
                           query_start_loc=wl.query_start_loc)
    assert_close(to_f64(dw.out_prefill), ref, dtype, call)

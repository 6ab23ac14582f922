"""Barriers in shared memory are initialised once: initialising one that is in use is undefined. (A
second pass over some of them, to change their counts, is what this finds.) CPU only."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parent.parent / "paged_kv_cache_238_gb300" / "csrc"


@pytest.mark.parametrize("name", ["prefill.cu", "prefill_scored.cu", "decode_balanced.cu", "decode_scored.cu"])
def test_one_place_initialises_a_kernels_barriers(name):
    source = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    assert len(re.findall(r"\bmbar_init\s*\(", source)) == 1

"""Counts next to 2^31, past what the step operators' 32-bit loops can take, are
refused before any CUDA call (this machine may have no GPU)."""
from __future__ import annotations

import pytest

from paged_kv_cache_445_b200 import _binding as b

F = 4096  # a stand-in pointer
L = b._lib


@pytest.mark.parametrize("n", [2**31 - 65536, 2**31 - 1])
def test_counts_next_to_the_end_of_int32(n):
    assert L.pa_step_slots(F, F, F, F, F, F, 8, F, F, F, n, 10, 16, F, F, F, 9, None, None) == b.PA_ERR_SHAPE
    assert L.pa_prefill_chunk_int4(F, F, F, F, F, F, 4, F, n, 9, 8, 2, 128, 16, 10, 0.1, F, 1 << 30, None,
                                   None) == b.PA_ERR_SHAPE
    assert L.pa_decode_int4(F, F, F, F, F, 4, F, n, 8, 2, 128, 16, 10, 0.1, F, 1 << 30, None, None) == b.PA_ERR_SHAPE
    for bf16 in (0, 1):
        assert L.pa_accept_drafts(F, F, F, n, F, n, bf16, F, F, F, 3, 9, n, F, F, None, None) == b.PA_ERR_SHAPE

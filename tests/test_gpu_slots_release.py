"""A bad block ID in a sequence that gives its blocks up is reported by that step."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import step_reference as ref
from tests.gpu_helpers import load_library
from tests.test_gpu_slots import run, state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    load_library()


@pytest.mark.parametrize("bad", [-1, -2**31, 2**31 - 1, "end"])
@pytest.mark.parametrize("b,max_tokens", [(5, 20), (1500, 3000), (1500, 40000)])
def test_a_bad_id_given_up_is_reported_and_queued(b, max_tokens, bad):
    """60 tokens in four blocks, a fifth held: the bad entry among those given up, or among those kept."""
    rng = np.random.default_rng(b)
    ctx, held, tables, ring, st = state(rng, b, 16, 20, b * 12, 100)
    s = b - 2
    ctx[s], held[s] = 60, 5
    new = np.zeros(b, np.int32)
    for given_up, entry, status in ((60, 2, ref.RANGE), (20, 3, ref.RANGE), (20, 2, 0), (5, 4, ref.RANGE), (5, 3, 0)):
        new[s] = -given_up
        tables[s, :5] = [1, 2, 3, 4, 5]
        tables[s, entry] = len(ring) if bad == "end" else bad
        want, _ = ref.step_slots(new, ctx, held, tables, ring, st, 16, max_tokens)
        got, bits = run(new, ctx, held, tables, ring, st, 16, max_tokens)
        for k in want:
            assert np.array_equal(got[k], want[k]), k
        assert bits == status, (given_up, entry)

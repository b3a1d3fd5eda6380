"""Lengths that leave a sequence without keys in the 4-bit attention: which status they set."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import step_reference as ref
from tests.gpu_helpers import load_library
from tests.test_gpu_int4 import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    load_library()


@pytest.mark.parametrize("length,status", [(0, 0), (-1, 0), (-7, 0), (-2**31, 0), (65, ref.RANGE), (2**31 - 1, ref.RANGE)])
@pytest.mark.parametrize("varlen", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_no_keys_give_zeros_and_one_status(d, varlen, length, status):
    """64 keys fit the table; the sequences beside it keep their results."""
    b = Batch([40, 64, 33], [1, 2, 1] if varlen else [1] * 3, 8, 2, d, 16, seed=40)
    assert b.run(varlen) == 0
    want = b.out.clone()
    b.ctx = np.array([40, length, 33])
    out = torch.full_like(b.out, -5.0)
    assert b.run(varlen, out) == status
    assert (out[1:-1] == 0).all()
    b.status.zero_()
    b.ctx = np.array([40, 64, 33])
    keep = b.run(varlen, b.out)
    assert keep == 0 and torch.equal(b.out, want)
    # the keys are cut at other places then: each run is within the attention tests' bound, 2^-8 |out| + 2^-9 max |v|
    err = (out[[0, -1]].float() - want[[0, -1]].float()).abs()
    assert (err <= 2.0**-7 * want[[0, -1]].float().abs() + 2.0**-8 * np.nanmax(np.abs(b.kv[1]))).all()

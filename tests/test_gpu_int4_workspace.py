"""One workspace for calls on the bf16, FP8 and 4-bit caches in turn: each gives the
bits that it gives on a fresh workspace."""
from __future__ import annotations

import pytest
import torch

from tests.gpu_helpers import load_library
from tests.test_gpu_int4 import Batch
from tests.test_gpu_workspace_reuse import BATCHES, KEYS, ROWS, SHAPES, Calls

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    load_library()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"Hq{s[0]}-Hkv{s[1]}-d{s[2]}-bs{s[3]}")
def test_calls_on_all_caches_share_a_workspace(shape):
    """4-bit calls whose items are cut between CTAs, between warps and not at all, between those of the other kinds."""
    import paged_kv_cache_445_b200 as pa
    hq, hkv, d, bs = shape
    ws = pa.make_workspace(ROWS, hq, hkv, d, KEYS // bs, bs)
    assert ws.numel() >= pa.pa_int4_workspace_bytes(hq, hkv, d)
    others = [Calls(shape, i, b) for i, b in enumerate(BATCHES[:6])]
    fours = [(Batch(ctx, rows, *shape, seed=60 + i), varlen) for i, (ctx, rows, varlen) in enumerate([
        ([9000], [1], False), ([700, 33, 2000], [1] * 3, False), ([3000, 50, 800], [6, 1, 40], True),
        ([60] * 400, [1] * 400, False), ([5000, 4000], [1, 1], False), ([130], [130], True)])]
    fresh = []
    for b, varlen in fours:
        b.ws = torch.zeros_like(ws)
        assert b.run(varlen) == 0
        b.check()
        fresh.append(b.out.clone())
        b.ws = ws
    kinds = [[k for k in c.kinds() if k != "cascade"] for c in others]
    want = [{k: c.run(k, torch.zeros_like(ws)) for k in ks} for c, ks in zip(others, kinds)]
    for turn in range(3):
        for i, (b, varlen) in enumerate(fours):
            out = torch.full_like(b.out, -5.0)
            assert b.run(varlen, out) == 0
            assert torch.equal(out, fresh[i]), (turn, i)
            c = (i + turn) % len(others)
            for k in kinds[c]:
                assert torch.equal(others[c].run(k, ws), want[c][k]), (turn, c, k)

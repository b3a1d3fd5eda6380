"""One workspace for calls of every size and kind, one after another, as an engine
makes them: each gives the bits that it gives on a fresh workspace."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_kv_cache_445_b200 import workloads
from tests.gpu_helpers import DeviceStep, i32, load_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    load_library()


ROWS, KEYS = 1000, 2400  # what the shared workspace is made for
# stored tokens and new ones of each sequence, in calls that grow and shrink
BATCHES = [
    ([2300], [1]),
    ([int(x) for x in np.linspace(3, 700, 120)], [1] * 120),
    ([1200, 90, 15, 700], [400, 1, 3, 150]),
    ([5], [1]),
    ([300 + 7 * i for i in range(40)], [4] * 40),
    ([0], [900]),
    ([2000, 2100], [1, 1]),
    ([40] * 300, [1] * 300),
    ([10, 600], [2, 500]),
    ([1500] * 3, [1] * 3),
]
SHAPES = [(16, 2, 128, 16), (8, 2, 64, 16), (24, 4, 256, 32), (12, 2, 128, 32)]


class Calls:
    """Every attention call that takes a batch, on a given workspace."""

    def __init__(self, shape, i, batch):
        import paged_kv_cache_445_b200 as pa
        self.pa = pa
        hq, hkv, d, bs = shape
        self.w = workloads.custom(*batch, hq, hkv, d, bs, seed=50 + i)
        self.ds = DeviceStep(self.w)
        self.ds.append()
        if d != 64:
            kc, vc, self.ks, self.vs = workloads.fp8_caches(self.w, seed=i)
            self.fp8 = torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda()

    def kinds(self):
        one = self.w.is_decode
        return ["bf16"] + (["fp8"] if self.w.head_dim != 64 else []) + (["cascade"] if one and int(self.w.context_lens[0]) > 64 else [])

    def run(self, kind, ws):
        d, w, pa = self.ds, self.w, self.pa
        out = torch.full_like(d.q, -5.0)
        if kind == "bf16" and w.is_decode:
            pa.pa_decode(out, d.q, d.k_cache, d.v_cache, d.block_tables, d.context_lens, w.scale, ws, d.status)
        elif kind == "bf16":
            pa.pa_prefill_chunk(out, d.q, d.query_start, d.k_cache, d.v_cache, d.block_tables, d.context_lens, w.scale,
                                ws, d.status)
        elif kind == "fp8":
            pa.pa_prefill_chunk_fp8(out, d.q, d.query_start, *self.fp8, d.block_tables, d.context_lens, w.scale, self.ks,
                                    self.vs, ws, d.status)
        else:  # a group of one sequence, its first 64 tokens as the prefix
            pa.pa_decode_cascade(out, d.q, d.k_cache, d.v_cache, d.block_tables, d.context_lens, w.scale, i32([0, 1]),
                                 i32([64]), ws, dev_status=d.status)
        torch.cuda.synchronize()
        assert int(d.status.item()) == 0, kind
        return out


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"Hq{s[0]}-Hkv{s[1]}-d{s[2]}-bs{s[3]}")
def test_calls_of_all_sizes_share_a_workspace(shape):
    import paged_kv_cache_445_b200 as pa
    hq, hkv, d, bs = shape
    ws = pa.make_cascade_workspace(ROWS, hq, hkv, d, KEYS // bs, bs)
    calls = [Calls(shape, i, b) for i, b in enumerate(BATCHES)]
    fresh = {}
    for i, c in enumerate(calls):
        for kind in c.kinds():
            fresh[i, kind] = c.run(kind, torch.zeros_like(ws))
    for order in (range(len(calls)), reversed(range(len(calls)))):
        for i in order:
            for kind in calls[i].kinds():
                assert torch.equal(calls[i].run(kind, ws), fresh[i, kind]), (i, kind)

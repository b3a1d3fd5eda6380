"""Attention launched straight behind the kernel that wrote its lengths and row
offsets.  Its prologue reads them before it waits for that kernel's stores, so
these have to be fenced on every path: the results are those of the same calls
with a synchronisation between them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.gpu_helpers import i32, load_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    load_library()


def rand(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("b", [1500, 300])
def test_varlen_attention_behind_the_slots(b):
    """Lengths and offsets go to other buffers than they come from, the rows fill several CTAs."""
    import paged_kv_cache_445_b200 as pa
    rng = np.random.default_rng(b)
    bs, width, hq, hkv, d, t = 16, 8, 4, 1, 64, 6000
    nb = b * width
    kc, vc, q = rand(rng, nb, hkv, bs, d), rand(rng, nb, hkv, bs, d), rand(rng, t, hq, d)
    ctx = rng.integers(0, 100, b)
    held = -(-ctx // bs)
    tables = i32(rng.permutation(nb).reshape(b, width))
    free = i32(rng.permutation(nb))
    ws = pa.make_workspace(t, hq, hkv, d, width, bs)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx_in, held_in, state = i32(ctx), i32(held), i32([0, nb])
    ctx_out, held_out, state_out = torch.zeros_like(ctx_in), torch.zeros_like(held_in), torch.zeros_like(state)
    qs = torch.zeros(b + 1, dtype=torch.int32, device="cuda")
    pos, slots = (torch.zeros(t, dtype=torch.int32, device="cuda") for _ in range(2))
    out = torch.zeros_like(q)
    for i in range(12):
        new = i32(rng.integers(0, 4, b))
        results = []
        for wait in (True, False):
            for x in (ctx_out, qs, out):
                x.zero_()
            pa.pa_step_slots(new, ctx_in, held_in, tables, free, state, bs, qs, pos, slots, context_lens_out=ctx_out,
                             blocks_held_out=held_out, free_state_out=state_out, dev_status=status)
            if wait:
                torch.cuda.synchronize()
            pa.pa_prefill_chunk(out, q, qs, kc, vc, tables, ctx_out, d**-0.5, ws, status)
            torch.cuda.synchronize()
            results.append((out.clone(), qs.clone(), ctx_out.clone()))
        assert int(status.item()) == 0
        assert all(torch.equal(x, y) for x, y in zip(*results)), i
        assert int(results[0][1][-1]) == int(new.sum()) and torch.equal(results[0][2], ctx_in + new)

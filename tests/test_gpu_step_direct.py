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


def test_decode_behind_the_verification():
    """Sequences with no rows, with bad offsets and with refused drafts write their lengths on three paths."""
    import paged_kv_cache_445_b200 as pa
    rng = np.random.default_rng(7)
    b, bs, width, hq, hkv, d, vocab = 96, 16, 8, 8, 2, 128, 300
    nb = b * width
    kc, vc, q = rand(rng, nb, hkv, bs, d), rand(rng, nb, hkv, bs, d), rand(rng, b, hq, d)
    tables = i32(rng.permutation(nb).reshape(b, width))
    rows = np.where(np.arange(b) % 3 == 0, 0, rng.integers(1, 5, b))
    start = np.concatenate([[0], np.cumsum(rows)])
    t = int(start[-1])
    start[-1] += 5  # the last sequence's rows end past the buffer: it keeps its length, with the RANGE bit
    ctx = rng.integers(10, width * bs, b)
    target, draft = (torch.from_numpy(rng.random((t, vocab)).astype(np.float32)).cuda() for _ in range(2))
    tokens, uniforms = i32(rng.integers(0, vocab, t)), torch.from_numpy(rng.random(t).astype(np.float32)).cuda()
    ctx_in, qs = i32(ctx), i32(start)
    ctx_out, accepted = torch.zeros_like(ctx_in), torch.zeros_like(ctx_in)
    out_tokens = torch.zeros(t, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    ws = pa.make_workspace(b, hq, hkv, d, width, bs)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for i in range(12):
        results = []
        for wait in (True, False):
            for x in (ctx_out, out):
                x.zero_()
            pa.pa_accept_drafts(out_tokens, accepted, target, draft, tokens, qs, uniforms, context_lens=ctx_in,
                                context_lens_out=ctx_out, dev_status=status)
            if wait:
                torch.cuda.synchronize()
            pa.pa_decode(out, q, kc, vc, tables, ctx_out, d**-0.5, ws, None)
            torch.cuda.synchronize()
            results.append((out.clone(), ctx_out.clone()))
        assert int(status.item()) == pa.status_bit(-5)
        assert all(torch.equal(x, y) for x, y in zip(*results)), i
        lost = np.where(rows > 0, rows - 1, 0)
        lost[-1] = 0
        kept = np.where(np.arange(b) == b - 1, 0, accepted.cpu().numpy())
        assert np.array_equal(results[0][1].cpu().numpy(), ctx - np.where(rows > 0, lost - kept, 0))

"""Tables, positions and slots of a step built on the GPU (pa_step_slots)
against a sequential walk over the batch and against the host allocator."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_kv_cache_445_b200.allocator import BlockAllocator
from tests import step_reference as ref
from tests.gpu_helpers import i32, load_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    load_library()


def state(rng, b, bs, width, nb, max_ctx, spare=0.3):
    """A consistent state: lengths, held blocks (some spare), tables, a wrapped queue."""
    ctx = rng.integers(0, max_ctx + 1, b)
    held = np.minimum(-(-ctx // bs) + (rng.random(b) < spare), width)
    ids = rng.permutation(nb)
    tables = np.full((b, width), -1, np.int64)
    at = 0
    for s in range(b):
        tables[s, :held[s]] = ids[at:at + held[s]]
        at += held[s]
    assert at <= nb
    head = int(rng.integers(0, nb))
    ring = np.full(nb, -7, np.int64)
    for j, x in enumerate(ids[at:]):
        ring[(head + j) % nb] = x
    to = lambda a: np.ascontiguousarray(a, dtype=np.int32)  # noqa: E731
    return to(ctx), to(held), to(tables), to(ring), to([head, nb - at])


def run(new, ctx, held, tables, ring, st, bs, max_tokens, in_place=False):
    import paged_kv_cache_445_b200 as pa
    d = dict(new=i32(new), ctx=i32(ctx), held=i32(held), tables=i32(tables), ring=i32(ring), state=i32(st))
    b = len(new)
    qs = torch.full((b + 1,), -9, dtype=torch.int32, device="cuda")
    pos = torch.full((max_tokens,), -9, dtype=torch.int32, device="cuda")
    slots = torch.full((max_tokens,), -9, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = {} if in_place else dict(context_lens_out=torch.full_like(d["ctx"], -9),
                                    blocks_held_out=torch.full_like(d["held"], -9),
                                    free_state_out=torch.full_like(d["state"], -9))
    pa.pa_step_slots(d["new"], d["ctx"], d["held"], d["tables"], d["ring"], d["state"], bs, qs, pos, slots,
                     dev_status=status, **outs)
    torch.cuda.synchronize()
    if not in_place:
        for k, v in (("ctx", ctx), ("held", held), ("state", st)):
            assert np.array_equal(d[k].cpu().numpy(), v), f"{k} was changed"
        d.update(ctx=outs["context_lens_out"], held=outs["blocks_held_out"], state=outs["free_state_out"])
    got = dict(query_start=qs, positions=pos, slots=slots, tables=d["tables"], ring=d["ring"], ctx=d["ctx"],
               held=d["held"], state=d["state"])
    return {k: v.cpu().numpy() for k, v in got.items()}, int(status.item())


def check(new, ctx, held, tables, ring, st, bs, max_tokens, in_place=False):
    want, bits = ref.step_slots(new, ctx, held, tables, ring, st, bs, max_tokens)
    got, status = run(new, ctx, held, tables, ring, st, bs, max_tokens, in_place)
    for k in want:
        assert np.array_equal(got[k], want[k]), k
    assert status == bits
    return bits


# batch, block size, rows of the buffer: one CTA and eight, one tile of 1024 sequences and three
@pytest.mark.parametrize("b,bs,max_tokens", [(1, 16, 1), (7, 32, 100), (128, 16, 4000), (1024, 16, 9000),
                                             (1025, 32, 40000), (2500, 16, 120000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_mixed_step(b, bs, max_tokens, in_place):
    rng = np.random.default_rng(b + bs)
    width = 1500 // bs
    nb = b * (600 // bs + 2) + 1500 // bs
    ctx, held, tables, ring, st = state(rng, b, bs, width, nb, 500)
    kind = rng.random(b)
    new = np.where(kind < 0.5, 1, np.where(kind < 0.6, 0, rng.integers(2, 90, b)))
    new = np.where(kind > 0.85, -np.minimum(ctx, rng.integers(0, 600, b)), new).astype(np.int32)
    check(new, ctx, held, tables, ring, st, bs, max_tokens, in_place)


def test_a_long_prompt_on_eight_ctas():
    rng = np.random.default_rng(3)
    ctx, held, tables, ring, st = state(rng, 3, 16, 5000, 6000, 40)
    new = np.array([1, 65537, 0], np.int32)
    assert check(new, ctx, held, tables, ring, st, 16, 70000) == 0


def test_too_few_blocks_refuses_in_order():
    rng = np.random.default_rng(4)
    ctx, held, tables, ring, st = state(rng, 40, 16, 30, 240, 60, spare=0.5)
    st[1] = 11
    new = np.full(40, 20, np.int32)
    assert check(new, ctx, held, tables, ring, st, 16, 1000) & ref.NO_BLOCKS
    st[1] = 0
    assert check(new, ctx, held, tables, ring, st, 16, 1000, in_place=True) & ref.NO_BLOCKS


def test_refused_sequences_keep_their_state():
    rng = np.random.default_rng(5)
    ctx, held, tables, ring, st = state(rng, 9, 16, 8, 90, 100)
    ctx[6] = max(ctx[6], 1)
    held[6] = -(-ctx[6] // 16)
    new = np.array([1, 200, 2, -ctx[3] - 1, 1, 3, 1, 2**31 - 1, -2**31], np.int32)  # past the table, more than stored
    held[4] = 9    # more than the table is wide
    ctx[5] = -2    # not a length
    held[6] -= 1   # too few for the tokens
    assert check(new, ctx, held, tables, ring, st, 16, 500) == ref.RANGE


def test_rows_past_the_buffer_are_refused():
    rng = np.random.default_rng(6)
    ctx, held, tables, ring, st = state(rng, 6, 32, 20, 80, 200)
    new = np.array([5, 0, 4, 3, -1, 1], np.int32)
    new[4] = -min(1, ctx[4])
    assert check(new, ctx, held, tables, ring, st, 32, 11) == ref.RANGE
    assert check(new, ctx, held, tables, ring, st, 32, 0) == ref.RANGE


@pytest.mark.parametrize("bad", [[-1, 5], [80, 5], [3, -1], [3, 81]])
def test_a_bad_queue_state_serves_nothing_new(bad):
    rng = np.random.default_rng(7)
    ctx, held, tables, ring, _ = state(rng, 6, 32, 20, 80, 200)
    new = np.array([500, 1, 0, 3, -1, 1], np.int32)
    ctx[4] = max(ctx[4], 1)
    held[4] = max(held[4], 1)
    assert check(new, ctx, held, tables, ring, np.array(bad, np.int32), 32, 600) & ref.RANGE


def test_bad_block_ids_give_no_slot():
    rng = np.random.default_rng(8)
    ctx, held, tables, ring, st = state(rng, 5, 16, 20, 100, 100)
    ctx[:] = [17, 16, 0, 30, 1]
    held[:] = [2, 1, 0, 2, 1]
    tables[0, 1] = 100
    tables[3, 1] = -3
    ring[st[0]] = 5000  # the first block taken
    new = np.array([2, 3, 1, 1, 1], np.int32)
    assert check(new, ctx, held, tables, ring, st, 16, 12) == ref.RANGE


def test_more_blocks_returned_than_the_pool_has():
    rng = np.random.default_rng(9)
    ctx, held, tables, ring, st = state(rng, 3, 16, 10, 40, 100)
    ctx[:] = 160
    held[:] = 10
    tables[:] = np.arange(30).reshape(3, 10)
    st[:] = [7, 25]
    assert check(np.full(3, -160, np.int32), ctx, held, tables, ring, st, 16, 4) == ref.RANGE


def test_an_empty_batch():
    z = np.zeros(0, np.int32)
    got, status = run(z, z, z, np.zeros((0, 4), np.int32), np.arange(9, dtype=np.int32), np.array([2, 5], np.int32), 16,
                      7)
    assert status == 0 and got["query_start"].tolist() == [0] and got["state"].tolist() == [2, 5]
    assert (got["positions"] == -1).all() and (got["slots"] == -1).all()


def test_steps_follow_the_host_allocator():
    """Twenty steps of decodes, prompts, finished and returning sequences: the same tables, slots and queue."""
    rng = np.random.default_rng(10)
    b, bs, nb, width, t = 17, 16, 300, 40, 17 * 120  # the first step adds up to 119 rows to each
    host = BlockAllocator(nb, bs, seed=3)
    for s in range(b):
        host.add_sequence(s)
    ring = i32(list(host._free))
    ctx = torch.zeros(b, dtype=torch.int32, device="cuda")
    held = torch.zeros_like(ctx)
    tables = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    st = i32([0, nb])
    qs = torch.empty(b + 1, dtype=torch.int32, device="cuda")
    pos, slots = (torch.empty(t, dtype=torch.int32, device="cuda") for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    import paged_kv_cache_445_b200 as pa
    for step in range(20):
        lens = [host.length(s) for s in range(b)]
        new = np.array([1 if n else int(rng.integers(1, 120)) for n in lens])
        done = [s for s in range(b) if lens[s] and rng.random() < 0.15]
        new[done] = [-lens[s] for s in done]
        pa.pa_step_slots(i32(new), ctx, held, tables, ring, st, bs, qs, pos, slots, dev_status=status)
        want = []
        for s in range(b):
            if new[s] > 0:
                want.append(host.append_slots(s, int(new[s])))
        for s in done:  # the queue gives blocks before it takes them back
            host.free(s)
            host.add_sequence(s)
        want = np.concatenate(want)
        assert int(status.item()) == 0
        assert np.array_equal(slots[:len(want)].cpu().numpy(), want), step
        assert (slots[len(want):] == -1).all()
        got, n = tables.cpu().numpy(), held.cpu().numpy()
        for s in range(b):
            assert got[s, :n[s]].tolist() == host.table(s)
        assert ctx.tolist() == [host.length(s) for s in range(b)]
        head, count = st.tolist()
        q = ring.tolist()
        assert [q[(head + j) % nb] for j in range(count)] == list(host._free)


def test_two_runs_of_one_state_give_the_same():
    rng = np.random.default_rng(11)
    args = state(rng, 300, 16, 60, 9000, 400)
    new = np.where(rng.random(300) < 0.2, -args[0], rng.integers(0, 60, 300)).astype(np.int32)
    a, b = (run(new, *args, 16, 20000)[0] for _ in range(2))
    assert all(np.array_equal(a[k], b[k]) for k in a)

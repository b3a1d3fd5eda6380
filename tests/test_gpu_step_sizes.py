"""The step operators where offsets pass 31 and 32 bits: caches, probability
rows and row buffers of several GB, compared with the same call on small ones."""
from __future__ import annotations

import pytest
import torch

from tests.gpu_helpers import load_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    load_library()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_slots_far_into_a_cache(kind):
    """Rows land in blocks past 4 GB as they do in the first ones; nothing else changes."""
    import paged_kv_cache_445_b200 as pa
    t, hq, hkv, d, bs = 40, 8, 8, 128, 16
    width = d * 9 // 16 if kind == "int4" else d
    dtype = torch.bfloat16 if kind == "bf16" else torch.uint8
    block = hkv * bs * width * (2 if kind == "bf16" else 1)  # bytes
    nb = (5 << 30) // block
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(t, h, d, generator=g, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    table = torch.empty(64, d, device="cuda")
    pa.pa_rope_table(table)
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = []
    for blocks, first in ((3, 0), (nb, nb - 3)):
        kc, vc = (torch.zeros(blocks, hkv, bs, width, dtype=dtype, device="cuda") for _ in range(2))
        args = (torch.empty_like(q), q, k, v, kc, vc, table, pos, first * bs + pos)
        if kind == "bf16":
            pa.pa_rope_append(*args, dev_status=status)
        elif kind == "fp8":
            pa.pa_rope_append_fp8(*args, 0.0625, 0.03125, dev_status=status)
        else:
            pa.pa_rope_append_int4(*args, dev_status=status)
        rows = [kc[first:].clone(), vc[first:].clone(), args[0]]
        if kind == "int4":
            ko, vo = (torch.empty(t, hkv, d, device="cuda") for _ in range(2))
            pa.pa_cache_read_int4(ko, vo, kc, vc, first * bs + pos, dev_status=status)
            rows += [ko, vo]
            kd, vd = torch.zeros_like(kc), torch.zeros_like(vc)
            pa.pa_cache_append_int4(k, v, kd, vd, first * bs + pos, dev_status=status)
            rows += [kd[first:].clone(), vd[first:].clone()]
            assert not kd[:first].any() and not vd[:first].any()
        assert not kc[:first].any() and not vc[:first].any()
        got.append(rows)
    assert int(status.item()) == 0
    for near, far in zip(*got):
        assert near.any() and torch.equal(near, far)


@pytest.mark.parametrize("varlen", [False, True])
@pytest.mark.parametrize("hq,hkv,d,bs", [(16, 8, 128, 16), (24, 4, 256, 32), (4, 4, 64, 16)])
def test_int4_attention_far_into_a_cache(hq, hkv, d, bs, varlen):
    """The same keys in blocks past 4 GB give the same rows, bit for bit."""
    import paged_kv_cache_445_b200 as pa
    record = bs * d * 9 // 16
    nb = (5 << 30) // (hkv * record)
    g = torch.Generator(device="cuda").manual_seed(2)
    ctx = torch.tensor([700, 33, 1], dtype=torch.int32, device="cuda")
    entries = -(-700 // bs)
    small = [torch.empty(3 * entries, hkv, bs, d * 9 // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    slots = torch.arange(3 * entries * bs, dtype=torch.int32, device="cuda")
    kv = [torch.randn(len(slots), hkv, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    pa.pa_cache_append_int4(*kv, *small, slots)
    tables = torch.arange(3 * entries, dtype=torch.int32, device="cuda").view(3, entries)
    far = [torch.empty(nb, hkv, bs, d * 9 // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for x, y in zip(far, small):
        x[nb - 3 * entries:] = y
    qs = torch.tensor([0, 4, 5, 6], dtype=torch.int32, device="cuda")
    q = torch.randn(6 if varlen else 3, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = pa.make_int4_workspace(hq, hkv, d)
    got = []
    for cache, bt in ((small, tables), (far, tables + (nb - 3 * entries))):
        out = torch.zeros_like(q)
        args = (*cache, bt, ctx, d ** -0.5, ws, status)
        if varlen:
            pa.pa_prefill_chunk_int4(out, q, qs, *args)
        else:
            pa.pa_decode_int4(out, q, *args)
        got.append(out)
    assert int(status.item()) == 0
    assert got[0].any() and torch.equal(*got)


def test_probability_rows_past_2_to_the_31():
    """17000 rows of 128000 bf16 probabilities; the second sequence's rows lie past element 2^31."""
    import paged_kv_cache_445_b200 as pa
    rows, vocab, n = 17000, 128000, 3
    target, draft = (torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    first = rows - n
    assert first * vocab > 2**31
    target[[0, first, first + 1, first + 2]] = 0
    draft[[first, first + 1]] = 0
    target[0, 99999] = 1.0
    target[first, 127000] = draft[first, 127000] = 1.0      # kept
    target[first + 1, 5] = draft[first + 1, 127999] = 1.0   # refused: 5 in its place
    tokens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    tokens[1] = -1                                          # no drafts
    tokens[first + 1:] = torch.tensor([127000, 127999], dtype=torch.int32)
    out = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    acc = torch.empty(2, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_accept_drafts(out, acc, target, draft, tokens,
                        torch.tensor([0, first, rows], dtype=torch.int32, device="cuda"),
                        torch.full((rows,), 0.5, device="cuda"), dev_status=status)
    assert acc.tolist() == [0, 1] and int(status.item()) == 0
    assert int(out[0]) == 99999 and bool((out[1:first] == -1).all())
    assert out[first:].tolist() == [127000, 5, -1]


@pytest.mark.parametrize("in_place", [False, True])
def test_the_largest_row_buffer(in_place):
    """2^31 - 1 rows of buffer: two sequences' rows, then padding to the end."""
    import paged_kv_cache_445_b200 as pa
    rows = 2**31 - 1

    def i32(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")
    pos, slots = (torch.empty(rows, dtype=torch.int32, device="cuda") for _ in range(2))
    new, ctx, held = i32(2, 3), i32(15, 0), i32(1, 0)
    tables = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    tables[0, 0] = 6
    ring, state, qs = i32(1, 4, 0, 2, 3, 5, 7, 6), i32(0, 7), i32(0, 0, 0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = {} if in_place else dict(context_lens_out=i32(0, 0), blocks_held_out=i32(0, 0), free_state_out=i32(0, 0))
    pa.pa_step_slots(new, ctx, held, tables, ring, state, 16, qs, pos, slots, dev_status=status, **outs)
    assert int(status.item()) == 0 and qs.tolist() == [0, 2, 5]
    assert pos[:5].tolist() == [15, 16, 0, 1, 2] and slots[:5].tolist() == [6 * 16 + 15, 16, 64, 65, 66]
    assert int(pos[5:].max()) == -1 and int(pos[5:].min()) == -1
    assert int(slots[5:].max()) == -1 and int(slots[5:].min()) == -1
    got = [outs.get(k, x).tolist() for k, x in (("context_lens_out", ctx), ("blocks_held_out", held),
                                                ("free_state_out", state))]
    assert got == [[17, 3], [2, 1], [2, 5]]


def test_a_table_past_2_to_the_32_bytes():
    """Far rows of a long table equal a short table's: the angles of one position do not depend on the table."""
    import paged_kv_cache_445_b200 as pa
    n = 2**26 + 8  # rows of 64 bytes
    table, start = torch.zeros(n, 16, device="cuda"), n - 40
    pa.pa_rope_table(table)
    p = torch.arange(start, n, dtype=torch.float64, device="cuda")[:, None]
    w = 10000.0 ** (-torch.arange(0, 16, 2, dtype=torch.float64, device="cuda") / 16)
    want = torch.cat([(p * w).cos(), (p * w).sin()], 1)
    # an angle near 2^26 carries 2^-27 of binary64 rounding on either side; the value's own rounding is 2^-25
    assert (table[start:].double() - want).abs().max().item() <= 2.0**-25 + 2.0**-25

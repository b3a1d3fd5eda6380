"""Attention over the 4-bit cache (pa_decode_int4, pa_prefill_chunk_int4)
against the definition in 64 bits.

Tolerance per output: bf16 rounding, 2^-8 of the value; the weights p enter the
products in fp16 (2^-11), once more against their sum (2^-11), and the scores,
sums of products in binary32, may move a weight by another 2^-10 at these sizes:
together 2^-9 of the largest |value| seen."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import step_reference as ref
from tests.gpu_helpers import i32, load_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    load_library()


class Batch:
    def __init__(self, ctx, rows, hq, hkv, d, bs, seed=0, poison=True, amp=0.5):
        rng = np.random.default_rng(seed)
        self.ctx, self.rows = np.array(ctx), np.array(rows)
        self.hq, self.hkv, self.d, self.bs = hq, hkv, d, bs
        need = -(-self.ctx // bs)
        self.width = max(1, int(need.max()))
        self.nb = int(need.sum()) + 3
        ids = rng.permutation(self.nb)
        self.tables = np.full((len(ctx), self.width), -1, np.int64)
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = ids[at:at + n]
            at += n
        self.kv, self.cache = [], []
        for _ in range(2):
            codes = rng.integers(1, 16, (self.nb, hkv, bs, d)).astype(np.uint8)
            scales = (rng.random((self.nb, hkv, bs, d // 32)) * 0.4 + 0.05).astype(np.float16)
            if poison:  # every place that holds no token: NaN scales
                live = np.zeros((self.nb, bs), bool)
                for s, n in enumerate(self.ctx):
                    for j in range(n):
                        live[self.tables[s, j // bs], j % bs] = True
                scales = np.where(live[:, None, :, None], scales, np.float16(np.nan))
            self.kv.append(ref.int4_values(codes, scales))
            self.cache.append(torch.from_numpy(ref.int4_pack(codes, scales)).cuda())
        self.qs = np.concatenate([[0], np.cumsum(rows)])
        t = int(self.qs[-1])
        self.q = torch.from_numpy(rng.standard_normal((t, hq, d)) * amp).to(torch.bfloat16).cuda()
        self.scale = d ** -0.5
        self.out = torch.full_like(self.q, -5.0)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        import paged_kv_cache_445_b200 as pa
        self.ws = pa.make_int4_workspace(hq, hkv, d)

    def run(self, varlen=False, out=None):
        import paged_kv_cache_445_b200 as pa
        out = self.out if out is None else out
        args = (*self.cache, i32(self.tables), i32(self.ctx), self.scale, self.ws, self.status)
        if varlen:
            pa.pa_prefill_chunk_int4(out, self.q, i32(self.qs), *args)
        else:
            pa.pa_decode_int4(out, self.q, *args)
        torch.cuda.synchronize()
        return int(self.status.item())

    def reference(self):
        q = self.q.float().cpu().numpy().astype(np.float64)
        kv = [np.nan_to_num(x, nan=0.0) for x in self.kv]
        return ref.attention(q, *kv, self.tables, self.ctx, self.qs, self.scale, self.bs)

    def check(self, out=None):
        want = self.reference()
        got = (self.out if out is None else out).float().cpu().numpy().astype(np.float64)
        assert np.isfinite(got).all()
        top = np.nanmax(np.abs(self.kv[1]))
        err = np.abs(got - want) - (2.0**-8 * np.abs(want) + 2.0**-9 * top)
        assert err.max() <= 0, f"{err.max()} past the bound"


DECODE = [  # contexts, Hq, Hkv, d, bs
    ([1], 2, 1, 64, 16),
    ([0, 5, 17, 33, 64, 0], 2, 1, 64, 16),
    ([15, 16, 17, 31, 32, 33, 700], 8, 1, 128, 16),
    ([31, 32, 33, 63, 64, 65, 1], 8, 2, 128, 32),
    ([40, 1000], 16, 1, 128, 16),        # 16 heads on a KV head
    ([300, 77], 11, 1, 128, 32),
    ([500, 3, 90], 24, 4, 256, 32),
    ([129, 250], 8, 1, 256, 16),
    ([200, 60, 333], 12, 12, 64, 32),    # one head a KV head
    ([333, 2], 15, 3, 128, 16),
    ([9000, 7000], 8, 1, 128, 16),       # cut between many warps
    ([3000], 64, 8, 128, 16),
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"Hq{c[1]}-Hkv{c[2]}-d{c[3]}-bs{c[4]}-n{len(c[0])}-{max(c[0])}")
def test_decode(case):
    ctx, hq, hkv, d, bs = case
    b = Batch(ctx, [1] * len(ctx), hq, hkv, d, bs, seed=len(ctx) + hq + d)
    assert b.run() == 0
    b.check()


ROWS = [  # contexts, rows, Hq, Hkv, d, bs
    ([40, 100, 17], [5, 0, 1], 8, 1, 128, 16),
    ([33, 64, 7, 300, 12], [2, 9, 7, 4, 0], 16, 2, 128, 32),
    ([3, 2, 10], [5, 2, 10], 4, 2, 64, 16),         # more rows than keys: rows without a key are zero
    ([150], [130], 4, 4, 64, 32),                   # a chunk from the start and past it
    ([600, 90], [33, 17], 24, 4, 256, 32),
    ([200], [3], 32, 2, 128, 16),
    ([1200, 50, 800], [6, 6, 6], 5, 5, 128, 16),
]


@pytest.mark.parametrize("case", ROWS, ids=lambda c: f"Hq{c[2]}-Hkv{c[3]}-d{c[4]}-bs{c[5]}-rows{sum(c[1])}")
def test_varlen(case):
    ctx, rows, hq, hkv, d, bs = case
    b = Batch(ctx, rows, hq, hkv, d, bs, seed=sum(rows) + hq)
    assert b.run(varlen=True) == 0
    b.check()


def test_many_sequences():
    rng = np.random.default_rng(1)
    ctx = rng.integers(0, 60, 1500)
    b = Batch(ctx, [1] * 1500, 4, 2, 64, 16, seed=5)
    assert b.run() == 0
    b.check()


@pytest.mark.parametrize("varlen", [False, True])
def test_repeats_bit_for_bit(varlen):
    """Pieces are merged in their order whoever brings the last one (the two entry points cut the keys at different
    places, so they agree up to rounding only)."""
    b = Batch([500, 33, 20000], [1, 1, 1], 16, 2, 128, 16, seed=3)
    assert b.run(varlen) == 0
    b.check()
    first = b.out.clone()
    for _ in range(5):
        out = torch.zeros_like(b.out)
        assert b.run(varlen, out) == 0
        assert torch.equal(out, first)


def test_rows_behind_the_last_sequence_stay():
    import paged_kv_cache_445_b200 as pa
    b = Batch([100, 50], [3, 2], 8, 2, 128, 16, seed=4)
    q = torch.cat([b.q, torch.full((4, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
    out = torch.full_like(q, -5.0)
    pa.pa_prefill_chunk_int4(out, q, i32(b.qs), *b.cache, i32(b.tables), i32(b.ctx), b.scale, b.ws, b.status)
    b.check(out[:5])
    assert (out[5:] == -5.0).all() and int(b.status.item()) == 0


def test_a_late_large_score_and_small_ones():
    """The maximum rises at the last key; the first keys' weights vanish."""
    b = Batch([900], [1], 8, 1, 128, 16, seed=6, amp=8.0)
    assert b.run() == 0
    b.check()
    b = Batch([900], [1], 8, 1, 128, 16, seed=6)
    b.scale = 0.0  # every key weighs the same
    assert b.run() == 0
    b.check()
    b.scale = -0.1
    assert b.run() == 0
    b.check()


@pytest.mark.parametrize("amp", [1e-30, 1e-6, 1e6, 1e30])
def test_queries_outside_the_fp16_range(amp):
    """q far below and above fp16: the scores are scale * q . k all the same (scale undoes amp)."""
    b = Batch([300, 20], [1, 1], 16, 2, 128, 32, seed=7, amp=amp)
    b.scale = 0.05 / amp
    assert b.run() == 0
    b.check()


def test_infinite_and_nan_queries_give_nan_rows_only():
    b = Batch([300, 40, 77], [1, 1, 1], 8, 2, 128, 16, seed=8)
    b.q[1, 2, 5] = float("nan")
    assert b.run() == 0
    got = b.out.float()
    assert torch.isnan(got[1, 2]).all()
    got[1, 2] = 0
    assert torch.isfinite(got).all()


def test_bad_blocks_are_skipped_and_reported():
    b = Batch([100, 90, 40], [1, 1, 1], 8, 2, 128, 16, seed=9)
    good = b.reference()
    b.tables[0, 2] = b.nb
    b.tables[1, 0] = -1
    assert b.run() == ref.RANGE
    got = b.out.float().cpu().numpy()
    assert np.isfinite(got).all()
    assert np.abs(got[2] - good[2]).max() < 2.0**-6 * 7  # the untouched sequence
    # the same keys left out of the definition
    keys = np.delete(np.arange(100), np.arange(32, 48))
    q = b.q.float().cpu().numpy().astype(np.float64)
    blocks = np.where(np.arange(b.width) == 2, 0, b.tables[0])
    k, v = (np.nan_to_num(x)[blocks].transpose(1, 0, 2, 3).reshape(2, -1, 128)[:, keys] for x in b.kv)
    for h in range(8):
        z = k[h // 4] @ q[0, h] * b.scale
        p = np.exp(z - z.max())
        want = p @ v[h // 4] / p.sum()
        assert np.abs(got[0, h] - want).max() <= 2.0**-8 * np.abs(want).max() + 2.0**-9 * np.nanmax(np.abs(b.kv[1]))


def test_a_context_longer_than_its_table_is_reported():
    b = Batch([64, 30], [1, 1], 8, 2, 128, 16, seed=10)
    b.ctx = np.array([65, 30])
    assert b.run() == ref.RANGE
    assert (b.out[0] == 0).all() and torch.isfinite(b.out[1].float()).all()


def test_negative_lengths_and_wild_row_offsets():
    b = Batch([64, 30, 20], [2, 1, 3], 8, 2, 128, 16, seed=11)
    b.ctx = np.array([64, -7, 20])
    assert b.run(varlen=True) in (0, ref.RANGE)
    assert (b.out[2] == 0).all()
    for qs in ([0, 2, 900, 901], [-3, 2, 3, 6], [0, 5, 2, 6]):
        b.qs = np.array(qs)
        assert b.run(varlen=True) == ref.RANGE
        b.status.zero_()


def test_workspace_is_clean_after_every_call():
    """One workspace, calls of different shapes one after another, on a stream of its own."""
    a = Batch([5000], [1], 8, 1, 128, 16, seed=12)
    c = Batch([33, 900, 2], [4, 3, 1], 8, 1, 128, 16, seed=13)
    c.ws = a.ws
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            assert a.run() == 0 and c.run(varlen=True) == 0
    a.check()
    c.check()


def test_graph_replay_equals_eager():
    import paged_kv_cache_445_b200 as pa
    b = Batch([700, 3, 90], [1, 1, 1], 16, 2, 128, 16, seed=14)
    tables, ctx = i32(b.tables), i32(b.ctx)
    assert b.run() == 0
    want = b.out.clone()
    out = torch.zeros_like(b.out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_decode_int4(out, b.q, *b.cache, tables, ctx, b.scale, b.ws, b.status)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)

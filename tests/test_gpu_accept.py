"""Verification of drafted tokens (pa_accept_drafts) against the definition in 64 bits."""
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


def softmax(x):
    e = np.exp(x - x.max(1, keepdims=True))
    return (e / e.sum(1, keepdims=True)).astype(np.float32)


def batch(seed, rows, vocab, near=0.5, temp=2.0):
    rng = np.random.default_rng(seed)
    t = int(sum(rows))
    z = rng.standard_normal((t, vocab)) * temp
    target = softmax(z)
    draft = softmax(z + near * rng.standard_normal((t, vocab)))
    tokens = np.zeros(t, np.int64)
    for r in range(t - 1):
        tokens[r + 1] = min(vocab - 1, int(np.searchsorted(np.cumsum(draft[r], dtype=np.float64), rng.random())))
    qs = np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)
    return target, draft, tokens, qs, rng.random(t).astype(np.float32)


def run(target, draft, tokens, qs, uniforms, dtype=torch.float32, pad=0, ctx=None, in_place=False):
    import paged_kv_cache_445_b200 as pa

    def probs(x):
        wide = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
        wide[:, :x.shape[1]] = torch.from_numpy(np.ascontiguousarray(x)).to(dtype)
        return wide[:, :x.shape[1]]

    out = torch.full((len(tokens),), -9, dtype=torch.int32, device="cuda")
    acc = torch.full((len(qs) - 1,), -9, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = {}
    if ctx is not None:
        kw["context_lens"] = i32(ctx)
        if not in_place:
            kw["context_lens_out"] = torch.full_like(kw["context_lens"], -9)
    pa.pa_accept_drafts(out, acc, probs(target), None if draft is None else probs(draft), i32(tokens), i32(qs),
                        torch.from_numpy(uniforms).cuda(), dev_status=status, **kw)
    torch.cuda.synchronize()
    after = kw.get("context_lens_out", kw.get("context_lens"))
    return out.cpu().numpy(), acc.cpu().numpy(), int(status.item()), None if after is None else after.cpu().numpy()


def check(target, draft, tokens, qs, uniforms, **kw):
    dtype = kw.get("dtype", torch.float32)
    r = lambda x: None if x is None else torch.from_numpy(x).to(dtype).double().numpy()  # noqa: E731
    out, acc, bits = ref.accept(r(target), r(draft), tokens, qs, uniforms)
    got, got_acc, status, ctx = run(target, draft, tokens, qs, uniforms, **kw)
    assert np.array_equal(got_acc, acc)
    assert np.array_equal(got, out)
    assert status == bits
    if kw.get("ctx") is not None:
        n = np.where((qs[:-1] < 0) | (qs[1:] > len(tokens)), 0, np.diff(qs))  # outside the rows: nothing lost
        assert np.array_equal(ctx, np.where(n > 0, kw["ctx"] - (n - 1 - acc), kw["ctx"]))
    return out, acc, bits


# vocabularies of one value, odd sizes, one slice short of and past whole slices, a large one
@pytest.mark.parametrize("vocab", [1, 2, 127, 997, 1024, 16384, 16385, 50001, 128000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_drafts_with_a_draft_distribution(vocab, dtype):
    rows = [5, 1, 3, 0, 2, 8, 1]
    check(*batch(vocab, rows, vocab), dtype=dtype, ctx=np.arange(20, 27), pad=3)


@pytest.mark.parametrize("vocab", [5, 997, 32000])
def test_drafts_that_were_looked_up(vocab):
    target, _, tokens, qs, u = batch(vocab, [4, 6, 1, 3, 9], vocab)
    target = target * 0.2
    for r in range(len(tokens) - 1):
        target[r, tokens[r + 1]] += 0.8
    check(target, None, tokens, qs, u, ctx=np.full(5, 50), in_place=True)


def test_more_drafts_than_a_warp_has_lanes():
    target, draft, tokens, qs, u = batch(3, [70, 40], 300, near=0.0)  # equal distributions: every draft is kept
    out, acc, _ = check(target, draft, tokens, qs, u)
    assert acc.tolist() == [69, 39]
    u2 = u.copy()
    target[50, :] = 0  # the target has nothing of draft 51
    target[50, 7] = 1
    tokens[51] = 9
    _, acc, _ = check(target, draft, tokens, qs, u2)
    assert acc.tolist() == [50, 39]


def test_every_uniform_at_its_ends():
    target, draft, tokens, qs, u = batch(4, [4, 4, 4], 1000)
    for x in (0.0, np.float32(1 - 2**-24), 1.0, 2.0, np.nan):
        check(target, draft, tokens, qs, np.full_like(u, x))


def test_ties_go_to_the_first_index_past_the_sum():
    target = np.full((6, 8), 0.125, np.float32)
    qs = np.arange(7)
    u = np.array([0.0, 0.125, 0.25, 0.5, 0.874, 0.875], np.float32)
    out, _, _ = check(target, None, np.zeros(6, np.int64), qs, u)
    assert out.tolist() == [0, 1, 2, 4, 6, 7]


def test_zeros_around_the_mass():
    target = np.zeros((4, 40000), np.float32)
    target[:, [77, 20000, 39000]] = [0.25, 0.5, 0.25]
    out, _, _ = check(target, None, np.zeros(4, np.int64), np.arange(5), np.array([0, 0.25, 0.74, 0.75], np.float32))
    assert out.tolist() == [77, 20000, 20000, 39000]


def test_the_draft_leaves_nothing():
    target, draft, tokens, qs, _ = batch(5, [2, 2], 500)
    draft = np.maximum(draft, target) + np.float32(1e-3)  # nowhere below the target: draw from the target itself
    tokens[1] = tokens[3] = 3
    target[0, 3] = target[2, 3] = 0
    check(target, draft, tokens, qs, np.array([0.5, 0.3, 0.5, 0.9], np.float32))
    only = np.zeros((2, 500), np.float32)  # looked up, and the target knows only the refused token
    only[:, 3] = 0.25
    check(only, None, np.array([0, 3]), np.array([0, 2]), np.array([0.5, 0.5], np.float32))


def test_odd_weights_count_as_zero():
    target = np.full((4, 3000), 1e-4, np.float32)
    target[0, 5] = np.nan
    target[1, 2000] = np.inf
    target[2, 100] = -3.0
    target[3, :] = [0.0] * 2999 + [np.nan]
    out, _, bits = check(target, None, np.zeros(4, np.int64), np.arange(5), np.full(4, 0.5, np.float32))
    assert out[3] == -1 and bits == ref.RANGE


def test_negative_and_wild_tokens_end_the_drafts():
    target, draft, tokens, qs, u = batch(6, [6, 6, 6], 700, near=0.0)
    tokens[3] = -1
    tokens[7] = -5
    tokens[14] = 700
    out, acc, bits = check(target, draft, tokens, qs, u, ctx=np.array([100, 200, 300]))
    assert acc.tolist() == [2, 0, 1] and bits == ref.RANGE


def test_bad_row_offsets_are_reported_and_skipped():
    target, draft, tokens, _, u = batch(7, [3, 3], 200)
    for qs in ([0, 3, 7], [-1, 3, 6], [4, 2, 6]):
        check(target, draft, tokens, np.array(qs), u, ctx=np.array([9, 9]))
    out, _, _ = check(target, draft, tokens, np.array([2, 4, 5]), u)  # rows outside every sequence
    assert out[[0, 1, 5]].tolist() == [-9] * 3


def test_tokens_follow_the_targets_distribution():
    """Keeping by min(1, p/q) and drawing from the rest gives p: 20000 sequences of one draft, 8 tokens.

    The count of each first token is binomial: its deviation stays under 5 sigma
    (probability of a false alarm under 1e-5)."""
    rng = np.random.default_rng(8)
    n, vocab = 20000, 8
    p, q = softmax(rng.standard_normal((1, vocab)))[0], softmax(rng.standard_normal((1, vocab)))[0]
    target, draft = np.tile(p, (2 * n, 1)), np.tile(q, (2 * n, 1))
    tokens = np.zeros(2 * n, np.int64)
    tokens[1::2] = np.minimum(np.searchsorted(np.cumsum(q, dtype=np.float64), rng.random(n)), vocab - 1)
    out, acc, _, _ = run(target, draft, tokens, np.arange(0, 2 * n + 1, 2), rng.random(2 * n).astype(np.float32))
    counts = np.bincount(out[0::2], minlength=vocab)
    sigma = np.sqrt(n * p.astype(np.float64) * (1 - p))
    assert (np.abs(counts - n * p.astype(np.float64)) < 5 * sigma).all()

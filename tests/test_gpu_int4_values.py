"""Attention over the 4-bit cache where V's size, or the spread of the weights,
leaves fp16's range: small and large scales, scales that differ between keys and
chunks, a first key that takes nearly all of the weight.

Bound per output, from the operator's own terms (p: the weights, v: the values, s
their scales):
- bf16 rounding, 2^-8 of the value.
- A weight enters the product with V in fp16 and is rounded once more with its scale,
  2^-11 each; a score off by e moves its weight by e ln 2 against the others and in
  their sum: with sums of binary32 over scores below 2^6 (|e| < 2^-13) another 2^-11.
  Together 1.5 * 2^-10 of sum p |v|.
- A product below fp16's normal range is off by 2^-25 where a weight may be 2^12 and the
  largest scale enters as 1/2 or more, and counts 7 times at most: 2^-36 of the chunk's
  largest |v| (7 of that scale) per key.
- The tensor core adds the 16 products of a step and the sum so far on one grid, 2^-25 of
  the largest product as its operands' exponent fields give it (measured: beside
  8 * 2^14 a product of 2^-25 of that is kept, one of 2^-26 is not).  A code u 2^-24 is
  a subnormal fp16 number, whose field stands for 2^-14, so the grid is at most
  2^-25 * 2^-14 / 2^-24 = 2^-15 of the step's largest p s, in units of p s: 17 terms a
  step, in the codes' product and in that of the 8 they carry too many, and the largest
  p s of the steps is at most their sum: 34 * 2^-15 of sum p s."""
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


def put(b, which, codes, scales):
    """Another K (0) or V (1) into the batch's pool; places without a token keep a NaN scale."""
    dead = np.isnan(b.kv[which]).reshape(*scales.shape, 32).any(-1)
    scales = np.where(dead, np.float16(np.nan), scales.astype(np.float16))
    b.kv[which] = ref.int4_values(codes, scales)
    b.scales = np.repeat(np.nan_to_num(scales.astype(np.float64), nan=0.0), 32, -1)  # of V, put last
    b.cache[which] = torch.from_numpy(ref.int4_pack(codes, scales)).cuda()


def parts(b, seed):
    rng = np.random.default_rng(seed)
    shape = (b.nb, b.hkv, b.bs, b.d)
    codes = rng.integers(1, 16, shape).astype(np.uint8)
    return rng, codes, (rng.random((*shape[:3], b.d // 32)) * 0.4 + 0.05)


def check(b):
    """Against 64 bits; returns the largest error over its bound."""
    q = b.q.float().cpu().numpy().astype(np.float64)
    k, v = (np.nan_to_num(x, nan=0.0) for x in b.kv)
    args = (b.tables, b.ctx, b.qs, b.scale, b.bs)
    want, spread, steps = (ref.attention(q, k, x, *args) for x in (v, np.abs(v), b.scales))
    top = np.repeat(np.abs(v).reshape(b.nb, b.hkv, b.bs, -1, 32).max((0, 2, 4)), 32, 1)  # [Hkv, d]
    top = np.repeat(top, b.hq // b.hkv, 0)[None]
    got = b.out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    bound = 2.0**-8 * np.abs(want) + 1.5 * 2.0**-10 * spread + 34 * 2.0**-15 * steps
    bound += 2.0**-36 * max(b.ctx) * top
    worst = (np.abs(got - want) / np.maximum(bound, 1e-300)).max()
    assert worst <= 1, f"{worst} times the bound"
    return worst


FORMS = [  # contexts, rows (None: the call for single rows), Hq, Hkv, d, bs: one case per form of the kernel
    ([700, 33, 5], None, 4, 2, 64, 16),
    ([700, 33, 5], None, 16, 1, 64, 32),
    ([900, 64, 17], None, 16, 2, 128, 16),
    ([900, 64, 17], None, 16, 1, 128, 32),
    ([600, 31, 90], None, 24, 4, 256, 32),
    ([300, 40], [5, 17], 8, 2, 64, 16),
    ([300, 40, 9], [3, 6, 9], 16, 2, 128, 32),
    ([250, 70], [4, 1], 8, 2, 256, 16),
]
IDS = [f"d{f[4]}-G{f[2] // f[3]}-{'rows' if f[1] else 'decode'}" for f in FORMS]


def batch(form, seed):
    ctx, rows, hq, hkv, d, bs = form
    return Batch(ctx, rows or [1] * len(ctx), hq, hkv, d, bs, seed=seed)


@pytest.mark.parametrize("power", [-18, -12, -6, 6, 12, 17])
@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_values_of_any_size(form, power):
    """V's scales from subnormal fp16 numbers to its largest: the error keeps its share of the values."""
    b = batch(form, 20)
    _, codes, scales = parts(b, 21)
    put(b, 1, codes, scales * 2.0**power)
    assert b.run(varlen=form[1] is not None) == 0
    check(b)


@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_scales_that_differ_between_keys_and_chunks(form):
    """Chunks of one row from 1e-6 to 1e3, and within a chunk keys a thousand times larger than others."""
    b = batch(form, 22)
    rng, codes, scales = parts(b, 23)
    chunk = 10.0 ** rng.integers(-6, 4, scales.shape[-1])
    put(b, 1, codes, scales * chunk * np.where(rng.random(scales.shape[:3]) < 0.02, 1.0, 1e-3)[..., None])
    assert b.run(varlen=form[1] is not None) == 0
    check(b)


@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_scales_that_rise_and_fall_along_the_keys(form, rising):
    """Every further key's values a little larger (the reference moves again and again), or smaller."""
    b = batch(form, 24)
    _, codes, scales = parts(b, 25)
    for s, n in enumerate(b.ctx):
        for j in range(int(n)):
            x = (j if rising else n - 1 - j) / max(1, n - 1)
            scales[b.tables[s, j // b.bs], :, j % b.bs] *= 2.0 ** (20 * x - 12)
    put(b, 1, codes, scales)
    assert b.run(varlen=form[1] is not None) == 0
    check(b)


def sink(b, nats, value_scale, seed):
    """Key 0 of every sequence `nats` above the others' mean score, its value zero; the other scores are small."""
    rng, codes, scales = parts(b, seed)
    first = np.unique(b.tables[:, 0])
    codes[..., 0] = 8                           # dim 0 tells the first key alone
    codes[first, :, 0] = 8
    codes[first, :, 0, 0] = 15
    scales = scales * 0.2
    scales[first, :, 0, 0] = nats / (7 * b.scale)
    put(b, 0, codes, scales)
    b.q[..., 0] = 1.0
    _, codes, scales = parts(b, seed + 1)
    codes[first, :, 0] = 8
    scales[first, :, 0] = 0.0
    put(b, 1, codes, scales * value_scale)


@pytest.mark.parametrize("nats,value_scale", [(8, 1e-4), (10, 1e-3), (12, 1e-2), (14, 1.0), (14, 1e-5)])
@pytest.mark.parametrize("d,hq,bs", [(64, 4, 16), (128, 4, 32), (256, 4, 16)])
def test_a_first_key_that_takes_the_weight(d, hq, bs, nats, value_scale):
    """One key far above thousands, its value zero, in one warp's walk: 300 sequences over one pool."""
    b = Batch([2048], [1], hq, 4, d, bs, seed=26)
    n = 300
    b.tables, b.ctx, b.rows = np.repeat(b.tables, n, 0), np.repeat(b.ctx, n), np.ones(n, int)
    b.qs = np.arange(n + 1)
    b.q = (torch.from_numpy(np.random.default_rng(27).standard_normal((n, hq, d)))).to(torch.bfloat16).cuda()
    b.out = torch.full_like(b.q, -5.0)
    sink(b, nats, value_scale, 28)
    assert b.run() == 0
    check(b)


def test_a_first_key_that_takes_the_weight_across_warps():
    """The same for one long sequence, cut between all warps, and for rows of several tokens."""
    b = Batch([20000], [1], 8, 1, 128, 16, seed=29)
    sink(b, 12, 1e-3, 30)
    assert b.run() == 0
    check(b)
    b = Batch([3000, 500], [5, 3], 16, 2, 128, 16, seed=31)
    sink(b, 12, 1e-3, 32)
    assert b.run(varlen=True) == 0
    check(b)


def test_a_nan_value_stays_in_its_chunk_and_rows():
    """A NaN scale of V in the last key: NaN in its 32 dims for the rows that see it, the rest as before."""
    b = Batch([200, 90], [3, 2], 8, 2, 128, 16, seed=33)
    _, codes, scales = parts(b, 34)
    scales = scales * 2.0**-12
    scales[b.tables[0, 199 // 16], 1, 199 % 16, 2] = np.nan
    with np.errstate(invalid="ignore"):
        put(b, 1, codes, scales)
    assert b.run(varlen=True) == 0
    got = b.out.float()
    assert torch.isnan(got[2, 4:, 64:96]).all()
    b.out[2, 4:, 64:96] = 0  # the reference without the NaN key's chunk: those outputs are told above
    b.kv[1] = np.where(np.isnan(b.kv[1]), 0.0, b.kv[1])
    want = b.reference()
    want[2, 4:, 64:96] = 0
    err = np.abs(b.out.float().cpu().numpy() - want)
    assert (err <= 2.0**-8 * np.abs(want) + 1.5 * 2.0**-10 * np.abs(b.kv[1]).max()).all()

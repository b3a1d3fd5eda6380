"""Rotated values where one product lies at a tie of bf16 and the other far below
it: the exact sum decides the rounding, however small the other product is."""
from __future__ import annotations

from fractions import Fraction

import numpy as np
import pytest
import torch

from tests.gpu_helpers import i32, load_library
from tests.test_gpu_rope import bf16, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    load_library()


def nearest_bf16(x: Fraction) -> float:
    """Ties to even; normal range."""
    if x == 0:
        return 0.0
    e = 0
    m = abs(x)
    while m >= 256:
        m, e = m / 2, e + 1
    while m < 128:
        m, e = m * 2, e - 1
    n = m.numerator // m.denominator
    rest = m - n
    if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and n & 1):
        n += 1
    return float((n if x > 0 else -n) * Fraction(2) ** e)


@pytest.mark.parametrize("inter", [False, True])
def test_a_tie_and_a_product_far_below_it(inter):
    import paged_kv_cache_445_b200 as pa
    d, half, rows = 64, 32, 120
    # cosines and sines are ties of bf16 in themselves: 1 + 2^-8 (the even neighbour lies below), 1 + 3 2^-8 (above)
    table = np.empty((2, d), np.float32)
    table[0, :half], table[0, half:] = 1 + 2.0**-8, 1 + 3 * 2.0**-8
    table[1, :half], table[1, half:] = -(1 + 3 * 2.0**-8), 1 + 2.0**-8
    rng = np.random.default_rng(1)
    big = np.ldexp(rng.choice([-1.0, 1.0], (rows, 1, half)), rng.integers(-2, 3, (rows, 1, half)))
    small = np.ldexp(rng.choice([-1.0, 1.0], (rows, 1, half)), -np.arange(5, 5 + rows)[:, None, None])
    first = rng.random((rows, 1, half)) < 0.5
    x, y = np.where(first, big, small), np.where(first, small, big)
    q = np.empty((rows, 1, d))
    if inter:
        q[..., 0::2], q[..., 1::2] = x, y
    else:
        q[..., :half], q[..., half:] = x, y
    pos = np.arange(rows) % 2
    qt = bf16(q).cuda()
    assert np.array_equal(f64(qt), q)
    out, status = torch.zeros_like(qt), torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = [torch.zeros(8, 1, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pa.pa_rope_append(out, qt, qt, qt, *cache, torch.from_numpy(table).cuda(), i32(pos), i32(np.arange(rows)),
                      interleaved=inter, dev_status=status)
    got = f64(out)[:, 0]
    for t in range(rows):
        for i in range(half):
            a, b = Fraction(x[t, 0, i]), Fraction(y[t, 0, i])
            c, s = Fraction(float(table[pos[t], i])), Fraction(float(table[pos[t], half + i]))
            at = (2 * i, 2 * i + 1) if inter else (i, half + i)
            assert got[t, at[0]] == nearest_bf16(a * c - b * s), (t, i)
            assert got[t, at[1]] == nearest_bf16(b * c + a * s), (t, i)
    assert torch.equal(cache[0].reshape(-1, d)[:rows], out[:, 0]) and int(status.item()) == 0

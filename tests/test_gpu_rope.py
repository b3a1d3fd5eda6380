"""Rotary positions fused with the append (pa_rope_append and its FP8 and 4-bit
forms), the 4-bit append and read-back, and the table of angles, against 64-bit
restatements.  Rotation and codes are rounded once, so they are compared bit
for bit."""
from __future__ import annotations

import math

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


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def make_table(p, rot, seed=0):
    rng = np.random.default_rng(seed)
    a = rng.random((p, rot // 2)) * 2 * math.pi
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


class Step:
    def __init__(self, t, hq, hkv, d, rot, bs, cache, seed=0, strided=True, positions=None):
        rng = np.random.default_rng(seed)
        heads = hq + 2 * hkv
        x = bf16(rng.standard_normal((t, heads, d)) * np.exp(rng.standard_normal((1, heads, d)))).cuda()
        self.qkv = x
        self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        if not strided:
            self.q, self.k, self.v = (y.contiguous() for y in (self.q, self.k, self.v))
        self.table = make_table(300, rot, seed)
        self.pos = rng.integers(0, 300, t) if positions is None else positions
        nb = t // bs + 3
        self.slots = rng.permutation(nb * bs)[:t].astype(np.int64)
        self.q_out = torch.full((t, hq, d), -5.0, dtype=torch.bfloat16, device="cuda")
        shape = {"bf16": (nb, hkv, bs, d), "fp8": (nb, hkv, bs, d), "int4": (nb, hkv, bs, d * 9 // 16)}[cache]
        dtype = torch.bfloat16 if cache == "bf16" else torch.uint8
        self.kc, self.vc = (torch.full(shape, 77, dtype=dtype, device="cuda") for _ in range(2))
        self.cache, self.bs = cache, bs
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, inter, q_out=None):
        import paged_kv_cache_445_b200 as pa
        fn = {"bf16": pa.pa_rope_append, "fp8": pa.pa_rope_append_fp8, "int4": pa.pa_rope_append_int4}[self.cache]
        scales = (0.5, 0.375) if self.cache == "fp8" else ()
        fn(self.q_out if q_out is None else q_out, self.q, self.k, self.v, self.kc, self.vc,
           torch.from_numpy(self.table).cuda(), i32(self.pos), i32(self.slots), *scales, interleaved=inter,
           dev_status=self.status)
        torch.cuda.synchronize()
        return int(self.status.item())

    def check(self, inter):
        live = (self.pos >= 0) & (self.pos < len(self.table))
        pos = np.where(live, self.pos, -1)
        q = ref.bf16_round(ref.rotate(f64(self.q), self.table, pos, inter))
        want_q = np.full(q.shape, -5.0)
        want_q[live] = q[live]
        assert np.array_equal(f64(self.q_out), want_q)
        k, v = ref.bf16_round(ref.rotate(f64(self.k), self.table, pos, inter)), f64(self.v)
        check_cache(self.kc, k, self.slots, live, self.cache, self.bs, 0.5)
        check_cache(self.vc, v, self.slots, live, self.cache, self.bs, 0.375)


def check_cache(cache, rows, slots, live, kind, bs, scale):
    """The cache holds `rows` at `slots` and its old bytes (77) everywhere else."""
    nb, hkv = cache.shape[:2]
    d = rows.shape[2]
    keep = live & (slots >= 0) & (slots < nb * bs)
    blk, off = slots[keep] // bs, slots[keep] % bs
    if kind == "int4":
        codes, s = ref.int4_quantise(rows)
        raw = cache.cpu().numpy().reshape(nb, hkv, -1)
        want = np.full_like(raw, 77)
        byte, shift, sb = ref.int4_places(bs, d)
        for t, b, o in zip(np.nonzero(keep)[0], blk, off):
            want[b, :, byte[o]] = 0
            for half in (0, 4):
                m = shift[o] == half
                want[b][:, byte[o][m]] |= codes[t][:, m] << half
            raw_s = np.ascontiguousarray(s[t]).view(np.uint8).reshape(hkv, -1, 2)
            want[b][:, sb[o]], want[b][:, sb[o] + 1] = raw_s[..., 0], raw_s[..., 1]
        assert np.array_equal(raw, want)
        return
    if kind == "fp8":
        inv = np.float32(1) / np.float32(scale)
        y = torch.from_numpy(rows.astype(np.float32) * inv).clamp(-448, 448).to(torch.float8_e4m3fn)
        want = torch.full(tuple(cache.shape), 77, dtype=torch.uint8)
        want[blk, :, off] = y.view(torch.uint8)[torch.from_numpy(keep)]
        assert torch.equal(cache.cpu(), want)
        return
    want = np.full(tuple(cache.shape), 77.0)
    want[blk, :, off] = rows[keep]
    assert np.array_equal(f64(cache), want)


SHAPES = [  # T, Hq, Hkv, d, rot, bs
    (1, 2, 1, 64, 64, 16),
    (5, 64, 8, 128, 128, 16),
    (37, 24, 4, 256, 256, 32),
    (130, 12, 12, 64, 32, 32),
    (33, 3, 1, 128, 80, 16),     # 5 vectors to a half: no power of two
    (19, 8, 2, 256, 64, 16),
    (700, 16, 1, 128, 16, 32),   # the smallest turned part
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("cache", ["bf16", "fp8", "int4"])
def test_rotation_and_append(shape, inter, cache):
    s = Step(*shape, cache, seed=sum(shape))
    assert s.run(inter) == 0
    s.check(inter)


@pytest.mark.parametrize("inter", [False, True])
def test_in_place(inter):
    s = Step(211, 24, 4, 256, 256, 16, "bf16", seed=3, strided=False)
    want = ref.bf16_round(ref.rotate(f64(s.q), s.table, s.pos, inter))
    assert s.run(inter, q_out=s.q) == 0
    assert np.array_equal(f64(s.q), want)


@pytest.mark.parametrize("cache", ["bf16", "fp8", "int4"])
def test_padding_and_places_out_of_range(cache):
    s = Step(40, 8, 2, 128, 128, 16, cache, seed=4)
    s.pos[[0, 7, 39]] = -1          # padding: nothing of the row is written
    s.slots[[3, 4]] = -1            # rotated, not stored
    s.check_before = None
    assert s.run(False) == 0
    s.check(False)
    s = Step(40, 8, 2, 128, 128, 16, cache, seed=5)
    s.pos[[5, 6]] = [300, 2**31 - 1]
    s.slots[9] = s.kc.shape[0] * 16
    s.slots[10] = 2**31 - 1
    assert s.run(True) == ref.RANGE
    s.check(True)


def test_no_tokens():
    s = Step(0, 8, 2, 128, 128, 16, "int4")
    assert s.run(False) == 0
    assert (s.kc == 77).all()


def test_values_next_to_a_bf16_tie():
    """cos = sin = 1/2 and neighbours of odd multiples of a half step: every sum lies on or by a tie."""
    t, d = 64, 64
    s = Step(t, 2, 1, d, d, 16, "bf16", seed=6, strided=False, positions=np.arange(64) % 4)
    rng = np.random.default_rng(6)
    m = rng.integers(128, 256, (t, 2, d)) * 2.0 ** rng.integers(-9, 2, (t, 2, d))
    s.q = bf16(m).cuda()
    s.table = np.zeros((4, d), np.float32)
    s.table[0] = 0.5
    s.table[1] = np.nextafter(np.float32(0.5), np.float32(1))
    s.table[2, :d // 2], s.table[2, d // 2:] = 0.5, -0.5 + 2.0**-25
    s.table[3, :d // 2], s.table[3, d // 2:] = 1.0, 2.0**-9 + 2.0**-33
    assert s.run(False) == 0
    s.check(False)


def test_infinities_turn_into_infinities():
    s = Step(2, 2, 1, 64, 64, 16, "bf16", seed=7, strided=False)
    s.table[:] = 0.5
    s.q[0, 0, 3] = float("inf")      # pairs with dim 35
    s.q[1, 1, 40] = float("nan")     # pairs with dim 8
    s.run(False)
    q = f64(s.q_out)
    assert q[0, 0, 3] == np.inf and q[0, 0, 35] == np.inf
    assert np.isnan(q[1, 1, [8, 40]]).all() and np.isfinite(q).sum() == q.size - 4


# ---- the 4-bit cache -------------------------------------------------------------
@pytest.mark.parametrize("t,hkv,d,bs", [(1, 1, 64, 16), (33, 8, 128, 16), (100, 3, 256, 32), (639, 5, 64, 32)])
def test_int4_append_and_read(t, hkv, d, bs):
    import paged_kv_cache_445_b200 as pa
    rng = np.random.default_rng(t)
    nb = t // bs + 2
    x = bf16(rng.standard_normal((2, t, hkv, d)) * 10.0 ** rng.integers(-6, 5, (2, t, hkv, d // 32, 1)).repeat(32, 4)
             .reshape(2, t, hkv, d)).cuda()
    slots = rng.permutation(nb * bs)[:t].astype(np.int64)
    slots[t // 2] = -1
    kc, vc = (torch.full((nb, hkv, bs, d * 9 // 16), 77, dtype=torch.uint8, device="cuda") for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_cache_append_int4(x[0], x[1], kc, vc, i32(slots), status)
    out = torch.full((2, t, hkv, d), -3.0, device="cuda")
    pa.pa_cache_read_int4(out[0], out[1], kc, vc, i32(slots), status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    live = np.ones(t, bool)
    check_cache(kc, f64(x[0]), slots, live, "int4", bs, 0)
    check_cache(vc, f64(x[1]), slots, live, "int4", bs, 0)
    for i in range(2):
        want = ref.int4_values(*ref.int4_quantise(f64(x[i])))
        want[slots < 0] = -3.0
        assert np.array_equal(out[i].cpu().numpy().astype(np.float64), want)


def test_int4_special_values():
    """Zeros, one outlier, ties, subnormals, the largest bf16, infinities and a NaN in 32 dims of its own."""
    import paged_kv_cache_445_b200 as pa
    d, bs = 256, 16
    x = np.zeros((1, 1, d))
    x[0, 0, 32] = 7.0                                   # one value in zeros
    x[0, 0, 64:96] = np.concatenate([[7], np.arange(31) * 0.5 - 7])  # scale 1: halves are ties
    x[0, 0, 96:128] = 2.0**-130 * np.arange(32)          # the scale underflows to zero
    x[0, 0, 128:160] = 3e38                              # the scale is clamped to 65504
    x[0, 0, 160], x[0, 0, 161], x[0, 0, 162] = np.inf, -np.inf, 1.0
    x[0, 0, 192], x[0, 0, 193] = np.nan, 5.0
    x[0, 0, 224:] = 7 * 2.0**-25 * np.array([1, 3] * 16)  # fp16 subnormal scale, a tie in it
    xb = bf16(x).cuda()
    kc, vc = (torch.zeros((1, 1, bs, d * 9 // 16), dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = i32([5])
    pa.pa_cache_append_int4(xb, xb, kc, vc, slots)
    out = torch.zeros((2, 1, 1, d), device="cuda")
    pa.pa_cache_read_int4(out[0], out[1], kc, vc, slots)
    want = ref.int4_values(*ref.int4_quantise(f64(xb)))
    assert np.array_equal(out[0].cpu().numpy().astype(np.float64), want, equal_nan=True)
    assert np.array_equal(out[1].cpu().numpy().astype(np.float64), want, equal_nan=True)
    got = out[0, 0, 0].cpu().numpy()
    assert np.isnan(got[192:224]).all() and not np.isnan(np.delete(got, np.arange(192, 224))).any()
    assert got[160] == 7 * 65504.0 and got[161] == -7 * 65504.0


def test_int4_slots_out_of_range():
    import paged_kv_cache_445_b200 as pa
    x = bf16(np.ones((3, 2, 64))).cuda()
    kc, vc = (torch.full((2, 2, 16, 36), 77, dtype=torch.uint8, device="cuda") for _ in range(2))
    out = torch.full((2, 3, 2, 64), -3.0, device="cuda")
    for slots in ([32, -1, 2**31 - 1], [-5, 40, -1]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pa.pa_cache_append_int4(x, x, kc, vc, i32(slots), status)
        assert int(status.item()) == ref.RANGE
        status.zero_()
        pa.pa_cache_read_int4(out[0], out[1], kc, vc, i32(slots), status)
        assert int(status.item()) == ref.RANGE
    assert (kc == 77).all() and (vc == 77).all() and (out == -3.0).all()


def test_int4_append_then_rope_append_write_the_same_codes():
    """The fused append gives the codes of the two calls."""
    import paged_kv_cache_445_b200 as pa
    s = Step(77, 8, 4, 128, 128, 16, "int4", seed=12)
    assert s.run(False) == 0
    k = bf16(ref.bf16_round(ref.rotate(f64(s.k), s.table, s.pos, False))).cuda()
    kc, vc = torch.full_like(s.kc, 77), torch.full_like(s.vc, 77)
    pa.pa_cache_append_int4(k, s.v.contiguous(), kc, vc, i32(s.slots))
    assert torch.equal(kc, s.kc) and torch.equal(vc, s.vc)


# ---- the table --------------------------------------------------------------------
def frequencies(rot, base, scaling, factor, orig, low, high, att):
    w, m = [], 1.0
    for i in range(rot // 2):
        x = base ** (-2 * i / rot)
        if scaling == "linear":
            x /= factor
        elif scaling == "ntk":
            x = (base * factor ** (rot / (rot - 2))) ** (-2 * i / rot)
        elif scaling == "yarn":
            at = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
            ramp = min(max((i - a) / max(b - a, 0.001), 0), 1)
            x = x * (1 - ramp) + x / factor * ramp
            m = 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
        elif scaling == "bands":
            turns = orig * x / (2 * math.pi)
            keep = min(max((turns - low) / (high - low), 0), 1)
            x = x * keep + x / factor * (1 - keep)
        w.append(x)
    return np.array(w), att or m


@pytest.mark.parametrize("rot,base,scaling,kw", [
    (128, 10000.0, "none", {}),
    (64, 500000.0, "linear", dict(factor=4.0)),
    (128, 10000.0, "ntk", dict(factor=8.0)),
    (128, 500000.0, "yarn", dict(factor=16.0, original_positions=4096)),
    (80, 10000.0, "yarn", dict(factor=4.0, original_positions=2048, low=2.0, high=20.0, attention_factor=1.25)),
    (16, 10000.0, "yarn", dict(factor=0.5, original_positions=100)),
    (256, 500000.0, "bands", dict(factor=8.0, original_positions=8192)),
    (128, 1e6, "bands", dict(factor=32.0, original_positions=8192, low=0.5, high=2.0)),
])
def test_table(rot, base, scaling, kw):
    import paged_kv_cache_445_b200 as pa
    p = 2500
    table = torch.full((p, rot), -9.0, device="cuda")
    pa.pa_rope_table(table, base, scaling, **kw)
    w, m = frequencies(rot, base, scaling, kw.get("factor", 1.0), kw.get("original_positions", 0),
                       kw.get("low", 1.0), kw.get("high", 4.0 if scaling == "bands" else 32.0),
                       kw.get("attention_factor", 0.0))
    a = np.arange(p)[:, None] * w[None, :]
    want = np.concatenate([np.cos(a), np.sin(a)], 1) * m
    # rounded to binary32 once (half a step of 2^-24 relative, values up to m), angles off by some 2^-52 of themselves
    assert np.abs(table.cpu().numpy() - want).max() <= m * (2.0**-24 + 2500 * 2.0**-50)


def test_far_positions():
    import paged_kv_cache_445_b200 as pa
    p, rot = 1 << 20, 16
    table = torch.empty(p, rot, device="cuda")
    pa.pa_rope_table(table, 10000.0)
    w, _ = frequencies(rot, 10000.0, "none", 1, 0, 1, 32, 0)
    a = np.arange(p - 1000, p)[:, None] * w[None, :]
    want = np.concatenate([np.cos(a), np.sin(a)], 1)
    assert np.abs(table[-1000:].cpu().numpy() - want).max() <= 2.0**-24 + 2.0**20 * 2.0**-50

"""Host-side refusals of the step operators: each answers before any CUDA call
(this machine may have no GPU)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from paged_kv_cache_445_b200 import _binding as b

F, ODD = 4096, 4100  # stand-in pointers: 16-byte aligned, and not
L = b._lib


def test_status_name():
    assert b.pa_status_string(b.PA_ERR_NO_BLOCKS).startswith("PA_ERR_NO_BLOCKS")
    assert b.status_bit(b.PA_ERR_NO_BLOCKS) == 256


def test_step_slots():
    def call(new=F, tables=F, width=8, ring=F, b_=4, nb=10, bs=16, qs=F, pos=F, t=9):
        return L.pa_step_slots(new, F, F, F, F, tables, width, ring, F, F, b_, nb, bs, qs, pos, F, t, None, None)
    for kw in (dict(b_=-1), dict(nb=0), dict(width=0), dict(t=-1), dict(nb=1 << 28), dict(width=1 << 28)):
        assert call(**kw) == b.PA_ERR_SHAPE, kw
    assert call(bs=8) == b.PA_ERR_UNSUPPORTED
    for kw in (dict(new=None), dict(tables=None), dict(ring=None), dict(qs=None), dict(pos=None)):
        assert call(**kw) == b.PA_ERR_NULL, kw


def test_rope_table():
    def call(table=F, n=10, rot=64, base=10000.0, type=0, factor=2.0, orig=4096, low=1.0, high=32.0, att=0.0):
        return L.pa_rope_table(table, n, rot, base, ctypes.byref(b.RopeScaling(type, orig, factor, low, high, att)),
                               None)
    inf, nan = float("inf"), float("nan")
    for kw in (dict(n=-1), dict(base=0.0), dict(base=inf), dict(base=nan), dict(type=1, factor=0.0),
               dict(type=2, factor=inf), dict(type=3, orig=0), dict(type=4, low=4.0, high=4.0), dict(type=4, low=0.0),
               dict(att=-1.0), dict(att=nan), dict(table=ODD), dict(type=3, base=1.0)):
        assert call(**kw) == b.PA_ERR_SHAPE, kw
    for kw in (dict(rot=0), dict(rot=24), dict(rot=272), dict(type=5), dict(type=-1)):
        assert call(**kw) == b.PA_ERR_UNSUPPORTED, kw
    assert call(table=None) == b.PA_ERR_NULL
    assert call(n=0, table=None) == b.PA_OK


@pytest.mark.parametrize("kind", ["", "_fp8", "_int4"])
def test_rope_append(kind):
    def call(qo=F, q=F, qs=8 * 128, ks=2 * 128, vs=2 * 128, kc=F, table=F, tl=100, rot=128, pos=F, t=3, nb=9, hq=8,
             hkv=2, d=128, bs=16, scales=(0.5, 0.25)):
        extra = scales if kind == "_fp8" else ()
        fn = getattr(L, "pa_rope_append" + kind)
        return fn(qo, q, qs, F + 32, ks, F, vs, kc, F, table, tl, rot, 0, pos, F, t, nb, hq, hkv, d, bs, *extra, None,
                  None)
    for kw in (dict(t=-1), dict(nb=0), dict(hq=0), dict(hkv=-1), dict(tl=0), dict(qs=1020), dict(ks=248),
               dict(vs=257), dict(qo=ODD), dict(kc=ODD), dict(table=ODD), dict(qs=2048)):  # the last: in place, strided
        assert call(**kw) == b.PA_ERR_SHAPE, kw
    for kw in (dict(d=96, qs=4096, rot=64), dict(bs=64), dict(rot=0), dict(rot=24), dict(rot=144)):
        assert call(**kw) == b.PA_ERR_UNSUPPORTED, kw
    for kw in (dict(qo=None), dict(kc=None), dict(table=None), dict(pos=None)):
        assert call(**kw) == b.PA_ERR_NULL, kw
    assert call(t=0, q=None) == b.PA_OK
    if kind == "_fp8":
        for s in ((0.0, 1.0), (1.0, -1.0), (float("inf"), 1.0), (1.0, float("nan"))):
            assert call(scales=s) == b.PA_ERR_SHAPE, s


def test_int4_cache():
    for fn in (L.pa_cache_append_int4, L.pa_cache_read_int4):
        def call(a=F, kc=F, sm=F, t=3, nb=9, hkv=2, d=128, bs=16):
            return fn(a, F, kc, F, sm, t, nb, hkv, d, bs, None, None)
        for kw in (dict(t=-1), dict(nb=0), dict(hkv=0), dict(a=ODD), dict(kc=ODD)):
            assert call(**kw) == b.PA_ERR_SHAPE, kw
        for kw in (dict(d=96), dict(bs=8)):
            assert call(**kw) == b.PA_ERR_UNSUPPORTED, kw
        for kw in (dict(a=None), dict(kc=None), dict(sm=None)):
            assert call(**kw) == b.PA_ERR_NULL, kw
        assert call(t=0, a=None) == b.PA_OK


def test_int4_attention():
    def decode(out=F, bt=F, width=4, n=4, hq=8, hkv=2, d=128, bs=16, nb=10, ws=F):
        return L.pa_decode_int4(out, F, F, F, bt, width, F, n, hq, hkv, d, bs, nb, 0.1, ws, 1 << 30, None, None)

    def chunk(qs=F, n=4, t=9):
        return L.pa_prefill_chunk_int4(F, F, qs, F, F, F, 4, F, n, t, 8, 2, 128, 16, 10, 0.1, F, 1 << 30, None, None)
    for kw in (dict(width=0), dict(n=-1), dict(hq=7), dict(hkv=0), dict(nb=0), dict(out=ODD), dict(ws=ODD),
               dict(width=1 << 28)):
        assert decode(**kw) == b.PA_ERR_SHAPE, kw
    for kw in (dict(d=96), dict(bs=8), dict(hq=17, hkv=1), dict(hq=9, hkv=1, d=256)):
        assert decode(**kw) == b.PA_ERR_UNSUPPORTED, kw
    for kw in (dict(out=None), dict(bt=None), dict(ws=None)):
        assert decode(**kw) == b.PA_ERR_NULL, kw
    assert decode(n=0) == b.PA_OK
    assert chunk(qs=None) == b.PA_ERR_NULL and chunk(t=-1) == b.PA_ERR_SHAPE and chunk(t=0) == b.PA_OK
    for args in ((7, 2, 128), (8, 0, 128), (8, 2, 96), (17, 1, 64)):
        assert L.pa_int4_workspace_bytes(*args) == 0, args


def test_accept_drafts():
    def call(out=F, acc=F, target=F, ts=100, draft=F, ds=100, tok=F, qs=F, uni=F, n=3, t=9, v=100, ctx=F, ctx_out=F):
        return L.pa_accept_drafts(out, acc, target, ts, draft, ds, 0, tok, qs, uni, n, t, v, ctx, ctx_out, None, None)
    for kw in (dict(n=-1), dict(t=-1), dict(v=0), dict(ts=99), dict(ds=99), dict(n=2**31 - 1)):
        assert call(**kw) == b.PA_ERR_SHAPE, kw
    for kw in (dict(out=None), dict(acc=None), dict(target=None), dict(tok=None), dict(qs=None), dict(uni=None),
               dict(ctx=None), dict(ctx_out=None)):
        assert call(**kw) == b.PA_ERR_NULL, kw
    assert call(n=0, acc=None) == b.PA_OK


def test_the_binding_checks_its_tensors():
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):  # host tensors
        b.pa_step_slots(t, t, t, t.view(2, 2), t, t, 16, t, t, t)
    with pytest.raises(ValueError):
        b.pa_rope_table(torch.zeros(4, 16), scaling="cubic")
    with pytest.raises(ValueError):
        b.pa_cache_read_int4(t, t, t, t, t)
    with pytest.raises(b.PAError):
        b.pa_int4_workspace_bytes(8, 2, 96)


def test_rope_table_refuses_bounds_without_end():
    inf, nan = float("inf"), float("nan")
    for type in (3, 4):
        for low, high in ((1.0, inf), (1.0, nan), (nan, 32.0), (inf, inf)):
            sc = b.RopeScaling(type, 4096, 2.0, low, high, 0.0)
            assert L.pa_rope_table(F, 10, 64, 10000.0, ctypes.byref(sc), None) == b.PA_ERR_SHAPE, (type, low, high)

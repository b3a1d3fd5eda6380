"""Plain 64-bit restatements of the step operators, for the tests: request
lengths to tables and slots, rotary positions, the 4-bit cache format, draft
verification.  Written from their definitions in include/pa.h, row by row."""
from __future__ import annotations

import math

import numpy as np

I32_MAX = 2**31 - 1
RANGE, NO_BLOCKS = 1 << 5, 1 << 8


def step_slots(new, ctx, held, tables, ring, state, bs, max_tokens):
    """Sequential walk over the batch; returns a dict of all results and the status bits."""
    nb, width = len(ring), tables.shape[1]
    tables, ring = tables.copy(), ring.copy()
    ctx_out, held_out = ctx.copy(), held.copy()
    head, count = int(state[0]), int(state[1])
    bits = 0
    bad = not (0 <= head < nb and 0 <= count <= nb)
    if bad:
        bits |= RANGE
        head, count = 0, 0
    qs = [0]
    pos = np.full(max_tokens, -1, np.int32)
    slot = np.full(max_tokens, -1, np.int32)
    need_sum = taken = back_sum = 0
    for s in range(len(new)):
        n, c, h = int(new[s]), int(ctx[s]), int(held[s])
        start = qs[-1]
        qs.append(start + max(n, 0))
        after = c + n
        if c < 0 or h < -(-c // bs) or h > width or after < 0:
            bits |= RANGE
            continue
        blocks = -(-after // bs)
        if n < 0:
            if bad:
                continue
            for j in range(blocks, h):
                if count + back_sum >= nb:
                    bits |= RANGE
                else:
                    ring[(head + count + back_sum) % nb] = tables[s, j]
                back_sum += 1
            ctx_out[s], held_out[s] = after, h - max(0, h - blocks)
            continue
        if blocks > width or qs[-1] > max_tokens:
            bits |= RANGE
            continue
        need = max(0, blocks - h)
        need_sum += need
        if need and need_sum > count:
            bits |= NO_BLOCKS
            continue
        for j in range(need):
            tables[s, h + j] = ring[(head + taken + j) % nb]
        taken += need
        ctx_out[s], held_out[s] = after, h + need
        for i in range(n):
            pos[start + i] = c + i
            b = int(tables[s, (c + i) // bs])
            if 0 <= b < nb:
                slot[start + i] = b * bs + (c + i) % bs
            else:
                bits |= RANGE
    state_out = np.array([(head + taken) % nb, min(nb, count - taken + back_sum)], np.int32)
    if bad:
        state_out = np.array(state, np.int32)
    return dict(query_start=np.minimum(qs, I32_MAX).astype(np.int32), positions=pos, slots=slot, tables=tables,
                ring=ring, ctx=ctx_out, held=held_out, state=state_out), bits


def bf16_round(x):
    """float64 -> the bf16 value nearest to it (ties to even), as float64; normal range only."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, 8)), e - 8)


def rotate(x, table, pos, interleaved):
    """x [T, H, d] float64, table [P, rot] float32: the exact rotation (products of at most 32 bits)."""
    rot = table.shape[1]
    h = rot // 2
    out = x.copy()
    for t, p in enumerate(pos):
        if p < 0:
            continue
        c, s = table[p, :h].astype(np.float64), table[p, h:].astype(np.float64)
        a, b = (x[t, :, 0:rot:2], x[t, :, 1:rot:2]) if interleaved else (x[t, :, :h], x[t, :, h:rot])
        ya, yb = a * c - b * s, b * c + a * s
        if interleaved:
            out[t, :, 0:rot:2], out[t, :, 1:rot:2] = ya, yb
        else:
            out[t, :, :h], out[t, :, h:rot] = ya, yb
    return out


def int4_quantise(x):
    """[..., d] float64 (bf16 values) -> codes 1..15, fp16 scales [..., d / 32]."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    nan = np.isnan(b).any(-1)
    with np.errstate(all="ignore"):
        s = np.minimum(np.abs(b).max(-1) / 7.0, 65504.0).astype(np.float16)
        f = s.astype(np.float64)[..., None]
        n = np.where(f > 0, np.rint(b / f), 0.0)
    n = np.where(np.isnan(n), 0.0, np.clip(n, -7, 7))
    s = np.where(nan, np.float16(np.nan), s)
    return (n + 8).astype(np.uint8).reshape(x.shape), s


def int4_values(codes, scales):
    b = codes.reshape(*codes.shape[:-1], -1, 32).astype(np.float64) - 8.0
    return (b * scales.astype(np.float64)[..., None]).reshape(codes.shape)


def int4_places(bs, d):
    """(byte, shift) of every (row, dim) of a record, and the byte of every (row, chunk)'s scale."""
    n = d // 32
    byte = np.zeros((bs, d), np.int64)
    shift = np.zeros((bs, d), np.int64)
    scale = np.zeros((bs, n), np.int64)
    for r in range(bs):
        for c in range(n):
            scale[r, c] = bs * d // 2 + (r * n + c) * 2
            place = c ^ ((r // (8 // n)) % n)
            for i in range(32):
                byte[r, c * 32 + i] = r * (d // 2) + place * 16 + 2 * (i % 8) + i // 16
                shift[r, c * 32 + i] = 4 * (i // 8 % 2)
    return byte, shift, scale


def int4_pack(codes, scales):
    """codes [NB, H, bs, d], scales [NB, H, bs, d / 32] -> the cache's bytes [NB, H, bs, 9 d / 16]."""
    nb, h, bs, d = codes.shape
    byte, shift, scale = int4_places(bs, d)
    rec = np.zeros((nb, h, bs * d * 9 // 16), np.uint8)
    for half in (0, 4):
        sel = shift == half
        rec[:, :, byte[sel]] |= codes[:, :, sel] << half
    raw = np.ascontiguousarray(scales.astype(np.float16)).view(np.uint8).reshape(nb, h, bs, d // 32, 2)
    rec[:, :, scale], rec[:, :, scale + 1] = raw[..., 0], raw[..., 1]
    return rec.reshape(nb, h, bs, d * 9 // 16)


def int4_unpack(cache, bs, d):
    """The cache's bytes -> values [NB, H, bs, d] in float64."""
    nb, h = cache.shape[:2]
    byte, shift, scale = int4_places(bs, d)
    rec = cache.reshape(nb, h, -1)
    codes = (rec[:, :, byte] >> shift) & 15
    raw = np.ascontiguousarray(np.stack([rec[:, :, scale], rec[:, :, scale + 1]], -1)).view(np.float16)[..., 0]
    return int4_values(codes.astype(np.uint8), raw)


def attention(q, k, v, tables, ctx, query_start, scale, bs):
    """q [T, Hq, d]; k, v values [NB, Hkv, bs, d]; zeros for a row without keys."""
    hq, hkv = q.shape[1], k.shape[1]
    out = np.zeros(q.shape)
    for s in range(len(ctx)):
        rows = int(query_start[s + 1] - query_start[s])
        idx = tables[s, :-(-int(ctx[s]) // bs)]
        ks = k[idx].transpose(1, 0, 2, 3).reshape(hkv, -1, q.shape[2])
        vs = v[idx].transpose(1, 0, 2, 3).reshape(hkv, -1, q.shape[2])
        for i in range(rows):
            m = int(ctx[s]) - rows + i + 1
            if m <= 0:
                continue
            t = int(query_start[s]) + i
            for h in range(hq):
                g = h // (hq // hkv)
                z = ks[g, :m] @ q[t, h] * scale
                p = np.exp(z - z.max())
                out[t, h] = p @ vs[g, :m] / p.sum()
    return out


def accept(target, draft, tokens, query_start, uniforms):
    """(out_tokens with -9 where nothing is written, num_accepted, status bits)."""
    out = np.full(len(tokens), -9, np.int64)
    acc_out, bits = [], 0
    vocab = target.shape[1]

    def clean(w):
        return np.where((w > 0) & np.isfinite(w), w, 0.0)

    for s in range(len(query_start) - 1):
        a, b = int(query_start[s]), int(query_start[s + 1])
        rows = b - a
        if rows <= 0 or a < 0 or b > len(tokens):
            if rows < 0 or a < 0 or b > len(tokens):
                bits |= RANGE
            acc_out.append(0)
            continue
        acc, refused = rows - 1, -1
        for i in range(rows - 1):
            d = int(tokens[a + i + 1])
            if d < 0 or d >= vocab:
                bits |= RANGE if d >= vocab else 0
                acc = i
                break
            p = float(target[a + i, d])
            q = 1.0 if draft is None else float(draft[a + i, d])
            if not float(uniforms[a + i]) * q < p:
                acc, refused = i, d
                break
        w = np.asarray(target[a + acc], np.float64)
        if refused >= 0:
            if draft is None:
                rest = clean(w)
                rest[refused] = 0.0
            else:
                rest = clean(w - np.asarray(draft[a + acc], np.float64))
            w = rest if rest.sum() > 0 else clean(w)
        else:
            w = clean(w)
        total = math.fsum(w)
        run = np.cumsum(w)
        hit = np.nonzero((run > float(uniforms[b - 1]) * total) & (w > 0))[0]
        some = np.nonzero(w > 0)[0]
        if len(hit):
            tok = int(hit[0])
        elif len(some):
            tok = int(some[-1])
        else:
            tok, bits = -1, bits | RANGE
        out[a:a + acc] = tokens[a + 1:a + 1 + acc]
        out[a + acc] = tok
        out[a + acc + 1:b] = -1
        acc_out.append(acc)
    return out, np.array(acc_out, np.int64), bits

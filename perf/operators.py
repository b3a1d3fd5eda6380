"""Cases of the serving-step operators around paged attention, with plain forms.

Four operators carry one engine step on the GPU, from request lengths to
accepted tokens:

* ``slots``  -- block tables, positions and slot mapping built from request
  lengths and a queue of free blocks (``pa_step_slots``);
* ``rope``, ``table`` -- rotary positions applied to a step's q and k while the
  rows go into the cache (``pa_rope_append``, ``_fp8``, ``_int4``), and the
  table of angles behind them (``pa_rope_table``);
* ``append4``, ``attn4`` -- a cache held in 4 bits: quantising append and read
  back (``pa_cache_append_int4``, ``pa_cache_read_int4``), decode and varlen
  attention over it (``pa_decode_int4``, ``pa_prefill_chunk_int4``);
* ``accept`` -- verification of drafted tokens against the target's
  probabilities (``pa_accept_drafts``).

``own`` False: the plain forms, elementary torch operations.  ``own`` True: the
package's calls.  ``exact`` computes the same definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
WORKSPACE = 160 << 20  # bytes a serving program sets aside for pa_decode_int4 / pa_prefill_chunk_int4


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of a full batch: one new token per sequence, a few new blocks
        dict(name="slots-decode-b128", op="slots", B=128, mode="decode", ctx=1500, bs=16),
        # an offline engine: 2000 requests, prompts up to 2000 tokens, drafts, idle and finished ones
        dict(name="slots-mixed-b2000", op="slots", B=2000, mode="mixed", ctx=1500, bs=32),
        # the rotary step of a decode batch, 64 query and 8 KV heads, bf16 cache
        dict(name="rope-bf16-decode-b128", op="rope", cache="bf16", T=128, Hq=64, Hkv=8, d=128, rot=128, inter=False,
             bs=16),
        # prefill of several prompts into an FP8 cache, interleaved pairs on half of the head
        dict(name="rope-fp8-partial-t1111", op="rope", cache="fp8", T=1111, Hq=24, Hkv=4, d=256, rot=128, inter=True,
             bs=32),
        # a long prefill into a 4-bit cache, rows read back for a prefix transfer
        dict(name="rope-int4-prefill-t8192", op="rope", cache="int4", T=8192, Hq=32, Hkv=8, d=128, rot=128, inter=False,
             bs=16),
        # the table of a long-context model, set up once: 131072 positions, YaRN
        dict(name="table-yarn-131072", op="table", P=131072, rot=128, base=500000.0, scaling="yarn", factor=8.0,
             orig=16384),
        # four short chats: latency
        dict(name="attn4-decode-b4", op="attn4", B=4, Hq=32, Hkv=8, d=128, bs=16, lo=5, hi=64, rows=1),
        # the headline decode batch: lognormal contexts, 64 query and 8 KV heads
        dict(name="attn4-decode-b128", op="attn4", B=128, Hq=64, Hkv=8, d=128, bs=16, lo=0, hi=8192, rows=1),
        # two very long documents, head_dim 256
        dict(name="attn4-decode-long-d256", op="attn4", B=2, Hq=24, Hkv=4, d=256, bs=32, lo=90000, hi=120000, rows=1),
        # drafts verified over the 4-bit cache: up to 5 rows a sequence, some without rows
        dict(name="attn4-verify-b64", op="attn4", B=64, Hq=64, Hkv=8, d=128, bs=16, lo=256, hi=4096, rows=5),
        # four drafts for each of 128 sequences against the target's probabilities
        dict(name="accept-b128-v128000", op="accept", B=128, k=4, V=128000, t="float32", draft=True),
        # one chat, drafts found by lookup (no draft probabilities)
        dict(name="accept-b1-v32000", op="accept", B=1, k=7, V=32000, t="float32", draft=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["slots", "rope", "rope", "append4", "attn4", "attn4", "attn4", "accept", "table"])
    Hq, Hkv, d = rng.choice([(64, 8, 128), (32, 8, 128), (24, 4, 256), (2, 1, 64), (12, 12, 64), (30, 6, 128),
                             (24, 2, 128), (16, 1, 128)])
    bs = rng.choice([16, 32])
    if op == "slots":
        return dict(op=op, B=_log(rng, 1, 2000), mode=rng.choice(["decode", "mixed"]), ctx=_log(rng, 20, 1500), bs=bs)
    if op == "rope":
        return dict(op=op, cache=rng.choice(["bf16", "fp8", "int4"]), T=_log(rng, 1, 4500), Hq=Hq, Hkv=Hkv, d=d,
                    rot=rng.choice([32, d // 2, d]), inter=rng.random() < 0.5, bs=bs)
    if op == "table":
        return dict(op=op, P=_log(rng, 500, 100000), rot=rng.choice([32, 64, 80, 128]),
                    base=rng.choice([10000.0, 500000.0]), scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                    factor=rng.choice([2.0, 4.0, 8.0, 32.0]), orig=rng.choice([2048, 8192]))
    if op == "append4":
        return dict(op=op, T=_log(rng, 1, 6000), Hkv=Hkv, d=d, bs=bs)
    if op == "attn4":
        rows = rng.choice([1, 1, 4, 9, 40])
        hi = _log(rng, 30, 3500)
        B = _log(rng, 1, 128 if rows < 10 else 12)
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, bs=bs, lo=1, hi=hi, rows=rows)
    return dict(op=op, B=_log(rng, 1, 100), k=rng.randint(1, 8), V=rng.choice([997, 32000, 50001, 100003, 128000]),
                t=rng.choice(["float32", "bfloat16"]), draft=rng.random() < 0.7)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 445)
    return g


def _randint(g, lo, hi, shape):  # lo .. hi inclusive
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV)


def _shuffled(g, values):
    return torch.tensor(values, device=DEV)[torch.randperm(len(values), generator=g, device=DEV)]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = _gen(seed)
    st = {"case": dict(case)}
    op = case["op"]
    if op == "slots":
        _prepare_slots(st, case, g)
    elif op in ("rope", "append4"):
        _prepare_rows(st, case, g)
    elif op == "table":
        st["table"] = torch.empty(case["P"], case["rot"], device=DEV)
        # another seed: another fine-tuned base, as models of one family have
        st["base"] = case["base"] * (1.0 + (int(seed) % 97) / 97.0)
    elif op == "attn4":
        _prepare_attn4(st, case, g)
    else:
        _prepare_accept(st, case, g)
    return st


def _lengths(g, case, B):
    if case.get("lo", 1) == 0:  # the lognormal mix of the headline batch
        z = torch.randn(B, generator=g, device=DEV, dtype=torch.float64)
        return torch.exp(math.log(1500) + 0.8 * z).round().clamp(16, case["hi"]).long()
    return _randint(g, case["lo"], case["hi"], (B,))


def _prepare_slots(st, case, g):
    B, bs = case["B"], case["bs"]
    ctx = _randint(g, 0, 2 * case["ctx"], (B,))
    if case["mode"] == "decode":
        n = torch.ones(B, dtype=torch.long, device=DEV)
    else:
        kind = torch.rand(B, generator=g, device=DEV)
        n = torch.where(kind < 0.55, 1, 0)                                      # decodes; the rest idle
        n = torch.where((kind >= 0.55) & (kind < 0.75), _randint(g, 2, 8, (B,)), n)  # drafts
        new = (kind >= 0.75) & (kind < 0.85)                                    # prompts
        ctx = torch.where(new, 0, ctx)
        n = torch.where(new, _randint(g, 1, 2000, (B,)), n)
        n = torch.where((kind >= 0.85) & (kind < 0.93), -ctx, n)                # finished
        back = torch.minimum(ctx, _randint(g, 1, 40, (B,)))
        n = torch.where((kind >= 0.93) & (kind < 0.97), -back, n)               # rolled back
    held = (ctx + bs - 1) // bs
    spare = (torch.rand(B, generator=g, device=DEV) < 0.1).long()              # a block kept from a rejected draft
    held = held + spare
    width = int(((2 * case["ctx"] + 2000) + bs - 1) // bs) + 2
    new_rows = 0 if case["mode"] == "decode" else 125
    NB = int(1.25 * B * ((case["ctx"] + new_rows) / bs + 2) + (4 * case["ctx"] + 4000) / bs) + 8
    ids = torch.randperm(NB, generator=g, device=DEV)
    col = torch.arange(width, device=DEV)
    used = col[None, :] < held[:, None]
    tables = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    total = int(held.sum().item())
    tables[used] = ids[:total].int()
    head = int(_randint(g, 0, NB - 1, (1,)).item())
    ring = torch.full((NB,), -1, dtype=torch.int32, device=DEV)
    at = (head + torch.arange(NB - total, device=DEV)) % NB
    ring[at] = ids[total:].int()
    Tmax = B + 64 if case["mode"] == "decode" else 130 * B + 4000  # the step's token budget
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    st.update(new_tokens=i32(n), context_lens=i32(ctx), blocks_held=i32(held), block_tables=tables, free_blocks=ring,
              free_state=torch.tensor([head, NB - total], dtype=torch.int32, device=DEV),
              context_out=torch.empty(B, dtype=torch.int32, device=DEV),
              held_out=torch.empty(B, dtype=torch.int32, device=DEV),
              state_out=torch.empty(2, dtype=torch.int32, device=DEV),
              query_start=torch.empty(B + 1, dtype=torch.int32, device=DEV),
              positions=torch.empty(Tmax, dtype=torch.int32, device=DEV),
              slots=torch.empty(Tmax, dtype=torch.int32, device=DEV))


def _angles(P, rot, base):
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(P, dtype=torch.float64, device=DEV)[:, None] * inv[None, :]
    return torch.cat([a.cos(), a.sin()], dim=1).float().contiguous()


def _prepare_rows(st, case, g):
    T, Hkv, d, bs = case["T"], case["Hkv"], case["d"], case["bs"]
    Hq = case.get("Hq", 0)
    # one projection's output, [T, (Hq + 2 Hkv) d]: q, k and v are views of it
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g, device=DEV)
    gain = torch.exp(0.7 * torch.randn(1, Hq + 2 * Hkv, d, generator=g, device=DEV))  # channels of unequal size
    qkv = (qkv * gain).to(torch.bfloat16)
    cache = case.get("cache", "int4")
    NB = (T + bs - 1) // bs + 3
    slots = torch.randperm(NB * bs, generator=g, device=DEV)[:T]
    pad = torch.rand(T, generator=g, device=DEV) < 0.01
    slots = torch.where(pad, -1, slots).int()
    st.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], slots=slots, bs=bs, pad=pad,
              k_scale=0.0625, v_scale=0.03125)
    if case["op"] == "append4":
        st.update(k=st["k"].contiguous(), v=st["v"].contiguous())
    else:
        P = 16384
        st["table"] = _angles(P, case["rot"], 10000.0)
        first = int(_randint(g, 0, P - T, (1,)).item()) if T > 256 else 0  # one long chunk, else a batch of decodes
        pos = first + torch.arange(T, device=DEV) if T > 256 else _randint(g, 0, P - 1, (T,))
        st["positions"] = torch.where(pad, -1, pos).int()
        st["q_out"] = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device=DEV)
    if cache == "bf16":
        shape, dtype = (NB, Hkv, bs, d), torch.bfloat16
    elif cache == "fp8":
        shape, dtype = (NB, Hkv, bs, d), torch.uint8
    else:
        shape, dtype = (NB, Hkv, bs, d * 9 // 16), torch.uint8
        st["k_read"] = torch.zeros(T, Hkv, d, device=DEV)
        st["v_read"] = torch.zeros(T, Hkv, d, device=DEV)
    st["k_cache"] = torch.zeros(shape, dtype=dtype, device=DEV)
    st["v_cache"] = torch.zeros(shape, dtype=dtype, device=DEV)


def _pack4(u, s):
    """Codes u [NB, Hkv, bs, d] (0..15, value u - 8) and fp16 scales s [NB, Hkv, bs, d/32] -> the cache's bytes
    [NB, Hkv, bs, 9 d / 16].  Byte 2 i + h of a 32-dim chunk holds dims i + 16 h (low nibble) and i + 16 h + 8; the
    16-byte chunk c of row r stands at position c ^ (r // (8 / (d/32)) % (d/32)); a block's scales follow its codes."""
    NB, H, bs, d = u.shape
    n = d // 32
    w = u.to(torch.uint8).view(NB, H, bs, n, 2, 2, 8)                # chunk, h, low/high, i
    b = (w[:, :, :, :, :, 0] | (w[:, :, :, :, :, 1] << 4)).transpose(4, 5).reshape(NB, H, bs, n, 16)
    r = torch.arange(bs, device=u.device)
    at = torch.arange(n, device=u.device)[None, :] ^ ((r // (8 // n)) % n)[:, None]  # an involution
    b = torch.gather(b, 3, at[None, None, :, :, None].expand(NB, H, bs, n, 16))
    codes = b.reshape(NB, H, bs * d // 2)
    sc = s.to(torch.float16).contiguous().view(torch.uint8).reshape(NB, H, bs * n * 2)
    return torch.cat([codes, sc], dim=2).view(NB, H, bs, d * 9 // 16).contiguous()


def _unpack4(c, bs, d):
    """The inverse of _pack4, as values [.., bs, d] in fp32 (exact: 4-bit code times 11-bit scale)."""
    n = d // 32
    flat = c.reshape(*c.shape[:-2], bs * d * 9 // 16)
    codes = flat[..., :bs * d // 2].reshape(*flat.shape[:-1], bs, n, 16)
    s = flat[..., bs * d // 2:].contiguous().view(torch.float16).reshape(*flat.shape[:-1], bs, n)
    r = torch.arange(bs, device=c.device)
    at = torch.arange(n, device=c.device)[None, :] ^ ((r // (8 // n)) % n)[:, None]
    codes = torch.gather(codes, -2, at[:, :, None].expand(codes.shape))
    by = codes.reshape(*codes.shape[:-1], 8, 2).transpose(-1, -2)    # h, i
    u = torch.stack([by & 15, by >> 4], dim=-2)                      # h, low/high, i
    return ((u.float() - 8.0).reshape(*codes.shape[:-1], 32) * s.float()[..., None]).flatten(-2)


def _prepare_attn4(st, case, g):
    B, Hq, Hkv, d, bs = case["B"], case["Hq"], case["Hkv"], case["d"], case["bs"]
    ctx = _lengths(g, case, B)
    if case["rows"] == 1:
        n = torch.ones(B, dtype=torch.long, device=DEV)
    else:
        n = _shuffled(g, [(case["rows"] - i) % (case["rows"] + 1) for i in range(B)])
        ctx = torch.maximum(ctx, n)
    blocks = (ctx + bs - 1) // bs
    width = int(blocks.max().item())
    total = int(blocks.sum().item())
    NB = int(total * 1.25) + 1
    ids = torch.randperm(NB, generator=g, device=DEV)[:total].int()
    tables = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    tables[torch.arange(width, device=DEV)[None, :] < blocks[:, None]] = ids

    def cache():
        u = torch.randn(NB, Hkv, bs, d, generator=g, device=DEV, dtype=torch.float16).mul_(3.0).add_(8.0).round_()
        u = u.clamp_(1, 15).to(torch.uint8)
        s = torch.rand(NB, Hkv, bs, d // 32, generator=g, device=DEV) * 0.3 + 0.2
        return _pack4(u, s)

    T = int(n.sum().item())
    q = (torch.randn(T, Hq, d, generator=g, device=DEV) * 0.5).to(torch.bfloat16)
    qs = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    qs[1:] = torch.cumsum(n, 0)
    st.update(q=q, k_cache=cache(), v_cache=cache(), tables=tables, ctx=ctx.int(), qs=qs, out=torch.zeros_like(q),
              scale=1.0 / math.sqrt(d), workspace=torch.zeros(WORKSPACE, dtype=torch.uint8, device=DEV),
              max_rows=int(n.max().item()), max_ctx=int(ctx.max().item()))


def _prepare_accept(st, case, g):
    B, k, V = case["B"], case["k"], case["V"]
    dt = getattr(torch, case["t"])
    n = _shuffled(g, [k + 1 - i % (k + 1) for i in range(B)])
    T = int(n.sum().item())
    z = torch.randn(T, V, generator=g, device=DEV) * 2.5
    # row r's draft token stands at row r + 1
    if case["draft"]:
        target = torch.softmax(z, dim=1).to(dt)
        z += torch.randn(T, V, generator=g, device=DEV) * 0.6  # the draft model: near the target
        draft = torch.softmax(z, dim=1)
        u = torch.rand(T, 1, generator=g, device=DEV, dtype=torch.float64)
        pick = torch.searchsorted(torch.cumsum(draft.double(), 1), u).clamp(max=V - 1)[:, 0]
    else:  # a text that repeats itself: the target is nearly sure of the token that was looked up
        draft = z
        pick = _randint(g, 0, V - 1, (T,))
        z[torch.arange(T, device=DEV), pick] += 2.5 * math.log(V)
        target = torch.softmax(z, dim=1).to(dt)
    del z
    tokens = torch.zeros(T, dtype=torch.int32, device=DEV)
    tokens[1:] = pick[:-1].int()
    qs = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    qs[1:] = torch.cumsum(n, 0)
    st.update(target=target, draft=draft.to(dt) if case["draft"] else None, tokens=tokens, qs=qs,
              uniforms=torch.rand(T, generator=g, device=DEV), rows=k + 1,
              ctx=_randint(g, k + 1, 4000, (B,)).int(), ctx_out=torch.empty(B, dtype=torch.int32, device=DEV),
              out=torch.empty(T, dtype=torch.int32, device=DEV), accepted=torch.empty(B, dtype=torch.int32, device=DEV))


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        import paged_kv_cache_445_b200 as pa
        if op == "slots":
            return _own_slots(pa, st)
        if op == "table":
            c = st["case"]
            pa.pa_rope_table(st["table"], st["base"], c["scaling"], factor=c["factor"], original_positions=c["orig"])
            return st["table"]
        if op == "rope":
            return _own_rope(pa, st)
        if op == "append4":
            pa.pa_cache_append_int4(st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"])
            pa.pa_cache_read_int4(st["k_read"], st["v_read"], st["k_cache"], st["v_cache"], st["slots"])
            return st["k_read"], st["v_read"]
        if op == "attn4":
            return _own_attn4(pa, st)
        return _own_accept(pa, st)
    return {"slots": _plain_slots, "table": _plain_table, "rope": _plain_rope, "append4": _plain_append4,
            "attn4": _plain_attn4, "accept": _plain_accept}[op](st)


def _own_slots(pa, st):
    pa.pa_step_slots(st["new_tokens"], st["context_lens"], st["blocks_held"], st["block_tables"], st["free_blocks"],
                     st["free_state"], st["case"]["bs"], st["query_start"], st["positions"], st["slots"],
                     context_lens_out=st["context_out"], blocks_held_out=st["held_out"],
                     free_state_out=st["state_out"])
    return _slots_out(st)


def _slots_out(st):
    return {k: st[k] for k in ("query_start", "positions", "slots", "block_tables", "free_blocks", "context_out",
                               "held_out", "state_out")}


def _own_rope(pa, st):
    c = st["case"]
    args = (st["q_out"], st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["positions"],
            st["slots"])
    if c["cache"] == "bf16":
        pa.pa_rope_append(*args, interleaved=c["inter"])
        return st["q_out"], st["k_cache"], st["v_cache"]
    if c["cache"] == "fp8":
        pa.pa_rope_append_fp8(*args, st["k_scale"], st["v_scale"], interleaved=c["inter"])
        return _fp8_out(st)
    pa.pa_rope_append_int4(*args, interleaved=c["inter"])
    pa.pa_cache_read_int4(st["k_read"], st["v_read"], st["k_cache"], st["v_cache"], st["slots"])
    return st["q_out"], st["k_read"], st["v_read"]


def _fp8_out(st):
    k, v = st["k_cache"].view(torch.float8_e4m3fn).float(), st["v_cache"].view(torch.float8_e4m3fn).float()
    return st["q_out"], k * st["k_scale"], v * st["v_scale"]


def _own_attn4(pa, st):
    if st["case"]["rows"] == 1:
        pa.pa_decode_int4(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["ctx"], st["scale"],
                          st["workspace"])
    else:
        pa.pa_prefill_chunk_int4(st["out"], st["q"], st["qs"], st["k_cache"], st["v_cache"], st["tables"], st["ctx"],
                                 st["scale"], st["workspace"])
    return st["out"]


def _own_accept(pa, st):
    pa.pa_accept_drafts(st["out"], st["accepted"], st["target"], st["draft"], st["tokens"], st["qs"], st["uniforms"],
                        context_lens=st["ctx"], context_lens_out=st["ctx_out"])
    return st["out"], st["accepted"], st["ctx_out"]


# ------------------------------------------------------------------ plain forms
def _plain_slots(st):
    bs = st["case"]["bs"]
    n, ctx, held = (st[k].long() for k in ("new_tokens", "context_lens", "blocks_held"))
    tables, ring = st["block_tables"], st["free_blocks"]
    B, width = tables.shape
    NB, T = ring.shape[0], st["positions"].shape[0]
    head, count = st["free_state"].long()
    rows = n.clamp(min=0)
    end = torch.cumsum(rows, 0)
    qs = torch.cat([torch.zeros_like(end[:1]), end])
    after = ctx + n
    blocks = (after.clamp(min=0) + bs - 1) // bs
    fits = (n >= 0) & (blocks <= width) & (end <= T)
    need = torch.where(fits, (blocks - held).clamp(min=0), 0)
    upto = torch.cumsum(need, 0)
    served = fits & ((need == 0) | (upto <= count))
    take = torch.where(served, need, 0)
    drops = (n < 0) & (after >= 0)
    back = torch.where(drops, (held - blocks).clamp(min=0), 0)
    # rows
    t = torch.arange(T, device=n.device)
    s = torch.searchsorted(end, t, right=True).clamp(max=B - 1)
    ok = (t < end[-1]) & served[s]
    pos = ctx[s] + (t - qs[s])
    blk = pos // bs
    fresh = blk >= held[s]
    k = upto[s] - need[s] + blk - held[s]
    taken = ring[torch.where(fresh & ok, (head + k) % NB, 0)].long()
    here = tables[s, blk.clamp(max=width - 1)].long()
    block = torch.where(fresh, taken, here)
    st["positions"].copy_(torch.where(ok, pos, -1))
    st["slots"].copy_(torch.where(ok, block * bs + pos % bs, -1))
    # released blocks go to the queue's tail, in order of sequence and position
    col = torch.arange(width, device=n.device)
    gone = (col[None, :] >= (held - back)[:, None]) & (col[None, :] < held[:, None])
    place = (head + count + torch.cumsum(back, 0) - back)[:, None] + col[None, :] - (held - back)[:, None]
    ring[(place % NB)[gone]] = tables[gone]
    # taken blocks into the tables
    got = (col[None, :] >= held[:, None]) & (col[None, :] < (held + take)[:, None])
    k = (upto - need)[:, None] + col[None, :] - held[:, None]
    tables[got] = ring[((head + k) % NB)[got]]
    st["query_start"].copy_(qs)
    st["context_out"].copy_(torch.where(served | drops, after, ctx))
    st["held_out"].copy_(held + take - back)
    st["state_out"].copy_(torch.stack([(head + take.sum()) % NB, count - take.sum() + back.sum()]))
    return _slots_out(st)


def _inv_freq(c, base):
    """Angles per position (float64) and the factor on cos and sin, for each scaling."""
    rot, f, orig = c["rot"], c["factor"], c["orig"]
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=DEV)
    if c["scaling"] == "ntk":
        base = base * f ** (rot / (rot - 2.0))
    inv = base ** (-i / rot)
    if c["scaling"] == "linear":
        return inv / f, 1.0
    if c["scaling"] == "yarn":
        at = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = ((i / 2 - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return inv / f * ramp + inv * (1 - ramp), 0.1 * math.log(f) + 1.0 if f > 1 else 1.0
    if c["scaling"] == "bands":
        turns = orig * inv / (2 * math.pi)  # whole turns within the trained context
        smooth = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return (1 - smooth) * inv / f + smooth * inv, 1.0
    return inv, 1.0


def _plain_table(st):
    inv, m = _inv_freq(st["case"], st["base"])
    a = torch.arange(st["case"]["P"], dtype=torch.float64, device=DEV)[:, None] * inv[None, :]
    return torch.cat([a.cos() * m, a.sin() * m], dim=1).float()


def _to_bf16(x):
    """float64 -> bf16, rounded once (through fp32 a value next to a tie would be rounded twice)."""
    f = x.float()
    tie = (f.view(torch.int32) & 0xFFFF) == 0x8000
    side = torch.sign(x.abs() - f.double().abs()).int()
    return (f.view(torch.int32) + torch.where(tie, side, torch.zeros_like(side))).view(torch.float32).bfloat16()


def _rotate(x, table, pos, inter):
    """x [T, H, d] in 64 bits (angles of far positions, values next to a border of the cache's codes)."""
    rot = table.shape[1]
    h = rot // 2
    row = table[pos.clamp(min=0).long()].double()[:, None, :]
    c, s = row[..., :h], row[..., h:]
    x = x.double()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :h], x[..., h:rot])
    y, z = a * c - b * s, b * c + a * s
    y = torch.stack([y, z], dim=-1).flatten(-2) if inter else torch.cat([y, z], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _quantise4(x):
    """bf16 [T, Hkv, d] -> (codes 1..15, fp16 scales): scale = max|x| / 7 of 32 dims, code = 8 + round(x / scale)."""
    b = x.float().unflatten(-1, (-1, 32))
    s = (b.abs().amax(-1) / 7.0).clamp(max=65504.0).half()
    f = s.float()[..., None]
    u = torch.where(f > 0, (b / f).round().clamp(-7, 7), torch.zeros_like(b)) + 8.0
    return u.flatten(-2), s


def _plain_rope(st):
    c = st["case"]
    live = st["positions"] >= 0
    q = _to_bf16(_rotate(st["q"], st["table"], st["positions"], c["inter"]))
    k = _to_bf16(_rotate(st["k"], st["table"], st["positions"], c["inter"]))
    st["q_out"][live] = q[live]
    keep = live & (st["slots"] >= 0)
    if c["cache"] == "int4":
        return (st["q_out"],) + _read_back(st, keep, _quantise4(k), _quantise4(st["v"]))
    slot = st["slots"][keep].long()
    blk, off = slot // c["bs"], slot % c["bs"]
    v = st["v"]
    if c["cache"] == "fp8":
        k = (k.float() * (1.0 / st["k_scale"])).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v.float() * (1.0 / st["v_scale"])).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    st["k_cache"][blk, :, off] = k[keep]
    st["v_cache"][blk, :, off] = v[keep]
    return _fp8_out(st) if c["cache"] == "fp8" else (st["q_out"], st["k_cache"], st["v_cache"])


def _read_back(st, keep, kq, vq):
    for out, (u, s) in ((st["k_read"], kq), (st["v_read"], vq)):
        x = ((u - 8.0).unflatten(-1, (-1, 32)) * s.float()[..., None]).flatten(-2)
        out[keep] = x[keep]
    return st["k_read"], st["v_read"]


def _plain_append4(st):
    return _read_back(st, st["slots"] >= 0, _quantise4(st["k"]), _quantise4(st["v"]))


def _plain_attn4(st):
    c = st["case"]
    B, Hkv, d, bs = c["B"], c["Hkv"], c["d"], c["bs"]
    G, R, L = c["Hq"] // Hkv, st["max_rows"], st["max_ctx"]
    qs, ctx = st["qs"].long(), st["ctx"].long()
    n = qs[1:] - qs[:-1]
    row = torch.arange(R, device=DEV)
    has = row[None, :] < n[:, None]
    at = torch.where(has, qs[:-1, None] + row, 0)
    q = st["q"].float()[at].view(B, R, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, d)
    tables = st["tables"].clamp(min=0).long()
    k = _unpack4(st["k_cache"][tables], bs, d).transpose(1, 2).reshape(B, Hkv, -1, d)[:, :, :L]
    s = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    del k
    seen = (ctx - n)[:, None] + row                                 # row's position: the last key it sees
    mask = torch.arange(L, device=DEV) <= seen[:, :, None]
    mask = mask[:, None, :, None, :].expand(B, Hkv, R, G, L).reshape(B, Hkv, R * G, L)
    s = s.masked_fill(~mask, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    v = _unpack4(st["v_cache"][tables], bs, d).transpose(1, 2).reshape(B, Hkv, -1, d)[:, :, :L]
    v = v.masked_fill(~(torch.arange(L, device=DEV) < ctx[:, None])[:, None, :, None], 0)
    o = torch.matmul(p, v).view(B, Hkv, R, G, d).permute(0, 2, 1, 3, 4).reshape(B, R, Hkv * G, d)
    st["out"][at[has]] = o[has].bfloat16()
    return st["out"]


def _weights(p, q, tok):
    """Residual weights in 64 bits: max(p - q, 0), or p without the rejected token where no draft distribution is."""
    if q is not None:
        return (p.double() - q.double()).clamp(min=0)
    return p.double().scatter(1, tok[:, None], 0.0)


def _plain_accept(st):
    qs, tok = st["qs"].long(), st["tokens"].long()
    start, n = qs[:-1], qs[1:] - qs[:-1]
    B, R, T = n.shape[0], st["rows"], tok.shape[0]
    i = torch.arange(R - 1, device=DEV)
    has = i[None, :] < (n - 1)[:, None]                             # draft i of a sequence: row start + i, token at + 1
    r = torch.where(has, start[:, None] + i, 0)
    d = tok[torch.where(has, r + 1, 0)]
    p = st["target"][r, d].double()
    q = st["draft"][r, d].double() if st["draft"] is not None else torch.ones_like(p)
    good = has & (st["uniforms"][r].double() * q < p)
    acc = torch.cumprod(good.long(), 1).sum(1)
    bonus = acc == n - 1
    last = start + acc
    w = st["target"][last].double()
    rejected = tok[torch.where(bonus, 0, last + 1)]
    rest = _weights(w, st["draft"][last] if st["draft"] is not None else None, rejected)
    w = torch.where(bonus[:, None], w, torch.where(rest.sum(1, keepdim=True) > 0, rest, w))
    total = torch.cumsum(w, 1)
    u = st["uniforms"][start + n - 1].double()[:, None] * total[:, -1:]
    hit = (total > u) & (w > 0)
    new = torch.argmax(hit.to(torch.uint8), dim=1)
    new = torch.where(hit.any(1), new, w.shape[1] - 1 - torch.argmax((w > 0).flip(1).to(torch.uint8), dim=1))
    t = torch.arange(T, device=DEV)
    s = torch.searchsorted(qs[1:].contiguous(), t, right=True)
    j = t - start[s]
    out = torch.where(j < acc[s], tok[(t + 1).clamp(max=T - 1)], torch.where(j == acc[s], new[s], -1))
    st["out"].copy_(out)
    st["accepted"].copy_(acc)
    st["ctx_out"].copy_(st["ctx"] - (n - 1 - acc))
    return st["out"], st["accepted"], st["ctx_out"]


# ------------------------------------------------------------------ the floor
def work(case):
    c, op = case, case["op"]
    if op == "slots":
        B, bs = c["B"], c["bs"]
        rows = B if c["mode"] == "decode" else int(B * (0.55 + 0.2 * 5 + 0.1 * 1000))
        # lengths in, counts and offsets out; a position and a slot per row; a table entry and queue entry per block
        return {"bytes": 4.0 * (3 * B + 3 * B + 2 * rows + 2 * rows / bs), "flops": 0.0}
    if op == "table":
        return {"bytes": 4.0 * c["P"] * c["rot"], "flops": 2.0 * c["P"] * c["rot"]}
    if op in ("rope", "append4"):
        T, Hkv, d = c["T"], c["Hkv"], c["d"]
        wide = {"bf16": 2.0, "fp8": 1.0, "int4": 0.5625}[c.get("cache", "int4")]
        kv = 2 * T * Hkv * d
        # rows in; codes out; where a pass reads the codes back, the codes in and fp32 values out
        b = kv * (2 + wide) + 4.0 * T
        if wide != 2.0:
            b += kv * (wide + 4)
        f = 0.0
        if op == "rope":
            b += 4.0 * T * c["Hq"] * d + 4.0 * T + min(T, 16384) * c["rot"] * 4
            f = 3.0 * T * (c["Hq"] + Hkv) * c["rot"]
        return {"bytes": b, "flops": f}
    if op == "attn4":
        B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
        # the lognormal mix: E[ctx] = 1500 exp(0.32)
        mean = 1500 * math.exp(0.32) if c["lo"] == 0 else (c["lo"] + c["hi"]) / 2
        rows = 1 if c["rows"] == 1 else c["rows"] / 2
        b = B * mean * Hkv * 2 * d * 0.5625 + B * rows * Hq * d * 4 + B * mean / c["bs"] * 4
        return {"bytes": b, "flops": 4.0 * B * mean * rows * Hq * d}
    V, B = c["V"], c["B"]
    e = 4 if c["t"] == "float32" else 2
    # one target row per sequence, and a draft row for the part of the sequences that reject (about half)
    return {"bytes": float(B * V * e * (1.5 if c["draft"] else 1.0)), "flops": 2.0 * B * V}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "slots":
        return None  # whole numbers only
    if op == "table":
        pos = torch.arange(case["P"], dtype=torch.float64, device=DEV)
        half = case["rot"] // 2
        out = torch.empty(case["P"], 2 * half, dtype=torch.float64, device=DEV)
        for i in range(half):
            w, m = _frequency(case, st["base"], i)
            out[:, i] = torch.cos(pos * w) * m
            out[:, half + i] = torch.sin(pos * w) * m
        return out
    if op == "attn4":
        return _exact_attn4(st)
    if op == "accept":
        return None  # whole numbers only
    return _exact_rows(st)


def _frequency(case, base, i):
    """Angle per position of pair i, and the factor on cos and sin."""
    rot, f, orig, how = case["rot"], case["factor"], case["orig"], case["scaling"]
    if how == "ntk":
        return (base * f ** (rot / (rot - 2))) ** (-2 * i / rot), 1.0
    w = base ** (-2 * i / rot)
    if how == "linear":
        return w / f, 1.0
    turns = orig * w / (2 * math.pi)  # turns of the pair within the trained context
    if how == "bands":                # over 4 turns: kept; under 1: stretched; a ramp between
        keep = min(max((turns - 1) / 3, 0.0), 1.0)
        return w * (keep + (1 - keep) / f), 1.0
    if how == "yarn":                 # a ramp over the pair's index, from 32 turns to 1
        first = max(math.floor(rot * math.log(orig / (64 * math.pi)) / (2 * math.log(base))), 0)
        last = min(math.ceil(rot * math.log(orig / (2 * math.pi)) / (2 * math.log(base))), rot - 1)
        keep = 1 - min(max((i - first) / max(last - first, 0.001), 0.0), 1.0)
        return w * (keep + (1 - keep) / f), 1.0 + 0.1 * math.log(f)
    return w, 1.0


def _exact_rows(st):
    import numpy as np
    c = st["case"]
    T, d = st["k"].shape[0], c["d"]
    rows = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    k, v = rows(st["k"]), rows(st["v"])
    slots = st["slots"].cpu().numpy()
    q = None
    if c["op"] == "rope":
        pos = st["positions"].cpu().numpy()
        tab = st["table"].double().cpu().numpy()[np.maximum(pos, 0)]
        rot = c["rot"]
        turn = tab[:, None, :rot // 2] + 1j * tab[:, None, rot // 2:]  # a pair is a complex number, rotated

        def rotated(x):
            y = x.copy()
            if c["inter"]:
                z = (x[..., 0:rot:2] + 1j * x[..., 1:rot:2]) * turn
                y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
            else:
                z = (x[..., :rot // 2] + 1j * x[..., rot // 2:rot]) * turn
                y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
            return y

        q, k = rotated(rows(st["q"])), rotated(k)
        q[pos < 0] = 0.0
        if c["cache"] != "bf16":  # the codes are those of the bf16 row
            k = _round_bits(k, 8)
    ok = slots >= 0
    if c.get("cache", "int4") == "int4":
        out = []
        for x in (k, v):
            b = x.reshape(T, -1, d // 32, 32)
            s = np.minimum(np.abs(b).max(-1) / 7.0, 65504.0).astype(np.float16).astype(np.float64)[..., None]
            u = np.clip(np.rint(np.divide(b, s, out=np.zeros_like(b), where=s > 0)), -7, 7)
            y = (u * s).reshape(T, -1, d)
            y[~ok] = 0.0
            out.append(torch.from_numpy(y))
        return tuple(out) if q is None else (torch.from_numpy(q), *out)
    if c["cache"] == "fp8":
        k, v = (_round_e4m3(x / s) * s for x, s in ((k, st["k_scale"]), (v, st["v_scale"])))
    full = []
    for x in (k, v):
        y = np.zeros(tuple(st["k_cache"].shape))
        y[slots[ok] // c["bs"], :, slots[ok] % c["bs"]] = x[ok]
        full.append(torch.from_numpy(y))
    return (torch.from_numpy(q), *full)


def _round_bits(x, bits):
    import numpy as np
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, bits)), e - bits)


def _round_e4m3(x):
    import numpy as np
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))
    return np.clip(np.rint(x / step) * step, -448, 448)


def _exact_attn4(st):
    c = st["case"]
    Hkv, d, bs = c["Hkv"], c["d"], c["bs"]
    G, n = c["Hq"] // Hkv, d // 32
    qs, ctx = st["qs"].tolist(), st["ctx"].tolist()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    # byte and shift of dim j of row r of a block, from the format's definition
    j = torch.arange(d, device=DEV)
    r = torch.arange(bs, device=DEV)
    chunk = (j // 32)[None, :] ^ (r // (8 // n) % n)[:, None]
    byte = r[:, None] * (d // 2) + chunk * 16 + 2 * (j % 8) + (j % 32) // 16
    shift = 4 * (j % 16 // 8)

    def values(cache, s):
        raw = cache[st["tables"][s, :-(-ctx[s] // bs)].long()].flatten(2)           # [blocks, Hkv, bytes]
        code = (raw[:, :, byte].int() >> shift) & 15
        sc = raw[:, :, bs * d // 2:].contiguous().view(torch.float16).view(-1, Hkv, bs, n).double()
        x = (code - 8).double() * sc.repeat_interleave(32, dim=3)
        return x.transpose(0, 1).reshape(Hkv, -1, d)[:, :ctx[s]]

    for s in range(c["B"]):
        rows = qs[s + 1] - qs[s]
        if not rows:
            continue
        k, v = values(st["k_cache"], s), values(st["v_cache"], s)
        q = st["q"][qs[s]:qs[s + 1]].double().view(rows, Hkv, G, d)
        for i in range(rows):
            m = ctx[s] - rows + i + 1
            p = torch.softmax(torch.einsum("hgd,hkd->hgk", q[i], k[:, :m]) * st["scale"], dim=-1)
            out[qs[s] + i] = torch.einsum("hgk,hkd->hgd", p, v[:, :m]).reshape(Hkv * G, d)
    return out

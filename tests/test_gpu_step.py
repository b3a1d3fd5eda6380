"""The step operators together, as an engine runs them: lengths to slots, rotary
append, attention, verification of drafts, lengths of the next step -- eagerly,
captured in a CUDA graph, and on two streams at once."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import step_reference as ref
from tests.gpu_helpers import i32, load_library
from tests.test_gpu_rope import bf16, f64, make_table

pytestmark = pytest.mark.gpu

B, BS, D, HQ, HKV, V, K = 6, 16, 128, 8, 2, 500, 3  # K drafts a sequence
WIDTH, NB, T = 24, 120, 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    load_library()


class Engine:
    """One layer's state on the GPU: every tensor a step reads or writes has a fixed place."""

    def __init__(self, seed, cache):
        import paged_kv_cache_445_b200 as pa
        self.pa, self.cache = pa, cache
        self.rng = np.random.default_rng(seed)
        z = lambda *s, **k: torch.zeros(*s, dtype=k.get("dtype", torch.int32), device="cuda")  # noqa: E731
        self.new, self.ctx, self.held = z(B), z(B), z(B)
        self.tables = torch.full((B, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.ring, self.state = i32(self.rng.permutation(NB)), i32([0, NB])
        self.qs, self.pos, self.slots = z(B + 1), z(T), z(T)
        self.q, self.k, self.v = (z(T, h, D, dtype=torch.bfloat16) for h in (HQ, HKV, HKV))
        self.q_rot, self.out = torch.zeros_like(self.q), torch.zeros_like(self.q)
        self.table = torch.from_numpy(make_table(WIDTH * BS, D)).cuda()
        wide, dtype = {"bf16": (D, torch.bfloat16), "fp8": (D, torch.uint8), "int4": (D * 9 // 16, torch.uint8)}[cache]
        self.kc, self.vc = z(NB, HKV, BS, wide, dtype=dtype), z(NB, HKV, BS, wide, dtype=dtype)
        self.ws = pa.make_int4_workspace(HQ, HKV, D) if cache == "int4" else pa.make_workspace(T, HQ, HKV, D, WIDTH, BS)
        self.tokens, self.uniforms = z(T), z(T, dtype=torch.float32)
        self.target, self.draft = z(T, V, dtype=torch.float32), z(T, V, dtype=torch.float32)
        self.accepted, self.out_tokens, self.status = z(B), z(T), z(1)

    def inputs(self, new):
        """Random rows, probabilities and uniforms for the next step."""
        r = self.rng
        self.new.copy_(i32(new))
        for t, h in ((self.q, HQ), (self.k, HKV), (self.v, HKV)):
            t.copy_(bf16(r.standard_normal((T, h, D))))
        p = np.exp(r.standard_normal((T, V)) * 2)
        q = p * np.exp(0.6 * r.standard_normal((T, V)))
        self.target.copy_(torch.from_numpy((p / p.sum(1, keepdims=True)).astype(np.float32)))
        self.draft.copy_(torch.from_numpy((q / q.sum(1, keepdims=True)).astype(np.float32)))
        self.tokens.copy_(i32(r.integers(0, V, T)))
        self.uniforms.copy_(torch.from_numpy(r.random(T).astype(np.float32)))

    def step(self):
        pa, s = self.pa, self.status
        pa.pa_step_slots(self.new, self.ctx, self.held, self.tables, self.ring, self.state, BS, self.qs, self.pos,
                         self.slots, dev_status=s)
        args = (self.q_rot, self.q, self.k, self.v, self.kc, self.vc, self.table, self.pos, self.slots)
        scale = D ** -0.5
        rows = (self.out, self.q_rot, self.qs, self.kc, self.vc, self.tables, self.ctx, scale)
        if self.cache == "bf16":
            pa.pa_rope_append(*args, dev_status=s)
            pa.pa_prefill_chunk(*rows, self.ws, s)
        elif self.cache == "fp8":
            pa.pa_rope_append_fp8(*args, 0.03125, 0.03125, dev_status=s)
            pa.pa_prefill_chunk_fp8(*rows, 0.03125, 0.03125, self.ws, s)
        else:
            pa.pa_rope_append_int4(*args, dev_status=s)
            pa.pa_prefill_chunk_int4(*rows, self.ws, s)
        pa.pa_accept_drafts(self.out_tokens, self.accepted, self.target, self.draft, self.tokens, self.qs,
                            self.uniforms, context_lens=self.ctx, dev_status=s)

    def snapshot(self):
        names = ("ctx", "held", "tables", "ring", "state", "qs", "pos", "slots", "q_rot", "out", "kc", "vc", "accepted",
                 "out_tokens")
        return {n: getattr(self, n).clone() for n in names}


class Model:
    """The same steps from the definitions, on the host: the rows of every sequence in full precision."""

    def __init__(self, e):
        self.e = e
        self.keys = [np.zeros((0, HKV, D)) for _ in range(B)]
        self.values = [np.zeros((0, HKV, D)) for _ in range(B)]

    def rounded(self, x):
        if self.e.cache == "bf16":
            return x
        if self.e.cache == "fp8":
            y = torch.from_numpy((x * 32).astype(np.float32)).clamp(-448, 448).to(torch.float8_e4m3fn)
            return y.double().numpy() / 32
        return ref.int4_values(*ref.int4_quantise(x))

    def check(self, new, before):
        e = self.e
        host = lambda t: t.cpu().numpy()  # noqa: E731
        want, bits = ref.step_slots(np.asarray(new, np.int32), *(host(before[k]) for k in ("ctx", "held", "tables", "ring", "state")),
                                    BS, T)
        assert bits == 0 and int(e.status.item()) == 0
        for name, key in (("qs", "query_start"), ("pos", "positions"), ("slots", "slots"), ("tables", "tables"),
                          ("held", "held"), ("state", "state")):
            assert np.array_equal(host(getattr(e, name)), want[key]), name
        pos, qs, ctx = want["positions"], want["query_start"], want["ctx"]
        q = ref.bf16_round(ref.rotate(f64(e.q), host(e.table), pos, False))
        k = self.rounded(ref.bf16_round(ref.rotate(f64(e.k), host(e.table), pos, False)))
        v = self.rounded(f64(e.v))
        got = f64(e.out)
        for s in range(B):
            a, b = qs[s], qs[s + 1]
            self.keys[s] = np.concatenate([self.keys[s][:ctx[s] - (b - a)], k[a:b]])[:ctx[s]]
            self.values[s] = np.concatenate([self.values[s][:ctx[s] - (b - a)], v[a:b]])[:ctx[s]]
            for i in range(b - a):
                m = ctx[s] - (b - a) + i + 1
                for h in range(HQ):
                    kk, vv = self.keys[s][:m, h // (HQ // HKV)], self.values[s][:m, h // (HQ // HKV)]
                    z = kk @ q[a + i, h] * D ** -0.5
                    p = np.exp(z - z.max())
                    o = p @ vv / p.sum()
                    # bf16 out (2^-8 of the value), weights of 8 bits in the bf16 kernels (2^-8 of the largest value)
                    assert np.abs(got[a + i, h] - o).max() <= 2.0**-8 * np.abs(o).max() + 2.0**-7 * np.abs(vv).max()
        out, acc, _ = ref.accept(host(e.target), host(e.draft), host(e.tokens), qs, host(e.uniforms))
        assert np.array_equal(host(e.accepted), acc)
        live = out != -9
        assert np.array_equal(host(e.out_tokens)[live], out[live])
        n = np.diff(qs)
        assert np.array_equal(host(e.ctx), np.where(n > 0, ctx - (n - 1 - acc), ctx))


def plan(step, e):
    """New tokens of a step: prompts, then drafts; a sequence finishes and comes back, one idles."""
    if step == 0:
        return [9, 1, 17, 4, 0, 2]
    new = [K + 1] * B
    if step == 2:
        new[2] = -int(e.ctx[2].item())
    if step == 3:
        new[2], new[4] = 12, 0
    return new


@pytest.mark.parametrize("cache", ["bf16", "fp8", "int4"])
def test_six_steps(cache):
    e = Engine(1, cache)
    m = Model(e)
    for step in range(6):
        new = plan(step, e)
        e.inputs(new)
        before = e.snapshot()
        e.step()
        torch.cuda.synchronize()
        m.check(new, before)


@pytest.mark.parametrize("cache", ["bf16", "int4"])
def test_a_captured_step_replays_as_the_eager_one(cache):
    eager, graph = Engine(2, cache), Engine(2, cache)
    g = None
    for step in range(5):
        for e in (eager, graph):
            e.inputs(plan(step, e))
        eager.step()
        if step == 0:
            graph.step()  # set-up of every kernel, before the capture
        else:
            if g is None:
                torch.cuda.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    graph.step()
            g.replay()
        torch.cuda.synchronize()
        a, b = eager.snapshot(), graph.snapshot()
        for k in a:
            if k == "out":  # rows behind the last sequence are not part of the step
                n = int(a["qs"][-1].item())
                assert torch.equal(a[k][:n].view(torch.int16), b[k][:n].view(torch.int16)), (step, k)
            else:
                same = a[k].view(torch.int16) if a[k].dtype == torch.bfloat16 else a[k]
                other = b[k].view(torch.int16) if b[k].dtype == torch.bfloat16 else b[k]
                assert torch.equal(same, other), (step, k)
    assert int(graph.status.item()) == 0


def test_two_engines_on_two_streams():
    engines = [Engine(3, "int4"), Engine(4, "int4")]
    alone = [Engine(3, "int4"), Engine(4, "int4")]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for step in range(4):
        for e in engines + alone:
            e.inputs(plan(step, e))
        torch.cuda.synchronize()
        for _ in range(1):
            for e, s in zip(engines, streams):
                with torch.cuda.stream(s):
                    e.step()
        torch.cuda.synchronize()
        for e in alone:
            e.step()
            torch.cuda.synchronize()
        for a, b in zip(engines, alone):
            n = int(b.qs[-1].item())
            assert torch.equal(a.out[:n].view(torch.int16), b.out[:n].view(torch.int16))
            assert torch.equal(a.ctx, b.ctx) and torch.equal(a.kc, b.kc) and torch.equal(a.out_tokens, b.out_tokens)


def test_decode_of_rotated_rows_equals_the_separate_calls():
    """bf16: the fused rotation and append, then pa_decode, against rotating with torch and appending."""
    import paged_kv_cache_445_b200 as pa
    e = Engine(5, "bf16")
    e.inputs([1, 5, 30, 3, 2, 1])
    e.step()
    e.inputs([1] * B)
    before = e.snapshot()
    pa.pa_step_slots(e.new, e.ctx, e.held, e.tables, e.ring, e.state, BS, e.qs, e.pos, e.slots, dev_status=e.status)
    kc, vc = before["kc"].clone(), before["vc"].clone()
    pa.pa_rope_append(e.q_rot, e.q, e.k, e.v, e.kc, e.vc, e.table, e.pos, e.slots, dev_status=e.status)
    out = torch.empty(B, HQ, D, dtype=torch.bfloat16, device="cuda")
    pa.pa_decode(out, e.q_rot[:B].contiguous(), e.kc, e.vc, e.tables, e.ctx, 0.1, e.ws, e.status)
    pos = e.pos.cpu().numpy()
    k = bf16(ref.bf16_round(ref.rotate(f64(e.k), e.table.cpu().numpy(), pos, False))).cuda()
    pa.pa_cache_append(k, e.v, kc, vc, e.slots, e.status)
    again = torch.empty_like(out)
    pa.pa_decode(again, e.q_rot[:B].contiguous(), kc, vc, e.tables, e.ctx, 0.1, e.ws, e.status)
    assert torch.equal(kc.view(torch.int16), e.kc.view(torch.int16))
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and int(e.status.item()) == 0

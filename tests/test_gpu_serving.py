"""Requests from prompt to tokens with all of it together: pages for the
prompts' tokens, rotary positions, rows into the 4-bit cache, the packed
prefill; then decode steps of one token a request, some requests ending and
new ones taking their places and pages.  The same loop in fp64 keeps every
request's rows by itself; results are held to the bars of each call."""
import numpy as np
import pytest
import torch

from gpu_util import TOL, dev
from serving_ref import decode_ref, packed_ref, q4_ref, rope_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_serving(dtype):
    import long_context_attention_causal_gb300 as pa
    B, Hq, Hkv, d, page, cols, pool = 6, 8, 2, 64, 16, 20, 80
    name = "bf16" if dtype == torch.bfloat16 else "f32"
    rng = np.random.default_rng(5)
    g = torch.Generator(device=dev()).manual_seed(5)
    inv_freq, scale = pa.rope_inv_freq(32, factor=2.0, scaling="bands", context=2048)
    w = torch.randn((Hq, d), generator=g, device=dev()) * 0.02
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev())  # noqa: E731
    table = torch.full((B, cols), -1, dtype=torch.int32, device=dev())
    lens, count = i32([0] * B), i32([pool])
    free = torch.randperm(pool, generator=g, device=dev()).to(torch.int32)
    kp, vp = pa.cache_q4(pool, Hkv, page, d)
    kept = [[torch.zeros((0, Hkv, d), dtype=torch.float64, device=dev())] * 2 for _ in range(B)]

    def tokens(n):
        qkv = torch.randn((n, Hq + 2 * Hkv, d), generator=g, device=dev()).to(dtype)
        mem = (torch.randn((n, Hq, d), generator=g, device=dev()) * 0.1).to(dtype)
        return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], mem

    def step(new):
        """New tokens of every request: rows, positions, cache; the turned q and k."""
        n = sum(new)
        q, k, v, mem = tokens(n)
        cu, pos, slots = pa.pages_extend(table, lens, i32(new), free, count, page, n)
        assert (slots >= 0).all()
        q2, k2 = pa.rope(q, k, pos, inv_freq, scale=scale)
        ref = rope_ref(k, pos, inv_freq, scale)
        lim = 2.0 ** -8 * ref.abs() + 2.0 ** -15 if name == "bf16" else torch.full_like(ref, 2e-5)
        assert ((k2.double() - ref).abs() <= lim).all()
        pa.cache_append_q4(k2, v, slots, kp, vp)
        at = cu.tolist()
        for b in range(B):
            s = slice(at[b], at[b + 1])
            kept[b] = [torch.cat([kept[b][0], q4_ref(k2[s])]), torch.cat([kept[b][1], q4_ref(v[s])])]
            assert pos[s].tolist() == list(range(len(kept[b][0]) - new[b], len(kept[b][0])))
        return q2, k2, v, mem, cu

    prompts = [40, 1, 130, 16, 75, 17]
    q, k, v, mem, cu = step(prompts)
    out, n_eff, conf = pa.fwd_packed(q, k, v, mem, w, cu, want_conf=True)
    for b in range(B):
        s = slice(int(cu[b]), int(cu[b + 1]))
        o, ne, c = packed_ref(q, k, v, mem, w, cu, b)
        assert (out[s].double() - o).abs().max() <= TOL[name]["out"]
        assert (n_eff[s].double() / ne - 1).abs().max() <= TOL["f32"]["neff"]
    for i in range(30):
        if i % 7 == 3:
            # one request ends; a new prompt takes its place at the next step
            gone = int(rng.integers(B))
            keep = lens.clone()
            keep[gone] = 0
            pa.pages_release(table, lens, keep, free, count, page)
            kept[gone] = [x[:0] for x in kept[gone]]
            new = [0] * B
            new[gone] = int(rng.integers(1, 90))
            step(new)
        q, k, v, mem, cu = step([1] * B)
        out, n_eff, conf = pa.decode_paged_q4(q, kp, vp, table, lens, mem, w, want_conf=True)
        assert lens.tolist() == [len(x[0]) for x in kept]
        used = sum(-(-len(x[0]) // page) for x in kept)
        assert int(count) == pool - used
        for b in range(B):
            o, ne, c = decode_ref(q[b], kept[b][0].transpose(0, 1), kept[b][1].transpose(0, 1), w,
                                  mem[b])
            assert (out[b].double() - o).abs().max() <= TOL[name]["out"]
            assert (n_eff[b].double() / ne - 1).abs().max() <= TOL["f32"]["neff"]
            assert (conf[b].double() - c).abs().max() <= TOL["f32"]["conf"]
    assert pa.device_status() == 0


def test_captured_decode_step():
    """A decode step (pages, positions, cache, decode) captured once: replays go
    on from one another and give the bits of the same calls made one by one."""
    import long_context_attention_causal_gb300 as pa
    B, Hq, Hkv, d, page, cols, pool = 5, 8, 2, 128, 8, 12, 60
    g = torch.Generator(device=dev()).manual_seed(9)
    inv_freq, _ = pa.rope_inv_freq(128)
    w = torch.randn((Hq, d), generator=g, device=dev()) * 0.02
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev())  # noqa: E731

    class Loop:
        def __init__(self):
            self.table = torch.full((B, cols), -1, dtype=torch.int32, device=dev())
            self.lens, self.count = i32([0] * B), i32([pool])
            self.free = torch.arange(pool, dtype=torch.int32, device=dev())
            self.cache = pa.cache_q4(pool, Hkv, page, d)
            self.one = i32([1] * B)
            self.qkv = torch.zeros((B, Hq + 2 * Hkv, d), device=dev(), dtype=torch.bfloat16)
            self.mem = torch.zeros((B, Hq, d), device=dev(), dtype=torch.bfloat16)

        def step(self):
            q, k, v = self.qkv.split([Hq, Hkv, Hkv], 1)
            _, pos, slots = pa.pages_extend(self.table, self.lens, self.one, self.free, self.count,
                                            page, B)
            q, k = pa.rope(q, k, pos, inv_freq)
            pa.cache_append_q4(k, v, slots, *self.cache)
            self.out = pa.decode_paged_q4(q, *self.cache, self.table, self.lens, self.mem, w,
                                          want_conf=True)

    eager, loop = Loop(), Loop()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop.step()
    for _ in range(90):
        x = torch.randn(eager.qkv.shape, generator=g, device=dev()).bfloat16()
        eager.qkv.copy_(x)
        loop.qkv.copy_(x)
        eager.step()
        graph.replay()
        for a, b in zip(eager.out, loop.out):
            assert torch.equal(a, b)
    assert loop.lens.tolist() == [90] * B and torch.equal(loop.table, eager.table)
    assert pa.device_status() == 0


def test_two_threads():
    """Two host threads run the whole chain at once, each on a stream of its own
    with tensors of its own, and get the bits of the same calls made alone."""
    import threading

    import long_context_attention_causal_gb300 as pa
    B, Hq, Hkv, d, page, cols, pool = 7, 16, 2, 128, 32, 16, 120
    inv_freq, _ = pa.rope_inv_freq(d)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev())  # noqa: E731
    w = torch.randn((Hq, d), generator=torch.Generator(device=dev()).manual_seed(1), device=dev()) * 0.02

    def chain(seed):
        """Every output of some rounds of a prompt and a token for each request."""
        g = torch.Generator(device=dev()).manual_seed(seed)
        table = torch.full((B, cols), -1, dtype=torch.int32, device=dev())
        lens, count = i32([0] * B), i32([pool])
        free, cache = torch.arange(pool, dtype=torch.int32, device=dev()), pa.cache_q4(pool, Hkv, page, d)
        got = []
        for i in range(12):
            new = [1] * B if i % 3 else [(37 * seed + 29 * i + 11 * b) % 90 for b in range(B)]
            n = sum(new)
            qkv = torch.randn((n, Hq + 2 * Hkv, d), generator=g, device=dev()).bfloat16()
            mem = torch.randn((n, Hq, d), generator=g, device=dev()).bfloat16()
            q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
            cu, pos, slots = pa.pages_extend(table, lens, i32(new), free, count, page, n)
            q, k = pa.rope(q, k, pos, inv_freq)
            pa.cache_append_q4(k, v, slots, *cache)
            if i % 3:
                got += pa.decode_paged_q4(q, *cache, table, lens, mem, w)[:2]
            else:
                got += pa.fwd_packed(q, k, v, mem, w, cu)[:2]
            if i % 4 == 3:
                pa.pages_release(table, lens, lens - lens % page, free, count, page)
        return got + [lens, count, table]

    alone = [chain(s) for s in (1, 2)]
    torch.cuda.synchronize()
    together, failed = [None, None], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(5):
                    together[i] = chain(i + 1)
            stream.synchronize()
        except BaseException as e:  # noqa: BLE001 (shown below)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for a, b in zip(alone, together):
        assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))
    assert pa.device_status() == 0

"""Decode over the paged 4-bit cache against fp64 on the values it holds.

Tolerances are those of the paged decode (gpu_util.TOL): bf16 rounds the
weights times the values' scales to 8 bits, one rounding, as the bf16 decode
rounds its weights; fp32 takes both products to 24 bits.  n_eff and conf come
from fp32 scores in both types and are held to fp32's bar.
"""
import pytest
import torch

from gpu_util import TOL, dev
from serving_ref import decode_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def case(B, Hq, Hkv, lens, d, page, dtype, seed, spare=3, kstd=1.0):
    """Arguments of decode_paged_q4 and, per sequence, the values (k, v) [Hkv, n, d]."""
    import long_context_attention_causal_gb300 as pa
    g = torch.Generator(device=dev()).manual_seed(seed)
    npg = [-(-n // page) for n in lens]
    pool = sum(npg) + spare
    perm = torch.randperm(pool, generator=g, device=dev()).to(torch.int32)
    cols = max(npg) + 1
    table = torch.full((B, cols), -7, dtype=torch.int32, device=dev())
    kp = torch.randint(0, 256, (pool, Hkv, page, 9 * d // 16), generator=g, device=dev(),
                       dtype=torch.uint8)   # unused rows hold anything, scales of NaN too
    vp = torch.randint(0, 256, kp.shape, generator=g, device=dev(), dtype=torch.uint8)
    kp.flatten(2)[..., page * d // 2:] = 0xFF
    vp.flatten(2)[..., page * d // 2:] = 0xFF
    values, at = [], 0
    for b, n in enumerate(lens):
        table[b, :npg[b]] = perm[at:at + npg[b]]
        at += npg[b]
        t = torch.arange(n, device=dev())
        slots = (table[b].long()[t // page] * page + t % page).to(torch.int32)
        k = torch.randn((n, Hkv, d), generator=g, device=dev()) * kstd
        v = torch.randn((n, Hkv, d), generator=g, device=dev())
        v = v * torch.exp(torch.randn((n, Hkv, 1), generator=g, device=dev()))
        pa.cache_append_q4(k, v, slots, kp, vp)
        k, v = pa.cache_read_q4(kp, vp, slots, dtype=torch.float32)
        values.append((k.transpose(0, 1), v.transpose(0, 1)))
    q = torch.randn((B, Hq, d), generator=g, device=dev()).to(DT[dtype])
    mem = (torch.randn((B, Hq, d), generator=g, device=dev()) * 0.1).to(DT[dtype])
    w = torch.randn((Hq, d), generator=g, device=dev()) * 0.02
    return [q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device=dev()), mem, w], values


def check(args, values, got, dtype, rows=None):
    q, mem, w = args[0], args[5], args[6]
    out, n_eff, conf = got
    for b in rows if rows is not None else range(q.shape[0]):
        o, ne, c = decode_ref(q[b], *values[b], w, mem[b])
        assert (out[b].double() - o).abs().max() <= TOL[dtype]["out"]
        assert (n_eff[b].double() / ne - 1).abs().max() <= TOL["f32"]["neff"]
        assert (conf[b].double() - c).abs().max() <= TOL["f32"]["conf"]


@pytest.mark.parametrize("Hq,Hkv,lens,d,page", [
    (1, 1, [1], 64, 8), (8, 1, [1, 2, 3], 128, 8), (4, 4, [100, 8, 9], 64, 8), (8, 2, [300, 15, 17], 128, 16),
    (16, 2, [777, 128, 129, 127], 64, 64), (4, 2, [1500, 1], 128, 128), (8, 8, [4000, 33], 128, 256),
    (32, 4, [1100, 1024, 1], 64, 1024), (6, 3, [513, 2500], 128, 32)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("runs", [0, 1, 5, 700])
def test_decode(Hq, Hkv, lens, d, page, dtype, runs):
    import long_context_attention_causal_gb300 as pa
    args, values = case(len(lens), Hq, Hkv, lens, d, page, dtype, 7 + d + len(lens))
    got = pa.decode_paged_q4(*args, max_seq_len=max(lens), num_runs=runs, want_conf=True)
    check(args, values, got, dtype)
    again = pa.decode_paged_q4(*args, max_seq_len=max(lens), num_runs=runs, want_conf=True)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert pa.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_growing_and_peaked_logits(dtype):
    """Running maxima that move at every step, and one key that takes it all."""
    import long_context_attention_causal_gb300 as pa
    lens = [700, 1300]
    args, values = case(2, 8, 2, lens, 128, 64, dtype, 3, kstd=6.0)
    for b, n in enumerate(lens):     # logits grow along the sequence: sort the rows by them
        q = args[0][b, 0].float()
        t = torch.arange(n, device=dev())
        slots = (args[3][b].long()[t // 64] * 64 + t % 64).to(torch.int32)
        k, v = (x.transpose(0, 1) for x in values[b])
        order = torch.argsort((k[:, 0] * q).sum(-1))
        k, v = k[order].contiguous(), v[order].contiguous()
        pa.cache_append_q4(k, v, slots, args[1], args[2])
        k, v = pa.cache_read_q4(args[1], args[2], slots, dtype=torch.float32)
        values[b] = (k.transpose(0, 1), v.transpose(0, 1))
    got = pa.decode_paged_q4(*args, max_seq_len=1300, num_runs=5, want_conf=True)
    check(args, values, got, dtype)


def test_bad_pages_and_lengths():
    import long_context_attention_causal_gb300 as pa
    lens = [200, 90, 50]
    args, values = case(3, 4, 2, lens, 64, 16, "bf16", 11)
    table = args[3]
    table[0, 3], table[0, 7] = args[1].shape[0], -1
    keep = torch.ones(200, dtype=torch.bool, device=dev())
    keep[48:64] = keep[112:128] = False
    got = pa.decode_paged_q4(*args, max_seq_len=200, want_conf=True)
    assert pa.device_status(reset=True) == 3
    check(args, values, got, "bf16", rows=[1, 2])
    # keys on bad pages are skipped (n stays the length)
    k, v = (x[:, keep] for x in values[0])
    o, _, _ = decode_ref(args[0][0], k, v, args[6], args[5][0])
    a = (got[0][0].double() - args[5][0].double())
    o = o - args[5][0].double()
    assert ((a - o).norm() / o.norm()) <= 0.05   # the gate differs a little with n
    # a length of 0: the memory stream passes; one past the bound is cut to it
    args[4][1], args[4][2] = 0, 1000
    values[2] = tuple(x[:, :40] for x in values[2])
    table[0, 3], table[0, 7] = 0, 1
    got = pa.decode_paged_q4(*args, max_seq_len=200, want_conf=True)
    assert pa.device_status(reset=True) == 3
    assert torch.equal(got[0][1], args[5][1]) and (got[1][1] == 0).all() and (got[2][1] == 0).all()


def test_nan_row_reaches_its_sequence_only():
    import long_context_attention_causal_gb300 as pa
    args, values = case(3, 4, 2, [150, 150, 150], 64, 16, "bf16", 12)
    slot = (args[3][1, 3] * 16 + 5).view(1)
    bad = torch.full((1, 2, 64), float("nan"), device=dev())
    pa.cache_append_q4(bad, bad, slot, args[1], args[2])
    got = pa.decode_paged_q4(*args, max_seq_len=150, want_conf=True)
    check(args, values, got, "bf16", rows=[0, 2])
    assert got[0][1].isnan().all()
    # the only key of a sequence
    args[4][1] = 1
    pa.cache_append_q4(bad, bad, args[3][1, :1] * 16, args[1], args[2])
    got = pa.decode_paged_q4(*args, max_seq_len=150, want_conf=True)
    check(args, values, got, "bf16", rows=[0, 2])
    assert got[0][1].isnan().all()
    assert pa.device_status() == 0


@pytest.mark.parametrize("scale", [2.0 ** -20, 2.0 ** 20])
def test_scaled_values(scale):
    """Rows times a power of two hold the same codes, and the sums keep their
    precision (below the projection's eps too, which the reference applies)."""
    import long_context_attention_causal_gb300 as pa
    args, values = case(1, 4, 2, [500], 128, 32, "bf16", 13)
    got = pa.decode_paged_q4(*args, max_seq_len=500)
    t = torch.arange(500, device=dev())
    slots = (args[3][0].long()[t // 32] * 32 + t % 32).to(torch.int32)
    k, v = (x.transpose(0, 1).contiguous() for x in values[0])
    pa.cache_append_q4(k, v * scale, slots, args[1], args[2])
    k2, v2 = pa.cache_read_q4(args[1], args[2], slots, dtype=torch.float32)
    assert torch.equal(k2, k) and torch.equal(v2, v * scale)
    other = pa.decode_paged_q4(*args, max_seq_len=500)
    o, _, _ = decode_ref(args[0][0], k2.transpose(0, 1), v2.transpose(0, 1), args[6], args[5][0])
    assert (other[0][0].double() - o).abs().max() <= TOL["bf16"]["out"]
    assert torch.equal(other[1], got[1])


def test_many_calls_and_streams():
    """One cache, the same bits every time, on two streams with a workspace each."""
    import long_context_attention_causal_gb300 as pa
    lens = [4096, 3000, 5000, 1]
    args, values = case(4, 16, 4, lens, 128, 64, "bf16", 15)
    need = pa.decode_paged_q4_workspace_bytes(4, 16, 4, 5000, 128)
    ws = [torch.empty(need, device=dev(), dtype=torch.uint8) for _ in range(2)]
    first = pa.decode_paged_q4(*args, max_seq_len=5000, want_conf=True, workspace=ws[0])
    check(args, values, first, "bf16")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(t) for t in first] for _ in range(2)]
    wrong = [torch.zeros(3, dtype=torch.int64, device=dev()) for _ in range(2)]
    for _ in range(100):
        for s, w, o, bad in zip(streams, ws, outs, wrong):
            pa.decode_paged_q4(*args, max_seq_len=5000, workspace=w, out=o[0], n_eff=o[1], conf=o[2],
                               stream=s)
            with torch.cuda.stream(s):
                bad += torch.stack([(a != b).any() for a, b in zip(o, first)])
    torch.cuda.synchronize()
    assert [w.tolist() for w in wrong] == [[0] * 3] * 2
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.decode_paged_q4(*args, max_seq_len=5000, workspace=ws[0], out=outs[0][0],
                           n_eff=outs[0][1], conf=outs[0][2])
    args[4].copy_(torch.tensor([100, 2999, 17, 1], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    values = [tuple(x[:, :n] for x in vs) for vs, n in zip(values, [100, 2999, 17, 1])]
    check(args, values, outs[0], "bf16")
    assert pa.device_status() == 0


def test_refusals():
    import long_context_attention_causal_gb300 as pa
    args, _ = case(1, 4, 2, [20], 64, 8, "bf16", 16)
    for i, bad in ((0, args[0][:, :3].contiguous()), (1, args[1].float()), (2, args[2][:1]),
                   (3, args[3].long()), (4, args[4][:0]), (5, args[5].float()), (6, args[6][:2])):
        a = list(args)
        a[i] = bad
        with pytest.raises((TypeError, ValueError, pa.PolarError)):
            pa.decode_paged_q4(*a, max_seq_len=20)
    with pytest.raises(ValueError):
        pa.decode_paged_q4(torch.zeros((1, 4, 128), device=dev()).bfloat16(), *args[1:])
    with pytest.raises(pa.PolarError):
        pa.decode_paged_q4(*args, max_seq_len=200)
    with pytest.raises(pa.PolarError):
        pa.decode_paged_q4(*args, max_seq_len=20,
                           workspace=torch.empty(16, device=dev(), dtype=torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_long_sequence(dtype):
    """400000 rows of one head, spread over all runs and joined from their records."""
    import long_context_attention_causal_gb300 as pa
    n = 400001
    args, values = case(1, 4, 1, [n], 64, 256, dtype, 61)
    got = pa.decode_paged_q4(*args, max_seq_len=n, want_conf=True)
    check(args, values, got, dtype)
    assert pa.device_status() == 0

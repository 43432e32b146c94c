"""Causal prefill of packed sequences with grouped heads against fp64, held to
the bars of the padded prefill (gpu_util.TOL); n_eff and conf come from fp32
scores in both types and are held to fp32's."""
import pytest
import torch

from gpu_util import TOL, dev
from serving_ref import packed_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def case(lens, Hq, Hkv, d, dtype, seed, lead=0, tail=0):
    """(q, k, v, mem, w_count, cu) with q, k, v parts of one buffer; `lead` and
    `tail` rows belong to no sequence."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    N = sum(lens) + lead + tail
    qkv = torch.randn((N, Hq + 2 * Hkv, d), generator=g, device=dev()).to(DT[dtype])
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    mem = (torch.randn((N, Hq, d), generator=g, device=dev()) * 0.1).to(DT[dtype])
    w = torch.randn((Hq, d), generator=g, device=dev()) * 0.02
    at = [lead]
    for n in lens:
        at.append(at[-1] + n)
    return [q, k, v, mem, w, torch.tensor(at, dtype=torch.int32, device=dev())]


def run(args, **kw):
    """Outputs with marked rows, so that one written where it should not be shows."""
    import long_context_attention_causal_gb300 as pa
    q = args[0]
    out = torch.full(q.shape, 77.0, dtype=q.dtype, device=dev())
    n_eff = torch.full(q.shape[:2], 77.0, device=dev())
    conf = n_eff.clone()
    pa.fwd_packed(*args, out=out, n_eff=n_eff, conf=conf, **kw)
    return out, n_eff, conf


def check(args, got, dtype, seqs=None):
    cu = args[5].tolist()
    out, n_eff, conf = got
    for b in seqs if seqs is not None else range(len(cu) - 1):
        lo, hi = cu[b], cu[b + 1]
        if lo == hi:
            continue
        o, ne, c = packed_ref(*args, b)
        assert (out[lo:hi].double() - o).abs().max() <= TOL[dtype]["out"], b
        assert (n_eff[lo:hi].double() / ne - 1).abs().max() <= TOL["f32"]["neff"], b
        assert (conf[lo:hi].double() - c).abs().max() <= TOL["f32"]["conf"], b
    for x in got:
        assert (x[:cu[0]] == 77.0).all() and (x[cu[-1]:] == 77.0).all()


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1], [1, 1, 1], [0, 5, 0, 0, 17, 0], [127, 128, 129], [255, 256, 257],
                                  [31, 32, 33, 15, 16, 64], [700, 3, 1025], [2600, 90]])
def test_packed(lens, dtype, d, G):
    import long_context_attention_causal_gb300 as pa
    args = case(lens, 2 * G, 2, d, dtype, sum(lens) + d + G, lead=3, tail=5)
    got = run(args)
    check(args, got, dtype)
    again = run(args)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert pa.device_status() == 0


@pytest.mark.parametrize("B,top,seed", [(300, 40, 1), (1500, 9, 2), (257, 300, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences(B, top, seed, dtype):
    """More sequences than a warp keeps in registers, many of them empty."""
    import long_context_attention_causal_gb300 as pa
    lens = torch.randint(0, top + 1, (B,), generator=torch.Generator().manual_seed(seed)).tolist()
    args = case(lens, 8, 4, 64, dtype, seed, tail=2)
    got = run(args)
    check(args, got, dtype, seqs=list(range(0, B, 7)) + [B - 1])
    live = got[1][:int(args[5][-1])]
    assert (live != 77.0).all() and pa.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 8])
def test_neighbours_do_not_leak(dtype, G):
    """NaN and infinities in the sequences around one, in the rows of no
    sequence, and a sequence's results do not depend on what is beside it."""
    import long_context_attention_causal_gb300 as pa
    lens = [70, 100, 130]
    args = case(lens, 2 * G, 2, 128, dtype, 5, lead=4, tail=100)
    clean = run(args)
    lo, hi = 74, 174
    for value in (float("nan"), float("inf"), -float("inf")):
        other = [a.clone() for a in args]
        for t in other[:4]:
            t[:lo] = value
            t[hi:] = value
        got = run(other)
        for a, b in zip(got, clean):
            assert torch.equal(a[lo:hi], b[lo:hi])
    assert pa.device_status() == 0


def test_same_rows_as_the_padded_prefill():
    """One head a KV head, equal lengths: the padded prefill's problem."""
    import long_context_attention_causal_gb300 as pa
    B, H, T, d = 2, 3, 300, 64
    args = case([T] * B, H, H, d, "f32", 9)
    got = run(args)
    pad = [t.contiguous().view(B, T, H, d).transpose(1, 2).contiguous() for t in args[:4]]
    out, n_eff, conf = pa.fwd(*pad, args[4], want_conf=True)
    assert (out.transpose(1, 2).reshape(B * T, H, d) - got[0]).abs().max() <= TOL["f32"]["out"]
    assert (n_eff.transpose(1, 2).reshape(B * T, H) / got[1] - 1).abs().max() <= TOL["f32"]["neff"]
    assert (conf.transpose(1, 2).reshape(B * T, H) - got[2]).abs().max() <= TOL["f32"]["conf"]


def test_constants_and_missing_conf():
    import math
    import long_context_attention_causal_gb300 as pa
    args = case([40, 9], 4, 2, 64, "bf16", 21)
    a = run(args, consts=pa.Consts(math.log(16.0), math.log(16.0), 0.5, 1e-6, 2))
    b = run(args)
    assert not torch.equal(a[0], b[0])
    flat = [t.contiguous() for t in args[:4]]
    for seq in (slice(0, 40), slice(40, 49)):
        kv = [t[seq].transpose(0, 1)[None] for t in flat]
        kv[1], kv[2] = kv[1].repeat_interleave(2, 1), kv[2].repeat_interleave(2, 1)
        out, _, conf = pa.fwd(*[t.contiguous() for t in kv], args[4], want_conf=True,
                              consts=pa.Consts(math.log(16.0), math.log(16.0), 0.5, 1e-6, 2))
        assert (out[0].transpose(0, 1).float() - a[0][seq].float()).abs().max() <= TOL["bf16"]["out"]
        assert (conf[0].t() - a[2][seq]).abs().max() <= TOL["f32"]["conf"]
    out, n_eff, none = pa.fwd_packed(*args)
    assert none is None and torch.equal(out, b[0]) and torch.equal(n_eff, b[1])


def test_bad_offsets():
    """Offsets out of bounds or descending are cut and recorded; nothing outside
    the tensors is touched, and rows that one sequence alone has are computed."""
    import long_context_attention_causal_gb300 as pa
    for dtype in DT:
        args = case([50, 60, 40], 4, 2, 64, dtype, 31)
        for cu in ([0, 50, 300, 150], [0, 50, 20, 150], [-5, 50, 110, 150], [0, 50, 1 << 30, 1 << 31 - 1]):
            bad = list(args)
            bad[5] = torch.tensor([max(min(x, (1 << 31) - 1), -5) for x in cu], dtype=torch.int32,
                                  device=dev())
            got = run(bad)
            assert pa.device_status(reset=True) == 3
            if cu[0] == 0:
                o, _, _ = packed_ref(*args, 0)
                own = min([50] + [x for x in cu[2:] if x >= 0])
                assert (got[0][:own].double() - o[:own]).abs().max() <= TOL[dtype]["out"]
    none = case([], 4, 2, 64, "bf16", 1, lead=6)
    assert (run(none)[0] == 77.0).all()


def test_elements_past_2_31():
    """Rows whose offsets pass 2^31 elements, in q, k, v (strided) and the outputs."""
    import long_context_attention_causal_gb300 as pa
    n, B = 1000, 1100
    Hq, Hkv, d = 16, 2, 128
    N = n * B
    qkv = torch.empty((N, Hq + 2 * Hkv, d), dtype=torch.bfloat16, device=dev())
    for o in range(0, N, 100000):
        qkv[o:o + 100000].normal_()
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    mem = torch.zeros((N, Hq, d), dtype=torch.bfloat16, device=dev())
    w = torch.randn((Hq, d), device=dev()) * 0.02
    cu = torch.arange(0, N + 1, n, dtype=torch.int32, device=dev())
    assert N * (Hq + 2 * Hkv) * d > 1 << 31 and N * Hq * d > 1 << 31
    out, n_eff, conf = pa.fwd_packed(q, k, v, mem, w, cu, want_conf=True)
    for b in (0, 1, 800, B - 2, B - 1):
        o, ne, c = packed_ref(q, k, v, mem, w, cu, b)
        s = slice(b * n, (b + 1) * n)
        assert (out[s].double() - o).abs().max() <= TOL["bf16"]["out"]
        assert (n_eff[s].double() / ne - 1).abs().max() <= TOL["f32"]["neff"]
        assert (conf[s].double() - c).abs().max() <= TOL["f32"]["conf"]
    assert pa.device_status() == 0


def test_long_sequence():
    """One long prompt among short ones: sampled rows (n - 400 .. n)."""
    import long_context_attention_causal_gb300 as pa
    from serving_ref import polar_ref
    for dtype, n in (("bf16", 40000), ("f32", 9000)):
        args = case([3, n, 50], 8, 1, 128, dtype, 41)
        got = run(args)
        lo, hi = 3, 3 + n
        t = lambda x: x.transpose(0, 1)  # noqa: E731
        first = n - 400
        o, ne, c = polar_ref(t(args[0][lo + first:hi]), t(args[1][lo:hi]).expand(8, -1, -1),
                             t(args[2][lo:hi]).expand(8, -1, -1), first, args[4],
                             t(args[3][lo + first:hi]))
        assert (t(got[0][lo + first:hi]).double() - o).abs().max() <= TOL[dtype]["out"]
        assert (t(got[1][lo + first:hi]).double() / ne - 1).abs().max() <= TOL["f32"]["neff"]
        check(args, got, dtype, seqs=[0, 2])
        assert pa.device_status() == 0


def test_streams_capture_and_refusals():
    import long_context_attention_causal_gb300 as pa
    args = case([300, 77, 1200], 8, 2, 128, "bf16", 51)
    first = run(args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.full_like(t, 77.0) for t in first] for _ in range(2)]
    for _ in range(50):
        for s, o in zip(streams, outs):
            pa.fwd_packed(*args, out=o[0], n_eff=o[1], conf=o[2], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.fwd_packed(*args, out=outs[0][0], n_eff=outs[0][1], conf=outs[0][2])
    args[5].copy_(torch.tensor([0, 10, 500, 1577], dtype=torch.int32))   # other lengths
    graph.replay()
    torch.cuda.synchronize()
    check(args, outs[0], "bf16")
    q, k, v, mem, w, cu = args
    for bad in ((q.transpose(0, 1), k, v, mem, w, cu), (q, k[:5], v, mem, w, cu),
                (q, k, v.float(), mem, w, cu), (q, k, v, mem.transpose(0, 1), w, cu),
                (q, k, v, mem, w[:3], cu), (q, k, v, mem, w, cu.long()), (q[:, :3], k, v, mem[:, :3].contiguous(), w[:3], cu)):
        with pytest.raises((TypeError, ValueError, pa.PolarError)):
            pa.fwd_packed(*bad)
    with pytest.raises(pa.PolarError):
        pa.fwd_packed(*args, out=mem)
    with pytest.raises(ValueError):
        pa.fwd_packed(*args, n_eff=torch.empty(3, device=dev()))
    with pytest.raises(ValueError):
        pa.fwd_packed(q, k, v, mem, w, cu[:0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B", [8300, 33000])
def test_thousands_of_sequences(B, dtype):
    """Short and empty sequences with some long ones far apart among them."""
    import long_context_attention_causal_gb300 as pa
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 4, (B,), generator=g).tolist()
    far = list(range(5, B, B // 9)) + [B - 1]
    for i, b in enumerate(far):
        lens[b] = 300 + 170 * i
    args = case(lens, 4, 2, 64, dtype, B, tail=3)
    got = run(args)
    check(args, got, dtype, seqs=far + list(range(0, B, B // 50)))
    assert (got[1][:sum(lens)] != 77.0).all() and pa.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_descending_offsets_end_the_list(dtype):
    """Sequences that would overlap are not computed, however many they are."""
    import long_context_attention_causal_gb300 as pa
    args = case([50, 0, 60, 40], 4, 2, 64, dtype, 33)
    want = run(args)
    for tail in ([109, 150], [0, 150] * 40000, [-1, 150], [50, 60, 70, 150] * 10):
        bad = args[:5] + [torch.tensor([0, 50, 50, 110] + tail, dtype=torch.int32, device=dev())]
        got = run(bad)
        assert pa.device_status(reset=True) == 3
        for a, b in zip(got, want):
            assert torch.equal(a[:110], b[:110]) and (a[110:] == 77.0).all()


def test_very_long_sequence():
    """200000 tokens: the last rows of the prompt."""
    import long_context_attention_causal_gb300 as pa
    from serving_ref import polar_ref
    n, m = 200000, 60
    args = case([n], 4, 1, 64, "bf16", 43)
    got = run(args)
    t = lambda x: x.transpose(0, 1)  # noqa: E731
    o, ne, c = polar_ref(t(args[0][n - m:]), t(args[1]).expand(4, -1, -1),
                         t(args[2]).expand(4, -1, -1), n - m, args[4], t(args[3][n - m:]))
    assert (t(got[0][n - m:]).double() - o).abs().max() <= TOL["bf16"]["out"]
    assert (t(got[1][n - m:]).double() / ne - 1).abs().max() <= TOL["f32"]["neff"]
    assert (t(got[2][n - m:]).double() - c).abs().max() <= TOL["f32"]["conf"]
    assert pa.device_status() == 0


def test_beside_the_padded_prefill():
    """Short prompts (two CTAs a SM) and padded batches on two streams at once:
    both kernels hold tensor memory, and each gives the bits it gives alone."""
    import long_context_attention_causal_gb300 as pa
    args = case([(37 * i) % 120 + 1 for i in range(300)], 8, 8, 64, "bf16", 61)
    g = torch.Generator(device=dev()).manual_seed(62)
    pad = [torch.randn((2, 8, 700, 64), generator=g, device=dev()).bfloat16() for _ in range(4)]
    want, wide = run(args), pa.fwd(*pad, args[4])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got, other = [], []
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            got.append(run(args))
        with torch.cuda.stream(streams[1]):
            other.append(pa.fwd(*pad, args[4]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x in got for a, b in zip(x, want))
    assert all(torch.equal(x[0], wide[0]) and torch.equal(x[1], wide[1]) for x in other)
    assert pa.device_status() == 0

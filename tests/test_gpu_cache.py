"""Accumulated attention weights of the paged decode, eviction by them, and
the serving loop that uses both beside the linear memory.

Weights: p = exp(s - lse) with |s| <= S.  The logit and the logsumexp each
round a few times at magnitude S log2(e), so the exponent is off by at most
about 8 u S log2(e) and p by 8 u S relative, u = 2^-24; the d-term dot
product adds d u sum|q k| <= d u |q||k| tau / sqrt d.  With |q||k| tau /
sqrt d <= 130 here and d <= 128 the worst case is (8 + 128) 130 u = 1.1e-3;
roundings do not all align, and 2e-5 (an eighth of one per cent of that per
rounding) is what fp32 results are held to throughout.  Evictions copy bits:
they are compared for equality.
"""
import numpy as np
import pytest
import torch

from gpu_util import TOL, dev
from linear_ref import evict_ref, linear_fwd_ref

pytestmark = pytest.mark.gpu


def paged(B, Hq, Hkv, T, d, page, dtype, seed, ragged=True):
    from long_context_attention_causal_gb300 import inputs
    wl = inputs.custom_paged(B, Hq, Hkv, T, d, page, dtype, seed, ragged)
    return inputs.make_paged_decode(wl, "cpu")


def gather(x, name, b):
    n = int(x["seq_lens"][b])
    rows = x[name][x["block_table"][b].long()].double()   # [cols, Hkv, page, d]
    return rows.transpose(0, 1).reshape(rows.shape[1], -1, rows.shape[-1])[:, :n]


def weights_ref(x, b, log_t0=np.log(2048.0)):
    n = int(x["seq_lens"][b])
    k = gather(x, "k_pages", b)
    Hkv, d = k.shape[0], k.shape[-1]
    q = x["q"][b].double().view(Hkv, -1, d)
    tau = max(1.0, np.log(n) / log_t0)
    return torch.softmax(tau / np.sqrt(d) * q @ k.transpose(1, 2), -1).sum(1)


@pytest.mark.parametrize("B,Hq,Hkv,T,d,page,dtype", [
    (2, 4, 4, 100, 64, 8, "bf16"), (3, 8, 4, 300, 128, 16, "bf16"), (2, 8, 2, 777, 64, 64, "bf16"),
    (2, 16, 2, 1500, 128, 128, "bf16"), (2, 8, 1, 5000, 128, 256, "bf16"),
    (2, 4, 4, 100, 128, 8, "f32"), (3, 8, 4, 300, 64, 16, "f32"), (2, 8, 2, 777, 128, 64, "f32"),
    (2, 16, 2, 1500, 64, 32, "f32"), (1, 1, 1, 1, 64, 8, "bf16"), (1, 2, 1, 1, 128, 8, "f32")])
@pytest.mark.parametrize("splits", [0, 3])
def test_weights(B, Hq, Hkv, T, d, page, dtype, splits):
    import long_context_attention_causal_gb300 as pa
    x = paged(B, Hq, Hkv, T, d, page, dtype, 900 + T + d)
    g = {k: t.to(dev()) for k, t in x.items()}
    stride = T + 5
    w = torch.full((B, Hkv, stride), 0.25, device=dev())
    args = [g[k] for k in ("q", "k_pages", "v_pages", "block_table", "seq_lens", "mem", "w_count")]
    got = pa.decode_paged_weights(*args, w, max_seq_len=T, num_splits=splits, want_conf=True)
    same = splits or pa.decode_paged_weights_num_splits(B, Hkv, T, d)
    plain = pa.decode_paged(*args, max_seq_len=T, num_splits=same, want_conf=True)
    for a, b in zip(got, plain):
        assert torch.equal(a, b)   # the decode itself is untouched
    for b in range(B):
        n = int(x["seq_lens"][b])
        ref = weights_ref(x, b)
        have = w[b].double().cpu()
        # 0.25 + p rounds to half a step of 2^-2 .. 2 more
        assert ((have[:, :n] - 0.25 - ref).abs() <= 2e-5 * ref + 2.0 ** -24 * (1 + ref)).all()
        assert (have[:, n:] == 0.25).all()
    pa.decode_paged_weights(*args, w, max_seq_len=T, num_splits=splits)
    first = w.clone()
    w.fill_(0.25)
    for _ in range(2):
        pa.decode_paged_weights(*args, w, max_seq_len=T, num_splits=splits)
    assert torch.equal(w, first)   # no timing in the sums
    assert pa.device_status() == 0


def test_weights_skip_bad_pages_and_clamp_lengths():
    """A page outside the pool gets no weight, and a length past max_seq_len
    does not write past the sums (both are recorded)."""
    import long_context_attention_causal_gb300 as pa
    for dtype in ("bf16", "f32"):
        x = paged(2, 4, 2, 200, 64, 16, dtype, 41, ragged=False)
        x["block_table"][0, 3] = 10 ** 6
        g = {k: t.to(dev()) for k, t in x.items()}
        args = [g[k] for k in ("q", "k_pages", "v_pages", "block_table", "seq_lens", "mem",
                               "w_count")]
        pa.device_status(reset=True)
        w = torch.zeros((2, 2, 200), device=dev())
        pa.decode_paged_weights(*args, w, max_seq_len=200)
        assert pa.device_status(reset=True) == 3
        assert (w[0, :, 48:64] == 0).all() and (w[0, :, 64:] > 0).all()
        torch.testing.assert_close(w[0].sum(-1), torch.full((2,), 2.0, device=dev()), rtol=1e-5,
                                   atol=0)
        # lengths beyond max_seq_len: rows past it get nothing, no other row is touched
        w = torch.full((2, 2, 200), 0.5, device=dev())
        pa.decode_paged_weights(*args, w, max_seq_len=190)
        pa.device_status(reset=True)
        assert torch.isfinite(w).all() and (w[:, :, 190:] == 0.5).all()
        # no valid length at all: nothing is added
        args[4] = torch.tensor([0, -5], dtype=torch.int32, device=dev())
        w.zero_()
        pa.decode_paged_weights(*args, w, max_seq_len=190)
        assert pa.device_status(reset=True) == 3
        assert (w == 0).all()


def test_weights_of_growing_logits():
    """Key norms rise along the sequence, so every split moves its maximum."""
    import long_context_attention_causal_gb300 as pa
    for dtype in ("bf16", "f32"):
        x = paged(2, 8, 2, 900, 128, 32, dtype, 43, ragged=False)
        for b in range(2):
            for j in range(900):
                x["k_pages"][int(x["block_table"][b, j // 32]), :, j % 32] *= 0.5 + 3.0 * j / 900
        g = {k: t.to(dev()) for k, t in x.items()}
        w = torch.zeros((2, 2, 900), device=dev())
        pa.decode_paged_weights(*(g[k] for k in ("q", "k_pages", "v_pages", "block_table",
                                                 "seq_lens", "mem", "w_count")), w)
        for b in range(2):
            ref = weights_ref(x, b)
            assert ((w[b].double().cpu() - ref).abs() <= 2e-5 * ref + 1e-12).all()


def evict_case(B, Hkv, T, d, page, dtype, seed, lens=None):
    g = torch.Generator().manual_seed(seed)
    cols = -(-T // page)
    lens = torch.tensor(lens if lens is not None
                        else [max(0, T - 7 * b * b) for b in range(B)], dtype=torch.int32)
    table = torch.randperm(B * cols, generator=g).to(torch.int32).view(B, cols)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    shape = (B * cols, Hkv, page, d)
    stride = T + 3
    return {"k": torch.randn(shape, generator=g).to(dt), "v": torch.randn(shape, generator=g).to(dt),
            "table": table, "lens": lens,
            "w": torch.exp(2 * torch.randn((B, Hkv, stride), generator=g)),
            "pos": torch.arange(stride, dtype=torch.int32).repeat(B, Hkv, 1)}


def evict_expect(x, keep, recent, page):
    k, v, w, pos = (x[n].clone() for n in ("k", "v", "w", "pos"))
    moves = evict_ref(x["lens"], x["w"].numpy(), x["pos"].numpy(), keep, recent)
    for (b, h), lst in moves.items():
        for src, dst in lst:
            ps, pd = int(x["table"][b, src // page]), int(x["table"][b, dst // page])
            k[pd, h, dst % page] = x["k"][ps, h, src % page]
            v[pd, h, dst % page] = x["v"][ps, h, src % page]
            w[b, h, dst] = x["w"][b, h, src]
            pos[b, h, dst] = x["pos"][b, h, src]
        n = int(x["lens"][b])
        if n > keep:
            w[b, h, keep:n] = 0
    return k, v, w, pos, torch.clamp(x["lens"], max=keep)


def run_evict(x, keep, recent, T, **kw):
    import long_context_attention_causal_gb300 as pa
    g = {n: t.to(dev()) for n, t in x.items()}
    new = pa.cache_evict(g["k"], g["v"], g["table"], g["lens"], g["w"], g["pos"], keep,
                         recent=recent, max_seq_len=T, **kw)
    torch.cuda.synchronize()
    return [t.cpu() for t in (g["k"], g["v"], g["w"], g["pos"], new)]


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("B,Hkv,T,d,page,dtype,keep,recent", [
    (1, 1, 9, 64, 8, "bf16", 1, 0), (1, 2, 9, 64, 8, "bf16", 8, 8), (3, 2, 100, 128, 16, "bf16", 60, 7),
    (2, 4, 257, 64, 64, "f32", 256, 256), (2, 3, 1000, 128, 32, "f32", 333, 50),
    (4, 2, 1025, 64, 8, "bf16", 1000, 100), (2, 1, 4100, 64, 128, "bf16", 2048, 0),
    (1, 1, 33000, 64, 256, "bf16", 5000, 300), (2, 2, 64, 64, 64, "bf16", 64, 3),
    (2, 2, 64, 64, 64, "bf16", 100, 3), (1, 1, 70001, 64, 1024, "bf16", 69000, 10)])
def test_evict(B, Hkv, T, d, page, dtype, keep, recent):
    x = evict_case(B, Hkv, T, d, page, dtype, 11 + T)
    want = evict_expect(x, keep, recent, page)
    for got, ref, name in zip(run_evict(x, keep, recent, T), want, ("k", "v", "w", "pos", "lens")):
        assert same_bits(got, ref), name


def test_evict_ties_and_odd_weights():
    """Equal weights, zeros of both signs, infinities, NaN and negatives."""
    T, keep, page = 500, 200, 16
    for pattern in ("equal", "zeros", "few", "special"):
        x = evict_case(2, 2, T, 64, page, "bf16", 77)
        w = x["w"]
        if pattern == "equal":
            w.fill_(0.125)
        elif pattern == "zeros":
            w.zero_()
            w[..., ::3] = -0.0
            w[..., 5::7] = 1e-30
        elif pattern == "few":
            w.copy_(torch.randint(0, 3, w.shape, generator=torch.Generator().manual_seed(1)))
        else:
            w[..., ::5] = float("nan")
            w[..., 1::11] = float("inf")
            w[..., 2::13] = -float("inf")
            w[..., 3::7] = -1.5
        for recent in (0, 13):
            want = evict_expect(x, keep, recent, page)
            for got, ref, name in zip(run_evict(x, keep, recent, T), want,
                                      ("k", "v", "w", "pos", "lens")):
                assert same_bits(got, ref), (pattern, recent, name)


@pytest.mark.parametrize("T,keep", [(40000, 17001), (40000, 39999), (70001, 30000)])
def test_evict_long_ties(T, keep):
    """Many equal rows on both sides of the cut and across the warps' runs, with
    the keys in shared memory and without."""
    x = evict_case(1, 2, T, 64, 256, "bf16", 78)
    g = torch.Generator().manual_seed(2)
    x["w"][0, 0] = torch.randint(0, 3, x["w"].shape[2:], generator=g).float()
    x["w"][0, 1] = (torch.arange(x["w"].shape[2]) // 5000).float()
    for recent in (0, 700):
        want = evict_expect(x, keep, recent, 256)
        for got, ref, name in zip(run_evict(x, keep, recent, T), want,
                                  ("k", "v", "w", "pos", "lens")):
            assert same_bits(got, ref), (recent, name)


def test_evict_permuted_and_equal_positions():
    """Protection goes by position, wherever the rows lie; more protected
    rows than `keep` (equal positions) still leave exactly `keep`."""
    T, page = 300, 16
    x = evict_case(1, 2, T, 64, page, "bf16", 5)
    perm = torch.stack([torch.randperm(T + 3, generator=torch.Generator().manual_seed(s))
                        for s in (1, 2)])
    x["pos"] = perm[None].to(torch.int32).contiguous()
    for got, ref in zip(run_evict(x, 100, 40, T), evict_expect(x, 100, 40, page)):
        assert same_bits(got, ref)
    x["pos"].fill_(7)
    for got, ref in zip(run_evict(x, 100, 40, T), evict_expect(x, 100, 40, page)):
        assert same_bits(got, ref)
    x["pos"].fill_(-2 ** 31)
    for got, ref in zip(run_evict(x, 100, 40, T), evict_expect(x, 100, 40, page)):
        assert same_bits(got, ref)


def test_evict_lengths_in_place_and_again():
    """new_lens may be seq_lens; a second call finds nothing to do."""
    import long_context_attention_causal_gb300 as pa
    x = evict_case(5, 2, 400, 64, 32, "bf16", 6, lens=[400, 0, 100, 101, 399])
    g = {n: t.to(dev()) for n, t in x.items()}
    pa.cache_evict(g["k"], g["v"], g["table"], g["lens"], g["w"], g["pos"], 100, recent=9,
                   max_seq_len=400, new_lens=g["lens"])
    assert g["lens"].tolist() == [100, 0, 100, 100, 100]
    for got, ref in zip((g["k"], g["v"], g["w"], g["pos"]), evict_expect(x, 100, 9, 32)):
        assert same_bits(got.cpu(), ref)
    before = {n: t.clone() for n, t in g.items()}
    pa.cache_evict(g["k"], g["v"], g["table"], g["lens"], g["w"], g["pos"], 100, recent=9,
                   max_seq_len=400, new_lens=g["lens"])
    for n in g:
        assert same_bits(g[n].cpu(), before[n].cpu())


def test_evict_bad_pages_and_lengths():
    """Pages outside the pool are not touched, lengths are clamped; both are
    recorded."""
    import long_context_attention_causal_gb300 as pa
    pa.device_status(reset=True)
    x = evict_case(1, 1, 200, 64, 16, "bf16", 8)
    x["table"][0, 2] = -1
    x["table"][0, 9] = 10 ** 6
    good = evict_case(1, 1, 200, 64, 16, "bf16", 8)
    want = evict_expect(good, 100, 0, 16)
    got = run_evict(x, 100, 0, 200)
    assert pa.device_status(reset=True) == 3
    assert same_bits(got[2], want[2]) and same_bits(got[3], want[3])
    for bad, clamped in ((999, 200), (-4, 0)):
        y = evict_case(1, 1, 200, 64, 16, "bf16", 8, lens=[bad])
        z = evict_case(1, 1, 200, 64, 16, "bf16", 8, lens=[clamped])
        got = run_evict(y, 100, 5, 200)
        assert pa.device_status(reset=True) == 3
        for a, b in zip(got, evict_expect(z, 100, 5, 16)):
            assert same_bits(a, b)


def test_evict_capture():
    import long_context_attention_causal_gb300 as pa
    x = evict_case(3, 2, 500, 64, 32, "bf16", 9)
    g = {n: t.to(dev()) for n, t in x.items()}
    ws = torch.empty(pa.cache_evict_workspace_bytes(3, 2, 500, 120), device=dev(),
                     dtype=torch.uint8)
    new = torch.empty_like(g["lens"])

    def call():
        pa.cache_evict(g["k"], g["v"], g["table"], g["lens"], g["w"], g["pos"], 120, recent=20,
                       max_seq_len=500, new_lens=new, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    y = evict_case(3, 2, 500, 64, 32, "bf16", 10)
    for n in g:
        g[n].copy_(y[n].to(dev()))
    graph.replay()
    torch.cuda.synchronize()
    for got, ref in zip((g["k"], g["v"], g["w"], g["pos"], new), evict_expect(y, 120, 20, 32)):
        assert same_bits(got.cpu(), ref)


def test_refusals():
    import long_context_attention_causal_gb300 as pa
    x = evict_case(2, 2, 100, 64, 16, "bf16", 3)
    g = {n: t.to(dev()) for n, t in x.items()}
    a = [g[n] for n in ("k", "v", "table", "lens", "w", "pos")]
    with pytest.raises(pa.PolarError):
        pa.cache_evict(*a, 0)
    with pytest.raises(pa.PolarError):
        pa.cache_evict(*a, 10, recent=11)
    with pytest.raises(pa.PolarError):
        pa.cache_evict(*a, 10, max_seq_len=10 ** 6)
    with pytest.raises(pa.PolarError):
        pa.cache_evict(*a, 10, workspace=torch.empty(16, device=dev(), dtype=torch.uint8))
    with pytest.raises(ValueError):
        pa.cache_evict(*a[:4], g["w"][:1].contiguous(), g["pos"], 10)
    with pytest.raises(ValueError):
        pa.cache_evict(*a[:5], g["pos"][..., :50].contiguous(), 10)
    with pytest.raises(TypeError):
        pa.cache_evict(*a[:5], g["pos"].long(), 10)
    with pytest.raises(TypeError):
        pa.cache_evict(*a[:3], g["lens"].cpu(), *a[4:], 10)
    p = paged(2, 4, 2, 100, 64, 16, "bf16", 1)
    h = [p[n].to(dev()) for n in ("q", "k_pages", "v_pages", "block_table", "seq_lens", "mem",
                                  "w_count")]
    with pytest.raises(ValueError):
        pa.decode_paged_weights(*h, torch.zeros((2, 4, 112), device=dev()))
    with pytest.raises(TypeError):
        pa.decode_paged_weights(*h, torch.zeros((2, 2, 112), device=dev(), dtype=torch.bfloat16))
    with pytest.raises(pa.PolarError):
        pa.decode_paged_weights(*h, torch.zeros((2, 2, 90), device=dev()), max_seq_len=100)


def test_serving_loop():
    """A prompt, then tokens: the linear memory makes the memory stream of
    the prefill and of every decode, the decode sums its rows' weights, and
    the cache is cut whenever it reaches its bound.  Every step is compared
    with the same loop in fp64 on the rows that the fp64 loop keeps."""
    import long_context_attention_causal_gb300 as pa
    B, H, d, page, T, steps, keep, recent = 2, 2, 64, 16, 90, 40, 96, 24
    bound = keep + 16
    g = torch.Generator(device=dev()).manual_seed(3)
    r = lambda *s, std=1.0: (torch.randn(s, generator=g, device=dev()) * std).bfloat16()  # noqa: E731
    n_all = T + steps
    q, k, v, mq, mk, mv = (r(B, H, n_all, d) for _ in range(6))
    w_count = torch.randn((H, d), generator=g, device=dev()) * 0.02
    ld = torch.tensor([-0.1, -0.01], device=dev())
    cut = lambda t: t[:, :, :T].contiguous()  # noqa: E731
    mem, state = pa.linear_fwd(cut(mq), cut(mk), cut(mv), ld, want_state=True)
    out, _, _ = pa.fwd(cut(q), cut(k), cut(v), mem, w_count)
    assert torch.isfinite(out.float()).all()
    cols = -(-bound // page)
    table = torch.arange(B * cols, dtype=torch.int32, device=dev()).view(B, cols)
    kp = torch.zeros((B * cols, H, page, d), dtype=torch.bfloat16, device=dev())
    vp = torch.zeros_like(kp)
    weights = torch.zeros((B, H, cols * page), device=dev())
    positions = torch.zeros((B, H, cols * page), dtype=torch.int32, device=dev())
    lens = torch.full((B,), T, dtype=torch.int32, device=dev())
    kept = [[list(range(T)) for _ in range(H)] for _ in range(B)]  # fp64 loop: token per row
    sums = torch.zeros((B, H, cols * page), dtype=torch.float64)

    def put(j, t):
        for b in range(B):
            pg = int(table[b, j // page])
            kp[pg, :, j % page] = k[b, :, t]
            vp[pg, :, j % page] = v[b, :, t]
        positions[:, :, j] = t

    for t in range(T):
        put(t, t)
    ref_mem, _ = linear_fwd_ref(mq, mk, mv, ld, d ** -0.5)
    evictions = 0
    for t in range(T, n_all):
        tok = lambda x: x[:, :, t].contiguous()  # noqa: E731
        m = pa.linear_step(state, tok(mq), tok(mk), tok(mv), ld)
        err = float((m.double() - ref_mem[:, :, t]).norm() / ref_mem[:, :, t].norm())
        assert err <= 4.6e-3
        j = int(lens[0])
        put(j, t)
        for b in range(B):
            for h in range(H):
                kept[b][h].append(t)
        lens += 1
        o, _, _ = pa.decode_paged_weights(tok(q), kp, vp, table, lens, m, w_count, weights,
                                          max_seq_len=bound)
        n = j + 1
        for b in range(B):
            for h in range(H):
                rows = torch.tensor(kept[b][h], device=dev())
                s = (k[b, h, rows].double() @ q[b, h, t].double()) * d ** -0.5
                p = torch.softmax(s, 0)
                sums[b, h, :n] += p.cpu()
                u = p @ v[b, h, rows].double()
                u = u / u.norm()
                floor = q[b, h, t].double().norm() * d ** -0.5 * np.sqrt(2 * np.log(n))
                conf = torch.sigmoid(torch.logsumexp(s, 0) - floor)
                count = conf * torch.tanh(-torch.log((p * p).sum()) / np.log(2048.0))
                ref = u + count * w_count[h].double() + m[b, h].double()
                # TOL is for results near 1; this memory reaches 14, and a bf16
                # result of size x is off by up to 2^-8 x by its rounding alone
                assert ((o[b, h].double() - ref).abs()
                        <= TOL["bf16"]["out"] + 2.0 ** -8 * ref.abs()).all()
        assert ((weights[:, :, :n].double().cpu() - sums[:, :, :n]).abs()
                <= 2e-5 * sums[:, :, :n] + 1e-9).all()
        if n == bound:
            # the library's own sums select on both sides (a near tie may
            # fall either way in fp32 and fp64)
            w, p = weights.cpu().numpy(), positions.cpu().numpy()
            moves = evict_ref([n] * B, w, p, keep, recent)
            pa.cache_evict(kp, vp, table, lens, weights, positions, keep, recent=recent,
                           max_seq_len=bound, new_lens=lens)
            for (b, h), lst in moves.items():
                for src, dst in lst:
                    kept[b][h][dst] = kept[b][h][src]
                    sums[b, h, dst] = sums[b, h, src]
                del kept[b][h][keep:]
                sums[b, h, keep:] = 0
                assert positions[b, h, :keep].tolist() == kept[b][h]
            assert lens.tolist() == [keep] * B
            evictions += 1
    assert evictions == 2 and pa.device_status() == 0

"""4-bit decode: outputs row by row in their 2-norm, and batches and lengths that
other tests do not reach.

A bf16 row: the result's rounding is at most 2^-8 of each channel, the weights'
(times V's scales) at most 2^-8 of each key's share, for values that are nearly
orthogonal 2^-8 of the norm: 2^-7 together.  Both are uniform in half a step, whose
rms is 2^-8 / sqrt(3) of the number at most: over all rows sqrt(2/3) 2^-8, 3.2e-3.
(One wrong row of V among n of equal weights moves a row by sqrt(2 / n).)
"""
import math

import pytest
import torch

from gpu_util import TOL, dev
from serving_ref import LOG_T0, decode_ref
from test_gpu_decode_q4 import case, check

pytestmark = pytest.mark.gpu

ROW = 2.0 ** -7
RMS = 3.2e-3


def distances(args, values, out, rows):
    """|out - reference| / |reference| of every row."""
    far = []
    for b in rows:
        o, _, _ = decode_ref(args[0][b], *values[b], args[6], args[5][b])
        far.append((out[b].double() - o).norm(dim=-1) / o.norm(dim=-1))
    return torch.stack(far)


@pytest.mark.parametrize("Hq,Hkv,lens,d,page", [
    (1, 1, [1], 64, 8), (8, 1, [1, 2, 3], 128, 8), (4, 4, [100, 8, 9], 64, 8),
    (16, 2, [777, 128, 129, 127], 64, 64), (8, 8, [4000, 33], 128, 256),
    (32, 4, [1100, 1024, 1], 64, 1024), (16, 4, [9000, 5000, 14000], 128, 64)])
@pytest.mark.parametrize("runs", [0, 5, 700])
def test_rows_in_norm(Hq, Hkv, lens, d, page, runs):
    import long_context_attention_causal_gb300 as pa
    args, values = case(len(lens), Hq, Hkv, lens, d, page, "bf16", 70 + d + len(lens))
    args[5].zero_()
    got = pa.decode_paged_q4(*args, max_seq_len=max(lens), num_runs=runs)
    far = distances(args, values, got[0], range(len(lens)))
    assert far.max() <= ROW and far.square().mean().sqrt() <= RMS
    assert pa.device_status() == 0


def masked_ref(q, k, v, w, mem, keep):
    """decode_ref with n the length and sums over the keys of `keep` alone."""
    G, n, d = q.shape[0] // k.shape[0], k.shape[1], q.shape[1]
    k, v = (t[:, keep].double().repeat_interleave(G, 0) for t in (k, v))
    q, w, mem = q.double(), w.double(), mem.double()
    tau = max(1.0, math.log(n) / LOG_T0)
    s = torch.einsum("hd,hnd->hn", q, k) * tau / math.sqrt(d)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    n_eff = 1.0 / p.square().sum(-1)
    conf = torch.sigmoid(lse - tau * q.norm(dim=-1) / math.sqrt(d) * math.sqrt(2 * math.log(n)))
    a = torch.einsum("hn,hnd->hd", p, v)
    a = a / a.norm(dim=-1, keepdim=True).clamp(min=1e-6)
    return a + (conf * torch.tanh(n_eff.log() / LOG_T0))[:, None] * w + mem, n_eff, conf


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [8, 16, 256])
def test_keys_of_bad_pages(dtype, page):
    """Pages outside the pool: their keys are left out of the sums; temperature
    and floor follow the length."""
    import long_context_attention_causal_gb300 as pa
    lens = [2900, 90]
    args, values = case(2, 4, 2, lens, 64, page, dtype, 21)
    bad = [1, 5, 11]
    keep = torch.ones(2900, dtype=torch.bool, device=dev())
    for i, at in enumerate(bad):
        args[3][0, at] = (args[1].shape[0], -1, 1 << 30)[i]
        keep[at * page:(at + 1) * page] = False
    got = pa.decode_paged_q4(*args, max_seq_len=2900, want_conf=True)
    assert pa.device_status(reset=True) == 3
    check(args, values, got, dtype, rows=[1])
    o, ne, c = masked_ref(args[0][0], *values[0], args[6], args[5][0], keep)
    if dtype == "bf16":
        assert ((got[0][0].double() - o).norm(dim=-1) / o.norm(dim=-1)).max() <= ROW
    else:
        assert (got[0][0].double() - o).abs().max() <= TOL["f32"]["out"]
    assert (got[1][0].double() / ne - 1).abs().max() <= TOL["f32"]["neff"]
    assert (got[2][0].double() - c).abs().max() <= TOL["f32"]["conf"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("limit", [200, 256, 1])
def test_lengths_past_the_limit(dtype, limit):
    """A length above max_seq_len is cut to it, and recorded."""
    import long_context_attention_causal_gb300 as pa
    lens = [90, 400, 130]
    args, values = case(3, 8, 2, lens, 128, 16, dtype, 22)
    got = pa.decode_paged_q4(*args, max_seq_len=limit, want_conf=True)
    assert pa.device_status(reset=True) == 3
    cut = [min(n, limit) for n in lens]
    check(args, [tuple(x[:, :n] for x in kv) for kv, n in zip(values, cut)], got, dtype)
    args[4].copy_(torch.tensor(cut, dtype=torch.int32))
    want = pa.decode_paged_q4(*args, max_seq_len=limit, want_conf=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and pa.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,top,runs", [(75, 700, 0), (97, 300, 37), (200, 260, 1000)])
def test_many_sequences(B, top, runs, dtype):
    """More sequences than lanes, empty ones between them."""
    import long_context_attention_causal_gb300 as pa
    g = torch.Generator().manual_seed(B)
    lens = [int(n) if n % 3 else 0 for n in torch.randint(1, top, (B,), generator=g)]
    lens[0] = lens[31] = lens[32] = lens[64] = 0
    lens[33], lens[B - 1] = top, 5
    args, values = case(B, 4, 2, lens, 64, 16, dtype, B)
    got = pa.decode_paged_q4(*args, max_seq_len=top, num_runs=runs, want_conf=True)
    assert pa.device_status(reset=True) == 3      # lengths of 0
    live = [b for b in range(B) if lens[b]]
    check(args, values, got, dtype, rows=live)
    if dtype == "bf16":
        assert distances(args, values, got[0], live).square().mean().sqrt() <= RMS
    for b in set(range(B)) - set(live):
        assert torch.equal(got[0][b], args[5][b])
        assert (got[1][b] == 0).all() and (got[2][b] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_more_records_than_threads(dtype, d):
    """One pair of 1501 records, joined in more than one block of them."""
    import long_context_attention_causal_gb300 as pa
    n = 1500 * 128 + 77
    args, values = case(1, 4, 1, [n], d, 64, dtype, 23)
    got = pa.decode_paged_q4(*args, max_seq_len=n, num_runs=3000, want_conf=True)
    check(args, values, got, dtype)
    if dtype == "bf16":
        assert distances(args, values, got[0], [0]).max() <= ROW
    assert pa.device_status() == 0

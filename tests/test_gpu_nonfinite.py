"""One NaN channel in one row of V.

The direction is acc / max(|acc|, eps), and |acc| of a row that saw the NaN is
not a number, so every channel of that row's out is none; l, sum p^2 and the
gate follow K alone, so n_eff and conf are those of the clean call to the bit.
Rows that do not see it keep their bits.
"""
import math

import pytest
import torch

from gpu_util import dev
from test_gpu_decode_q4 import case as q4_case
from test_gpu_packed import case as packed_case, run as run_packed

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,G", [(64, 1), (128, 2), (64, 8), (128, 4)])
def test_packed_prefill(dtype, d, G):
    import long_context_attention_causal_gb300 as pa
    args = packed_case([70, 300, 40], 2 * G, 2, d, dtype, 3)
    clean = run_packed(args)
    token = 70 + 137      # of the second sequence, inside a key tile
    args[2][token, 1, 5] = math.nan
    got = run_packed(args)
    own = slice(G, 2 * G)  # query heads of KV head 1
    assert got[0][token:370, own].isnan().all()
    for a, b in zip(got[1:], clean[1:]):
        assert torch.equal(a, b)
    for rows in (slice(0, 70), slice(370, 410)):
        assert torch.equal(got[0][rows], clean[0][rows])
    assert torch.equal(got[0][:, :G], clean[0][:, :G])
    assert pa.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,Hq,runs", [(64, 4, 0), (128, 16, 0), (128, 2, 1), (64, 8, 700)])
def test_decode_q4(dtype, d, Hq, runs):
    """The scale NaN in one group of 32 channels, as the append leaves it."""
    import long_context_attention_causal_gb300 as pa
    page, lens = 16, [150, 400, 150]
    args, _ = q4_case(3, Hq, 2, lens, d, page, dtype, 12)
    clean = pa.decode_paged_q4(*args, max_seq_len=400, num_runs=runs, want_conf=True)
    block = args[2].flatten(2)[int(args[3][1, 13]), 1]   # rows 208 .. 223, KV head 1
    at = page * d // 2 + 5 * (d // 16) + 2
    block[at], block[at + 1] = 0xFF, 0x7F
    got = pa.decode_paged_q4(*args, max_seq_len=400, num_runs=runs, want_conf=True)
    own = slice(Hq // 2, Hq)
    assert got[0][1, own].isnan().all()
    for a, b in zip(got[1:], clean[1:]):
        assert torch.equal(a, b)
    assert torch.equal(got[0][1, :Hq // 2], clean[0][1, :Hq // 2])
    assert torch.equal(got[0][0], clean[0][0]) and torch.equal(got[0][2], clean[0][2])
    assert pa.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_padded_prefill_and_decode(dtype, d):
    import long_context_attention_causal_gb300 as pa
    g = torch.Generator(device=dev()).manual_seed(8)
    q, k, v, mem = (torch.randn((2, 3, 200, d), generator=g, device=dev()).to(DT[dtype])
                    for _ in range(4))
    w = torch.randn((3, d), generator=g, device=dev()) * 0.02
    bad = v.clone()
    bad[1, 2, 131, 7] = math.nan
    clean, got = (pa.fwd(q, k, x, mem, w, want_conf=True) for x in (v, bad))
    assert got[0][1, 2, 131:].isnan().all()
    assert torch.equal(got[0][0], clean[0][0]) and torch.equal(got[0][1, :2], clean[0][1, :2])
    assert torch.equal(got[1], clean[1]) and torch.equal(got[2], clean[2])
    q1, mem1 = q[:, :, 0].contiguous(), mem[:, :, 0].contiguous()
    clean, got = (pa.decode(q1, k, x, mem1, w, want_conf=True) for x in (v, bad))
    assert got[0][1, 2].isnan().all()
    assert torch.equal(got[0][0], clean[0][0]) and torch.equal(got[0][1, :2], clean[0][1, :2])
    assert torch.equal(got[1], clean[1]) and torch.equal(got[2], clean[2])
    assert pa.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32", "bf16 statistics"])
@pytest.mark.parametrize("d", [64, 128])
def test_gradients(dtype, d):
    """The rows that see the NaN have no gradient of a direction: every row of
    the head's dv (all are seen by one of them) and theirs of dq hold NaN alone,
    not the gradient of a direction of norm eps.  Other heads keep their bits."""
    import long_context_attention_causal_gb300 as pa
    dt = DT[dtype.split()[0]]
    g = torch.Generator(device=dev()).manual_seed(9)
    q, k, v, mem, dout = (torch.randn((2, 2, 300, d), generator=g, device=dev()).to(dt)
                          for _ in range(5))
    w = torch.randn((2, d), generator=g, device=dev()) * 0.02
    bad = v.clone()
    bad[1, 0, 201, 7] = math.nan

    def grads(v):
        if dtype == dtype.split()[0]:
            return pa.bwd(q, k, v, w, dout)
        return pa.bwd_stats(q, k, v, mem, w, *pa.fwd_stats(q, k, v, mem, w), dout)

    clean, got = grads(v), grads(bad)
    assert got[2][1, 0].isnan().all() and got[0][1, 0, 201:].isnan().all()
    assert got[1][1, 0, :202].isnan().all()
    for a, b in zip(got[:3], clean[:3]):
        assert torch.isfinite(b).all()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1, 1], b[1, 1])
    assert pa.device_status() == 0

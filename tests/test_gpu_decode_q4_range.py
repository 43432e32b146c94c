"""4-bit decode at the ends of its ranges."""
import pytest
import torch

from gpu_util import TOL, dev
from serving_ref import decode_ref

pytestmark = pytest.mark.gpu

ROW = 2.0 ** -7   # bf16, in a row's 2-norm: the result's rounding and the weights', 2^-8 each


def pages_of(k, v, page):
    """(k_pages, v_pages, table, seq_lens) of one sequence of rows [n, Hkv, d]."""
    import long_context_attention_causal_gb300 as pa
    n, Hkv, d = k.shape
    pool = -(-n // page)
    kp, vp = pa.cache_q4(pool, Hkv, page, d)
    pa.cache_append_q4(k, v, torch.arange(n, dtype=torch.int32, device=dev()), kp, vp)
    table = torch.arange(pool, dtype=torch.int32, device=dev())[None]
    return kp, vp, table, torch.tensor([n], dtype=torch.int32, device=dev())


@pytest.mark.parametrize("dtype,tol", [("bf16", ROW), ("f32", 2.0 ** -17)])
@pytest.mark.parametrize("power", [-30, -10, 40, 50])
@pytest.mark.parametrize("d,runs", [(128, 0), (64, 1)])
def test_scales_of_values(power, d, runs, dtype, tol):
    """Aligned rows of V with scales at both ends of the range.  fp32: a weight
    is off by 2^-22 (ex2), 2^-20 (its exponent) and 2^-19 (a score below 8 of 24
    bits), a sum by 2^-20."""
    import long_context_attention_causal_gb300 as pa
    g = torch.Generator(device=dev()).manual_seed(31)
    n, Hq, Hkv = 4000, 8, 2
    k = torch.randn((n, Hkv, d), generator=g, device=dev())
    v = torch.rand((1, Hkv, d), generator=g, device=dev()) * 6.0 + \
        torch.rand((n, Hkv, d), generator=g, device=dev())
    v[..., ::32] = 7.0                       # a group's scale: 2^power
    v = v * 2.0 ** power
    kp, vp, table, lens = pages_of(k, v, 64)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    q = torch.randn((1, Hq, d), generator=g, device=dev()).to(dt)
    zero, w = torch.zeros_like(q), torch.zeros((Hq, d), device=dev())
    out, n_eff, _ = pa.decode_paged_q4(q, kp, vp, table, lens, zero, w, num_runs=runs)
    slots = torch.arange(n, dtype=torch.int32, device=dev())
    k4, v4 = (x.transpose(0, 1) for x in pa.cache_read_q4(kp, vp, slots, dtype=torch.float32))
    o, ne, _ = decode_ref(q[0], k4, v4, w, zero[0])
    assert ((out[0].double() - o).norm(dim=-1) / o.norm(dim=-1)).max() <= tol
    assert (n_eff[0].double() / ne - 1).abs().max() <= TOL["f32"]["neff"]
    assert pa.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("power", [-30, 50])
def test_scales_of_keys(power, dtype):
    """K times a power of two and q by its inverse: the same scores, bit for bit."""
    import long_context_attention_causal_gb300 as pa
    g = torch.Generator(device=dev()).manual_seed(32)
    n, Hq, Hkv, d = 2500, 8, 2, 128
    k = torch.rand((n, Hkv, d), generator=g, device=dev()) * 2.0 - 1.0
    k[..., ::32] = 1.75                      # a group's scale: 1/4
    v = torch.randn((n, Hkv, d), generator=g, device=dev())
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    q = torch.randn((1, Hq, d), generator=g, device=dev()).to(dt)
    mem = torch.randn((1, Hq, d), generator=g, device=dev()).to(dt)
    w = torch.zeros((Hq, d), device=dev())
    want = pa.decode_paged_q4(q, *pages_of(k, v, 32), mem, w)
    by = 2.0 ** (power + 2)
    got = pa.decode_paged_q4(q / by, *pages_of(k * by, v, 32), mem, w)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert pa.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_keep_fp32(dtype):
    """n_eff of one key of weight 1 beside 1023 of one weight w = 2^-6 to 2^-8, whose
    scores are exact: q and k have one channel each, d = 64 and no temperature.
    With S = 1023 w and R = 1023 w^2, an error e of w moves n_eff by 2 e (S / (1 + S) -
    R / (1 + R)), below 1.8 e.  e: the exponent, below 8, is rounded to half of
    2^-21, ln 2 times that (rms 1 / sqrt(3) of it) 1e-7; ex2 2.4e-7; log2(e) in the
    scale 0.7e-7; a sum of 1023 equal numbers 1.5e-7 rms.  In all below 2^-20 rms (with
    exponents near 40, half of 2^-18, it is 1.3e-6)."""
    import long_context_attention_causal_gb300 as pa
    B, Hq, d, n, page = 64, 8, 64, 1024, 64
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    scale = ((1.0 + torch.arange(B, device=dev()) / 512.0).bfloat16()).float()
    k = torch.zeros((B, n, 1, d), device=dev())
    k[:, :, 0, 3] = -7.0 * scale[:, None]
    k[:, 500, 0, 3] *= -1.0
    v = torch.ones((B * n, 1, d), device=dev())
    kp, vp = pa.cache_q4(B * n // page, 1, page, d)
    slots = torch.arange(B * n, dtype=torch.int32, device=dev())
    pa.cache_append_q4(k.view(B * n, 1, d), v, slots, kp, vp)
    back, _ = pa.cache_read_q4(kp, vp, slots, dtype=torch.float32)
    assert torch.equal(back, k.view(B * n, 1, d))
    q = torch.zeros((B, Hq, d), device=dev(), dtype=dt)
    q[..., 3] = (2.4 + 0.05 * torch.arange(Hq, device=dev())).bfloat16().to(dt)
    table = torch.arange(B * n // page, dtype=torch.int32, device=dev()).view(B, -1)
    lens = torch.full((B,), n, dtype=torch.int32, device=dev())
    got = pa.decode_paged_q4(q, kp, vp, table, lens, torch.zeros_like(q),
                             torch.zeros((Hq, d), device=dev()))
    x = -14.0 * q[..., 3].double() * scale.double()[:, None] / 8.0
    weight = torch.exp(x)
    assert (weight > 2.0 ** -8).all() and (weight < 2.0 ** -5.5).all()
    want = (1 + (n - 1) * weight) ** 2 / (1 + (n - 1) * weight ** 2)
    far = (got[1].double() / want - 1).square().mean().sqrt()
    assert far <= 2.0 ** -20
    assert pa.device_status() == 0

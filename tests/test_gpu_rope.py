"""Rotary positions against fp64.

|y| <= scale (|x_a| + |x_b|).  Rounding of one result: the cosine and sine are
off by at most 2^-32 of a turn in the angle, 2^-25 pi from the angle's
rounding to fp32 half turns, and 2^-22 from their own evaluation and the
scale's product, together below 4 2^-22; the two products and the sum add 2
2^-24.  So fp32 results are within 5 2^-22 (|x_a| + |x_b|) scale; bf16 ones
add half a step, 2^-8 of the result at most (2^-9 of its binade's top).
"""
import math

import pytest
import torch

from gpu_util import dev
from serving_ref import rope_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(N, Hq, Hkv, d, dtype, seed, far=1 << 20):
    g = torch.Generator(device=dev()).manual_seed(seed)
    qkv = torch.randn((N, Hq + 2 * Hkv, d), generator=g, device=dev()).to(DT[dtype])
    pos = torch.randint(0, far, (N,), generator=g, device=dev(), dtype=torch.int32)
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], pos


def check(got, x, pos, f, scale=1.0, interleaved=False, inverse=False):
    want = rope_ref(x, pos, f, scale, interleaved, inverse)
    rot = 2 * f.shape[0]
    assert got.dtype == x.dtype
    assert torch.equal(got[..., rot:], x[..., rot:])
    size = x.double().abs()
    pair = torch.zeros_like(size)
    if interleaved:
        both = size[..., :rot:2] + size[..., 1:rot:2]
        pair[..., :rot:2] = pair[..., 1:rot:2] = both
    else:
        both = size[..., :rot // 2] + size[..., rot // 2:rot]
        pair[..., :rot // 2] = pair[..., rot // 2:rot] = both
    tol = 5 * 2.0 ** -22 * pair * abs(scale)
    if x.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("N,Hq,Hkv,d,rot", [
    (1, 1, 1, 64, 64), (1, 16, 2, 128, 128), (3, 8, 8, 64, 16), (77, 6, 3, 128, 96), (200, 32, 8, 128, 64),
    (1000, 5, 1, 64, 48), (31, 4, 2, 64, 26), (50, 4, 4, 128, 2), (9, 3, 1, 128, 126), (5000, 16, 4, 128, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(N, Hq, Hkv, d, rot, dtype, interleaved, inverse):
    import long_context_attention_causal_gb300 as pa
    q, k, pos = make(N, Hq, Hkv, d, dtype, N + rot)
    f, _ = pa.rope_inv_freq(rot)
    kw = dict(scale=1.25, interleaved=interleaved, inverse=inverse)
    q0, k0 = q.clone(), k.clone()
    qo, ko = pa.rope(q, k, pos, f, **kw)
    assert qo.is_contiguous() and torch.equal(q, q0) and torch.equal(k, k0)
    check(qo, q, pos, f, **kw)
    check(ko, k, pos, f, **kw)
    # in place, inside the projection's output: the same bits
    a, b = pa.rope(q, k, pos, f, q_out=q, k_out=k, **kw)
    assert a is q and torch.equal(q, qo) and torch.equal(k, ko)
    # q alone
    qo2, none = pa.rope(q0, None, pos, f, **kw)
    assert none is None and torch.equal(qo2, qo)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_and_negative_positions(dtype):
    import long_context_attention_causal_gb300 as pa
    far = [0, 1, -1, 1 << 24, (1 << 24) + 1, -(1 << 30), (1 << 31) - 1, -(1 << 31), 1048577, 999983]
    q, k, _ = make(len(far), 2, 1, 128, dtype, 5)
    pos = torch.tensor(far, dtype=torch.int32, device=dev())
    f, _ = pa.rope_inv_freq(128)
    # a double frequency turns 2^31 tokens to 2^-53 * 2^31 / (2 pi) = 4e-8 of a turn
    # in fp64 as well: the slow pairs are exact, the fastest are held to that
    f = torch.round(f * 2.0 ** 24) / 2.0 ** 24
    qo, ko = pa.rope(q, k, pos, f)
    near = torch.tensor([abs(p) <= 1 << 24 for p in far], device=dev())
    check(qo[near], q[near], pos[near], f)
    check(ko[near], k[near], pos[near], f)
    ref = rope_ref(q, pos, f)
    # fp64 angles of 2^31 radians are off by 2^-22, the library's by 2^-53 2^31 turns
    tol = (2.0 ** -20 + 2.0 ** -19 + (2.0 ** -8 if dtype == "bf16" else 0)) * 2 * q.double().abs().amax()
    assert ((qo.double() - ref).abs() <= tol).all()
    assert not torch.equal(qo[3], qo[4])  # neighbours that one fp32 number would name


def test_strides_that_are_not_16_bytes():
    """Tokens an odd number of elements apart: the narrow accesses, the same
    results as the wide ones up to the last bit's rounding (none)."""
    import long_context_attention_causal_gb300 as pa
    N, H, d = 40, 3, 64
    f, _ = pa.rope_inv_freq(d)
    for dtype in DT.values():
        x = torch.randn((N, H, d), device=dev()).to(dtype)
        pos = torch.arange(N, dtype=torch.int32, device=dev()) * 37
        buf = torch.zeros((N, H * d + 7), device=dev(), dtype=dtype)
        view = buf[:, :H * d].unflatten(1, (H, d))
        view.copy_(x)
        want, _ = pa.rope(x, None, pos, f)
        got, _ = pa.rope(view, None, pos, f)
        assert torch.equal(got, want)
        pa.rope(view, None, pos, f, q_out=view)
        assert torch.equal(view, want) and (buf[:, H * d:] == 0).all()


def test_gradient():
    """<g, rope(x + e) - rope(x - e)> = <inverse(g), 2 e>: rope is linear, so
    its difference quotient is its derivative; and against autograd of the
    formula in fp64."""
    import long_context_attention_causal_gb300 as pa
    f, s = pa.rope_inv_freq(32, factor=4.0, scaling="bands", context=4096)
    for interleaved in (False, True):
        q, k, pos = make(60, 4, 2, 64, "f32", 3)
        kw = dict(scale=s, interleaved=interleaved)
        gq, gk = torch.randn_like(q.contiguous()), torch.randn_like(k.contiguous())
        dq, dk = pa.rope(gq, gk, pos, f, inverse=True, **kw)
        for x, g, dx in ((q, gq, dq), (k, gk, dk)):
            e = torch.randn_like(g)
            up, _ = pa.rope((x + e), None, pos, f, **kw)
            dn, _ = pa.rope((x - e), None, pos, f, **kw)
            lhs = (g.double() * (up.double() - dn.double())).sum()
            rhs = 2 * (dx.double() * e.double()).sum()
            # each side sums x.numel() products with relative errors of 2^-20
            assert abs(float(lhs - rhs)) <= 2.0 ** -18 * float((g.double() * up.double()).abs().sum())
            leaf = x.double().clone().requires_grad_()
            rope_ref_torch(leaf, pos, f, s, interleaved).backward(g.double())
            assert ((dx.double() - leaf.grad).abs() <= 5 * 2.0 ** -22 * s * 2 * g.abs().max()).all()


def rope_ref_torch(x, pos, f, scale, interleaved):
    """The formula without writes in place, for autograd."""
    rot = 2 * f.shape[0]
    a = pos.double()[:, None, None] * f
    c, s = scale * a.cos(), scale * a.sin()
    if interleaved:
        p, q = x[..., :rot:2], x[..., 1:rot:2]
        turned = torch.stack([p * c - q * s, q * c + p * s], -1).flatten(-2)
    else:
        p, q = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([p * c - q * s, q * c + p * s], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def test_stream_capture_and_refusals():
    import long_context_attention_causal_gb300 as pa
    f, _ = pa.rope_inv_freq(64)
    q, k, pos = make(300, 4, 2, 64, "bf16", 8)
    q, k = q.contiguous(), k.contiguous()
    want = pa.rope(q, k, pos, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pa.rope(q, k, pos, f, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = torch.empty_like(q), torch.empty_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.rope(q, k, pos, f, q_out=out[0], k_out=out[1])
    pos.add_(17)
    graph.replay()
    torch.cuda.synchronize()
    check(out[0], q, pos, f)
    with pytest.raises(ValueError):
        pa.rope(q.transpose(0, 1), k, pos, f)
    with pytest.raises(ValueError):
        pa.rope(q, k[:10], pos, f)
    with pytest.raises(TypeError):
        pa.rope(q, k.float(), pos, f)
    with pytest.raises(TypeError):
        pa.rope(q, k, pos.long(), f)
    with pytest.raises(TypeError):
        pa.rope(q, k, pos, f.float())
    with pytest.raises(TypeError):
        pa.rope(q.half(), None, pos, f)
    with pytest.raises(pa.PolarError):
        pa.rope(q, k, pos, pa.rope_inv_freq(66)[0])
    with pytest.raises(pa.PolarError):
        pa.rope(q, k, pos, f, q_out=q[:, :, :], k_out=k, scale=math.nan)
    empty, _ = pa.rope(q[:0], None, pos[:0], f)
    assert empty.shape == (0, 4, 64)

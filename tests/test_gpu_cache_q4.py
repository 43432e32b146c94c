"""Rows into and out of the paged 4-bit cache.  Rounding is exact by
definition, so rows are compared for equality with fp64's."""
import math

import pytest
import torch

from gpu_util import dev
from serving_ref import q4_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def same(a, b):
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


def store(k, v, slots, page, num_pages, fill=0):
    import long_context_attention_causal_gb300 as pa
    kp, vp = pa.cache_q4(num_pages, k.shape[1], page, k.shape[2])
    kp.fill_(fill)
    vp.fill_(fill)
    pa.cache_append_q4(k, v, slots, kp, vp)
    return kp, vp


@pytest.mark.parametrize("N,Hkv,d,page", [(1, 1, 64, 8), (7, 3, 128, 8), (100, 2, 64, 16),
                                          (333, 4, 128, 64), (64, 8, 64, 1024), (2000, 5, 128, 256),
                                          (1031, 1, 64, 32)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_round_trip(N, Hkv, d, page, dtype):
    import long_context_attention_causal_gb300 as pa
    g = torch.Generator(device=dev()).manual_seed(N + d)
    kv = torch.randn((N, 2 * Hkv + 1, d), generator=g, device=dev())
    kv = (kv * torch.exp(2 * torch.randn((1, 2 * Hkv + 1, d), generator=g, device=dev()))).to(DT[dtype])
    k, v = kv[:, :Hkv], kv[:, Hkv:2 * Hkv]
    pool = -(-N // page) + 2
    slots = torch.randperm(pool * page, generator=g, device=dev())[:N].to(torch.int32)
    kp, vp = store(k, v, slots, page, pool)
    rk, rv = pa.cache_read_q4(kp, vp, slots, dtype=torch.float32)
    assert torch.equal(rk.double(), q4_ref(k)) and torch.equal(rv.double(), q4_ref(v))
    bk, bv = pa.cache_read_q4(kp, vp, slots)
    assert torch.equal(bk, rk.bfloat16()) and torch.equal(bv, rv.bfloat16())
    # the documented layout, byte by byte
    t, h = N // 2, Hkv - 1
    p, row = int(slots[t]) // page, int(slots[t]) % page
    raw = kp[p, h].flatten().cpu()
    codes = raw[:page * d // 2].view(page, d // 2)[row].tolist()
    scales = raw[page * d // 2:].clone().view(torch.bfloat16).view(page, d // 32)[row]
    for ch in range(d):
        w, j = ch // 8, ch % 4
        at = 4 * (w % 4 * (d // 32) + w // 4) + 2 * (ch // 4 % 2)
        bits = codes[at] | codes[at + 1] << 8
        n = (bits >> (4, 0, 12, 8)[j] & 7) * (-1 if bits >> (15, 11, 7, 3)[j] & 1 else 1)
        assert n * float(scales[ch // 32]) == float(rk[t, h, ch])
    # rows that no slot names keep their bytes
    kp2, _ = store(k[: N // 2], v[: N // 2], slots[: N // 2], page, pool, fill=0x5A)
    seen = torch.zeros(pool * page, dtype=torch.bool, device=dev())
    seen[slots[: N // 2].long()] = True
    codes = kp2.flatten(2)[..., :page * d // 2].reshape(pool, Hkv, page, -1).transpose(1, 2)
    scales = kp2.flatten(2)[..., page * d // 2:].reshape(pool, Hkv, page, -1).transpose(1, 2)
    for part in (codes, scales):
        assert (part.flatten(0, 1)[~seen] == 0x5A).all()


def test_ties_and_odd_values():
    """Ties go to even, groups of zeros, of one value, of subnormals, with
    infinities and NaN, the largest numbers."""
    import long_context_attention_causal_gb300 as pa
    rows = []
    s = 0.25
    ties = [7 * s] + [(i + 0.5) * s for i in range(-7, 7)] + [i * s for i in range(-7, 8)]
    rows.append(ties + [0.0] * (64 - len(ties)))
    near = []
    for i in range(-7, 7):
        x = torch.tensor((i + 0.5) * s)
        near += [float(torch.nextafter(x, torch.tensor(-9.0))), float(torch.nextafter(x, torch.tensor(9.0)))]
    rows.append([7 * s] + near + [0.0] * 3 + [0.0] * 32)
    rows.append([0.0] * 64)
    rows.append([-0.0] * 32 + [1e-45] * 32)
    rows.append([1e-39 * i for i in range(32)] + [1e-42 * (i - 16) for i in range(32)])
    rows.append([3.3e38 * (1 if i % 2 else -1) for i in range(32)] + [1e-30 * i for i in range(32)])
    rows.append([math.inf] + [1.0] * 31 + [1.0] * 32)
    rows.append([1.0] * 32 + [math.nan] + [-2.0] * 31)
    rows.append([-math.inf] * 64)
    rows.append([1.0] * 64)
    x = torch.tensor(rows, device=dev())[:, None, :]
    for dtype in DT.values():
        k = x.to(dtype)
        slots = torch.arange(len(rows), dtype=torch.int32, device=dev())
        kp, vp = store(k, k.flip(-1).contiguous(), slots, 8, 2)
        rk, rv = pa.cache_read_q4(kp, vp, slots, dtype=torch.float32)
        want = q4_ref(k).float().double()   # s n below fp32's range is rounded by the read
        assert same(rk.double(), want)
        assert same(rv.double(), q4_ref(k.flip(-1)).float().double())
        assert rk[2].abs().sum() == 0 and rk[6, 0, :32].isnan().all() and not rk[6, 0, 32:].isnan().any()
        fin = torch.isfinite(want)
        step = k.double().abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True) / 7
        err = (rk.double() - k.double()).unflatten(-1, (-1, 32)).abs()
        # s / 2, the scale's own rounding (2^-9) times 7, the subnormals' steps
        ok = err <= step * (0.5 + 7.5 * 2.0 ** -9) + 4e-40
        assert (ok | ~fin.unflatten(-1, (-1, 32))).all()


def test_border_of_every_code():
    """fp32 numbers around every border of many scales: a code is the nearest,
    whatever a product with the reciprocal would say."""
    import long_context_attention_causal_gb300 as pa
    g = torch.Generator(device=dev()).manual_seed(4)
    N = 4000
    s = torch.exp(20 * torch.rand((N, 1), generator=g, device=dev()) - 10).bfloat16().float()
    n = torch.randint(-7, 7, (N, 32), generator=g, device=dev()).float() + 0.5
    x = n * s                       # exact: 8 and 4 bits
    ulp = torch.randint(-2, 3, (N, 32), generator=g, device=dev())
    x = (x.view(torch.int32) + ulp.int()).view(torch.float32)
    x[:, 0] = 7 * s[:, 0]
    x = torch.cat([x, x.flip(1)], 1)[:, None, :].contiguous()
    slots = torch.arange(N, dtype=torch.int32, device=dev())
    kp, vp = store(x, x, slots, 16, N // 16)
    rk, rv = pa.cache_read_q4(kp, vp, slots, dtype=torch.float32)
    assert torch.equal(rk.double(), q4_ref(x)) and torch.equal(rv, rk)


def test_slots_without_rows():
    import long_context_attention_causal_gb300 as pa
    k = torch.randn((5, 2, 64), device=dev())
    slots = torch.tensor([3, -1, 31, -(1 << 31), 0], dtype=torch.int32, device=dev())
    kp, vp = store(k, k, slots, 16, 2)
    rk, _ = pa.cache_read_q4(kp, vp, slots, dtype=torch.float32)
    assert torch.equal(rk[[0, 2, 4]].double(), q4_ref(k)[[0, 2, 4]]) and rk[[1, 3]].abs().sum() == 0
    assert pa.device_status() == 0
    before = kp.clone()
    far = torch.tensor([32, (1 << 31) - 1], dtype=torch.int32, device=dev())
    pa.cache_append_q4(k[:2], k[:2], far, kp, vp)
    assert pa.device_status(reset=True) == 3 and torch.equal(kp, before)
    rk, _ = pa.cache_read_q4(kp, vp, far, dtype=torch.float32)
    assert rk.abs().sum() == 0 and pa.device_status(reset=True) == 3
    none = slots[:0]
    pa.cache_append_q4(k[:0], k[:0], none, kp, vp)
    a, b = pa.cache_read_q4(kp, vp, none)
    assert a.shape == (0, 2, 64) and torch.equal(kp, before)


def test_pool_past_2_31_bytes():
    """Rows whose bytes lie past 2^31 and 2^32 of a large pool."""
    import long_context_attention_causal_gb300 as pa
    page, Hkv, d = 64, 4, 128
    num = (1 << 33) // (Hkv * page * 9 * d // 16) + 5
    kp = torch.empty((num, Hkv, page, 9 * d // 16), dtype=torch.uint8, device=dev())
    vp = torch.empty_like(kp)
    ids = torch.tensor([0, num // 4 + 1, num // 2 + 1, num - 1], device=dev())
    slots = (ids[:, None] * page + torch.tensor([0, 33, page - 1], device=dev())).flatten().to(torch.int32)
    k = torch.randn((12, Hkv, d), device=dev()).bfloat16()
    v = torch.randn((12, Hkv, d), device=dev()).bfloat16()
    pa.cache_append_q4(k, v, slots, kp, vp)
    rk, rv = pa.cache_read_q4(kp, vp, slots, dtype=torch.float32)
    assert torch.equal(rk.double(), q4_ref(k)) and torch.equal(rv.double(), q4_ref(v))
    assert pa.device_status() == 0


def test_stream_capture_and_refusals():
    import long_context_attention_causal_gb300 as pa
    k = torch.randn((30, 2, 64), device=dev()).bfloat16()
    slots = torch.arange(30, dtype=torch.int32, device=dev())
    kp, vp = pa.cache_q4(4, 2, 8, 64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.cache_append_q4(k, k, slots, kp, vp)
    k.mul_(-3.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph.replay()
    rk, _ = pa.cache_read_q4(kp, vp, slots, dtype=torch.float32, stream=s)
    s.synchronize()
    assert torch.equal(rk.double(), q4_ref(k))
    with pytest.raises(ValueError):
        pa.cache_append_q4(k[:, :1], k, slots, kp, vp)
    with pytest.raises(ValueError):
        pa.cache_append_q4(k.transpose(0, 1), k, slots, kp, vp)
    with pytest.raises(TypeError):
        pa.cache_append_q4(k, k.float(), slots, kp, vp)
    with pytest.raises(TypeError):
        pa.cache_append_q4(k, k, slots.long(), kp, vp)
    with pytest.raises(TypeError):
        pa.cache_append_q4(k, k, slots, kp.int(), vp)
    with pytest.raises(ValueError):
        pa.cache_append_q4(k, k, slots, kp[..., :35].contiguous(), vp)
    with pytest.raises(pa.PolarError):
        pa.cache_append_q4(k, k, slots, kp, kp)
    with pytest.raises(TypeError):
        pa.cache_read_q4(kp, vp, slots, dtype=torch.float16)
    with pytest.raises(ValueError):
        pa.cache_q4(1, 1, 8, 40)

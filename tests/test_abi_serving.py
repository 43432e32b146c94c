"""Host-side checks of the entry points between requests and tokens (no GPU
needed, nothing launched): refusals with the documented status, workspace
sizes, the frequencies of the rotary positions."""
import ctypes
import math
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
# addresses that are never dereferenced: validation or the missing device comes first
A = [P((1 + i) << 32) for i in range(14)]
NULL = P(0)
BIG = 1 << 40


def odd(i, by):
    return P(((1 + i) << 32) + by)


@pytest.fixture(scope="module")
def L():
    from long_context_attention_causal_gb300 import _build
    _build.build()
    import long_context_attention_causal_gb300 as pa
    return pa.lib()


@pytest.fixture(scope="module")
def valid(L):
    """Statuses that a call with valid arguments may end with here: no device,
    which is the only thing that keeps these calls from launching."""
    if torch.cuda.is_available():
        pytest.skip("valid calls would launch on addresses that are not the device's")
    return 6


def test_every_declared_symbol_is_exported(L):
    text = open(os.path.join(ROOT, "include", "polar_attn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(polar_[a-z_0-9]+)\s*\(", text))
    assert {"polar_pages_extend", "polar_pages_release", "polar_rope", "polar_cache_append_q4",
            "polar_cache_read_q4", "polar_attn_decode_paged_q4", "polar_attn_fwd_packed"} <= names
    assert not [n for n in names if not hasattr(L, n)]


def extend(L, p=None, B=4, cols=8, page=16, pool=32, cap=32, tokens=10, ws=A[10], wsb=BIG):
    a = dict(enumerate(A))
    a.update(p or {})
    return L.polar_pages_extend(*[a[i] for i in range(10)], B, cols, page, pool, cap, tokens, ws, wsb,
                                NULL)


def test_pages_extend_refusals(L):
    assert extend(L, B=-1) == 1 and extend(L, cols=0) == 1 and extend(L, pool=0) == 1
    assert extend(L, cap=-1) == 1 and extend(L, tokens=-1) == 1
    assert extend(L, page=4) == 2 and extend(L, page=2048) == 2 and extend(L, page=24) == 2
    assert extend(L, pool=1 << 28) == 2 and extend(L, cols=1 << 28) == 2
    assert extend(L, B=1 << 20, cols=1 << 12) == 2
    for i in range(10):
        assert extend(L, {i: NULL}) == 1, i
        assert extend(L, {i: odd(i, 2)}) == 3, i
    assert extend(L, {8: NULL, 9: NULL}, B=0) == 0
    assert extend(L, ws=NULL) == 4 and extend(L, wsb=39) == 4 and extend(L, ws=odd(10, 8)) == 3
    # written arrays over others; lengths and count may be updated in place
    for i, j in ((0, 1), (0, 2), (0, 3), (5, 2), (7, 1), (8, 9), (9, 0), (6, 5), (3, 4), (8, 7)):
        assert extend(L, {i: A[j]}) == 1, (i, j)
    assert extend(L, ws=A[0]) == 1
    assert L.polar_pages_workspace_bytes(4) == 40 and L.polar_pages_workspace_bytes(-1) == 0


def test_pages_valid_calls_reach_the_device(L, valid):
    assert extend(L, {3: NULL}, cap=0) == valid
    assert extend(L) == valid and extend(L, {5: A[1], 6: A[4]}) == valid
    assert extend(L, {8: NULL, 9: NULL}, tokens=0) == valid
    assert release(L) == valid and release(L, {5: A[1], 6: A[4]}) == valid


def release(L, p=None, B=4, cols=8, page=16, pool=32, cap=32, ws=A[10], wsb=BIG):
    a = dict(enumerate(A))
    a.update(p or {})
    return L.polar_pages_release(*[a[i] for i in range(7)], B, cols, page, pool, cap, ws, wsb, NULL)


def test_pages_release_refusals(L):
    assert release(L, B=-1) == 1 and release(L, cols=0) == 1 and release(L, page=12) == 2
    for i in range(7):
        assert release(L, {i: NULL}) == 1, i
    assert release(L, {3: A[0]}) == 1 and release(L, {5: A[2]}) == 1 and release(L, {6: A[3]}) == 1
    assert release(L, ws=NULL) == 4 and release(L, wsb=8) == 4 and release(L, B=0) == 0


def rope(L, p=None, qs=256, ks=128, qos=256, kos=128, N=7, Hq=4, Hkv=2, d=64, rot=64, dtype=1,
         inter=0, inv=0, scale=1.0):
    a = dict(enumerate(A))
    a.update(p or {})
    return L.polar_rope(*[a[i] for i in range(6)], qs, ks, qos, kos, N, Hq, Hkv, d, rot, dtype,
                        inter, inv, scale, NULL)


def test_rope_refusals(L):
    assert rope(L, N=-1) == 1 and rope(L, Hq=-1) == 1 and rope(L, rot=0) == 1
    assert rope(L, rot=66) == 1 and rope(L, rot=31) == 1 and rope(L, scale=math.inf) == 1
    assert rope(L, d=96) == 2 and rope(L, dtype=2) == 2 and rope(L, Hq=5000) == 2
    for i in range(6):
        assert rope(L, {i: NULL}) == 1, i
    for i in (0, 1, 4, 5):
        assert rope(L, {i: odd(i, 8)}) == 3, i
    assert rope(L, {2: odd(2, 2)}) == 3 and rope(L, {3: odd(3, 4)}) == 3
    assert rope(L, qs=255) == 1 and rope(L, ks=100) == 1 and rope(L, qos=0) == 1
    assert rope(L, N=0) == 0
    # overlaps: the outputs with each other, over the other input, partly over their own
    assert rope(L, {4: A[5]}) == 1 and rope(L, {4: A[1]}) == 1 and rope(L, {5: A[0]}) == 1
    assert rope(L, {4: odd(0, 16)}) == 1 and rope(L, {4: A[0]}, qs=512) == 1
    assert rope(L, {4: A[2]}) == 1 and rope(L, {5: A[3]}) == 1


def test_rope_interleaved_windows(L, valid):
    """q and k of one projection, turned in place: their windows of a token
    interleave and do not meet; k's moved by a head into q's does."""
    base = 1 << 33
    q, k = P(base), P(base + 4 * 64 * 2)
    kw = dict(qs=512, ks=512, qos=512, kos=512)
    assert rope(L, {0: q, 4: q, 1: k, 5: k}, **kw) == valid
    assert rope(L, {0: q, 4: q, 1: P(base + 3 * 64 * 2), 5: P(base + 3 * 64 * 2)}, **kw) == 1
    # k's window wraps into the next token's q
    assert rope(L, {0: q, 4: q, 1: P(base + 7 * 64 * 2), 5: P(base + 7 * 64 * 2)}, **kw) == 1
    assert rope(L) == valid and rope(L, {1: NULL, 5: NULL}, Hkv=0) == valid
    assert rope(L, qs=257, qos=259) == valid  # odd strides take narrow accesses


def append(L, p=None, ks=128, vs=128, N=7, Hkv=2, d=64, page=16, pool=8, dtype=1):
    a = dict(enumerate(A))
    a.update(p or {})
    return L.polar_cache_append_q4(*[a[i] for i in range(5)], ks, vs, N, Hkv, d, page, pool, dtype,
                                   NULL)


def test_append_and_read_refusals(L):
    def read(p=None, N=7, Hkv=2, d=64, page=16, pool=8, dtype=1):
        a = dict(enumerate(A))
        a.update(p or {})
        return L.polar_cache_read_q4(*[a[i] for i in range(5)], N, Hkv, d, page, pool, dtype, NULL)
    for f in (lambda *x, **k: append(L, *x, **k), read):
        assert f(N=-1) == 1 and f(Hkv=0) == 1 and f(pool=0) == 1
        assert f(d=32) == 2 and f(dtype=3) == 2 and f(page=4) == 2 and f(page=2048) == 2
        assert f(pool=1 << 28) == 2 and f(Hkv=5000) == 2
        for i in range(5):
            assert f({i: NULL}) == 1, i
            assert f({i: odd(i, 2)}) == 3, i
        assert f({3: A[4]}) == 1 and f({3: A[0]}) == 1 and f({4: A[2]}) == 1
        assert f(N=0) == 0
    assert append(L, ks=127) == 1 and append(L, ks=132) == 3 and append(L, vs=100) == 1


def test_append_valid_calls_reach_the_device(L, valid):
    assert append(L) == valid and append(L, ks=132, dtype=0) == valid


def decode(L, p=None, B=2, Hq=4, Hkv=2, d=64, page=16, pool=8, cols=4, top=50, dtype=1, c=None,
           runs=0, ws=A[11], wsb=BIG):
    a = dict(enumerate(A))
    a.update(p or {})
    return L.polar_attn_decode_paged_q4(*[a[i] for i in range(10)], B, Hq, Hkv, d, page, pool, cols,
                                        top, dtype, c, runs, ws, wsb, NULL)


def test_decode_q4_refusals(L):
    import long_context_attention_causal_gb300 as pa
    assert decode(L, B=-1) == 1 and decode(L, runs=-1) == 1 and decode(L, pool=0) == 1
    assert decode(L, top=0) == 1 and decode(L, top=65) == 1 and decode(L, cols=0) == 1
    assert decode(L, Hq=6) == 2 and decode(L, Hq=3) == 2 and decode(L, Hq=32) == 2
    assert decode(L, d=96) == 2 and decode(L, dtype=2) == 2 and decode(L, page=4) == 2
    assert decode(L, page=48) == 2 and decode(L, pool=1 << 28) == 2 and decode(L, runs=(1 << 20) + 1) == 2
    assert decode(L, B=0) == 0
    bad = pa.Consts(math.log(2048.0), -1.0, 1.0, 1e-6, 1)
    assert decode(L, c=ctypes.byref(bad)) == 1
    for i in range(10):
        want = 1 if i != 9 else None      # conf may be missing
        if want:
            assert decode(L, {i: NULL}) == want, i
    for i in (0, 1, 2, 5, 6, 7):
        assert decode(L, {i: odd(i, 8)}) == 3, i
    for i in (3, 4, 8, 9):
        assert decode(L, {i: odd(i, 2)}) == 3, i


def test_decode_q4_workspace(L, valid):
    n = L.polar_attn_decode_paged_q4_workspace_bytes
    assert n(2, 4, 2, 50, 64, 1, 3) == (3 + 4) * 2 * 68 * 4 + 4 * 8
    assert n(2, 6, 2, 50, 64, 1, 0) == 0 and n(2, 4, 2, 0, 64, 1, 0) == 0
    assert n(2, 4, 2, 50, 64, 1, -1) == 0 and n(2, 4, 2, 50, 64, 2, 0) == 0
    runs = L.polar_attn_decode_paged_q4_num_runs
    for dtype in (0, 1):
        s = runs(2, 2, 5000, dtype)
        assert s >= 1 and n(2, 4, 2, 5000, 64, dtype, 0) == (s + 4) * 2 * 68 * 4 + 4 * 8
    assert runs(1, 2, 300, 1) == 6 and runs(0, 2, 300, 1) == 1   # a stage is 128 keys
    assert runs(2, 2, 0, 1) == 0 and runs(2, 2, 50, 5) == 0
    assert decode(L) == valid


def packed(L, p=None, qs=256, ks=128, vs=128, N=7, B=2, Hq=4, Hkv=2, d=64, dtype=1, c=None):
    a = dict(enumerate(A))
    a.update(p or {})
    return L.polar_attn_fwd_packed(*[a[i] for i in range(9)], qs, ks, vs, N, B, Hq, Hkv, d, dtype, c,
                                   NULL)


def test_packed_refusals(L):
    assert packed(L, N=-1) == 1 and packed(L, B=-1) == 1 and packed(L, Hq=0) == 1
    assert packed(L, Hkv=0) == 1 and packed(L, Hq=3) == 2 and packed(L, Hq=6) == 2
    assert packed(L, Hq=32) == 2 and packed(L, d=256) == 2 and packed(L, dtype=7) == 2
    for i in range(8):
        assert packed(L, {i: NULL}) == 1, i
    for i in (0, 1, 2, 3, 4, 6):
        assert packed(L, {i: odd(i, 8)}) == 3, i
    for i in (5, 7, 8):
        assert packed(L, {i: odd(i, 2)}) == 3, i
    assert packed(L, qs=255) == 1 and packed(L, ks=64) == 1 and packed(L, vs=0) == 1
    assert packed(L, qs=260) == 3 and packed(L, ks=129) == 3 and packed(L, qs=1 << 38) == 2
    assert packed(L, N=0) == 0 and packed(L, B=0) == 0 and packed(L, B=(1 << 18) + 1) == 2
    for i, j in ((6, 0), (6, 1), (6, 2), (6, 3), (6, 4), (6, 5), (7, 8), (7, 6), (8, 0)):
        assert packed(L, {i: A[j]}) == 1, (i, j)


def test_packed_valid_calls_reach_the_device(L, valid):
    assert packed(L) == valid and packed(L, {8: NULL}) == valid
    assert packed(L, qs=264, ks=136, vs=512) == valid
    # parts of one projection's output: the inputs interleave
    b = 1 << 33
    assert packed(L, {0: P(b), 1: P(b + 512), 2: P(b + 768)}, qs=512, ks=512, vs=512) == valid


def test_inv_freq():
    import long_context_attention_causal_gb300 as pa
    f, s = pa.rope_inv_freq(64, device="cpu")
    assert s == 1.0 and f.dtype == torch.float64 and f.shape == (32,)
    i = torch.arange(32, dtype=torch.float64)
    assert torch.allclose(f, 10000.0 ** (-i / 32), rtol=1e-14, atol=0)
    lin, _ = pa.rope_inv_freq(64, factor=4.0, scaling="linear", device="cpu")
    assert torch.allclose(lin, f / 4, rtol=1e-15, atol=0)
    base, _ = pa.rope_inv_freq(64, factor=4.0, scaling="base", device="cpu")
    assert base[0] == 1.0 and abs(float(base[-1] / f[-1]) - 0.25) < 1e-12
    mix, s = pa.rope_inv_freq(64, factor=4.0, scaling="bands", context=4096, device="cpu")
    assert abs(s - (0.1 * math.log(4.0) + 1.0)) < 1e-15
    turns = f * 4096 / (2 * math.pi)
    assert torch.equal(mix[turns > 32], f[turns > 32])
    assert torch.allclose(mix[turns < 1], f[turns < 1] / 4, rtol=1e-15, atol=0)
    assert ((mix <= f) & (mix >= f / 4)).all() and (mix[1:] < mix[:-1]).all()
    for kw in (dict(scaling="other"), dict(scaling="bands"), dict(factor=0.5),
               dict(scaling="bands", context=100, fast=1.0, slow=2.0), dict(base=1.0)):
        with pytest.raises(ValueError):
            pa.rope_inv_freq(64, device="cpu", **kw)
    for rot in (0, 7):
        with pytest.raises(ValueError):
            pa.rope_inv_freq(rot, device="cpu")
    with pytest.raises(ValueError):
        pa.rope_inv_freq(2, factor=2.0, scaling="base", device="cpu")

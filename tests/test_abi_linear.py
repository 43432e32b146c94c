"""Host-side checks of the linear attention and cache eviction entry points
(no GPU needed, nothing launched): refusals with the documented status, and
the workspace sizes."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

OK = ctypes.c_void_p(1 << 20)            # never dereferenced: validation fails first
OUT = [ctypes.c_void_p((2 + i) << 20) for i in range(3)]  # distinct outputs
ODD = ctypes.c_void_p((1 << 20) + 8)
ODD2 = ctypes.c_void_p((1 << 20) + 2)
NULL = ctypes.c_void_p(0)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from long_context_attention_causal_gb300 import _build
    _build.build()
    import long_context_attention_causal_gb300 as pa
    return pa.lib()


def test_every_declared_symbol_is_exported(L):
    text = open(os.path.join(ROOT, "include", "polar_attn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(polar_[a-z_0-9]+)\s*\(", text))
    assert {"polar_linear_fwd", "polar_linear_step", "polar_linear_bwd", "polar_cache_evict",
            "polar_attn_decode_paged_weights"} <= names
    assert not [n for n in names if not hasattr(L, n)]


def fwd(L, q=OK, ld=OK, lens=NULL, s_in=NULL, mem=OUT[0], s_out=NULL, B=1, H=2, T=64, d=64, dtype=1,
        scale=1.0, ws=OK, wsb=BIG):
    return L.polar_linear_fwd(q, OK, OK, ld, lens, s_in, mem, s_out, B, H, T, d, dtype, scale, ws,
                              wsb, NULL)


def test_linear_fwd_validation(L):
    assert fwd(L, B=-1) == 1 and fwd(L, T=-1) == 1
    assert fwd(L, scale=float("inf")) == 1 and fwd(L, scale=float("nan")) == 1
    assert fwd(L, d=96) == 2 and fwd(L, dtype=2) == 2
    assert fwd(L, B=1 << 15, H=1 << 15) == 2 and fwd(L, T=(1 << 28) + 1) == 2
    assert fwd(L, q=NULL) == 1 and fwd(L, ld=NULL) == 1 and fwd(L, mem=NULL) == 1
    assert fwd(L, q=ODD) == 3 and fwd(L, s_in=ODD) == 3 and fwd(L, s_out=ODD) == 3
    assert fwd(L, ld=ODD2) == 3 and fwd(L, lens=ODD2) == 3
    assert fwd(L, mem=OK) == 1                      # over an input
    assert fwd(L, B=1 << 10, H=1 << 10, T=1 << 28) == 2
    assert fwd(L, B=0, q=NULL) == 0 and fwd(L, T=0, q=NULL) == 0


def test_linear_bwd_validation(L):
    def bwd(dq=OUT[0], dk=OUT[1], dmem=OK, ds_out=NULL, ds=NULL, T=64, d=64, B=1):
        return L.polar_linear_bwd(OK, OK, OK, OK, NULL, NULL, dmem, ds_out, dq, dk, OUT[2], ds, B,
                                  2, T, d, 1, 1.0, OK, BIG, NULL)
    assert bwd(dq=OK) == 1 and bwd(dk=OUT[0]) == 1 and bwd(dk=OUT[2]) == 1
    assert bwd(d=80) == 2 and bwd(T=-2) == 1
    assert bwd(dq=NULL) == 1 and bwd(dmem=NULL) == 1
    assert bwd(dq=ODD) == 3 and bwd(ds_out=ODD) == 3 and bwd(ds=ODD) == 3
    assert bwd(B=0, dq=NULL) == 0 and bwd(T=0, dq=NULL) == 0


def test_linear_step_validation(L):
    def step(state=OK, q=OK, B=1, d=64, dtype=0, scale=1.0):
        return L.polar_linear_step(state, q, OK, OK, OK, OK, B, 2, d, dtype, scale, NULL)
    assert step(state=NULL) == 1 and step(q=ODD) == 3 and step(d=32) == 2
    assert step(dtype=5) == 2 and step(scale=float("nan")) == 1 and step(B=0, q=NULL) == 0


def test_linear_overlaps_are_refused(L):
    """Outputs that meet another tensor of the call, at their first or last
    bytes; a state may be updated in place.  Two heads of 4000 tokens are cut
    and need a workspace, which is not given: nothing can launch anywhere."""
    at = [1 << 24 | i << 22 for i in range(4)] + [1 << 26 | i << 22 for i in range(8)]
    n, ns = 2 * 4000 * 64 * 2, 2 * 64 * 64 * 4
    P = ctypes.c_void_p

    def fwd(q=at[0], k=at[1], v=at[2], s_in=at[3], mem=at[4], s_out=at[5]):
        return L.polar_linear_fwd(P(q), P(k), P(v), OK, NULL, P(s_in), P(mem), P(s_out), 1, 2,
                                  4000, 64, 1, 1.0, NULL, 0, NULL)
    free = fwd()
    assert free != 1                     # past validation: no device, or no workspace
    assert fwd(s_out=at[3]) == free and fwd(mem=at[0] + n) == free and fwd(mem=at[0] - n) == free
    for other in at[:3]:
        assert fwd(mem=other + n - 16) == 1 and fwd(mem=other - n + 16) == 1
        assert fwd(s_out=other + n - 16) == 1 and fwd(s_out=other - ns + 16) == 1
    assert fwd(mem=at[3] + ns - 16) == 1 and fwd(mem=at[5]) == 1
    assert fwd(s_out=at[3] + 16) == 1

    def step(state=at[0], q=at[1], k=at[2], v=at[3], mem=at[4]):
        return L.polar_linear_step(P(state), P(q), P(k), P(v), OK, P(mem), 1, 2, 64, 1, 1.0, NULL)
    one = 2 * 64 * 2
    for other in at[1:4]:
        assert step(mem=other) == 1 and step(mem=other + one - 16) == 1
    assert step(mem=at[0] + ns - 16) == 1 and step(q=at[0]) == 1

    def bwd(dq=at[4], dk=at[5], dv=at[6], s_in=at[7], ds_out=at[8], ds=at[9]):
        return L.polar_linear_bwd(P(at[0]), P(at[1]), P(at[2]), OK, NULL, P(s_in), P(at[3]),
                                  P(ds_out), P(dq), P(dk), P(dv), P(ds), 1, 2, 4000, 64, 1,
                                  1.0, NULL, 0, NULL)
    free = bwd()
    assert free != 1 and bwd(ds=at[8]) == free
    for other in at[:4] + at[7:10]:
        assert bwd(dq=other + 16) == 1 and bwd(dv=other - 16) == 1
    assert bwd(dk=at[4] + n - 16) == 1 and bwd(ds=at[7]) == 1 and bwd(ds=at[8] + 16) == 1
    assert bwd(ds=at[6]) == 1


def test_linear_workspace(L):
    ws = L.polar_linear_workspace_bytes
    assert ws(1, 1, 0, 64, 1) == 0 and ws(1, 1, 10, 96, 1) == 0 and ws(-1, 1, 10, 64, 1) == 0
    assert ws(1, 1, 128, 64, 1) == 0               # one tile: no head is cut
    assert ws(1 << 10, 152, 4096, 64, 1) == 0      # whole heads fill every SM
    one = 128 * 128 * 4
    for B, H, T in ((1, 16, 65536), (2, 16, 16384), (1, 1, 100000)):
        for dtype in (0, 1):
            n = ws(B, H, T, 128, dtype)
            assert n > 0 and n % one == 0
            assert n // one <= B * H * ((T + 127) // 128)
            assert L.polar_linear_bwd_workspace_bytes(B, H, T, 128, dtype) == 2 * n


def test_decode_paged_weights_validation(L):
    def dec(w=OK, stride=64, msl=64, Hq=4, page=16, pages=8, B=1, wsb=BIG, d=64):
        return L.polar_attn_decode_paged_weights(OK, OK, OK, OK, OK, OK, OK, OK, OK, NULL, w,
                                                 stride, B, Hq, 2, d, page, 8, pages, msl, 1, None,
                                                 0, OK, wsb, NULL)
    assert dec(w=NULL) == 1 and dec(stride=63) == 1 and dec(w=ODD2) == 3
    assert dec(Hq=6) == 2 and dec(page=12) == 2 and dec(pages=3) == 1 and dec(d=32) == 2
    assert dec(B=0, w=NULL) == 0
    size = L.polar_attn_decode_paged_weights_workspace_bytes
    assert size(2, 8, 2, 1000, 64, 4) == \
        L.polar_attn_decode_paged_workspace_bytes(2, 8, 2, 1000, 64, 4) + 2 * 8 * 1000 * 4
    assert size(2, 6, 2, 1000, 64, 4) == 0
    count = L.polar_attn_decode_paged_weights_num_splits
    own = L.polar_attn_decode_paged_num_splits
    assert size(2, 8, 2, 1000, 64, 0) == size(2, 8, 2, 1000, 64, count(2, 2, 1000, 64))
    for B, Hkv, T in ((1, 1, 1), (4, 4, 1500), (1, 1, 32768), (32, 4, 32768), (1, 2, 100)):
        s = count(B, Hkv, T, 64)
        assert s >= own(B, Hkv, T, 64)
        assert s == own(B, Hkv, T, 64) or (s <= 64 and s * 128 <= T and s * B * Hkv <= 2 * 160)
    assert count(1, 0, 5, 64) == 0


def test_cache_evict_validation(L):
    def ev(kp=OK, w=OK, pos=OK, new=OK, B=2, Hkv=2, d=64, page=16, pages=8, msl=64, stride=64,
           dtype=1, keep=32, recent=4, ws=OK, wsb=BIG):
        return L.polar_cache_evict(kp, OK, OK, OK, w, pos, new, B, Hkv, d, page, 8, pages, msl,
                                   stride, dtype, keep, recent, ws, wsb, NULL)
    assert ev(keep=0) == 1 and ev(recent=-1) == 1 and ev(recent=33) == 1 and ev(stride=63) == 1
    assert ev(msl=0) == 1 and ev(pages=3) == 1 and ev(B=-1) == 1
    assert ev(d=32) == 2 and ev(dtype=9) == 2 and ev(page=24) == 2 and ev(B=40000) == 2
    assert ev(kp=NULL) == 1 and ev(w=NULL) == 1 and ev(pos=NULL) == 1 and ev(new=NULL) == 1
    assert ev(kp=ODD) == 3 and ev(w=ODD2) == 3 and ev(new=ODD2) == 3 and ev(ws=ODD) == 3
    assert ev(wsb=16) == 4 and ev(ws=NULL) == 4
    assert ev(B=0, kp=NULL) == 0
    size = L.polar_cache_evict_workspace_bytes
    assert size(2, 3, 100, 100) == 2 * 3 * 8           # nothing can move
    assert size(2, 3, 100, 70) == 2 * 3 * (30 * 8 + 8)
    assert size(2, 3, 100, 20) == 2 * 3 * (20 * 8 + 8)
    assert size(2, 3, 100, 0) == 0

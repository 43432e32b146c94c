"""Outputs of the linear attention that meet the decay, the lengths or the
workspace of the call are refused, at their first and last bytes and when one
holds the other (host-side: nothing is launched, no pointer is read).

Two heads of 4000 tokens are cut at any number of SMs from 2 up, so these
calls need a workspace; the tests that place one also make it too small, and
nothing can launch anywhere."""
import ctypes

import pytest

MB = 1 << 20
AT = [64 * MB + i * 4 * MB for i in range(12)]
H, T, D = 2, 4000, 64
N, NS = H * T * D * 2, H * D * D * 4      # bytes of a bf16 row tensor and of the states
SMALL = 1 * MB                            # log_decay and lengths, far from the rest
WS = 32 * MB
P = ctypes.c_void_p
INVALID, WORKSPACE, DEVICE = 1, 4, 6


@pytest.fixture(scope="module")
def L():
    from long_context_attention_causal_gb300 import _build
    _build.build()
    import long_context_attention_causal_gb300 as pa
    return pa.lib()


def fwd(L, ld=SMALL, lens=SMALL + 64, ws=0, wsb=0, mem=AT[4], s_out=AT[5], s_in=AT[3], q=AT[0],
        t=T):
    return L.polar_linear_fwd(P(q), P(AT[1]), P(AT[2]), P(ld), P(lens), P(s_in), P(mem), P(s_out),
                              1, H, t, D, 1, 1.0, P(ws), wsb, None)


def bwd(L, ld=SMALL, lens=SMALL + 64, ws=0, wsb=0, dq=AT[4], ds=AT[9], t=T):
    return L.polar_linear_bwd(P(AT[0]), P(AT[1]), P(AT[2]), P(ld), P(lens), P(AT[7]), P(AT[3]),
                              P(AT[8]), P(dq), P(AT[5]), P(AT[6]), P(ds), 1, H, t, D, 1, 1.0,
                              P(ws), wsb, None)


def step(L, ld=SMALL, state=AT[0], mem=AT[4]):
    return L.polar_linear_step(P(state), P(AT[1]), P(AT[2]), P(AT[3]), P(ld), P(mem), 1, H, D, 1,
                               1.0, None)


def test_decay_under_an_output(L):
    assert fwd(L) in (WORKSPACE, DEVICE) and bwd(L) in (WORKSPACE, DEVICE)
    for out, size in ((AT[4], N), (AT[5], NS)):
        for at in (out, out + 64, out + size - 4, out - 4 * H + 4):
            assert fwd(L, ld=at) == INVALID
        assert fwd(L, ld=out + size) != INVALID and fwd(L, ld=out - 4 * H) != INVALID
    for out, size in ((AT[4], N), (AT[5], N), (AT[6], N), (AT[9], NS)):
        for at in (out, out + size - 4, out - 4 * H + 4):
            assert bwd(L, ld=at) == INVALID
        assert bwd(L, ld=out + size) != INVALID
    one = H * D * 2
    for out, size in ((AT[0], NS), (AT[4], one)):
        for at in (out, out + size - 4, out - 4 * H + 4):
            assert step(L, ld=at) == INVALID


def test_lengths_under_an_output(L):
    for out, size in ((AT[4], N), (AT[5], NS)):
        for at in (out, out + size - 4):
            assert fwd(L, lens=at) == INVALID
        assert fwd(L, lens=out + size) != INVALID and fwd(L, lens=out - 4) != INVALID
    for out, size in ((AT[4], N), (AT[5], N), (AT[6], N), (AT[9], NS)):
        for at in (out, out + size - 4):
            assert bwd(L, lens=at) == INVALID
        assert bwd(L, lens=out - 4) != INVALID


@pytest.mark.parametrize("call,rows,states,small", [
    (fwd, (0, 1, 2, 4), (3, 5), ("ld", "lens")),
    (bwd, (0, 1, 2, 3, 4, 5, 6), (7, 8, 9), ("ld", "lens"))])
def test_workspace_over_a_tensor(L, call, rows, states, small):
    """The workspace is written: it may meet no tensor of the call."""
    size = (L.polar_linear_workspace_bytes if call is fwd else L.polar_linear_bwd_workspace_bytes)
    need = size(1, H, T, D, 1)
    assert 0 < need < 4 * MB
    short = need - 16                     # too small: refused even where it meets nothing
    assert call(L, ws=WS, wsb=short) in (WORKSPACE, DEVICE)
    for i, n in [(i, N) for i in rows] + [(i, NS) for i in states]:
        for at in (AT[i], AT[i] + n - 16, AT[i] - short + 16):
            assert call(L, ws=at, wsb=short) == INVALID, (i, at)
        assert call(L, ws=AT[i] - short, wsb=short) in (WORKSPACE, DEVICE)
    for name in small:
        assert call(L, ws=WS, wsb=short, **{name: WS + short - 4}) == INVALID
        assert call(L, ws=WS, wsb=short, **{name: WS + short}) in (WORKSPACE, DEVICE)

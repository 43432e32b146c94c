"""Calls repeated many times give the same bits every time.

The state's warps of the bf16 kernel read a tile's y into registers and let
the next tile be loaded over it.  Where the CTAs hold several short heads that
start from given states, those warps reach a tile late and one by one, while
the loads of the states and the zeros of rows past the sequences keep the SM's
memory pipeline busy: a read of y that is still under way is then overwritten
by the next head's rows.  Values are compared with the token-by-token
recurrence in fp64 too, with the bound of test_gpu_linear.py.
"""
import pytest
import torch

from gpu_util import dev
from linear_ref import linear_bwd_ref, linear_fwd_ref

pytestmark = pytest.mark.gpu

CALLS = 400


@pytest.mark.parametrize("B,H,T,d,lens", [
    (2, 90, 666, 64, (137, 137)), (2, 90, 666, 64, (0, 137)), (2, 90, 666, 128, (137, 140)),
    (1, 304, 300, 64, (200,)), (4, 100, 200, 64, None)])
@pytest.mark.parametrize("want", [False, True])
def test_repeated_calls(B, H, T, d, lens, want):
    import long_context_attention_causal_gb300 as pa
    gen = torch.Generator(device=dev()).manual_seed(T + d)
    r = lambda *s: torch.randn(s, generator=gen, device=dev())  # noqa: E731
    q, k, v, g = (r(B, H, T, d).bfloat16() for _ in range(4))
    S, R = r(B, H, d, d), r(B, H, d, d)
    ld = -torch.exp2(-torch.rand(H, generator=gen, device=dev()) * 8 - 2)
    lengths = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev())
    scale = d ** -0.5
    outs = [torch.empty_like(q) for _ in range(4)]
    states = [torch.empty_like(S) if want else None for _ in range(2)]

    def call():
        pa.linear_fwd(q, k, v, ld, state=S, lengths=lengths, mem=outs[0], state_out=states[0])
        pa.linear_bwd(q, k, v, ld, g, state=S, dstate_out=R, lengths=lengths, dq=outs[1],
                      dk=outs[2], dv=outs[3], dstate=states[1])

    call()
    ref = [linear_fwd_ref(q, k, v, ld, scale, S, lens)[0],
           *linear_bwd_ref(q, k, v, ld, scale, g, S, R, lens)[:3]]
    for a, b in zip(outs, ref):
        # every head by itself: one wrong tile does not hide in the others
        err = (a.double() - b).flatten(2).norm(dim=2) / b.flatten(2).norm(dim=2).clamp(min=1e-30)
        assert float(err.max()) <= 4.6e-3
    first = [o.clone() for o in (*outs, *states) if o is not None]
    wrong = torch.zeros(len(first), dtype=torch.int64, device=dev())
    for _ in range(CALLS):
        call()
        now = [o for o in (*outs, *states) if o is not None]
        wrong += torch.stack([(a != b).any() for a, b in zip(now, first)])
    assert wrong.tolist() == [0] * len(first)
    assert pa.device_status() == 0

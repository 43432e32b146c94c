"""How the fp32 state of fp32 prompts rounds over many tokens.

Positive inputs and no decay: the state grows to T products of one sign, so
what is rounded at the state's size counts most.  u = 2^-24; a rounding has an
rms of at most u / sqrt 3 of the rounded value.  64 tokens are summed on their
own: 64 roundings of partial sums, sqrt(64 / 3) units of a chunk's sum, and
C = T / 64 chunks average that to sqrt(64 / (3 C)) of the state.  Each chunk is
joined to the state with one rounding, at c / C of its final size: sqrt(C / 3).
Cutting a head into runs joins no more often.  Twice the sum of both, in the
2-norm, holds for a state rounded once a chunk (8 u at T = 8192); one rounded
once a token has sqrt(T / 3) units, 30 u there.
"""
import math

import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu


# whole heads; heads cut into long runs; whole heads, d = 128; two heads in many runs
@pytest.mark.parametrize("H,T,d", [(304, 8192, 64), (100, 8192, 64), (76, 8192, 128),
                                   (2, 16384, 128)])
def test_fp32_state_rounds_once_a_chunk(H, T, d):
    import long_context_attention_causal_gb300 as pa
    gen = torch.Generator(device=dev()).manual_seed(90 + d)
    q, k, v, g = (torch.randn((1, H, T, d), generator=gen, device=dev()).abs_() for _ in range(4))
    zero = torch.zeros(H, device=dev())
    state = pa.linear_fwd(q, k, v, zero, want_state=True)[1]
    dstate = pa.linear_bwd(q, k, v, zero, g, scale=1.0, want_dstate=True)[3]
    chunks = T / 64
    tol = 2 * (math.sqrt(chunks / 3) + math.sqrt(64 / (3 * chunks))) * 2.0 ** -24 / math.sqrt(3)
    worst = [0.0, 0.0]
    for h in range(0, H, max(1, H // 16)):
        for i, (got, z, y) in enumerate(((state, v, k), (dstate, g, q))):
            ref = z[0, h].double().T @ y[0, h].double()
            worst[i] = max(worst[i], float((got[0, h].double() - ref).norm() / ref.norm()))
    assert max(worst) <= tol, (worst, tol)

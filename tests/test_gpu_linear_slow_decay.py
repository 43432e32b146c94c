"""States that live through many slow decays, fp32 prompts and single tokens.

The decay of a chunk or a token is a number near 1.  Rounded to fp32 it is up
to u / 2 off (u = 2^-24), each time by the same factor, so a state that lives
through N decays would be off by up to N u / 2.  The library applies it in two
parts.  Bounds in units u, 2-norm, positive inputs (nothing cancels):
a prompt of C chunks: rounding of the state once a chunk and of the chunk's
own sum, twice their rms as in test_gpu_linear_rounding.py; powers inside a
chunk, exp2f (2) and its exponent (1), the same in every chunk; x = log_decay
n and e^x - 1 are right to 3 |x| together, and the state lives through 1 / |x|
chunks: 3.  Single tokens: one rounding a token at the state's size, twice
sqrt(T / 3) / sqrt 3, and 3.
"""
import math

import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def exact(z, y, log_decay, first):
    """sum_t g^(T - 1 - t) z_t y_t^T, or from the first token's side g^(t + 1)."""
    T = z.shape[0]
    n = torch.arange(T, device=z.device, dtype=torch.float64)
    w = torch.exp(float(log_decay) * (n + 1 if first else T - 1 - n))
    return (z.double() * w[:, None]).T @ y.double()


def decays(H):
    """From exp(-2^-9) to exp(-2^-14) a token, odd numbers among them."""
    return -torch.exp2(-torch.linspace(9, 14, H, device=dev()))


@pytest.mark.parametrize("H,T,d", [(152, 16384, 64), (76, 8192, 128), (3, 65536, 64)])
def test_prompt(H, T, d):
    import long_context_attention_causal_gb300 as pa
    gen = torch.Generator(device=dev()).manual_seed(140 + d)
    q, k, v, g = (torch.randn((1, H, T, d), generator=gen, device=dev()).abs_() for _ in range(4))
    ld = decays(H)
    state = pa.linear_fwd(q, k, v, ld, want_state=True)[1]
    dstate = pa.linear_bwd(q, k, v, ld, g, scale=1.0, want_dstate=True)[3]
    chunks = T / 64
    tol = (2 * (math.sqrt(chunks / 3) + math.sqrt(64 / (3 * chunks))) / math.sqrt(3) + 6) * U
    worst = [0.0, 0.0]
    for h in sorted({*range(0, H, max(1, H // 24)), H - 1}):
        for i, (got, z, y) in enumerate(((state, v, k), (dstate, g, q))):
            ref = exact(z[0, h], y[0, h], ld[h], first=i == 1)
            worst[i] = max(worst[i], float((got[0, h].double() - ref).norm() / ref.norm()))
    assert max(worst) <= tol, (worst, tol)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_single_tokens(dtype):
    import long_context_attention_causal_gb300 as pa
    H, T, d = 12, 4096, 64
    gen = torch.Generator(device=dev()).manual_seed(150)
    q, k, v = (torch.randn((T, 1, H, d), generator=gen, device=dev()).abs_().to(dtype)
               for _ in range(3))
    ld = decays(H)
    S = torch.zeros((1, H, d, d), device=dev())
    mem = torch.empty_like(q[0])
    for t in range(T):
        pa.linear_step(S, q[t], k[t], v[t], ld, mem=mem)
    tol = (2 * math.sqrt(T / 3) / math.sqrt(3) + 3) * U
    worst = 0.0
    for h in range(H):
        ref = exact(v[:, 0, h], k[:, 0, h], ld[h], first=False)
        worst = max(worst, float((S[0, h].double() - ref).norm() / ref.norm()))
    assert worst <= tol, (worst, tol)


@pytest.mark.parametrize("signs", ["positive", "both"])
@pytest.mark.parametrize("H,T,d", [(152, 16384, 64), (76, 8192, 128), (3, 65536, 128),
                                   (300, 700, 64)])
def test_prompt_of_bf16(H, T, d, signs):
    """bf16 inputs are exact, but weighted by a power of the decay they are
    not: they enter as three bf16 terms, 2^-25 of them and less is left out
    (two terms would leave up to 2^-17, 2^-18.7 rms: 40 u).  The tensor core
    cuts off what it adds, less than 2 u of the sum so far, in the eight steps
    of a tile's largest term: 9 u.  A state is joined once a tile, C = T / 128
    times: twice sqrt(C / 3) / sqrt 3.  Powers of the decay, by the bounds
    above: exp2f 2, exponents 2, the state's decay 3."""
    import long_context_attention_causal_gb300 as pa
    gen = torch.Generator(device=dev()).manual_seed(160 + d + T)
    q, k, v, g = (torch.randn((1, H, T, d), generator=gen, device=dev()).bfloat16()
                  for _ in range(4))
    if signs == "positive":
        q, k, v, g = (t.abs() for t in (q, k, v, g))
    ld = decays(H)
    state = pa.linear_fwd(q, k, v, ld, want_state=True)[1]
    dstate = pa.linear_bwd(q, k, v, ld, g, scale=1.0, want_dstate=True)[3]
    tol = (2 * math.sqrt(T / 128 / 3) / math.sqrt(3) + 9 + 7) * U
    worst = [0.0, 0.0]
    for h in sorted({*range(0, H, max(1, H // 24)), H - 1}):
        for i, (got, z, y) in enumerate(((state, v, k), (dstate, g, q))):
            ref = exact(z[0, h], y[0, h], ld[h], first=i == 1)
            worst[i] = max(worst[i], float((got[0, h].double() - ref).norm() / ref.norm()))
    assert max(worst) <= tol, (worst, tol)

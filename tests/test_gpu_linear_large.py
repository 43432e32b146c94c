"""Linear attention and eviction on tensors of more than 2^31 elements, and
from several host threads at once."""
import threading

import pytest
import torch

from gpu_util import dev
from linear_ref import evict_ref

pytestmark = pytest.mark.gpu


def test_forward_and_backward_past_2_31_elements():
    """Heads on both sides of the boundary against the same heads alone, which
    the small tests hold to the recurrence.  Both sides round bf16 results
    from fp32 sums that are cut at different tiles: 4.6e-3 each in the 2-norm
    (see test_gpu_linear.py)."""
    import long_context_attention_causal_gb300 as pa
    H, T, d = 132, 131072, 128
    ld = -torch.exp2(-torch.linspace(3, 12, H, device=dev()))
    x = {}
    for i, n in enumerate(("q", "k", "v", "g")):
        x[n] = torch.empty((1, H, T, d), device=dev(), dtype=torch.bfloat16)
        for h in range(H):
            gen = torch.Generator(device=dev()).manual_seed(1000 * i + h)
            x[n][0, h] = torch.randn((T, d), generator=gen, device=dev())
    assert x["q"].numel() > 2 ** 31
    mem, S = pa.linear_fwd(x["q"], x["k"], x["v"], ld, want_state=True)
    grads = pa.linear_bwd(x["q"], x["k"], x["v"], ld, x["g"], want_dstate=True)
    torch.cuda.synchronize()
    for h in (0, 127, 128, 131):
        one = {n: t[:, h:h + 1].contiguous() for n, t in x.items()}
        want = pa.linear_fwd(one["q"], one["k"], one["v"], ld[h:h + 1], want_state=True)
        gwant = pa.linear_bwd(one["q"], one["k"], one["v"], ld[h:h + 1], one["g"],
                              want_dstate=True)
        for a, b in zip((mem, *grads[:3]), (want[0], *gwant[:3])):
            a, b = a[:, h:h + 1].float(), b.float()
            assert float((a - b).norm() / b.norm()) <= 2 * 4.6e-3, h
        for a, b in zip((S, grads[3]), (want[1], gwant[3])):
            a = a[:, h:h + 1]
            assert float((a - b).norm() / b.norm()) <= 1e-4, h
    assert pa.device_status() == 0


def test_evict_in_a_pool_past_2_31_elements():
    import long_context_attention_causal_gb300 as pa
    pages, Hkv, page, d, T, keep = 70000, 4, 64, 128, 640, 200
    kp = torch.empty((pages, Hkv, page, d), device=dev(), dtype=torch.bfloat16)
    vp = torch.empty_like(kp)
    assert kp.numel() > 2 ** 31
    cols = T // page
    table = torch.stack([torch.arange(pages - 1, pages - 1 - cols, -1),
                         torch.arange(0, 7 * cols, 7)]).to(torch.int32)
    gen = torch.Generator().manual_seed(2)
    rows = torch.randn((2, cols, Hkv, page, d), generator=gen).bfloat16()
    for b in range(2):
        kp[table[b].long().to(dev())] = rows[b].to(dev())
        vp[table[b].long().to(dev())] = -rows[b].to(dev())
    w = torch.rand((2, Hkv, T), generator=gen)
    pos = torch.arange(T, dtype=torch.int32).repeat(2, Hkv, 1)
    lens = torch.full((2,), T, dtype=torch.int32)
    moves = evict_ref(lens, w.numpy(), pos.numpy(), keep, 10)
    pa.cache_evict(kp, vp, table.to(dev()), lens.to(dev()), w.to(dev()), pos.to(dev()), keep,
                   recent=10)
    want = rows.clone()
    for (b, h), lst in moves.items():
        for src, dst in lst:
            want[b, dst // page, h, dst % page] = rows[b, src // page, h, src % page]
    for b in range(2):
        at = table[b].long().to(dev())
        assert torch.equal(kp[at].cpu(), want[b]) and torch.equal(vp[at].cpu(), -want[b])


def test_four_host_threads():
    """Each thread on its own stream; every result equals the serial one."""
    import long_context_attention_causal_gb300 as pa
    gen = torch.Generator(device=dev()).manual_seed(4)
    r = lambda *s: torch.randn(s, generator=gen, device=dev())  # noqa: E731
    work = []
    for T, d, dt in ((1500, 128, torch.bfloat16), (700, 64, torch.bfloat16),
                     (300, 64, torch.float32), (2000, 128, torch.bfloat16)):
        q, k, v, g = (r(1, 3, T, d).to(dt) for _ in range(4))
        work.append((q, k, v, torch.tensor([-0.2, -0.01, -0.001], device=dev()), g))

    def calls(q, k, v, ld, g):
        mem, S = pa.linear_fwd(q, k, v, ld, want_state=True)
        grads = pa.linear_bwd(q, k, v, ld, g, state=S, want_dstate=True)
        tok = [t[:, :, 0].contiguous() for t in (q, k, v)]
        return (mem, S.clone(), *grads, pa.linear_step(S, *tok, ld))

    want = [calls(*w) for w in work]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def run(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(3):
                    got[i] = calls(*work[i])
            s.synchronize()
        except Exception as e:  # reported by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    assert pa.device_status() == 0

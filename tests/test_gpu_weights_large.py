"""The weighted decode with more than 2^31 logits: sequences past the boundary
get the bits of the same sequences decoded alone with as many splits."""
import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu


def test_logits_past_2_31_elements():
    import long_context_attention_causal_gb300 as pa
    B, Hq, Hkv, d, page, most = 136, 16, 2, 64, 1024, 1 << 20
    assert B * Hq * most > 2 ** 31
    gen = torch.Generator(device=dev()).manual_seed(12)
    r = lambda *s: torch.randn(s, generator=gen, device=dev()).bfloat16()  # noqa: E731
    cols = most // page
    k, v = r(cols, Hkv, page, d), r(cols, Hkv, page, d)
    q, mem = r(B, Hq, d), r(B, Hq, d)
    w_count = torch.randn((Hq, d), generator=gen, device=dev())
    table = torch.arange(cols, dtype=torch.int32, device=dev()).repeat(B, 1)  # all share the pages
    lens = torch.full((B,), 90, dtype=torch.int32, device=dev())
    lens[0], lens[127], lens[128], lens[B - 1] = 2000, 70001, most - 1, most
    w = torch.zeros((B, Hkv, most), device=dev())
    out, n_eff, conf = pa.decode_paged_weights(q, k, v, table, lens, mem, w_count, w,
                                               num_splits=16, want_conf=True)
    for b in (0, 5, 127, 128, B - 1):
        one = torch.zeros((1, Hkv, most), device=dev())
        got = pa.decode_paged_weights(q[b:b + 1], k, v, table[:1], lens[b:b + 1], mem[b:b + 1],
                                      w_count, one, num_splits=16, want_conf=True)
        for a, t in zip((out, n_eff, conf, w), (*got, one)):
            assert torch.equal(a[b:b + 1], t), b
        assert (one[..., int(lens[b]):] == 0).all()
        torch.testing.assert_close(one.double().sum(-1),
                                   torch.full((1, Hkv), Hq / Hkv, device=dev(),
                                              dtype=torch.float64), rtol=2e-5, atol=0)
    assert pa.device_status() == 0

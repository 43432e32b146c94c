"""Packed prefill with so many heads that the offsets inside one tile, and of
one head in a token, pass 2^31 elements (held to the bars of test_gpu_packed)."""
import pytest
import torch

from gpu_util import TOL, dev
from serving_ref import packed_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def randn(*shape, dtype=torch.float32):
    """Normal numbers, made in pieces of the leading dimension's rows."""
    x = torch.empty(shape, dtype=dtype, device=dev())
    flat = x.view(-1)
    for o in range(0, flat.numel(), 1 << 29):
        flat[o:o + (1 << 29)].normal_()
    return x


def outputs(N, Hq, d, dtype):
    return (torch.full((N, Hq, d), 77.0, dtype=dtype, device=dev()),
            torch.full((N, Hq), 77.0, device=dev()), torch.full((N, Hq), 77.0, device=dev()))


# (both widths of the bf16 kernel's CTAs: one long sequence, two short ones)
@pytest.mark.parametrize("lens,d,H", [([128], 128, 135000), ([100, 28], 64, 345000)])
def test_rows_of_a_tile_past_2_31(lens, d, H):
    import long_context_attention_causal_gb300 as pa
    N = sum(lens)
    assert (lens[0] - 1) * H * d > 1 << 31
    q, k, v, mem = (randn(N, H, d, dtype=torch.bfloat16) for _ in range(4))
    mem.mul_(0.1)
    w = randn(H, d).mul_(0.02)
    cu = torch.tensor([0, lens[0], N][:len(lens) + 1], dtype=torch.int32, device=dev())
    out, n_eff, conf = outputs(N, H, d, torch.bfloat16)
    pa.fwd_packed(q, k, v, mem, w, cu, out=out, n_eff=n_eff, conf=conf)
    assert pa.device_status() == 0
    some = [0, 1, H // 2, (1 << 31) // ((lens[0] - 1) * d), H - 2, H - 1]
    part = [t[:, some] for t in (q, k, v, mem)] + [w[some]]
    for b in range(len(lens)):
        s = slice(int(cu[b]), int(cu[b + 1]))
        o, ne, c = packed_ref(*part, cu, b)
        assert (out[s, some].double() - o).abs().max() <= TOL["bf16"]["out"]
        assert (n_eff[s, some].double() / ne - 1).abs().max() <= TOL["f32"]["neff"]
        assert (conf[s, some].double() - c).abs().max() <= TOL["f32"]["conf"]
    assert bool((n_eff != 77.0).all()) and bool((out[..., d - 1] != 77.0).all())


@pytest.mark.parametrize("dtype,G,Hkv", [("f32", 1, (1 << 24) + 5), ("f32", 8, (1 << 21) + 1),
                                         ("bf16", 1, (1 << 24) + 5)])
def test_heads_of_a_token_past_2_31(dtype, G, Hkv):
    """One token: u = v / |v|, a count of one key gates nothing."""
    import long_context_attention_causal_gb300 as pa
    torch.cuda.empty_cache()
    d, Hq = 128, G * Hkv
    assert Hq * d > 1 << 31
    q, mem = randn(1, Hq, d, dtype=DT[dtype]), randn(1, Hq, d, dtype=DT[dtype])
    k, v = randn(1, Hkv, d, dtype=DT[dtype]), randn(1, Hkv, d, dtype=DT[dtype])
    mem.mul_(0.1)
    w = randn(Hq, d)
    cu = torch.tensor([0, 1], dtype=torch.int32, device=dev())
    out, n_eff, conf = outputs(1, Hq, d, DT[dtype])
    pa.fwd_packed(q, k, v, mem, w, cu, out=out, n_eff=n_eff, conf=conf)
    assert pa.device_status() == 0
    for hs in (range(0, 40), range(Hq // 2, Hq // 2 + 40), range(Hq - 40, Hq)):
        hs = list(hs)
        kv = [h // G for h in hs]
        qq, kk, vv = q[0, hs].double(), k[0, kv].double(), v[0, kv].double()
        o = vv / vv.norm(dim=-1, keepdim=True) + mem[0, hs].double()
        c = torch.sigmoid((qq * kk).sum(-1) / d ** 0.5)
        assert (out[0, hs].double() - o).abs().max() <= TOL[dtype]["out"]
        assert (n_eff[0, hs] - 1).abs().max() <= TOL["f32"]["neff"]
        assert (conf[0, hs].double() - c).abs().max() <= TOL["f32"]["conf"]
    assert bool((n_eff != 77.0).all()) and bool((out[..., d - 1] != 77.0).all())
    del q, k, v, mem, w, out
    torch.cuda.empty_cache()

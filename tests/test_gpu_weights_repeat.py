"""The weighted decode repeated many times on one cache: the same bits every
time, however the stores of logits and the copies of the next pages meet."""
import pytest
import torch

from gpu_util import dev
from test_gpu_cache import paged, weights_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,Hq,Hkv,T,d,page,dtype", [
    (8, 16, 4, 4096, 128, 64, "f32"), (4, 32, 4, 5000, 64, 16, "f32"), (4, 8, 8, 3000, 128, 8, "f32"),
    (8, 16, 4, 8192, 128, 64, "bf16")])
def test_repeated_calls(B, Hq, Hkv, T, d, page, dtype):
    import long_context_attention_causal_gb300 as pa
    x = paged(B, Hq, Hkv, T, d, page, dtype, 33 + d)
    g = {k: t.to(dev()) for k, t in x.items()}
    args = [g[k] for k in ("q", "k_pages", "v_pages", "block_table", "seq_lens", "mem", "w_count")]
    w = torch.zeros((B, Hkv, T), device=dev())
    out, n_eff, conf = pa.decode_paged_weights(*args, w, want_conf=True, max_seq_len=T)
    ref = weights_ref(x, 0)
    assert ((w[0, :, :ref.shape[1]].double().cpu() - ref).abs() <= 2e-5 * ref + 1e-12).all()
    first = [t.clone() for t in (out, n_eff, conf, w)]
    wrong = torch.zeros(4, dtype=torch.int64, device=dev())
    for _ in range(200):
        w.zero_()
        pa.decode_paged_weights(*args, w, out=out, n_eff=n_eff, conf=conf, max_seq_len=T)
        wrong += torch.stack([(a != b).any() for a, b in zip((out, n_eff, conf, w), first)])
    assert wrong.tolist() == [0] * 4
    assert pa.device_status() == 0

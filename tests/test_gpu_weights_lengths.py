"""Lengths past max_seq_len in the weighted decode, among them lengths that
the last split's whole pages would still cover: each is cut to max_seq_len
and recorded, and the weights are those of a call with the cut length, bit
for bit.  Their sum is then one per query head: every row counted in the
softmax is a row that gets its weight."""
import pytest
import torch

from gpu_util import dev
from test_gpu_cache import paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,most,page,splits,over", [
    (200, 190, 16, 0, (191, 200)),      # 191 and 192: inside the last page
    (200, 190, 16, 3, (192, 193)),
    (300, 257, 256, 0, (258, 300)),
    (2048, 2000, 256, 1, (2040, 2001)),
    (2048, 2000, 256, 5, (2048, 2000)),
    (64, 1, 8, 0, (2, 64)),
])
def test_lengths_past_the_limit(T, most, page, splits, over, dtype):
    import long_context_attention_causal_gb300 as pa
    x = paged(2, 4, 2, T, 64, page, dtype, 500 + T + splits, ragged=False)
    g = {k: t.to(dev()) for k, t in x.items()}
    names = ("q", "k_pages", "v_pages", "block_table", "seq_lens", "mem", "w_count")

    def run(lengths):
        g["seq_lens"] = torch.tensor(lengths, dtype=torch.int32, device=dev())
        w = torch.zeros((2, 2, T), device=dev())
        pa.decode_paged_weights(*(g[n] for n in names), w, max_seq_len=most, num_splits=splits)
        return w, pa.device_status(reset=True)

    pa.device_status(reset=True)
    want, clean = run((most, most))
    assert clean == 0
    got, status = run(over)
    assert status == 3
    assert (got[:, :, most:] == 0).all()
    # two query heads a KV head; a weight is within 2e-5 of its value
    torch.testing.assert_close(got.sum(-1), torch.full((2, 2), 2.0, device=dev()), rtol=2e-5,
                               atol=0)
    assert torch.equal(got, want)

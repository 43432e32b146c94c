"""Packed prefill, bf16: outputs row by row in their 2-norm, and offsets at the
ends of their type.

A row: the result's rounding is at most 2^-8 of each channel, the probabilities'
at most 2^-8 of each key's share, for values that are nearly orthogonal 2^-8 of the
norm: 2^-7 together.  Both are uniform in half a step, whose rms is 2^-8 / sqrt(3)
of the number at most: over all rows sqrt(2/3) 2^-8, 3.2e-3.  (One wrong row of V
among n of equal weights moves a row by sqrt(2 / n).)
"""
import pytest
import torch

from gpu_util import dev
from serving_ref import packed_ref
from test_gpu_packed import case, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1, 1, 1], [127, 128, 129], [255, 256, 257], [31, 32, 33, 15, 16, 64],
                                  [700, 3, 1025], [3000, 90], [50] * 40])
def test_rows_in_norm(lens, d, G):
    import long_context_attention_causal_gb300 as pa
    args = case(lens, 2 * G, 2, d, "bf16", 80 + sum(lens) + d + G, lead=3, tail=5)
    args[3].zero_()
    got = run(args)
    far, at = [], args[5].tolist()
    for b in range(len(lens)):
        o, _, _ = packed_ref(*args, b)
        far.append(((got[0][at[b]:at[b + 1]].double() - o).norm(dim=-1) / o.norm(dim=-1)).flatten())
    far = torch.cat(far)
    assert far.max() <= 2.0 ** -7 and far.square().mean().sqrt() <= 3.2e-3
    assert pa.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cu", [[0, 50, 110, (1 << 31) - 1], [-(1 << 31), 50, 110, 150],
                                [0, 50, 110, 150, (1 << 31) - 1, -(1 << 31)]])
def test_offsets_of_any_size(cu, dtype):
    """Cut to the tokens there are, and recorded."""
    import long_context_attention_causal_gb300 as pa
    args = case([50, 60, 40], 4, 2, 64, dtype, 91)
    want = run(args)
    got = run(args[:5] + [torch.tensor(cu, dtype=torch.int32, device=dev())])
    assert pa.device_status(reset=True) == 3
    assert all(torch.equal(a, b) for a, b in zip(got, want))

"""Page calls of many sequences without tokens, and of stacks whose heights pass
2^31 with what is given back."""
import pytest
import torch

from gpu_util import dev
from serving_ref import release_ref
from test_gpu_pages import pool_state, run_extend, t32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [1, 2048, 2049, 5000])
@pytest.mark.parametrize("late", [False, True])
def test_no_tokens(B, late):
    """max_tokens 0: the table, lengths and stack stay; `late`: sequences that
    ask for tokens all the same are past max_tokens, which is recorded."""
    import long_context_attention_causal_gb300 as pa
    lens = [(7 * b) % 40 for b in range(B)]
    table, free, pool = pool_state(B, 6, 8, lens, 9, B)
    new = [0] * B
    if late:
        new[B // 2] = 3
    want = run_extend(table, lens, new, free, 9, 8, 0, pool)
    assert want[1] == lens and want[2] == 9 and want[3] == [0] * (B + 1)
    assert pa.device_status(reset=True) == (3 if late else 0)
    # and what is asked of the stream afterwards runs as ever
    run_extend(table, lens, [1] * B, free, 9, 8, B, pool)
    assert pa.device_status(reset=True) == 0


def test_stack_past_2_31():
    """Stack height plus entries given back above 2^31: what does not fit the
    stack is dropped and recorded, what does is in its place."""
    import long_context_attention_causal_gb300 as pa
    page, cols, B = 8, (1 << 28) - 1, 4
    room, top = 2048, (1 << 30) + 2048
    assert top + B * cols > 1 << 31
    table = torch.arange(B * cols, dtype=torch.int32, device=dev()).remainder_((1 << 28) - 7)
    table = table.view(B, cols)
    stack = torch.full((top + room,), -9, dtype=torch.int32, device=dev())
    lens, keep, count = t32([cols * page] * B), t32([0] * B), t32([top])
    pa.pages_release(table, lens, keep, stack, count, page, num_pages=(1 << 28) - 7)
    assert pa.device_status(reset=True) == 3
    assert lens.tolist() == [0] * B and count.tolist() == [top + room]
    assert torch.equal(stack[top:], table[0, :room])
    assert bool((stack[:top] == -9).all())
    del stack
    torch.cuda.empty_cache()


def test_release_to_a_full_stack():
    """The same at a small size, against the bookkeeping in Python."""
    import long_context_attention_causal_gb300 as pa
    lens = [40, 17, 64, 8]
    table, free, pool = pool_state(4, 8, 8, lens, 5, 1)
    T, L, F, C = t32(table, (4, -1)), t32(lens), t32(free + [-1] * 3), t32([5])
    want = release_ref(table, lens, [0, 8, 1, 0], free + [-1] * 3, 5, 8, pool)
    pa.pages_release(T, L, t32([0, 8, 1, 0]), F, C, 8, num_pages=pool)
    assert F.tolist() == want[0] and L.tolist() == want[1] and C.tolist() == [want[2]]
    assert pa.device_status(reset=True) == 3

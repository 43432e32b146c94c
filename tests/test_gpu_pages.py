"""Pages handed out and taken back on the device, against the bookkeeping in
Python: integers, compared for equality."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from serving_ref import extend_ref, release_ref

pytestmark = pytest.mark.gpu

I32 = torch.int32


def t32(x, shape=None):
    t = torch.tensor(x, dtype=I32, device=dev())
    return t if shape is None else t.reshape(shape)


def pool_state(B, cols, page, lens, spare, seed):
    """A table with the pages of `lens` and a stack of `spare` others."""
    rng = np.random.default_rng(seed)
    have = [-(-n // page) for n in lens]
    ids = rng.permutation(sum(have) + spare).tolist()
    table = [[-1] * cols for _ in range(B)]
    at = 0
    for b, n in enumerate(have):
        table[b][:n] = ids[at:at + n]
        at += n
    return table, ids[at:], max(sum(have) + spare, 1)  # a pool has a page at least


def run_extend(table, lens, new, free, count, page, tokens, num_pages, **kw):
    import long_context_attention_causal_gb300 as pa
    B = len(lens)
    T = t32(table, (B, -1))
    L, C, F = t32(lens), t32([count]), t32(free)
    got = pa.pages_extend(T, L, t32(new), F, C, page, tokens, num_pages=num_pages, **kw)
    want = extend_ref(table, lens, new, free, count, page, tokens, num_pages)
    assert T.tolist() == want[0]
    assert L.tolist() == want[1] and C.tolist() == [want[2]]
    assert [x.tolist() for x in got] == [want[3], want[4], want[5]]
    assert F.tolist() == free
    return want


@pytest.mark.parametrize("B,page,top,new,seed", [
    (1, 8, 0, 1, 0), (1, 8, 100, 300, 1), (3, 16, 50, 1, 2), (37, 8, 100, 20, 3), (256, 64, 2000, 1, 4),
    (1023, 8, 60, 9, 5), (1024, 16, 60, 3, 6), (1025, 8, 30, 5, 7), (2500, 32, 200, 2, 8),
    (40, 1024, 5000, 3000, 9), (96, 16, 500, 700, 10), (5000, 8, 20, 4, 11)])
@pytest.mark.parametrize("share", [1.0, 0.4, 0.0])
def test_extend(B, page, top, new, seed, share):
    """share: the part of the needed pages that the stack holds."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, top + 1, B).tolist()
    add = rng.integers(0, new + 1, B).tolist()
    need = sum(-(-(n + a) // page) - -(-n // page) for n, a in zip(lens, add))
    cols = -(-(top + new) // page)
    table, free, pool = pool_state(B, cols, page, lens, int(need * share) + (3 if share == 1 else 0),
                                   seed)
    free = free + [77777] * 2               # room above the top
    w = run_extend(table, lens, add, free, len(free) - 2, page, sum(add) + 3, pool)
    if share == 1.0:
        assert w[1] == [n + a for n, a in zip(lens, add)]
    else:
        stuck = [n != m for n, m in zip([n + a for n, a in zip(lens, add)], w[1])]
        assert any(stuck) or need == 0


def test_extend_edges():
    """Lengths at page borders, no new tokens, an empty call, few slots, bounds
    that are met exactly."""
    import long_context_attention_causal_gb300 as pa
    page = 8
    lens = [0, 7, 8, 9, 15, 16, 0, 24]
    new = [8, 1, 1, 0, 2, 0, 0, 0]
    table, free, pool = pool_state(8, 3, page, lens, 3, 1)
    run_extend(table, lens, new, free, 3, page, sum(new), pool)
    assert pa.device_status() == 0
    # one slot fewer: the last sequence with tokens gets none
    table, free, pool = pool_state(8, 3, page, lens, 3, 2)
    w = run_extend(table, lens, new, free, 3, page, sum(new) - 1, pool)
    assert w[1][4] == 15 and w[3][-1] == sum(new) - 1
    assert pa.device_status(reset=True) == 3
    none = torch.empty((0, 4), dtype=I32, device=dev())
    z = torch.empty((0,), dtype=I32, device=dev())
    cu, pos, slots = pa.pages_extend(none, z, z, t32([1, 2]), t32([2]), 8, 0)
    assert cu.tolist() == [0] and pos.numel() == 0 and slots.numel() == 0
    assert pa.device_status() == 0


def test_extend_bad_inputs():
    """Such sequences are left as they are, and recorded; the others are served."""
    import long_context_attention_causal_gb300 as pa
    page, cols = 8, 4
    for lens, new in (([5, -1, 6], [3, 2, 4]), ([5, 33, 6], [3, 0, 4]), ([5, 30, 6], [3, 3, 4]),
                      ([5, 9, 6], [3, -4, 4])):
        good = [min(max(n, 0), 32) for n in lens]
        table, free, pool = pool_state(3, cols, page, good, 4, 5)
        w = run_extend(table, lens, new, free, 4, page, 20, pool)
        assert w[1][0] == 8 and w[1][1] == lens[1] and w[1][2] == 10
        assert pa.device_status(reset=True) == 3
    # a count past the stack, and below it
    table, free, pool = pool_state(3, cols, page, [5, 9, 6], 4, 6)
    run_extend(table, [5, 9, 6], [9, 9, 9], free, 9, page, 30, pool)
    assert pa.device_status(reset=True) == 3
    run_extend(table, [5, 9, 6], [9, 9, 9], free, -2, page, 30, pool)
    assert pa.device_status(reset=True) == 3
    # numbers outside the pool, in the table and on the stack
    table, free, pool = pool_state(3, cols, page, [5, 9, 6], 4, 7)
    table[0][0], free[3] = pool, -5
    w = run_extend(table, [5, 9, 6], [2, 9, 9], free, 4, page, 30, pool)
    assert -1 in w[5][:2] and pa.device_status(reset=True) == 3


@pytest.mark.parametrize("B,page,top,seed", [(1, 8, 9, 0), (33, 16, 300, 1), (1030, 8, 40, 2),
                                             (300, 8, 3000, 3), (64, 1024, 9000, 4)])
def test_release(B, page, top, seed):
    import long_context_attention_causal_gb300 as pa
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, top + 1, B)
    keep = np.where(rng.random(B) < 0.4, 0, (lens * rng.random(B)).astype(int)).tolist()
    lens = lens.tolist()
    cols = -(-top // page)
    table, free, pool = pool_state(B, cols, page, lens, 5, seed)
    back = sum(-(-n // page) - -(-k // page) for n, k in zip(lens, keep))
    for room in (back + 2, back, max(back - 3, 0)):
        F, L, C = t32(free + [-9] * room), t32(lens), t32([5])
        T = t32(table, (B, -1))
        want = release_ref(table, lens, keep, free + [-9] * room, 5, page, pool)
        out, n = torch.empty_like(L), torch.empty_like(C)
        pa.pages_release(T, L, t32(keep), F, C, page, num_pages=pool, lens_out=out, count_out=n)
        assert F.tolist() == want[0] and out.tolist() == want[1] and n.tolist() == [want[2]]
        assert L.tolist() == lens and C.tolist() == [5] and T.tolist() == table
        assert pa.device_status(reset=True) == (3 if room < back else 0)


def test_release_bad_inputs():
    import long_context_attention_causal_gb300 as pa
    table, free, pool = pool_state(4, 4, 8, [20, 9, 30, 8], 2, 3)
    table[2][1] = pool + 4
    for lens, keep in (([20, 9, 30, 8], [5, 10, 0, 0]), ([20, -9, 30, 8], [5, 0, 0, 0]),
                       ([20, 40, 30, 8], [5, 0, 8, 0]), ([20, 9, 30, 8], [5, -1, 30, 8])):
        stack = free + [-9] * 12
        F, L, C = t32(stack), t32(lens), t32([2])
        want = release_ref(table, lens, keep, stack, 2, 8, pool)
        pa.pages_release(t32(table, (4, -1)), L, t32(keep), F, C, 8, num_pages=pool)
        assert F.tolist() == want[0] and L.tolist() == want[1] and C.tolist() == [want[2]]
        assert pa.device_status(reset=True) == 3


@pytest.mark.parametrize("B,steps,tokens", [(9, 60, 9), (500, 12, 5000)])
def test_captured_loop(B, steps, tokens):
    """Replays of one captured step (release, then extend) go on from one
    another, on a stream of their own."""
    import long_context_attention_causal_gb300 as pa
    rng = np.random.default_rng(1)
    page, cols = 8, 40
    lens = rng.integers(1, 100, B).tolist()
    table, free, pool = pool_state(B, cols, page, lens, 10 * B, 4)
    free = free + [-1] * (pool - len(free))
    T, L, F, C = t32(table, (B, -1)), t32(lens), t32(free), t32([10 * B])
    keep, new = t32(lens), t32([1] * B)
    bufs = [torch.empty((n,), dtype=I32, device=dev()) for n in (B + 1, tokens, tokens)]
    ws = torch.empty((8 * B + 8,), dtype=torch.uint8, device=dev())

    def step():
        pa.pages_release(T, L, keep, F, C, page, workspace=ws, num_pages=pool)
        pa.pages_extend(T, L, new, F, C, page, tokens, num_pages=pool, cu_seqlens=bufs[0],
                        positions=bufs[1], slots=bufs[2], workspace=ws)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    count = 10 * B
    for i in range(steps):
        k = [0 if rng.random() < 0.05 else n for n in lens]
        a = rng.integers(0, 3, B).tolist() if B < 100 else [1] * B
        while sum(a) > tokens:
            a[a.index(max(a))] -= 1
        keep.copy_(t32(k))
        new.copy_(t32(a))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        free, lens, count = release_ref(table, lens, k, free, count, page, pool)
        table, lens, count, cu, pos, slots = extend_ref(table, lens, a, free, count, page, tokens,
                                                        pool)
        assert T.tolist() == table and L.tolist() == lens and C.tolist() == [count]
        assert F.tolist() == free
        assert [x.tolist() for x in bufs] == [cu, pos, slots]
        rows = [s for s in slots if s >= 0]
        assert len(set(rows)) == len(rows)
    assert pa.device_status() == 0


def test_binding_refusals():
    import long_context_attention_causal_gb300 as pa
    T, L, F, C = t32([[0, 1]]), t32([3]), t32([2, 3]), t32([2])
    n = t32([1])
    with pytest.raises(TypeError):
        pa.pages_extend(T.cpu(), L, n, F, C, 8, 4)
    with pytest.raises(TypeError):
        pa.pages_extend(T, L.long(), n, F, C, 8, 4)
    with pytest.raises(ValueError):
        pa.pages_extend(T, L, t32([1, 1]), F, C, 8, 4)
    with pytest.raises(ValueError):
        pa.pages_extend(T, L, n, F, C, 8, -1)
    with pytest.raises(ValueError):
        pa.pages_extend(T, L, n, F, C, 8, 4, slots=t32([0] * 5))
    with pytest.raises(pa.PolarError):
        pa.pages_extend(T, L, n, F, C, 12, 4)
    with pytest.raises(pa.PolarError):
        pa.pages_extend(T, L, n, F, C, 8, 4, workspace=torch.empty(8, device=dev(), dtype=torch.uint8))
    with pytest.raises(pa.PolarError):
        pa.pages_release(T, L, n, F, C, 8, lens_out=n)
    pa.pages_release(T, L, L, F, C, 8)   # keeps all rows
    with pytest.raises(TypeError):
        pa.pages_release(T, L, None, F, C, 8)
    assert T.tolist() == [[0, 1]] and L.tolist() == [3] and C.tolist() == [2]


def test_no_sequences_and_no_stack():
    """Without sequences every token is one without a row; a stack of no pages
    serves tokens that need none."""
    import long_context_attention_causal_gb300 as pa
    none = torch.empty((0, 4), dtype=I32, device=dev())
    z = torch.empty((0,), dtype=I32, device=dev())
    count, left = t32([2]), t32([9])
    cu, pos, slots = pa.pages_extend(none, z, z, t32([1, 2]), count, 8, 3, count_out=left)
    assert cu.tolist() == [0] and pos.tolist() == [0] * 3 and slots.tolist() == [-1] * 3
    assert left.tolist() == [2]
    left = t32([9])
    pa.pages_release(none, z, z, t32([1, 2]), count, 8, count_out=left)
    assert left.tolist() == [2]
    lens = t32([5, 8])
    cu, pos, slots = pa.pages_extend(t32([[3, 7], [1, 7]]), lens, t32([2, 1]), z, t32([0]), 8, 4,
                                     num_pages=8)
    assert lens.tolist() == [7, 8] and slots.tolist() == [29, 30, -1, -1]
    assert cu.tolist() == [0, 2, 3] and pa.device_status() == 0

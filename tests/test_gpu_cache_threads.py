"""Eviction and the weighted decode from several host threads at once, each
on its own stream with a cache of another size: every call succeeds and every
result has the bits of the same calls made one after another.

An eviction whose lengths are already cut leaves everything as it is, so a
thread repeats the call in place on one cache: the host side of the calls is
what overlaps, with selections that ask for 1.2 to 160 KB of shared memory.
Half of that is made of bare calls of the C entry point, whose host side is
short enough for the threads to meet inside it.
"""
import threading
from ctypes import c_int, c_size_t, c_void_p

import pytest
import torch

from gpu_util import dev
from test_gpu_cache import evict_case, paged

pytestmark = pytest.mark.gpu

CALLS = 300
EVICT = [(300, 64, 16, 100), (40000, 64, 64, 900), (2112, 128, 64, 2048), (20000, 64, 256, 5000)]
DECODE = [(2, 8, 2, 300, 64, 16, "bf16"), (1, 4, 4, 700, 64, 64, "f32"),
          (2, 4, 1, 1500, 128, 64, "bf16"), (1, 8, 4, 90, 128, 8, "f32")]


def make(i):
    T, d, page, keep = EVICT[i]
    x = {n: t.to(dev()) for n, t in evict_case(2, 2, T, d, page, "bf16", 60 + i).items()}
    y = {n: t.to(dev()) for n, t in paged(*DECODE[i], 70 + i).items()}
    B, _, Hkv, S = DECODE[i][:4]
    return x, y, torch.zeros((B, Hkv, S), device=dev()), T, keep, S


def calls(x, y, w, T, keep, S):
    import long_context_attention_causal_gb300 as pa
    args = [y[n] for n in ("q", "k_pages", "v_pages", "block_table", "seq_lens", "mem", "w_count")]
    for n in range(CALLS):
        pa.cache_evict(x["k"], x["v"], x["table"], x["lens"], x["w"], x["pos"], keep, recent=9,
                       max_seq_len=T, new_lens=x["lens"])
        if n % 10 == 0:
            out = pa.decode_paged_weights(*args, w, max_seq_len=S, want_conf=True)
    return [x[n] for n in ("k", "v", "lens", "w", "pos")] + [w, *out]


def bare_call(x, T, keep, stream):
    """The eviction of `calls` as a C call with its arguments converted once."""
    import long_context_attention_causal_gb300 as pa
    pages, Hkv, page, d = x["k"].shape
    B, cols = x["table"].shape
    need = pa.cache_evict_workspace_bytes(B, Hkv, T, keep)
    x["ws"] = torch.empty(need, dtype=torch.uint8, device=dev())
    ptrs = [c_void_p(x[n].data_ptr()) for n in ("k", "v", "table", "lens", "w", "pos", "lens")]
    ints = [c_int(i) for i in (B, Hkv, d, page, pages, cols, T, x["w"].shape[2], 1, keep, 9)]
    args = (*ptrs, *ints, c_void_p(x["ws"].data_ptr()), c_size_t(need),
            c_void_p(stream.cuda_stream))
    f = pa.lib().polar_cache_evict
    return lambda: f(*args)


def in_threads(n, f):
    errors, gate = [], threading.Barrier(n)

    def run(i):
        try:
            torch.cuda.set_device(dev())
            gate.wait()
            f(i)
        except Exception as e:  # reported by the assertion below
            errors.append((i, e))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_bare_calls_with_caches_of_different_sizes():
    import long_context_attention_causal_gb300 as pa
    n = len(EVICT)
    want = [calls(*make(i)) for i in range(n)]
    work = [make(i) for i in range(n)]
    streams = [torch.cuda.Stream() for _ in range(n)]
    todo = [bare_call(w[0], w[3], w[4], s) for w, s in zip(work, streams)]
    torch.cuda.synchronize()
    failed = [0] * n

    def run(i):
        for _ in range(4000):
            failed[i] += todo[i]() != 0

    in_threads(n, run)
    torch.cuda.synchronize()
    assert failed == [0] * n, (failed, pa.lib().polar_attn_last_error())
    for a, (x, *_) in zip(want, work):
        for p, r in zip(a, (x[m] for m in ("k", "v", "lens", "w", "pos"))):
            assert torch.equal(p, r)
    assert pa.device_status() == 0


def test_threads_with_caches_of_different_sizes():
    import long_context_attention_causal_gb300 as pa
    want = [calls(*make(i)) for i in range(len(EVICT))]
    work = [make(i) for i in range(len(EVICT))]
    torch.cuda.synchronize()
    got = [None] * len(work)

    def run(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got[i] = calls(*work[i])
        stream.synchronize()

    in_threads(len(work), run)
    for a, b in zip(want, got):
        for p, r in zip(a, b):
            assert torch.equal(p, r)
    assert pa.device_status() == 0

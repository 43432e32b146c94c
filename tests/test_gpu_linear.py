"""Decayed linear attention on the GPU: prompt, single token and gradients
against the token-by-token recurrence in fp64.

Bounds.  u = 2^-24.  A result is a sum of products; `mag` is the same sum
over absolute values (the reference run on |q|, |k|, |v|, |S|).  fp32: the
dot products round at most d times, the chunk sums 128 times, the state once
a chunk, and a power of the decay is off by at most 200 u relative (its
exponent up to 126, two roundings, ln 2 each): 2 (d + 128) + 3 T / 64 + 400
units u of mag.  bf16 tensors: the scores, the state as an operand and the
values that enter the state inside a segment are each rounded to bf16 (half
a step, 2^-8), and the result once more: 3 2^-8 mag + 2^-8 |ref|.  Roundings
are independent, so in the 2-norm four of rms 2^-8 / sqrt 3: 4.6e-3.  States
are fp32 for both types; bf16 inputs enter them as two bf16 terms, 2^-16.
"""
import pytest
import torch

from gpu_util import dev
from linear_ref import linear_bwd_ref, linear_fwd_ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def decay(H, lo=3.0, hi=9.0):
    return -torch.exp2(-torch.linspace(lo, hi, H)) if H > 1 else torch.tensor([-0.02])


def make(B, H, T, d, dtype, seed, state=False):
    g = torch.Generator(device=dev()).manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    r = lambda *s: torch.randn(s, generator=g, device=dev())  # noqa: E731
    x = {n: r(B, H, T, d).to(dt) for n in ("q", "k", "v", "dmem")}
    x["state"] = r(B, H, d, d) if state else None
    x["dstate"] = r(B, H, d, d) if state else None
    x["log_decay"] = decay(H).to(dev())
    return x


def units(T, d):
    return (2 * (d + 128) + 3 * T / 64 + 400) * U


def check(got, ref, mag, dtype, T, d, what, is_state=False):
    got = got.double()
    err = (got - ref).abs()
    if is_state:
        tol = (units(T, d) + (2.0 ** -16 if dtype == "bf16" else 0.0)) * mag
    elif dtype == "f32":
        tol = units(T, d) * mag
    else:
        tol = 3 * 2.0 ** -8 * mag + 2.0 ** -8 * ref.abs()
    bad = ~(err <= tol + 1e-30)
    assert not bad.any(), (what, int(bad.sum()), float(err.max()), float((err / (tol + 1e-30)).max()))
    if dtype == "bf16" and not is_state and ref.norm() > 0:
        assert float((got - ref).norm() / ref.norm()) <= 4.6e-3, what


def absolute(x, names):
    return [x[n].abs() if x[n] is not None else None for n in names]


CASES = [  # B, H, T, d, lengths, state
    (1, 1, 1, 64, None, False), (2, 3, 1, 128, None, True), (1, 2, 2, 128, None, True),
    (2, 2, 63, 64, None, True), (1, 3, 64, 128, None, False), (1, 2, 65, 64, None, True),
    (2, 1, 127, 128, None, True), (1, 2, 128, 64, None, False), (1, 2, 129, 128, None, True),
    (1, 2, 256, 64, None, True), (1, 4, 300, 128, None, True), (3, 2, 385, 64, None, False),
    (1, 1, 1000, 128, None, True), (1, 2, 2100, 64, None, True),
    (4, 2, 300, 128, (300, 0, 1, 257), True), (5, 1, 640, 64, (639, 128, 129, 0, 640), False),
    (3, 3, 200, 128, (0, 0, 0), True), (2, 160, 130, 64, None, True),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:4])))
def test_forward(case, dtype):
    import long_context_attention_causal_gb300 as pa
    B, H, T, d, lens, state = case
    x = make(B, H, T, d, dtype, 31 * T + d, state)
    lengths = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev())
    if lens is not None:  # padding may hold anything
        for b, n in enumerate(lens):
            for name in ("q", "k", "v"):
                x[name][b, :, n:] = float("nan")
    scale = 0.37
    mem, S = pa.linear_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"],
                           lengths=lengths, scale=scale, want_state=True)
    ref, S_ref = linear_fwd_ref(x["q"], x["k"], x["v"], x["log_decay"], scale, x["state"], lens)
    mag, S_mag = linear_fwd_ref(*absolute(x, ("q", "k", "v")), x["log_decay"], scale,
                                *absolute(x, ("state",)), lens)
    check(mem, ref, mag, dtype, T, d, "mem")
    check(S, S_ref, S_mag, dtype, T, d, "state", is_state=True)
    # without the state the outputs are right too
    mem2, none = pa.linear_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"],
                               lengths=lengths, scale=scale)
    assert none is None
    check(mem2, ref, mag, dtype, T, d, "mem alone")
    assert pa.device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:4])))
def test_backward(case, dtype):
    import long_context_attention_causal_gb300 as pa
    B, H, T, d, lens, state = case
    x = make(B, H, T, d, dtype, 37 * T + d, state)
    lengths = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev())
    if lens is not None:
        for b, n in enumerate(lens):
            for name in ("q", "k", "v", "dmem"):
                x[name][b, :, n:] = float("nan")
    scale = 0.37
    got = pa.linear_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["dmem"], state=x["state"],
                        dstate_out=x["dstate"], lengths=lengths, scale=scale, want_dstate=True)
    ref = linear_bwd_ref(x["q"], x["k"], x["v"], x["log_decay"], scale, x["dmem"], x["state"],
                         x["dstate"], lens)
    mag = linear_bwd_ref(*absolute(x, ("q", "k", "v")), x["log_decay"], scale,
                         *absolute(x, ("dmem", "state", "dstate")), lens)
    for name, a, r, m in zip(("dq", "dk", "dv", "dstate"), got, ref, mag):
        check(a, r, m, dtype, T, d, name, is_state=name == "dstate")
    # without the state's gradient the others are right too
    got = pa.linear_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["dmem"], state=x["state"],
                        dstate_out=x["dstate"], lengths=lengths, scale=scale)
    assert got[3] is None
    for name, a, r, m in zip(("dq", "dk", "dv"), got, ref, mag):
        check(a, r, m, dtype, T, d, name + " alone")
    assert pa.device_status() == 0


MANY = [  # enough heads to fill the SMs: whole heads, runs that hold parts of several
    (2, 40, 100, 64, None, True), (2, 20, 300, 128, (300, 171), True),
    (1, 45, 1000, 128, None, True), (3, 30, 777, 64, (777, 1, 500), True),
    (1, 160, 3000, 64, None, True),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", MANY, ids=lambda c: "x".join(map(str, c[:4])))
def test_many_heads(case, dtype):
    test_forward(case, dtype)
    test_backward(case, dtype)


@pytest.mark.parametrize("d,T,H", [(64, 130, 640), (64, 256, 2000), (128, 200, 900), (128, 40, 3000)])
def test_many_short_heads_repeat(d, T, H):
    """Runs of many whole heads change from one head's state to the next all
    the time.  Ten calls into buffers that hold NaN give the same bits, and
    single heads what they give alone (other tile cuts do not arise: one head
    is one or two tiles)."""
    import long_context_attention_causal_gb300 as pa
    x = make(1, H, T, d, "bf16", 5 * d + T, state=True)
    args = [x[n] for n in ("q", "k", "v", "log_decay", "dmem")]
    first = None
    for _ in range(10):
        out = [torch.full_like(x["q"], float("nan")) for _ in range(4)]
        S = pa.linear_fwd(*args[:4], state=x["state"], mem=out[0], want_state=True)[1]
        pa.linear_bwd(*args, state=x["state"], dstate_out=x["dstate"], dq=out[1], dk=out[2],
                      dv=out[3])
        first = first or (*out, S)
        for a, b in zip(first, (*out, S)):
            assert torch.equal(a, b)
    for h in (0, 1, H // 2, H - 1):
        cut = lambda t: t[:, h:h + 1].contiguous()  # noqa: E731
        one = [cut(x[n]) for n in ("q", "k", "v")]
        mem, S = pa.linear_fwd(*one, x["log_decay"][h:h + 1], state=cut(x["state"]),
                               want_state=True)
        got = pa.linear_bwd(*one, x["log_decay"][h:h + 1], cut(x["dmem"]), state=cut(x["state"]),
                            dstate_out=cut(x["dstate"]))
        for a, b in zip((mem, *got[:3], S), first):
            assert torch.equal(a, cut(b)), h
    assert pa.device_status() == 0


def test_gradients_are_differences_of_the_loss():
    """The loss sum(dmem * mem) + sum(dstate * state) is linear in each of q,
    k, v and the state, so its difference along a direction is exact."""
    import long_context_attention_causal_gb300 as pa
    B, H, T, d, scale = 2, 2, 150, 64, 0.2
    x = make(B, H, T, d, "f32", 5, True)
    dq, dk, dv, ds = pa.linear_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["dmem"],
                                   state=x["state"], dstate_out=x["dstate"], scale=scale,
                                   want_dstate=True)

    def loss(**over):
        y = {**x, **over}
        mem, S = linear_fwd_ref(y["q"], y["k"], y["v"], y["log_decay"], scale, y["state"])
        return float((mem * x["dmem"].double()).sum() + (S * x["dstate"].double()).sum())

    g = torch.Generator(device=dev()).manual_seed(9)
    for name, grad in (("q", dq), ("k", dk), ("v", dv), ("state", ds)):
        u = torch.randn(x[name].shape, generator=g, device=dev(), dtype=torch.float64)
        num = (loss(**{name: x[name].double() + u}) - loss(**{name: x[name].double() - u})) / 2
        ana = float((grad.double() * u).sum())
        # fp32 gradients: the units of the bound above over the inner product
        assert abs(num - ana) <= units(T, d) * float((grad.double().abs() * u.abs()).sum()), name


@pytest.mark.parametrize("dtype,d,B,H", [("f32", 64, 1, 1), ("bf16", 128, 3, 5), ("f32", 128, 2, 3),
                                         ("bf16", 64, 7, 1)])
def test_steps_continue_a_prompt(dtype, d, B, H):
    """A prompt of T tokens, then single tokens, equals one longer prompt."""
    import long_context_attention_causal_gb300 as pa
    T, more = 140, 5
    x = make(B, H, T + more, d, dtype, 77 + d, True)
    scale = d ** -0.5
    cut = lambda n: x[n][:, :, :T].contiguous()  # noqa: E731
    _, S = pa.linear_fwd(cut("q"), cut("k"), cut("v"), x["log_decay"], state=x["state"],
                         want_state=True)
    ref, S_ref = linear_fwd_ref(x["q"], x["k"], x["v"], x["log_decay"], scale, x["state"])
    mag, S_mag = linear_fwd_ref(*absolute(x, ("q", "k", "v")), x["log_decay"], scale,
                                x["state"].abs())
    for t in range(T, T + more):
        q, k, v = (x[n][:, :, t].contiguous() for n in ("q", "k", "v"))
        mem = pa.linear_step(S, q, k, v, x["log_decay"])
        err = (mem.double() - ref[:, :, t]).abs()
        own = 2.0 ** -8 * ref[:, :, t].abs() if dtype == "bf16" else 0.0
        assert (err <= (units(T, d) + 2.0 ** -16) * mag[:, :, t] + own).all(), t
    check(S, S_ref, S_mag, "bf16", T, d, "state", is_state=True)


def test_decay_extremes():
    """No decay, a decay whose first power vanishes, and -inf."""
    import long_context_attention_causal_gb300 as pa
    B, T, d = 1, 300, 64
    for dtype in ("f32", "bf16"):
        x = make(B, 4, T, d, dtype, 3, True)
        x["log_decay"] = torch.tensor([0.0, -1e4, -float("inf"), -1e-7], device=dev())
        mem, S = pa.linear_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"],
                               scale=1.0, want_state=True)
        ref, S_ref = linear_fwd_ref(x["q"], x["k"], x["v"], x["log_decay"], 1.0, x["state"])
        mag, S_mag = linear_fwd_ref(*absolute(x, ("q", "k", "v")), x["log_decay"], 1.0,
                                    x["state"].abs())
        check(mem, ref, mag, dtype, T, d, "mem")
        check(S, S_ref, S_mag, dtype, T, d, "state", is_state=True)
        step = pa.linear_step(S, *(x[n][:, :, 0].contiguous() for n in ("q", "k", "v")),
                              x["log_decay"])
        assert torch.isfinite(step.float()).all()


@pytest.mark.parametrize("H,T,d", [(2, 16384, 128), (304, 8192, 64)])
def test_state_without_decay_stays_fp32(H, T, d):
    """Positive inputs and no decay: the state grows to T products of one sign,
    where accumulation errors show.  w = 1 exactly and bf16 inputs are exact as
    hi, so per element, relative: the tensor core adds 16 products a tile into
    the tile's own sum (cut off, 2^-22 each of a sum that holds T / tiles), and
    each tile rounds the fp32 state once, 2^-24; joining runs once more each.
    2^-18 covers inputs that need lo."""
    import long_context_attention_causal_gb300 as pa

    g = torch.Generator(device=dev()).manual_seed(40 + d)
    q, k, v = (torch.randn(1, H, T, d, generator=g, device=dev()).abs().bfloat16()
               for _ in range(3))
    state = pa.linear_fwd(q, k, v, torch.zeros(H, device=dev()), want_state=True)[1]
    tol = 2.0 ** -18 + 16 * 2.0 ** -22 + 2 * (T / 128) * 2.0 ** -24
    for h in (0, H // 2, H - 1):
        ref = v[0, h].double().T @ k[0, h].double()
        assert float(((state[0, h].double() - ref).abs() / ref).max()) <= tol


def test_state_in_place_and_repeats():
    """state_out may be state; the same call gives the same bits."""
    import long_context_attention_causal_gb300 as pa
    for dtype, T in (("bf16", 700), ("f32", 700), ("bf16", 90), ("bf16", 9000)):
        x = make(2, 3, T, 128, dtype, 8, True)
        # the second sequence ends early: the CTAs of its end have nothing to
        # walk and write its state at once
        lens = torch.tensor([T, 30], dtype=torch.int32, device=dev())
        a = pa.linear_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"],
                          lengths=lens, want_state=True)
        S = x["state"].clone()
        b = pa.linear_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=S, state_out=S,
                          lengths=lens)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], S)
        ga = pa.linear_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["dmem"], state=x["state"],
                           dstate_out=x["dstate"], want_dstate=True)
        R = x["dstate"].clone()
        gb = pa.linear_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["dmem"], state=x["state"],
                           dstate_out=R, dstate=R)
        for p, r in zip(ga, gb):
            assert torch.equal(p, r)


def test_tensors_on_odd_16_byte_boundaries():
    """Pointers need 16-byte alignment only."""
    import long_context_attention_causal_gb300 as pa
    B, H, T, d = 1, 3, 333, 64
    for dtype in ("bf16", "f32"):
        x = make(B, H, T, d, dtype, 6, True)
        want = pa.linear_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"],
                             want_state=True)
        gwant = pa.linear_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["dmem"],
                              state=x["state"], want_dstate=True)

        def shifted(t):
            buf = torch.empty(t.numel() + 64, dtype=t.dtype, device=t.device)
            off = next(o for o in range(64) if (buf.data_ptr() + o * t.element_size()) % 32 == 16)
            return buf[off:off + t.numel()].view(t.shape).copy_(t)

        y = {n: shifted(t) for n, t in x.items() if n != "log_decay"}
        mem, S = shifted(x["q"]), shifted(x["state"])
        pa.linear_fwd(y["q"], y["k"], y["v"], x["log_decay"], state=y["state"], mem=mem,
                      state_out=S)
        assert torch.equal(mem, want[0]) and torch.equal(S, want[1])
        g = [shifted(x["q"]) for _ in range(3)] + [shifted(x["state"])]
        pa.linear_bwd(y["q"], y["k"], y["v"], x["log_decay"], y["dmem"], state=y["state"], dq=g[0],
                      dk=g[1], dv=g[2], dstate=g[3])
        for a, b in zip(g, gwant):
            assert torch.equal(a, b)
        tok = [shifted(x[n][:, :, 0].contiguous()) for n in ("q", "k", "v")]
        S1, S2 = x["state"].clone(), shifted(x["state"])
        a = pa.linear_step(S1, *(x[n][:, :, 0].contiguous() for n in ("q", "k", "v")),
                           x["log_decay"])
        b = pa.linear_step(S2, *tok, x["log_decay"], mem=shifted(a))
        assert torch.equal(a, b) and torch.equal(S1, S2)


def test_empty_prompt_passes_the_state():
    import long_context_attention_causal_gb300 as pa
    z = torch.empty((2, 3, 0, 64), device=dev())
    ld = decay(3).to(dev())
    S = torch.randn((2, 3, 64, 64), device=dev())
    mem, out = pa.linear_fwd(z, z, z, ld, state=S, want_state=True)
    assert mem.shape == z.shape and torch.equal(out, S)
    assert torch.equal(pa.linear_fwd(z, z, z, ld, want_state=True)[1], torch.zeros_like(S))
    assert torch.equal(pa.linear_bwd(z, z, z, ld, z, dstate_out=S, want_dstate=True)[3], S)
    n = torch.empty((0, 3, 5, 64), device=dev())
    assert pa.linear_fwd(n, n, n, ld)[0].numel() == 0


def test_lengths_out_of_range_are_clamped_and_reported():
    import long_context_attention_causal_gb300 as pa
    pa.device_status(reset=True)
    for dtype in ("f32", "bf16"):
        x = make(2, 2, 200, 64, dtype, 4)
        bad = torch.tensor([-3, 999], dtype=torch.int32, device=dev())
        good = torch.tensor([0, 200], dtype=torch.int32, device=dev())
        a = pa.linear_fwd(x["q"], x["k"], x["v"], x["log_decay"], lengths=bad, want_state=True)
        assert pa.device_status(reset=True) == 3
        b = pa.linear_fwd(x["q"], x["k"], x["v"], x["log_decay"], lengths=good, want_state=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert pa.device_status() == 0


def test_capture_replays_on_new_inputs():
    import long_context_attention_causal_gb300 as pa
    B, H, T, d = 1, 4, 600, 128
    x = make(B, H, T, d, "bf16", 12, True)
    ws = torch.empty(max(16, pa.linear_bwd_workspace_bytes(B, H, T, d)), device=dev(),
                     dtype=torch.uint8)
    mem, S = torch.empty_like(x["q"]), torch.empty_like(x["state"])
    grads = [torch.empty_like(x["q"]) for _ in range(3)]
    tok = [x[n][:, :, 0].contiguous() for n in ("q", "k", "v")]
    step = torch.empty_like(tok[0])

    def calls():
        pa.linear_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"], mem=mem,
                      state_out=S, workspace=ws)
        pa.linear_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["dmem"], state=x["state"],
                      dstate_out=x["dstate"], dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws)
        pa.linear_step(S, *tok, x["log_decay"], mem=step)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    y = make(B, H, T, d, "bf16", 13, True)
    for n in ("q", "k", "v", "dmem", "state", "dstate"):
        x[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (mem, S, step, *grads)]
    for t in (mem, S, step, *grads):
        t.fill_(float("nan"))
    calls()
    torch.cuda.synchronize()
    for a, b in zip(got, (mem, S, step, *grads)):
        assert torch.equal(a, b)


def test_two_streams_with_two_workspaces():
    import long_context_attention_causal_gb300 as pa
    xs = [make(1, 3, 900, 128, "bf16", s, True) for s in (21, 22)]
    want = [pa.linear_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"],
                          want_state=True) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for x, s in zip(xs, streams):
        with torch.cuda.stream(s):
            got.append([pa.linear_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"],
                                      want_state=True) for _ in range(4)])
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        for g in many:
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_given_stream_owns_what_is_allocated():
    """Results and workspaces of a call on a given stream are not handed out
    again by the current stream's allocations while it still runs."""
    import long_context_attention_causal_gb300 as pa
    x = make(1, 3, 3000, 128, "bf16", 31, True)
    args = (x["q"], x["k"], x["v"], x["log_decay"])
    want = pa.linear_fwd(*args, state=x["state"], want_state=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(6):
        got.append(pa.linear_fwd(*args, state=x["state"], want_state=True, stream=side))
        junk = [torch.full((1 << 20,), float("nan"), device=dev()) for _ in range(8)]
        del junk
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])


def test_arguments_by_name():
    """Every argument may be given by name, the first included, with or
    without a stream."""
    import long_context_attention_causal_gb300 as pa
    x = make(1, 2, 200, 64, "bf16", 3, state=True)
    args = {n: x[n] for n in ("q", "k", "v", "log_decay", "state")}
    want = pa.linear_fwd(*args.values(), want_state=True)
    for stream in (None, torch.cuda.Stream()):
        got = pa.linear_fwd(want_state=True, stream=stream, **args)
        one = pa.linear_step(state=x["state"].clone(), log_decay=x["log_decay"], stream=stream,
                             **{n: x[n][:, :, 0].contiguous() for n in ("q", "k", "v")})
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.isfinite(one.float()).all()


def test_refusals():
    import long_context_attention_causal_gb300 as pa
    x = make(1, 2, 16, 64, "f32", 1)
    a = (x["q"], x["k"], x["v"], x["log_decay"])
    with pytest.raises(ValueError):
        pa.linear_fwd(x["q"], x["k"][:, :, :8].contiguous(), x["v"], x["log_decay"])
    with pytest.raises(TypeError):
        pa.linear_fwd(x["q"], x["k"].bfloat16(), x["v"], x["log_decay"])
    with pytest.raises(ValueError):
        pa.linear_fwd(x["q"], x["k"], x["v"], x["log_decay"][:1])
    with pytest.raises(ValueError):
        pa.linear_fwd(x["q"].transpose(1, 2).contiguous().transpose(1, 2), *a[1:])
    with pytest.raises(TypeError):
        pa.linear_fwd(*a, lengths=torch.tensor([3], device=dev()))
    with pytest.raises(TypeError):
        pa.linear_fwd(x["q"].cpu(), *a[1:])
    y = make(1, 2, 4000, 64, "f32", 1)  # few long heads are cut: a workspace is needed
    with pytest.raises(pa.PolarError):
        pa.linear_fwd(y["q"], y["k"], y["v"], y["log_decay"],
                      workspace=torch.empty(16, device=dev(), dtype=torch.uint8))
    with pytest.raises(pa.PolarError):
        pa.linear_fwd(*a, scale=float("nan"))
    h = [t.half() for t in a[:3]]
    with pytest.raises(TypeError):
        pa.linear_fwd(*h, x["log_decay"])
    w = torch.zeros((1, 2, 16, 96), device=dev())
    with pytest.raises(pa.PolarError):
        pa.linear_fwd(w, w, w, x["log_decay"])
    with pytest.raises(ValueError):
        pa.linear_step(torch.zeros((1, 2, 64, 32), device=dev()), *(t[:, :, 0].contiguous()
                                                                   for t in a[:3]), a[3])
    with pytest.raises(ValueError):
        pa.linear_bwd(*a, x["dmem"][:, :1].contiguous())

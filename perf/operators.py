"""Workloads of the linear-memory and cache-eviction operators, in plain torch
and through the library.

Five operators, each in two forms: `run` with `own` false computes them with
elementary torch operations in fp32 (exponents of the decay in fp64), with
`own` true it makes the calls a program makes of
long_context_attention_causal_gb300.

  linear_fwd   S_t = g S_{t-1} + v_t k_t^T,  mem_t = scale S_t q_t over a prompt
  linear_bwd   its gradients dq, dk, dv and the incoming state's
  linear_step  one token of it, the state updated in place
  decode       paged grouped-query Polar decode that also adds every cache
               row's attention weight to a running sum
  evict        keep the rows of largest accumulated weight, in place
"""
import math

import torch

own = False

DEV = "cuda"
CHUNK = 128
LOG_T0 = math.log(2048.0)  # neutral length of the temperature, and kappa


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # the framework's smallest prefill in length and heads: latency
        dict(name="linear_fwd_tiny", op="linear_fwd", B=1, H=2, T=100, d=64, dtype="f32",
             ragged=False, state=False),
        # a training or prefill batch of the headline prefill's shape
        dict(name="linear_fwd_16k", op="linear_fwd", B=2, H=16, T=16384, d=128, dtype="bf16",
             ragged=False, state=False),
        # one long prompt, continued from a state kept from earlier text
        dict(name="linear_fwd_64k", op="linear_fwd", B=1, H=16, T=65536, d=128, dtype="bf16",
             ragged=False, state=True),
        # a padded serving batch of prompts of different, odd lengths
        dict(name="linear_fwd_ragged", op="linear_fwd", B=8, H=8, T=1111, d=64, dtype="bf16",
             ragged=True, state=True),
        # the backward of the headline prefill's shape
        dict(name="linear_bwd_16k", op="linear_bwd", B=2, H=16, T=16384, d=128, dtype="bf16",
             ragged=False, state=False),
        # a small fp32 training step on padded sequences, state gradients included
        dict(name="linear_bwd_ragged", op="linear_bwd", B=3, H=4, T=777, d=64, dtype="f32",
             ragged=True, state=True),
        # one decode step of a large serving batch
        dict(name="linear_step_256", op="linear_step", B=256, H=16, T=1, d=128, dtype="bf16",
             ragged=False, state=True),
        # one decode step of a single sequence: latency
        dict(name="linear_step_1", op="linear_step", B=1, H=16, T=1, d=64, dtype="f32",
             ragged=False, state=True),
        # the framework's paged decode workload, weights accumulated
        dict(name="decode_weights_32k", op="decode", B=32, Hq=16, Hkv=4, T=32768, d=128, page=64,
             dtype="bf16", ragged=False),
        # a small ragged batch on small pages
        dict(name="decode_weights_ragged", op="decode", B=4, Hq=8, Hkv=4, T=1500, d=64, page=16,
             dtype="f32", ragged=True),
        # long prompts cut to a quarter of their rows after the prefill
        dict(name="evict_32k", op="evict", B=32, Hkv=4, T=32768, d=128, page=64, dtype="bf16",
             keep=8192, recent=512, ragged=False),
        # the running cut of a decode loop: a page's worth of rows at a time
        dict(name="evict_step", op="evict", B=16, Hkv=8, T=2112, d=64, page=64, dtype="bf16",
             keep=2048, recent=256, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear_fwd", "linear_fwd", "linear_bwd", "linear_bwd", "linear_step", "decode",
                     "decode", "evict", "evict"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("linear_fwd", "linear_bwd"):
        H = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        B = rng.choice([1, 1, 2, 3, 4, 8])
        top = (1 << 19) // (B * H)  # token-heads of the largest drawn case
        if dtype == "f32":
            top //= 4
        return dict(op=op, B=B, H=H, T=_log_int(rng, 1, min(top, 40000)), d=d, dtype=dtype,
                    ragged=rng.random() < 0.4, state=rng.random() < 0.5)
    if op == "linear_step":
        return dict(op=op, B=_log_int(rng, 1, 200), H=rng.choice([1, 2, 4, 5, 8, 16]), T=1, d=d,
                    dtype=dtype, ragged=False, state=True)
    page = rng.choice([8, 16, 32, 64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    B = _log_int(rng, 1, 24)
    T = _log_int(rng, 1, min(32768, (1 << 21) // (B * Hkv)))
    if op == "decode":
        return dict(op=op, B=B, Hq=Hkv * rng.choice([1, 2, 4, 8]), Hkv=Hkv, T=T, d=d, page=page,
                    dtype=dtype, ragged=rng.random() < 0.5)
    T = max(T, 8)
    keep = max(1, int(T * rng.uniform(0.1, 0.98)))
    return dict(op=op, B=B, Hkv=Hkv, T=T, d=d, page=page, dtype=dtype, keep=keep,
                recent=int(keep * rng.choice([0.0, 0.05, 0.3])), ragged=rng.random() < 0.5)


def _lengths(case):
    """Rows of each sequence: all T, or spread evenly down to a short one."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [max(1, T * (B - b) // B - 3 * (b % 2)) for b in range(B)]


# ----------------------------------------------------------------- inputs --

def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 1009 + 17)

    def randn(*shape, std=1.0, dtype=torch.float32):
        out = torch.empty(shape, device=DEV, dtype=dtype)
        flat, n = out.view(-1), 1 << 26
        for o in range(0, flat.numel(), n):  # bounds the fp32 scratch
            part = torch.randn(min(n, flat.numel() - o), generator=g, device=DEV)
            flat[o:o + n] = part * std
        return out

    op, B, d, dt = case["op"], case["B"], case["d"], _dtype(case)
    lens = _lengths(case)
    st = {"case": case, "op": op}
    if op.startswith("linear"):
        H, T = case["H"], case["T"]
        # heads forget over 2^3 ... 2^11 tokens, spread geometrically
        span = torch.linspace(3.0, 11.0, H) if H > 1 else torch.tensor([7.0])
        st["log_decay"] = (-torch.exp2(-span)).to(DEV)
        st["scale"] = d ** -0.5
        st["state"] = randn(B, H, d, d, std=0.5) if case["state"] else None
        if op == "linear_step":
            for n in ("q", "k", "v"):
                st[n] = randn(B, H, d, dtype=dt)
            return st
        for n in ("q", "k", "v"):
            st[n] = randn(B, H, T, d, dtype=dt)
        st["lengths"] = (torch.tensor(lens, dtype=torch.int32, device=DEV) if case["ragged"]
                         else None)
        if op == "linear_bwd":
            st["dmem"] = randn(B, H, T, d, dtype=dt)
            st["dstate"] = randn(B, H, d, d, std=0.5) if case["state"] else None
        return st
    Hkv, page = case["Hkv"], case["page"]
    npg = [(n + page - 1) // page for n in lens]
    gc = torch.Generator().manual_seed(int(seed) * 7919 + 5)
    perm = torch.randperm(sum(npg), generator=gc).to(torch.int32)
    cols = max(npg)
    table = torch.zeros((B, cols), dtype=torch.int32)
    o = 0
    for b in range(B):
        table[b, :npg[b]] = perm[o:o + npg[b]]
        o += npg[b]
    st["table"] = table.to(DEV)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["k_pages"] = randn(sum(npg), Hkv, page, d, dtype=dt)
    st["v_pages"] = randn(sum(npg), Hkv, page, d, dtype=dt)
    cap = cols * page
    if op == "decode":
        Hq = case["Hq"]
        st["q"] = randn(B, Hq, d, dtype=dt)
        st["mem"] = randn(B, Hq, d, std=0.1, dtype=dt)
        st["w_count"] = randn(Hq, d, std=0.02)
        st["weights"] = torch.zeros((B, Hkv, cap), device=DEV)
        return st
    # accumulated weights are heavy-tailed; every slot holds its own token
    st["weights"] = torch.exp(2.0 * randn(B, Hkv, cap)) / case["T"]
    st["positions"] = torch.arange(cap, dtype=torch.int32, device=DEV).repeat(B, Hkv, 1)
    return st


# ------------------------------------------------------------ plain forms --

def _powers(log_decay, n):
    """exp(log_decay * n) in fp32 for integer n >= 0 (0 where n < 0), fp64 inside."""
    e = log_decay.double().reshape(-1, *([1] * n.dim())) * n.clamp(min=0).double()
    return torch.where(n >= 0, torch.exp(e), torch.zeros_like(e)).float()


def _mix(x, y, z, log_decay, init, scale):
    """scale * sum_{s <= t} g^(t-s) (x_t . y_s) z_s + scale * g^(t+1) init x_t, by chunks."""
    B, H, T, d = x.shape
    N = -(-T // CHUNK)
    pad = (0, 0, 0, N * CHUNK - T)
    x, y, z = (torch.nn.functional.pad(t, pad).view(B, H, N, CHUNK, d) for t in (x, y, z))
    i = torch.arange(CHUNK, device=x.device)
    n = torch.arange(N, device=x.device)
    local = (x @ y.transpose(-1, -2)) * _powers(log_decay, i[:, None] - i[None, :])[None, :, None]
    out = local @ z
    ends = _powers(log_decay, CHUNK - 1 - i)[None, :, None, :, None]
    parts = (z * ends).transpose(-1, -2) @ y
    carry = _powers(log_decay * CHUNK, n[:, None] - 1 - n[None, :])
    states = (carry[None] @ parts.reshape(B, H, N, d * d)).view(B, H, N, d, d)
    if init is not None:
        states = states + _powers(log_decay * CHUNK, n)[None, :, :, None, None] * init[:, :, None]
    starts = _powers(log_decay, i + 1)[None, :, None, :, None]
    out = out + (x * starts) @ states.transpose(-1, -2)
    return scale * out.reshape(B, H, N * CHUNK, d)[:, :, :T]


def _tokens(st):
    """Which tokens exist, [B, 1, T, 1], and the lengths [B, 1, 1] as int64."""
    B, T = st["q"].shape[0], st["q"].shape[2]
    t = torch.arange(T, device=DEV)
    lens = (torch.full((B,), T, device=DEV) if st["lengths"] is None else st["lengths"].long())
    return t, lens, (t[None, :] < lens[:, None])[:, None, :, None]


def _to_end(log_decay, t, lens):
    """g^(len - 1 - t) per (b, h, token), 0 past the end: [B, H, T, 1]."""
    w = _powers(log_decay, lens[:, None] - 1 - t[None, :])  # [H, B, T]
    return w.transpose(0, 1)[..., None]


def _run_linear_fwd(st):
    t, lens, here = _tokens(st)
    q, k, v = (st[n].float() * here for n in ("q", "k", "v"))
    mem = _mix(q, k, v, st["log_decay"], st["state"], st["scale"])
    last = (v * _to_end(st["log_decay"], t, lens)).transpose(-1, -2) @ k
    if st["state"] is not None:
        last = last + _powers(st["log_decay"], lens).t()[..., None, None] * st["state"]
    return {"mem": mem.to(st["q"].dtype), "state": last}


def _run_linear_bwd(st):
    ld, scale, dt = st["log_decay"], st["scale"], st["q"].dtype
    t, lens, here = _tokens(st)
    q, k, v, g = (st[n].float() * here for n in ("q", "k", "v", "dmem"))
    init = None if st["state"] is None else st["state"].transpose(-1, -2)
    dq = _mix(g, v, k, ld, init, scale)

    def flip(*ts):
        return [x.flip(2) for x in ts]

    def back(x, y, z):
        # the sums run from the last token, which takes no decay itself
        return _mix(*flip(x, y, z), ld, None, scale).flip(2)

    dk, dv = back(v, g, q), back(k, q, g)
    first = _powers(ld, t + 1)[None, :, :, None]
    dstate = scale * ((g * first).transpose(-1, -2) @ q)
    if st["dstate"] is not None:
        ends = _to_end(ld, t, lens)
        dk = dk + ends * (v @ st["dstate"])
        dv = dv + ends * (k @ st["dstate"].transpose(-1, -2))
        dstate = dstate + _powers(ld, lens).t()[..., None, None] * st["dstate"]
    out = {"dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt)}
    if st["state"] is not None:
        out["dstate"] = dstate
    return out


def _run_linear_step(st):
    S = st["state"]
    q, k, v = (st[n].float() for n in ("q", "k", "v"))
    decay = torch.exp(st["log_decay"].double()).float()[None, :, None, None]
    S.copy_(decay * S + v[..., :, None] * k[..., None, :])
    mem = st["scale"] * (S * q[..., None, :]).sum(-1)
    return {"mem": mem.to(st["q"].dtype), "state": S}


def _run_decode(st):
    q, w = st["q"].float(), st["weights"]
    B, Hq, d = q.shape
    Hkv = w.shape[1]
    G = Hq // Hkv

    def gather(pages):
        x = pages[st["table"].long()]  # [B, cols, Hkv, page, d]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d).float()

    k = gather(st["k_pages"])
    n = st["lens"].float()[:, None, None, None]
    tau = (torch.log(n) / LOG_T0).clamp(min=1.0)
    s = tau * d ** -0.5 * (q.view(B, Hkv, G, d) @ k.transpose(-1, -2))
    del k
    seen = torch.arange(s.shape[-1], device=DEV)[None, :] < st["lens"][:, None]
    s = torch.where(seen[:, None, None], s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    p = p / l
    lse = m + torch.log(l)
    n_eff = 1.0 / (p * p).sum(-1, keepdim=True)
    norm = q.view(B, Hkv, G, d).square().sum(-1, keepdim=True).sqrt()
    floor = tau * norm * d ** -0.5 * torch.sqrt(2.0 * torch.log(n))
    conf = 1.0 / (1.0 + torch.exp(floor - lse))
    a = p @ gather(st["v_pages"])
    u = a / a.square().sum(-1, keepdim=True).sqrt().clamp(min=1e-6)
    count = conf * torch.tanh(torch.log(n_eff) / LOG_T0)
    out = (u + count * st["w_count"].view(Hkv, G, d)).view(B, Hq, d) + st["mem"].float()
    w += p.sum(2)
    return {"out": out.to(st["q"].dtype), "n_eff": n_eff.view(B, Hq), "conf": conf.view(B, Hq),
            "weights": w}


def _run_evict(st):
    keep, recent = st["case"]["keep"], st["case"]["recent"]
    w, pos = st["weights"].clone(), st["positions"].clone()
    kp, vp, lens = st["k_pages"], st["v_pages"], st["lens"].long()
    B, Hkv, cap = w.shape
    page = kp.shape[2]
    slot = torch.arange(cap, device=DEV)
    live = (slot[None, :] < lens[:, None])[:, None, :].expand(B, Hkv, cap)
    over = (lens > keep)[:, None, None]
    newest = torch.where(live, pos, torch.full_like(pos, -1)).amax(-1, keepdim=True)
    guard = live & (pos > newest - recent)
    rank_by = torch.where(guard, torch.full_like(w, math.inf), w)
    rank_by = torch.where(live, rank_by, torch.full_like(w, -math.inf))
    order = torch.sort(rank_by, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(live)
    kept = kept.scatter(-1, order[..., :keep], True)
    hole = over & ~kept & (slot < keep)
    mover = over & kept & (slot >= keep)
    # both are in ascending order of (b, head, slot), and as many in each head
    bh_hole, bh_mover = hole.nonzero(), mover.nonzero()
    if bh_hole.numel():
        b, h, dst = bh_hole.unbind(1)
        src = bh_mover[:, 2]
        p_dst, p_src = st["table"][b, dst // page].long(), st["table"][b, src // page].long()
        for pool in (kp, vp):
            pool[p_dst, h, dst % page] = pool[p_src, h, src % page]
        w[b, h, dst] = w[b, h, src]
        pos[b, h, dst] = pos[b, h, src]
    w = torch.where(over & live & (slot >= keep), torch.zeros_like(w), w)
    return {"k_pages": kp, "v_pages": vp, "weights": w, "positions": pos,
            "lens": torch.minimum(lens, torch.full_like(lens, keep)).to(torch.int32)}


# -------------------------------------------------------- library's calls --

def _own(st):
    import long_context_attention_causal_gb300 as pa
    op = st["op"]
    if op == "linear_fwd":
        mem, state = pa.linear_fwd(st["q"], st["k"], st["v"], st["log_decay"], state=st["state"],
                                   lengths=st["lengths"], scale=st["scale"], want_state=True)
        return {"mem": mem, "state": state}
    if op == "linear_bwd":
        dq, dk, dv, dstate = pa.linear_bwd(st["q"], st["k"], st["v"], st["log_decay"], st["dmem"],
                                           state=st["state"], dstate_out=st["dstate"],
                                           lengths=st["lengths"], scale=st["scale"],
                                           want_dstate=st["state"] is not None)
        out = {"dq": dq, "dk": dk, "dv": dv}
        if dstate is not None:
            out["dstate"] = dstate
        return out
    if op == "linear_step":
        mem = pa.linear_step(st["state"], st["q"], st["k"], st["v"], st["log_decay"],
                             scale=st["scale"])
        return {"mem": mem, "state": st["state"]}
    if op == "decode":
        out, n_eff, conf = pa.decode_paged_weights(
            st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"], st["mem"],
            st["w_count"], st["weights"], max_seq_len=st["case"]["T"], want_conf=True)
        return {"out": out, "n_eff": n_eff, "conf": conf, "weights": st["weights"]}
    # the sums and positions go on from the same start in every pass
    w, pos = st["weights"].clone(), st["positions"].clone()
    lens = pa.cache_evict(st["k_pages"], st["v_pages"], st["table"], st["lens"], w, pos,
                          st["case"]["keep"], recent=st["case"]["recent"],
                          max_seq_len=st["case"]["T"])
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"], "weights": w, "positions": pos,
            "lens": lens}


def run(state):
    if own:
        return _own(state)
    return {"linear_fwd": _run_linear_fwd, "linear_bwd": _run_linear_bwd,
            "linear_step": _run_linear_step, "decode": _run_decode,
            "evict": _run_evict}[state["op"]](state)


# ------------------------------------------------------------------- work --

def work(case):
    op, B, d = case["op"], case["B"], case["d"]
    es = 4 if case["dtype"] == "f32" else 2
    rows = float(sum(_lengths(case)))
    if op.startswith("linear"):
        H = case["H"]
        state = 4.0 * B * H * d * d
        if op == "linear_step":
            return {"bytes": 2 * state + 4.0 * B * H * d * es, "flops": 4.0 * B * H * d * d}
        if op == "linear_fwd":
            return {"bytes": 4.0 * rows * H * d * es + state * (2 if case["state"] else 1),
                    "flops": 4.0 * rows * H * d * d}
        return {"bytes": 7.0 * rows * H * d * es + (3 * state if case["state"] else 0),
                "flops": 10.0 * rows * H * d * d}
    Hkv = case["Hkv"]
    if op == "decode":
        return {"bytes": rows * Hkv * (2.0 * d * es + 8) + B * case["Hq"] * (3.0 * d * es + 8),
                "flops": 4.0 * rows * case["Hq"] * d}
    # a kept row sits past the cut with the share of the rows that do; the
    # protected newest rows always do where they fit there
    moved = 0.0
    for n in _lengths(case):
        if n > case["keep"]:
            past, newest = n - case["keep"], case["recent"]
            free = max(0, past - newest) / max(1, n - newest)
            moved += min(past, newest) + (case["keep"] - newest) * free
    return {"bytes": rows * Hkv * 8.0 + moved * Hkv * 2 * (2.0 * d * es + 8), "flops": 0.0}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    """The definitions, token by token or sequence by sequence, in 64 bits."""
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("linear"):
        return _exact_linear(st, case)
    return _exact_decode(st, case) if op == "decode" else _exact_evict(st, case)


def _exact_linear(st, case):
    B, H, T, d = case["B"], case["H"], case["T"], case["d"]
    q, k, v = (st[n].double().view(B * H, T, d) for n in ("q", "k", "v"))
    scale = st["scale"]
    lens = torch.tensor(_lengths(case), device=DEV).repeat_interleave(H)
    gam = torch.exp(st["log_decay"].double()).repeat(B)
    S = (torch.zeros((B * H, d, d), dtype=torch.float64, device=DEV) if st["state"] is None
         else st["state"].double().view(B * H, d, d).clone())
    there = (torch.arange(T, device=DEV)[:, None] < lens[None, :]).double()[..., None, None]
    step = torch.where(there > 0, gam[:, None, None], torch.ones_like(gam)[:, None, None])
    first = torch.zeros((T, B * H, d, 1), dtype=torch.float64, device=DEV)
    cols = k.transpose(0, 1)[:, :, None, :] * there      # [T, BH, 1, d]
    vals = v.transpose(0, 1)[..., None]
    grad = case["op"] == "linear_bwd"
    reads = ((st["dmem"].double().view(B * H, T, d) if grad else q).transpose(0, 1)[..., None]
             * there * scale)
    for t in range(T):
        S.mul_(step[t]).baddbmm_(vals[t], cols[t])
        torch.bmm(S.transpose(1, 2) if grad else S, reads[t], out=first[t])
    first = first[..., 0].transpose(0, 1).reshape(B, H, T, d)
    if not grad:
        mem = first if case["op"] == "linear_fwd" else first[:, :, 0]
        return {"mem": mem, "state": S.view(B, H, d, d)}
    R = (torch.zeros((B * H, d, d), dtype=torch.float64, device=DEV) if st["dstate"] is None
         else st["dstate"].double().view(B * H, d, d).clone())
    dk, dv = torch.zeros_like(vals), torch.zeros_like(vals)
    qrow = q.transpose(0, 1)[:, :, None, :]
    kcol = cols.transpose(2, 3)
    vcol = vals * there
    for t in range(T - 1, -1, -1):
        R.baddbmm_(reads[t], qrow[t])
        torch.bmm(R.transpose(1, 2), vcol[t], out=dk[t])
        torch.bmm(R, kcol[t], out=dv[t])
        R.mul_(step[t])
    out = {"dq": first}
    for n, x in (("dk", dk), ("dv", dv)):
        out[n] = x[..., 0].transpose(0, 1).reshape(B, H, T, d)
    if st["state"] is not None:
        out["dstate"] = R.view(B, H, d, d)
    return out


def _exact_decode(st, case):
    B, Hq, Hkv, d, page = (case[n] for n in ("B", "Hq", "Hkv", "d", "page"))
    out, n_eff = torch.zeros((B, Hq, d), dtype=torch.float64, device=DEV), []
    conf, weights = [], st["weights"].double().clone()
    for b, n in enumerate(_lengths(case)):
        ids = st["table"][b, :-(-n // page)].long()
        k = st["k_pages"][ids].double().transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
        v = st["v_pages"][ids].double().transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
        k, v = (x.repeat_interleave(Hq // Hkv, 0) for x in (k, v))
        q = st["q"][b].double()
        tau = max(1.0, math.log(n) / LOG_T0)
        s = torch.einsum("hd,hnd->hn", q, k) * (tau / math.sqrt(d))
        p = torch.softmax(s, -1)
        weights[b, :, :n] += p.view(Hkv, -1, n).sum(1)
        n_eff.append(1.0 / p.square().sum(-1))
        floor = tau * torch.linalg.vector_norm(q, dim=-1) / math.sqrt(d) * math.sqrt(2 * math.log(n))
        conf.append(torch.sigmoid(torch.logsumexp(s, -1) - floor))
        a = torch.einsum("hn,hnd->hd", p, v)
        a = a / torch.linalg.vector_norm(a, dim=-1, keepdim=True).clamp(min=1e-6)
        gate = conf[-1] * torch.tanh(torch.log(n_eff[-1]) / LOG_T0)
        out[b] = a + gate[:, None] * st["w_count"].double() + st["mem"][b].double()
    return {"out": out, "n_eff": torch.stack(n_eff), "conf": torch.stack(conf), "weights": weights}


def _exact_evict(st, case):
    keep, recent, page = case["keep"], case["recent"], case["page"]
    w, pos = st["weights"], st["positions"]
    lens = _lengths(case)
    for b, n in enumerate(lens):
        if n <= keep:
            continue
        for h in range(case["Hkv"]):
            ws, ps = w[b, h, :n], pos[b, h, :n]
            old = torch.nonzero(ps <= ps.max() - recent).flatten()
            spare = torch.argsort(ws[old], stable=True, descending=True)
            stay = torch.ones(n, dtype=torch.bool, device=DEV)
            stay[old[spare[max(0, keep - (n - old.numel())):]]] = False
            to = torch.nonzero(~stay[:keep]).flatten()
            fro = keep + torch.nonzero(stay[keep:]).flatten()
            row = st["table"][b].long()
            for pool in (st["k_pages"], st["v_pages"]):
                pool[row[to // page], h, to % page] = pool[row[fro // page], h, fro % page]
            ws[to], ps[to] = ws[fro], ps[fro]
            ws[keep:] = 0
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"], "weights": w, "positions": pos,
            "lens": torch.tensor([min(n, keep) for n in lens], dtype=torch.int32, device=DEV)}

"""Workloads of the operators between a batch of requests and its tokens, in
plain torch and through the library.

Five operators, each in two forms: `run` with `own` false computes them with
elementary torch operations in fp32 (angles and quantisation borders in
fp64), with `own` true it makes the calls a program makes of
long_context_attention_causal_gb300.

  pages    requests that ended give their pages back, the others get pages for
           their new tokens: block table, slot of every token, positions
  rope     rotary positions of q and k (forward, or its gradient)
  prefill  causal Polar attention over packed prompts with grouped heads
  store    k and v rows into a paged 4-bit cache, and back as their values
  decode   Polar decode against the paged 4-bit cache

The 4-bit cache: pages [num_pages, Hkv, page, 9 d / 16] of bytes.  The block
of a (page, head) holds page * d / 2 bytes of codes, row after row, then page *
d / 32 bf16 scales, row after row.  32 consecutive channels share a scale s =
bf16(max |x| / 7); a code is n = round(x / s), -7 <= n <= 7, as a sign and
three bits.  Channels 4 p + j, j < 4, make 16 bits: signs in bits 15, 11, 7, 3,
|n| from bits 4, 0, 12, 8 on.  Two of them make a 32-bit word, and word w = 4 i
+ c (i < d / 32, c < 4) of a row stands in place c * d / 32 + i.
"""
import math

import torch

own = False

DEV = "cuda"
LOG_T0 = math.log(2048.0)  # neutral length of the temperature, and kappa
GROUP = 32  # channels that share a scale
SIGN_AT, SIZE_AT = (15, 11, 7, 3), (4, 0, 12, 8)  # bits of a code in its 16


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token for each sequence of a large serving batch, some requests
        # ended: latency
        dict(name="pages_step_256", op="pages", B=256, T=2048, new=1, page=64, ended=0.05,
             short=False),
        # new prompts of different lengths on small pages
        dict(name="pages_prompts", op="pages", B=96, T=500, new=8000, page=16, ended=0.0,
             short=False),
        # q and k of the headline prefill's tokens, halves, whole head
        dict(name="rope_32k", op="rope", N=32768, Hq=16, Hkv=4, d=128, rot=128, dtype="bf16",
             interleaved=False, inverse=False, far=1 << 17),
        # gradient of a small fp32 batch: pairs side by side, half of the head
        dict(name="rope_bwd_part", op="rope", N=1555, Hq=6, Hkv=2, d=64, rot=32, dtype="f32",
             interleaved=True, inverse=True, far=1 << 20),
        # the headline prefill's tokens as two prompts, four query heads a KV head
        dict(name="prefill_16k", op="prefill", B=2, T=16384, Hq=16, Hkv=4, d=128, dtype="bf16",
             ragged=False),
        # prompts of a serving step: from one token to thousands
        dict(name="prefill_ragged", op="prefill", B=24, T=2900, Hq=16, Hkv=2, d=128, dtype="bf16",
             ragged=True),
        # many short prompts, a KV head for each query head
        dict(name="prefill_short", op="prefill", B=200, T=190, Hq=8, Hkv=8, d=64, dtype="bf16",
             ragged=True),
        # the framework's smallest prefill in length and heads: latency
        dict(name="prefill_tiny", op="prefill", B=3, T=100, Hq=2, Hkv=1, d=64, dtype="f32",
             ragged=True),
        # the headline prefill's rows into the cache, and read back
        dict(name="store_32k", op="store", N=32768, Hkv=4, d=128, page=64, dtype="bf16"),
        # one decode step of a batch: latency
        dict(name="store_step", op="store", N=257, Hkv=8, d=64, page=16, dtype="f32"),
        # the framework's paged decode workload
        dict(name="decode_32k", op="decode", B=32, Hq=16, Hkv=4, T=32768, d=128, page=64,
             dtype="bf16", ragged=False),
        # a small ragged batch on small pages
        dict(name="decode_ragged", op="decode", B=5, Hq=8, Hkv=2, T=1500, d=64, page=16,
             dtype="f32", ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["pages", "rope", "rope", "prefill", "prefill", "prefill", "store", "store",
                     "decode", "decode", "decode"])
    if op == "pages":
        return dict(op=op, B=_log_int(rng, 1, 1000), T=_log_int(rng, 1, 4000),
                    new=rng.choice([1, 1, _log_int(rng, 2, 4000)]),
                    page=rng.choice([8, 16, 32, 64, 128, 256]), ended=rng.choice([0.0, 0.05, 0.3]),
                    short=rng.random() < 0.2)
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    if op == "rope":
        rot = rng.choice([d, d, d // 2, d // 4, d * 3 // 4, 26])
        return dict(op=op, N=_log_int(rng, 1, (1 << 18) // (Hq + Hkv)), Hq=Hq, Hkv=Hkv, d=d, rot=rot,
                    dtype=dtype, interleaved=rng.random() < 0.5, inverse=rng.random() < 0.4,
                    far=_log_int(rng, 1000, 1 << 22))
    if op == "store":
        return dict(op=op, N=_log_int(rng, 1, 60000 // Hkv), Hkv=Hkv, d=d,
                    page=rng.choice([8, 16, 32, 64, 128, 256]), dtype=dtype)
    if op == "prefill":
        B = _log_int(rng, 1, 64)
        # pairs of a row and a key over all heads: an eighth of the largest
        # listed case's, less in fp32
        room = (1 << 30) // (4 if dtype == "f32" else 1)
        T = _log_int(rng, 1, min(8000, int(math.sqrt(room / (B * Hq)))))
        return dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, ragged=rng.random() < 0.7)
    B = _log_int(rng, 1, 32)
    T = _log_int(rng, 1, min(100000, (1 << 21) // (B * Hkv)))
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, page=rng.choice([8, 16, 32, 64, 128, 256]),
                dtype=dtype, ragged=rng.random() < 0.5)


def _lengths(case):
    """Tokens of each sequence: all T, or spread evenly from one token to T."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [max(1, T * (b + 1) // B - 3 * (b % 2)) if b else 1 for b in range(B)]


# ----------------------------------------------------------------- inputs --

def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _inv_freq(rot):
    """Frequencies of a context stretched four times: the slow half of the
    pairs turns four times slower, the fast half as before."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    return torch.where(2 * i < rot // 2, f, f / 4.0)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 1009 + 17)
    gc = torch.Generator().manual_seed(int(seed) * 7919 + 5)

    def randn(*shape, std=1.0, dtype=torch.float32):
        out = torch.empty(shape, device=DEV, dtype=dtype)
        flat, n = out.view(-1), 1 << 26
        for o in range(0, flat.numel(), n):  # bounds the fp32 scratch
            part = torch.randn(min(n, flat.numel() - o), generator=g, device=DEV)
            flat[o:o + n] = part * std
        return out

    op = case["op"]
    st = {"case": case, "op": op}
    if op == "pages":
        return _prepare_pages(case, st, gc)
    d, dt = case["d"], _dtype(case)
    if op == "rope":
        N, Hq, Hkv = case["N"], case["Hq"], case["Hkv"]
        # q and k (and v, not touched) as the projection leaves them; a
        # gradient comes in tensors of its own
        if case["inverse"]:
            st["q"], st["k"] = randn(N, Hq, d, dtype=dt), randn(N, Hkv, d, dtype=dt)
        else:
            qkv = randn(N, Hq + 2 * Hkv, d, dtype=dt)
            st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        start = torch.randint(0, case["far"], (1,), generator=gc).item()
        # two requests: one that starts, one far into its text
        pos = torch.arange(N)
        pos = torch.where(pos < N // 2, pos, pos + start)
        st["positions"] = pos.to(torch.int32).to(DEV)
        st["inv_freq"] = _inv_freq(case["rot"]).to(DEV)
        st["scale"] = 0.1 * math.log(4.0) + 1.0
        return st
    if op == "prefill":
        lens = _lengths(case)
        N, Hq, Hkv = sum(lens), case["Hq"], case["Hkv"]
        qkv = randn(N, Hq + 2 * Hkv, d, dtype=dt)
        st["q"], st["k"], st["v"] = qkv.split([Hq, Hkv, Hkv], 1)
        st["mem"] = randn(N, Hq, d, std=0.1, dtype=dt)
        st["w_count"] = randn(Hq, d, std=0.02)
        st["cu"] = torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32,
                                device=DEV)
        return st
    if op == "store":
        N, Hkv, page = case["N"], case["Hkv"], case["page"]
        kv = randn(N, 2 * Hkv, d, dtype=dt)
        # channels differ in size, as those of trained keys do
        kv.mul_(torch.exp(0.5 * randn(2 * Hkv, d)).to(dt))
        st["k"], st["v"] = kv.split([Hkv, Hkv], 1)
        pool = (N + page - 1) // page + 3
        slots = torch.randperm(pool, generator=gc)[:, None] * page + torch.arange(page)[None, :]
        st["slots"] = slots.reshape(-1)[:N].to(torch.int32).to(DEV)
        st["k_pages"] = torch.zeros((pool, Hkv, page, 9 * d // 16), dtype=torch.uint8, device=DEV)
        st["v_pages"] = torch.zeros_like(st["k_pages"])
        return st
    B, Hq, Hkv, page = case["B"], case["Hq"], case["Hkv"], case["page"]
    lens = _lengths(case)
    npg = [(n + page - 1) // page for n in lens]
    table = torch.zeros((B, max(npg)), dtype=torch.int32)
    perm = torch.randperm(sum(npg), generator=gc).to(torch.int32)
    for b, n in enumerate(npg):
        table[b, :n] = perm[sum(npg[:b]):sum(npg[:b]) + n]
    st["table"] = table.to(DEV)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for name in ("k_pages", "v_pages"):
        pages = torch.empty((sum(npg), Hkv, page, 9 * d // 16), dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 26) // (Hkv * page * d))
        for o in range(0, sum(npg), step):
            pages[o:o + step] = _pack(*_quantise(randn(min(step, sum(npg) - o), Hkv, page, d)))
        st[name] = pages
    st["q"] = randn(B, Hq, d, dtype=dt)
    st["mem"] = randn(B, Hq, d, std=0.1, dtype=dt)
    st["w_count"] = randn(Hq, d, std=0.02)
    return st


def _prepare_pages(case, st, gc):
    B, T, page = case["B"], case["T"], case["page"]
    # spread evenly, in an order of the seed's: the buffers have one size
    order = [torch.randperm(B, generator=gc) for _ in range(3)]
    lens = (T * torch.arange(1, B + 1) // B)[order[0]]
    new = (1 + (case["new"] - 1) * torch.arange(1, B + 1) // B)[order[1]]
    ended = torch.arange(B)[order[2]] < int(case["ended"] * B)
    tokens = int(new.sum())
    new[ended] = 0
    have = (lens + page - 1) // page
    cols = int(((T + case["new"] + page - 1) // page))
    used = int(have.sum())
    # with too few pages left the last sequences get none
    pool = used + (tokens // page * 3 // 5 if case["short"] else tokens // page + B)
    perm = torch.randperm(pool, generator=gc).to(torch.int32)
    table = torch.full((B, cols), -1, dtype=torch.int32)
    inside = torch.arange(cols)[None, :] < have[:, None]
    table[inside] = perm[:used]
    free = torch.full((max(pool, 1),), -1, dtype=torch.int32)
    free[:pool - used] = perm[used:]
    st["pool"], st["tokens"] = pool, tokens
    for name, x in (("table", table), ("lens", lens), ("keep", torch.where(ended, 0, lens)),
                    ("new", new), ("free", free), ("count", torch.tensor([pool - used]))):
        st[name] = x.to(torch.int32).to(DEV)
    st["lens2"], st["count2"] = torch.empty_like(st["lens"]), torch.empty_like(st["count"])
    return st


# ------------------------------------------------------------ plain forms --

def _quantise(x):
    """Codes n [..., d] and scales [..., d / 32] of rows x."""
    x = x.double().unflatten(-1, (-1, GROUP))
    s = (x.abs().amax(-1) / 7.0).to(torch.bfloat16)
    n = torch.round(x / s.double()[..., None])
    n = torch.where((s == 0)[..., None], torch.zeros_like(n), n).clamp(-7, 7)
    return n.flatten(-2).to(torch.int32), s


def _bits(at):
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def _pack(n, s):
    """Page blocks of codes and scales [..., page, :]."""
    n = n.unflatten(-1, (-1, 4))
    c = (((n < 0).int() << _bits(SIGN_AT)) + (n.abs() << _bits(SIZE_AT))).sum(-1)  # [..., d / 4]
    c = torch.stack([c & 255, c >> 8], -1).to(torch.uint8).flatten(-2)
    c = c.unflatten(-1, (-1, 4, 4)).transpose(-2, -3).flatten(-4)
    s = s.contiguous().view(torch.uint8).flatten(-2)
    return torch.cat([c, s], -1).unflatten(-1, (n.shape[-3], -1))


def _unpack(pages, d):
    """fp32 values [..., page, d] of page blocks."""
    page = pages.shape[-2]
    flat = pages.flatten(-2)
    c = flat[..., :page * d // 2].unflatten(-1, (page, 4, d // GROUP, 4))
    c = c.transpose(-2, -3).reshape(*flat.shape[:-1], page, -1, 2).int()
    c = (c[..., 0] + (c[..., 1] << 8))[..., None]
    n = ((c >> _bits(SIZE_AT)) & 7) * (1 - 2 * ((c >> _bits(SIGN_AT)) & 1))
    s = flat[..., page * d // 2:].contiguous().view(torch.bfloat16).float()
    s = s.unflatten(-1, (page, d // GROUP, 1))
    return (n.flatten(-2).float().unflatten(-1, (-1, GROUP)) * s).flatten(-2)


def _run_pages(st):
    page, tokens = st["case"]["page"], st["tokens"]
    table, free, lens, keep, new = (st[n].long() for n in ("table", "free", "lens", "keep", "new"))
    count, B, cols = st["count"].long(), st["lens"].shape[0], st["table"].shape[1]
    col = torch.arange(cols, device=DEV)

    def pages(n):
        return (n + page - 1) // page

    # the pages past keep go back, sequence by sequence
    back = (col >= pages(keep)[:, None]) & (col < pages(lens)[:, None])
    given = table[back]
    free.scatter_(0, count + torch.arange(given.shape[0], device=DEV), given)
    count = count + given.shape[0]
    # the new tokens' pages come from the end of the stack, in order
    need = pages(keep + new) - pages(keep)
    before = need.cumsum(0) - need
    ok = (need == 0) | (before + need <= count)
    fresh = (col >= pages(keep)[:, None]) & (col < pages(keep + new)[:, None]) & ok[:, None]
    at = count - 1 - before[:, None] - (col - pages(keep)[:, None])
    table = torch.where(fresh, free[at.clamp(0, free.shape[0] - 1)], table)
    count = count - (need * ok).sum()
    after = keep + new * ok
    cu = torch.cat([torch.zeros_like(count), new.cumsum(0)])
    t = torch.arange(tokens, device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    p = keep[b] + t - cu[b]
    here = (t < cu[-1]) & ok[b]
    slot = table[b, (p // page).clamp(max=cols - 1)] * page + p % page
    out = {"table": table, "free": free, "count": count, "lens": after, "cu": cu,
           "positions": torch.where(here, p, torch.zeros_like(p)),
           "slots": torch.where(here, slot, torch.full_like(slot, -1))}
    return {n: x.to(torch.int32) for n, x in out.items()}


def _run_rope(st):
    rot = st["case"]["rot"]
    angle = st["positions"].double()[:, None] * st["inv_freq"]
    sign = -1.0 if st["case"]["inverse"] else 1.0
    cos = (st["scale"] * torch.cos(angle)).float()[:, None]
    sin = (sign * st["scale"] * torch.sin(angle)).float()[:, None]

    def turn(x):
        y = x.float().clone()
        if st["case"]["interleaved"]:
            a, b = x[..., :rot:2].float(), x[..., 1:rot:2].float()
            y[..., :rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :rot // 2].float(), x[..., rot // 2:rot].float()
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        return y.to(x.dtype)

    return {"q": turn(st["q"]), "k": turn(st["k"])}


def _polar(s, tau, n, v, q_norm, w_count, mem):
    """out, n_eff, conf from masked logits s [..., keys] (natural units)."""
    d = v.shape[-1]
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    p = p / l
    lse = m + torch.log(l)
    n_eff = 1.0 / (p * p).sum(-1, keepdim=True)
    floor = tau * q_norm * d ** -0.5 * torch.sqrt(2.0 * torch.log(n))
    conf = 1.0 / (1.0 + torch.exp(floor - lse))
    a = p @ v
    u = a / a.square().sum(-1, keepdim=True).sqrt().clamp(min=1e-6)
    count = conf * torch.tanh(torch.log(n_eff) / LOG_T0)
    return u + count * w_count + mem, n_eff[..., 0], conf[..., 0]


def _run_prefill(st):
    q, k, v, mem, cu = (st[n] for n in ("q", "k", "v", "mem", "cu"))
    N, Hq, d = q.shape
    Hkv = k.shape[1]
    G, lens = Hq // Hkv, (cu[1:] - cu[:-1]).long()
    B, T = lens.shape[0], st["case"]["T"]
    t = torch.arange(T, device=DEV)
    rows = (cu[:-1].long()[:, None] + t).clamp(max=N - 1)  # [B, T], those past an end unused

    def batch(x, r):  # [N, Hkv * n, d] -> [B, Hkv, n * rows, d]
        x = x[r].float().unflatten(2, (Hkv, -1))
        return x.permute(0, 2, 3, 1, 4).flatten(2, 3)

    there = (t < lens[:, None])[:, None, :, None]
    kb = batch(k, rows).transpose(-1, -2)
    vb = torch.where(there, batch(v, rows), torch.zeros((), device=DEV))
    out = torch.empty((N, Hq, d), device=DEV)
    n_eff, conf = torch.empty((N, Hq), device=DEV), torch.empty((N, Hq), device=DEV)
    step = max(1, (1 << 31) // (B * Hq * T))
    for o in range(0, T, step):  # bounds the scores held at once
        r = rows[:, o:o + step]
        n = (t[o:o + step] + 1).float().repeat(G)[:, None]
        tau = (torch.log(n) / LOG_T0).clamp(min=1.0)
        qb = batch(q, r)
        s = tau * d ** -0.5 * (qb @ kb)
        s = s.masked_fill(t[None, :] >= n, -math.inf)
        w = st["w_count"].view(Hkv, G, 1, d).expand(Hkv, G, r.shape[1], d).flatten(1, 2)
        y = _polar(s, tau, n, vb, qb.square().sum(-1, keepdim=True).sqrt(), w, batch(mem, r))
        live = (t[o:o + step] < lens[:, None])
        for dst, x in zip((out, n_eff, conf), y):
            x = x.unflatten(2, (G, -1)).movedim(3, 1).flatten(2, 3)  # [B, rows, Hq, ...]
            dst[r[live]] = x[live]
    return {"out": out.to(q.dtype), "n_eff": n_eff, "conf": conf}


def _run_store(st):
    page, d = st["case"]["page"], st["case"]["d"]
    slots = st["slots"].long()
    out = {}
    for name in ("k", "v"):
        n, s = _quantise(st[name])
        pool = st[name + "_pages"]
        # the rows' bytes, where the block's layout has them
        row = _pack(n[:, :, None], s[:, :, None])[:, :, 0]  # [N, Hkv, 9 d / 16]
        flat = pool.flatten(2)
        codes = flat[..., :page * d // 2].unflatten(-1, (page, -1))
        scales = flat[..., page * d // 2:].unflatten(-1, (page, -1))
        codes[slots // page, :, slots % page] = row[..., :d // 2]
        scales[slots // page, :, slots % page] = row[..., d // 2:]
        out[name] = _unpack(pool, d)[slots // page, :, slots % page]
    return out


def _run_decode(st):
    q, table = st["q"].float(), st["table"].long()
    B, Hq, d = q.shape
    Hkv = st["k_pages"].shape[1]
    G = Hq // Hkv

    def gather(pages):
        return _unpack(pages, d)[table].transpose(1, 2).flatten(2, 3)  # [B, Hkv, rows, d]

    n = st["lens"].float()[:, None, None, None]
    tau = (torch.log(n) / LOG_T0).clamp(min=1.0)
    q = q.view(B, Hkv, G, d)
    s = tau * d ** -0.5 * (q @ gather(st["k_pages"]).transpose(-1, -2))
    s = s.masked_fill(torch.arange(s.shape[-1], device=DEV) >= n, -math.inf)
    w, mem = st["w_count"].view(Hkv, G, d), st["mem"].float().view(B, Hkv, G, d)
    out, n_eff, conf = _polar(s, tau, n, gather(st["v_pages"]),
                              q.square().sum(-1, keepdim=True).sqrt(), w, mem)
    return {"out": out.view(B, Hq, d).to(st["q"].dtype), "n_eff": n_eff.reshape(B, Hq),
            "conf": conf.reshape(B, Hq)}


# -------------------------------------------------------- library's calls --

def _own(st):
    import long_context_attention_causal_gb300 as pa
    op, case = st["op"], st["case"]
    if op == "pages":
        pa.pages_release(st["table"], st["lens"], st["keep"], st["free"], st["count"],
                         case["page"], num_pages=st["pool"], lens_out=st["lens2"],
                         count_out=st["count2"])
        cu, pos, slots = pa.pages_extend(st["table"], st["lens2"], st["new"], st["free"],
                                         st["count2"], case["page"], st["tokens"],
                                         num_pages=st["pool"])
        return {"table": st["table"], "free": st["free"], "count": st["count2"],
                "lens": st["lens2"], "cu": cu, "positions": pos, "slots": slots}
    if op == "rope":
        q, k = pa.rope(st["q"], st["k"], st["positions"], st["inv_freq"], scale=st["scale"],
                       interleaved=case["interleaved"], inverse=case["inverse"])
        return {"q": q, "k": k}
    if op == "prefill":
        out, n_eff, conf = pa.fwd_packed(st["q"], st["k"], st["v"], st["mem"], st["w_count"],
                                         st["cu"], want_conf=True)
        return {"out": out, "n_eff": n_eff, "conf": conf}
    if op == "store":
        pa.cache_append_q4(st["k"], st["v"], st["slots"], st["k_pages"], st["v_pages"])
        k, v = pa.cache_read_q4(st["k_pages"], st["v_pages"], st["slots"], dtype=torch.float32)
        return {"k": k, "v": v}
    out, n_eff, conf = pa.decode_paged_q4(
        st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"], st["mem"], st["w_count"],
        max_seq_len=max(_lengths(case)), want_conf=True)
    return {"out": out, "n_eff": n_eff, "conf": conf}


def run(state):
    if own:
        return _own(state)
    return {"pages": _run_pages, "rope": _run_rope, "prefill": _run_prefill, "store": _run_store,
            "decode": _run_decode}[state["op"]](state)


# ------------------------------------------------------------------- work --

def work(case):
    op = case["op"]
    if op == "pages":
        # lengths and prefix sums, a page's number twice, a token's two numbers
        tokens = case["B"] * (case["new"] + 1) / 2.0
        gone = case["ended"] * case["B"] * case["T"] / 2.0
        return {"bytes": 20.0 * case["B"] + 8.0 * (tokens + gone) / case["page"] + 8.0 * tokens,
                "flops": 0.0}
    d, es = case["d"], 4 if case["dtype"] == "f32" else 2
    if op == "rope":
        rows = float(case["N"]) * (case["Hq"] + case["Hkv"])
        return {"bytes": 2.0 * rows * d * es + 4.0 * case["N"], "flops": 3.0 * rows * case["rot"]}
    row = 9.0 * d / 16
    if op == "store":
        rows = 2.0 * case["N"] * case["Hkv"]
        return {"bytes": rows * (d * es + 2 * row + 4 * d) + 8.0 * case["N"], "flops": 4.0 * rows * d}
    lens, Hq, Hkv = _lengths(case), case["Hq"], case["Hkv"]
    if op == "prefill":
        pairs = sum(n * (n + 1) / 2 for n in lens)
        return {"bytes": sum(lens) * ((3.0 * Hq + 2 * Hkv) * d * es + 8.0 * Hq),
                "flops": 4.0 * pairs * Hq * d}
    return {"bytes": sum(lens) * Hkv * 2 * row + case["B"] * Hq * (3.0 * d * es + 8),
            "flops": 4.0 * sum(lens) * Hq * d}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    """The definitions, sequence by sequence, in 64 bits."""
    st = prepare(case, seed)
    return {"pages": _exact_pages, "rope": _exact_rope, "prefill": _exact_prefill,
            "store": _exact_store, "decode": _exact_decode}[case["op"]](st, case)


def _exact_pages(st, case):
    page = case["page"]
    table, free, lens = (st[n].tolist() for n in ("table", "free", "lens"))
    keep, new, top = st["keep"].tolist(), st["new"].tolist(), st["count"].item()
    for b, n in enumerate(lens):
        for j in range(-(-keep[b] // page), -(-n // page)):
            free[top] = table[b][j]
            top += 1
    bottom, cu, pos, slots, after = top, [0], [], [], []
    for b, n in enumerate(keep):
        first, last = -(-n // page), -(-(n + new[b]) // page)
        cu.append(cu[-1] + new[b])
        ok = last == first or top - (last - first) >= 0
        for j in range(first, last):
            top -= 1
            if ok:
                table[b][j] = free[top]
                bottom -= 1
        after.append(n + new[b] if ok else n)
        for t in range(n, n + new[b]):
            pos.append(t if ok else 0)
            slots.append(table[b][t // page] * page + t % page if ok else -1)
    pad = st["tokens"] - len(pos)
    out = {"table": table, "free": free, "count": [bottom], "lens": after, "cu": cu,
           "positions": pos + [0] * pad, "slots": slots + [-1] * pad}
    return {n: torch.tensor(x, dtype=torch.int32, device=DEV) for n, x in out.items()}


def _exact_rope(st, case):
    rot = case["rot"]
    f = st["inv_freq"] * (-1 if case["inverse"] else 1)
    turn = torch.polar(torch.full((), st["scale"], dtype=torch.float64, device=DEV),
                       st["positions"].double()[:, None, None] * f)
    out = {}
    for name in ("q", "k"):
        x = st[name].double()
        if case["interleaved"]:
            z = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous())
            z = torch.view_as_real(z * turn).flatten(-2)
        else:
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
            z = torch.cat([z.real, z.imag], -1)
        out[name] = torch.cat([z, x[..., rot:]], -1)
    return out


def _exact_attention(q, k, v, first, w_count, mem):
    """q, mem [h, m, d], the rows first, first + 1, ... of k, v [h, n, d]."""
    h, m, d = q.shape
    n = torch.arange(first + 1, first + m + 1, device=DEV, dtype=torch.float64)
    tau = torch.clamp(n.log() / LOG_T0, min=1.0)
    s = torch.einsum("hmd,hnd->hmn", q, k) * (tau / math.sqrt(d))[None, :, None]
    s = s + torch.full((m, k.shape[1]), -math.inf, device=DEV, dtype=torch.float64).triu(first + 1)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    n_eff = 1.0 / p.square().sum(-1)
    norm = torch.linalg.vector_norm(q, dim=-1)
    conf = torch.sigmoid(lse - tau * norm / math.sqrt(d) * torch.sqrt(2 * n.log()))
    a = torch.einsum("hmn,hnd->hmd", p, v)
    a = a / torch.linalg.vector_norm(a, dim=-1, keepdim=True).clamp(min=1e-6)
    gate = conf * torch.tanh(torch.log(n_eff) / LOG_T0)
    return a + gate[..., None] * w_count[:, None] + mem, n_eff, conf


def _exact_prefill(st, case):
    Hq, G = case["Hq"], case["Hq"] // case["Hkv"]
    out = {"out": torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)}
    for name in ("n_eff", "conf"):
        out[name] = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device=DEV)
    at, w = 0, st["w_count"].double()
    for n in _lengths(case):
        q, k, v, mem = (st[x][at:at + n].transpose(0, 1) for x in ("q", "k", "v", "mem"))
        for h in range(0, Hq, G):
            kh, vh = (x[h // G].double().expand(G, n, -1) for x in (k, v))
            step = 2048
            for o in range(0, n, step):
                e = min(n, o + step)
                y = _exact_attention(q[h:h + G, o:e].double(), kh[:, :e], vh[:, :e], o, w[h:h + G],
                                     mem[h:h + G, o:e].double())
                for name, x in zip(("out", "n_eff", "conf"), y):
                    out[name][at + o:at + e, h:h + G] = x.transpose(0, 1)
        at += n
    return out


def _exact_store(st, case):
    out = {}
    for name in ("k", "v"):
        x = st[name].double().unflatten(-1, (-1, GROUP))
        s = (x.abs().amax(-1, keepdim=True) / 7.0).to(torch.bfloat16).double()
        s_or_1 = torch.where(s == 0, torch.ones_like(s), s)
        out[name] = (s * torch.round(x / s_or_1).clamp(-7, 7)).flatten(-2)
    return out


def _exact_values(pages, d):
    """Rows [heads, rows, d] of page blocks, by each channel's place in them."""
    P, H, page, _ = pages.shape
    raw = pages.reshape(P, H, -1)
    row, ch = torch.arange(page, device=DEV)[:, None], torch.arange(d, device=DEV)[None, :]
    word = (ch // 8) % 4 * (d // 32) + ch // 32
    at = row * (d // 2) + 4 * word + 2 * (ch // 4 % 2)
    code = raw[:, :, at].int() + 256 * raw[:, :, at + 1].int()
    sign = torch.where((code << (4 * (ch % 4)).int()) & 0x8000 != 0, -1, 1)
    n = sign * torch.where(ch % 4 < 2, code << (4 * (ch % 4)).int() >> 4, code >> (20 - 4 * (ch % 4)).int()).bitwise_and(7)
    lo = page * (d // 2) + 2 * (row * (d // 32) + ch // 32)
    bits = raw[:, :, lo].int() + 256 * raw[:, :, lo + 1].int()
    s = (bits << 16).view(torch.float32).double()
    return (s * n.double()).transpose(0, 1).reshape(H, P * page, d)


def _exact_decode(st, case):
    Hq, Hkv, d, page = (case[n] for n in ("Hq", "Hkv", "d", "page"))
    got = []
    for b, n in enumerate(_lengths(case)):
        ids = st["table"][b, :-(-n // page)].long()
        k, v = (_exact_values(st[x][ids], d)[:, :n].repeat_interleave(Hq // Hkv, 0)
                for x in ("k_pages", "v_pages"))
        y = _exact_attention(st["q"][b].double()[:, None], k, v, n - 1, st["w_count"].double(),
                             st["mem"][b].double()[:, None])
        got.append([x[:, 0] for x in y])
    return {name: torch.stack([y[i] for y in got]) for i, name in enumerate(("out", "n_eff", "conf"))}

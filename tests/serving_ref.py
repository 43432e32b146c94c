"""References of the operators between requests and tokens (imported by test
files only): page bookkeeping in Python, rotary positions, 4-bit rounding and
Polar rows in fp64."""
import math

import torch

LOG_T0 = math.log(2048.0)


# ------------------------------------------------------------------ pages --

def extend_ref(table, lens, new, free, count, page, max_tokens, num_pages):
    """(table, lens, count, cu, positions, slots) after pages_extend; lists."""
    table = [list(r) for r in table]
    cols = len(table[0]) if table else 0
    cu, pos, slots, after = [0], [], [], []
    run, taken, tokens = 0, 0, 0
    count0 = min(max(count, 0), len(free))
    for b, n in enumerate(lens):
        add = new[b]
        bad = n < 0 or n > cols * page or add < 0
        add = 0 if bad else add
        tokens += add
        fits = not bad and n + add <= cols * page and tokens <= max_tokens
        need = -(-(n + add) // page) - -(-n // page) if fits else 0
        ok = fits and (need == 0 or run + need <= count0)
        if ok:
            for i in range(need):
                table[b][-(-n // page) + i] = free[count0 - 1 - run - i]
            taken += need
        run += need
        after.append(n + add if ok else n)
        cu.append(min(tokens, max_tokens))
        for t in range(n, n + add):
            pid = table[b][t // page] if ok else -1
            pos.append(t if ok else 0)
            slots.append(pid * page + t % page if ok and 0 <= pid < num_pages else -1)
    pos, slots = pos[:max_tokens], slots[:max_tokens]
    pad = max_tokens - len(pos)
    return table, after, count0 - taken, cu, pos + [0] * pad, slots + [-1] * pad


def release_ref(table, lens, keep, free, count, page, num_pages):
    """(free, lens, count) after pages_release; lists."""
    free, after = list(free), []
    cols = len(table[0]) if table else 0
    top = min(max(count, 0), len(free))
    for b, n in enumerate(lens):
        bad = n < 0 or n > cols * page or keep[b] < 0 or keep[b] > n
        k = n if bad else keep[b]
        after.append(k)
        if bad:
            continue
        for j in range(-(-k // page), -(-n // page)):
            if top < len(free):
                free[top] = table[b][j] if 0 <= table[b][j] < num_pages else -1
            top += 1
    return free, after, min(top, len(free))


# ------------------------------------------------------------------- rope --

def rope_ref(x, positions, inv_freq, scale=1.0, interleaved=False, inverse=False):
    """fp64 rotation of [N, heads, d]."""
    rot = 2 * inv_freq.shape[0]
    a = positions.double()[:, None, None] * inv_freq.double()
    c, s = scale * torch.cos(a), scale * torch.sin(a) * (-1.0 if inverse else 1.0)
    y = x.double().clone()
    if interleaved:
        p, q = x[..., :rot:2].double(), x[..., 1:rot:2].double()
        y[..., :rot:2], y[..., 1:rot:2] = p * c - q * s, q * c + p * s
    else:
        p, q = x[..., :rot // 2].double(), x[..., rot // 2:rot].double()
        y[..., :rot // 2], y[..., rot // 2:rot] = p * c - q * s, q * c + p * s
    return y


# ------------------------------------------------------------------ 4 bit --

def q4_ref(x):
    """What rows [..., d] are held as, fp64: s n per group of 32 channels."""
    g = x.double().unflatten(-1, (-1, 32))
    top = g.abs().amax(-1, keepdim=True)
    s = (top / 7.0).float().to(torch.bfloat16).double()
    n = torch.where(s == 0, torch.zeros_like(g), torch.round(g / s)).clamp(-7, 7)
    out = torch.where(torch.isfinite(top), s * n, torch.full_like(g, math.nan))
    return out.flatten(-2)


# ------------------------------------------------------------------ polar --

def polar_ref(q, k, v, first, w, mem):
    """fp64 (out, n_eff, conf): q, mem [h, m, d] at positions first, first + 1,
    ... over k, v [h, n, d] with causal visibility; w [h, d]."""
    h, m, d = q.shape
    q, k, v, mem, w = (t.double() for t in (q, k, v, mem, w))
    n = torch.arange(first + 1, first + m + 1, device=q.device, dtype=torch.float64)
    tau = (n.log() / LOG_T0).clamp(min=1.0)
    s = torch.einsum("hmd,hnd->hmn", q, k) * (tau / math.sqrt(d))[None, :, None]
    seen = torch.arange(k.shape[1], device=q.device)[None, :] < n[:, None]
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    n_eff = 1.0 / p.square().sum(-1)
    conf = torch.sigmoid(lse - tau * torch.linalg.vector_norm(q, dim=-1) / math.sqrt(d)
                         * torch.sqrt(2 * n.log()))
    a = torch.einsum("hmn,hnd->hmd", p, v)
    a = a / torch.linalg.vector_norm(a, dim=-1, keepdim=True).clamp(min=1e-6)
    gate = conf * torch.tanh(torch.log(n_eff) / LOG_T0)
    return a + gate[..., None] * w[:, None] + mem, n_eff, conf


def packed_ref(q, k, v, mem, w, cu, b):
    """polar_ref of sequence b of packed tensors: out [n, Hq, d], n_eff, conf [n, Hq]."""
    lo, hi = int(cu[b]), int(cu[b + 1])
    G = q.shape[1] // k.shape[1]
    t = lambda x: x[lo:hi].transpose(0, 1)  # noqa: E731
    o, ne, c = polar_ref(t(q), t(k).repeat_interleave(G, 0), t(v).repeat_interleave(G, 0), 0, w,
                         t(mem))
    return o.transpose(0, 1), ne.t(), c.t()


def decode_ref(q, k, v, w, mem):
    """One query token q, mem [Hq, d] over k, v [Hkv, n, d]: out [Hq, d], n_eff, conf [Hq]."""
    G, n = q.shape[0] // k.shape[0], k.shape[1]
    o, ne, c = polar_ref(q[:, None], k.repeat_interleave(G, 0), v.repeat_interleave(G, 0), n - 1, w,
                         mem[:, None])
    return o[:, 0], ne[:, 0], c[:, 0]

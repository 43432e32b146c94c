"""fp64 references of the decayed linear attention and of the cache eviction
(imported by test files only): the definitions, token by token and row by
row, in plain torch on the CPU or the device of the inputs."""
import numpy as np
import torch


def _prep(log_decay, lengths, B, T, dev):
    g = torch.exp(torch.as_tensor(log_decay, device=dev).double())
    lens = [T] * B if lengths is None else [int(n) for n in lengths]
    return g, lens


def linear_fwd_ref(q, k, v, log_decay, scale, state=None, lengths=None):
    """(mem, state) in fp64; q, k, v [B, H, T, d]."""
    B, H, T, d = q.shape
    dev = q.device
    g, lens = _prep(log_decay, lengths, B, T, dev)
    mem = torch.zeros((B, H, T, d), dtype=torch.float64, device=dev)
    S = (torch.zeros((B, H, d, d), dtype=torch.float64, device=dev) if state is None
         else state.double().clone())
    for b in range(B):
        n = lens[b]
        qb, kb, vb = q[b, :, :n].double(), k[b, :, :n].double(), v[b, :, :n].double()
        for t in range(n):
            S[b] = g[:, None, None] * S[b] + vb[:, t, :, None] * kb[:, t, None, :]
            mem[b, :, t] = scale * (S[b] @ qb[:, t, :, None])[..., 0]
    return mem, S


def linear_bwd_ref(q, k, v, log_decay, scale, dmem, state=None, dstate_out=None, lengths=None):
    """(dq, dk, dv, dstate) in fp64."""
    B, H, T, d = q.shape
    dev = q.device
    g, lens = _prep(log_decay, lengths, B, T, dev)
    dq, dk, dv = (torch.zeros((B, H, T, d), dtype=torch.float64, device=dev) for _ in range(3))
    R = (torch.zeros((B, H, d, d), dtype=torch.float64, device=dev) if dstate_out is None
         else dstate_out.double().clone())
    for b in range(B):
        n = lens[b]
        qb, kb, vb, db = (x[b, :, :n].double() for x in (q, k, v, dmem))
        S = (torch.zeros((H, d, d), dtype=torch.float64, device=dev) if state is None
             else state[b].double().clone())
        for t in range(n):
            S = g[:, None, None] * S + vb[:, t, :, None] * kb[:, t, None, :]
            dq[b, :, t] = scale * (S.transpose(1, 2) @ db[:, t, :, None])[..., 0]
        for t in range(n - 1, -1, -1):
            R[b] = R[b] + scale * db[:, t, :, None] * qb[:, t, None, :]
            dk[b, :, t] = (R[b].transpose(1, 2) @ vb[:, t, :, None])[..., 0]
            dv[b, :, t] = (R[b] @ kb[:, t, :, None])[..., 0]
            R[b] = g[:, None, None] * R[b]
    return dq, dk, dv, R


def evict_ref(lens, weights, positions, keep, recent):
    """Per (b, h): the list of (from, to) moves, in order; numpy, row by row."""
    B, Hkv, _ = weights.shape
    moves = {}
    for b in range(B):
        n = int(lens[b])
        for h in range(Hkv):
            if n <= keep:
                moves[b, h] = []
                continue
            w = weights[b, h, :n].astype(np.float64)
            p = positions[b, h, :n].astype(np.int64)
            newest = p.max()

            def rank(j):
                # larger weight first, NaN last, lower row first
                return (np.isnan(w[j]), -w[j] if not np.isnan(w[j]) else 0.0, j)

            guarded = [j for j in range(n) if p[j] > newest - recent]
            rest = sorted((j for j in range(n) if not p[j] > newest - recent), key=rank)
            kept = set((guarded + rest)[:keep])
            holes = [j for j in range(keep) if j not in kept]
            movers = [j for j in range(keep, n) if j in kept]
            assert len(holes) == len(movers)
            moves[b, h] = list(zip(movers, holes))
    return moves

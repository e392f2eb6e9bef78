"""Plain 64-bit implementations of the calls for bounded caches, and the error bounds that their
results are held to (roundings as in spec_reference)."""
from __future__ import annotations

import math

import torch

from tests.spec_reference import U32, values


def visible(pos, n, window, first):
    """bool [tokens, n]: the keys that tokens at `pos` see."""
    j = torch.arange(n)
    p = pos.cpu().long()[:, None]
    see = j <= p
    if window > 0:
        see &= (j > p - window) | (j < first)
    return see


def window_attention(q, kb, vb, qsl, lens, positions, tables, scale, window=0, first=0, sinks=None,
                     k_scales=None, v_scales=None, weight_u=2.0 ** -16, q_u=0.0, weight_min=0.0,
                     observed=0, weights_len=0):
    """A dict of out [T, H, D], lse [H, T] and key weights [S, Hkv, weights_len] in 64 bits and
    their bounds (of out before its own rounding).

    weight_u, q_u, weight_min: as in spec_reference.tree_attention."""
    T, H, D = q.shape
    NB, bs, Hkv, _ = kb.shape
    G, S = H // Hkv, lens.numel()
    qd, kd, vd = values(q), values(kb).view(NB * bs, Hkv, D), values(vb).view(NB * bs, Hkv, D)
    ks = torch.ones(Hkv, dtype=torch.float64) if k_scales is None else values(k_scales)
    vs = torch.ones(Hkv, dtype=torch.float64) if v_scales is None else values(v_scales)
    out = torch.zeros(T, H, D, dtype=torch.float64)
    lse = torch.full((H, T), -math.inf, dtype=torch.float64)
    W = torch.zeros(S, Hkv, weights_len, dtype=torch.float64)
    out_b, lse_b, W_b = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(W)
    qsl, lens = qsl.cpu().tolist(), lens.cpu().tolist()
    pos, tables = positions.cpu().long(), tables.cpu().long()
    for s, L in enumerate(lens):
        a, b = qsl[s], qsl[s + 1]
        if a == b:
            continue
        see = visible(pos[a:b], L, window, first)
        used = see.any(0).nonzero()[:, 0]  # (entries of the others' blocks may be anything)
        see = see[:, used]
        slots = tables[s, used // bs] * bs + used % bs
        counted = 0 if observed == 0 else max(0, b - a - observed)
        for h in range(H):
            g = h // G
            K, V = kd[slots, g] * ks[g], vd[slots, g] * vs[g]
            x = (qd[a:b, h] @ torch.nan_to_num(K).t()) * scale
            # an fp32 dot product of D terms: (D + 2) u of the terms' magnitudes, scale included
            d = (qd[a:b, h].abs() @ torch.nan_to_num(K).abs().t()) * abs(scale) * (D + 4) * U32
            if q_u:
                d = d + q_u * qd[a:b, h].abs().amax(1, keepdim=True) * \
                    torch.nan_to_num(K).abs().sum(1) * abs(scale)
            dm = torch.where(see, d, 0.0).amax(1, keepdim=True)
            x = torch.where(see, x, -math.inf)
            y = x if sinks is None else torch.cat([x, values(sinks)[h].expand(b - a, 1)], 1)
            m = y.amax(1, keepdim=True)
            m = torch.where(m == -math.inf, 0.0, m)
            l = (y - m).exp().sum(1, keepdim=True)
            p = torch.where(l > 0, (x - m).exp() / l.clamp_min(1e-300), 0.0)
            Vn = torch.nan_to_num(V)
            out[a:b, h] = p @ Vn
            lse[h, a:b] = torch.where(l > 0, m + l.log(), -math.inf)[:, 0]
            n = used.numel()
            # as in spec_reference.tree_attention
            big = torch.where(see, x.abs(), 0.0).amax(1, keepdim=True) + m.abs()
            e = 4 * dm + 4 * big * U32 + 2.0 ** -20 + weight_u + 2 * n * U32
            out_b[a:b, h] = (p @ Vn.abs()) * e + weight_min * (see.double() @ Vn.abs())
            lb = 2 * dm + 4 * big * U32 + 2.0 ** -20 + n * U32
            lb = lb + 4 * U32 * torch.nan_to_num(lse[h, a:b, None], neginf=0.0).abs()
            lse_b[h, a:b] = lb[:, 0]
            if weights_len:
                pc = p[counted:]
                W[s, g, used] += pc.sum(0)
                # a weight: the score's error, the lse's, the argument's rounding, the exponential
                ew = dm + lb + 4 * big * U32 + 2.0 ** -20
                W_b[s, g, used] += (pc * ew[counted:]).sum(0)
        if weights_len:  # fp32 sums over all rows
            W_b[s] += W[s] * ((b - a) * G + 2) * U32
    return {"out": out, "lse": lse, "weights": W, "out_b": out_b, "lse_b": lse_b, "weights_b": W_b}


def evict(rows, weights, lens, new_lens, first, recent):
    """rows: a list (over sequences) of lists (over kv heads) of lists of anything, one entry to a
    key; weights [S][Hkv][n] of floats or None.  Both are changed as pa_evict_keys does."""
    for s, (n, new) in enumerate(zip(lens, new_lens)):
        if new >= n:
            continue
        f = min(first, new)
        r = min(recent, new - f)
        for g in range(len(rows[s])):
            w = weights[s][g] if weights is not None else [0.0] * n
            size = lambda i: (1, 0.0) if math.isnan(w[i]) else (0, w[i])
            order = sorted(range(f, n - r), key=lambda i: (tuple(-x for x in size(i)), i))
            kept = sorted(order[:new - f - r])
            stay = {i for i in kept if i < new - r}
            to = [i for i in range(f, new - r) if i not in stay] + list(range(new - r, new))
            frm = [i for i in kept if i >= new - r] + list(range(n - r, n))
            old, old_w = list(rows[s][g]), list(w)
            for a, b in zip(frm, to):
                rows[s][g][b] = old[a]
                if weights is not None:
                    w[b] = old_w[a]
            if weights is not None:
                w[new:n] = [0.0] * (n - new)


class Batch:
    """Inputs of an attention call over a permuted pool."""

    def __init__(self, seqs, H, Hkv, D, bs=16, src=torch.bfloat16, kv=torch.bfloat16, seed=0,
                 device="cuda", extra_blocks=3, spread=1.0):
        """seqs: (context, new tokens) of each sequence."""
        g = torch.Generator().manual_seed(seed)
        self.seqs = seqs
        lens = [c + n for c, n in seqs]
        need = [-(-n // bs) for n in lens]
        num = sum(need) + extra_blocks
        ids = torch.randperm(num, generator=g)
        width = max(max(need), 1) + 1
        tables = torch.full((len(seqs), width), -7, dtype=torch.int32)  # (unused entries: anything)
        at = 0
        for s, k in enumerate(need):
            tables[s, :k] = ids[at:at + k].int()
            at += k
        T = sum(n for _, n in seqs)

        def pool():
            x = torch.randn(num, bs, Hkv, D, generator=g) * spread
            return (x * 8).to(kv) if kv == torch.float8_e4m3fn else x.to(kv)

        self.q = torch.randn(T, H, D, generator=g).to(src).to(device)
        self.kb, self.vb = pool().to(device), pool().to(device)
        self.out = torch.full((T, H, D), 7.0, dtype=src, device=device)
        self.lse = torch.full((H, T), 7.0, device=device)
        self.qsl = torch.tensor([0] + [sum(n for _, n in seqs[:i + 1]) for i in range(len(seqs))],
                                dtype=torch.int32, device=device)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=device)
        pos = [torch.arange(c, c + n) for c, n in seqs]
        self.positions = torch.cat(pos).int().to(device) if T else torch.zeros(0, dtype=torch.int32,
                                                                               device=device)
        self.tables = tables.to(device)
        self.scale = 1.0 / math.sqrt(D)
        self.bs, self.H, self.Hkv, self.D, self.T = bs, H, Hkv, D, T

    def args(self):
        return (self.q, self.kb, self.vb, self.out, self.qsl, self.lens, self.positions, self.tables)

    def poison_unread(self, window, first):
        """Garbage in what the call must not look at: rows past the ends, keys that nobody sees
        (K) and the table entries of the blocks between the first tokens' and the window's."""
        bad_k, bad_v = [], []
        for s, (c, n) in enumerate(self.seqs):
            L = c + n
            row = self.tables[s].cpu()
            blocks = -(-L // self.bs)
            tail = [int(row[j // self.bs]) * self.bs + j % self.bs for j in range(L, blocks * self.bs)]
            bad_k += tail
            bad_v += tail
            if n == 0:
                self.tables[s] = -99
                continue
            pos = self.positions[int(self.qsl[s]):int(self.qsl[s + 1])].cpu()
            unseen = (~visible(pos, L, window, first).any(0)).nonzero()[:, 0]
            bad_k += (row.long()[unseen // self.bs] * self.bs + unseen % self.bs).tolist()
            if window > 0:
                front = -(-first // self.bs)
                lo = max(0, c - window + 1) // self.bs
                for b in range(front, lo):
                    self.tables[s, b] = 2 ** 30 if b % 2 else -5
        for pool, bad in ((self.kb, bad_k), (self.vb, bad_v)):
            rows = pool.view(-1, *pool.shape[2:])
            at = torch.tensor(bad, dtype=torch.long, device=pool.device)
            if pool.dtype == torch.float8_e4m3fn:
                rows.view(torch.uint8)[at] = 0x7F  # NaN
            else:
                rows[at] = float("nan")

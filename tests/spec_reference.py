"""Plain 64-bit implementations of the speculative-decoding calls, and the error bounds that
their results are held to.

Bounds.  A rounding to a type is off by at most half a step: u = eps / 2 relative (bf16 2^-8,
fp16 2^-11, fp32 2^-24, e4m3 2^-4, and half its smallest step, 2^-10, below its normal range)."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24
OUT_U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}
OUT_MIN = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float8_e4m3fn: 2.0 ** -10}


def values(t):
    """The values of a tensor of any type, in 64 bits on the CPU."""
    return t.detach().cpu().float().double()


def rotate(x, positions, inv_freq, interleaved, factor):
    """x [T, N, D] in 64 bits -> (rotated, bound on an fp32 evaluation's error)."""
    R = 2 * inv_freq.numel()
    y, err = x.clone(), torch.zeros_like(x)
    t = positions.cpu().double()[:, None] * inv_freq.cpu()
    c, s = (t.cos() * factor)[:, None], (t.sin() * factor)[:, None]
    ia = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    ib = ia + 1 if interleaved else ia + R // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    # the angle, in half turns, is off by 2^-25 from the conversion of 32 bits to fp32 (pi 2^-25
    # radians < 2^-23), sincospi by a few u, the factor's product, two products and a sum by
    # one u each: under 9 u of |a| + |b| in all
    e = 9 * U32 * abs(factor) * (a.abs() + b.abs())
    err[..., ia], err[..., ib] = e, e
    return y, err


def stored(y, err, dtype):
    """What a value y computed with error err may be after rounding to dtype: (value, bound)."""
    if dtype == torch.float8_e4m3fn:
        y = y.clamp(-448.0, 448.0)
    return y, err + (y.abs() + err) * OUT_U[dtype] + OUT_MIN[dtype]


def assert_within(got, want, bound, what=""):
    got = values(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(torch.isinf(got), torch.isinf(want)), f"{what}: infinities differ"
    fin = torch.isfinite(want)
    assert torch.isfinite(got[fin]).all(), f"{what}: not finite"
    assert torch.equal(got[~fin], want[~fin]), f"{what}: infinities differ"
    off = (got - want).abs()[fin] - bound.expand_as(want)[fin]
    assert off.numel() == 0 or float(off.max()) <= 0, (
        f"{what}: {int((off > 0).sum())} of {off.numel()} outside their bound, "
        f"by up to {float(off.max()):.3e}")


def unpack_mask(mask, nodes):
    """int32 [n, words] -> bool [n, nodes]."""
    bits = mask.cpu().to(torch.int64) & 0xFFFFFFFF
    j = torch.arange(nodes)
    return (bits[:, j // 32] >> (j % 32)) & 1 == 1


def tree_attention(q, kb, vb, qsl, lens, positions, mask, tables, scale, window=0, sinks=None,
                   k_scales=None, v_scales=None, weight_u=2.0 ** -16, q_u=0.0,
                   weight_min=0.0):
    """(out [T, H, D], lse [H, T], bound of out before its own rounding, bound of lse), 64 bits.

    k_scales, v_scales: per kv head (or None).  weight_u: the softmax weights' rounding where they
    enter the product with V (a bf16 pair 2^-16, f16 2^-11, fp32 less than either).  q_u: what q's
    elements may be off by, relative to their row's largest (0: q is used as it is; a pair of
    e4m3 terms 2^-17: half of e4m3's smallest step, 2^-10, where the largest is at least 2^7).
    weight_min: what a small weight is off by, relative to a sum of 1 (f16: half its smallest step,
    2^-25, where the row's largest weight is at least 2^7: 2^-32)."""
    T, H, D = q.shape
    NB, bs, Hkv, _ = kb.shape
    G = H // Hkv
    qd, kd, vd = values(q), values(kb).view(NB * bs, Hkv, D), values(vb).view(NB * bs, Hkv, D)
    ks = torch.ones(Hkv, dtype=torch.float64) if k_scales is None else values(k_scales)
    vs = torch.ones(Hkv, dtype=torch.float64) if v_scales is None else values(v_scales)
    out = torch.zeros(T, H, D, dtype=torch.float64)
    lse = torch.full((H, T), -math.inf, dtype=torch.float64)
    out_b, lse_b = torch.zeros_like(out), torch.zeros_like(lse)
    qsl, lens = qsl.cpu().tolist(), lens.cpu().tolist()
    pos, tables = positions.cpu().long(), tables.cpu().long()
    for s, L in enumerate(lens):
        a, b = qsl[s], qsl[s + 1]
        n = b - a
        if n == 0:
            continue
        ctx = L - n
        j = torch.arange(L)
        slots = tables[s, j // bs] * bs + j % bs
        see = torch.ones(n, L, dtype=torch.bool)
        see[:, ctx:] = unpack_mask(mask[a:b], n)
        key_pos = torch.cat([j[:ctx], pos[a:b]])
        if window > 0:
            see &= key_pos[None] > pos[a:b, None] - window
        for h in range(H):
            g = h // G
            K, V = kd[slots, g] * ks[g], vd[slots, g] * vs[g]
            x = (qd[a:b, h] @ K.t()) * scale
            # an fp32 dot product of D terms: (D + 2) u of the terms' magnitudes, scale included
            d = ((qd[a:b, h].abs() @ torch.nan_to_num(K).abs().t()) * abs(scale))
            d = torch.where(see, d, 0.0).amax(1, keepdim=True) * (D + 4) * U32
            if q_u:
                e = torch.where(see, torch.nan_to_num(K).abs().sum(1), 0.0).amax(1, keepdim=True)
                d = d + q_u * qd[a:b, h].abs().amax(1, keepdim=True) * e * abs(scale)
            x = torch.where(see, x, -math.inf)
            if sinks is not None:
                x = torch.cat([x, values(sinks)[h].expand(n, 1)], 1)
            m = x.amax(1, keepdim=True)
            m = torch.where(m == -math.inf, 0.0, m)
            p = (x - m).exp()
            l = p.sum(1, keepdim=True)
            p = torch.where(l > 0, p / l.clamp_min(1e-300), 0.0)[:, :L]
            Vn = torch.nan_to_num(V)
            out[a:b, h] = p @ Vn
            lse[h, a:b] = torch.where(l > 0, m + l.log(), -math.inf)[:, 0]
            # weights: twice the scores' error (numerator and sum), the exponential (2^-21 and
            # the scaled argument's rounding, |x| u each for score and maximum), their rounding
            # for the product, and fp32 sums over L keys
            big = torch.where(see, x[:, :L].abs(), 0.0).amax(1, keepdim=True) + m.abs()
            e = 4 * d + 4 * big * U32 + 2.0 ** -20 + weight_u + 2 * L * U32
            out_b[a:b, h] = (p @ Vn.abs()) * e + weight_min * (see.double() @ Vn.abs())
            lse_b[h, a:b] = (2 * d + 4 * big * U32 + 2.0 ** -20 + L * U32)[:, 0]
    lse_b += 4 * U32 * torch.nan_to_num(lse, neginf=0.0).abs()
    return out, lse, out_b, lse_b


def tree(rng, n, ctx, spread=6):
    """A random tree: parents, mask words [n, ceil(n / 32)] (ancestors and self), positions."""
    words = max(1, -(-n // 32))
    mask = [[0] * words for _ in range(n)]
    pos = [0] * n
    parents = []
    for i in range(n):
        p = rng.randrange(max(0, i - spread), i) if i else -1
        parents.append(p)
        if p >= 0:
            mask[i] = list(mask[p])
        pos[i] = pos[p] + 1 if p >= 0 else ctx
        mask[i][i // 32] |= 1 << (i % 32)
    return parents, mask, pos


def to_int32(words):
    return [[w - (1 << 32) if w >= 1 << 31 else w for w in row] for row in words]


class Pages:
    """The page bookkeeping in plain Python: the state and what each call makes of it."""

    def __init__(self, tables, lens, refs, free, block):
        self.tables = [list(r) for r in tables]
        self.lens, self.refs, self.free, self.block = list(lens), list(refs), list(free), block

    def _blocks(self, n):
        return -(-n // self.block)

    def fork(self, parents, children):
        pairs = []
        for p, c in zip(parents, children):
            n = self.lens[p]
            row = self.tables[p][:self._blocks(n)]
            pair = (-1, -1)
            if n % self.block:
                page = self.free.pop()
                pair = (row[-1], page)
                row[-1] = page
            for b in row:
                self.refs[b] += 1
            self.tables[c][:len(row)] = row
            pairs.append(pair)
        for p, c in zip(parents, children):
            self.lens[c] = self.lens[p]
        return pairs

    def grow(self, rows, new):
        for r, n in zip(rows, new):
            for i in range(self._blocks(self.lens[r]), self._blocks(n)):
                page = self.free.pop()
                self.refs[page] += 1
                self.tables[r][i] = page
            self.lens[r] = n

    def end(self, rows, new=None):
        gone = []
        for i, r in enumerate(rows):
            n = new[i] if new else 0
            for b in self.tables[r][self._blocks(n):self._blocks(self.lens[r])]:
                self.refs[b] -= 1
                if self.refs[b] == 0:
                    gone.append(b)
            self.lens[r] = n
        self.free += sorted(gone)

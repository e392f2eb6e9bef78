"""A K/V cache of bounded size: the cases its operators are measured on.

Long conversations either see only a window of the cache and its first tokens (window), or keep
in the cache what earlier queries looked at: every step adds up the attention weight that each
cached key receives (weigh), and now and then the keys with the least of it are evicted and the
rows that stay are moved together (evict).

``own`` False: the operators written out in elementary torch operations.  ``own`` True: the
calls a user makes of the library.
"""
import math
import zlib

import numpy as np
import torch

own = False

DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TYPES = {"bf16": BF16, "f32": F32, "e4m3": E4M3}
BLOCK = 16


def _attend(op, name=None, **c):
    """A batch of `chunks` sequences with chunk_lo to chunk_hi new tokens each and `decodes`
    with one, behind contexts of ctx_lo to ctx_hi cached tokens."""
    case = {"op": op, "chunks": 0, "chunk_lo": 0, "chunk_hi": 0, "decodes": 0, "ctx_lo": 0,
            "ctx_hi": 0, "heads": 32, "kv_heads": 8, "dim": 128, "window": 0, "first": 0,
            "observed": 0, "sinks": False, "lse": False, "src": "bf16", "kv": "bf16", **c}
    return {"name": name, **case} if name else case


def listed():
    return [
        # one user's long chat behind a window of 4096 and its first tokens: the smallest call
        _attend("window", "window_chat_1", decodes=1, ctx_lo=60001, ctx_hi=60001, window=4096,
                first=4),
        # a serving batch of 64 long chats
        _attend("window", "window_decode_64", decodes=64, ctx_lo=2048, ctx_hi=16384, window=4096,
                first=4),
        # continuous batching: prompt chunks beside decoding sequences
        _attend("window", "window_mixed", chunks=6, chunk_lo=257, chunk_hi=2048, decodes=58,
                ctx_lo=1000, ctx_hi=12000, window=4096, first=4),
        # e4m3 pools, a short window, learned sink logits and the log-sum-exp for a later merge
        _attend("window", "window_decode_48_e4m3", decodes=48, ctx_lo=1024, ctx_hi=8192,
                window=1024, first=17, sinks=True, lse=True, kv="e4m3"),
        # one user's chat over a cache held at about 2048 keys: latency counts
        _attend("weigh", "weigh_chat_1", decodes=1, ctx_lo=2047, ctx_hi=2047),
        # the 64-sequence serving batch (contexts 512 to 4096)
        _attend("weigh", "weigh_decode_64", decodes=64, ctx_lo=512, ctx_hi=4096),
        # a long prompt whose every query counts
        _attend("weigh", "weigh_prompt_8191", chunks=1, chunk_lo=8191, chunk_hi=8191),
        # ragged prompts of which the last 32 queries count, e4m3 pools
        _attend("weigh", "weigh_prompts_32_e4m3", chunks=5, chunk_lo=700, chunk_hi=4096,
                observed=32, kv="e4m3"),
        # a chat's cache, grown by one page, cut back to 1024 keys
        {"name": "evict_chat_1", "op": "evict", "seqs": 1, "len_lo": 1040, "len_hi": 1040,
         "keep": 0.9847, "first": 4, "recent": 64, "kv_heads": 8, "dim": 128, "block": 16,
         "kv": "bf16"},
        # long prompts cut to half before they decode
        {"name": "evict_64_half", "op": "evict", "seqs": 64, "len_lo": 2048, "len_hi": 8192,
         "keep": 0.5, "first": 4, "recent": 256, "kv_heads": 8, "dim": 128, "block": 16,
         "kv": "bf16"},
        # a large decoding batch held at about 1024 keys, half of them the most recent ones
        {"name": "evict_256_steady_e4m3", "op": "evict", "seqs": 256, "len_lo": 1030,
         "len_hi": 1060, "keep": 0.98, "first": 0, "recent": 512, "kv_heads": 8, "dim": 128,
         "block": 16, "kv": "e4m3"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "weigh", "weigh", "weigh", "evict", "evict"])
    if op == "evict":
        hi = _log(rng, 40, 16384)
        seqs = min(_log(rng, 1, 256), max(1, 300_000 // hi))
        lo = max(1, hi // rng.choice([1, 2, 4]))
        return {"op": op, "seqs": seqs, "len_lo": lo, "len_hi": hi,
                "keep": rng.choice([0.25, 0.5, 0.75, 0.97]), "first": rng.choice([0, 1, 4, 17]),
                "recent": rng.choice([0, 1, hi // 16, hi // 8]),
                "kv_heads": rng.choice([1, 4, 8]), "dim": rng.choice([64, 128, 128]),
                "block": rng.choice([16, 16, 32]), "kv": rng.choice(["bf16", "bf16", "e4m3", "f32"])}
    src, kv = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "e4m3"),
                          ("bf16", "e4m3"), ("f32", "f32")])
    dim = rng.choice([64, 128, 128]) if kv != "e4m3" else 128
    kvh, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 4, 5, 8])
    kind = rng.choice(["decode", "decode", "chunks", "mixed"])
    decodes = _log(rng, 1, 96) if kind != "chunks" else 0
    chunks = rng.randint(1, 6) if kind != "decode" else 0
    hi = _log(rng, 2, 4096 if src == "bf16" else 512) if chunks else 0
    ctx = _log(rng, 16, 16384 if src == "bf16" else 2048)
    most = 4e9 if src == "bf16" else 3e8  # products of queries and keys, times heads
    while (chunks * hi + decodes) * (ctx + hi) * kvh * group > most or decodes * ctx > 250_000:
        ctx, decodes, hi = max(1, ctx * 3 // 4), decodes * 3 // 4, hi * 3 // 4
        if not decodes and not hi:
            decodes = 1
    chunks = chunks if hi else 0
    window = rng.choice([max(1, ctx // 4), max(1, ctx // 2), 512]) if op == "window" else 0
    return _attend(op, chunks=chunks, chunk_lo=max(1, hi // 3) if chunks else 0,
                   chunk_hi=hi if chunks else 0, decodes=decodes, ctx_lo=max(0, ctx // 4), ctx_hi=ctx,
                   heads=kvh * group, kv_heads=kvh, dim=dim, window=window,
                   first=rng.choice([1, 4, 33]) if window else 0,
                   observed=rng.choice([0, 0, 1, 32]) if op == "weigh" else 0,
                   sinks=rng.random() < 0.3, lse=rng.random() < 0.5, src=src, kv=kv)


# ---- inputs ---------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _pool(gen, shape, kv):
    x = torch.randn(shape, generator=gen, device=DEV)
    return (x * 8).to(E4M3) if kv == "e4m3" else x.to(TYPES[kv])


def _sizes(case):
    """A generator for a batch's lengths: another seed shuffles them, so its outputs keep
    their shapes."""
    return np.random.default_rng(zlib.crc32(repr(sorted(
        (k, v) for k, v in case.items() if k != "name")).encode()))


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _tables(rng, lens, block):
    """Block tables over a permuted pool (blocks in use, rounded up to 16) and its size."""
    need = [-(-int(n) // block) for n in lens]
    num = -(-max(1, sum(need)) // 16) * 16
    ids = rng.permutation(num)
    t = np.zeros((len(need), max(1, max(need))), np.int64)
    at = 0
    for s, n in enumerate(need):
        t[s, :n] = ids[at:at + n]
        at += n
    return t, num


def _prepare_attend(c, seed):
    rng, gen, sizes = np.random.default_rng(seed), _gen(seed), _sizes(c)
    H, G, D = c["heads"], c["kv_heads"], c["dim"]
    S = c["chunks"] + c["decodes"]
    n = np.ones(S, np.int64)
    if c["chunks"]:
        n[:c["chunks"]] = sizes.integers(c["chunk_lo"], c["chunk_hi"] + 1, c["chunks"])
        n[0] = c["chunk_hi"]
    ctx = sizes.integers(c["ctx_lo"], c["ctx_hi"] + 1, S)
    ctx[0] = c["ctx_hi"]
    order = rng.permutation(S)
    n, ctx = n[order], ctx[order]
    lens = n + ctx
    T = int(n.sum())
    tables, num = _tables(rng, lens, BLOCK)
    src = TYPES[c["src"]]
    state = {
        "c": c, "q": torch.randn(T, H, D, generator=gen, device=DEV).to(src),
        "kb": _pool(gen, (num, BLOCK, G, D), c["kv"]),
        "vb": _pool(gen, (num, BLOCK, G, D), c["kv"]),
        "out": torch.empty(T, H, D, dtype=src, device=DEV),
        "lse": torch.empty(H, T, device=DEV) if c["lse"] else None,
        "sinks": torch.randn(H, generator=gen, device=DEV) if c["sinks"] else None,
        "qsl": _int(np.concatenate([[0], np.cumsum(n)])), "seq_lens": _int(lens),
        "positions": _int(np.concatenate([np.arange(a, b) for a, b in zip(ctx, lens)])),
        "tables": _int(tables), "scale": 1.0 / math.sqrt(D),
        "ks": 0.125 if c["kv"] == "e4m3" else 1.0, "vs": 0.25 if c["kv"] == "e4m3" else 1.0,
        "host_n": n.tolist(), "host_lens": lens.tolist()}  # (a scheduler knows them, too)
    if c["op"] == "weigh":
        # what earlier steps have added up; the largest length is the same for every seed
        most = int(lens.max())
        state["weights"] = torch.rand(S, G, most, generator=gen, device=DEV)
    return state


def _lengths(c, sizes):
    lens = sizes.integers(c["len_lo"], c["len_hi"] + 1, c["seqs"])
    lens[0] = c["len_hi"]
    return lens


def _prepare_evict(c, seed):
    rng, gen = np.random.default_rng(seed), _gen(seed)
    lens = rng.permutation(_lengths(c, _sizes(c)))
    new = np.maximum(1, (lens * c["keep"]).astype(np.int64))
    tables, num = _tables(rng, lens, c["block"])
    shape = (num, c["block"], c["kv_heads"], c["dim"])
    most = int(lens.max())
    # summed attention weights: heavy-tailed, and some keys that no query has looked at
    w = torch.randn(c["seqs"], c["kv_heads"], most, generator=gen, device=DEV).mul(2).exp()
    w[torch.rand(w.shape, generator=gen, device=DEV) < 0.05] = 0.0
    return {"c": c, "kb": _pool(gen, shape, c["kv"]), "vb": _pool(gen, shape, c["kv"]),
            "tables": _int(tables), "seq_lens": _int(lens), "new_lens": _int(new),
            "summed": w, "weights": torch.empty_like(w)}


def prepare(case, seed):
    return (_prepare_evict if case["op"] == "evict" else _prepare_attend)(case, seed)


# ---- one pass -------------------------------------------------------------------------------


def _take(pool, slots, scale):
    """Rows [..., Hkv, D] of a pool in 32 bits."""
    rows = pool.view(-1, *pool.shape[2:])
    if pool.dtype == E4M3:
        rows = rows.view(torch.uint8)[slots].view(E4M3)
    else:
        rows = rows[slots]
    return rows.float() * scale


def _softmax(x, sink):
    """Weights and log-sum-exp of the last axis; a sink logit joins the sum."""
    m = x.amax(-1, keepdim=True)
    if sink is not None:
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    if sink is not None:
        total = total + (sink - m).exp()
    lse = m + total.log()
    return x.div_(torch.where(total > 0, total, torch.ones_like(total))), lse


def _plain_decodes(s, rows):
    """The sequences with one new token, together."""
    c, G, D = s["c"], s["c"]["kv_heads"], s["c"]["dim"]
    w, f = c["window"], c["first"]
    seqs = torch.tensor(rows, device=DEV)
    lens = s["seq_lens"].long()[seqs]
    tok = s["qsl"].long()[seqs]
    longest = max(s["host_lens"][i] for i in rows)
    span = min(longest, w) if w else longest
    j = torch.arange(span, device=DEV) + (lens - span)[:, None]  # a window's keys end with the query
    here = j >= 0
    if w and f:
        i = torch.arange(f, device=DEV).expand(len(rows), f)
        j = torch.cat([i, j], 1)
        here = torch.cat([i < (lens - w)[:, None], here], 1)
    j = j.clamp_min(0)
    slots = s["tables"].long()[seqs].gather(1, j // BLOCK) * BLOCK + j % BLOCK
    K, V = _take(s["kb"], slots, s["ks"]), _take(s["vb"], slots, s["vs"])
    V = V.masked_fill_(~here[:, :, None, None], 0.0)
    q = s["q"][tok].float().view(len(rows), G, -1, D)
    x = q @ K.permute(0, 2, 3, 1) * s["scale"]
    x = x.masked_fill_(~here[:, None, None], -math.inf)
    sink = s["sinks"].view(1, G, -1, 1) if s["sinks"] is not None else None
    p, lse = _softmax(x, sink)
    s["out"][tok] = (p @ V.permute(0, 2, 1, 3)).flatten(1, 2).to(s["q"].dtype)
    if s["lse"] is not None:
        s["lse"][:, tok] = lse.flatten(1).t()
    if c["op"] == "weigh":
        got = p.sum(2)
        W = s["weights"]
        at = (seqs[:, None, None] * G + torch.arange(G, device=DEV)[:, None]) * W.shape[2] + j[:, None]
        W.view(-1).index_add_(0, at.flatten(), got.flatten())


def _plain_chunk(s, i):
    """Sequence i, whose new tokens are its last ones."""
    c, G, D = s["c"], s["c"]["kv_heads"], s["c"]["dim"]
    w, f, n, L = c["window"], c["first"], s["host_n"][i], s["host_lens"][i]
    t0 = sum(s["host_n"][:i])
    lo = max(0, L - n - w + 1) if w else 0
    j = torch.arange(lo, L, device=DEV)
    if lo > 0 and f:
        j = torch.cat([torch.arange(min(f, lo), device=DEV), j])
    pos = torch.arange(L - n, L, device=DEV)[:, None]
    see = j <= pos
    if w:
        see &= (j > pos - w) | (j < f)
    slots = s["tables"][i].long()[j // BLOCK] * BLOCK + j % BLOCK
    K, V = _take(s["kb"], slots, s["ks"]), _take(s["vb"], slots, s["vs"])
    counted = n if c["observed"] == 0 else min(n, c["observed"])
    for g in range(G):
        hs = slice(g * (c["heads"] // G), (g + 1) * (c["heads"] // G))
        q = s["q"][t0:t0 + n, hs].float().transpose(0, 1)
        x = (q @ K[:, g].t()).mul_(s["scale"]).masked_fill_(~see, -math.inf)
        sink = s["sinks"][hs].view(-1, 1, 1) if s["sinks"] is not None else None
        p, lse = _softmax(x, sink)
        s["out"][t0:t0 + n, hs] = (p @ V[:, g]).transpose(0, 1).to(s["q"].dtype)
        if s["lse"] is not None:
            s["lse"][hs, t0:t0 + n] = lse.squeeze(-1)
        if c["op"] == "weigh":
            s["weights"][i, g].index_add_(0, j, p[:, n - counted:].sum((0, 1)))


def _attended(s):
    got = {"out": s["out"]}
    if s["lse"] is not None:
        got["lse"] = s["lse"]
    if s["c"]["op"] == "weigh":
        got["key_weights"] = s["weights"]
    return got


def _plain_attend(s):
    ones = [i for i, n in enumerate(s["host_n"]) if n == 1]
    if ones:
        _plain_decodes(s, ones)
    for i, n in enumerate(s["host_n"]):
        if n > 1:
            _plain_chunk(s, i)
    return _attended(s)


def _plain_evict(s):
    c, W = s["c"], s["weights"]
    S, G, L = W.shape
    b = c["block"]
    W.copy_(s["summed"])
    n, new = s["seq_lens"].long()[:, None, None], s["new_lens"].long()[:, None, None]
    f = new.clamp_max(c["first"])
    r = (new - f).clamp_max(c["recent"])
    j = torch.arange(L, device=DEV).expand(S, G, L)
    # the m heaviest of the keys between the first and the recent ones; ties to the lowest index
    middle = (j >= f) & (j < n - r)
    order = W.masked_fill(~middle, -1.0).sort(dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, j)
    kept = middle & (rank < new - f - r)
    # those that stay in place, the places that become free, and the keys that fill them in order
    hole = middle & ~kept & (j < new - r)
    filler = kept & (j >= new - r)
    src = torch.where((j >= new - r) & (j < new), j + n - new, j)
    at = torch.cumsum(filler.long(), -1) - 1
    filled = torch.zeros(S, G, L + 1, dtype=torch.long, device=DEV)
    filled.scatter_(-1, torch.where(filler, at, L), j)
    src = torch.where(hole, filled.gather(-1, (torch.cumsum(hole.long(), -1) - 1).clamp_min(0)), src)
    src = torch.where((n > new) & (j < new), src, j).clamp_max(L - 1)
    slot = lambda p: (s["tables"].long()[:, None].expand(S, G, -1).gather(2, p // b) * b + p % b)
    live = j < n
    own_row = torch.where(live, j, torch.zeros_like(j))
    src_row = torch.where(live, src, torch.zeros_like(j))
    g = torch.arange(G, device=DEV)[:, None]
    to, frm = (slot(own_row) * G + g).flatten(), (slot(src_row) * G + g).flatten()
    for pool in (s["kb"], s["vb"]):
        rows = pool.view(-1, pool.shape[3])
        rows = rows.view(torch.uint8) if pool.dtype == E4M3 else rows
        # (positions past a sequence's end repeat its first row)
        frm_first = torch.where(live.flatten(), frm, (slot(src[..., :1].expand(S, G, L)) * G + g).flatten())
        rows[to] = rows[frm_first]
    moved = W.gather(-1, src)
    W.copy_(torch.where((j < new) | (n <= new), moved, torch.where(live, torch.zeros_like(W), W)))
    return {"k_blocks": s["kb"], "v_blocks": s["vb"], "key_weights": W}


def _own(s):
    from paged_kv_cache_31_gb300 import binding as pa

    c = s["c"]
    if c["op"] == "evict":
        s["weights"].copy_(s["summed"])
        pa.pa_evict_keys(s["kb"], s["vb"], s["tables"], s["seq_lens"], s["new_lens"], s["weights"],
                         keep_first=c["first"], keep_recent=c["recent"])
        return {"k_blocks": s["kb"], "v_blocks": s["vb"], "key_weights": s["weights"]}
    batch = (s["q"], s["kb"], s["vb"], s["out"], s["qsl"], s["seq_lens"], s["positions"],
             s["tables"])
    extras = {"sinks": s["sinks"], "lse": s["lse"], "k_scale": s["ks"], "v_scale": s["vs"]}
    if c["op"] == "window":
        pa.pa_window_attention(*batch, s["scale"], sliding_window=c["window"],
                               first_tokens=c["first"], **extras)
    else:
        pa.pa_attention_key_weights(*batch, s["weights"], s["scale"],
                                    observed_tokens=c["observed"], **extras)
    return _attended(s)


def run(state):
    if own:
        return _own(state)
    return (_plain_evict if state["c"]["op"] == "evict" else _plain_attend)(state)


# ---- what a pass cannot do without ----------------------------------------------------------


def work(case):
    c = case
    size = {"bf16": 2, "f32": 4, "e4m3": 1}
    if c["op"] == "evict":
        n = (c["len_lo"] + c["len_hi"]) / 2
        new = n * c["keep"]
        f = min(c["first"], new)
        r = min(c["recent"], new - f)
        # the recent rows, and of the others that stay those that lie behind their new end
        moved = r + (new - f - r) * (n - new) / max(n - f - r, 1)
        heads = c["seqs"] * c["kv_heads"]
        return {"bytes": heads * (moved * 2 * 2 * c["dim"] * size[c["kv"]] + 4 * (n + moved + n - new)),
                "flops": 0}
    H, G, D = c["heads"], c["kv_heads"], c["dim"]
    ctx = (c["ctx_lo"] + c["ctx_hi"]) / 2
    chunk = (c["chunk_lo"] + c["chunk_hi"]) / 2
    w, f = c["window"], c["first"]
    total, flops = 0.0, 0.0
    for count, n in ((c["chunks"], chunk), (c["decodes"], 1)):
        if not count:
            continue
        keys = min(ctx + n, w + f + n - 1) if w else ctx + n
        # the mean number of keys that a query sees
        seen = (ctx + (n + 1) / 2) if not w else min(ctx + (n + 1) / 2, w + f)
        total += count * (2 * keys * G * D * size[c["kv"]]
                          + n * H * (2 * D * size[c["src"]] + (4 if c["lse"] else 0)))
        if c["op"] == "weigh":
            total += count * 2 * 4 * keys * G
        flops += count * 4 * n * seen * H * D
    return {"bytes": total, "flops": flops}


# ---- the definitions in 64 bits -------------------------------------------------------------


def _exact_attend(c, s):
    H, G, D = c["heads"], c["kv_heads"], c["dim"]
    T = s["q"].shape[0]
    out = torch.zeros(T, H, D, dtype=torch.float64, device=DEV)
    lse = torch.full((H, T), -math.inf, dtype=torch.float64, device=DEV)
    weights = s["weights"].double() if c["op"] == "weigh" else None
    qsl, lens = s["qsl"].tolist(), s["seq_lens"].tolist()
    for i, L in enumerate(lens):
        a, b = qsl[i], qsl[i + 1]
        ids = s["tables"][i, :-(-L // BLOCK)].long()
        pos = s["positions"][a:b].double()[:, None]
        keys = torch.arange(L, device=DEV, dtype=torch.float64)
        hidden = keys > pos
        if c["window"]:
            hidden |= (pos - keys >= c["window"]) & (keys >= c["first"])
        whole = lambda p: p.view(torch.uint8)[ids].view(p.dtype).flatten(0, 1)[:L]
        kd, vd = whole(s["kb"]), whole(s["vb"])
        for h in range(H):
            k, v = kd[:, h * G // H].double() * s["ks"], vd[:, h * G // H].double() * s["vs"]
            for r0 in range(0, b - a, 2048):  # (rows at a time: the scores of all may not fit)
                r1 = min(b - a, r0 + 2048)
                x = torch.einsum("td,kd->tk", s["q"][a + r0:a + r1, h].double(), k) * s["scale"]
                x.masked_fill_(hidden[r0:r1], -math.inf)
                l = torch.logsumexp(x, -1)
                if s["sinks"] is not None:
                    l = torch.logaddexp(l, s["sinks"][h].double())
                p = torch.exp(x - l[:, None])
                out[a + r0:a + r1, h] = p @ v
                lse[h, a + r0:a + r1] = l
                if weights is not None:
                    skip = max(0, b - a - c["observed"] - r0) if c["observed"] else 0
                    weights[i, h * G // H, :L] += p[skip:].sum(0)
    got = {"out": out}
    if c["lse"]:
        got["lse"] = lse
    if weights is not None:
        got["key_weights"] = weights
    return got


def _exact_evict(c, s):
    kb, vb = s["kb"].double(), s["vb"].double()
    k_old, v_old = kb.clone(), vb.clone()
    W = s["summed"].double().cpu().numpy()
    tables = s["tables"].cpu().numpy()
    b = c["block"]
    moves = []  # (old page, row, head) and (new page, row, head)
    for i, (n, new) in enumerate(zip(s["seq_lens"].tolist(), s["new_lens"].tolist())):
        if new >= n:
            continue
        f = min(c["first"], new)
        r = min(c["recent"], new - f)
        for g in range(c["kv_heads"]):
            w = W[i, g].copy()
            mid = np.arange(f, n - r)
            heavy = mid[np.lexsort((mid, -w[mid]))][:new - f - r]
            stay = set(heavy[heavy < new - r].tolist())
            free = [x for x in range(f, new - r) if x not in stay]
            frm = np.concatenate([np.sort(heavy[heavy >= new - r]), np.arange(n - r, n)])
            to = np.concatenate([np.array(free, np.int64), np.arange(new - r, new)])
            W[i, g, to] = w[frm.astype(np.int64)]
            W[i, g, new:n] = 0.0
            page = lambda p: np.stack([tables[i, p // b], p % b, np.full(len(p), g)])
            moves.append(np.concatenate([page(frm.astype(np.int64)), page(to)]))
    if moves:
        m = torch.from_numpy(np.concatenate(moves, 1)).to(DEV)
        kb[m[3], m[4], m[5]] = k_old[m[0], m[1], m[2]]
        vb[m[3], m[4], m[5]] = v_old[m[0], m[1], m[2]]
    return {"k_blocks": kb, "v_blocks": vb, "key_weights": torch.from_numpy(W).to(DEV)}


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_evict if case["op"] == "evict" else _exact_attend)(case, s)

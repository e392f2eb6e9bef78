"""Speculative decoding over the paged K/V cache: the cases its operators are measured on.

A drafted step puts a tree of candidate tokens behind every sequence: their queries and keys
are rotated and their rows cached (rope), the tree attends to the cached context and to the
ancestors of each node (tree), the accepted path's rows are moved together (commit), and the
pages are copied (copy) and shared, taken and given back (pages) as sequences fork and end.

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


def listed():
    return [
        # one decoding step of a 64-sequence batch, Llama-3-8B heads: latency counts
        {"name": "rope_decode_64", "op": "rope", "tokens": 64, "heads": 32, "kv_heads": 8,
         "dim": 128, "rotary": 128, "interleaved": False, "scaling": "llama3", "max_pos": 8192,
         "src": "bf16", "kv": "bf16"},
        # a long prompt's rows taken out of one fused q/k/v product, half of each head rotated
        # in interleaved pairs, into e4m3 pools with scales, at far positions
        {"name": "rope_prompt_16381_e4m3", "op": "rope", "tokens": 16381, "heads": 32,
         "kv_heads": 8, "dim": 128, "rotary": 64, "interleaved": True, "scaling": "yarn",
         "max_pos": 1000000, "src": "bf16", "kv": "e4m3"},
        # a single user's chat with a small tree: the smallest call
        {"name": "tree_1x8_ctx700", "op": "tree", "seqs": 1, "nodes_lo": 8, "nodes_hi": 8,
         "ctx_lo": 700, "ctx_hi": 700, "heads": 32, "kv_heads": 8, "dim": 128, "window": 0,
         "lse": False, "src": "bf16", "kv": "bf16"},
        # the 64-sequence serving batch (contexts 512 to 4096), ragged trees of 1 to 32 nodes
        {"name": "tree_64x32_ragged", "op": "tree", "seqs": 64, "nodes_lo": 1, "nodes_hi": 32,
         "ctx_lo": 512, "ctx_hi": 4096, "heads": 32, "kv_heads": 8, "dim": 128, "window": 0,
         "lse": True, "src": "bf16", "kv": "bf16"},
        # e4m3 pools behind a sliding window of 4096, contexts 1024 to 8192
        {"name": "tree_48x16_e4m3_window", "op": "tree", "seqs": 48, "nodes_lo": 5, "nodes_hi": 16,
         "ctx_lo": 1024, "ctx_hi": 8192, "heads": 32, "kv_heads": 8, "dim": 128, "window": 4096,
         "lse": False, "src": "bf16", "kv": "e4m3"},
        # long documents with wide trees, 64 query heads: 512 rows share each key
        {"name": "tree_4x64_ctx65536", "op": "tree", "seqs": 4, "nodes_lo": 64, "nodes_hi": 64,
         "ctx_lo": 65533, "ctx_hi": 65536, "heads": 64, "kv_heads": 8, "dim": 128, "window": 0,
         "lse": True, "src": "bf16", "kv": "bf16"},
        # accepting up to 4 drafted tokens of one tree
        {"name": "commit_1x24", "op": "commit", "seqs": 1, "nodes": 24, "max_accept": 4,
         "ctx_hi": 2048, "kv_heads": 8, "dim": 128, "block": 16, "kv": "bf16"},
        # the 256-sequence batch accepting up to 8 of 64 nodes each
        {"name": "commit_256x64", "op": "commit", "seqs": 256, "nodes": 64, "max_accept": 8,
         "ctx_hi": 4096, "kv_heads": 8, "dim": 128, "block": 16, "kv": "bf16"},
        # a fork of a few sequences: their last, partly filled pages
        {"name": "copy_7", "op": "copy", "pairs": 7, "kv_heads": 8, "dim": 128, "block": 16,
         "kv": "bf16"},
        # moving a large part of a pool
        {"name": "copy_4096", "op": "copy", "pairs": 4096, "kv_heads": 8, "dim": 128,
         "block": 16, "kv": "bf16"},
        # one prompt answered four ways: fork, room for the drafts, and the end of all four
        {"name": "pages_4_of_1", "op": "pages", "parents": 1, "children": 4, "len_lo": 1000,
         "len_hi": 1000, "grow_hi": 24, "block": 16},
        # the same for 256 children of 16 long parents
        {"name": "pages_256_of_16", "op": "pages", "parents": 16, "children": 256,
         "len_lo": 2048, "len_hi": 16384, "grow_hi": 64, "block": 16},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "tree", "tree", "tree", "tree", "commit", "copy", "pages"])
    if op == "rope":
        src, kv = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "e4m3"),
                              ("f32", "f32")])
        dim = rng.choice([64, 128, 128])
        kvh = rng.choice([1, 2, 4, 8])
        return {"op": op, "tokens": _log(rng, 1, 8192), "heads": kvh * rng.choice([1, 4, 5, 8]),
                "kv_heads": kvh, "dim": dim, "rotary": rng.choice([dim, dim, dim // 2, dim // 4]),
                "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "ntk", "yarn", "llama3"]),
                "max_pos": _log(rng, 2048, 1000000), "src": src, "kv": kv}
    if op == "tree":
        src, kv = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "e4m3"),
                              ("f32", "f32")])
        dim = rng.choice([64, 128, 128]) if kv != "e4m3" else 128
        seqs, nodes = _log(rng, 1, 96), _log(rng, 1, 64)
        ctx = _log(rng, 16, 16384)
        kvh, group = rng.choice([2, 4, 8]), rng.choice([1, 4, 5, 8])
        most = 24_000_000 if kv != "f32" else 2_000_000  # query rows of a kv head x keys
        while seqs * nodes * group * (ctx + nodes) > most or seqs * ctx > 250_000:
            ctx = max(16, ctx * 3 // 4)
            seqs = max(1, seqs * 3 // 4)
        return {"op": op, "seqs": seqs, "nodes_lo": max(1, nodes // 3), "nodes_hi": nodes,
                "ctx_lo": max(1, ctx // 4), "ctx_hi": ctx, "heads": kvh * group, "kv_heads": kvh,
                "dim": dim, "window": rng.choice([0, 0, max(1, ctx // 2)]),
                "lse": rng.random() < 0.5, "src": src, "kv": kv}
    heads = {"kv_heads": rng.choice([1, 4, 8]), "dim": rng.choice([64, 128]),
             "block": rng.choice([16, 16, 32]), "kv": rng.choice(["bf16", "e4m3", "f32"])}
    if op == "commit":
        most = rng.randint(1, 10)
        return {"op": op, "seqs": _log(rng, 1, 256), "nodes": rng.randint(2 * most, 64),
                "max_accept": most, "ctx_hi": _log(rng, 1, 4096), **heads}
    if op == "copy":
        return {"op": op, "pairs": _log(rng, 1, 2048), **heads}
    parents = _log(rng, 1, 32)
    lo = _log(rng, 1, 4096)
    return {"op": op, "parents": parents, "children": _log(rng, 1, 256), "len_lo": lo,
            "len_hi": 4 * lo, "grow_hi": rng.randint(1, 64), "block": rng.choice([16, 16, 32])}


# ---- inputs ---------------------------------------------------------------------------------


def _frequencies(rotary, scaling):
    """Radians per position of each rotated pair, in 64 bits, and the attention factor."""
    i = np.arange(rotary // 2, dtype=np.float64)
    base, factor, trained = 500000.0, 8.0, 8192
    if scaling == "ntk":
        base *= factor ** (rotary / max(rotary - 2, 1))
    f = base ** (-2.0 * i / rotary)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "llama3":
        wave, low, high = 2 * math.pi / f, 1.0, 4.0
        mid = np.clip((trained / wave - low) / (high - low), 0.0, 1.0)
        return (1 - mid) * f / factor + mid * f, 1.0
    if scaling == "yarn":
        turn = lambda n: rotary * math.log(trained / (n * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(turn(32)), 0), min(math.ceil(turn(1)), rotary - 1)
        keep = 1 - np.clip((i - low) / max(high - low, 0.001), 0.0, 1.0)
        return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0
    return f, 1.0


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


def _scales(kv):
    return (0.125, 0.25) if kv == "e4m3" else (1.0, 1.0)


def _prepare_rope(c, seed):
    rng, gen = np.random.default_rng(seed), _gen(seed)
    T, H, G, D = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
    src = TYPES[c["src"]]
    qkv = torch.randn(T, (H + 2 * G) * D, generator=gen, device=DEV).to(src)
    q, k, v = (x.view(T, -1, D) for x in qkv.split([H * D, G * D, G * D], dim=1))
    num = -(-T // BLOCK) + 16
    slots = rng.permutation(num * BLOCK)[:T]
    f, factor = _frequencies(c["rotary"], c["scaling"])
    ks, vs = _scales(c["kv"])
    return {"c": c, "q": q, "k": k, "v": v,
            "q_out": torch.empty(T, H, D, dtype=src, device=DEV),
            "kb": _pool(gen, (num, BLOCK, G, D), c["kv"]),
            "vb": _pool(gen, (num, BLOCK, G, D), c["kv"]),
            "positions": _int(rng.integers(0, c["max_pos"], T)), "slots": _int(slots),
            "inv_freq": torch.from_numpy(f).to(DEV), "factor": factor, "ks": ks, "vs": vs}


def _prepare_tree(c, seed):
    rng, gen = np.random.default_rng(seed), _gen(seed)
    S, H, G, D = c["seqs"], c["heads"], c["kv_heads"], c["dim"]
    sizes, order = _sizes(c), rng.permutation(S)
    n = sizes.integers(c["nodes_lo"], c["nodes_hi"] + 1, S)
    ctx = sizes.integers(c["ctx_lo"], c["ctx_hi"] + 1, S)
    n[0], ctx[0] = c["nodes_hi"], c["ctx_hi"]
    n, ctx = n[order], ctx[order]
    lens = n + ctx
    T = int(n.sum())
    words = -(-c["nodes_hi"] // 32)
    mask = np.zeros((T, words), np.uint32)
    pos = np.zeros(T, np.int64)
    t = 0
    for s in range(S):
        parent = [-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, n[s])]
        for i in range(n[s]):
            depth = 0
            if parent[i] >= 0:
                mask[t + i] = mask[t + parent[i]]
                depth = pos[t + parent[i]] - ctx[s] + 1
            mask[t + i, i // 32] |= np.uint32(1 << (i % 32))
            pos[t + i] = ctx[s] + depth
        t += n[s]
    tables, num = _tables(rng, lens, BLOCK)
    ks, vs = _scales(c["kv"])
    src = TYPES[c["src"]]
    return {"c": c, "q": torch.randn(T, H, D, generator=gen, device=DEV).to(src),
            "kb": _pool(gen, (num, BLOCK, G, D), c["kv"]),
            "vb": _pool(gen, (num, BLOCK, G, D), c["kv"]),
            "out": torch.empty(T, H, D, dtype=src, device=DEV),
            "lse": torch.empty(H, T, device=DEV) if c["lse"] else None,
            "qsl": _int(np.concatenate([[0], np.cumsum(n)])), "seq_lens": _int(lens),
            "positions": _int(pos), "mask": torch.from_numpy(mask.view(np.int32)).to(DEV),
            "tables": _int(tables), "scale": 1.0 / math.sqrt(D), "ks": ks, "vs": vs,
            "most_nodes": int(c["nodes_hi"]), "most_keys": int(lens.max())}


def _prepare_commit(c, seed):
    rng, gen = np.random.default_rng(seed), _gen(seed)
    S, n, most = c["seqs"], c["nodes"], c["max_accept"]
    ctx = rng.permutation(_sizes(c).integers(max(1, c["ctx_hi"] // 8), c["ctx_hi"] + 1, S))
    tables, num = _tables(rng, ctx + n, c["block"])
    # a path of a tree laid out level by level: the root, then nodes of deeper levels
    count = rng.integers(1, most + 1, S)
    acc = np.sort(np.stack([rng.permutation(np.arange(most, n))[:most] for _ in range(S)]), 1)
    acc = np.concatenate([np.zeros((S, 1), np.int64), acc[:, :most - 1]], 1)
    shape = (num, c["block"], c["kv_heads"], c["dim"])
    return {"c": c, "kb": _pool(gen, shape, c["kv"]), "vb": _pool(gen, shape, c["kv"]),
            "tables": _int(tables), "ctx": _int(ctx), "accepted": _int(acc),
            "count": _int(count)}


def _prepare_copy(c, seed):
    rng, gen = np.random.default_rng(seed), _gen(seed)
    n = c["pairs"]
    num = -(-2 * n // 16) * 16
    dst = rng.permutation(num)[:n]
    src = rng.choice(np.setdiff1d(np.arange(num), dst), n)  # a page may be copied twice
    shape = (num, c["block"], c["kv_heads"], c["dim"])
    return {"c": c, "kb": _pool(gen, shape, c["kv"]), "vb": _pool(gen, shape, c["kv"]),
            "pairs": _int(np.stack([src, dst], 1))}


def _prepare_pages(c, seed):
    rng = np.random.default_rng(seed)
    P, C, b = c["parents"], c["children"], c["block"]
    lens = _sizes(c).integers(c["len_lo"], c["len_hi"] + 1, P)
    lens[0] = c["len_hi"]
    lens = rng.permutation(lens)
    parents = rng.integers(0, P, C)
    grown = lens[parents] + rng.integers(0, c["grow_hi"] + 1, C)
    cols = -(-(c["len_hi"] + c["grow_hi"]) // b)
    used = -(-lens // b)
    extra = C * (2 + c["grow_hi"] // b)
    num = -(-(int(used.sum()) + extra) // 16) * 16
    ids = rng.permutation(num)
    tables = np.zeros((P + C, cols), np.int64)
    at = 0
    for p in range(P):
        tables[p, :used[p]] = ids[at:at + used[p]]
        at += used[p]
    refs = np.zeros(num, np.int64)
    refs[ids[:at]] = 1
    free = np.zeros(num, np.int64)
    free[:num - at] = np.sort(ids[at:])
    return {"c": c, "tables": _int(tables),
            "seq_lens": _int(np.concatenate([lens, np.zeros(C, np.int64)])),
            "parents": _int(parents), "children": _int(P + rng.permutation(C)),
            "grown": _int(grown), "refs": _int(refs), "free": _int(free),
            "free_count": _int([num - at]),
            "pairs": torch.empty(C, 2, dtype=torch.int32, device=DEV)}


def prepare(case, seed):
    return {"rope": _prepare_rope, "tree": _prepare_tree, "commit": _prepare_commit,
            "copy": _prepare_copy, "pages": _prepare_pages}[case["op"]](case, seed)


# ---- one pass -------------------------------------------------------------------------------


def _rotate(x, cos, sin, rotary, interleaved):
    """x [T, N, D] in 32 bits; cos, sin [T, 1, rotary / 2]."""
    r, rest = x[..., :rotary], x[..., rotary:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = r[..., :rotary // 2], r[..., rotary // 2:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, rest], -1)


def _store(x, dtype):
    return x.clamp(-448.0, 448.0).to(E4M3) if dtype == E4M3 else x.to(dtype)


def _bytes(pool):
    """The pool's rows [rows, Hkv, D], as bytes where torch does not index the type."""
    rows = pool.view(-1, *pool.shape[2:])
    return rows.view(torch.uint8) if pool.dtype == E4M3 else rows


def _run_rope(s):
    c = s["c"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos = (angle.cos() * s["factor"]).float()[:, None]
    sin = (angle.sin() * s["factor"]).float()[:, None]
    q = _rotate(s["q"].float(), cos, sin, c["rotary"], c["interleaved"])
    k = _rotate(s["k"].float(), cos, sin, c["rotary"], c["interleaved"])
    s["q_out"].copy_(q)
    slots = s["slots"].long()
    kb, vb = s["kb"], s["vb"]
    k, v = _store(k / s["ks"], kb.dtype), _store(s["v"].float() / s["vs"], vb.dtype)
    _bytes(kb)[slots] = k.view(torch.uint8) if kb.dtype == E4M3 else k
    _bytes(vb)[slots] = v.view(torch.uint8) if vb.dtype == E4M3 else v
    return {"q": s["q_out"], "k_blocks": kb, "v_blocks": vb}


def _run_tree(s):
    c, q = s["c"], s["q"]
    T, H, D = q.shape
    G, N, L, w = c["kv_heads"], s["most_nodes"], s["most_keys"], c["window"]
    qsl, lens = s["qsl"].long(), s["seq_lens"].long()
    S = lens.numel()
    n = qsl[1:] - qsl[:-1]
    ctx = lens - n
    # queries padded to [S, N], keys to [S, L]
    node = torch.arange(N, device=DEV)
    tok = (qsl[:-1, None] + node).clamp_max(T - 1)
    here = node < n[:, None]
    j = torch.arange(L, device=DEV)
    cached = j < lens[:, None]
    slot = s["tables"].long()[:, j // BLOCK] * BLOCK + j % BLOCK
    slot = torch.where(cached, slot, torch.zeros_like(slot))
    gap = ~cached[:, :, None, None]
    kb, vb = s["kb"].view(-1, G, D), s["vb"].view(-1, G, D)
    take = lambda p: (p.view(torch.uint8)[slot].view(E4M3) if p.dtype == E4M3 else p[slot])
    K = (take(kb).float() * s["ks"]).masked_fill_(gap, 0.0)
    V = (take(vb).float() * s["vs"]).masked_fill_(gap, 0.0)
    # which key each node sees
    k_node = j - ctx[:, None]  # the key's own node, where it is one
    in_tree = (k_node >= 0) & cached
    k_node = k_node.clamp(0, N - 1)
    words = s["mask"].long()[tok]  # [S, N, words]
    word = words.gather(2, (k_node // 32)[:, None].expand(S, N, L))
    bit = (word >> (k_node % 32)[:, None]) & 1
    key_pos = torch.where(in_tree, s["positions"].long()[tok].gather(1, k_node), j)
    see = torch.where(in_tree[:, None], bit != 0, cached[:, None])
    if w > 0:
        see &= key_pos[:, None] > s["positions"].long()[tok][:, :, None] - w
    # softmax in 32 bits
    qp = q[tok].float().view(S, N, G, H // G, D).permute(0, 2, 1, 3, 4).reshape(S, G, -1, D)
    x = qp @ K.permute(0, 2, 3, 1) * s["scale"]
    x = x.view(S, G, N, H // G, L).masked_fill_(~see[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(S, G, -1, L) @ V.permute(0, 2, 1, 3)).view(S, G, N, H // G, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 2, 1, 3, 4).reshape(S * N, H, D)
    # padded nodes write the row of a real one: node 0 of their sequence
    flat = torch.where(here, node, torch.zeros_like(node))
    at = (torch.arange(S, device=DEV)[:, None] * N + flat).view(-1)
    row = (qsl[:-1, None] + flat).view(-1)
    s["out"][row] = o[at].to(q.dtype)
    if s["lse"] is None:
        return s["out"]
    lse = (m + total.log()).squeeze(-1).permute(0, 2, 1, 3).reshape(S * N, H)
    s["lse"][:, row] = lse[at].t()
    return s["out"], s["lse"]


def _run_commit(s):
    b = s["c"]["block"]
    i = torch.arange(s["accepted"].shape[1], device=DEV)
    ctx, tables = s["ctx"].long()[:, None], s["tables"].long()
    live = i < s["count"].long()[:, None]
    to = ctx + i
    frm = torch.where(live, ctx + s["accepted"].long(), to)
    slot = lambda p: (tables.gather(1, p // b) * b + p % b).view(-1)
    src, dst = slot(frm), slot(to)
    kb, vb = _bytes(s["kb"]), _bytes(s["vb"])
    kb[dst] = kb[src]
    vb[dst] = vb[src]
    return s["kb"], s["vb"]


def _run_copy(s):
    src, dst = s["pairs"].long().unbind(1)
    for_bytes = lambda p: p.view(torch.uint8) if p.dtype == E4M3 else p
    kb, vb = for_bytes(s["kb"]), for_bytes(s["vb"])
    kb[dst] = kb[src]
    vb[dst] = vb[src]
    return s["kb"], s["vb"]


def _run_pages(s):
    b = s["c"]["block"]
    tables, lens, refs, free, count = (s[x] for x in ("tables", "seq_lens", "refs", "free",
                                                      "free_count"))
    par, chi, grown = s["parents"].long(), s["children"].long(), s["grown"]
    num = refs.numel()
    cols = torch.arange(tables.shape[1], device=DEV)
    n = lens[par].long()
    full, part = (n // b)[:, None], n % b > 0
    # fork: whole pages are shared, the last partly filled one becomes a page of its own
    taken = torch.cumsum(part.long(), 0)
    page = free[(count.long() - taken).clamp_min(0)]
    page = torch.where(part, page, torch.full_like(page, -1))
    rows, old = tables[par], tables[chi]
    own_page = (cols == full) & part[:, None]
    tail = rows.gather(1, full.clamp_max(tables.shape[1] - 1)).squeeze(1)
    s["pairs"][:, 0] = torch.where(part, tail, torch.full_like(tail, -1))
    s["pairs"][:, 1] = page
    new = torch.where(cols < full, rows, torch.where(own_page, page[:, None], old))
    add = (cols < full) | own_page
    refs.index_add_(0, new.long().view(-1), add.int().view(-1))
    left = count.long() - taken[-1]
    # growth: pages for the positions up to the new length
    have, want = -(-n // b), -(-grown.long() // b)
    more = (want - have).clamp_min(0)
    before = torch.cumsum(more, 0) - more
    k = cols - have[:, None]
    fresh = (k >= 0) & (k < more[:, None])
    at = left - 1 - before[:, None] - k
    new = torch.where(fresh, free[at.clamp(0, num - 1)], new)
    refs.index_add_(0, new.long().view(-1), fresh.int().view(-1))
    tables[chi] = new
    lens[chi] = grown
    left = left - more.sum()
    # the end: every page of the children is given back; those that nobody holds are free,
    # in ascending order
    held = cols < want[:, None]
    drop = torch.zeros_like(refs).index_add_(0, new.long().view(-1), held.int().view(-1))
    gone = (drop > 0) & (refs == drop)
    refs -= drop
    rank = torch.cumsum(gone.long(), 0) - 1
    slots = torch.where(gone, left + rank, torch.full_like(rank, num))
    longer = torch.cat([free, free[:1]])
    longer.scatter_(0, slots, torch.arange(num, dtype=torch.int32, device=DEV))
    free.copy_(longer[:num])
    count.copy_(left + gone.sum())
    lens[chi] = 0
    return {"tables": tables, "seq_lens": lens, "refs": refs, "free": free, "count": count,
            "pairs": s["pairs"]}


def _own(s):
    from paged_kv_cache_31_gb300 import binding as pa

    c = s["c"]
    if c["op"] == "rope":
        pa.pa_rope_and_cache(s["q"], s["k"], s["v"], s["q_out"], s["kb"], s["vb"],
                             s["positions"], s["slots"], s["inv_freq"],
                             interleaved=c["interleaved"], attn_factor=s["factor"],
                             k_scale=s["ks"], v_scale=s["vs"])
        return {"q": s["q_out"], "k_blocks": s["kb"], "v_blocks": s["vb"]}
    if c["op"] == "tree":
        pa.pa_tree_attention(s["q"], s["kb"], s["vb"], s["out"], s["qsl"], s["seq_lens"],
                             s["positions"], s["mask"], s["tables"], s["scale"],
                             sliding_window=c["window"], lse=s["lse"], k_scale=s["ks"],
                             v_scale=s["vs"])
        return s["out"] if s["lse"] is None else (s["out"], s["lse"])
    if c["op"] == "commit":
        pa.pa_tree_commit(s["kb"], s["vb"], s["tables"], s["ctx"], s["accepted"], s["count"])
        return s["kb"], s["vb"]
    if c["op"] == "copy":
        pa.pa_copy_blocks(s["kb"], s["vb"], s["pairs"])
        return s["kb"], s["vb"]
    pages = (s["refs"], s["free"], s["free_count"], c["block"])
    pa.pa_fork_sequences(s["tables"], s["seq_lens"], s["parents"], s["children"], *pages,
                         block_pairs=s["pairs"])
    pa.pa_grow_sequences(s["tables"], s["seq_lens"], s["children"], s["grown"], *pages)
    pa.pa_free_sequences(s["tables"], s["seq_lens"], s["children"], *pages)
    return {"tables": s["tables"], "seq_lens": s["seq_lens"], "refs": s["refs"],
            "free": s["free"], "count": s["free_count"], "pairs": s["pairs"]}


def run(state):
    if own:
        return _own(state)
    return {"rope": _run_rope, "tree": _run_tree, "commit": _run_commit, "copy": _run_copy,
            "pages": _run_pages}[state["c"]["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------------------


def work(case):
    c = case
    size = {"bf16": 2, "f32": 4, "e4m3": 1}
    if c["op"] == "rope":
        T, H, G, D = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
        return {"bytes": T * D * (2 * H * size[c["src"]] + 2 * G * (size[c["src"]] + size[c["kv"]]))
                + 8 * T + 4 * c["rotary"], "flops": 3 * T * (H + G) * c["rotary"]}
    if c["op"] == "tree":
        S, H, G, D = c["seqs"], c["heads"], c["kv_heads"], c["dim"]
        n, ctx = (c["nodes_lo"] + c["nodes_hi"]) / 2, (c["ctx_lo"] + c["ctx_hi"]) / 2
        keys = min(ctx, c["window"]) if c["window"] else ctx
        T = S * n
        return {"bytes": 2 * S * (keys + n) * G * D * size[c["kv"]]
                + T * H * (2 * D * size[c["src"]] + (4 if c["lse"] else 0))
                + 4 * S * (keys + n) / BLOCK + 4 * T * (1 + -(-c["nodes_hi"] // 32)),
                "flops": 4 * T * H * D * (keys + n / 2)}
    row = 2 * c.get("kv_heads", 0) * c.get("dim", 0) * size[c.get("kv", "bf16")]
    if c["op"] == "commit":
        # the root's row stays where it is
        return {"bytes": c["seqs"] * (2 * row * (c["max_accept"] - 1) / 2
                                      + 4 * (2 + c["max_accept"])), "flops": 0}
    if c["op"] == "copy":
        return {"bytes": c["pairs"] * (2 * row * c["block"] + 8), "flops": 0}
    pages = (c["len_lo"] + c["len_hi"]) / 2 / c["block"]
    grow = c["grow_hi"] / 2 / c["block"]
    # parents' tables read, children's written; each distinct page's count read and written
    # twice, the new pages through the free list
    return {"bytes": 4 * ((c["parents"] + c["children"]) * pages + 4 * c["parents"] * pages
                          + c["children"] * (6 * (1 + grow) + 6)), "flops": 0}


# ---- the definitions in 64 bits -------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        T, half = c["tokens"], c["rotary"] // 2
        theta = s["positions"].cpu().double()[:, None] * s["inv_freq"].cpu()
        turn = torch.polar(torch.full_like(theta, s["factor"]), theta).to(DEV)[:, None]

        def rotated(x):
            y = x.double()
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
                z = torch.complex(y[..., a], y[..., b]) * turn[..., i]
                y[..., a], y[..., b] = z.real, z.imag
            return y

        q, k = rotated(s["q"].clone()), rotated(s["k"].clone()) / s["ks"]
        v = s["v"].double() / s["vs"]
        slots = s["slots"].long()
        pools = []
        for pool, rows in ((s["kb"], k), (s["vb"], v)):
            whole = pool.double()
            whole.view(-1, *whole.shape[2:])[slots] = rows
            pools.append(whole)
        return {"q": q, "k_blocks": pools[0], "v_blocks": pools[1]}
    if c["op"] == "tree":
        q = s["q"]
        T, H, D = q.shape
        G, w = c["kv_heads"], c["window"]
        out = torch.zeros(T, H, D, dtype=torch.float64, device=DEV)
        lse = torch.full((H, T), -math.inf, dtype=torch.float64, device=DEV)
        qsl, lens = s["qsl"].tolist(), s["seq_lens"].tolist()
        masks = s["mask"].cpu().numpy().view(np.uint32)
        places = s["positions"].cpu().numpy()
        for i, n in enumerate(lens):
            a, b = qsl[i], qsl[i + 1]
            ctx = n - (b - a)
            see = np.ones((b - a, n), bool)
            where = np.arange(n)
            where[ctx:] = places[a:b]
            for x in range(b - a):
                for y in range(b - a):
                    see[x, ctx + y] = bool(masks[a + x, y // 32] >> (y % 32) & 1)
                if w:
                    see[x] &= where > places[a + x] - w
            see = torch.from_numpy(see).to(DEV)
            ids = s["tables"][i, :-(-n // BLOCK)].long()
            k = s["kb"].view(torch.uint8)[ids].view(s["kb"].dtype).double().flatten(0, 1)[:n]
            v = s["vb"].view(torch.uint8)[ids].view(s["vb"].dtype).double().flatten(0, 1)[:n]
            for g in range(G):
                rows = q[a:b, g * (H // G):(g + 1) * (H // G)].double()
                x = torch.einsum("thd,kd->thk", rows, k[:, g] * s["ks"]) * s["scale"]
                x = x.masked_fill(~see[:, None], -math.inf)
                l = torch.logsumexp(x, -1)
                p = torch.where(see[:, None], (x - l[..., None]).exp(), 0.0)
                out[a:b, g * (H // G):(g + 1) * (H // G)] = torch.einsum(
                    "thk,kd->thd", p, v[:, g] * s["vs"])
                lse[g * (H // G):(g + 1) * (H // G), a:b] = l.t()
        return (out, lse) if c["lse"] else out
    if c["op"] == "pages":
        return None  # whole numbers
    rows = []  # (page, row) of each moved row and of where it goes
    b = c["block"]
    if c["op"] == "copy":
        rows = [((x, i), (y, i)) for x, y in s["pairs"].tolist() for i in range(b)]
    else:
        tables = s["tables"].tolist()
        for i, (ctx, n) in enumerate(zip(s["ctx"].tolist(), s["count"].tolist())):
            place = lambda p: (tables[i][p // b], p % b)
            rows += [(place(ctx + a), place(ctx + k))
                     for k, a in enumerate(s["accepted"][i, :n].tolist())]
    (sp, si), (dp, di) = (torch.tensor(x, device=DEV).t() for x in zip(*rows))
    pools = []
    for pool in (s["kb"], s["vb"]):
        whole = pool.double()
        whole[dp, di] = whole[sp, si]
        pools.append(whole)
    return tuple(pools)

"""Speculative decoding as a user runs it: prompts cached, a sequence forked, then drafted steps --
grow, slots, rotary caching, tree attention, the accepted rows moved, the rest given back -- with
every step's pools, attention, tables and counts checked against plain 64-bit code; captured in a
graph; tree attention whose waits run out; what the Python calls refuse."""
import contextlib
import os
import random

import pytest
import torch

from tests.spec_reference import (OUT_U, Pages, assert_within, rotate, stored, to_int32, tree,
                                  tree_attention, values)

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
H, HKV, D, BLOCK = 8, 2, 128, 16


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_31_gb300 import binding

    assert binding.pa_device_status() == binding.PA_OK
    return binding


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Server:
    """Four rows over one pool; `kept[r]` holds the K and V rows that row r's positions must have."""

    def __init__(self, pa, kv, seed):
        self.pa, self.kv = pa, kv
        self.scale = 0.25 if kv == E4M3 else 1.0
        self.gen = torch.Generator().manual_seed(seed)
        self.rng = random.Random(seed)
        NB, cols = 90, 20
        ids = list(range(NB))
        self.rng.shuffle(ids)
        self.p = Pages([[0] * cols for _ in range(4)], [0] * 4, [0] * NB, ids, BLOCK)
        self.tables, self.lens = _i32(self.p.tables), _i32(self.p.lens)
        self.refs, self.free, self.count = _i32(self.p.refs), _i32(ids), _i32([NB])
        self.kb, self.vb = (torch.zeros(NB, BLOCK, HKV, D, dtype=kv, device=DEV) for _ in range(2))
        self.inv, self.factor = pa.pa_rope_frequencies(D, base=500000.0, scaling="bands",
                                                       factor=8.0, original_max_position=8192)
        self.kept = [[] for _ in range(4)]

    def books(self):
        return self.refs, self.free, self.count, BLOCK

    def row(self, r, pos):
        b = self.p.tables[r][pos // BLOCK]
        return [x[b, pos % BLOCK].cpu().float() for x in (self.kb, self.vb)]

    def check_pages(self):
        p = self.p
        assert self.lens.tolist() == p.lens and self.refs.tolist() == p.refs
        assert self.free[:self.count.item()].tolist() == p.free
        for r in range(4):
            n = -(-p.lens[r] // BLOCK)
            assert self.tables[r, :n].tolist() == p.tables[r][:n]
            for pos, want in enumerate(self.kept[r][:p.lens[r]]):
                for a, b in zip(self.row(r, pos), want):
                    assert torch.equal(a, b), (r, pos)

    def grow(self, rows, new):
        self.pa.pa_grow_sequences(self.tables, self.lens, _i32(rows), _i32(new), *self.books())
        self.p.grow(rows, new)

    def write(self, rows, first, counts, positions):
        """New tokens of `rows` at cache positions first[i] .., rotated to `positions`."""
        T = sum(counts)
        x = torch.randn(T, (H + 2 * HKV) * D, generator=self.gen).to(BF16).to(DEV)
        q, k, v = (x[:, :H * D].view(T, H, D), x[:, H * D:(H + HKV) * D].view(T, HKV, D),
                   x[:, (H + HKV) * D:].view(T, HKV, D))
        qsl = [0]
        for n in counts:
            qsl.append(qsl[-1] + n)
        at = [f + i for f, n in zip(first, counts) for i in range(n)]
        qsl, tables = _i32(qsl), self.tables[rows].contiguous()
        slots = self.pa.pa_slot_mapping(qsl, _i32(at), tables, BLOCK, self.kb.shape[0])
        q_out = torch.empty(T, H, D, dtype=BF16, device=DEV)
        pos = _i32(positions)
        self.pa.pa_rope_and_cache(q, k, v, q_out, self.kb, self.vb, pos, slots, self.inv,
                                  attn_factor=self.factor, k_scale=self.scale, v_scale=self.scale)
        y, e = rotate(values(q), pos, self.inv, False, self.factor)
        assert_within(q_out, *stored(y, e, BF16), "q")
        y, e = rotate(values(k), pos, self.inv, False, self.factor)
        u = 2.0 ** -24
        y, e = y / self.scale, (e + y.abs() * u) / self.scale
        t, got = 0, []
        for r, f, n in zip(rows, first, counts):
            for i in range(n):
                got.append(self.row(r, f + i))
        assert_within(torch.stack([g[0] for g in got]), *stored(y, e, self.kv), "k")
        y = values(v) / self.scale
        assert_within(torch.stack([g[1] for g in got]), *stored(y, y.abs() * u, self.kv), "v")
        for r, f, n in zip(rows, first, counts):
            self.kept[r][f:] = got[t:t + n]
            t += n
        return q_out, qsl, tables, pos

    def attend(self, q, qsl, tables, rows, pos, mask):
        lens = self.lens[rows].contiguous()
        out, lse = torch.empty_like(q), torch.empty(H, q.shape[0], device=DEV)
        self.pa.pa_tree_attention(q, self.kb, self.vb, out, qsl, lens, pos, mask, tables, D ** -0.5,
                                  lse=lse, k_scale=self.scale, v_scale=self.scale)
        assert self.pa.pa_device_status() == self.pa.PA_OK
        # the reference reads a cache of its own, laid out row after row from `kept`
        own, table, at = [], [], 0
        for r in rows:
            n = self.p.lens[r]
            own += self.kept[r][:n]
            table.append(list(range(at, at + n)))
            at += n
        wide = max(len(t) for t in table)
        kb, vb = (torch.stack([x[i] for x in own])[:, None] for i in (0, 1))
        sc = torch.full((HKV,), self.scale)
        want, wl, ob, lb = tree_attention(
            q, kb, vb, qsl, lens, pos, mask, torch.tensor([t + [0] * (wide - len(t)) for t in table]),
            D ** -0.5, 0, None, sc, sc, weight_u=2.0 ** -11 if self.kv == E4M3 else 2.0 ** -16)
        assert_within(out, want, ob + (want.abs() + ob) * OUT_U[BF16] + 2.0 ** -126, "out")
        assert_within(lse, wl, lb, "lse")

    def drafted_step(self, rows, nodes):
        ctx = [self.p.lens[r] for r in rows]
        self.grow(rows, [c + n for c, n in zip(ctx, nodes)])
        mask, pos, paths = [], [], []
        words = -(-max(nodes) // 32)
        for c, n in zip(ctx, nodes):
            parents, m, ps = tree(self.rng, n, c)
            mask += [w + [0] * (words - len(w)) for w in m]
            pos += ps
            node, path = self.rng.randrange(n), []
            while node >= 0:  # an accepted path: a node and its ancestors
                path.append(node)
                node = parents[node]
            paths.append(path[::-1])
        q, qsl, tables, pos = self.write(rows, ctx, nodes, pos)
        self.attend(q, qsl, tables, rows, pos, _i32(to_int32(mask)).view(-1, words))
        most = max(map(len, paths)) + 1
        self.pa.pa_tree_commit(self.kb, self.vb, tables, _i32(ctx),
                               _i32([p + [-1] * (most - len(p)) for p in paths]),
                               _i32([len(p) for p in paths]))
        new = [c + len(p) for c, p in zip(ctx, paths)]
        self.pa.pa_trim_sequences(self.tables, self.lens, _i32(rows), _i32(new), *self.books())
        self.p.end(rows, new)
        for r, c, p in zip(rows, ctx, paths):
            tail = self.kept[r][c:]
            self.kept[r][c:] = [tail[i] for i in p]
        self.check_pages()


@pytest.mark.parametrize("kv", [BF16, E4M3])
def test_drafted_steps(pa, kv):
    s = Server(pa, kv, 31)
    prompts = [40, 17, 3]
    s.grow([0, 1, 2], prompts)
    q, qsl, tables, pos = s.write([0, 1, 2], [0, 0, 0], prompts,
                                  [i for n in prompts for i in range(n)])
    words = 2
    chain = [[(1 << (i + 1)) - 1 >> (32 * w) & 0xFFFFFFFF for w in range(words)]
             for n in prompts for i in range(n)]
    s.attend(q, qsl, tables, [0, 1, 2], pos, _i32(to_int32(chain)))
    pairs = pa.pa_fork_sequences(s.tables, s.lens, _i32([0]), _i32([3]), *s.books())
    assert [tuple(x) for x in pairs.tolist()] == s.p.fork([0], [3])
    pa.pa_copy_blocks(s.kb, s.vb, pairs)
    s.kept[3] = list(s.kept[0])
    s.check_pages()
    for rows, nodes in (([0, 1, 2, 3], [24, 1, 40, 7]), ([3, 0], [33, 16]), ([0, 1, 2, 3], [5] * 4),
                        ([2, 1], [64, 30])):
        s.drafted_step(rows, nodes)
    pa.pa_free_sequences(s.tables, s.lens, _i32([2, 0, 3, 1]), *s.books())
    s.p.end([2, 0, 3, 1])
    s.check_pages()
    assert not any(s.p.refs) and pa.pa_device_status() == pa.PA_OK


def test_a_drafted_step_in_a_graph(pa):
    """The whole step captured once and replayed on other contents gives what separate calls give."""
    gen = torch.Generator().manual_seed(41)
    rng = random.Random(41)
    NB, n, S = 60, 20, 3

    def start():
        free = torch.arange(NB, dtype=torch.int32, device=DEV)
        refs, lens = torch.zeros_like(free), torch.zeros(S, dtype=torch.int32, device=DEV)
        tables, count = torch.zeros(S, 12, dtype=torch.int32, device=DEV), _i32([NB])
        pool = [torch.zeros(NB, BLOCK, HKV, D, dtype=BF16, device=DEV) for _ in range(2)]
        return dict(tables=tables, lens=lens, refs=refs, free=free, count=count, kb=pool[0],
                    vb=pool[1], out=torch.zeros(S * n, H, D, dtype=BF16, device=DEV))

    rows, qsl = _i32(list(range(S))), _i32([i * n for i in range(S + 1)])
    inp = dict(x=torch.empty(S * n, (H + 2 * HKV) * D, dtype=BF16, device=DEV),
               ctx=_i32([0] * S), grown=_i32([0] * S), at=_i32([0] * S * n), pos=_i32([0] * S * n),
               mask=_i32([[0]] * S * n), acc=_i32([[0] * 4] * S), num=_i32([0] * S),
               kept=_i32([0] * S))
    inv, _ = pa.pa_rope_frequencies(D)
    slots = torch.empty(S * n, dtype=torch.int32, device=DEV)
    q_out = torch.empty(S * n, H, D, dtype=BF16, device=DEV)

    def step(st):
        books = st["refs"], st["free"], st["count"], BLOCK
        pa.pa_grow_sequences(st["tables"], st["lens"], rows, inp["grown"], *books)
        pa.pa_slot_mapping(qsl, inp["at"], st["tables"], BLOCK, NB, out=slots)
        x = inp["x"]
        pa.pa_rope_and_cache(x[:, :H * D].view(-1, H, D), x[:, H * D:(H + HKV) * D].view(-1, HKV, D),
                             x[:, (H + HKV) * D:].view(-1, HKV, D), q_out, st["kb"], st["vb"],
                             inp["pos"], slots, inv)
        pa.pa_tree_attention(q_out, st["kb"], st["vb"], st["out"], qsl, st["lens"], inp["pos"],
                             inp["mask"], st["tables"], D ** -0.5)
        pa.pa_tree_commit(st["kb"], st["vb"], st["tables"], inp["ctx"], inp["acc"], inp["num"])
        pa.pa_trim_sequences(st["tables"], st["lens"], rows, inp["kept"], *books)

    def fill(ctx):
        mask, pos, at, acc, num = [], [], [], [], []
        for c in ctx:
            _, m, p = tree(rng, n, c)
            mask += m
            pos += p
            at += range(c, c + n)
            k = rng.randint(0, 4)
            acc.append(sorted(rng.sample(range(n), k)) + [0] * (4 - k))
            num.append(k)
        kept = [c + k for c, k in zip(ctx, num)]
        for name, v in (("ctx", ctx), ("grown", [c + n for c in ctx]), ("at", at), ("pos", pos),
                        ("mask", to_int32(mask)), ("acc", acc), ("num", num), ("kept", kept)):
            inp[name].copy_(_i32(v))
        inp["x"].copy_(torch.randn(inp["x"].shape, generator=gen))
        return kept

    a, b = start(), start()
    g = torch.cuda.CUDAGraph()
    fill([0] * S)
    step(start())
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(b)
    ctx = [0] * S
    for _ in range(5):
        nxt = fill(ctx)
        step(a)
        g.replay()
        for name in a:
            assert torch.equal(a[name].view(torch.uint8), b[name].view(torch.uint8)), name
        ctx = nxt
    assert a["lens"].tolist() == ctx and pa.pa_device_status() == pa.PA_OK


@contextlib.contextmanager
def _stalled_waits(ns):
    os.environ["PA_DEBUG_STALL_NS"] = str(ns)
    try:
        yield
    finally:
        del os.environ["PA_DEBUG_STALL_NS"]


@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("nodes", [[5, 9, 2], [24, 40, 3]])
@pytest.mark.parametrize("columns", [100, 1200])
def test_tree_attention_timeout_unwinds_and_the_device_stays_usable(pa, kv, nodes, columns):
    """PA_DEBUG_STALL_NS points the softmax waits at a barrier that nothing signals, each wait
    bounded at 20 ms: the status says so, nothing is written, the next call gives the same bits
    (short tables: clusters that join their states; long ones: planned shares)."""
    gen = torch.Generator().manual_seed(51)
    S, T, ctx, NB = len(nodes), sum(nodes), 1500, 330
    q = torch.randn(T, H, D, generator=gen).to(BF16).to(DEV)
    kb, vb = (torch.randn(NB, BLOCK, HKV, D, generator=gen).to(kv).to(DEV) for _ in range(2))
    qsl = _i32([sum(nodes[:i]) for i in range(S + 1)])
    lens = _i32([ctx + n for n in nodes])
    tables = torch.zeros(S, columns, dtype=torch.int32, device=DEV)
    tables[:, :100] = torch.randperm(NB, generator=gen)[:S * 100].int().view(S, 100).to(DEV)
    mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (T, 2), generator=gen).int().to(DEV)
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)

    def call():
        out, lse = torch.full_like(q, 7.0), torch.full((H, T), 7.0, device=DEV)
        pa.pa_tree_attention(q, kb, vb, out, qsl, lens, pos, mask, tables, D ** -0.5, lse=lse)
        return out, lse

    ref = call()
    assert pa.pa_device_status() == pa.PA_OK
    with _stalled_waits(20_000_000):
        for _ in range(2):
            got = call()
            assert pa.pa_device_status() == pa.PA_ETIMEOUT
            assert all(bool((x == 7.0).all()) for x in got), "a timed-out call wrote output"
    again = call()
    assert pa.pa_device_status() == pa.PA_OK
    for x, y in zip(again, ref):
        assert torch.equal(x, y)


def test_python_refusals(pa):
    q = torch.zeros(4, H, D, dtype=BF16, device=DEV)
    k, v = (torch.zeros(4, HKV, D, dtype=BF16, device=DEV) for _ in range(2))
    kb, vb = (torch.zeros(3, BLOCK, HKV, D, dtype=BF16, device=DEV) for _ in range(2))
    i4, i2, i1 = _i32([0, 1, 2, 3]), _i32([0, 4]), _i32([4])
    inv, _ = pa.pa_rope_frequencies(D)
    mask, table = _i32([[1]] * 4), _i32([[0]])

    def rope(**kw):
        a = dict(q=q, k=k, v=v, q_out=q.clone(), k_blocks=kb, v_blocks=vb, positions=i4,
                 slot_mapping=i4, inv_freq=inv)
        a.update(kw)
        with pytest.raises((ValueError, KeyError, TypeError)):
            pa.pa_rope_and_cache(**a)

    for kw in (dict(q=q.cpu()), dict(k=k.cpu()), dict(positions=i4.long()), dict(positions=i4[:3]),
               dict(slot_mapping=i4.cpu()), dict(slot_mapping=_i32([0, 0, 1, 0, 2, 0, 3, 0])[::2]),
               dict(inv_freq=inv.float()), dict(inv_freq=inv.cpu()), dict(q=None), dict(q_out=None),
               dict(q_out=q.float()), dict(v=v.float()), dict(v=v[:3]), dict(q=q[:, :, :64]),
               dict(k=k.transpose(0, 1)), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
               dict(k_blocks=kb.float()), dict(k_blocks=kb[:, :, :1]), dict(k=k.half(), v=v.half()),
               dict(k_scales=torch.ones(3, device=DEV)), dict(v_scales=torch.ones(2))):
        rope(**kw)

    def attend(**kw):
        a = dict(q=q, k_blocks=kb, v_blocks=vb, out=q.clone(), query_start_loc=i2, seq_lens=i1,
                 positions=i4, tree_mask=mask, block_tables=table, scale=1.0)
        a.update(kw)
        with pytest.raises((ValueError, KeyError, TypeError)):
            pa.pa_tree_attention(**a)

    for kw in (dict(q=q.cpu()), dict(out=q.float()), dict(out=q[:3]), dict(k_blocks=kb[..., :64]),
               dict(v_blocks=vb.float()), dict(tree_mask=mask[:3]), dict(tree_mask=mask.long()),
               dict(tree_mask=mask.view(-1)), dict(seq_lens=i4), dict(block_tables=table.view(-1)),
               dict(block_tables=_i32([[0], [0]])), dict(positions=i4[:2]),
               dict(sinks=torch.zeros(H - 1, device=DEV)), dict(sinks=torch.zeros(H)),
               dict(lse=torch.zeros(4, H, device=DEV)), dict(workspace=torch.zeros(9)),
               dict(q=q.half(), out=q.half()), dict(k_scales=torch.ones(HKV + 1, device=DEV)),
               dict(query_start_loc=torch.tensor([0, 4], dtype=torch.int32))):
        attend(**kw)
    refs, free, count = _i32([1, 0, 0]), _i32([1, 2, 0]), _i32([2])
    lens = _i32([4])
    for bad in (lambda: pa.pa_copy_blocks(kb, vb, _i32([0, 1])),
                lambda: pa.pa_copy_blocks(kb, vb.float(), _i32([[0, 1]])),
                lambda: pa.pa_copy_blocks(kb, vb, _i32([[0, 1]]).long()),
                lambda: pa.pa_tree_commit(kb, vb, table, i2, _i32([[0]]), i1),
                lambda: pa.pa_tree_commit(kb, vb, table, i1, _i32([0]), i1),
                lambda: pa.pa_fork_sequences(table, lens, i1, i2, refs, free, count, 16),
                lambda: pa.pa_fork_sequences(table, lens, i1, i1, refs, free, count, 16,
                                             block_pairs=_i32([0, 0])),
                lambda: pa.pa_grow_sequences(table, i2, i1, i1, refs, free, count, 16),
                lambda: pa.pa_trim_sequences(table, lens, i1, i1, refs, free[:2], count, 16),
                lambda: pa.pa_free_sequences(table, lens, i1, refs, free, i2, 16),
                lambda: pa.pa_free_sequences(table, lens.cpu(), i1, refs, free, count, 16)):
        with pytest.raises((ValueError, KeyError, TypeError)):
            bad()
    assert pa.pa_device_status() == pa.PA_OK

"""Eviction of keys by their accumulated attention weight, and a cache kept at a bounded size by all
the calls that belong to it."""
import math
import random

import pytest
import torch

from tests import bounded_reference as ref
from tests.spec_reference import U32, assert_within, stored, values

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_31_gb300 import binding

    return binding


class Cache:
    def __init__(self, lens, Hkv, D, bs=16, kv=BF16, seed=0, extra=5, ties=False):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // bs) for n in lens]
        num = sum(need) + extra
        ids = torch.randperm(num, generator=g)
        self.tables = torch.full((len(lens), max(max(need), 1) + 2), -3, dtype=torch.int32)
        at = 0
        for s, k in enumerate(need):
            self.tables[s, :k] = ids[at:at + k].int()
            at += k
        # every byte of the pools is its own, so a wrong row cannot pass for another
        size = {BF16: 2, F32: 4, E4M3: 1}[kv]
        raw = lambda: torch.randint(0, 256, (num, bs, Hkv, D * size), dtype=torch.uint8, generator=g)
        self.kv = kv
        self.kb, self.vb = (raw().view(kv).cuda() for _ in range(2))
        self.lens, self.bs, self.Hkv = list(lens), bs, Hkv
        self.w = torch.rand(len(lens), Hkv, max(lens) + 3, generator=g)
        if ties:
            self.w = (self.w * 3).floor()
            self.w[self.w == 0] *= -1  # both zeros
        self.tables = self.tables.cuda()
        self.w = self.w.cuda()

    def slots(self, s, n):
        j = torch.arange(n)
        return self.tables[s].cpu().long()[j // self.bs] * self.bs + j % self.bs

    def expected(self, new, first, recent, weights=True):
        bytes_of = lambda t: t.cpu().view(torch.uint8).view(t.shape[0] * self.bs, self.Hkv, -1).clone()
        kb, vb = bytes_of(self.kb), bytes_of(self.vb)
        slots = [self.slots(s, n) for s, n in enumerate(self.lens)]
        rows = [[[int(x) for x in slots[s]] for _ in range(self.Hkv)] for s in range(len(self.lens))]
        w = self.w.cpu().tolist() if weights else None
        ref.evict(rows, w, self.lens, new, first, recent)
        k2, v2 = kb.clone(), vb.clone()
        for s, n in enumerate(self.lens):
            for g in range(self.Hkv):
                frm = torch.tensor(rows[s][g], dtype=torch.long)
                k2[slots[s], g], v2[slots[s], g] = kb[frm, g], vb[frm, g]
        return k2, v2, torch.tensor(w) if weights else None

    def check(self, pa, new, first=0, recent=0, weights=True, **kw):
        k2, v2, w2 = self.expected(new, first, recent, weights)
        before = self.w.clone()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        pa.pa_evict_keys(self.kb, self.vb, self.tables, i32(self.lens), i32(new),
                         self.w if weights else None, first, recent, **kw)
        assert pa.pa_device_status() == pa.PA_OK
        for got, want in ((self.kb, k2), (self.vb, v2)):
            # rows behind a new end may hold anything: they are compared up to it
            got = got.cpu().view(torch.uint8).view(want.shape)
            gone = torch.zeros(want.shape[0], dtype=torch.bool)
            for s, n in enumerate(self.lens):
                gone[self.slots(s, n)[min(new[s], n):]] = True
            assert torch.equal(got[~gone], want[~gone])
            assert torch.equal(got[gone], want[gone])  # (nothing is written there)
        if weights:
            assert torch.equal(self.w.cpu().nan_to_num(77.0), w2.nan_to_num(77.0))
        else:
            assert torch.equal(self.w, before)


@pytest.mark.parametrize("first,recent", [(0, 0), (4, 0), (0, 7), (4, 16), (1, 1), (300, 0), (0, 300),
                                          (50, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("ties", [False, True])
def test_rules(pa, first, recent, ties):
    lens = [100, 64, 1, 33, 257, 0, 16, 40]
    new = [60, 64, 0, 32, 17, 0, 15, 90]
    Cache(lens, 3, 64, seed=first % 11 + recent % 7, ties=ties).check(pa, new, first, recent)


@pytest.mark.parametrize("kv", [BF16, F32, E4M3])
@pytest.mark.parametrize("D,bs", [(128, 16), (64, 32), (40, 8), (1, 1), (7, 5), (256, 16), (96, 16)])
def test_types_and_sizes(pa, kv, D, bs):
    Cache([90, 200, 31], 2, D, bs, kv, seed=D).check(pa, [45, 190, 31], 3, 20)


@pytest.mark.parametrize("n,new", [(2, 1), (17, 16), (1040, 1024), (4097, 2000), (5000, 4999),
                                   (9000, 1000), (40000, 20000)])
@pytest.mark.parametrize("ties", [False, True])
def test_lengths(pa, n, new, ties):
    Cache([n], 1, 16, seed=n, ties=ties).check(pa, [new], 4, min(64, n // 8))


@pytest.mark.parametrize("recent", [0, 1, 500, 900, 1500])
def test_the_recent_rows_move_up_by_little_or_much(pa, recent):
    for new in (1990, 1500, 700):
        Cache([2000, 1995], 2, 128, seed=recent).check(pa, [new, new], 2, recent)


def test_without_weights(pa):
    Cache([100, 40, 70], 2, 64, seed=1).check(pa, [30, 40, 60], 4, 20, weights=False)


def test_values_that_are_not_ordinary(pa):
    c = Cache([300], 2, 32, seed=2)
    w = c.w
    w[0, 0, 5::7] = float("nan")
    w[0, 0, 1::9] = float("inf")
    w[0, 0, 3::11] = -float("inf")
    w[0, 1, :] = -w[0, 1, :]
    w[0, 1, ::5] = 0.0
    w[0, 1, 1::5] = -0.0
    w[0, 1, 2::50] = 1e-45
    c.check(pa, [120], 3, 10)
    c = Cache([300], 1, 32, seed=3)
    c.w[:] = float("nan")
    c.check(pa, [120], 3, 10)


def test_misaligned_pools(pa):
    c = Cache([90, 200], 2, 64, seed=4)
    for off in (1, 4):
        for name in ("kb", "vb"):
            t = getattr(c, name)
            moved = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")[off:].view(t.shape)
            moved.copy_(t)
            setattr(c, name, moved)
        c.check(pa, [45, 190], 3, 20)


def test_far_blocks(pa):
    """Rows past 2^31 elements of a pool."""
    Hkv, D = 8, 128
    num = 2 ** 31 // (16 * Hkv * D) + 40
    kb, vb = (torch.empty(num, 16, Hkv, D, dtype=BF16, device="cuda") for _ in range(2))
    c = Cache([300, 90], Hkv, D, seed=5)
    blocks = c.kb.shape[0]
    kb[num - blocks:], vb[num - blocks:] = c.kb, c.vb
    tables = torch.where(c.tables >= 0, c.tables + (num - blocks), c.tables)
    lens, new = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([300, 90], [150, 80]))
    w = c.w.clone()
    pa.pa_evict_keys(kb, vb, tables, lens, new, w, 4, 30)
    c.check(pa, [150, 80], 4, 30)
    bits = lambda t: t.view(torch.int16)
    assert torch.equal(bits(kb[num - blocks:]), bits(c.kb)) and torch.equal(w, c.w)
    assert torch.equal(bits(vb[num - blocks:]), bits(c.vb))


@pytest.mark.parametrize("what", ["id", "id_high", "length", "length_table", "new", "weights"])
def test_refusals_leave_everything(pa, what):
    c = Cache([100, 64, 90], 2, 64, seed=6)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    new = torch.tensor([50, 64, 80], dtype=torch.int32, device="cuda")
    w = c.w
    if what.startswith("id"):
        c.tables[2, 3] = -1 if what == "id" else c.kb.shape[0]
    elif what == "length":
        lens[1] = -1
    elif what == "length_table":
        lens[0] = 16 * c.tables.shape[1] + 1
    elif what == "new":
        new[2] = -1
    else:
        w = w[..., :99].contiguous()
    before = [t.clone() for t in (c.kb, c.vb, w)]
    pa.pa_evict_keys(c.kb, c.vb, c.tables, lens, new, w, 4, 10)
    assert pa.pa_device_status() == pa.PA_EINVAL
    for t, b in zip((c.kb, c.vb, w), before):
        assert torch.equal(t.view(torch.uint8), b.view(torch.uint8))


def test_tables_of_sequences_that_stay_are_not_looked_at(pa):
    c = Cache([100, 64], 2, 64, seed=7)
    c.tables[1] = -1
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    pa.pa_evict_keys(c.kb, c.vb, c.tables, lens, torch.tensor([50, 64], dtype=torch.int32, device="cuda"),
                     c.w, 4, 10)
    assert pa.pa_device_status() == pa.PA_OK


def test_streams_and_graphs(pa):
    cs = [Cache([700, 30, 260], 2, 64, seed=8), Cache([500, 400, 410], 2, 64, seed=9)]
    new = [[300, 30, 250], [490, 100, 400]]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    want = [c.expected(n, 4, 32) for c, n in zip(cs, new)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    args = [(c.kb, c.vb, c.tables, i32(c.lens), i32(n), c.w, 4, 32) for c, n in zip(cs, new)]
    saved = [[t.clone() for t in (c.kb, c.vb, c.w)] for c in cs]
    torch.cuda.synchronize()

    def right():
        torch.cuda.synchronize()
        assert pa.pa_device_status() == pa.PA_OK
        for c, (k2, v2, w2) in zip(cs, want):
            assert torch.equal(c.kb.cpu().view(torch.uint8).view(k2.shape), k2)
            assert torch.equal(c.vb.cpu().view(torch.uint8).view(v2.shape), v2)
            assert torch.equal(c.w.cpu(), w2)

    def restore():
        for c, old in zip(cs, saved):
            for t, o in zip((c.kb, c.vb, c.w), old):
                t.view(torch.uint8).copy_(o.view(torch.uint8))
        torch.cuda.synchronize()

    for a, st in zip(args, streams):
        pa.pa_evict_keys(*a, stream=st)
    right()
    restore()
    graphs = []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.pa_evict_keys(*a)
        graphs.append(g)
    for _ in range(2):
        restore()
        for g in graphs:
            g.replay()
        right()


def test_a_cache_kept_at_a_bounded_size(pa):
    """Steps of a serving loop: new rows are cached at rotated positions, attention adds up the keys'
    weights, sequences past their budget are cut and their pages given back."""
    torch.manual_seed(0)
    rng = random.Random(0)
    S, H, Hkv, D, bs, budget, cut = 3, 8, 2, 128, 16, 96, 64
    first, recent = 4, 16
    num, width = 40, 12
    kb, vb = (torch.full((num, bs, Hkv, D), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    tables = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    lens = i32([0] * S)
    refs, free, count = i32([0] * num), torch.arange(num, dtype=torch.int32, device="cuda"), i32([num])
    pages = (refs, free, count, bs)
    rows = i32(list(range(S)))
    w = torch.zeros(S, Hkv, width * bs, device="cuda")
    inv_freq, factor = pa.pa_rope_frequencies(D, base=10000.0)
    seen = [0] * S  # tokens so far: their rotary positions
    have = [0] * S  # keys in the cache
    model_k = [[[] for _ in range(Hkv)] for _ in range(S)]  # the rows that should be there
    model_v = [[[] for _ in range(Hkv)] for _ in range(S)]
    evictions = 0
    for step in range(30):
        new = [rng.choice([1, 1, 1, 5, 20]) if step else 50 for _ in range(S)]
        T = sum(new)
        grown = [a + b for a, b in zip(have, new)]
        pa.pa_grow_sequences(tables, lens, rows, i32(grown), *pages)
        qsl = i32([0] + [sum(new[:i + 1]) for i in range(S)])
        cache_pos = i32([p for s in range(S) for p in range(have[s], grown[s])])
        rope_pos = i32([p for s in range(S) for p in range(seen[s], seen[s] + new[s])])
        slots = pa.pa_slot_mapping(qsl, cache_pos, tables, bs, num)
        q, k, v = (torch.randn(T, n, D, device="cuda").to(BF16) for n in (H, Hkv, Hkv))
        pa.pa_rope_and_cache(q, k, v, q, kb, vb, rope_pos, slots, inv_freq, attn_factor=factor)
        rk, rv = kb.view(-1, Hkv, D)[slots.long()].cpu(), vb.view(-1, Hkv, D)[slots.long()].cpu()
        t = 0
        for s in range(S):
            for _ in range(new[s]):
                for g in range(Hkv):
                    model_k[s][g].append(rk[t, g])
                    model_v[s][g].append(rv[t, g])
                t += 1
        out = torch.empty(T, H, D, dtype=BF16, device="cuda")
        before = w.clone()
        pa.pa_attention_key_weights(q, kb, vb, out, qsl, lens, cache_pos, tables, w, 1 / math.sqrt(D))
        assert pa.pa_device_status() == pa.PA_OK
        # the same over the model's dense rows
        most = max(grown)
        dk = torch.zeros(S, most, Hkv, D, dtype=BF16)
        dv = torch.zeros_like(dk)
        for s in range(S):
            for g in range(Hkv):
                dk[s, :grown[s], g] = torch.stack(model_k[s][g])
                dv[s, :grown[s], g] = torch.stack(model_v[s][g])
        want = ref.window_attention(q, dk, dv, qsl, lens, cache_pos,
                                    torch.arange(S, dtype=torch.int32)[:, None], 1 / math.sqrt(D),
                                    weights_len=w.shape[2])
        y, bound = stored(want["out"], want["out_b"], BF16)
        assert_within(out, y, bound, "out")
        total = before.cpu().double() + want["weights"]
        assert_within(w, total, want["weights_b"] + 2 * U32 * total, "weights")
        cutting = [cut if n > budget else n for n in grown]
        keys = [[list(range(n)) for _ in range(Hkv)] for n in grown]
        summed = [[row[:n].tolist() for row in heads] for n, heads in zip(grown, values(w))]
        ref.evict(keys, summed, grown, cutting, first, recent)
        pa.pa_evict_keys(kb, vb, tables, lens, i32(cutting), w, first, recent)
        pa.pa_trim_sequences(tables, lens, rows, i32(cutting), *pages)
        assert pa.pa_device_status() == pa.PA_OK
        for s in range(S):
            seen[s] += new[s]
            evictions += grown[s] > cutting[s]
            have[s] = cutting[s]
            j = torch.arange(have[s])
            slot = tables[s].cpu().long()[j // bs] * bs + j % bs
            for g in range(Hkv):
                for pool, model in ((kb, model_k), (vb, model_v)):
                    model[s][g] = [model[s][g][x] for x in keys[s][g][:have[s]]]
                    assert torch.equal(pool.view(-1, Hkv, D)[slot, g].cpu(), torch.stack(model[s][g]))
                assert values(w[s, g, :grown[s]]).tolist() == summed[s][g]
        assert lens.tolist() == have
        assert int(count) == num - sum(-(-n // bs) for n in have)
    assert evictions > 5

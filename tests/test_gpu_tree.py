"""pa_tree_attention against softmax attention in 64 bits: tree masks, ragged batches, GQA groups,
head sizes, types, windows, sinks, scales, empty rows, contexts from nothing to long ones."""
import random

import pytest
import torch

from tests.spec_reference import OUT_U, assert_within, to_int32, tree, tree_attention

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_31_gb300 import binding

    assert binding.pa_device_status() == binding.PA_OK
    return binding


class Batch:
    def __init__(self, nodes, ctx, H, Hkv, D, src=BF16, kv=BF16, bs=16, seed=0, words=None,
                 sharp=1.0):
        gen = torch.Generator().manual_seed(seed)
        rng = random.Random(seed)
        T = sum(nodes)
        words = words or max(1, -(-max(nodes) // 32))
        mask, pos = [], []
        for n, c in zip(nodes, ctx):
            _, m, p = tree(rng, n, c)
            mask += [r + [0] * (words - len(r)) for r in m]
            pos += p
        lens = [n + c for n, c in zip(nodes, ctx)]
        need = [-(-x // bs) for x in lens]
        NB = sum(need) + 2
        ids = torch.randperm(NB, generator=gen)
        tables = torch.zeros(len(nodes), max(1, max(need)), dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            tables[s, :n] = ids[at:at + n].int()
            at += n
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        self.q = (torch.randn(T, H, D, generator=gen) * sharp).to(src).to(DEV)
        m = 8.0 if kv == E4M3 else 1.0
        self.kb = (torch.randn(NB, bs, Hkv, D, generator=gen) * m).to(kv).to(DEV)
        self.vb = (torch.randn(NB, bs, Hkv, D, generator=gen) * m).to(kv).to(DEV)
        self.qsl = i32([sum(nodes[:i]) for i in range(len(nodes) + 1)])
        self.lens, self.pos = i32(lens), i32(pos)
        self.mask = i32(to_int32(mask)).view(T, words)
        self.tables = tables.to(DEV)
        self.scale = D ** -0.5 / m
        self.nodes, self.ctx, self.bs = nodes, ctx, bs

    def call(self, pa, window=0, lse=True, **kw):
        T, H, _ = self.q.shape
        out = torch.full_like(self.q, float("nan"))
        ls = torch.full((H, T), float("nan"), device=DEV) if lse else None
        pa.pa_tree_attention(self.q, self.kb, self.vb, out, self.qsl, self.lens, self.pos,
                             self.mask, self.tables, self.scale, sliding_window=window, lse=ls,
                             **kw)
        return out, ls

    def check(self, pa, window=0, sinks=None, k_scale=1.0, v_scale=1.0, k_scales=None,
              v_scales=None):
        Hkv = self.kb.shape[2]
        out, lse = self.call(pa, window=window, sinks=sinks, k_scale=k_scale, v_scale=v_scale,
                             k_scales=k_scales, v_scales=v_scales)
        assert pa.pa_device_status() == pa.PA_OK
        ks = k_scales if k_scales is not None else torch.full((Hkv,), k_scale)
        vs = v_scales if v_scales is not None else torch.full((Hkv,), v_scale)
        # e4m3 pools on the tensor cores: weights in f16
        u = 2.0 ** -11 if self.kb.dtype == E4M3 else 2.0 ** -16
        want, wl, ob, lb = tree_attention(self.q, self.kb, self.vb, self.qsl, self.lens, self.pos,
                                          self.mask, self.tables, self.scale, window, sinks, ks,
                                          vs, weight_u=u,
                                          q_u=2.0 ** -17 if self.kb.dtype == E4M3 else 0.0,
                                          weight_min=2.0 ** -32 if self.kb.dtype == E4M3 else 0.0)
        assert_within(out, want, ob + (want.abs() + ob) * OUT_U[self.q.dtype] + 2.0 ** -126, "out")
        assert_within(lse, wl, lb, "lse")
        kw = dict(window=window, sinks=sinks, k_scale=k_scale, v_scale=v_scale, k_scales=k_scales,
                  v_scales=v_scales)
        out2, _ = self.call(pa, lse=False, **kw)
        assert torch.equal(out.view(torch.uint8), out2.view(torch.uint8))
        # small calls over short tables are one launch of clusters: over long tables (whose
        # entries past the sequences are not read) they take the planned shares
        tables = self.tables
        if tables.shape[1] < 1100:
            self.tables = torch.full((tables.shape[0], 1100), -9, dtype=torch.int32, device=DEV)
            self.tables[:, :tables.shape[1]] = tables
            o, ls = self.call(pa, **kw)
            self.tables = tables
            assert pa.pa_device_status() == pa.PA_OK
            assert_within(o, want, ob + (want.abs() + ob) * OUT_U[self.q.dtype] + 2.0 ** -126, "out")
            assert_within(ls, wl, lb, "lse")
        return out, lse


RAGGED = ([1, 5, 32, 17, 0, 3], [0, 700, 33, 15, 40, 16])


@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2), (10, 2), (7, 1), (16, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_groups_ragged(pa, H, Hkv, D):
    Batch(*RAGGED, H, Hkv, D, seed=H + D).check(pa)


@pytest.mark.parametrize("D", [32, 80, 96, 100, 6, 256])
def test_other_head_sizes(pa, D):
    Batch([9, 1, 30], [100, 0, 257], 4, 2, D, seed=D).check(pa)


@pytest.mark.parametrize("src,kv", [(F32, F32), (F32, BF16), (BF16, F32), (F32, E4M3), (BF16, E4M3)])
@pytest.mark.parametrize("D", [64, 128])
def test_types(pa, src, kv, D):
    Batch(*RAGGED, 8, 2, D, src=src, kv=kv, seed=5).check(pa)


@pytest.mark.parametrize("bs", [1, 5, 32, 64])
def test_block_sizes(pa, bs):
    Batch([9, 1, 30], [100, 0, 257], 4, 2, 128, bs=bs, seed=bs).check(pa)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 100, 250])
def test_tree_sizes(pa, n):
    Batch([n, 1, n], [130, 500, 3], 8, 2, 128, seed=n).check(pa)


@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 111, 112, 127, 128, 129, 255, 256, 1000, 4095])
def test_context_lengths(pa, ctx):
    Batch([8], [ctx], 8, 2, 128, seed=ctx).check(pa)
    Batch([33, 4], [ctx, 60], 8, 2, 128, seed=ctx).check(pa)


@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("window", [1, 2, 5, 16, 100, 129, 100000])
def test_windows(pa, window, kv):
    Batch([12, 40, 3], [300, 90, 0], 8, 2, 128, kv=kv, seed=window).check(pa, window=window)


@pytest.mark.parametrize("kv", [BF16, E4M3, F32])
def test_the_widest_windows_hide_nothing(pa, kv):
    """A key's distance behind the window's edge must not leave 32 bits."""
    src = F32 if kv == F32 else BF16
    b = Batch([12, 40, 3], [300, 90, 0], 8, 2, 128, src=src, kv=kv, seed=29)
    want, _ = b.check(pa)
    b.pos.zero_()
    for window in (2 ** 31 - 1, 2 ** 31 - 200, 2 ** 30):
        out, _ = b.check(pa, window=window)
        assert torch.equal(out, want)


def test_long_context_many_pieces(pa):
    """One sequence over the whole GPU: every item is cut into many pieces."""
    Batch([7], [9001], 8, 1, 128, seed=1).check(pa)
    Batch([40], [9001], 16, 1, 128, seed=2).check(pa)
    Batch([40], [6001], 16, 1, 128, kv=E4M3, seed=3).check(pa, k_scale=0.5, v_scale=0.25)
    Batch([7], [3001], 4, 1, 64, src=F32, kv=F32, seed=4).check(pa)


@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("n", [7, 30, 45])
def test_many_tiles_to_a_cta(pa, n, kv):
    """Shares of dozens of key tiles over several items: the copies' ring goes round many times."""
    ctx = [700, 9000, 1, 4000, 129, 2500, 6000, 900]
    Batch([n, 1, n, 3, n, 2, n, n], [c * 4 for c in ctx], 16, 4, 128, kv=kv, seed=n).check(
        pa, k_scale=0.25, v_scale=0.5)


def test_many_sequences(pa):
    rng = random.Random(7)
    n = [rng.randint(0, 12) for _ in range(300)]
    Batch(n, [rng.randint(0, 90) for _ in n], 4, 2, 64, seed=9).check(pa)
    n = [1] * 1100
    Batch(n, [rng.randint(0, 40) for _ in n], 2, 1, 128, seed=10).check(pa, window=9)


def test_sinks(pa):
    sinks = torch.tensor([0.5, -float("inf"), 4.0, -3.0, 0.0, 30.0, 1.0, -60.0], device=DEV)
    Batch(*RAGGED, 8, 2, 128, seed=11).check(pa, sinks=sinks)
    Batch([5], [5000], 8, 2, 128, seed=12).check(pa, sinks=sinks, window=50)


def test_scales(pa):
    for kv in (BF16, E4M3):
        b = Batch(*RAGGED, 8, 2, 128, kv=kv, seed=13)
        b.check(pa, k_scale=0.5, v_scale=3.0)
        b.check(pa, k_scales=torch.tensor([0.25, 1.5], device=DEV),
                v_scales=torch.tensor([2.0, 0.125], device=DEV))
        b.check(pa, v_scales=torch.tensor([2.0, 0.125], device=DEV), k_scale=0.75)


def test_sharp_and_negative_scales(pa):
    """Large scores (one key takes all the weight) and a softmax scale of the other sign."""
    b = Batch([20, 6], [300, 900], 8, 2, 128, seed=14, sharp=30.0)
    b.check(pa)
    b.scale = -b.scale
    b.check(pa)
    b.scale = 0.0
    b.check(pa)


def test_uneven_queries_over_e4m3_pools(pa):
    """Rows of q with one large element, tiny rows, rows of zeros; scales at both ends."""
    b = Batch([30, 5], [300, 90], 8, 2, 128, kv=E4M3, seed=27)
    b.q *= 2.0 ** -9
    b.q[::2, ::3, 5] = 40.0
    b.q[3], b.q[7] = 0.0, b.q[7] * 2.0 ** -100
    b.check(pa)
    b.q[11] *= 2.0 ** 90
    b.check(pa, k_scale=2.0 ** -90, v_scale=2.0 ** 20)
    b.q[11] = 0.0
    b.scale = 2.0 ** -40
    b.check(pa, k_scale=2.0 ** -40)
    b.mask[9] = 0
    b.check(pa, window=3)


def test_many_small_weights(pa):
    """One key far above thousands whose weights are small but make up the whole output."""
    for kv, gap in ((E4M3, 26.0), (E4M3, 30.0), (BF16, 30.0)):
        S, ctx = 16, 1900
        b = Batch([4] * S, [ctx] * S, 8, 8, 128, kv=kv, seed=34)
        b.q[:] = 0.0
        b.q[:, :, 0] = 1.0
        b.kb[:, :, :, 0] = 0.0
        b.vb[:] = 8.0
        for s in range(S):
            b.kb[b.tables[s, 3], 5, :, 0] = 32.0
            b.vb[b.tables[s, 3], 5] = 0.0
        b.scale = gap * 0.6931471805599453 / 32.0  # the other weights are 2^-gap of the largest
        out, _ = b.check(pa)
        assert abs(float(out[0, 0, 0]) / (ctx * 2.0 ** -gap * 8.0) - 1.0) < 2.0 ** -6


def test_rows_that_see_nothing(pa):
    """Nodes without a bit and without a context, between ordinary ones."""
    for kv in (BF16, E4M3):
        b = Batch([6, 40, 3], [0, 0, 50], 8, 2, 128, kv=kv, seed=15)
        b.mask[2] = 0
        b.mask[6:30] = 0
        out, lse = b.check(pa)
        assert not out[2].any() and torch.isinf(lse[:, 6:30]).all()
    b = Batch([4], [0], 2, 2, 64, src=F32, kv=F32, seed=16)
    b.mask[:] = 0
    out, lse = b.check(pa)
    assert not out.any()


def test_any_mask_is_taken(pa):
    """Bits need not form a tree: random ones, nodes behind the token, bits past the nodes."""
    b = Batch([33, 12, 64], [40, 0, 300], 8, 2, 128, seed=17)
    gen = torch.Generator().manual_seed(18)
    b.mask.copy_(torch.randint(-2 ** 31, 2 ** 31 - 1, b.mask.shape, generator=gen).int())
    b.check(pa)
    b.check(pa, window=30)


def test_wider_masks_than_needed(pa):
    Batch([5, 33], [70, 10], 4, 2, 128, words=7, seed=19).check(pa)


def test_shared_pages(pa):
    """Forked sequences read the same context blocks."""
    b = Batch([6, 6, 6], [160, 160, 160], 8, 2, 128, seed=20)
    b.tables[1, :10] = b.tables[0, :10]
    b.tables[2, :10] = b.tables[0, :10]
    b.check(pa)


@pytest.mark.parametrize("kv", [BF16, E4M3, F32])
def test_garbage_behind_the_sequence_and_in_masked_keys(pa, kv):
    """Rows past the last position, and K rows of nodes that nobody sees, may hold anything."""
    src = F32 if kv == F32 else BF16
    b = Batch([20, 7], [101, 130], 8, 2, 128, src=src, kv=kv, seed=21)
    nan = float("nan")
    ok, ol = b.call(pa)
    hidden = [3, 11]
    for h in hidden:
        b.mask[:20] &= ~(1 << h)
    want = b.check(pa)
    for s, n in enumerate([121, 137]):
        last = b.tables[s, (n - 1) // 16]
        for pool in (b.kb, b.vb):
            x = pool.float()
            x[last, (n - 1) % 16 + 1:] = nan
            pool.copy_(x.to(kv))
    x = b.kb.float()
    for h in hidden:
        p = 101 + h
        x[b.tables[0, p // 16], p % 16] = nan
    b.kb.copy_(x.to(kv))
    got = b.call(pa)
    for g, w in zip(got, want):
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))
    assert pa.pa_device_status() == pa.PA_OK


def test_a_chain_is_causal_attention(pa):
    """A tree without branches gives what pa_varlen_forward gives for the same tokens."""
    b = Batch([9, 24], [200, 41], 8, 2, 128, seed=22)
    m, t = [], 0
    for n in b.nodes:
        m += [[(1 << (i + 1)) - 1] for i in range(n)]
    b.mask.copy_(torch.tensor(to_int32(m), dtype=torch.int32))
    b.pos.copy_(torch.cat([torch.arange(c, c + n) for n, c in zip(b.nodes, b.ctx)]).int())
    for window in (0, 37):
        out, lse = b.check(pa, window=window)
        ref, rl = torch.empty_like(out), torch.empty_like(lse)
        pa.pa_varlen_forward(b.q, b.kb, b.vb, ref, b.qsl, b.lens, b.pos, b.tables, b.scale,
                             sliding_window=window, lse=rl)
        assert pa.pa_device_status() == pa.PA_OK
        assert torch.allclose(lse, rl, atol=2e-4, rtol=0)
        assert torch.allclose(out.float(), ref.float(), atol=1e-3, rtol=2 ** -6)


def _bad(pa, b, change, **kw):
    out, lse = torch.zeros_like(b.q), torch.zeros(b.q.shape[1], b.q.shape[0], device=DEV)
    saved = {k: getattr(b, k).clone() for k in ("qsl", "lens", "pos", "tables", "mask")}
    change(b)
    pa.pa_tree_attention(b.q, b.kb, b.vb, out, b.qsl, b.lens, b.pos, b.mask, b.tables, b.scale,
                         lse=lse, **kw)
    assert pa.pa_device_status() == pa.PA_EINVAL
    assert not out.any() and not lse.any()
    for k, v in saved.items():
        getattr(b, k).copy_(v)


@pytest.mark.parametrize("kv,wide", [(BF16, False), (BF16, True), (E4M3, False), (E4M3, True),
                                     (F32, False)])
def test_bad_metadata_writes_nothing(pa, kv, wide):
    b = Batch([5, 40, 3], [60, 20, 0], 8, 2, 128, src=F32 if kv == F32 else BF16, kv=kv, seed=23)
    if wide:  # (long tables: the planned shares)
        b.tables = torch.cat([b.tables, b.tables.new_zeros(3, 1100)], 1).contiguous()
    NB = b.kb.shape[0]

    def put(name, at, value):
        def f(x):
            getattr(x, name)[at] = value
        return f

    _bad(pa, b, put("tables", (0, 2), NB))
    _bad(pa, b, put("tables", (1, 3), -1))
    _bad(pa, b, put("lens", 1, 39))          # fewer positions than nodes
    _bad(pa, b, put("lens", 2, 16 * b.tables.shape[1] + 1))  # beyond the table
    _bad(pa, b, put("lens", 0, -5))
    _bad(pa, b, put("qsl", 0, 1))
    _bad(pa, b, put("qsl", 1, 50))
    _bad(pa, b, put("qsl", 3, 47))
    _bad(pa, b, put("qsl", 3, 1000))
    _bad(pa, b, put("pos", 3, -1), sliding_window=8)
    _bad(pa, b, lambda x: None, k_scales=torch.tensor([1.0, 0.0], device=DEV))
    _bad(pa, b, lambda x: None, v_scales=torch.tensor([float("inf"), 1.0], device=DEV))
    b.mask = b.mask[:, :1].contiguous()      # 40 nodes need two words
    _bad(pa, b, lambda x: None)
    # a table entry past the sequence's blocks is not read
    b = Batch([5, 40, 3], [60, 20, 0], 8, 2, 128, seed=23)
    b.tables[2, 1:] = -9
    b.check(pa)


def test_empty_calls(pa):
    b = Batch([5], [60], 8, 2, 128, seed=24)
    none = torch.empty(0, 8, 128, dtype=BF16, device=DEV)
    i0 = torch.empty(0, dtype=torch.int32, device=DEV)
    pa.pa_tree_attention(none, b.kb, b.vb, none.clone(), torch.zeros(1, dtype=torch.int32, device=DEV),
                         i0, i0, i0.view(0, 1), torch.empty(0, 4, dtype=torch.int32, device=DEV), 1.0)
    pa.pa_tree_attention(none, b.kb, b.vb, none.clone(), torch.zeros(3, dtype=torch.int32, device=DEV),
                         b.lens.repeat(2), i0, i0.view(0, 1), b.tables.repeat(2, 1), 1.0)
    assert pa.pa_device_status() == pa.PA_OK


def test_streams_graphs_and_repeats(pa):
    """Equal bits on every call, on another stream, and replayed with new lengths."""
    b = Batch([24, 24, 24], [900, 130, 2000], 8, 2, 128, seed=25)
    first, _ = b.check(pa)
    n = pa.pa_tree_attention_workspace_size(3, 72, 8, 2, 128, b.tables.shape[1], 16)
    for _ in range(3):
        ws = torch.randint(0, 255, (n,), dtype=torch.uint8, device=DEV)  # any workspace contents
        out, _ = b.call(pa, workspace=ws)
        assert torch.equal(out, first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(first)
    pa.pa_tree_attention(b.q, b.kb, b.vb, out, b.qsl, b.lens, b.pos, b.mask, b.tables, b.scale,
                         stream=s, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_tree_attention(b.q, b.kb, b.vb, out, b.qsl, b.lens, b.pos, b.mask, b.tables,
                             b.scale, workspace=ws)
    out.zero_()
    g.replay()
    assert torch.equal(out, first)
    b.lens -= 500 * (b.lens > 900).int()
    out.zero_()
    g.replay()
    want, _ = b.check(pa)
    assert torch.equal(out, want)


def test_calls_on_two_streams_at_once(pa):
    """Small and large calls, each stream with a workspace of its own."""
    cases = [Batch([8], [700], 32, 8, 128, seed=30), Batch([30] * 6, [2500] * 6, 32, 8, 128, seed=31),
             Batch([7] * 5, [400] * 5, 8, 2, 128, kv=E4M3, seed=32),
             Batch([16] * 20, [900] * 20, 32, 8, 128, kv=E4M3, seed=33)]
    want = [b.call(pa, lse=False)[0] for b in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(40):
        for k, s in enumerate(streams):
            j = (i + 2 * k + k * i) % 4
            b = cases[j]
            with torch.cuda.stream(s):
                out = torch.empty_like(b.q)
                if i % 2:  # the current stream, or given by name
                    pa.pa_tree_attention(b.q, b.kb, b.vb, out, b.qsl, b.lens, b.pos, b.mask, b.tables,
                                         b.scale)
            if i % 2 == 0:
                pa.pa_tree_attention(b.q, b.kb, b.vb, out, b.qsl, b.lens, b.pos, b.mask, b.tables,
                                     b.scale, stream=s)
            got[k].append((j, out))
    torch.cuda.synchronize()
    assert pa.pa_device_status() == pa.PA_OK
    for j, out in got[0] + got[1]:
        assert torch.equal(out, want[j])


@pytest.mark.parametrize("S,n,ctx", [(16, 8, 4000), (3, 40, 3000), (64, 4, 600)])
def test_hundreds_of_calls(pa, S, n, ctx):
    """Every one of many calls over all SMs gives the first one's bits: no wait runs out, no buffer
    is taken before it is free, whatever the copies' and products' timing."""
    for kv in (BF16, E4M3):
        b = Batch([n] * S, [ctx - 3 * i for i in range(S)], 32, 8, 128, kv=kv, seed=28)
        T = S * n
        ws = torch.empty(pa.pa_tree_attention_workspace_size(S, T, 32, 8, 128, b.tables.shape[1], 16),
                         dtype=torch.uint8, device=DEV)
        want, _ = b.call(pa, lse=False, workspace=ws)
        out = torch.empty_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(20):
                pa.pa_tree_attention(b.q, b.kb, b.vb, out, b.qsl, b.lens, b.pos, b.mask, b.tables,
                                     b.scale, workspace=ws)
        for _ in range(30):
            out.zero_()
            g.replay()
            assert torch.equal(out, want)
        assert pa.pa_device_status() == pa.PA_OK


def test_unaligned_and_small_workspace(pa):
    b = Batch([5], [60], 8, 2, 128, seed=26)
    n = pa.pa_tree_attention_workspace_size(1, 5, 8, 2, 128, b.tables.shape[1], 16)
    ws = torch.empty(n + 256, dtype=torch.uint8, device=DEV)
    for bad in (ws[8:8 + n], ws[:n - 256]):
        with pytest.raises(pa.PaError):
            b.call(pa, workspace=bad)
    # q, out and pools off a 16-byte boundary take the general kernel
    def shifted(t):
        raw = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape)
        return raw.copy_(t)
    want, wl = b.check(pa)
    b.q, b.kb, b.vb = shifted(b.q), shifted(b.kb), shifted(b.vb)
    got, gl = b.check(pa)

"""Attention that adds up the weight each cached key receives, against 64 bits."""
import pytest
import torch

from tests import bounded_reference as ref
from tests.spec_reference import U32, assert_within, stored
from tests.test_gpu_window import BF16, BIG, CHUNKS, E4M3, F32, MIXED, roundings

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_31_gb300 import binding

    return binding


def check(pa, b, observed=0, window=0, first=0, sinks=None, scales=(1.0, 1.0), lse=False, room=9,
          per_head=None, v_bits=0.0):
    L = int(b.lens.max()) + room
    ks = torch.full((b.Hkv,), scales[0]) if per_head is None else per_head[0].cpu()
    vs = torch.full((b.Hkv,), scales[1]) if per_head is None else per_head[1].cpu()
    want = ref.window_attention(b.q, b.kb, b.vb, b.qsl, b.lens, b.positions, b.tables, b.scale, window,
                                first, sinks, ks, vs, observed=observed, weights_len=L, **roundings(b))
    start = torch.rand(len(b.seqs), b.Hkv, L, device="cuda")
    w = start.clone()
    extra = {"k_scale": scales[0], "v_scale": scales[1]} if per_head is None else {
        "k_scales": per_head[0], "v_scales": per_head[1]}
    pa.pa_attention_key_weights(*b.args(), w, b.scale, observed_tokens=observed, sliding_window=window,
                                first_tokens=first, sinks=sinks, lse=b.lse if lse else None, **extra)
    assert pa.pa_device_status() == pa.PA_OK
    y, bound = stored(want["out"], want["out_b"] + v_bits, b.out.dtype)
    assert_within(b.out, y, bound, "out")
    if lse:
        assert_within(b.lse, want["lse"], want["lse_b"], "lse")
    total = start.cpu().double() + want["weights"]
    assert_within(w, total, want["weights_b"] + 2 * U32 * total, "key weights")
    # (keys that nobody counted sees, and what lies behind a sequence's end, keep their bits)
    idle = want["weights"] == 0
    assert torch.equal(w.cpu()[idle], start.cpu()[idle])
    return w, start


@pytest.mark.parametrize("observed", [0, 1, 5, 32, BIG])
@pytest.mark.parametrize("src,kv", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
def test_mixed_batch(pa, src, kv, observed):
    b = ref.Batch(MIXED, 8, 2, 128, src=src, kv=kv, seed=observed % 89)
    b.poison_unread(0, 0)
    check(pa, b, observed, scales=(0.125, 0.25) if kv == E4M3 else (1.0, 1.0), lse=observed == 5)


@pytest.mark.parametrize("window,first", [(1, 0), (7, 3), (100, 4), (129, 140), (BIG, 5)])
@pytest.mark.parametrize("kv", [BF16, E4M3, F32])
def test_behind_a_window(pa, kv, window, first):
    b = ref.Batch(MIXED, 8, 2, 128, src=F32 if kv == F32 else BF16, kv=kv, seed=window % 83)
    b.poison_unread(window, first)
    check(pa, b, 20, window, first, scales=(0.125, 0.25) if kv == E4M3 else (1.0, 1.0))


@pytest.mark.parametrize("H,Hkv", [(4, 4), (5, 1), (32, 8), (34, 2), (64, 1), (160, 1), (1, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads(pa, H, Hkv, D):
    b = ref.Batch([(0, 1), (700, 1), (90, 33), (260, 1), (0, 70)], H, Hkv, D, seed=H)
    check(pa, b)


@pytest.mark.parametrize("src,kv", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, E4M3), (BF16, E4M3),
                                    (F32, F32)])
@pytest.mark.parametrize("D,bs", [(40, 16), (256, 16), (128, 8), (65, 5), (1, 1), (128, 16)])
def test_other_sizes(pa, src, kv, D, bs):
    b = ref.Batch([(0, 1), (200, 1), (40, 9), (77, 0)], 6, 3, D, bs=bs, src=src, kv=kv, seed=D + bs)
    check(pa, b, 3, scales=(0.5, 0.25) if kv == E4M3 else (1.0, 1.0))


@pytest.mark.parametrize("kv", [BF16, E4M3, F32])
def test_decoding_batch(pa, kv):
    seqs = [((37 * i * i) % 2900, 1) for i in range(40)]
    b = ref.Batch(seqs, 8, 2, 128, src=F32 if kv == F32 else BF16, kv=kv, seed=3)
    check(pa, b, scales=(0.125, 0.25) if kv == E4M3 else (1.0, 1.0))


@pytest.mark.parametrize("ctx", [0, 15, 16, 127, 128, 1023, 5000, 20000])
@pytest.mark.parametrize("n", [1, 2, 16])
def test_one_sequence(pa, ctx, n):
    b = ref.Batch([(ctx, n)], 8, 2, 128, seed=ctx + n)
    check(pa, b)


@pytest.mark.parametrize("kv", [BF16, E4M3])
def test_long_chunk(pa, kv):
    b = ref.Batch([(1700, 900), (0, 1300), (2100, 1)], 8, 2, 128, kv=kv, seed=8)
    for observed in (0, 77):
        check(pa, b, observed, scales=(0.125, 0.25) if kv == E4M3 else (1.0, 1.0))


@pytest.mark.parametrize("observed,window,first", [(0, 0, 0), (25, 0, 0), (0, 300, 4), (1, 64, 70)])
def test_many_chunks(pa, observed, window, first):
    """Enough rows for the prefill kernel, with decoding sequences beside it."""
    b = ref.Batch(CHUNKS, 64, 8, 128, seed=observed)
    b.poison_unread(window, first)
    check(pa, b, observed, window, first, lse=observed == 25, v_bits=2.0 ** -25)


@pytest.mark.parametrize("kv", [BF16, E4M3])
def test_sinks_and_head_scales(pa, kv):
    b = ref.Batch(MIXED, 8, 2, 128, kv=kv, seed=5)
    sinks = torch.randn(8, device="cuda") * 3
    sinks[1], sinks[2] = -float("inf"), 40.0
    per_head = (torch.tensor([0.11, 0.3], device="cuda"), torch.tensor([0.5, 0.02], device="cuda"))
    check(pa, b, sinks=sinks, per_head=per_head)


def test_weights_of_a_row_sum_to_its_heads(pa):
    """Without sinks every counted (token, head) gives a weight of 1 in all."""
    b = ref.Batch([(4000, 1), (600, 200), (0, 64)], 32, 8, 128, seed=6)
    w = torch.zeros(3, 8, 4001, device="cuda")
    pa.pa_attention_key_weights(*b.args(), w, b.scale)
    assert pa.pa_device_status() == pa.PA_OK
    # (1024 rows of 4 heads at most, each off by some 2^-18)
    want = torch.tensor([1.0, 200.0, 64.0], device="cuda")[:, None] * 4
    assert ((w.double().sum(-1) / want - 1).abs() < 2.0 ** -16).all()


def test_equal_calls_give_equal_bits(pa):
    for seqs in ([(2000, 1), (900, 1), (37, 1)], [(2000, 90), (900, 1), (0, 400)]):
        b = ref.Batch(seqs, 32, 8, 128, seed=40)
        first = None
        for _ in range(20):
            w = torch.zeros(3, 8, 2100, device="cuda")
            pa.pa_attention_key_weights(*b.args(), w, b.scale)
            first = w if first is None else first
            assert torch.equal(w, first)
    assert pa.pa_device_status() == pa.PA_OK


def test_streams_and_graphs(pa):
    bs = [ref.Batch([(900, 1), (500, 1), (70, 1)], 8, 2, 128, seed=20),
          ref.Batch([(600, 40), (0, 300), (1000, 1)], 8, 2, 128, seed=21)]
    ws = [torch.zeros(3, 2, 1001, device="cuda") for _ in bs]
    run = lambda b, w, **kw: pa.pa_attention_key_weights(*b.args(), w, b.scale, **kw)
    one = []
    for b in bs:
        w = torch.zeros(3, 2, 1001, device="cuda")
        run(b, w)
        one.append(w)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for b, w, st in zip(bs, ws, streams):
        run(b, w, stream=st)
    torch.cuda.synchronize()
    for w, o in zip(ws, one):
        assert torch.equal(w, o)
    graphs = []
    for b, w in zip(bs, ws):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(b, w)
        graphs.append(g)
    for w in ws:
        w.zero_()
    for _ in range(4):  # (powers of two keep the sums exact multiples)
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert pa.pa_device_status() == pa.PA_OK
    for w, o in zip(ws, one):
        assert ((w - 4 * o).abs() <= 4 * U32 * 4 * o).all()


def test_lengths_past_the_weights_are_refused(pa):
    for seqs in ([(300, 1), (20, 1)], [(300, 40), (20, 1)]):
        b = ref.Batch(seqs, 8, 2, 128, seed=30)
        n = sum(seqs[0])
        w = torch.full((2, 2, n - 1), 0.5, device="cuda")
        pa.pa_attention_key_weights(*b.args(), w, b.scale, lse=b.lse)
        assert pa.pa_device_status() == pa.PA_EINVAL
        assert (w == 0.5).all() and (b.out == 7.0).all() and (b.lse == 7.0).all()
        w = torch.full((2, 2, n), 0.5, device="cuda")
        b.tables[1, 1] = b.kb.shape[0]
        pa.pa_attention_key_weights(*b.args(), w, b.scale, lse=b.lse)
        assert pa.pa_device_status() == pa.PA_EINVAL
        assert (w == 0.5).all() and (b.out == 7.0).all() and (b.lse == 7.0).all()


def test_rows_with_nan_scores_spoil_what_they_see(pa):
    b = ref.Batch([(300, 1), (40, 8), (70, 1)], 8, 2, 128, seed=12)
    b.q[3, 5, 7] = float("nan")
    w = torch.zeros(3, 2, 301, device="cuda")
    pa.pa_attention_key_weights(*b.args(), w, b.scale)
    assert pa.pa_device_status() == pa.PA_OK
    bad = w.isnan()
    p = int(b.positions[3])
    assert bad[1, 1, :p + 1].all() and int(bad.sum()) == p + 1

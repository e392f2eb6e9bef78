"""Attention behind a sliding window whose first tokens stay visible, against 64 bits."""
import pytest
import torch

from tests import bounded_reference as ref
from tests.spec_reference import OUT_U, OUT_MIN, assert_within, stored

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_31_gb300 import binding

    return binding


def roundings(b, tc=None):
    """What the kernels round softmax weights and q to (see spec_reference.tree_attention)."""
    many = b.T * (b.H // b.Hkv) // 256 * b.Hkv >= 304  # (the prefill kernel)
    if b.kb.dtype == E4M3 and b.q.dtype == BF16:
        if many:
            # weights as below; q's f16 rows, their largest element in [2^14, 2^15), keep 2^-25
            return {"weight_u": 2.0 ** -11, "weight_min": 2.0 ** -25, "q_u": 2.0 ** -39}
        return {"weight_u": 2.0 ** -11, "q_u": 2.0 ** -17, "weight_min": 2.0 ** -32}
    if many:
        # the prefill kernel: one f16 weight, at least 2^-8 for the row's largest (its reference may lie
        # 8 powers of two above): below its normal range half its smallest step, 2^-25
        return {"weight_u": 2.0 ** -11, "weight_min": 2.0 ** -25}
    return {"weight_u": 2.0 ** -16}


def check(pa, b, window, first, sinks=None, scales=(1.0, 1.0), per_head=None, lse=True, v_bits=0.0,
          **kw):
    ks = torch.full((b.Hkv,), scales[0]) if per_head is None else per_head[0].cpu()
    vs = torch.full((b.Hkv,), scales[1]) if per_head is None else per_head[1].cpu()
    want = ref.window_attention(b.q, b.kb, b.vb, b.qsl, b.lens, b.positions, b.tables, b.scale,
                                window, first, sinks, ks, vs, **roundings(b))
    extra = {"k_scale": scales[0], "v_scale": scales[1]} if per_head is None else {
        "k_scales": per_head[0], "v_scales": per_head[1]}
    pa.pa_window_attention(*b.args(), b.scale, sliding_window=window, first_tokens=first, sinks=sinks,
                           lse=b.lse if lse else None, **extra, **kw)
    assert pa.pa_device_status() == pa.PA_OK
    # v_bits: f16's rounding of V below its normal range (half its smallest step)
    y, bound = stored(want["out"], want["out_b"] + v_bits, b.out.dtype)
    assert_within(b.out, y, bound, "out")
    if lse:
        assert_within(b.lse, want["lse"], want["lse_b"], "lse")
    return want


MIXED = [(0, 1), (130, 1), (0, 17), (300, 37), (5, 0), (1000, 1), (511, 130), (15, 1), (16, 2)]


@pytest.mark.parametrize("window,first", [(0, 0), (0, 5), (1, 0), (1, 1), (7, 3), (16, 16), (100, 4),
                                          (128, 130), (257, 1), (4096, 4), (BIG, BIG), (33, BIG),
                                          (BIG, 0), (64, 0)])
@pytest.mark.parametrize("src,kv", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
def test_mixed_batch(pa, src, kv, window, first):
    b = ref.Batch(MIXED, 8, 2, 128, src=src, kv=kv, seed=window % 97)
    scales = (0.125, 0.25) if kv == E4M3 else (1.0, 1.0)
    b.poison_unread(window, first)
    check(pa, b, window, first, scales=scales)


@pytest.mark.parametrize("H,Hkv", [(4, 4), (5, 1), (32, 8), (12, 4), (34, 2), (64, 1), (160, 1), (1, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads(pa, H, Hkv, D):
    b = ref.Batch([(0, 1), (700, 1), (90, 33), (260, 1), (0, 70)], H, Hkv, D, seed=H)
    b.poison_unread(50, 20)
    check(pa, b, 50, 20)


@pytest.mark.parametrize("src,kv", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, E4M3), (BF16, E4M3),
                                    (F32, F32)])
@pytest.mark.parametrize("D,bs", [(40, 16), (256, 16), (128, 8), (64, 32), (65, 5), (1, 1), (128, 16)])
def test_other_sizes(pa, src, kv, D, bs):
    b = ref.Batch([(0, 1), (200, 1), (40, 9), (77, 0)], 6, 3, D, bs=bs, src=src, kv=kv, seed=D + bs)
    b.poison_unread(21, 6)
    check(pa, b, 21, 6, scales=(0.5, 0.25) if kv == E4M3 else (1.0, 1.0))


@pytest.mark.parametrize("kv", [BF16, E4M3, F32])
def test_decoding_batch(pa, kv):
    seqs = [((37 * i * i) % 2900, 1) for i in range(40)]
    b = ref.Batch(seqs, 8, 2, 128, src=F32 if kv == F32 else BF16, kv=kv, seed=3)
    b.poison_unread(300, 17)
    check(pa, b, 300, 17, scales=(0.125, 0.25) if kv == E4M3 else (1.0, 1.0))


@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 127, 128, 1023, 5000])
@pytest.mark.parametrize("n", [1, 2, 4, 16])
def test_one_sequence(pa, ctx, n):
    b = ref.Batch([(ctx, n)], 8, 2, 128, seed=ctx + n)
    b.poison_unread(200, 3)
    check(pa, b, 200, 3)


@pytest.mark.parametrize("kv", [BF16, E4M3])
def test_sinks_and_head_scales(pa, kv):
    b = ref.Batch(MIXED, 8, 2, 128, kv=kv, seed=5)
    sinks = torch.randn(8, device="cuda") * 3
    sinks[1], sinks[2] = -float("inf"), 40.0
    per_head = (torch.tensor([0.11, 0.3], device="cuda"), torch.tensor([0.5, 0.02], device="cuda"))
    check(pa, b, 90, 4, sinks=sinks, per_head=per_head)


def test_long_chunk(pa):
    b = ref.Batch([(3000, 1500), (0, 700), (9000, 1), (2100, 1)], 8, 2, 128, seed=8)
    b.poison_unread(1024, 4)
    check(pa, b, 1024, 4)


CHUNKS = [(300, 700), (0, 500), (1000, 1), (2000, 2), (40, 3), (900, 20), (7, 0), (0, 1)]


@pytest.mark.parametrize("window,first", [(0, 0), (1, 1), (300, 4), (128, 130), (64, 0), (BIG, 7)])
@pytest.mark.parametrize("H,Hkv", [(64, 8), (16, 16)])
def test_many_chunks(pa, H, Hkv, window, first):
    """Enough rows for the prefill kernel, with decoding sequences beside it."""
    seqs = CHUNKS if H == 64 else [(c, 4 * n if n > 100 else n) for c, n in CHUNKS]
    b = ref.Batch(seqs, H, Hkv, 128, seed=window % 91)
    b.poison_unread(window, first)
    sinks = torch.randn(H, device="cuda") if first == 4 else None
    check(pa, b, window, first, sinks=sinks, v_bits=2.0 ** -25)


def test_values_past_f16(pa):
    """V values that f16 cannot hold: the items that meet them are done again.  (Values above 2^100 are
    outside the call's domain: the sums before the division are fp32, weights up to 2^8 times V over all
    keys, so 3e38 = 2^127.8 overflows there with the first such key.)"""
    b = ref.Batch(CHUNKS, 64, 8, 128, seed=3)
    b.vb.view(-1, 8, 128)[5::97, 3, 10] = 1e30
    b.vb.view(-1, 8, 128)[7::89, 5, 100] = -1e6
    check(pa, b, 200, 4)


def test_no_window_is_causal_attention(pa):
    b = ref.Batch([(100, 30), (0, 200), (512, 1), (64, 1)], 8, 2, 64, seed=9)
    b.tables.clamp_(min=0)
    pa.pa_window_attention(*b.args(), b.scale)
    out = torch.empty_like(b.out)
    pa.pa_varlen_forward(b.q, b.kb, b.vb, out, b.qsl, b.lens, b.positions, b.tables, b.scale)
    assert pa.pa_device_status() == pa.PA_OK
    # both round once to bf16, and are off by less than a sixteenth of a step before that
    assert ((b.out.float() - out.float()).abs() <= out.float().abs() * 2.0 ** -7 + 2e-3).all()


def test_positions_may_repeat_and_skip(pa):
    b = ref.Batch([(200, 6), (50, 3)], 4, 2, 128, seed=11)
    b.positions[:] = torch.tensor([3, 3, 150, 180, 180, 205, 0, 51, 52], dtype=torch.int32)
    check(pa, b, 40, 2)


def test_rows_with_nan_scores(pa):
    """NaN in q gives NaN in its own row; no other row changes."""
    b = ref.Batch([(300, 1), (40, 8), (70, 1)], 8, 2, 128, seed=12)
    want = torch.empty_like(b.out)
    pa.pa_window_attention(b.q, b.kb, b.vb, want, *b.args()[4:], b.scale, sliding_window=64, first_tokens=2)
    b.q[3, 5, 7] = float("nan")
    pa.pa_window_attention(*b.args(), b.scale, sliding_window=64, first_tokens=2, lse=b.lse)
    assert pa.pa_device_status() == pa.PA_OK
    assert b.out[3, 5].isnan().all() and b.lse[5, 3].isnan()
    keep = torch.ones(b.T, 8, dtype=torch.bool)
    keep[3, 5] = False
    assert torch.equal(b.out[keep], want[keep])
    assert b.lse.t()[keep].isfinite().all()


def test_far_blocks(pa):
    """Blocks past 2^31 elements of a pool, and past 2^32 bytes."""
    H, Hkv, D = 8, 8, 128
    num = 2 ** 31 // (16 * Hkv * D) + 40
    kb = torch.empty(num, 16, Hkv, D, dtype=BF16, device="cuda")
    vb = torch.empty_like(kb)
    for n, ctx in ((1, 290), (40, 100)):
        b = ref.Batch([(ctx, n), (33, n)], H, Hkv, D, seed=13)
        blocks = b.kb.shape[0]
        kb[num - blocks:], vb[num - blocks:] = b.kb, b.vb
        tables = torch.where(b.tables >= 0, b.tables + (num - blocks), b.tables)
        out = torch.empty_like(b.out)
        pa.pa_window_attention(b.q, kb, vb, out, b.qsl, b.lens, b.positions, tables, b.scale,
                               sliding_window=100, first_tokens=4)
        check(pa, b, 100, 4)
        assert torch.equal(out, b.out)


def test_misaligned(pa):
    """Tensors off a 16-byte boundary take the general kernel."""
    b = ref.Batch(MIXED, 8, 2, 128, seed=14)
    for name in ("q", "kb", "vb", "out"):
        t = getattr(b, name)
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        moved = flat[1:].view(t.shape)
        moved.copy_(t)
        setattr(b, name, moved)
        check(pa, b, 70, 5)
        setattr(b, name, t)


def test_scale_not_positive(pa):
    b = ref.Batch([(100, 1), (30, 20)], 4, 2, 128, seed=15)
    for scale in (-0.1, 0.0):
        b.scale = scale
        check(pa, b, 40, 4)


def test_streams_and_graphs(pa):
    """Calls on two streams at once, and captured calls replayed over changed inputs."""
    bs = [ref.Batch([(900, 1), (500, 1), (70, 1)], 8, 2, 128, seed=20),
          ref.Batch([(600, 40), (0, 300), (1000, 1)], 8, 2, 128, seed=21)]
    run = lambda b, **kw: pa.pa_window_attention(*b.args(), b.scale, sliding_window=256, first_tokens=4,
                                                 lse=b.lse, **kw)
    want = []
    for b in bs:
        run(b)
        torch.cuda.synchronize()
        want.append((b.out.clone(), b.lse.clone()))
        b.out.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, st in zip(bs, streams):
            run(b, stream=st)
    torch.cuda.synchronize()
    for b, (o, l) in zip(bs, want):
        assert torch.equal(b.out, o) and torch.equal(b.lse, l)
    graphs = []
    for b in bs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(b)
            run(b)
        graphs.append(g)
    for b in bs:
        b.q.copy_(b.q.flip(0))
        b.out.zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert pa.pa_device_status() == pa.PA_OK
    for b in bs:
        got = b.out.clone()
        run(b)
        assert torch.equal(got, b.out)


def refused(pa, b, window=64, first=4):
    b.out.fill_(7.0)
    b.lse.fill_(7.0)
    pa.pa_window_attention(*b.args(), b.scale, sliding_window=window, first_tokens=first, lse=b.lse)
    assert pa.pa_device_status() == pa.PA_EINVAL
    assert (b.out == 7.0).all() and (b.lse == 7.0).all()


@pytest.mark.parametrize("seqs", [[(300, 1), (200, 1)], [(300, 1), (200, 30)], [(10, 1)]])
@pytest.mark.parametrize("kv", [BF16, F32])
def test_device_refusals(pa, seqs, kv):
    fresh = lambda: ref.Batch(seqs, 8, 2, 128, src=BF16, kv=kv, seed=30)
    last = len(seqs) - 1
    b = fresh()
    end = (b.seqs[last][0] + b.seqs[last][1] - 1) // 16
    for bad in (-1, b.kb.shape[0]):
        b = fresh()
        b.tables[last, end] = bad
        refused(pa, b)
        b = fresh()
        b.tables[last, 0] = bad  # the first tokens' block
        refused(pa, b)
    for bad in (0, -3, 16 * b.tables.shape[1] + 1):
        b = fresh()
        b.lens[last] = bad
        refused(pa, b)
    for bad in (-1, sum(b.seqs[last])):
        b = fresh()
        b.positions[-1] = bad
        refused(pa, b)
    if seqs[last][1] > 2:
        b = fresh()
        b.positions[-2] = b.positions[-3] - 1
        refused(pa, b)
    b = fresh()
    b.qsl[0] = 1
    refused(pa, b)
    b = fresh()
    b.qsl[-1] -= 1
    refused(pa, b)
    b = fresh()
    b.qsl[-1] += 1
    refused(pa, b)
    if last:
        b = fresh()
        b.qsl[1] = -1
        refused(pa, b)
        b = fresh()
        b.qsl[1] = 100000
        refused(pa, b)
    b = fresh()
    bad = torch.tensor([1.0, float("nan")], device="cuda")
    pa.pa_window_attention(*b.args(), b.scale, sliding_window=64, first_tokens=4, lse=b.lse, v_scales=bad)
    assert pa.pa_device_status() == pa.PA_EINVAL
    assert (b.out == 7.0).all() and (b.lse == 7.0).all()
    b = fresh()
    check(pa, b, 64, 4)


def test_empty(pa):
    b = ref.Batch([(20, 0), (5, 0)], 4, 2, 128)
    b.tables.fill_(-1)
    pa.pa_window_attention(*b.args(), b.scale, sliding_window=8)
    assert pa.pa_device_status() == pa.PA_OK


def test_equal_calls_give_equal_bits(pa):
    for seqs in ([(2000, 1), (900, 1), (37, 1)], [(2000, 90), (900, 1), (0, 400)]):
        b = ref.Batch(seqs, 32, 8, 128, seed=40)
        pa.pa_window_attention(*b.args(), b.scale, sliding_window=700, first_tokens=4)
        want = b.out.clone()
        for _ in range(50):
            b.out.zero_()
            pa.pa_window_attention(*b.args(), b.scale, sliding_window=700, first_tokens=4)
            assert torch.equal(b.out, want)
    assert pa.pa_device_status() == pa.PA_OK

"""pa_rope_and_cache against rotation in 64 bits: both pair layouts, parts of the head, strided
rows, every type, far positions, odd sizes, in place, on other streams and in a captured graph."""
import pytest
import torch

from tests.spec_reference import assert_within, rotate, stored, values

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


def _rows(gen, T, H, Hkv, D, dtype, pad):
    """q, k, v as views of one fused product with `pad` extra elements per token."""
    w = (H + 2 * Hkv) * D
    x = torch.randn(T, w + pad, generator=gen).to(dtype).to(DEV)
    return (x[:, :H * D].view(T, H, D), x[:, H * D:(H + Hkv) * D].view(T, Hkv, D),
            x[:, (H + Hkv) * D:w].view(T, Hkv, D))


def _case(pa, T, H, Hkv, D, R, src, kv, interleaved, *, bs=16, pad=0, max_pos=5000, ks=1.0,
          vs=1.0, k_scales=None, v_scales=None, factor=1.0, seed=0, negative=False):
    gen = torch.Generator().manual_seed(seed)
    q, k, v = _rows(gen, T, H, Hkv, D, src, pad)
    NB = -(-T // bs) + 3
    kb = (torch.randn(NB, bs, Hkv, D, generator=gen)).to(kv).to(DEV)
    vb = (torch.randn(NB, bs, Hkv, D, generator=gen)).to(kv).to(DEV)
    slots = torch.randperm(NB * bs, generator=gen)[:T].int().to(DEV)
    pos = torch.randint(-max_pos if negative else 0, max_pos, (T,), generator=gen).int().to(DEV)
    inv, _ = pa.pa_rope_frequencies(R, base=500000.0)
    kb0, vb0 = kb.clone(), vb.clone()
    q_out = torch.full((T, H, D), float("nan"), dtype=src, device=DEV)
    pa.pa_rope_and_cache(q, k, v, q_out, kb, vb, pos, slots, inv, interleaved=interleaved,
                         attn_factor=factor, k_scale=ks, v_scale=vs, k_scales=k_scales,
                         v_scales=v_scales)
    assert pa.pa_device_status() == pa.PA_OK
    y, e = rotate(values(q), pos, inv, interleaved, factor)
    assert_within(q_out, *stored(y, e, src), "q")
    y, e = rotate(values(k), pos, inv, interleaved, factor)
    kdiv = torch.full((Hkv, 1), ks, dtype=torch.float64) if k_scales is None else values(k_scales)[:, None]
    vdiv = torch.full((Hkv, 1), vs, dtype=torch.float64) if v_scales is None else values(v_scales)[:, None]
    u = 2.0 ** -24
    want_k, want_v = values(kb0), values(vb0)
    bk, bv = torch.zeros_like(want_k), torch.zeros_like(want_v)
    sl = slots.cpu().long()
    y, e = y / kdiv, (e + y.abs() * u) / kdiv
    want_k.view(-1, Hkv, D)[sl], bk.view(-1, Hkv, D)[sl] = stored(y, e, kv)
    y = values(v) / vdiv
    want_v.view(-1, Hkv, D)[sl], bv.view(-1, Hkv, D)[sl] = stored(y, y.abs() * u, kv)
    assert_within(kb, want_k, bk, "k_blocks")
    assert_within(vb, want_v, bv, "v_blocks")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (64, 64), (64, 16), (80, 80), (80, 20),
                                 (256, 256), (6, 6), (7, 4)])
def test_layouts_and_head_sizes(pa, D, R, interleaved):
    if D % 2 and interleaved:
        pytest.skip("refused (see test_refusals)")
    _case(pa, 37, 6, 2, D, R, BF16, BF16, interleaved, pad=3 if D == 6 else 0, seed=D + R)


@pytest.mark.parametrize("src,kv", [(BF16, BF16), (BF16, E4M3), (BF16, F32), (F32, F32),
                                    (F32, BF16), (F32, E4M3)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types(pa, src, kv, interleaved):
    _case(pa, 33, 8, 2, 128, 128, src, kv, interleaved, ks=0.25, vs=0.125, seed=3)


@pytest.mark.parametrize("T", [1, 2, 15, 64, 2048, 2049, 5003])
def test_token_counts(pa, T):
    _case(pa, T, 4, 1, 64, 64, BF16, BF16, False, seed=T)


@pytest.mark.parametrize("pad", [8, 1, 64])
def test_strided_rows(pa, pad):
    _case(pa, 19, 5, 5, 128, 64, BF16, BF16, False, pad=pad, seed=pad)


def test_far_and_negative_positions(pa):
    _case(pa, 41, 4, 2, 128, 128, F32, F32, False, max_pos=2_000_000_000, seed=8)
    _case(pa, 41, 4, 2, 128, 128, F32, F32, True, max_pos=3_000_000, negative=True, seed=9)


def test_attention_factor_and_head_scales(pa):
    ks = torch.tensor([0.5, 2.0, 0.0625], device=DEV)
    vs = torch.tensor([1.0, 0.25, 3.0], device=DEV)
    _case(pa, 50, 9, 3, 128, 128, BF16, E4M3, False, factor=1.2079, k_scales=ks, v_scales=vs)
    _case(pa, 50, 9, 3, 128, 96, F32, F32, True, factor=1.2079, k_scales=ks)


def test_odd_block_sizes(pa):
    _case(pa, 50, 3, 1, 128, 128, BF16, BF16, False, bs=5)


def test_keys_only_and_in_place(pa):
    gen = torch.Generator().manual_seed(1)
    q, k, v = _rows(gen, 23, 4, 2, 128, BF16, 0)
    inv, _ = pa.pa_rope_frequencies(128)
    pos = torch.arange(23, dtype=torch.int32, device=DEV) * 77
    slots = torch.arange(23, dtype=torch.int32, device=DEV)
    pools = [torch.zeros(2, 16, 2, 128, dtype=BF16, device=DEV) for _ in range(4)]
    out = torch.empty(23, 4, 128, dtype=BF16, device=DEV)
    pa.pa_rope_and_cache(q, k, v, out, pools[0], pools[1], pos, slots, inv)
    pa.pa_rope_and_cache(None, k, v, None, pools[2], pools[3], pos, slots, inv)
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    before_k, before_v = k.clone(), v.clone()
    pa.pa_rope_and_cache(q, k, v, q, pools[2], pools[3], pos, slots, inv)  # strided, in place
    assert torch.equal(q, out) and torch.equal(pools[0], pools[2])
    assert torch.equal(k, before_k) and torch.equal(v, before_v)
    assert pa.pa_device_status() == pa.PA_OK


def test_values_go_in_as_the_scatter_puts_them(pa):
    """V rows, and K rows at position 0, are pa_reshape_and_cache's bit for bit."""
    gen = torch.Generator().manual_seed(4)
    _, k, v = _rows(gen, 30, 0, 4, 128, BF16, 0)
    k, v = k.contiguous(), v.contiguous()
    slots = torch.randperm(48, generator=gen)[:30].int().to(DEV)
    pos = torch.zeros(30, dtype=torch.int32, device=DEV)
    inv, _ = pa.pa_rope_frequencies(128)
    for kv, s in ((BF16, 1.0), (E4M3, 0.37)):
        a = [torch.zeros(3, 16, 4, 128, device=DEV).to(kv) for _ in range(2)]
        b = [torch.zeros(3, 16, 4, 128, device=DEV).to(kv) for _ in range(2)]
        pa.pa_reshape_and_cache(k, v, a[0], a[1], slots, k_scale=s, v_scale=s)
        pa.pa_rope_and_cache(None, k, v, None, b[0], b[1], pos, slots, inv, k_scale=s, v_scale=s)
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_bad_slot_or_scale_writes_nothing(pa):
    for T, bad in ((20, -1), (20, 48), (3000, 3008), (3000, -7)):
        gen = torch.Generator().manual_seed(T)
        q, k, v = _rows(gen, T, 2, 1, 64, BF16, 0)
        NB = -(-T // 16) + (1 if T == 20 else 0)
        slots = torch.arange(T, dtype=torch.int32)
        slots[T // 2] = bad
        out = torch.zeros(T, 2, 64, dtype=BF16, device=DEV)
        kb, vb = (torch.zeros(NB, 16, 1, 64, dtype=BF16, device=DEV) for _ in range(2))
        inv, _ = pa.pa_rope_frequencies(64)
        pos = torch.zeros(T, dtype=torch.int32, device=DEV)
        pa.pa_rope_and_cache(q, k, v, out, kb, vb, pos, slots.to(DEV), inv)
        assert pa.pa_device_status() == pa.PA_EINVAL
        assert not out.any() and not kb.any() and not vb.any()
        ok = torch.arange(T, dtype=torch.int32, device=DEV)
        scales = torch.tensor([float("nan")], device=DEV)
        pa.pa_rope_and_cache(q, k, v, out, kb, vb, pos, ok, inv, k_scales=scales)
        assert pa.pa_device_status() == pa.PA_EINVAL
        assert not out.any() and not kb.any() and not vb.any()


def test_other_stream_and_captured_graph(pa):
    gen = torch.Generator().manual_seed(6)
    q, k, v = _rows(gen, 40, 4, 2, 128, BF16, 0)
    slots = torch.arange(40, dtype=torch.int32, device=DEV)
    pos = torch.arange(40, dtype=torch.int32, device=DEV)
    inv, _ = pa.pa_rope_frequencies(128)
    kb, vb = (torch.zeros(3, 16, 2, 128, dtype=BF16, device=DEV) for _ in range(2))
    want, out = (torch.empty(40, 4, 128, dtype=BF16, device=DEV) for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pa.pa_rope_and_cache(q, k, v, out, kb, vb, pos, slots, inv, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_rope_and_cache(q, k, v, out, kb, vb, pos, slots, inv)
    pos += 1000
    g.replay()
    k1 = kb.clone()
    pa.pa_rope_and_cache(q, k, v, want, kb, vb, pos, slots, inv)
    assert torch.equal(out, want) and torch.equal(k1, kb)
    assert pa.pa_device_status() == pa.PA_OK

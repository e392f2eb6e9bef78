"""The speculative-decoding calls at the ends of what they accept: pools whose offsets pass 32 bits,
thousands of sequences, the widest trees and groups, odd and large head sizes, positions in any
order."""
import random

import pytest
import torch

from tests.spec_reference import assert_within, rotate, stored, values
from tests.test_gpu_tree import BF16, DEV, E4M3, F32, Batch, pa  # noqa: F401
from tests.test_gpu_tree_forms import check_general, form

pytestmark = pytest.mark.gpu


def far(b, blocks):
    """The batch's blocks moved to the end of pools of `blocks` blocks (the rest is not touched)."""
    for name in ("kb", "vb"):
        p = getattr(b, name)
        big = torch.empty(blocks, *p.shape[1:], dtype=p.dtype, device=DEV)
        big[-p.shape[0]:] = p
        setattr(b, name, big)
    b.tables += blocks - p.shape[0]


@pytest.mark.parametrize("src,kv,D,blocks", [(BF16, BF16, 128, 300_000), (BF16, E4M3, 128, 300_000),
                                             (F32, F32, 128, 150_000), (BF16, BF16, 96, 300_000)])
def test_tree_over_pools_past_32_bits(pa, src, kv, D, blocks):
    """2^31 elements of a pool lie in front of its last 131 072 blocks (of 16 x 8 x 128)."""
    b = Batch([9, 40], [300, 17], 16, 8, D, src=src, kv=kv, seed=70)
    want = b.call(pa)
    far(b, blocks)
    assert (blocks - 60) * 16 * 8 * D > 2 ** 31
    got = b.call(pa)
    assert pa.pa_device_status() == pa.PA_OK
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("kv", [BF16, E4M3])
def test_rows_and_blocks_past_32_bits(pa, kv):
    """Rotary caching, commit and copies at the end of a pool of 5 * 10^9 elements."""
    NB, Hkv, D, T = 300_000, 8, 128, 21
    gen = torch.Generator().manual_seed(71)
    kb, vb = (torch.empty(NB, 16, Hkv, D, dtype=kv, device=DEV) for _ in range(2))
    for p in (kb, vb):
        p.view(torch.uint8)[-4:] = 0
        p.view(torch.uint8)[:4] = 0
    k, v = (torch.randn(T, Hkv, D, generator=gen).to(BF16).to(DEV) for _ in range(2))
    first = (NB - 2) * 16
    slots = torch.arange(first, first + T, dtype=torch.int32, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    inv, _ = pa.pa_rope_frequencies(D)
    pa.pa_rope_and_cache(None, k, v, None, kb, vb, pos, slots, inv)
    y, e = rotate(values(k), pos, inv, False, 1.0)
    assert_within(kb[-2:].view(32, Hkv, D)[:T], *stored(y, e, kv), "k")
    x = values(v)
    assert_within(vb[-2:].view(32, Hkv, D)[:T], *stored(x, torch.zeros_like(x), kv), "v")
    bits = lambda p: p.contiguous().view(torch.uint8)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    before = bits(kb[-2:]).view(32, -1).clone()
    pa.pa_tree_commit(kb, vb, i32([[NB - 2, NB - 1]]), i32([10]), i32([[2, 8, 10]]), i32([3]))
    want = before.clone()
    want[[10, 11, 12]] = before[[12, 18, 20]]
    assert torch.equal(bits(kb[-2:]).view(32, -1), want)
    pa.pa_copy_blocks(kb, vb, i32([[NB - 2, NB - 4], [NB - 1, 1]]))
    assert torch.equal(bits(kb[-4]), bits(kb[-2])) and torch.equal(bits(kb[1]), bits(kb[-1]))
    assert torch.equal(bits(vb[-4]), bits(vb[-2])) and torch.equal(bits(vb[1]), bits(vb[-1]))
    assert pa.pa_device_status() == pa.PA_OK


@pytest.mark.parametrize("kv", [BF16, E4M3, F32])
def test_thousands_of_sequences(pa, kv):
    rng = random.Random(72)
    n = [rng.choice([0, 1, 1, 2, 5]) for _ in range(2600)]
    b = Batch(n, [rng.randint(0, 60) for _ in n], 2, 1, 128, src=F32 if kv == F32 else BF16, kv=kv,
              seed=72)
    b.check(pa, window=31)


@pytest.mark.parametrize("src,kv", [(BF16, BF16), (BF16, E4M3), (F32, BF16)])
def test_the_widest_tree(pa, src, kv):
    """2048 nodes, 64 words to a mask row."""
    b = Batch([2048, 3], [130, 2000], 4, 2, 128, src=src, kv=kv, seed=73)
    assert b.mask.shape[1] == 64
    b.check(pa)
    b.check(pa, window=77)


@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("group", [3, 127, 128, 129, 200])
def test_wide_groups(pa, group, kv):
    b = Batch([3, 1, 7], [200, 0, 33], 2 * group, 2, 128, kv=kv, seed=group)
    assert (form(pa, b)[0] == 0) == (group > 128)
    b.check(pa)


@pytest.mark.parametrize("D", [1, 3, 127, 129, 255])
def test_odd_head_sizes(pa, D):
    for src, kv in ((BF16, BF16), (F32, E4M3)):
        b = Batch([9, 1, 30], [100, 0, 3000], 4, 2, D, src=src, kv=kv, seed=D)
        check_general(b, b.call(pa))


@pytest.mark.parametrize("src,kv", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
def test_positions_in_any_order(pa, src, kv):
    """With a window, nodes need not lie behind the context, nor at or behind one another."""
    for seed in range(6):
        rng = random.Random(seed)
        b = Batch([12, 40, 3], [300, 90, 700], 8, 2, 128, src=src, kv=kv, seed=seed)
        top = rng.choice([10, 200, 1500, 2 ** 31 - 1])
        b.pos.copy_(torch.tensor([rng.randint(0, top) for _ in range(55)], dtype=torch.int32))
        for window in (1, 9, 150, 1000, 2 ** 31 - 1):
            b.check(pa, window=window)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(320, 64), (512, 256), (2, 2), (258, 130)])
def test_rotary_at_large_head_sizes(pa, D, R, interleaved):
    from tests.test_gpu_rope import _case

    _case(pa, 29, 3, 2, D, R, BF16, BF16, interleaved, seed=D)
    _case(pa, 29, 3, 2, D, R, F32, E4M3, interleaved, seed=D, pad=2)

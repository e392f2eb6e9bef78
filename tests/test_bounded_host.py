"""Argument checks of the calls for bounded caches, and their plain implementations, without a GPU."""
import math
import random

import pytest
import torch

from tests import bounded_reference as ref


@pytest.fixture(scope="module")
def b():
    from paged_kv_cache_31_gb300 import _build

    _build.build()
    from paged_kv_cache_31_gb300 import binding

    return binding


FAKE = 1 << 20  # a non-null address: these calls return before they use it


def window(b, weights=False, **kw):
    a = dict(q=FAKE, kb=FAKE, vb=FAKE, out=FAKE, qsl=FAKE, lens=FAKE, pos=FAKE, tables=FAKE, w=FAKE,
             wlen=64, observed=0, S=2, T=2, H=8, Hkv=2, D=128, bs=16, NB=8, width=4, qt=b.PA_BF16,
             kvt=b.PA_BF16, scale=1.0, window=16, first=4, sinks=None, lse=None, ks=1.0, vs=1.0,
             kss=None, vss=None, ws=None, bytes=0)
    a.update(kw)
    one = [a[x] for x in "q kb vb out qsl lens pos tables".split()]
    two = [a[x] for x in "S T H Hkv D bs NB width qt kvt scale window first sinks lse ks vs kss vss ws "
           "bytes".split()]
    if weights:
        return b._lib.pa_attention_key_weights(*one, a["w"], a["wlen"], a["observed"], *two, None)
    return b._lib.pa_window_attention(*one, *two, None)


@pytest.mark.parametrize("weights", [False, True])
def test_attention_refusals(b, weights):
    w = lambda **kw: window(b, weights, **kw)
    for bad in ({"H": 7}, {"Hkv": 0}, {"D": 0}, {"bs": 0}, {"H": -8}):
        assert w(**bad) == b.PA_ESHAPE, bad
    for bad in ({"qt": 2}, {"kvt": 5}, {"D": 257}, {"T": 2 ** 31}, {"width": 2 ** 30},
                {"T": 2 ** 29, "H": 16}):
        assert w(**bad) == b.PA_EUNSUPPORTED, bad
    nan = float("nan")
    for bad in ({"q": None}, {"kb": None}, {"vb": None}, {"out": None}, {"qsl": None}, {"lens": None},
                {"pos": None}, {"tables": None}, {"S": -1}, {"T": -1}, {"NB": -1}, {"width": -1},
                {"window": -1}, {"first": -1}, {"ks": 0.0}, {"vs": nan}, {"ks": math.inf},
                {"scale": nan}, {"scale": math.inf}, {"kss": FAKE, "ks": 2.0}, {"vss": FAKE, "vs": 2.0},
                {"S": 0}, {}, {"ws": FAKE + 8, "bytes": 1 << 30}, {"ws": FAKE, "bytes": 100}):
        assert w(**bad) == b.PA_EINVAL, bad  # ({}: no workspace)
    if weights:
        for bad in ({"w": None}, {"wlen": -1}, {"observed": -1}):
            assert w(ws=FAKE, bytes=1 << 40, **bad) == b.PA_EINVAL, bad
    assert w(S=0, T=0, q=None, kb=None) == b.PA_OK
    assert w(T=0, q=None, qsl=None, out=None) == b.PA_OK


def evict(b, **kw):
    a = dict(kb=FAKE, vb=FAKE, tables=FAKE, lens=FAKE, new=FAKE, w=FAKE, wlen=64, first=0, recent=0, S=2,
             Hkv=2, D=128, bs=16, NB=8, width=4, kvt=b.PA_BF16, ws=None, bytes=0)
    a.update(kw)
    return b._lib.pa_evict_keys(*a.values(), None)


def test_eviction_refusals(b):
    for bad in ({"Hkv": 0}, {"D": 0}, {"bs": -1}):
        assert evict(b, **bad) == b.PA_ESHAPE, bad
    for bad in ({"kvt": 7}, {"S": 65536}, {"Hkv": 65536}, {"D": 2 ** 20},
                {"width": 2 ** 15 + 1, "w": None}, {"width": 2 ** 16, "wlen": 2 ** 19 + 1},
                {"width": 2 ** 28}):
        assert evict(b, **bad) == b.PA_EUNSUPPORTED, bad
    for bad in ({"kb": None}, {"vb": None}, {"tables": None}, {"lens": None}, {"new": None}, {"S": -1},
                {"NB": -1}, {"width": -1}, {"first": -1}, {"recent": -1}, {"wlen": -1}, {},
                {"ws": FAKE + 4, "bytes": 1 << 30}, {"ws": FAKE, "bytes": 64}):
        assert evict(b, **bad) == b.PA_EINVAL, bad
    assert evict(b, S=0, kb=None) == b.PA_OK


def test_workspace_sizes(b):
    size = b.pa_window_attention_workspace_size
    assert size(4, 4, 8, 3, 128, 4, 16) == 0 and size(-1, 4, 8, 2, 128, 4, 16) == 0
    a, c = size(4, 4, 8, 2, 128, 4, 16), size(64, 8192, 32, 8, 128, 1024, 16)
    assert 0 < a < c and a % 256 == c % 256 == 0
    more = b.pa_attention_key_weights_workspace_size(64, 8192, 32, 8, 128, 1024, 16)
    assert more >= c + 4 * 8192 * 32
    assert b.pa_evict_keys_workspace_size(2, 0, 4, 16) == 0
    assert b.pa_evict_keys_workspace_size(2, 8, 4, 16) >= 2 * 8 * 4 * 16 * 4


def test_visible_keys():
    see = ref.visible(torch.tensor([0, 5, 9]), 10, 3, 2)
    assert see[0].nonzero()[:, 0].tolist() == [0]
    assert see[1].nonzero()[:, 0].tolist() == [0, 1, 3, 4, 5]
    assert see[2].nonzero()[:, 0].tolist() == [0, 1, 7, 8, 9]
    assert ref.visible(torch.tensor([4]), 10, 0, 2)[0].sum() == 5


def test_plain_attention_and_weights():
    c = ref.Batch([(5, 3), (0, 2)], 4, 2, 8, src=torch.float32, kv=torch.float32, device="cpu")
    c.tables.clamp_(min=0)
    got = ref.window_attention(c.q, c.kb, c.vb, c.qsl, c.lens, c.positions, c.tables, c.scale, window=3,
                               first=1, weights_len=9, observed=2)
    # token 2 of sequence 0 (position 7), head 3, by hand
    slot = lambda j: (int(c.tables[0, j // 16]), j % 16)
    keys = [0, 5, 6, 7]
    k = torch.stack([c.kb[slot(j)][1] for j in keys]).double()
    v = torch.stack([c.vb[slot(j)][1] for j in keys]).double()
    p = ((k @ c.q[2, 3].double()) * c.scale).softmax(0)
    assert torch.allclose(got["out"][2, 3], p @ v)
    w = got["weights"]
    assert torch.allclose(w.sum(-1), torch.tensor(4.0).double())  # two tokens, two heads
    assert (w[0, :, 1:4] == 0).all() and (w[0, :, 8] == 0).all()


def test_plain_eviction():
    rows = [[list("abcdefghij")]]
    w = [[[0.0, 5.0, 1.0, 4.0, 0.5, 9.0, 4.0, 8.0, 0.0, 0.0]]]
    ref.evict(rows, w, [10], [6], 1, 2)
    # a stays; of b .. h the heaviest are f, h, b; i, j move up; f and h fill c and d
    assert rows[0][0][:6] == list("abfhij")
    assert w[0][0] == [0.0, 5.0, 9.0, 8.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0]
    rng = random.Random(1)
    for _ in range(50):
        n = rng.randrange(1, 30)
        new, f, r = rng.randrange(0, n + 1), rng.randrange(0, 9), rng.randrange(0, 9)
        rows, ws = [[list(range(n))]], [[[float(rng.randrange(4)) for _ in range(n)]]]
        old = list(ws[0][0])
        ref.evict(rows, ws, [n], [new], f, r)
        kept = rows[0][0][:new]
        assert len(set(kept)) == new
        assert kept[:min(f, new)] == list(range(min(f, new)))
        gone = set(range(n)) - set(kept)
        ff = min(f, new)
        mid = [x for x in kept if ff <= x < n - min(r, new - ff)]
        assert all(old[x] <= old[y] for x in gone for y in mid)

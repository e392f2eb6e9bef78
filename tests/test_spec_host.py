"""Host side of the speculative-decoding calls: the rotary frequencies against their formulas,
and the argument errors that are returned before anything touches the device.  No GPU."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def b():
    from paged_kv_cache_31_gb300 import _build

    _build.build()
    from paged_kv_cache_31_gb300 import binding

    return binding


def _plain(R, base):
    return torch.tensor([base ** (-2 * i / R) for i in range(R // 2)], dtype=torch.float64)


# pow, the quotients and the ramp in fp64: a few units of 2^-53, pow's argument up to 20 of them
TOL = dict(rtol=1e-13, atol=0)


@pytest.mark.parametrize("R", [2, 4, 64, 128, 80])
def test_plain_linear_and_ntk_frequencies(b, R):
    f, a = b.pa_rope_frequencies(R, base=10000.0, device="cpu")
    assert f.dtype == torch.float64 and a == 1.0
    torch.testing.assert_close(f, _plain(R, 10000.0), **TOL)
    f, a = b.pa_rope_frequencies(R, base=500000.0, scaling="linear", factor=8.0, device="cpu")
    torch.testing.assert_close(f, _plain(R, 500000.0) / 8, **TOL)
    if R > 2:
        f, _ = b.pa_rope_frequencies(R, scaling="ntk", factor=4.0, device="cpu")
        torch.testing.assert_close(f, _plain(R, 10000.0 * 4.0 ** (R / (R - 2))), **TOL)
        # the slowest pair is stretched by the factor, the fastest is left alone
        assert math.isclose(float(f[-1]), float(_plain(R, 10000.0)[-1]) / 4, rel_tol=1e-12)
        assert float(f[0]) == 1.0


def test_yarn_frequencies(b):
    R, base, s, n = 128, 10000.0, 16.0, 4096
    f, a = b.pa_rope_frequencies(R, base=base, scaling="yarn", factor=s, original_max_position=n,
                                 device="cpu")
    assert math.isclose(a, 0.1 * math.log(s) + 1, rel_tol=1e-7)
    plain = _plain(R, base)
    low = math.floor(R * math.log(n / (32 * 2 * math.pi)) / (2 * math.log(base)))
    high = math.ceil(R * math.log(n / (2 * math.pi)) / (2 * math.log(base)))
    for i in range(R // 2):
        r = min(1.0, max(0.0, (i - low) / (high - low)))
        want = plain[i] * (1 - r) + plain[i] / s * r
        assert math.isclose(float(f[i]), float(want), rel_tol=1e-12)
    assert torch.equal(f[:low], plain[:low])


def test_band_frequencies(b):
    R, base, s, n = 128, 500000.0, 8.0, 8192
    f, a = b.pa_rope_frequencies(R, base=base, scaling="bands", factor=s, original_max_position=n,
                                 device="cpu")
    assert a == 1.0
    for x, got in zip(_plain(R, base).tolist(), f.tolist()):
        wave = 2 * math.pi / x
        if wave < n / 4.0:
            want = x
        elif wave > n / 1.0:
            want = x / s
        else:
            t = (n / wave - 1.0) / 3.0
            want = (1 - t) * x / s + t * x
        assert math.isclose(got, want, rel_tol=1e-12)


def test_frequency_refusals(b):
    E, S, U = b.PA_EINVAL, b.PA_ESHAPE, b.PA_EUNSUPPORTED
    for kw, st in ((dict(rotary_dim=0), S), (dict(rotary_dim=7), S), (dict(rotary_dim=-2), S),
                   (dict(rotary_dim=8, base=1.0), E), (dict(rotary_dim=8, base=float("nan")), E),
                   (dict(rotary_dim=8, scaling="linear", factor=0.5), E),
                   (dict(rotary_dim=2, scaling="ntk", factor=2.0), U),
                   (dict(rotary_dim=8, scaling="yarn", factor=2.0), E),
                   (dict(rotary_dim=8, scaling="yarn", factor=2.0, original_max_position=64,
                         beta_fast=1.0, beta_slow=1.0), E),
                   (dict(rotary_dim=8, scaling="bands", factor=2.0, original_max_position=64,
                         low_freq_factor=4.0, high_freq_factor=1.0), E)):
        with pytest.raises(b.PaError) as e:
            b.pa_rope_frequencies(device="cpu", **kw)
        assert e.value.status == st, kw
    with pytest.raises(ValueError):
        b.pa_rope_frequencies(8, scaling="other", device="cpu")


FAKE = ctypes.c_void_p(256)  # never dereferenced: every refusal comes first


def _rope(b, **kw):
    a = dict(q=FAKE, qs=8 * 64, qo=FAKE, qos=8 * 64, k=FAKE, ks=2 * 64, v=FAKE, vs=2 * 64, kb=FAKE,
             vb=FAKE, pos=FAKE, slots=FAKE, freq=FAKE, rot=64, il=0, af=1.0, T=4, H=8, Hkv=2, D=64,
             bs=16, NB=8, src=b.PA_BF16, kv=b.PA_BF16, ksc=1.0, vsc=1.0, kss=None, vss=None, st=None)
    a.update(kw)
    return b._lib.pa_rope_and_cache(*a.values())


def test_rope_refusals(b):
    E, S, U = b.PA_EINVAL, b.PA_ESHAPE, b.PA_EUNSUPPORTED
    for kw, st in ((dict(D=0), S), (dict(Hkv=0), S), (dict(bs=0), S), (dict(rot=63), S),
                   (dict(rot=0), S), (dict(rot=66), S), (dict(H=0), S),
                   (dict(src=b.PA_FP8_E4M3), U), (dict(kv=7), U),
                   (dict(D=512, rot=258, qs=8 * 512, qos=8 * 512, ks=1024, vs=1024), U),
                   (dict(D=65, rot=64, il=1, qs=520, qos=520, ks=130, vs=130), U),
                   (dict(NB=1 << 28), U), (dict(T=1 << 31), U), (dict(T=-1), E),
                   (dict(ksc=0.0), E), (dict(vsc=float("nan")), E), (dict(af=float("inf")), E),
                   (dict(ksc=2.0, kss=FAKE), E), (dict(vsc=2.0, vss=FAKE), E),
                   (dict(k=None), E), (dict(v=None), E), (dict(kb=None), E), (dict(pos=None), E),
                   (dict(slots=None), E), (dict(freq=None), E), (dict(qo=None), E),
                   (dict(q=None), E), (dict(ks=127), E), (dict(vs=0), E), (dict(qs=511), E),
                   (dict(qos=-512), E)):
        assert _rope(b, **kw) == st, kw
    assert _rope(b, T=0, k=None) == b.PA_OK


def _tree(b, **kw):
    a = dict(q=FAKE, kb=FAKE, vb=FAKE, out=FAKE, qsl=FAKE, lens=FAKE, pos=FAKE, mask=FAKE, tab=FAKE,
             S=2, T=6, words=1, H=8, Hkv=2, D=64, bs=16, NB=8, MB=4, qt=b.PA_BF16, kv=b.PA_BF16,
             scale=0.1, win=0, sinks=None, lse=None, ks=1.0, vs=1.0, kss=None, vss=None, ws=FAKE,
             wsb=1 << 40, st=None)
    a.update(kw)
    return b._lib.pa_tree_attention(*a.values())


def test_tree_refusals(b):
    E, S, U = b.PA_EINVAL, b.PA_ESHAPE, b.PA_EUNSUPPORTED
    for kw, st in ((dict(H=7), S), (dict(D=0), S), (dict(bs=0), S), (dict(Hkv=0), S),
                   (dict(D=257), U), (dict(qt=b.PA_FP8_E4M3), U), (dict(kv=9), U),
                   (dict(words=65), U), (dict(MB=1 << 28), U), (dict(T=1 << 30, S=1), U),
                   (dict(words=0), E), (dict(words=-1), E), (dict(mask=None), E), (dict(S=0), E),
                   (dict(S=-1), E), (dict(scale=float("nan")), E), (dict(scale=float("inf")), E),
                   (dict(ks=0.0), E), (dict(vs=-1.0), E), (dict(ks=2.0, kss=FAKE), E),
                   (dict(q=None), E), (dict(kb=None), E), (dict(out=None), E), (dict(qsl=None), E),
                   (dict(lens=None), E), (dict(pos=None), E), (dict(tab=None), E),
                   (dict(ws=None), E), (dict(ws=ctypes.c_void_p(128)), E), (dict(wsb=255), E)):
        assert _tree(b, **kw) == st, kw
    assert _tree(b, S=0, T=0, q=None) == b.PA_OK
    small = b.pa_tree_attention_workspace_size(1, 8, 32, 8, 128, 4, 16)
    large = b.pa_tree_attention_workspace_size(64, 2048, 32, 8, 128, 300, 16)
    assert 0 < small < large and small % 256 == large % 256 == 0
    assert b.pa_tree_attention_workspace_size(1, 8, 32, 5, 128, 4, 16) == 0


def test_page_refusals(b):
    L, E, S, U = b._lib, b.PA_EINVAL, b.PA_ESHAPE, b.PA_EUNSUPPORTED
    bf = b.PA_BF16

    def copy(kb=FAKE, vb=FAKE, pairs=FAKE, n=3, Hkv=2, D=64, bs=16, NB=8, kv=bf):
        return L.pa_copy_blocks(kb, vb, pairs, n, Hkv, D, bs, NB, kv, None)

    assert copy(Hkv=0) == copy(D=0) == copy(bs=-1) == S
    assert copy(kv=5) == copy(n=257, NB=(1 << 23) + 1) == copy(n=1 << 31) == U
    assert copy(kb=None) == copy(pairs=None) == copy(n=-1) == copy(NB=-1) == E
    assert copy(pairs=ctypes.c_void_p(4)) == E
    assert copy(n=0, kb=None) == b.PA_OK

    def commit(kb=FAKE, vb=FAKE, tab=FAKE, ctx=FAKE, acc=FAKE, cnt=FAKE, n=2, most=4, Hkv=2, D=64,
               bs=16, NB=8, MB=3, kv=bf):
        return L.pa_tree_commit(kb, vb, tab, ctx, acc, cnt, n, most, Hkv, D, bs, NB, MB, kv, None)

    assert commit(Hkv=0) == commit(D=0) == commit(bs=0) == S
    assert commit(kv=5) == commit(D=1 << 22) == U
    for kw in (dict(kb=None), dict(vb=None), dict(tab=None), dict(ctx=None), dict(acc=None),
               dict(cnt=None), dict(n=-1), dict(most=-1), dict(MB=-1), dict(NB=-1)):
        assert commit(**kw) == E, kw
    assert commit(n=0, kb=None) == commit(most=0, acc=None) == b.PA_OK

    def fork(tab=FAKE, lens=FAKE, par=FAKE, kid=FAKE, n=2, rows=4, MB=3, bs=16, refs=FAKE, fl=FAKE,
             fc=FAKE, NB=8, pairs=FAKE):
        return L.pa_fork_sequences(tab, lens, par, kid, n, rows, MB, bs, refs, fl, fc, NB, pairs, None)

    def grow(tab=FAKE, lens=FAKE, seqs=FAKE, new=FAKE, n=2, rows=4, MB=3, bs=16, refs=FAKE, fl=FAKE,
             fc=FAKE, NB=8):
        return L.pa_grow_sequences(tab, lens, seqs, new, n, rows, MB, bs, refs, fl, fc, NB, None)

    def free(tab=FAKE, lens=FAKE, seqs=FAKE, n=2, rows=4, MB=3, bs=16, refs=FAKE, fl=FAKE, fc=FAKE,
             NB=8):
        return L.pa_free_sequences(tab, lens, seqs, n, rows, MB, bs, refs, fl, fc, NB, None)

    def trim(tab=FAKE, lens=FAKE, seqs=FAKE, new=FAKE, n=2, rows=4, MB=3, bs=16, refs=FAKE, fl=FAKE,
             fc=FAKE, NB=8):
        return L.pa_trim_sequences(tab, lens, seqs, new, n, rows, MB, bs, refs, fl, fc, NB, None)

    for f in (fork, grow, trim, free):
        assert f(bs=0) == S
        assert f(rows=65537) == f(NB=(1 << 23) + 1) == f(MB=1 << 30) == U
        for kw in (dict(n=5), dict(n=-1), dict(rows=-1), dict(MB=-1), dict(NB=-1), dict(tab=None),
                   dict(lens=None), dict(refs=None), dict(fl=None), dict(fc=None)):
            assert f(**kw) == E, (f, kw)
        assert f(n=0, tab=None) == b.PA_OK
    assert fork(par=None) == fork(kid=None) == fork(pairs=None) == E
    assert grow(seqs=None) == grow(new=None) == free(seqs=None) == E
    assert trim(seqs=None) == trim(new=None) == E

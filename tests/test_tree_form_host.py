"""What pa_tree_attention_form refuses, and what it says without a device.  No GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def b():
    from paged_kv_cache_31_gb300 import _build

    _build.build()
    from paged_kv_cache_31_gb300 import binding

    return binding


def _form(b, **kw):
    t, c = ctypes.c_int32(-7), ctypes.c_int32(-7)
    a = dict(S=2, T=6, words=1, H=8, Hkv=2, D=128, MB=4, bs=32, qt=b.PA_BF16, kv=b.PA_BF16,
             tiles=ctypes.byref(t), cluster=ctypes.byref(c))
    a.update(kw)
    return b._lib.pa_tree_attention_form(*a.values()), t.value, c.value


def test_refusals(b):
    E, S, U = b.PA_EINVAL, b.PA_ESHAPE, b.PA_EUNSUPPORTED
    for kw, st in ((dict(H=7), S), (dict(D=0), S), (dict(bs=0), S), (dict(Hkv=0), S),
                   (dict(D=257), U), (dict(qt=b.PA_FP8_E4M3), U), (dict(kv=9), U),
                   (dict(words=65), U), (dict(MB=1 << 28), U), (dict(T=1 << 30), U),
                   (dict(words=0), E), (dict(S=0), E), (dict(S=-1), E), (dict(T=0), E),
                   (dict(T=-1), E), (dict(MB=-1), E), (dict(tiles=None), E),
                   (dict(cluster=None), E)):
        assert _form(b, **kw) == (st, -7, -7), kw
    with pytest.raises(b.PaError):
        b.pa_tree_attention_form(2, 6, 1, 7, 2, 128, 4, 16)


def test_the_general_kernel_needs_no_device_to_tell(b):
    for kw in (dict(), dict(bs=16, D=96), dict(bs=16, qt=b.PA_F32), dict(bs=16, H=258, Hkv=1),
               dict(bs=16, kv=b.PA_FP8_E4M3, D=64), dict(bs=16, kv=b.PA_F32)):
        assert _form(b, **kw) == (b.PA_OK, 0, 0), kw

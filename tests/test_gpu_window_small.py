"""Small softmax weights and small values of V in every form of the attention behind a window: what f16
would round to nothing is kept."""
import pytest
import torch

from tests import bounded_reference as ref
from tests.spec_reference import assert_within, stored
from tests.test_gpu_window import BF16, E4M3, pa  # noqa: F401

pytestmark = pytest.mark.gpu

# (the prefill kernel; even shares; decoding clusters)
FORMS = {"prefill": ([(90, 1300)], 64, 8), "prefill, mixed": ([(300, 700), (0, 600), (1000, 1), (40, 20)], 64, 8),
         "shares": ([(700, 40), (0, 300)], 8, 2), "decode": ([(900, 1), (300, 1)], 8, 2)}


def check(pa, b, want, v_scale=1.0):
    pa.pa_window_attention(*b.args(), b.scale, sliding_window=b.window, first_tokens=b.first, lse=b.lse,
                           v_scale=v_scale)
    assert pa.pa_device_status() == pa.PA_OK
    y, bound = stored(want["out"], want["out_b"], b.out.dtype)
    assert_within(b.out, y, bound, "out")
    assert_within(b.lse, want["lse"], want["lse_b"], "lse")


def expected(b, **kw):
    return ref.window_attention(b.q, b.kb, b.vb, b.qsl, b.lens, b.positions, b.tables, b.scale, b.window, b.first,
                                **kw)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("window,first", [(0, 0), (400, 16)])
def test_weights_of_2_to_the_minus_26(pa, form, kv, window, first):
    """Position 0 takes nearly all of the weight and has V zero: the output is the sum of the others', each
    2^-26 of it."""
    seqs, H, Hkv = FORMS[form]
    b = ref.Batch(seqs, H, Hkv, 128, kv=kv, seed=len(form))
    b.window, b.first = window, first
    b.q.fill_(1.0)
    b.kb.view(torch.uint8).zero_()
    for s, (c, n) in enumerate(seqs):
        at = int(b.tables[s, 0])
        b.kb[at, 0].fill_(1.625)  # 128 * 1.625 / sqrt(128) = 18.4: 2^26.5
        b.vb.view(torch.uint8)[at, 0].zero_()
    # f16 weights 2^-11 of their value and, below f16's normal range, half its smallest step, 2^-25, of a row
    # whose largest weight is at least 2^7
    want = expected(b, weight_u=2.0 ** -11, weight_min=2.0 ** -32)
    assert float(want["out"].abs().max()) > 1e-7
    check(pa, b, want)


@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("size", [1.0, 30.0, 1000.0, 2.0 ** 20])
def test_scores_of_any_magnitude(pa, kv, size):
    """Maxima that rise from tile to tile by less than the reference follows, and by far more."""
    b = ref.Batch([(700, 1300)], 64, 8, 128, kv=kv, seed=7)
    b.window, b.first = 0, 0
    b.q.fill_(1.0)
    up = torch.arange(int(b.lens[0]), device="cuda")
    rows = b.tables[0].long()[up // 16] * 16 + up % 16
    level = (up // 128).float() * 0.11 * size / 16  # 128 * 0.11 / sqrt(128) / ln 2 = 1.8 a tile at size 16
    b.kb.view(-1, 8, 128)[rows] = level.clamp(max=400.0)[:, None, None].expand(-1, 8, 128).to(kv)
    check(pa, b, expected(b, weight_u=2.0 ** -11, weight_min=2.0 ** -32))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("size", [2.0 ** -12, 1e-6, 1e-9, 1e-20, 1e-36])
@pytest.mark.parametrize("heads", [slice(None), slice(3, 4)])
def test_small_values(pa, form, size, heads):
    """V all below 2^-9, or that of one kv head: as exact as V of any other size."""
    seqs, H, Hkv = FORMS[form]
    b = ref.Batch(seqs, H, Hkv, 128, seed=len(form))
    b.window, b.first = 4, 2  # (few keys: nothing averages out)
    b.vb[:, :, heads] = (b.vb[:, :, heads].float().clamp(-4, 4) * size).to(BF16)
    check_bound = dict(weight_u=2.0 ** -11, weight_min=2.0 ** -32)
    want = expected(b, **check_bound)
    if heads != slice(None):  # (the other heads' own values below 2^-14 are off by 2^-25)
        G = H // Hkv
        other = [h for h in range(H) if h // G != 3]
        want["out_b"][:, other] += 2.0 ** -25
    check(pa, b, want)


def test_a_prompt_of_few_values(pa):
    """V of zeros but for a few places is exact in f16 or done again: parts of a tile without any value
    are neither."""
    b = ref.Batch([(0, 1300)], 64, 8, 128, seed=1)
    b.window, b.first = 0, 0
    b.vb.zero_()
    b.vb[int(b.tables[0, 2]), 5, 3, 100] = 1e-7
    b.vb[int(b.tables[0, 7]), 1, 4, 7] = 3.0
    check(pa, b, expected(b, weight_u=2.0 ** -11, weight_min=2.0 ** -32))

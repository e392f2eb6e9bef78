"""Key weights of rows with an infinity: whatever the signs of their scores, a row whose log-sum-exp is NaN
spoils the keys that it sees and no others."""
import pytest
import torch

from tests import bounded_reference as ref
from tests.spec_reference import values
from tests.test_gpu_window import BF16, CHUNKS, E4M3, F32, pa  # noqa: F401
from tests.test_gpu_window_forms import FORMS, ragged, widen

pytestmark = pytest.mark.gpu


def spoil(pa, b, row, window, first, observed=0):
    """One row with an infinity in q: its scores are of both signs."""
    t, h = row
    L, G = int(b.lens.max()), b.H // b.Hkv
    s = next(i for i in range(len(b.seqs)) if int(b.qsl[i]) <= t < int(b.qsl[i + 1]))

    def run():
        w = torch.zeros(len(b.seqs), b.Hkv, L, device="cuda")
        pa.pa_attention_key_weights(*b.args(), w, b.scale, observed_tokens=observed, sliding_window=window,
                                    first_tokens=first, lse=b.lse)
        assert pa.pa_device_status() == pa.PA_OK
        return w

    want = run()
    b.q[t, h] = 0
    b.q[t, h, b.D // 2] = float("inf")
    w = run()
    see = ref.visible(b.positions[t:t + 1], L, window, first)[0]
    bad = torch.zeros(w.shape, dtype=torch.bool)
    j = see.nonzero()[:, 0]
    k = values(b.kb[b.tables[s].long()[j.cuda() // b.bs], j.cuda() % b.bs, h // G, b.D // 2])
    # the formula's: scores of +inf, or of 0 * inf, give NaN; a row of -inf alone (with an infinity over e4m3
    # pools the row is NaN by the contract) has no weights
    if (k >= 0).any() or (b.kb.dtype == E4M3 and b.q.dtype == BF16):
        bad[s, h // G] = see
        assert b.lse[h, t].isnan() and b.out[t, h].isnan().all() and int(b.lse.isnan().sum()) == 1
    else:
        assert b.lse[h, t] == -float("inf") and (b.out[t, h] == 0).all()
    assert torch.equal(w.isnan().cpu(), bad)
    assert torch.equal(w.cpu()[~bad][want.cpu()[~bad] == 0], want.cpu()[~bad][want.cpu()[~bad] == 0])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("D,kv", [(128, BF16), (64, BF16), (128, E4M3)])
@pytest.mark.parametrize("window,first", [(0, 0), (150, 20)])
def test_decoding_forms(pa, form, D, kv, window, first):
    S, longest, H, Hkv, columns = FORMS[form]
    b = ref.Batch(ragged(S, longest, len(form)) if S > 1 else [(longest - 5, 1)], H, Hkv, D, kv=kv, seed=len(form))
    widen(b, columns)
    spoil(pa, b, (S // 2, H - 1), window, first)


BATCHES = {"tiles": ([(700, 16)], 32, 8, 128), "shares": ([(900, 40), (0, 100), (2000, 1)], 8, 2, 128),
           "prefill": (CHUNKS, 64, 8, 128), "other sizes": ([(90, 1), (40, 9)], 6, 3, 40),
           "past the room": ([(37 * i % 90, 1) for i in range(299)] + [(4050, 1)], 64, 4, 128)}


TYPES = [(batch, *t) for batch in BATCHES for t in ((BF16, BF16), (BF16, E4M3), (F32, F32))
         if t[0] == BF16 or batch not in ("prefill", "past the room")]


@pytest.mark.parametrize("batch,src,kv", TYPES)
@pytest.mark.parametrize("window,first", [(0, 0), (60, 4)])
def test_batches(pa, batch, src, kv, window, first):
    seqs, H, Hkv, D = BATCHES[batch]
    b = ref.Batch(seqs, H, Hkv, D, src=src, kv=kv, seed=len(seqs))
    spoil(pa, b, (b.T - 1, H - 2), window, first)
    b = ref.Batch(seqs, H, Hkv, D, src=src, kv=kv, seed=len(seqs))
    spoil(pa, b, (0, 1), window, first)

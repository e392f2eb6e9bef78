"""The calls for bounded caches with a workspace of exactly the size that they report, cut from the middle
of a larger buffer: nothing outside it is written, and the results are those of any other workspace."""
import pytest
import torch

from tests import bounded_reference as ref
from tests import test_gpu_key_weights as weights_test
from tests import test_gpu_window as window_test
from tests.test_gpu_window import BF16, E4M3, F32, pa  # noqa: F401

pytestmark = pytest.mark.gpu

EDGE = 1 << 20  # bytes before and behind


class Exact:
    def __init__(self, bytes):
        self.all = torch.full((bytes + 2 * EDGE,), 0xA5, dtype=torch.uint8, device="cuda")
        self.own = self.all[EDGE:EDGE + bytes]
        assert self.own.data_ptr() % 256 == 0

    def intact(self):
        return bool((self.all[:EDGE] == 0xA5).all()) and bool((self.all[EDGE + self.own.numel():] == 0xA5).all())


def attend(pa, b, window=64, first=4, weigh=True, short=0):
    """One call of each with an exact workspace: (out, lse, weights)."""
    S, width = b.tables.shape
    sizes = (S, b.T, b.H, b.Hkv, b.D, width, b.bs)
    w = torch.zeros(S, b.Hkv, int(b.lens.max()), device="cuda")
    b.out.fill_(7.0)
    b.lse.fill_(7.0)
    if weigh:
        ws = Exact(pa.pa_attention_key_weights_workspace_size(*sizes) - short)
        pa.pa_attention_key_weights(*b.args(), w, b.scale, sliding_window=window, first_tokens=first, lse=b.lse,
                                    workspace=ws.own)
    else:
        ws = Exact(pa.pa_window_attention_workspace_size(*sizes) - short)
        pa.pa_window_attention(*b.args(), b.scale, sliding_window=window, first_tokens=first, lse=b.lse,
                               workspace=ws.own)
    assert pa.pa_device_status() == pa.PA_OK
    assert ws.intact()
    return b.out.clone(), b.lse.clone(), w


def both(pa, b):
    """With the right results, and with the same bits on a second workspace."""
    if b.kb.dtype != E4M3 or b.q.dtype != BF16:  # (their pools want scales: those tests have them)
        window_test.check(pa, b, 64, 4)
        weights_test.check(pa, b, window=64, first=4)
    for weigh in (False, True):
        a, c = attend(pa, b, weigh=weigh), attend(pa, b, weigh=weigh)
        for x, y in zip(a, c):
            assert torch.equal(x, y)


@pytest.mark.parametrize("H,Hkv", [(64, 16), (128, 32), (60, 12), (96, 16), (48, 48), (8, 2), (5, 1)])
@pytest.mark.parametrize("off", [-1, 0, 1])
@pytest.mark.parametrize("D,kv", [(128, BF16), (64, BF16), (128, E4M3)])
def test_one_row_tile(pa, H, Hkv, off, D, kv):
    """One sequence of a row tile's tokens, one fewer and one more, behind a table of 1 to 9 columns."""
    n = 128 // (H // Hkv) + off
    for ctx in (0, 20):
        both(pa, ref.Batch([(ctx, n)], H, Hkv, D, kv=kv, seed=n + ctx))


BATCHES = {"decode": ([(900, 1), (300, 1), (2000, 1)], 8, 2),
           "decode, one": ([(900, 1)], 8, 2),
           "decode, many": ([(37 * i % 300, 1) for i in range(80)], 16, 8),
           "shares": ([(900, 40), (0, 100), (2000, 1)], 8, 2),
           "prefill": ([(300, 800), (0, 500), (1000, 1), (2000, 2)], 64, 8),
           "two row tiles": ([(0, 64)], 64, 16)}


@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("src,kv", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
def test_batches(pa, batch, src, kv):
    seqs, H, Hkv = BATCHES[batch]
    both(pa, ref.Batch(seqs, H, Hkv, 128, src=src, kv=kv, seed=len(seqs)))


@pytest.mark.parametrize("weigh", [False, True])
@pytest.mark.parametrize("batch", BATCHES)
def test_shorter_ones_are_refused(pa, batch, weigh):
    seqs, H, Hkv = BATCHES[batch]
    b = ref.Batch(seqs, H, Hkv, 128, seed=2)
    with pytest.raises(pa.PaError):
        attend(pa, b, weigh=weigh, short=1)
    assert bool((b.out == 7.0).all()) and bool((b.lse == 7.0).all())


@pytest.mark.parametrize("lens,width", [([90, 200, 31], 16), ([8192, 5], 512), ([9000, 700], 600),
                                        ([100] * 40, 8), ([3000], 520)])
def test_eviction(pa, lens, width):
    from tests.test_gpu_evict import Cache

    c = Cache(lens, 2, 64, seed=len(lens))
    tables = torch.full((len(lens), width), -3, dtype=torch.int32, device="cuda")
    n = min(width, c.tables.shape[1])
    tables[:, :n] = c.tables[:, :n]
    c.tables = tables
    wide = torch.zeros(len(lens), 2, max(width * 16, c.w.shape[2]), device="cuda")
    wide[:, :, :c.w.shape[2]] = c.w
    c.w = wide
    ws = Exact(pa.pa_evict_keys_workspace_size(len(lens), 2, width, 16))
    c.check(pa, [n // 2 for n in lens], 4, 20, workspace=ws.own)
    assert ws.intact()
    with pytest.raises(pa.PaError):
        c.check(pa, [n // 4 for n in lens], workspace=ws.own[:-1])


def test_eviction_of_empty_sequences(pa):
    """Tables without a column: nothing to do, as in any other batch of sequences without keys."""
    kb, vb = (torch.ones(3, 16, 2, 64, dtype=BF16, device="cuda") for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    tables = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    pa.pa_evict_keys(kb, vb, tables, i32([0, 0]), i32([0, 0]))
    assert pa.pa_device_status() == pa.PA_OK
    none = kb[:0].contiguous()
    pa.pa_evict_keys(none, none, tables, i32([0, 0]), i32([0, 0]), torch.zeros(2, 2, 0, device="cuda"))
    assert pa.pa_device_status() == pa.PA_OK
    pa.pa_evict_keys(kb, vb, tables, i32([0, 1]), i32([0, 0]))
    assert pa.pa_device_status() == pa.PA_EINVAL
    assert bool((kb == 1).all()) and bool((vb == 1).all())


def test_weights_of_no_column_are_not_none(pa):
    from tests.test_gpu_evict import Cache

    c = Cache([40, 20], 2, 64, seed=3)
    before = c.kb.clone()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    args = (c.kb, c.vb, c.tables, i32([40, 20]), i32([30, 20]))
    pa.pa_evict_keys(*args, c.w[:, :, :0].contiguous(), 0, 5)
    assert pa.pa_device_status() == pa.PA_EINVAL  # 40 keys, 0 weights
    assert torch.equal(c.kb.view(torch.uint8), before.view(torch.uint8))
    c.check(pa, [30, 20], 0, 5, weights=False)

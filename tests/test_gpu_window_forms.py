"""The attention calls of bounded caches in each form of their kernels: narrow, plain and broad CTAs,
clusters of 1 to 16, longest sequences first, several row tiles, scores past the room that is kept for
them, and rows of NaN; waits that run out; and bad arguments while another stream clears the status
word."""
import os

import pytest
import torch

from tests import bounded_reference as ref
from tests import test_gpu_key_weights as weights_test
from tests import test_gpu_window as window_test
from tests.test_gpu_spec_bounds import Clearing, inside, margins
from tests.test_gpu_window import BF16, E4M3, F32, pa  # noqa: F401

pytestmark = pytest.mark.gpu


def widen(b, columns):
    """The table of a server that allows long sequences; entries past a sequence's are not read."""
    t = torch.full((b.tables.shape[0], columns), -9, dtype=torch.int32, device="cuda")
    t[:, :b.tables.shape[1]] = b.tables
    b.tables = t


def both(pa, b, window, first, observed=0):
    scales = (0.125, 0.25) if b.kb.dtype == E4M3 else (1.0, 1.0)
    window_test.check(pa, b, window, first, scales=scales)
    b.out.fill_(7.0)
    weights_test.check(pa, b, observed, window, first, scales=scales, lse=True)


def ragged(n, longest, seed):
    g = torch.Generator().manual_seed(seed)
    return [(int(c), 1) for c in torch.randint(0, longest, (n,), generator=g)]


# sequences, longest context, query and kv heads, columns of the table
FORMS = {"narrow": (80, 300, 16, 8, 24),           # 640 units, short
         "narrow, many": (130, 700, 16, 8, 256),   # 1040 units: more than are resident, longest first
         "narrow, over 256": (300, 200, 8, 4, 256),
         "plain": (20, 900, 16, 8, 256),
         "plain, longest first": (50, 1500, 16, 8, 256),
         "clusters of 2": (16, 2000, 16, 8, 512),
         "clusters of 4": (4, 1500, 16, 8, 100),
         "clusters of 8": (2, 3000, 16, 8, 200),
         "one": (1, 3000, 16, 8, 200),
         "one, wide": (1, 3000, 16, 8, 2048),
         "one head": (1, 3000, 4, 1, 2048)}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("D,kv", [(128, BF16), (64, BF16), (128, E4M3)])
@pytest.mark.parametrize("window,first", [(0, 0), (400, 20)])
def test_forms(pa, form, D, kv, window, first):
    S, longest, H, Hkv, columns = FORMS[form]
    seqs = ragged(S, longest, len(form))
    if S == 1:
        seqs = [(longest - 5, 1)]
    b = ref.Batch(seqs, H, Hkv, D, kv=kv, seed=len(form))
    widen(b, columns)
    b.poison_unread(window, first)
    both(pa, b, window, first)


@pytest.mark.parametrize("D,kv", [(128, BF16), (64, BF16), (128, E4M3)])
@pytest.mark.parametrize("S,H,Hkv,n", [(3, 40, 1, 1), (40, 40, 1, 1), (1, 16, 1, 4), (1, 32, 8, 16),
                                       (1, 10, 2, 7), (1, 64, 1, 1), (300, 17, 1, 1)])
def test_row_tiles(pa, S, H, Hkv, n, D, kv):
    """More rows of a kv head than a tile of 16 (8 over e4m3): tokens of one sequence, many heads."""
    b = ref.Batch([((137 * i * i + 300) % 700, n) for i in range(S)], H, Hkv, D, kv=kv, seed=S + n)
    b.poison_unread(150, 20)
    both(pa, b, 150, 20, observed=2)


@pytest.mark.parametrize("kv", [BF16, E4M3])
def test_scores_past_the_room(pa, kv):
    """1200 units of 16 rows share 256 MB for their scores: room for some 3500 keys, so the longest
    sequences' last keys are multiplied again."""
    seqs = [(37 * i % 90, 1) for i in range(300)]
    seqs[11], seqs[150] = (4050, 1), (3700, 1)
    b = ref.Batch(seqs, 64, 4, 128, kv=kv, seed=4)
    weights_test.check(pa, b, scales=(0.125, 0.25) if kv == E4M3 else (1.0, 1.0))


@pytest.mark.parametrize("window,first", [(0, 0), (1, 1), (300, 4), (128, 130), (2 ** 31 - 1, 7)])
@pytest.mark.parametrize("H,Hkv", [(64, 8), (16, 16)])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -30, 2.0 ** 40])
def test_many_chunks_over_e4m3(pa, H, Hkv, size, window, first):
    """The prefill kernel over e4m3 pools, q of any magnitude."""
    seqs = [(c, n if H == 64 or n <= 100 else 4 * n) for c, n in window_test.CHUNKS]
    b = ref.Batch(seqs, H, Hkv, 128, kv=E4M3, seed=window % 91)
    b.q *= size
    b.q[::3] *= 2.0 ** -9  # rows of one tile
    b.scale /= size
    b.poison_unread(window, first)
    both(pa, b, window, first, observed=30 if window == 300 else 0)


@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("window,first", [(0, 0), (300, 20)])
def test_one_long_chunk(pa, kv, window, first):
    """The prefill kernel without decoding sequences beside it; calls one behind the other."""
    b = ref.Batch([(90, 1300)], 64, 8, 128, kv=kv, seed=5)
    b.poison_unread(window, first)
    both(pa, b, window, first)
    want = b.out.clone()
    for _ in range(20):
        b.out.zero_()
        scale = 0.125 if kv == E4M3 else 1.0
        for _ in range(2):
            pa.pa_window_attention(*b.args(), b.scale, sliding_window=window, first_tokens=first,
                                   k_scale=scale, v_scale=2 * scale if kv == E4M3 else 1.0)
        assert torch.equal(b.out, want)
    assert pa.pa_device_status() == pa.PA_OK


def test_some_sequences_have_no_token(pa):
    """As many sequences as tokens, though one has them all and others none."""
    for seqs in ([(300, 1), (20, 0), (0, 1), (77, 2), (40, 0)], [(90, 0), (200, 5), (30, 0), (9, 0), (10, 0)]):
        b = ref.Batch(seqs, 8, 2, 128, seed=len(seqs))
        b.poison_unread(50, 3)
        both(pa, b, 50, 3)


@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("seqs", [[(301, 1), (40, 1), (70, 1)], [(200, 4)], [(3000, 1)], [(300, 2), (20, 40)]])
def test_a_row_of_nan_spoils_only_the_keys_it_sees(pa, kv, seqs):
    b = ref.Batch(seqs, 8, 2, 128, kv=kv, seed=12)
    L = int(b.lens.max())
    run = lambda w: pa.pa_attention_key_weights(*b.args(), w, b.scale, sliding_window=50, first_tokens=3)
    want = torch.zeros(len(seqs), 2, L, device="cuda")
    run(want)
    b.q[0, 5, 7] = float("nan")  # kv head 1
    w = torch.zeros_like(want)
    run(w)
    assert pa.pa_device_status() == pa.PA_OK
    see = ref.visible(b.positions[:1], L, 50, 3)[0].cuda()
    assert w[0, 1][see].isnan().all()
    same = torch.ones_like(w, dtype=torch.bool)
    same[0, 1] = ~see
    # (in that row's tile nothing else is summed in another order)
    assert torch.equal(w[same], want[same])


@pytest.mark.parametrize("H,n", [(64, 300), (8, 40)])
def test_far_blocks(pa, H, n):
    """Key weights over blocks past 2^31 elements of a pool."""
    num = 2 ** 31 // (16 * 8 * 128) + 80
    kb = torch.empty(num, 16, 8, 128, dtype=BF16, device="cuda")
    vb = torch.empty_like(kb)
    for seqs in ([(290, 1), (33, 1)], [(290, n), (33, n), (0, 4 * n)]):
        b = ref.Batch(seqs, H, 8, 128, seed=13)
        blocks = b.kb.shape[0]
        kb[num - blocks:], vb[num - blocks:] = b.kb, b.vb
        tables = torch.where(b.tables >= 0, b.tables + (num - blocks), b.tables)
        w = torch.zeros(2, len(seqs), 8, int(b.lens.max()), device="cuda")
        out = torch.empty_like(b.out)
        pa.pa_attention_key_weights(b.q, kb, vb, out, *b.args()[4:7], tables, w[0], b.scale)
        pa.pa_attention_key_weights(*b.args(), w[1], b.scale)
        assert pa.pa_device_status() == pa.PA_OK
        assert torch.equal(out, b.out) and torch.equal(w[0], w[1])


PATHS = {"decode": ([(900, 1), (300, 1), (2000, 1)], 8, 2, BF16),
         "decode e4m3": ([(900, 1), (300, 1), (2000, 1)], 8, 2, E4M3),
         "shares": ([(900, 40), (0, 100), (2000, 1)], 8, 2, BF16),
         "shares e4m3": ([(900, 40), (0, 100), (2000, 1)], 8, 2, E4M3),
         "prefill e4m3": ([(300, 800), (0, 500), (1000, 1), (2000, 2)], 64, 8, E4M3),
         "prefill": ([(300, 800), (0, 500), (1000, 1), (2000, 2)], 64, 8, BF16)}


@pytest.mark.parametrize("path", PATHS)
def test_timeouts_unwind_and_the_device_stays_usable(pa, path):
    """PA_DEBUG_STALL_NS points waits at a barrier that nothing signals, each bounded at 20 ms: the status
    says so, nothing is written, the next call gives the same bits."""
    seqs, H, Hkv, kv = PATHS[path]
    b = ref.Batch(seqs, H, Hkv, 128, kv=kv, seed=51)

    def call(weigh):
        b.out.fill_(7.0)
        b.lse.fill_(7.0)
        w = torch.full((len(seqs), Hkv, int(b.lens.max())), 7.0, device="cuda")
        if weigh:
            pa.pa_attention_key_weights(*b.args(), w, b.scale, sliding_window=700, first_tokens=4, lse=b.lse)
        else:
            pa.pa_window_attention(*b.args(), b.scale, sliding_window=700, first_tokens=4, lse=b.lse)
        return b.out.clone(), b.lse.clone(), w

    for weigh in (False, True):
        want = call(weigh)
        assert pa.pa_device_status() == pa.PA_OK
        os.environ["PA_DEBUG_STALL_NS"] = "20000000"
        try:
            for _ in range(2):
                got = call(weigh)
                assert pa.pa_device_status() == pa.PA_ETIMEOUT
                assert all(bool((x == 7.0).all()) for x in got), "a timed-out call wrote output"
        finally:
            del os.environ["PA_DEBUG_STALL_NS"]
        again = call(weigh)
        assert pa.pa_device_status() == pa.PA_OK
        for x, y in zip(again, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("path", [*PATHS, "general"])
@pytest.mark.parametrize("bad", [-2 ** 31, 2 ** 31 - 1])
def test_farthest_positions_are_refused(pa, path, bad):
    """Positions at both ends of int32 behind the widest windows: refused, with everything as it was."""
    seqs, H, Hkv, kv = PATHS.get(path, ([(300, 1), (90, 30)], 8, 2, F32))
    b = ref.Batch(seqs, H, Hkv, 128, src=F32 if path == "general" else BF16, kv=kv, seed=81)
    w = torch.full((len(seqs), Hkv, int(b.lens.max())), 0.5, device="cuda")
    fine = b.positions.clone()
    for at in (0, -1):
        b.positions.copy_(fine)
        b.positions[at] = bad
        for window, first in ((2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 0), (1, 0)):
            b.out.fill_(7.0)
            pa.pa_window_attention(*b.args(), b.scale, sliding_window=window, first_tokens=first)
            assert pa.pa_device_status() == pa.PA_EINVAL
            pa.pa_attention_key_weights(*b.args(), w, b.scale, sliding_window=window, first_tokens=first)
            assert pa.pa_device_status() == pa.PA_EINVAL
            assert (b.out == 7.0).all() and (w == 0.5).all()


@pytest.mark.parametrize("path", [*PATHS, "general"])
@pytest.mark.parametrize("bad", ["table", "lens", "qsl", "positions"])
def test_bad_batches_while_the_status_is_cleared(pa, path, bad):
    """Whatever the later launches then see, reads and writes stay inside the arrays.  Each array is a
    view in the middle of a larger one, and bad indices point into its margins."""
    seqs, H, Hkv, kv = PATHS.get(path, ([(300, 1), (90, 30)], 8, 2, F32))
    b = ref.Batch(seqs, H, Hkv, 128, src=F32 if path == "general" else BF16, kv=kv, seed=80)
    L, NB, last = int(b.lens.max()), b.kb.shape[0], len(seqs) - 1
    _, b.kb = inside(b.kb)
    _, b.vb = inside(b.vb)
    widen(b, b.tables.shape[1] + 200)
    if bad == "table":
        b.tables[0, 3], b.tables[1, 0], b.tables[last, 2], b.tables[last, 1] = -1, NB, NB + 7, -8
    elif bad == "lens":
        b.lens[1] = L + 100
    elif bad == "qsl":
        b.qsl[1] = b.T + 3
    else:
        b.positions[0], b.positions[-1] = -5, L + 60
    _, b.tables = inside(b.tables)
    obig, b.out = inside(torch.zeros_like(b.q))
    wbig, w = inside(torch.zeros(len(seqs), Hkv, L, device="cuda"))
    with Clearing(pa):
        for _ in range(300):
            pa.pa_window_attention(*b.args(), b.scale, sliding_window=200, first_tokens=4)
            pa.pa_attention_key_weights(*b.args(), w, b.scale)
    assert margins(obig) and margins(wbig)


def test_bad_evictions_while_the_status_is_cleared(pa):
    from tests.test_gpu_evict import Cache

    c = Cache([700, 300, 90, 260], 2, 64, seed=3)
    NB = c.kb.shape[0]
    kbig, kb = inside(torch.ones_like(c.kb))
    vbig, vb = inside(torch.ones_like(c.vb))
    wbig, w = inside(c.w)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    for what in ("table", "lens", "new"):
        lens, new, tables = [700, 300, 90, 260], [300, 200, 90, 100], c.tables.clone()
        if what == "table":
            tables[0, 3], tables[1, 0], tables[3, 7], tables[3, 1] = -1, NB, NB + 7, -8
        elif what == "lens":
            lens[1] = c.tables.shape[1] * 16 + 5
        else:
            new[0], new[3] = -1, 261
        with Clearing(pa):
            for _ in range(500):
                pa.pa_evict_keys(kb, vb, tables, i32(lens), i32(new), w, 4, 10)
    assert margins(kbig) and margins(vbig) and margins(wbig)
    assert bool((kb == 1).all()) and bool((vb == 1).all())


def test_python_refusals(pa):
    def fresh():
        b = ref.Batch([(40, 1), (20, 3)], 8, 2, 128, seed=1)
        return dict(q=b.q, k_blocks=b.kb, v_blocks=b.vb, out=b.out, query_start_loc=b.qsl, seq_lens=b.lens,
                    positions=b.positions, block_tables=b.tables, scale=b.scale)

    a = fresh()
    w = torch.zeros(2, 2, 41, device="cuda")
    pa.pa_window_attention(**a)
    pa.pa_attention_key_weights(key_weights=w, **a)
    for name in ("q", "k_blocks", "out", "query_start_loc", "seq_lens", "positions", "block_tables"):
        t = a[name]
        for other in (t.cpu(), t.double(), t[:1] if t.dim() == 1 else t[:, :1], None):
            if name == "block_tables" and other is not None and other.dtype == torch.int32 and other.is_cuda:
                continue  # (narrower tables are not wrong by themselves)
            bad = dict(a)
            bad[name] = other
            with pytest.raises((ValueError, KeyError, TypeError)):
                pa.pa_window_attention(**bad)
            with pytest.raises((ValueError, KeyError, TypeError)):
                pa.pa_attention_key_weights(key_weights=w, **bad)
    for kw in (dict(lse=w), dict(sinks=torch.zeros(7, device="cuda")), dict(k_scales=torch.ones(3, device="cuda")),
               dict(workspace=torch.zeros(8)), dict(sliding_window=1.5), dict(first_tokens="2")):
        with pytest.raises((ValueError, KeyError, TypeError)):
            pa.pa_window_attention(**a, **kw)
    for bad in (w.cpu(), w.double(), w[:1], w[:, :1], w[0], w.transpose(1, 2), None):
        with pytest.raises((ValueError, KeyError, TypeError)):
            pa.pa_attention_key_weights(key_weights=bad, **a)
        if bad is None:
            continue
        with pytest.raises((ValueError, KeyError, TypeError)):
            pa.pa_evict_keys(a["k_blocks"], a["v_blocks"], a["block_tables"], a["seq_lens"], a["seq_lens"], bad)
    for new in (a["seq_lens"][:1], a["seq_lens"].cpu(), a["seq_lens"].long(), None):
        with pytest.raises((ValueError, KeyError, TypeError)):
            pa.pa_evict_keys(a["k_blocks"], a["v_blocks"], a["block_tables"], a["seq_lens"], new)
    with pytest.raises(pa.PaError):
        pa.pa_window_attention(**a, sliding_window=-1)
    with pytest.raises(pa.PaError):
        pa.pa_evict_keys(a["k_blocks"], a["v_blocks"], a["block_tables"], a["seq_lens"], a["seq_lens"],
                         keep_first=-1)
    assert pa.pa_device_status() == pa.PA_OK


@pytest.mark.parametrize("S,longest", [(120, 1900), (70, 3500)])
def test_evictions_longest_first(pa, S, longest):
    """More (sequence, kv head) units than are resident at once, but not twice as many; some sequences stay."""
    from tests.test_gpu_evict import Cache

    g = torch.Generator().manual_seed(S)
    lens = torch.randint(1, longest, (S,), generator=g).tolist()
    lens[5] = 0
    new = [n if i % 7 == 0 else n + 3 if i % 11 == 0 else n // 2 for i, n in enumerate(lens)]
    Cache(lens, 8, 64, seed=S).check(pa, new, 4, 30)


@pytest.mark.parametrize("D,bs", [(64, 16), (1, 16)])
def test_eviction_with_the_most_keys(pa, D, bs):
    """Tables and weights for 524288 keys: the largest lists and the least room beside them."""
    from tests.test_gpu_evict import Cache

    c = Cache([30000, 700], 1, D, bs=bs, seed=9)
    tables = torch.full((2, 524288 // bs), -3, dtype=torch.int32, device="cuda")
    tables[:, :c.tables.shape[1]] = c.tables
    w = torch.zeros(2, 1, 524288, device="cuda")
    w[:, :, :c.w.shape[2]] = c.w
    c.tables, c.w = tables, w
    c.check(pa, [17000, 600], 4, 500)

"""Calls of several launches whose arguments are bad, while another stream reads and clears the status
word that the launches pass the finding on with: whatever they then write stays inside the arrays.
Every array is a view in the middle of a larger one, and bad indices point into its margins."""
import threading

import pytest
import torch

from tests.test_gpu_tree import BF16, DEV, E4M3, F32, Batch, pa  # noqa: F401

pytestmark = pytest.mark.gpu
MARGIN = 8


def inside(t):
    """(the whole array, a copy of t in its middle); the margins hold zeros."""
    big = torch.zeros(t.shape[0] + 2 * MARGIN, *t.shape[1:], dtype=t.dtype, device=DEV)
    big[MARGIN:-MARGIN] = t
    return big, big[MARGIN:-MARGIN]


def margins(big):
    b = big.view(torch.uint8)
    return not b[:MARGIN].any() and not b[-MARGIN:].any()


class Clearing:
    """Another thread that reads and clears the status word, on a stream of its own."""

    def __init__(self, pa):
        self.pa, self.stream, self.end, self.seen = pa, torch.cuda.Stream(), False, set()

    def _loop(self):
        while not self.end:
            self.seen.add(self.pa.pa_device_status(self.stream))

    def __enter__(self):
        self.thread = threading.Thread(target=self._loop)
        self.thread.start()
        return self

    def __exit__(self, *_):
        self.end = True
        self.thread.join()
        torch.cuda.synchronize()
        self.seen.add(self.pa.pa_device_status())
        assert self.seen <= {self.pa.PA_OK, self.pa.PA_EINVAL}


def test_rotary_slots(pa):
    T, NB, D = 3000, 190, 64
    kbig, kb = inside(torch.zeros(NB, 16, 2, D, dtype=BF16, device=DEV))
    vbig, vb = inside(torch.zeros(NB, 16, 2, D, dtype=BF16, device=DEV))
    k = torch.ones(T, 2, D, dtype=BF16, device=DEV)
    slots = torch.randperm(NB * 16)[:T].int()
    slots[::500] = torch.tensor([-1, -128, NB * 16, NB * 16 + 127, -77, NB * 16 + 9], dtype=torch.int32)
    slots = slots.to(DEV)
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)
    inv, _ = pa.pa_rope_frequencies(D)
    with Clearing(pa):
        for _ in range(2000):
            pa.pa_rope_and_cache(None, k, k, None, kb, vb, pos, slots, inv)
    assert margins(kbig) and margins(vbig)


def test_copies(pa):
    NB, n = 700, 300
    big, kb = inside(torch.ones(NB, 16, 1, 64, dtype=BF16, device=DEV))
    pairs = torch.stack([torch.arange(n), torch.arange(n) + n], 1).int()
    pairs[::75] = torch.tensor([[3, -1], [5, NB + 7], [-8, 600], [NB, 601]], dtype=torch.int32)
    pairs = pairs.to(DEV)
    with Clearing(pa):
        for _ in range(2000):
            pa.pa_copy_blocks(kb, None, pairs)
    assert margins(big)
    assert bool((kb == 1).all())  # nothing came in from the margins either


def test_commit(pa):
    S, most, NB = 64, 8, 200
    gen = torch.Generator().manual_seed(3)
    big, kb = inside(torch.ones(NB, 16, 1, 64, dtype=BF16, device=DEV))
    vb = kb.clone()
    tables = torch.randperm(NB, generator=gen)[:S * 3].view(S, 3).int()
    acc = torch.arange(most).int().repeat(S, 1) * 2 + 1
    ctx = torch.full((S,), 10, dtype=torch.int32)
    count = torch.full((S,), most, dtype=torch.int32)
    tables[5, 0], tables[6, 1], tables[7, 0], tables[8, 1] = -1, -8, NB, NB + 7
    acc[9, 3] = 45       # beyond the table
    acc[10, 0] = -3
    acc[11, 4] = 2       # not increasing
    count[12], count[13] = 2 ** 31 - 1, -1
    ctx[14], ctx[15] = -1, 2 ** 31 - 1
    _, tables = inside(tables.to(DEV))
    _, acc = inside(acc.to(DEV))
    ctx, count = ctx.to(DEV), count.to(DEV)
    with Clearing(pa):
        for _ in range(2000):
            pa.pa_tree_commit(kb, vb, tables, ctx, acc, count)
    assert margins(big) and bool((kb == 1).all())


@pytest.mark.parametrize("src,kv,bad", [(F32, F32, "table"), (BF16, BF16, "table"),
                                        (BF16, E4M3, "table"), (F32, BF16, "lens"),
                                        (BF16, BF16, "lens"), (BF16, E4M3, "qsl")])
def test_tree(pa, src, kv, bad):
    b = Batch([12, 40, 3], [300, 90, 700], 8, 2, 128, src=src, kv=kv, seed=80)
    wide = torch.zeros(3, 1100, dtype=torch.int32, device=DEV)
    wide[:, :b.tables.shape[1]] = b.tables
    _, b.tables = inside(wide)  # planned shares
    NB = b.kb.shape[0]
    _, b.kb = inside(b.kb)
    _, b.vb = inside(b.vb)
    if bad == "table":
        b.tables[0, 3], b.tables[1, 0], b.tables[2, 7], b.tables[2, 20] = -1, NB, NB + 7, -8
    elif bad == "lens":
        b.lens[1] = 1100 * 16 + 5
    else:
        b.qsl[1] = 50
    obig, out = inside(torch.zeros_like(b.q))
    ws = torch.empty(pa.pa_tree_attention_workspace_size(3, 55, 8, 2, 128, 1100, 16),
                     dtype=torch.uint8, device=DEV)
    with Clearing(pa):
        for _ in range(1000):
            pa.pa_tree_attention(b.q, b.kb, b.vb, out, b.qsl, b.lens, b.pos, b.mask, b.tables,
                                 b.scale, workspace=ws)
    assert margins(obig)

"""pa_tree_attention in each of its forms (clusters of one and of several CTAs, planned shares, the
general kernel): which one a call takes, clusters over items of two row tiles, many calls each with
an output of its own, the general kernel at its own bounds, tensors off a 16-byte boundary, and inputs
that are not finite."""
import pytest
import torch

from tests.spec_reference import OUT_U, assert_within, tree_attention
from tests.test_gpu_tree import BF16, DEV, E4M3, F32, RAGGED, Batch, pa  # noqa: F401

pytestmark = pytest.mark.gpu


def widen(b, columns):
    """The table of a server that allows long sequences; entries past a sequence's are not read."""
    t = torch.full((b.tables.shape[0], columns), -9, dtype=torch.int32, device=DEV)
    t[:, :b.tables.shape[1]] = b.tables
    b.tables = t


def form(pa, b):
    """(row tiles of an item, CTAs of a cluster) that the batch's call takes."""
    T, H, D = b.q.shape
    return pa.pa_tree_attention_form(len(b.nodes), T, b.mask.shape[1], H, b.kb.shape[2], D,
                                     b.tables.shape[1], b.bs, b.q.dtype, b.kb.dtype)


def batch(pa, name, kv, seed):
    ctx = [60, 31] if name == "one CTA" else [700, 300]
    b = Batch([12, 5], ctx, 32, 8, 128, src=F32 if name == "general" else BF16, kv=kv, seed=seed)
    if name == "shares":
        widen(b, 1100)
    tiles, cluster = form(pa, b)
    assert tiles == (0 if name == "general" else 1)
    assert cluster == 1 if name == "one CTA" else cluster > 1 if name == "cluster" else cluster == 0
    return b


@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("window", [0, 3, 700])
def test_clusters_of_one_over_two_row_tiles(pa, kv, window):
    """Ten trees of up to 40 nodes x 4 heads: 160 rows, 80 items of two row tiles, a CTA to each."""
    b = Batch([40, 33, 1, 40, 32, 17, 40, 0, 39, 40], [530 - 50 * i for i in range(10)], 32, 8, 128,
              kv=kv, seed=61)
    assert form(pa, b) == (2, 1)
    b.check(pa, window=window)


@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("window", [0, 40, 700])
def test_clusters_of_several_over_two_row_tiles(pa, kv, window):
    """Trees of up to 160 nodes x 4 heads over up to 6400 positions, a cluster to each 256 rows.  The
    last item of 160 and of 150 nodes has one row tile, 17 nodes are one; the third sequence's
    clusters have CTAs without a key tile, with a window all have."""
    b = Batch([160, 150, 90, 17], [6400, 900, 64, 3000], 4, 1, 128, kv=kv, seed=62)
    widen(b, 418)
    tiles, cluster = form(pa, b)
    assert tiles == 2 and cluster > 1
    b.check(pa, window=window)
    b.mask[200:230] = 0  # rows that see only the context, and with a narrow window little of it
    b.check(pa, window=window)


def test_two_row_tiles_of_head_size_64(pa):
    for nodes, ctx, H, Hkv in (([40] * 10, [500] * 10, 32, 8), ([160, 70, 33, 1], [6400, 10, 0, 90], 4, 1),
                               ([30, 26, 25] * 4, [200, 31, 90] * 4, 40, 8)):
        b = Batch(nodes, ctx, H, Hkv, 64, seed=63)
        if ctx[0] == 6400:
            widen(b, 418)
        tiles, cluster = form(pa, b)
        assert tiles == 2 and cluster >= 1
        b.check(pa)
        b.check(pa, window=100)


def test_which_form(pa):
    """The sizes alone decide: the width of the table, not the lengths."""
    ask = pa.pa_tree_attention_form
    assert ask(1, 8, 1, 32, 8, 128, 45, 16)[0] == 1 and ask(1, 8, 1, 32, 8, 128, 45, 16)[1] > 1
    assert ask(1, 8, 1, 32, 8, 128, 8193, 16) == (1, 0)      # more entries than a CTA checks
    assert ask(64, 1024, 1, 32, 8, 128, 258, 16) == (1, 0)   # more units than SMs
    assert ask(4, 256, 2, 64, 8, 128, 4200, 16) == (2, 0)
    assert ask(1, 8, 1, 32, 8, 128, 45, 32) == ask(1, 8, 1, 32, 8, 96, 45, 16) == (0, 0)
    assert ask(1, 8, 1, 32, 8, 64, 45, 16, kv_dtype=E4M3) == (0, 0)
    assert ask(1, 8, 1, 32, 8, 128, 45, 16, F32, BF16) == (0, 0)


def same_but(got, want, spoiled):
    """NaN in the rows `spoiled` [T, H], the bits of `want` in all others."""
    out, lse = got
    assert spoiled.any() and not spoiled.all()
    assert torch.isnan(out[spoiled]).all() and torch.isnan(lse.t()[spoiled]).all()
    assert torch.equal(out[~spoiled], want[0][~spoiled])
    assert torch.equal(lse.t()[~spoiled], want[1].t()[~spoiled])


@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("name", ["one CTA", "cluster", "shares", "general"])
def test_a_nan_in_q_is_not_an_empty_row(pa, name, kv):
    """Every score of the row is NaN, so are its output and its lse; other rows do not notice."""
    b = batch(pa, name, kv, 50)
    want = b.call(pa)
    spoiled = torch.zeros(17, 32, dtype=torch.bool, device=DEV)
    for t, h, d in ((2, 5, 17), (11, 31, 127), (13, 0, 0)):
        b.q[t, h, d] = float("nan")
        spoiled[t, h] = True
    same_but(b.call(pa), want, spoiled)
    assert pa.pa_device_status() == pa.PA_OK


@pytest.mark.parametrize("name", ["one CTA", "cluster", "shares", "general"])
def test_an_infinity_in_q_is_not_an_empty_row(pa, name):
    """Some scores are +inf (the keys' elements have both signs), and inf - inf is NaN."""
    b = batch(pa, name, BF16, 51)
    want = b.call(pa)
    spoiled = torch.zeros(17, 32, dtype=torch.bool, device=DEV)
    for t, h, d, x in ((0, 3, 64, float("inf")), (12, 30, 1, float("-inf"))):
        b.q[t, h, d] = x
        spoiled[t, h] = True
    same_but(b.call(pa), want, spoiled)
    assert pa.pa_device_status() == pa.PA_OK


@pytest.mark.parametrize("name", ["one CTA", "cluster", "shares", "general"])
def test_an_infinity_in_q_over_e4m3_pools(pa, name):
    """The tensor cores' forms split q into e4m3 terms, which have no infinity."""
    b = batch(pa, name, E4M3, 53)
    want = b.call(pa)
    spoiled = torch.zeros(17, 32, dtype=torch.bool, device=DEV)
    for t, h, d, x in ((0, 3, 64, float("inf")), (12, 30, 1, float("-inf"))):
        b.q[t, h, d] = x
        spoiled[t, h] = True
    same_but(b.call(pa), want, spoiled)
    assert pa.pa_device_status() == pa.PA_OK


@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("name", ["one CTA", "cluster", "shares", "general"])
def test_a_nan_in_a_visible_key(pa, name, kv):
    """One key of one kv head: the rows that see it, and they alone, come out as NaN, whichever of
    the pieces of the context it lies in."""
    b = batch(pa, name, kv, 52)
    want = b.call(pa)
    x = b.kb.float()
    x[b.tables[0, 1], 3, 2, 9] = float("nan")
    b.kb.copy_(x.to(kv))
    spoiled = torch.zeros(17, 32, dtype=torch.bool, device=DEV)
    spoiled[:12, 8:12] = True  # sequence 0, the four heads of kv head 2
    same_but(b.call(pa), want, spoiled)
    assert pa.pa_device_status() == pa.PA_OK


@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("S,n,ctx", [(16, 8, 4000), (3, 40, 3000), (64, 4, 600), (10, 40, 500)])
def test_every_call_of_many_gives_the_same_bits(pa, S, n, ctx, kv):
    """4000 calls in captured graphs, each with an output and an lse of its own, all of them compared.
    (This finds what goes wrong once in some thousand calls, not what does once in 50 000.)"""
    b = Batch([n] * S, [ctx - 3 * i for i in range(S)], 32, 8, 128, kv=kv, seed=28)
    ws = torch.empty(pa.pa_tree_attention_workspace_size(S, S * n, 32, 8, 128, b.tables.shape[1], 16),
                     dtype=torch.uint8, device=DEV)
    out, lse = b.call(pa, workspace=ws)
    outs, lses = (torch.empty(20, *x.shape, dtype=x.dtype, device=DEV) for x in (out, lse))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for o, ls in zip(outs, lses):
            pa.pa_tree_attention(b.q, b.kb, b.vb, o, b.qsl, b.lens, b.pos, b.mask, b.tables, b.scale,
                                 workspace=ws, lse=ls)
    wrong = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(200):
        outs.zero_()
        lses.zero_()
        g.replay()
        wrong += (outs != out).sum() + (lses != lse).sum()
    assert int(wrong) == 0
    assert pa.pa_device_status() == pa.PA_OK


def check_general(b, got, window=0):
    """The bounds of fp32 weights and of q as it is: no bf16 pairs, no f16, no terms of e4m3."""
    out, lse = got
    want, wl, ob, lb = tree_attention(b.q, b.kb, b.vb, b.qsl, b.lens, b.pos, b.mask, b.tables, b.scale,
                                      window, weight_u=2.0 ** -24)
    assert_within(out, want, ob + (want.abs() + ob) * OUT_U[b.q.dtype] + 2.0 ** -126, "out")
    assert_within(lse, wl, lb, "lse")


@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("src,kv,D,bs", [
    (F32, F32, 128, 16), (F32, F32, 64, 5), (F32, BF16, 64, 16), (F32, E4M3, 128, 16),
    (BF16, F32, 128, 16), (BF16, BF16, 96, 16), (BF16, BF16, 128, 64), (BF16, E4M3, 64, 16),
    (BF16, E4M3, 128, 32), (BF16, BF16, 256, 16), (F32, F32, 100, 16)])
def test_the_general_kernel_keeps_32_bits(pa, src, kv, D, bs, window):
    b = Batch(*RAGGED, 8, 2, D, src=src, kv=kv, bs=bs, seed=64)
    assert form(pa, b) == (0, 0)
    check_general(b, b.call(pa, window=window), window)


def shifted(t):
    """A copy that begins one element behind a 16-byte boundary."""
    x = torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)[1:t.numel() + 1].view(t.shape)
    assert x.data_ptr() % 16 != 0
    return x.copy_(t)


@pytest.mark.parametrize("kv", [BF16, E4M3])
def test_one_tensor_off_a_boundary(pa, kv):
    """Any of q, the pools and out by itself sends the call to the general kernel."""
    b = Batch([9, 40, 1], [300, 17, 60], 8, 2, 128, kv=kv, seed=65)
    first = None
    for name in ("q", "kb", "vb", "out"):
        keep = getattr(b, name, None)
        out = torch.full_like(b.q, float("nan"))
        if name == "out":
            out = shifted(out)
        else:
            setattr(b, name, shifted(keep))
        lse = torch.full((8, 50), float("nan"), device=DEV)
        pa.pa_tree_attention(b.q, b.kb, b.vb, out, b.qsl, b.lens, b.pos, b.mask, b.tables, b.scale,
                             lse=lse)
        assert pa.pa_device_status() == pa.PA_OK
        check_general(b, (out, lse))
        first = first or (out.clone(), lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
        if name != "out":
            setattr(b, name, keep)
    b.check(pa)  # and all of them on boundaries, the tensor cores' kernel

"""pa_tree_attention in each of its forms (clusters of one and of several CTAs, planned shares, the
general kernel): inputs that are not finite."""
import pytest
import torch

from tests.test_gpu_tree import BF16, DEV, E4M3, F32, Batch, pa  # noqa: F401

pytestmark = pytest.mark.gpu


def widen(b, columns):
    """The table of a server that allows long sequences; entries past a sequence's are not read."""
    t = torch.full((b.tables.shape[0], columns), -9, dtype=torch.int32, device=DEV)
    t[:, :b.tables.shape[1]] = b.tables
    b.tables = t


def batch(form, kv, seed):
    ctx = [60, 31] if form == "one CTA" else [700, 300]
    b = Batch([12, 5], ctx, 32, 8, 128, src=F32 if form == "general" else BF16, kv=kv, seed=seed)
    if form == "shares":
        widen(b, 1100)
    return b


def same_but(got, want, spoiled):
    """NaN in the rows `spoiled` [T, H], the bits of `want` in all others."""
    out, lse = got
    assert spoiled.any() and not spoiled.all()
    assert torch.isnan(out[spoiled]).all() and torch.isnan(lse.t()[spoiled]).all()
    assert torch.equal(out[~spoiled], want[0][~spoiled])
    assert torch.equal(lse.t()[~spoiled], want[1].t()[~spoiled])


@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("form", ["one CTA", "cluster", "shares", "general"])
def test_a_nan_in_q_is_not_an_empty_row(pa, form, kv):
    """Every score of the row is NaN, so are its output and its lse; other rows do not notice."""
    b = batch(form, kv, 50)
    want = b.call(pa)
    spoiled = torch.zeros(17, 32, dtype=torch.bool, device=DEV)
    for t, h, d in ((2, 5, 17), (11, 31, 127), (13, 0, 0)):
        b.q[t, h, d] = float("nan")
        spoiled[t, h] = True
    same_but(b.call(pa), want, spoiled)
    assert pa.pa_device_status() == pa.PA_OK


@pytest.mark.parametrize("form", ["one CTA", "cluster", "shares", "general"])
def test_an_infinity_in_q_is_not_an_empty_row(pa, form):
    """Some scores are +inf (the keys' elements have both signs), and inf - inf is NaN."""
    b = batch(form, BF16, 51)
    want = b.call(pa)
    spoiled = torch.zeros(17, 32, dtype=torch.bool, device=DEV)
    for t, h, d, x in ((0, 3, 64, float("inf")), (12, 30, 1, float("-inf"))):
        b.q[t, h, d] = x
        spoiled[t, h] = True
    same_but(b.call(pa), want, spoiled)
    assert pa.pa_device_status() == pa.PA_OK


@pytest.mark.parametrize("form", ["one CTA", "cluster", "shares", "general"])
def test_an_infinity_in_q_over_e4m3_pools(pa, form):
    """The tensor cores' forms split q into e4m3 terms, which have no infinity."""
    b = batch(form, E4M3, 53)
    want = b.call(pa)
    spoiled = torch.zeros(17, 32, dtype=torch.bool, device=DEV)
    for t, h, d, x in ((0, 3, 64, float("inf")), (12, 30, 1, float("-inf"))):
        b.q[t, h, d] = x
        spoiled[t, h] = True
    same_but(b.call(pa), want, spoiled)
    assert pa.pa_device_status() == pa.PA_OK


@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("form", ["one CTA", "cluster", "shares", "general"])
def test_a_nan_in_a_visible_key(pa, form, kv):
    """One key of one kv head: the rows that see it, and they alone, come out as NaN, whichever of
    the pieces of the context it lies in."""
    b = batch(form, kv, 52)
    want = b.call(pa)
    x = b.kb.float()
    x[b.tables[0, 1], 3, 2, 9] = float("nan")
    b.kb.copy_(x.to(kv))
    spoiled = torch.zeros(17, 32, dtype=torch.bool, device=DEV)
    spoiled[:12, 8:12] = True  # sequence 0, the four heads of kv head 2
    same_but(b.call(pa), want, spoiled)
    assert pa.pa_device_status() == pa.PA_OK

"""The workspace sizes of the calls for bounded caches against what their launches lay out in it,
restated here, without a GPU."""
import itertools

import pytest


@pytest.fixture(scope="module")
def b():
    from paged_kv_cache_31_gb300 import _build

    _build.build()
    from paged_kv_cache_31_gb300 import binding

    return binding


def planned_end(S, T, H, Hkv, D, keys, rows_per_item, key_tile, most_ctas, weights):
    """Where the arrays of a planned call end: items of rows_per_item query rows of a kv head, key
    tiles of key_tile keys, cut into shares for up to most_ctas CTAs."""
    up = lambda n: -(-n // 256) * 256
    rows = T * (H // Hkv)
    pieces = min((rows // rows_per_item + S) * Hkv, most_ctas) * (keys // key_tile + 2)
    grid = max(1, min(most_ctas, pieces))
    end = up(32 * S) + up(8 * (S + 1)) + up(16 * (grid + 1))  # sequences, weights before them, shares
    end += up(2 * grid * rows_per_item * 8) + up(2 * grid * rows_per_item * D * 4)  # two states a CTA
    items = -(-rows // rows_per_item) + S
    end += up(16 * items) + up(8 * (items + 1)) + up(4 * (16 + 6 * items + 64 + S * Hkv))
    if weights:
        tiles = min(S, T) * -(-keys // 256)
        end += up(4 * T * H) + up(32 * S) + up(16 * tiles) + up(8 * (tiles + 1))
        end += up(16 * (152 + 1)) + up(2 * 152 * 256 * 4)
    return end


def tile_rows(group):
    return 128 // group * group


SEQS = [1, 2, 3, 40]
HEADS = [(64, 16), (128, 32), (4, 4), (8, 2), (5, 1), (60, 12), (96, 16), (34, 2), (160, 1), (48, 48)]


@pytest.mark.parametrize("D", [64, 128, 40, 256])
@pytest.mark.parametrize("weights", [False, True])
def test_planned_calls_fit(b, D, weights):
    size = b.pa_attention_key_weights_workspace_size if weights else b.pa_window_attention_workspace_size
    for S, (H, Hkv), (width, bs) in itertools.product(SEQS, HEADS, [(1, 16), (2, 16), (3, 16), (9, 16),
                                                                    (200, 16), (2, 32), (7, 5)]):
        group, keys = H // Hkv, width * bs
        tile = tile_rows(group) // group if group <= 128 else 0
        for T in {1, 2, 7, tile - 1, tile, tile + 1, 2 * tile - 1, 2 * tile, 2 * tile + 1, 900, 5000}:
            if T < 1:
                continue
            # the general kernel, or the tensor cores' by one or two row tiles to an item
            ends = [planned_end(S, T, H, Hkv, D, keys, 32, 32, 608, weights)]
            if group <= 128 and D in (64, 128):
                rows = tile_rows(group) * (2 if T * group > tile_rows(group) else 1)
                ends.append(planned_end(S, T, H, Hkv, D, keys, rows, 128, 152, weights))
            got = size(S, T, H, Hkv, D, width, bs)
            assert got >= max(ends), (S, T, H, Hkv, width, bs, got, ends)


@pytest.mark.parametrize("weights", [False, True])
def test_more_tokens_or_sequences_never_need_less(b, weights):
    """So a workspace for a server's largest batch serves its smaller ones (key weights: of batches with
    prompt chunks; decoding ones keep scores there)."""
    size = b.pa_attention_key_weights_workspace_size if weights else b.pa_window_attention_workspace_size
    for (H, Hkv), width in itertools.product(HEADS, [2, 40]):
        for S in (1, 2, 9):
            least = max(S, 64 * Hkv // H) + 1 if weights else 1
            sizes = [size(S, T, H, Hkv, 128, width, 16) for T in range(least, 600)]
            assert sizes == sorted(sizes), (H, Hkv, width, S)
        sizes = [size(S, 600, H, Hkv, 128, width, 16) for S in range(2, 40)]
        assert sizes == sorted(sizes), (H, Hkv, width)


def test_eviction_lists(b):
    """A list of moves lies in the workspace only where shared memory does not hold it."""
    size = b.pa_evict_keys_workspace_size
    for S, Hkv, width, bs in [(256, 8, 512, 16), (65535, 65535, 256, 32), (1, 1, 0, 16), (3, 2, 8192, 1)]:
        assert size(S, Hkv, width, bs) == 4096
    for S, Hkv, width, bs in [(256, 8, 513, 16), (2, 3, 8193, 1), (64, 8, 8192, 16)]:
        assert size(S, Hkv, width, bs) == 4096 + 4 * S * Hkv * width * bs


def test_scores_of_decoding_batches(b):
    """They take 256 MB or 8 KB a (sequence, kv head), whichever is more, beside the planned calls' arrays."""
    size, plain = b.pa_attention_key_weights_workspace_size, b.pa_window_attention_workspace_size
    for S, (H, Hkv), width in itertools.product([1, 64, 4000, 16384, 100000], [(32, 8), (64, 64), (128, 1)],
                                                [4, 256, 100000]):
        got, units = size(S, S, H, Hkv, 128, width, 16), S * Hkv
        tiles = S * -(-width * 16 // 256)  # (the plan of a batch with prompt chunks, which this is not)
        planned = plain(S, S, H, Hkv, 128, width, 16) + 4 * S * H + 32 * S + 24 * tiles + 320000
        assert got <= max(2 ** 28, 2 ** 13 * units, planned), (S, H, Hkv, width, got)

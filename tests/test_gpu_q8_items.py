"""Many short items in a row of the tensor-core kernel over an 8-bit cache: row tiles of a few rows, whose epilogues
use the second query tile's room, between pairs of row tiles, which need it for their queries."""
import random

import pytest
import torch

import chunk_ref as R
import q8_ref as Q
from test_gpu_q8 import attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import eagle_speculative_decoding_parent_gb300 as m
    return m


def same_and_right(tv, c, **kw):
    out, status = attend(tv, c, **kw)
    ref, A, S = Q.attention(c, **kw)
    tol = R.attention_tolerance(c, ref, A, S, c["q"].shape[2])
    off = (out.double() - ref).abs() > tol
    start = c["q_start"].tolist()
    for b in range(len(c["n"])):
        assert status[b] == 0 and not bool(off[start[b]:start[b + 1]].any()), (b, c["n"][b], c["P"][b])
    assert torch.isfinite(out.double()).all()
    for _ in range(3):
        assert torch.equal(attend(tv, c, **kw)[0], out)


@pytest.mark.parametrize("heads", [(16, 4), (5, 5), (24, 3), (14, 2), (64, 2)])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("keys", [0, 60, 300])
def test_short_items_between_pairs_of_row_tiles(tv, heads, d, keys):
    """One to five tokens, one of which fill a row tile or a few rows of it, between chunks of two row tiles and of
    two and a part; after nothing, less than a tile of keys and a few tiles."""
    r = random.Random(keys + d + heads[0])
    tile = 128 // (heads[0] // heads[1])                         # tokens of a row tile
    n = []
    while len(n) < 160:
        n += [r.randrange(1, 6) for _ in range(r.randrange(1, 5))]
        n.append(r.choice([2 * tile, 2 * tile + 1, tile + 1, 2 * tile + 3, tile, tile - 1 or 1]))
    P = [r.randrange(0, keys + 1) for _ in n]
    c = Q.cache_case(n, P, Hq=heads[0], Hkv=heads[1], d=d, bs=16, seed=keys)
    same_and_right(tv, c)
    same_and_right(tv, c, window=5, sinks=2, softcap=20.0)


@pytest.mark.parametrize("heads", [(16, 4), (2, 2), (64, 2)])
@pytest.mark.parametrize("d", [128, 64])
def test_refused_short_sequences_between_pairs_of_row_tiles(tv, heads, d):
    """Short sequences that are refused, among chunks of two row tiles, whose queries may be there already."""
    r = random.Random(d + heads[0])
    tile = 128 // (heads[0] // heads[1])
    n, bad = [], []
    while len(n) < 150:
        for _ in range(r.randrange(1, 4)):
            bad.append(len(n))
            n.append(r.randrange(1, 4))
        n += [2 * tile] * r.randrange(1, 3)
    P = [r.randrange(16, 200) for _ in n]
    c = Q.cache_case(n, P, Hq=heads[0], Hkv=heads[1], d=d, bs=16, seed=d)
    c["table"] = c["table"].clone()
    for b in bad:
        c["table"][b, 0] = -1
    good = [b for b in range(len(n)) if b not in bad]
    whole = dict(c, n=[0 if b in bad else a for b, a in enumerate(n)])
    out, status = attend(tv, c)
    ref, A, S = Q.attention(whole)
    tol = R.attention_tolerance(c, ref, A, S, d)
    start = c["q_start"].tolist()
    for b in range(len(n)):
        rows = slice(start[b], start[b + 1])
        if b in bad:
            assert status[b] == 3 and bool((out[rows] == 0).all()), b
        else:
            assert status[b] == 0 and bool(((out[rows].double() - ref[rows]).abs() <= tol[rows]).all()), b
    assert good and torch.equal(attend(tv, c)[0], out)

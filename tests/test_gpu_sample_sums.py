"""Top-p cuts that hang on the sum of a whole row whose far entries are many.  Of that sum an entry below
2^-13 of the largest is off by at most 2^-18 of itself and 2^-39; every other weight by 2^-38, so that sums
of a row are off by less than 2^-30 of themselves."""
import pytest
import torch

from test_gpu_sample import sample

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import eagle_speculative_decoding_parent_gb300 as m
    return m


# depth of the far entries in units of the temperature (one value each: rounded alike), and how many
FAR = [(9.26, 60000), (9.9, 120000), (10.5, 120000), (10.7, 120000), (12.3, 128000), (13.1, 128000), (15.0, 128000)]


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("far", range(len(FAR)))
def test_cuts_by_the_whole_sum(tv, far, many):
    """3,000 entries down to a depth of nine and the far ones behind; top-p where the small ones of the former
    are cut.  Few rows, and the distributions of more than the GPU holds at once."""
    depth, count = FAR[far]
    V, B, N = 3000 + count + 1, 8, 16 if many else 1
    g = torch.Generator().manual_seed(far)
    row = torch.cat([torch.zeros(1), -9.0 * torch.rand(3000, generator=g), torch.full((count,), -depth)])
    row = row[torch.randperm(V, generator=g)]
    x = row.expand(B, N, V).contiguous()               # (times a power of two below: exact)
    u = torch.rand((B, N), generator=g)
    w = torch.exp(row.double())
    order = torch.argsort(row, descending=True, stable=True)
    cum = torch.cumsum(w[order], 0)
    S, tail = float(cum[-1]), float(w[row == -depth].sum())
    top_p = torch.tensor([float(cum[3001 - 40 * b - 2]) / S for b in range(B)], dtype=torch.float32)
    temp = [[1.0], [0.5]][far % 2] * B
    tokens, status, probs = sample(tv, x * temp[0], u, temp=temp, p=top_p.tolist())
    assert status.eq(0).all()
    for b in range(B):
        need = float(top_p[b]) * S
        off = float(top_p[b]) * (2.0 ** -18 * tail + count * 2.0 ** -39) + 2.0 ** -30 * S
        for i in range(N):
            kept = probs[b, i] > 0
            k = int(kept.sum())
            assert bool(kept[order[:k]].all())
            # the last one begins below top-p of the sum, the next one does not
            assert (float(cum[k - 2]) if k > 1 else 0.0) < need + off and float(cum[k - 1]) >= need - off, (b, i, k)
            assert kept[int(tokens[b, i])]

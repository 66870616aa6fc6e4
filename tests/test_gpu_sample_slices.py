"""Distributions of many rows at vocabularies whose last slice is short.  A row is cut into slices of a
multiple of 2,048 entries, and what a slice leaves for the second kernel lies in its own part of the
distribution: nothing may be written outside of it."""
import pytest
import torch

from test_gpu_sample import check, rows, sample

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import eagle_speculative_decoding_parent_gb300 as m
    return m


GUARD = 64


def guarded(tv, x, u, offset=0, **filters):
    """logits_sample with the distributions inside a larger buffer; (tokens, probs)."""
    B, N, V = x.shape
    wide = torch.full((B * N * V + 2 * GUARD,), 5.0, device="cuda")
    probs = wide[GUARD + offset:GUARD + offset + B * N * V].view(B, N, V)
    tokens, status = (torch.full((B, N), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    tv.logits_sample(x.cuda(), u.cuda(), tokens, status, probs=probs, **filters)
    torch.cuda.synchronize()
    wide = wide.cpu()
    assert bool((wide[:GUARD + offset] == 5.0).all()) and bool((wide[GUARD + offset + B * N * V:] == 5.0).all())
    assert status.eq(0).all()
    return tokens.cpu(), wide[GUARD + offset:GUARD + offset + B * N * V].view(B, N, V)


def settings(B):
    """Filters in turn with none: the rows that the first kernel finishes lie beside those that it leaves."""
    f = lambda v, dt: torch.tensor([v[b % len(v)] for b in range(B)], dtype=dt)  # noqa: E731
    return dict(temperature=f([1.0, 0.7, 1.0, 0.0, 0.9], torch.float32), top_k=f([0, 0, 0, 0, 40], torch.int32),
                top_p=f([1.0, 0.9, 1.0, 1.0, 0.95], torch.float32), min_p=f([0.0, 0.0, 0.05, 0.0, 0.0], torch.float32))


def around(tv, V, dtype, B, N, offset):
    """Every row among many as in a call of few rows (which the first kernel finishes), token 0 and the last
    ones, which lie at the slices' ends, among what is kept; some of them against the definition."""
    x, u = rows(B, N, V, V, dtype)
    x[..., 0] = 12.0                                             # kept by most rows
    x[B // 2:, :, 0] = 9.0
    x[::7, 0, -1] = 11.5                                         # near entries in the last slice, too
    kw = settings(B)
    tokens, probs = guarded(tv, x, u, offset, **{a: b.cuda() for a, b in kw.items()})
    assert bool((probs[::5, :, 0] > 0).all())                    # (no filter)
    assert bool(((probs.double().sum(-1) - 1).abs() < 1e-5).all())
    arg = lambda b, c: dict(temp=kw["temperature"][b:c].tolist(), k=kw["top_k"][b:c].tolist(),  # noqa: E731
                            p=kw["top_p"][b:c].tolist(), m=kw["min_p"][b:c].tolist())
    for b in range(B):
        few, status, want = sample(tv, x[b:b + 1], u[b:b + 1], **arg(b, b + 1))
        assert status.eq(0).all() and torch.equal(few[0], tokens[b]), b
        assert torch.equal(want[0] > 0, probs[b] > 0), b
        # (the same weights, summed and divided alike but for the last bits)
        assert bool(((want[0] - probs[b]).abs() <= 2.0 ** -18 * want[0]).all()), b
    for b in range(0, B, 7):
        check(tv, x[b:b + 1, :1], u[b:b + 1, :1], **arg(b, b + 1))


@pytest.mark.parametrize("V", [114695, 131079, 245767])
@pytest.mark.parametrize("offset", [0, 1])
def test_last_slice_of_seven_entries(tv, V, offset):
    around(tv, V, torch.float32, 28, 3, offset)


def test_last_slice_of_seven_entries_half_precision(tv):
    around(tv, 491527, torch.bfloat16, 14, 3, 0)


@pytest.mark.parametrize("V", [114689, 114690, 114696, 114698, 131075, 262208, 300000])
def test_last_slice_empty_or_short(tv, V):
    """One entry, two, as many as the header, one pair more; an empty slice (262,208 entries: sixteen slices of
    18,432)."""
    around(tv, V, torch.float32, 28, 3, V % 2)


@pytest.mark.parametrize("V", [5, 7, 8, 9, 2047, 2049, 2055, 2056])
def test_many_short_rows(tv, V):
    """Rows shorter than a slice, or than a dump's header."""
    around(tv, V, torch.float32, 35, 64, 0)

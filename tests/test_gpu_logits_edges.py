"""tree_logits_process at the edges of its arguments."""
import math

import pytest
import torch

import chunk_ref as R
from test_gpu_logits import case, process

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import eagle_speculative_decoding_parent_gb300 as m
    return m


# ------------------------------------------------------------------ absent nodes

@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("V", [1000, 40001, 270000])
def test_absent_rows_of_a_failed_sequence_are_not_written(tv, probs, V):
    """A bad temperature, or a bad token, with a count that is good: only the present nodes' rows
    take the error's value."""
    c = case(4, 5, V, seed=2, grammar=False)
    counts = torch.tensor([3, 5, 2, 1], dtype=torch.int32)
    c["kw"]["temp"][0] = 0.0
    c["kw"]["tokens"][2, 1] = V
    c["kw"]["rep"][3] = float("inf")
    out, status = process(tv, c, probs, node_counts=counts)
    assert status.tolist() == [7, 0, 3, 7]
    for b, n in enumerate(counts.tolist()):
        assert out[b, n:].eq(7.0).all(), b
        if b != 1:
            assert out[b, :n].eq(0.0 if probs else -math.inf).all(), b


# ------------------------------------------------------------------ the smallest temperatures

@pytest.mark.parametrize("V", [300, 20001, 151669, 262144, 300007])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_smallest_temperatures_give_the_largest_entry_everything(tv, V, dtype):
    """Ordinary logits, whose quotients by the temperature float32 cannot hold: the row's mass is
    on its largest entries, in equal shares, and every other entry is 0."""
    c = case(4, 2, V, dtype, seed=V, penalties=False, bias=False, grammar=False)
    c["kw"]["temp"] = torch.tensor([2.0 ** -100, 2.0 ** -126, 1e-30, 2.0 ** -127], dtype=torch.float32)
    out, status = process(tv, c, True)
    assert status.tolist() == [0, 0, 0, 7] and out[3].eq(0).all()
    z = c["z"][:3].float()
    top = z == z.amax(-1, keepdim=True)
    want = top / top.sum(-1, keepdim=True)
    assert torch.equal(out[:3] != 0, top)
    # a sum of at most V ones (exact) and the division
    assert ((out[:3] - want).abs() <= want * 2.0 ** -20).all()
    # the formula in 64 bits says the same
    ref = R.logits(c["z"][:3], probs=True, temp=c["kw"]["temp"][:3])
    assert ((ref - want).abs() <= 1e-12).all()


@pytest.mark.parametrize("V", [262144, 300007])
def test_rows_that_no_cluster_holds(tv, V):
    """Masked rows, rows with NaN or infinity, and each row's own sequence's temperature."""
    c = case(3, 2, V, seed=5, penalties=False)
    c["kw"]["temp"] = torch.tensor([0.01, 1.0, 40.0], dtype=torch.float32)
    c["kw"]["grammar"][0, 1] = 0
    bits = c["kw"]["grammar"].long()[..., torch.arange(V) // 32] >> (torch.arange(V) % 32) & 1
    c["z"][2, 0, int(bits[2, 0].nonzero()[5])] = float("nan")
    c["z"][2, 1, int((bits[2, 1] == 0).nonzero()[5])] = float("nan")
    out, status = process(tv, c, True)
    assert status.eq(0).all() and out[0, 1].eq(0).all() and out[2, 0].isnan().all()
    ref = R.logits(c["z"], probs=True, **c["kw"])
    # u = 2^-24; three roundings of a logit (bias, reciprocal, product), of at most M / temp; the
    # sum of V terms in at least 512 partial sums; 2^-20 for the exponential and the division
    u = 2.0 ** -24
    M = c["z"].double().nan_to_num().abs().amax((1, 2)) + c["kw"]["bias"].double().abs().amax(1)
    rel = (6 * u * M / c["kw"]["temp"].double())[:, None, None] + (V / 512 + 24) * u + 2.0 ** -20
    for b, i in ((0, 0), (1, 0), (1, 1), (2, 1)):
        assert ((out[b, i].double() - ref[b, i]).abs() <= ref[b, i] * rel[b] + 2.0 ** -126).all(), (b, i)


# ------------------------------------------------------------------ waits that run out

def plain(c, out, probs, keep):
    """Rows of the sequences `keep` of a case with temperatures only."""
    z = c["z"].double()[keep] / c["kw"]["temp"].double()[keep][:, None, None]
    # float32: the reciprocal and the product, 2 u of at most |z| each, and the softmax as above; a
    # probability below float32's smallest normal number, 2^-126, becomes 0 (here |z| reaches 60
    # and more, and e^-88 is below it)
    u, top, V = 2.0 ** -24, float(z.abs().max()), z.shape[-1]
    ref = torch.softmax(z, -1) if probs else z
    tol = ref * (6 * u * top + (V / 512 + 24) * u + 2.0 ** -20) + 2.0 ** -126 if probs else 3 * u * z.abs()
    assert ((out[keep].double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("B,N,V", [(5, 9, 40000), (1500, 1, 500), (300, 5, 2000), (2, 3, 270000)])
def test_waits_that_run_out(tv, monkeypatch, probs, B, N, V):
    """Every sequence with a row behind the wait says so, those included that the group of CTAs
    had not come to, and no row of theirs looks right.  (The test-only variable makes the first
    wait for a row count as run out.)"""
    c = case(B, N, V, seed=1, penalties=False, bias=False, grammar=False)
    counts = torch.full((B,), N, dtype=torch.int32)
    counts[B // 2] = N - 1 if N > 1 else 7
    monkeypatch.setenv("TV_TEST_WAITS_RUN_OUT", "0")
    out, status = process(tv, c, probs, node_counts=counts)
    want = torch.where(counts <= N, 6, 3)
    assert torch.equal(status, want.int())
    bad = torch.full_like(out, 0.0 if probs else -math.inf)
    if N > 1:
        bad[B // 2, N - 1] = 7.0
    assert torch.equal(out, bad)
    monkeypatch.delenv("TV_TEST_WAITS_RUN_OUT")
    out, status = process(tv, c, probs)
    assert status.eq(0).all()
    plain(c, out, probs, slice(None))


@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("cta", [0, 3, 40])
def test_a_wait_that_runs_out_in_one_cta(tv, monkeypatch, probs, cta):
    """The other CTAs' sequences are right."""
    c = case(1500, 1, 500, seed=1, penalties=False, bias=False, grammar=False)
    monkeypatch.setenv("TV_TEST_WAITS_RUN_OUT", f"0@{cta}")
    out, status = process(tv, c, probs)
    late = (status == 6).nonzero().view(-1).tolist()
    assert late == list(range(late[0], late[-1] + 1)) and 1 < len(late) < 20
    assert out[late].eq(0.0 if probs else -math.inf).all()
    good = status == 0
    assert int(good.sum()) == 1500 - len(late)
    plain(c, out, probs, good)

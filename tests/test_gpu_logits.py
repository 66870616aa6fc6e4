"""tree_logits_process and token_counts_update on the GPU against their definitions in 64
bits, with bounds derived from float32 arithmetic."""
import math

import numpy as np
import pytest
import torch

import chunk_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import eagle_speculative_decoding_parent_gb300 as m
    return m


def tree_masks(rng, B, N):
    """Ancestor-or-self bits of random trees, int64 [B, N]."""
    out = np.zeros((B, N), np.uint64)
    for b in range(B):
        out[b, 0] = 1
        for i in range(1, N):
            out[b, i] = out[b, int(rng.integers(i))] | (np.uint64(1) << np.uint64(i))
    return torch.from_numpy(out.view(np.int64))


def case(B, N, V, dtype=torch.float32, seed=0, penalties=True, bias=True, grammar=True):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    c = dict(z=(torch.randn((B, N, V), generator=g) * 4).to(dtype), kw={})
    kw = c["kw"]
    kw["temp"] = torch.tensor(rng.uniform(0.3, 2.0, B), dtype=torch.float32)
    if bias:
        kw["bias"] = torch.randn((B, V), generator=g)
    if grammar:
        kw["grammar"] = torch.randint(-2**31, 2**31, (B, N, (V + 31) // 32), generator=g).to(torch.int32)
    if penalties:
        kw["mask"] = tree_masks(rng, B, N)
        kw["tokens"] = torch.randint(0, V, (B, N), generator=g).to(torch.int32)
        if N > 3:
            kw["tokens"][:, 2] = kw["tokens"][:, 1]          # repeated on some paths
        cnt = torch.randint(0, 4, (B, V), generator=g) * (torch.rand((B, V), generator=g) < 0.2)
        flag = torch.rand((B, V), generator=g) < 0.1
        kw["counts"] = torch.where(flag, cnt - 2**31, cnt).to(torch.int32)
        kw["rep"] = torch.tensor(rng.uniform(0.7, 1.6, B), dtype=torch.float32)
        kw["freq"] = torch.tensor(rng.uniform(-0.5, 0.5, B), dtype=torch.float32)
        kw["pres"] = torch.tensor(rng.uniform(-0.5, 0.9, B), dtype=torch.float32)
    return c


NAMES = dict(mask="mask", tokens="draft_tokens", counts="counts", bias="bias", grammar="grammar",
             rep="repetition", freq="frequency", pres="presence", temp="temperature")


def process(tv, c, probs, out=None, node_counts=None):
    z = c["z"].cuda()
    B, N, V = z.shape
    out = torch.full((B, N, V), 7.0, device="cuda") if out is None else out
    status = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    tv.tree_logits_process(z, out, status, probs=probs,
                           node_counts=None if node_counts is None else node_counts.cuda(),
                           **{NAMES[k]: v.cuda() for k, v in c["kw"].items()})
    torch.cuda.synchronize()
    return out.cpu(), status.cpu()


def tolerance(ref_logits, ref, c, probs):
    """u = 2^-24.  A processed logit has at most seven float32 roundings (bias, penalty, frequency
    product and difference, presence, temperature twice over), each of a value at most M, the
    largest intermediate magnitude (|z| max(rep, 1/rep) plus the subtractions), divided by the
    temperature at the end: off by at most 7 u M / temp.
    A probability moves by that factor for itself and for the sum, and by the float32 sum of V
    terms (V u at most, but the terms are added in at least 512 partial sums: V / 512 + 24
    additions deep), and by 2^-20 for the exponential and the division."""
    B, N, V = ref.shape
    u = 2.0 ** -24
    k = c["kw"]
    one = torch.ones(B)
    rep = torch.maximum(k.get("rep", one), 1 / k.get("rep", one)).double()
    z = c["z"].double().abs().amax((1, 2)) + (k["bias"].double().abs().amax(1) if "bias" in k else 0.0)
    many = 70.0 * (k.get("freq", one * 0).abs() + k.get("pres", one * 0).abs()).double()
    d = 7 * u * ((z * rep + many) / k["temp"].double())[:, None, None]
    if not probs:
        return d + 0 * ref
    return ref * (2 * d + (V / 512 + 24) * u + 2.0 ** -20) + 2.0 ** -126


@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,N,V", [(2, 1, 1), (1, 3, 31), (3, 5, 1000), (2, 7, 4099), (1, 64, 20000),
                                   (2, 3, 50001), (1, 2, 128256), (1, 2, 151669)])
def test_logits(tv, probs, dtype, B, N, V):
    c = case(B, N, V, dtype, seed=V + N)
    out, status = process(tv, c, probs)
    assert status.eq(0).all()
    ref = R.logits(c["z"], probs=probs, **c["kw"])
    none = torch.isinf(ref) if not probs else ref == 0
    assert torch.equal(out.double()[none], ref[none])
    tol = tolerance(None, ref, c, probs)
    ok = ~none
    assert ((out.double() - ref).abs()[ok] <= tol.expand_as(ref)[ok]).all()


@pytest.mark.parametrize("what", [dict(penalties=False), dict(bias=False), dict(grammar=False),
                                  dict(penalties=False, bias=False, grammar=False)])
@pytest.mark.parametrize("probs", [False, True])
def test_logits_parts_left_out(tv, what, probs):
    c = case(2, 5, 3333, seed=5, **what)
    out, status = process(tv, c, probs)
    assert status.eq(0).all()
    ref = R.logits(c["z"], probs=probs, **c["kw"])
    none = torch.isinf(ref)
    assert torch.equal(out.double()[none], ref[none])
    tol = tolerance(None, ref, c, probs).expand_as(ref)
    assert ((out.double() - ref).abs()[~none] <= tol[~none]).all()


def test_probs_longer_than_a_cluster_holds(tv):
    """More entries than eight CTAs keep in shared memory: the rest is read again."""
    V = 520003
    c = case(1, 2, V, seed=2)
    out, status = process(tv, c, True)
    assert status.eq(0).all()
    ref = R.logits(c["z"], probs=True, **c["kw"])
    assert ((out.double() - ref).abs() <= tolerance(None, ref, c, True)).all()
    V = 520000
    c = case(1, 1, V, torch.bfloat16, seed=3)
    out, _ = process(tv, c, True)
    ref = R.logits(c["z"], probs=True, **c["kw"])
    assert ((out.double() - ref).abs() <= tolerance(None, ref, c, True)).all()


@pytest.mark.parametrize("V", [500, 40000])
def test_rows_without_an_allowed_token(tv, V):
    c = case(2, 4, V, seed=1)
    c["kw"]["grammar"][0, 2] = 0
    c["kw"]["grammar"][1, 1] = 0
    c["kw"]["grammar"][1, 1, 3] = 1 << 7                 # one token only
    c["z"][1, 3] = -math.inf
    p, status = process(tv, c, True)
    assert status.eq(0).all()
    assert p[0, 2].eq(0).all() and p[1, 3].eq(0).all()
    assert p[1, 1].nonzero().tolist() == [[3 * 32 + 7]] and p[1, 1, 3 * 32 + 7] == 1.0
    z, _ = process(tv, c, False)
    assert z[0, 2].eq(-math.inf).all()
    # what a masked entry holds does not matter; an allowed NaN or +infinity spoils the row only
    c = case(2, 4, V, seed=1)
    bits = c["kw"]["grammar"].long()[..., torch.arange(V) // 32] >> (torch.arange(V) % 32) & 1
    clean, _ = process(tv, c, True)
    dirty = dict(c, z=torch.where(bits == 0, torch.tensor(float("nan")), c["z"]))
    got, _ = process(tv, dirty, True)
    assert torch.equal(got, clean)
    at = int(bits[0, 1].nonzero()[0])
    for bad in (float("nan"), float("inf")):
        dirty["z"][0, 1, at] = bad
        got, _ = process(tv, dirty, True)
        assert got[0, 1].isnan().all()
        keep = torch.ones(2, 4, dtype=torch.bool)
        keep[0, 1] = False
        assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("probs", [False, True])
def test_in_place_and_repeated(tv, probs):
    c = case(3, 6, 30000, seed=4)
    first, _ = process(tv, c, probs)
    again, _ = process(tv, c, probs)
    assert torch.equal(first, again)
    z = c["z"].cuda()
    st = torch.zeros(3, dtype=torch.int32, device="cuda")
    tv.tree_logits_process(z, z, st, probs=probs, **{NAMES[k]: v.cuda() for k, v in c["kw"].items()})
    assert torch.equal(z.cpu(), first)


@pytest.mark.parametrize("probs", [False, True])
def test_node_counts_and_bad_sequences(tv, probs):
    B, N, V = 8, 6, 20000
    c = case(B, N, V, seed=6)
    ref = R.logits(c["z"], probs=probs, **c["kw"])
    tol = tolerance(None, ref, c, probs).expand_as(ref)
    counts = torch.tensor([6, 1, 3, 0, 7, 6, 6, 6], dtype=torch.int32)
    c["kw"]["tokens"][2, 3:] = 1 << 30            # absent nodes may hold anything
    c["kw"]["tokens"][5, 4] = V                   # a token past the vocabulary
    c["kw"]["temp"][6] = 0.0
    c["kw"]["rep"][7] = float("nan")
    out, status = process(tv, c, probs, node_counts=counts)
    assert status.tolist() == [0, 0, 0, 3, 3, 3, 7, 7]
    bad = 0.0 if probs else -math.inf
    for b, n in enumerate([6, 1, 3]):
        none = torch.isinf(ref[b, :n])
        assert ((out[b, :n].double() - ref[b, :n]).abs()[~none] <= tol[b, :n][~none]).all()
        assert out[b, n:].eq(7.0).all()
    assert out[3:].eq(bad).all()


@pytest.mark.parametrize("k", range(1, 17))
def test_probs_of_every_cluster_size(tv, k):
    """Rows that k CTAs just hold, of odd lengths."""
    V = 16352 * k - 7
    c = case(1, 3, V, seed=k)
    out, status = process(tv, c, True)
    assert status.eq(0).all()
    ref = R.logits(c["z"], probs=True, **c["kw"])
    assert ((out.double() - ref).abs() <= tolerance(None, ref, c, True)).all()


@pytest.mark.parametrize("probs", [False, True])
def test_smallest_temperatures(tv, probs):
    """Down to the smallest normal number, whose reciprocal is finite; below it the sequence is
    refused.  Logits of at most 2^-20 keep z / temperature finite."""
    c = case(5, 2, 300, seed=4, penalties=False, grammar=False, bias=False)
    c["z"] = (c["z"] * 2.0 ** -24).float()
    c["kw"]["temp"] = torch.tensor([1e-3, 2.0 ** -100, 2.0 ** -126, 2.0 ** -127, 1e-45], dtype=torch.float32)
    out, status = process(tv, c, probs)
    assert status.tolist() == [0, 0, 0, 7, 7]
    ref = R.logits(c["z"], probs=probs, temp=c["kw"]["temp"])[:3]
    # one float32 rounding of the reciprocal and one of the product; a probability moves by that
    # times the largest |z| / temperature in the exponent, at most all of itself
    z = (c["z"].double().abs().amax((1, 2)) / c["kw"]["temp"].double())[:3, None, None]
    rel = 4 * 2.0 ** -24
    tol = ref.abs() * rel if not probs else \
        torch.minimum(ref * (2 * rel * z + (300 / 512 + 24) * 2.0 ** -24 + 2.0 ** -20), torch.tensor(1.0).double()) + 2.0 ** -126
    assert ((out[:3].double() - ref).abs() <= tol).all()
    assert out[3:].eq(0.0 if probs else -math.inf).all()


def test_logits_refusals(tv):
    z = torch.zeros(1, 2, 64, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda")
    with pytest.raises(tv.TreeVerifyError):       # a penalty without a history
        tv.tree_logits_process(z, z, st, probs=True, repetition=one)
    with pytest.raises(tv.TreeVerifyError):
        tv.tree_logits_process(z, z, st, probs=True, mask=torch.zeros(1, 2, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        tv.tree_logits_process(z.half(), z, st, probs=True)
    with pytest.raises(ValueError):
        tv.tree_logits_process(z, z, st, probs=True, grammar=torch.zeros(1, 2, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(tv.TreeVerifyError):
        z65 = torch.zeros(1, 65, 8, device="cuda")
        tv.tree_logits_process(z65, z65, st, probs=True)


# ------------------------------------------------------------------ counts

def counts_ref(hist, rows, clear, prompt):
    out = hist.clone()
    for b, r in enumerate(rows):
        if clear:
            out[b] = 0
        for x in r:
            if x < 0:
                continue
            v = int(out[b, x]) & 0xFFFFFFFF
            v = (v | 0x80000000) if prompt else v + 1
            out[b, x] = v - (1 << 32) if v >= 1 << 31 else v
    return out


@pytest.mark.parametrize("clear", [False, True])
@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("V", [1, 70, 8193, 20001])
@pytest.mark.parametrize("ragged", [False, True])
def test_counts(tv, clear, prompt, V, ragged):
    rng = np.random.default_rng(V)
    B = 5
    hist = torch.from_numpy(rng.integers(0, 5, (B, V)).astype(np.int32))
    hist[1] |= -(1 << 31)
    lens = [0, 3, 700, 1, 40] if ragged else [37] * B
    rows = [[int(x) for x in (rng.random(m) ** 2 * V)] for m in lens]
    starts = None
    if ragged:
        starts = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
        tokens = torch.tensor(sum(rows, []), dtype=torch.int32).cuda()
    else:
        for b in range(B):
            rows[b][b:] = [-1] * (37 - b) if b < 3 else rows[b][b:]
        tokens = torch.tensor(rows, dtype=torch.int32).cuda()
    got = hist.cuda()
    st = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    tv.token_counts_update(got, tokens, st, starts=starts, clear=clear, prompt=prompt)
    assert st.eq(0).all()
    assert torch.equal(got.cpu(), counts_ref(hist, rows, clear, prompt))


@pytest.mark.parametrize("clear", [False, True])
def test_counts_bad_sequences(tv, clear):
    V = 9000
    hist = torch.arange(4 * V, dtype=torch.int32).reshape(4, V)
    tokens = torch.tensor([[1, 2, -1], [5, V, 3], [-2, 1, 1], [8999, 8999, 0]], dtype=torch.int32)
    got, st = hist.cuda(), torch.full((4,), -9, dtype=torch.int32, device="cuda")
    tv.token_counts_update(got, tokens.cuda(), st, clear=clear)
    assert st.tolist() == [0, 3, 3, 0]
    want = counts_ref(hist, [[1, 2], [], [], [8999, 8999, 0]], clear, False)
    want[1:3] = hist[1:3]
    assert torch.equal(got.cpu(), want)
    for starts in ([0, 3, 2, 5, 12], [0, 3, 6, 9, 13], [-1, 3, 6, 9, 12]):
        got = hist.cuda()
        tv.token_counts_update(got, tokens.cuda().view(-1), st, clear=clear,
                               starts=torch.tensor(starts, dtype=torch.int32).cuda())
        assert st.eq(3).all() and torch.equal(got.cpu(), hist)

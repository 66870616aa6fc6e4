"""Sampling on the GPU against its definition in 64 bits.  A token or a cut may differ only where an
exact sum comes within 2^-30 of its border (weights are off by 2^-38 of themselves and half a step
of 2^-42, so that sums of up to 2^20 of them are off by less than 2^-30 of theirs)."""
import math

import pytest
import torch

import q8_ref as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import eagle_speculative_decoding_parent_gb300 as m
    return m


def sample(tv, x, u, *, temp=None, k=None, p=None, m=None, probs=True, counts=None):
    B, N, V = x.shape
    tokens = torch.full((B, N), -7, dtype=torch.int32, device="cuda")
    status = torch.full((B, N), -9, dtype=torch.int32, device="cuda")
    out = torch.full((B, N, V), 5.0, device="cuda") if probs else None
    f = lambda t, dt: None if t is None else torch.tensor(t, dtype=dt, device="cuda")  # noqa: E731
    tv.logits_sample(x.cuda(), u.cuda(), tokens, status, temperature=f(temp, torch.float32), top_k=f(k, torch.int32),
                     top_p=f(p, torch.float32), min_p=f(m, torch.float32), probs=out,
                     node_counts=f(counts, torch.int32))
    torch.cuda.synchronize()
    return tokens.cpu(), status.cpu(), None if out is None else out.cpu()


def check(tv, x, u, temp=None, k=None, p=None, m=None):
    B, N, V = x.shape
    tokens, status, probs = sample(tv, x, u, temp=temp, k=k, p=p, m=m)
    bare, status2, _ = sample(tv, x, u, temp=temp, k=k, p=p, m=m, probs=False)
    assert status.eq(0).all() and status2.eq(0).all() and torch.equal(tokens, bare)
    r32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    for b in range(B):
        t, kk, pp, mm = (d if v is None else r32(v[b]) for v, d in ((temp, 1.0), (k, 0), (p, 1.0), (m, 0.0)))
        for i in range(N):
            w, kept, near = Q.sample_sets(x[b, i].float(), t, int(kk), pp, mm)
            got = probs[b, i].double()
            # (a weight below the smallest float32 may be written as zero)
            assert bool(((got > 0) == kept)[~near & (w > 1e-30)].all()), (b, i)
            kept = torch.where(near, got > 0, kept)
            w = torch.where(kept, w, 0.0)
            Z = float(w.sum())
            # 2^-20, and the rounding of the exponent (three roundings of 2^-24 of its size)
            size = ((x[b, i].double().max() - x[b, i].double()) / (t if t > 0 else 1.0)).clamp(max=200)
            tol = w / Z * (2.0 ** -20 + 4 * 2.0 ** -24 * size) + 1e-30
            assert bool(((got - w / Z).abs() <= tol).all()), (b, i, float(((got - w / Z).abs() / tol).max()))
            tok, goal = int(tokens[b, i]), float(u[b, i]) * Z
            below, upto = float(w[:tok].sum()), float(w[:tok + 1].sum())
            assert kept[tok] and below <= goal + 2.0 ** -30 * Z and upto > goal - 2.0 ** -30 * Z, (b, i)


def rows(B, N, V, seed, dtype=torch.float32, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, N, V), generator=g) * spread).to(dtype), torch.rand((B, N), generator=g)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 7, 128, 1000, 4097, 32000, 50257])
def test_filters(tv, dtype, V):
    x, u = rows(8, 2, V, V, dtype)
    check(tv, x, u)
    check(tv, x, u, temp=[0.7, 1.0, 2.0, 0.1, 0.0, 1.3, 0.5, 1.0], k=[0, 1, 5, 50, 3, 1000, V, V + 1],
          p=[0.9, 1.0, 0.5, 0.99, 0.3, 0.95, 1e-6, 0.999], m=[0.0, 0.1, 0.0, 0.01, 1.0, 0.0, 0.0, 0.3])
    check(tv, x, u, p=[0.1, 0.3, 0.5, 0.7, 0.9, 0.95, 0.99, 1.0])
    check(tv, x, u, m=[0.001, 0.01, 0.1, 0.5, 1.0, 0.0, 0.2, 0.05])


@pytest.mark.parametrize("V", [128256, 152064, 262144, 300001])
def test_long_rows(tv, V):
    for dtype in (torch.float32, torch.bfloat16):
        x, u = rows(3, 1, V, V, dtype)
        check(tv, x, u, temp=[0.7, 1.0, 1.5], k=[0, 50, 4000], p=[0.95, 0.9, 1.0], m=[0.0, 0.02, 0.0])


def test_many_rows(tv):
    x, u = rows(20, 20, 3000, 2)
    check(tv, x, u, temp=[0.5 + 0.1 * b for b in range(20)], p=[0.5 + 0.02 * b for b in range(20)], k=[0, 7] * 10)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,N,V", [(60, 22, 3001), (20, 13, 40000), (41, 16, 2100)])
def test_distributions_of_many_rows(tv, dtype, B, N, V):
    """More rows than the GPU holds at once; each sequence with filters of its own."""
    x, u = rows(B, N, V, V, dtype)
    x[1] = 0.25                                                  # rows of equal entries,
    x[2] = (torch.arange(V) % 3).to(dtype)                       # of few different ones,
    x[3, :, ::2] = -math.inf                                     # masked ones,
    x[4] *= 0.01                                                 # nearly flat ones
    x[5, :, 7] = 100.0
    some = [0.0, 0.3, 0.7, 1.0, 1.6]
    check(tv, x, u, temp=[some[b % 5] for b in range(B)], k=[[0, 40, 3, 2000][b % 4] for b in range(B)],
          p=[[1.0, 0.9, 0.99, 0.2, 0.95, 0.5][b % 6] for b in range(B)], m=[[0.0, 0.0, 0.05][b % 3] for b in range(B)])
    # rows that cannot be sampled beside the others
    x[6, 0, 3] = math.nan
    x[7] = -math.inf
    u[8, 1] = 2.0
    tokens, status, probs = sample(tv, x, u, p=[0.9] * B, counts=[N if b != 9 else 3 for b in range(B)])
    assert status[6, 0] == 7 and status[7].eq(7).all() and status[8, 1] == 7 and status[9, 3:].eq(-9).all()
    assert bool((probs[6, 0] == 0).all()) and bool((probs[7] == 0).all()) and bool((probs[9, 3:] == 5.0).all())
    good = torch.ones((B, N), dtype=torch.bool)
    good[6, 0], good[7], good[8, 1], good[9, 3:] = False, False, False, False
    assert status[good].eq(0).all() and bool(((probs[good].double().sum(-1) - 1).abs() < 1e-5).all())


@pytest.mark.parametrize("V", [5, 3000, 40000])
def test_equal_logits(tv, V):
    """Rows with long runs of equal entries, which are taken by their index: whole rows of one value, of a
    few, and runs around the cut."""
    x = torch.zeros((6, 1, V))
    x[1] = torch.arange(V) % 3
    x[2, 0, V // 2:] = 1.0
    x[3] = -0.0
    x[3, 0, ::2] = 0.0
    x[4, 0, :V // 3] = -5.0
    x[5] = (torch.arange(V) % 7 == 2) * 2.0
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 0.1]).view(6, 1)
    for dtype in (torch.float32, torch.bfloat16):
        check(tv, x.to(dtype), u, k=[3, V // 2, 1, V - 1, 2, 2000])
        check(tv, x.to(dtype), u, p=[0.37, 0.5, 0.251, 0.999, 1e-3, 0.7])
        check(tv, x.to(dtype), u, k=[V - 1, V // 2 + 1, 2, V - 2, V // 4 + 1, V // 2], p=[0.3, 0.9, 0.2, 0.5, 0.6, 0.77], m=[0.5] * 6)


def test_wide_and_narrow_temperatures(tv):
    x, u = rows(8, 1, 20000, 9)
    check(tv, x, u, temp=[1e-3, 0.01, 10.0, 1000.0, 1e30, 2.0 ** -126, 0.3, 5.0], p=[0.9] * 8)
    check(tv, x, u, temp=[1e-3, 0.01, 10.0, 1000.0, 1e30, 2.0 ** -126, 0.3, 5.0], k=[100, 5000] * 4)
    check(tv, x * 1e30, u, temp=[1e30, 1e29, 1e31, 3e38, 1.0, 1e28, 1e30, 2e30], p=[0.5] * 8)


def test_masked_entries(tv):
    """-infinity is never drawn, whatever the filters."""
    x, u = rows(5, 1, 10000, 4)
    x[0, 0, 1:] = -math.inf                                     # one entry is left: the first,
    x[1, 0, :-1] = -math.inf                                    # the last
    x[2, 0, ::2] = -math.inf
    x[3, 0, 17:9990] = -math.inf
    x[4, 0, :9000] = -3.4e38
    for kw in (dict(), dict(k=[5000] * 5), dict(p=[0.99] * 5), dict(temp=[0.0] * 5), dict(k=[2] * 5, p=[0.9] * 5, m=[0.01] * 5)):
        check(tv, x, u, **kw)


def test_refused_rows(tv):
    nan, inf = math.nan, math.inf
    x, u = rows(6, 1, 5000, 4)
    x[0, 0, 4000] = nan
    x[1, 0, 3] = inf
    x[2] = -inf
    u[3] = 1.0
    u[4] = nan
    tokens, status, probs = sample(tv, x, u, k=[5] * 6, p=[0.9] * 6)
    assert status.view(-1).tolist() == [7, 7, 7, 7, 7, 0] and bool((tokens[:5] == -1).all())
    assert bool((probs[:5] == 0).all()) and abs(float(probs[5].sum()) - 1) < 1e-4
    x, u = rows(9, 1, 500, 5)
    tokens, status, probs = sample(tv, x, u, temp=[-1.0, nan, inf, 1e-40, 1, 1, 1, 1, 1], p=[1, 1, 1, 1, 0.0, 1.5, nan, 1, 1],
                                   m=[0, 0, 0, 0, 0, 0, 0, -0.1, 1.1])
    assert status.eq(7).all() and tokens.eq(-1).all() and bool((probs == 0).all())


def test_node_counts(tv):
    x, u = rows(4, 5, 700, 6)
    tokens, status, probs = sample(tv, x, u, p=[0.9] * 4, counts=[5, 2, 0, 6])
    assert status[0].eq(0).all() and status[1].tolist() == [0, 0, -9, -9, -9]
    assert status[2].eq(3).all() and status[3].eq(3).all()
    assert tokens[1, 2:].eq(-7).all() and bool((probs[1, 2:] == 5.0).all()) and bool((probs[2:] == 0).all())
    full, _, want = sample(tv, x, u, p=[0.9] * 4)
    assert torch.equal(tokens[0], full[0]) and torch.equal(probs[0], want[0]) and torch.equal(tokens[1, :2], full[1, :2])


def test_misaligned_rows(tv):
    for dtype in (torch.float32, torch.bfloat16):
        x, u = rows(2, 3, 4099, 8, dtype)
        wide = torch.zeros(x.numel() + 1, dtype=dtype, device="cuda")
        wide[1:] = x.view(-1).cuda()
        tokens, status = (torch.zeros((2, 3), dtype=torch.int32, device="cuda") for _ in range(2))
        tv.logits_sample(wide[1:].view(2, 3, 4099), u.cuda(), tokens, status, top_p=torch.tensor([0.8, 0.9], device="cuda"))
        want, _, _ = sample(tv, x, u, p=[0.8, 0.9])
        assert torch.equal(tokens.cpu(), want) and bool((status == 0).all())


def test_draws_follow_the_distribution(tv):
    """20,000 rows of one distribution: every count within six standard deviations."""
    V, n = 40, 20000
    x = torch.linspace(-1, 2, V).expand(n // 50, 50, V).contiguous()
    u = torch.rand((n // 50, 50), generator=torch.Generator().manual_seed(1))
    tokens, status, _ = sample(tv, x, u, k=[30] * (n // 50), probs=False)
    assert status.eq(0).all()
    w, kept, _ = Q.sample_sets(x[0, 0], 1.0, 30, 1.0, 0.0)
    p = torch.where(kept, w, 0.0) / w[kept].sum()
    got = torch.bincount(tokens.view(-1).long(), minlength=V).double()
    assert bool(((got - n * p).abs() <= 6 * (n * p * (1 - p)).sqrt() + 1e-9).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_flat_rows(tv, dtype):
    """Rows in which thousands of entries carry the mass, few of them and more than the GPU holds at once."""
    for B, N, V, spread in ((3, 1, 128256, 3.0), (2, 1, 60000, 2.0), (30, 20, 32000, 2.5), (8, 12, 128256, 3.0)):
        x, u = rows(B, N, V, B + V, dtype, spread)
        if B * N > 200:                                          # (the reference on the CPU: some sequences)
            x[3:] = x[0] * 0.5
        keep = [0, 1, 2, B - 1]
        p, k, temp = ([v[b % 4] for b in range(B)] for v in ([0.95, 0.9, 0.97, 0.6], [0, 20000, 0, 3000], [1.0, 1.2, 0.9, 1.5]))
        m = [[0.0, 0.0, 2e-4, 0.0][b % 4] for b in range(B)]
        tokens, status, probs = sample(tv, x, u, temp=temp, k=k, p=p, m=m)
        assert status.eq(0).all() and bool(((probs.double().sum(-1) - 1).abs() < 1e-5).all())
        for b in keep[:B]:
            some = lambda v: [v[b]]  # noqa: E731
            check(tv, x[b:b + 1, :2], u[b:b + 1, :2], temp=some(temp), k=some(k), p=some(p), m=some(m))
            for i in range(min(N, 2)):                           # alone or among many: the same token, the same entries
                t1, _, p1 = sample(tv, x[b:b + 1, i:i + 1], u[b:b + 1, i:i + 1], temp=some(temp), k=some(k), p=some(p), m=some(m))
                assert int(t1) == int(tokens[b, i]) and torch.equal(p1[0, 0] > 0, probs[b, i] > 0)
                assert bool(((p1[0, 0] - probs[b, i]).abs() <= 2.0 ** -18 * p1[0, 0]).all())


def test_longest_rows(tv):
    for dtype in (torch.float32, torch.bfloat16):
        x, u = rows(2, 1, 786432, 3, dtype)
        check(tv, x, u, k=[50, 0], p=[0.9, 0.3])
        x, u = rows(1, 1, 786433, 3, dtype)
        tokens = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
        if dtype == torch.float32:
            with pytest.raises(tv.TreeVerifyError):
                tv.logits_sample(x.cuda(), u.cuda(), tokens, tokens.clone())


def test_streams_and_graphs(tv):
    """Two calls at once on streams of their own; a captured call replayed on other rows and filters."""
    f = lambda v, dt=torch.float32: torch.tensor(v, dtype=dt, device="cuda")  # noqa: E731
    for B, N, V in ((4, 1, 20000), (80, 10, 5000)):
        data = [rows(B, N, V, s) for s in (1, 2)]
        p = [[0.9, 0.5, 1.0, 0.97][b % 4] for b in range(B)]
        k = [[0, 40, 7][b % 3] for b in range(B)]
        want = [sample(tv, x, u, p=p, k=k) for x, u in data]
        bufs = [dict(x=x.cuda(), u=u.cuda(), tok=torch.zeros((B, N), dtype=torch.int32, device="cuda"),
                     st=torch.full((B, N), -9, dtype=torch.int32, device="cuda"), pr=torch.full((B, N, V), 5.0, device="cuda"))
                for x, u in data]
        P, K = f(p), f(k, torch.int32)
        streams = [torch.cuda.Stream() for _ in bufs]
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s in zip(bufs, streams):
                tv.logits_sample(g["x"], g["u"], g["tok"], g["st"], top_p=P, top_k=K, probs=g["pr"], stream=s)
        torch.cuda.synchronize()
        for g, (tokens, _, probs) in zip(bufs, want):
            assert g["st"].eq(0).all() and torch.equal(g["tok"].cpu(), tokens) and torch.equal(g["pr"].cpu(), probs)
        g = bufs[0]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tv.logits_sample(g["x"], g["u"], g["tok"], g["st"], top_p=P, top_k=K, probs=g["pr"])
        for i in (1, 0, 1):
            g["x"].copy_(data[i][0])
            g["u"].copy_(data[i][1])
            g["pr"].fill_(3.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(g["tok"].cpu(), want[i][0]) and torch.equal(g["pr"].cpu(), want[i][2])
        P.fill_(0.4)
        graph.replay()
        torch.cuda.synchronize()
        again = sample(tv, data[1][0], data[1][1], p=[0.4] * B, k=k)
        assert torch.equal(g["tok"].cpu(), again[0]) and torch.equal(g["pr"].cpu(), again[2])


def test_the_same_bits_alone_or_with_distributions(tv):
    """Tokens do not depend on whether the distributions are asked for, nor on the rows around them."""
    x, u = rows(100, 10, 6000, 7)
    p, k = [[0.9, 1.0, 0.6][b % 3] for b in range(100)], [[0, 30][b % 2] for b in range(100)]
    tokens, _, probs = sample(tv, x, u, p=p, k=k)
    bare, _, _ = sample(tv, x, u, p=p, k=k, probs=False)
    assert torch.equal(tokens, bare)
    for b in (0, 17, 99):
        one, _, _ = sample(tv, x[b:b + 1], u[b:b + 1], p=p[b:b + 1], k=k[b:b + 1])
        assert torch.equal(one[0], tokens[b])

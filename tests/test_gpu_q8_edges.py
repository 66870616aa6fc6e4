"""Attention over an 8-bit cache where it can go wrong: refused sequences, NaN among the codes, the whole
range of codes and scales, strides, streams, graphs, caches past 2^31 bytes.  Both kernels: a few rows
per sequence, and more."""
import pytest
import torch

import chunk_ref as R
import q8_ref as Q
from test_gpu_q8 import attend, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import eagle_speculative_decoding_parent_gb300 as m
    return m


FEW, MORE = [1, 2, 1, 3, 1, 0], [40, 33, 64, 5, 17, 0]


def matches(c, out, status, keep=None, **kw):
    ref, A, S = Q.attention(c, **kw)
    tol = R.attention_tolerance(c, ref, A, S, c["q"].shape[2])
    nan = ref.isnan()
    at = c["q_start"].tolist()
    for b in range(len(c["n"])) if keep is None else keep:
        rows = slice(at[b], at[b + 1])
        assert status[b] == 0, b
        assert torch.equal(out[rows].isnan(), nan[rows]), b
        assert ((out[rows].double() - ref[rows]).abs() <= tol[rows])[~nan[rows]].all(), b


# ------------------------------------------------------------------ refused sequences

@pytest.mark.parametrize("n", [FEW, MORE])
@pytest.mark.parametrize("d", [128, 64])
def test_refused_sequences(tv, n, d):
    """Their rows are zero and the others right."""
    P = [300, 70, 500, 20, 33, 9]
    c = Q.cache_case(n, P, Hq=8, Hkv=2, d=d, bs=16, seed=1)
    bad = dict(c, table=c["table"].clone(), prefix=c["prefix"].clone())
    bad["table"][0, 7] = 10 ** 6
    bad["table"][1, 0] = -5
    bad["prefix"][2] = -1
    bad["prefix"][4] = c["table"].shape[1] * 16 - n[4] + 1
    out, status = attend(tv, bad)
    assert status.tolist() == [3, 3, 3, 0, 3, 0]
    matches(c, out, status, [3, 5])
    at = c["q_start"].tolist()
    for b in (0, 1, 2, 4):
        assert bool((out[at[b]:at[b + 1]] == 0).all()), b
    # a bad q_start: everyone is refused
    for starts in ([0, 5, 4, 5, 6, 7, 7], [-1, 0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5, 10 ** 6]):
        out, status = attend(tv, dict(c, q_start=torch.tensor(starts, dtype=torch.int32)))
        assert status.eq(3).all()


@pytest.mark.parametrize("n", [[1, 2, 1], [30, 50, 40]])
def test_blocks_that_a_window_needs(tv, n):
    """Blocks wholly before the window may be gone, but not those of the first tokens."""
    c = Q.cache_case(n, [200, 310, 90], Hq=4, Hkv=2, d=64, bs=16, seed=3, first_block=[9, 16, 2])
    out, status = attend(tv, c, window=50)
    matches(c, out, status, window=50)
    c["table"][0, 0] = c["table"][1, 0] = c["table"][2, 0] = int(c["table"][0, 10])
    out, status = attend(tv, c, window=50, sinks=16)
    matches(c, out, status, window=50, sinks=16)
    _, status = attend(tv, c, window=50, sinks=17)             # the second block's first token
    assert status.eq(3).all()
    _, status = attend(tv, c)
    assert status.eq(3).all()


@pytest.mark.parametrize("d", [128, 64])
def test_more_than_64_rows_with_a_mask(tv, d):
    n = [64, 65, 3]
    c = Q.cache_case(n, [10, 20, 30], Hq=4, Hkv=4, d=d, bs=16, seed=2)
    mask = torch.full((sum(n),), -1, dtype=torch.int64)
    out, status = attend(tv, c, mask=mask)
    assert status.tolist() == [0, 3, 0] and bool((out[64:129] == 0).all())
    matches(c, out, status, [0, 2], mask=mask)
    few = Q.cache_case([1] * 70 + [65], [5] * 71, Hq=1, Hkv=1, d=d, bs=16, seed=2)
    mask = torch.full((135,), -1, dtype=torch.int64)
    out, status = attend(tv, few, mask=mask)
    assert status.tolist() == [0] * 70 + [3] and bool((out[70:] == 0).all())
    matches(few, out, status, range(70), mask=mask)


# ------------------------------------------------------------------ NaN

def poison(c, name, b, t, g, col=None):
    blk, row = int(c["table"][b, t // c["bs"]]), t % c["bs"]
    code = c[name + "_cache"].view(torch.uint8)
    code[blk, g, row, slice(None) if col is None else col] = 0x7F if t % 2 else 0xFF


@pytest.mark.parametrize("n", [[1, 3, 2], [40, 64, 9]])
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 32), (128, 48)])
def test_nan_where_no_row_looks(tv, n, d, bs):
    """Every row of the caches that no row attends to is NaN."""
    P = [150, 37, 260]
    for kw in (dict(), dict(window=33), dict(window=33, sinks=5), dict(mask=Q.trees(n, 5))):
        c = Q.cache_case(n, P, Hq=8, Hkv=2, d=d, bs=bs, seed=n[0] + d)
        some = torch.zeros(c["k_cache"].shape[:3], dtype=torch.bool)
        for b in range(3):
            seen = Q.seen_keys(c, b, kw.get("window", 0), kw.get("sinks", 0), kw.get("mask")).any(0).nonzero().view(-1)
            some[c["table"][b][seen // bs].long(), :, seen % bs] = True
        for x in ("k_cache", "v_cache"):
            c[x].view(torch.uint8)[~some] = 0x7F
        out, status = attend(tv, c, **kw)
        assert torch.isfinite(out.double()).all()
        matches(c, out, status, **kw)


@pytest.mark.parametrize("n", [[1, 3, 2], [40, 64, 9]])
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 32)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_nan_that_some_rows_see(tv, n, d, bs, which):
    """A NaN reaches the rows (K) or the columns of the rows (V) that attend to it and no others."""
    P = [150, 37, 260]
    for kw in (dict(), dict(window=20), dict(window=20, sinks=5), dict(mask=Q.trees(n, 5)), dict(softcap=20.0)):
        c = Q.cache_case(n, P, Hq=8, Hkv=2, d=d, bs=bs, seed=n[0] + d)
        poison(c, which, 0, P[0] + n[0] - 1, 1, 7)             # the last row's own
        poison(c, which, 1, P[1] + 1, 0, 63)                   # a node in the middle
        poison(c, which, 1, P[1] + 2, 0)
        poison(c, which, 2, P[2] - 15, 1, 3)                   # some windows hold it
        poison(c, which, 2, 2, 0, 5)
        out, status = attend(tv, c, **kw)
        ref = Q.attention(c, **kw)[0]
        assert ref.isnan().any() and not ref.isnan().all()
        matches(c, out, status, **kw)


# ------------------------------------------------------------------ numbers

@pytest.mark.parametrize("n", [[1, 3, 2], [40, 64, 9]])
@pytest.mark.parametrize("d", [128, 64])
def test_every_code(tv, n, d):
    c = Q.cache_case(n, [150, 37, 260], Hq=8, Hkv=2, d=d, bs=16, seed=d)
    for x in ("k", "v"):
        codes = (torch.arange(c[x + "_cache"].numel()) * 37 % 254)
        codes = torch.where(codes >= 127, codes + 1, codes)     # not 0x7f, 0xff
        c[x + "_cache"] = codes.to(torch.uint8).view(c[x + "_cache"].shape).view(Q.E4M3)
        c[x + "_scale"] *= 2.0 ** -4
    check(tv, c)
    check(tv, c, mask=Q.trees(n, 2), softcap=10.0)


@pytest.mark.parametrize("n", [[1, 3, 2], [40, 64, 9]])
@pytest.mark.parametrize("d", [128, 64])
def test_scales_of_the_whole_range(tv, n, d):
    """Blocks of values whose scales lie 2^200 apart, among them blocks of zeros (with the smallest
    scale), whose keys have their weight all the same; keys of almost nothing beside ordinary ones."""
    g = torch.Generator().manual_seed(d)
    for exps in ([-100, 100], [-100, -60, 0, 30, 60, 100], [100], [-100], [-100, 45], [-70, -61, -60, -59, 10]):
        c = Q.cache_case(n, [150, 37, 260], Hq=8, Hkv=2, d=d, bs=16, seed=d)
        shape = c["v_scale"].shape
        e = torch.tensor(exps, dtype=torch.float64)[torch.randint(0, len(exps), shape, generator=g)]
        c["v_scale"] = torch.exp2(e).float()
        c["v_cache"] = (torch.randn(c["v_cache"].shape, generator=g) * 40).clamp(-120, 120).to(Q.E4M3)
        zero = torch.rand(shape, generator=g) < 0.3
        c["v_cache"].view(torch.uint8)[zero] = 0
        c["v_scale"][zero] = 2.0 ** -100
        c["k_scale"][torch.rand(shape, generator=g) < 0.3] = 2.0 ** -100
        check(tv, c)
        check(tv, c, window=40, sinks=3)


@pytest.mark.parametrize("n", [[1, 3, 2], [40, 64, 9]])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("by", [2.0 ** -120, 2.0 ** -30, 40.0, 2.0 ** 40])
def test_small_and_large_queries(tv, n, d, by):
    """Scores of thousands (one key takes it all, or two that are equal) and of nothing; scales that
    bring queries of any size back."""
    c = Q.cache_case(n, [150, 37, 260], Hq=8, Hkv=2, d=d, bs=16, seed=d)
    c["q"] *= by
    if by == 40.0:
        check(tv, c)
        check(tv, c, softcap=30.0)
    else:
        c["k_scale"] *= 2.0 ** -30 if by > 1 else 1.0
        check(tv, c, scale=0.1 * 2.0 ** -10 if by > 1 else 0.0)


@pytest.mark.parametrize("n", [[1, 3, 2], [40, 64, 9]])
def test_odd_query_rows(tv, n):
    """Zero rows take the mean; rows with NaN or infinity give NaN, and only they."""
    for d in (128, 64):
        c = Q.cache_case(n, [150, 37, 260], Hq=8, Hkv=2, d=d, bs=16, seed=d)
        c["q"][0] = 0.0
        c["q"][2, 3, 5], c["q"][2, 4, 0], c["q"][1, 7, d - 1] = float("nan"), float("inf"), float("-inf")
        out, status = attend(tv, c)
        assert status.eq(0).all()
        odd = torch.zeros(c["q"].shape[:2], dtype=torch.bool)
        odd[2, 3], odd[2, 4], odd[1, 7] = True, True, True
        assert bool(out[odd].isnan().all())
        fine = dict(c, q=torch.where(odd[..., None], 0.0, c["q"]))
        ref, A, S = Q.attention(fine)
        tol = R.attention_tolerance(fine, ref, A, S, d)
        assert ((out.double() - ref).abs() <= tol)[~odd].all()


@pytest.mark.parametrize("n", [[1, 2], [40, 20]])
def test_nothing_to_see(tv, n):
    """A row whose mask is empty, with nothing before its sequence, is zero."""
    c = Q.cache_case(n, [0, 3], Hq=8, Hkv=2, d=128, bs=16, seed=3)
    mask = torch.zeros(sum(n), dtype=torch.int64)
    out, status = attend(tv, c, mask=mask)
    assert bool((out[:n[0]] == 0).all())
    matches(c, out, status, mask=mask)


# ------------------------------------------------------------------ buffers

@pytest.mark.parametrize("n", [FEW, MORE])
@pytest.mark.parametrize("d", [128, 64])
def test_strided_rows_and_rows_of_no_sequence(tv, n, d):
    c = Q.cache_case(n, [30, 200, 17, 90, 0, 4], Hq=8, Hkv=2, d=d, bs=16, seed=1)
    T = sum(n)
    wide_q = torch.randn((T + 7, 12, d), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    wide_o = torch.full((T + 7, 9, d), 5.0, dtype=torch.bfloat16, device="cuda")
    wide_q[3:T + 3, 2:10] = c["q"].cuda()
    shifted = dict(c, q_start=c["q_start"] + 3)
    out, status = attend(tv, shifted, q=wide_q[:, 2:10], out=wide_o[:, :8])
    matches(c, out[3:T + 3], status)
    wide_o = wide_o.cpu()
    assert bool((wide_o[:3] == 5.0).all()) and bool((wide_o[T + 3:] == 5.0).all()) and bool((wide_o[:, 8:] == 5.0).all())


def test_no_rows(tv):
    c = Q.cache_case([0, 0, 0], [5, 0, 40], Hq=4, Hkv=2, d=64, bs=16, seed=1)
    c["prefix"][1] = -3
    _, status = attend(tv, c)
    assert status.tolist() == [0, 3, 0]
    q = torch.zeros((4, 4, 64), dtype=torch.bfloat16, device="cuda")       # rows, but of no sequence
    out = torch.full_like(q, 3.0)
    _, status = attend(tv, c, q=q, out=out)
    assert status.tolist() == [0, 3, 0] and bool((out == 3.0).all())


@pytest.mark.parametrize("d", [128, 64])
def test_caches_past_32_bits(tv, d):
    """Append, attention and moving in caches of more than 2^31 bytes, in their last blocks."""
    n, P = [5, 30, 1], [100, 40, 260]
    c = Q.cache_case(n, P, Hq=8, Hkv=8, d=d, bs=16, seed=d)
    small = c["k_cache"].shape[0]
    total = (1 << 31) // (8 * 16 * d) + 1000
    far = dict(c, table=torch.where(c["table"] >= 0, c["table"] + (total - small), c["table"]))
    g = {}
    for x in ("k_cache", "v_cache"):
        g[x] = torch.zeros((total, 8, 16, d), dtype=torch.uint8, device="cuda").view(Q.E4M3)
        g[x][total - small:] = c[x].cuda()
    for x in ("k_scale", "v_scale"):
        g[x] = torch.full((total, 8), 2.0 ** 60, device="cuda")
        g[x][total - small:] = c[x].cuda()
    args = [g["k_cache"], g["v_cache"], g["k_scale"], g["v_scale"], far["table"].cuda()]
    T, pre, start = sum(n), c["prefix"].cuda(), c["q_start"].cuda()
    status = torch.full((3,), -9, dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.randn((T, 8, d), generator=gen).bfloat16() for _ in range(2))
    tv.chunk_kv_append_q8(None, k.cuda(), v.cuda(), *args, start, pre, status)
    assert status.eq(0).all()
    for x, rows in (("k", k), ("v", v)):
        code, scale = Q.append(c, x, rows.double())
        c[x + "_cache"], c[x + "_scale"] = code.view(Q.E4M3), scale.float()
        assert torch.equal(g[x + "_cache"][total - small:].view(torch.uint8).cpu(), code)
        assert torch.equal(g[x + "_scale"][total - small:].cpu().double(), scale)
    for few in (False, True):
        h = c if not few else dict(c, n=[1, 1, 1], q=c["q"][:3], q_start=torch.arange(4, dtype=torch.int32))
        q = h["q"].cuda()
        out = torch.zeros_like(q)
        ws = torch.zeros(tv.chunk_attention_q8_workspace(q.shape[0], 3, 8, 8, d), dtype=torch.uint8, device="cuda")
        tv.chunk_attention_q8(q, *args, h["q_start"].cuda(), pre, out, status, ws)
        matches(h, out.cpu(), status.cpu())
    path = torch.tensor([[0, 2, 4], [0, 9, 29], [0, -1, -1]], dtype=torch.int32)
    accept = torch.tensor([2, 2, 0], dtype=torch.int32)
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    tv.kv_compact_q8(*args, pre, path.cuda(), accept.cuda(), new, status)
    assert status.eq(0).all()
    for x in ("k", "v"):
        code, scale = Q.compact(c, x, path, accept)
        assert torch.equal(g[x + "_cache"][total - small:].cpu().float(), code.view(Q.E4M3).float())
        assert torch.equal(g[x + "_scale"][total - small:].cpu().double(), scale)


# ------------------------------------------------------------------ streams and graphs

def on_gpu(tv, c):
    g = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    T, Hq, d = c["q"].shape
    B = len(c["n"])
    g["out"] = torch.zeros_like(g["q"])
    g["status"] = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    g["need"] = tv.chunk_attention_q8_workspace(T, B, Hq, c["k_cache"].shape[1], d)
    return g


def run(tv, g, ws, **kw):
    tv.chunk_attention_q8(g["q"], g["k_cache"], g["v_cache"], g["k_scale"], g["v_scale"], g["table"], g["q_start"], g["prefix"],
                          g["out"], g["status"], ws, **kw)


@pytest.mark.parametrize("n,other", [(FEW, [2, 1, 1, 1, 2, 1]), (MORE, [64, 5, 33, 17, 40, 0])])
def test_captured_calls_and_a_shared_workspace(tv, n, other):
    """Two captured calls with one workspace, replayed in turn; the rows split anew between replays."""
    P = [500, 300, 77, 0, 1000, 60]
    a, b = (Q.cache_case(n, P, Hq=8, Hkv=2, d=128, bs=16, seed=s) for s in (1, 2))
    ga, gb = on_gpu(tv, a), on_gpu(tv, b)
    ws = torch.zeros(max(ga["need"], gb["need"]), dtype=torch.uint8, device="cuda")
    run(tv, ga, ws)
    torch.cuda.synchronize()
    graphs = []
    for g in (ga, gb):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(tv, g, ws)
        graphs.append(graph)
    split = torch.tensor([0] + other).cumsum(0).to(torch.int32)
    for starts, m in ((a["q_start"], n), (split, other)):
        for g in (ga, gb):
            g["q_start"].copy_(starts)
            g["out"].fill_(7.0)
        for graph in graphs * 2:
            graph.replay()
        torch.cuda.synchronize()
        for c, g in ((a, ga), (b, gb)):
            # (positions past the first case's own have codes too: the table is as long as the longest)
            ok = [i for i in range(6) if P[i] + m[i] <= P[i] + n[i]]
            h = dict(c, n=m, q_start=starts)
            h["n"] = [x if i in ok else 0 for i, x in enumerate(m)]
            matches(h, g["out"].cpu(), g["status"].cpu(), ok)


@pytest.mark.parametrize("n", [FEW, MORE])
def test_streams(tv, n):
    """On streams of their own, two calls at once with a workspace each."""
    P = [500, 300, 77, 0, 1000, 60]
    cases = [Q.cache_case(n, P, Hq=8, Hkv=2, d=64, bs=16, seed=s) for s in (3, 4)]
    gs = [on_gpu(tv, c) for c in cases]
    ws = [torch.zeros(g["need"], dtype=torch.uint8, device="cuda") for g in gs]
    streams = [torch.cuda.Stream() for _ in gs]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, w, s in zip(gs, ws, streams):
            run(tv, g, w, stream=s)
    torch.cuda.synchronize()
    for c, g in zip(cases, gs):
        matches(c, g["out"].cpu(), g["status"].cpu())


def test_same_bits_every_time(tv):
    for n in (FEW, MORE):
        c = Q.cache_case(n, [5000, 300, 77, 0, 1000, 60], Hq=8, Hkv=2, d=128, bs=16, seed=3)
        first = attend(tv, c)[0]
        for _ in range(5):
            assert torch.equal(first, attend(tv, c)[0])


# ------------------------------------------------------------------ shapes between the two kernels

@pytest.mark.parametrize("heads", [(128, 1), (24, 1), (28, 4), (5, 5), (65, 1)])
def test_query_heads_per_kv_head_of_128(tv, heads):
    for n, P in (([5, 1, 40], [30, 260, 0]), ([1, 1], [300, 17]), ([130, 3], [5, 600])):
        c = Q.cache_case(n, P, Hq=heads[0], Hkv=heads[1], d=128, bs=16, seed=heads[0])
        check(tv, c)
        if max(n) <= 64:
            check(tv, c, mask=Q.trees(n, 4))


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("G,each", [(1, 8), (1, 9), (1, 16), (1, 17), (1, 24), (1, 25), (4, 2), (4, 3), (4, 4), (4, 5), (4, 6),
                                    (4, 7), (8, 1), (7, 3), (3, 5), (24, 1)])
def test_rows_per_sequence(tv, d, G, each):
    """Around the numbers of rows at which another form is taken; lengths around the average."""
    n = [max(0, each + e) for e in (0, 1, -1, 0, 2, -2)]
    c = Q.cache_case(n, [40, 200, 7, 1000, 0, 128], Hq=2 * G, Hkv=2, d=d, bs=16, seed=each)
    check(tv, c)
    check(tv, c, window=30, sinks=6, softcap=15.0)
    check(tv, c, mask=Q.trees(n, each))


@pytest.mark.parametrize("d", [128, 64])
def test_prompt_among_decoding_sequences(tv, d):
    """Few rows on average, but a long chunk among them."""
    n, P = [300] + [1] * 150, [700] + [(b * 53) % 900 for b in range(150)]
    c = Q.cache_case(n, P, Hq=8, Hkv=2, d=d, bs=16, seed=1)
    check(tv, c)
    check(tv, c, window=100, sinks=4)

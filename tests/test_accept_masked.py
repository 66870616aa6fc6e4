"""Greedy acceptance of rows that a grammar or a failed sequence has masked: -infinity never wins,
so a row without a token above it chooses nothing."""
import ctypes

import numpy as np
import pytest

from test_chunk_host import NZ, I, P, SZ, lib  # noqa: F401  (the fixture)


def test_host_checks(lib):  # noqa: F811
    f = lib.tree_accept
    f.argtypes = [I, P, P, P, P, I, I, P, I, ctypes.c_uint64, ctypes.c_uint64, P, P, P, I, P, P, SZ, P]
    call = lambda mode, B=0, draft=None: f(  # noqa: E731
        mode, NZ, NZ, NZ, draft, B, 4, None, 10, 0, 0, NZ, NZ, NZ, 4, NZ, None, 0, None)
    assert [call(m) for m in (0, 1, 2)] == [0, 0, 0]
    assert call(3) == 1 and call(-1) == 1
    assert call(1, B=2) == 1                     # stochastic: needs draft_probs
    ws = lib.tree_accept_workspace
    ws.restype, ws.argtypes = SZ, [I] * 4
    for shape in ((1, 8, 128256), (3, 26, 1000), (64, 26, 128256), (300, 12, 37)):
        assert ws(2, *shape) == ws(0, *shape)    # the same kernels as unmasked greedy


torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import eagle_speculative_decoding_parent_gb300 as m
    return m


def accept(tv, mode, par, tok, z, max_path):
    B, N, V = z.shape
    par, tok = (torch.from_numpy(x).cuda() for x in (par, tok))
    out = [torch.full(s, -9, dtype=torch.int32, device="cuda") for s in ((B,), (B, max_path), (B, max_path), (B,))]
    ws = torch.zeros(max(16, tv.tree_accept_workspace(mode, B, N, V)), dtype=torch.uint8, device="cuda")
    tv.tree_accept(mode, par, tok, torch.from_numpy(z).cuda(), None, *out, workspace=ws)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in out]


@gpu
@pytest.mark.parametrize("B", [2, 40, 300])       # the row scan, and the walk level by level
@pytest.mark.parametrize("V", [1, 37, 4096, 20001])
def test_masked_greedy_is_greedy_with_nan_for_masked_rows(tv, orc, B, V):
    """Against the unmasked rule's oracle on rows whose -infinity-only ones are NaN."""
    rng = np.random.default_rng(B + V)
    N = 9
    par = np.full((B, N), -1, np.int32)
    for i in range(1, N):
        par[:, i] = rng.integers(0, i, B)
    z = rng.integers(-2, 3, (B, N, V)).astype(np.float32)
    z[rng.random((B, N, V)) < 0.5] = -np.inf
    z[rng.random((B, N)) < 0.3] = -np.inf
    z[0] = -np.inf
    z[1, 0, :] = np.nan
    am = np.where(np.isnan(z), -np.inf, z).argmax(2)
    # drafts that follow the unmasked rule, token 0 behind a masked row among them
    tok = np.take_along_axis(am, np.maximum(par, 0), 1).astype(np.int32)
    tok[:, 1::4] = rng.integers(0, V, tok[:, 1::4].shape)
    nan = z.copy()
    nan[(z == -np.inf).all(2)] = np.nan
    got = accept(tv, tv.GREEDY_MASKED, par, tok, z, N)
    want = orc.accept_greedy(par, tok, nan, N)
    for x, y in zip(got, want):
        assert np.array_equal(x, y)
    assert got[3][0] == 7 and (got[2][0] == -1).all()
    # the unmasked rule keeps its results
    for x, y in zip(accept(tv, tv.GREEDY, par, tok, z, N), orc.accept_greedy(par, tok, z, N)):
        assert np.array_equal(x, y)


@gpu
@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("reps", [1, 30])
@pytest.mark.parametrize("captured", [False, True])
def test_verify_step_emits_nothing_for_failed_sequences(tv, mode, reps, captured):
    """A temperature of 0, a root whose grammar allows nothing, a good sequence, a grammar that
    allows nothing after the first accepted draft, a token past the vocabulary: the four that
    cannot choose a token emit none, and their history and cache stay as they were."""
    from eagle_speculative_decoding_parent_gb300.pipeline import VerifyStep
    N, V, Hq, Hkv, d, bs, blocks = 4, 64, 4, 2, 64, 16, 3
    B = 5 * reps
    g = torch.Generator().manual_seed(mode)
    i32 = dict(dtype=torch.int32, device="cuda")
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    par = torch.tensor([[-1, 0, 1, 2], [-1, 0, 0, 1], [-1, 0, 1, 2], [-1, 0, 1, 2], [-1, 0, 0, 0]] * reps, **i32)
    draft = torch.tensor([[9, 0, 0, 0], [9, 0, 3, 0], [9, 5, 6, 7], [9, 5, 0, 0], [9, 5, 6, V]] * reps, **i32)
    raw = rand(B, N, V)
    raw[:, 0, 5] = 40.0                         # token 5 follows the root
    raw[:, 1, 6], raw[:, 2, 7] = 40.0, 40.0
    grammar = torch.full((B, N, V // 32), -1, dtype=torch.int32)
    grammar[1::5, 0] = 0
    grammar[3::5, 1] = 0
    temp = torch.tensor([0.0, 1.0, 1.0, 1.0, 1.0] * reps)
    probs = torch.softmax(rand(B, N, V), -1).cuda() if mode else None
    cache = [rand(B * blocks, Hkv, bs, d).to(torch.bfloat16).cuda() for _ in range(2)]
    table = torch.arange(B * blocks, **i32).view(B, blocks)
    prefix = torch.tensor([20, 3, 17, 30, 8] * reps, **i32)
    counts = torch.randint(0, 3, (B, V), generator=g).to(torch.int32).cuda()
    step = VerifyStep(B=B, N=N, Hq=Hq, Hkv=Hkv, d=d, max_blocks=blocks, bs=bs, dtype=torch.bfloat16,
                      max_path=N, V=V, mode=mode, process=True)
    args = dict(parents=par, q=rand(B, N, Hq, d).to(torch.bfloat16).cuda(), k_cache=cache[0], v_cache=cache[1],
                block_table=table, prefix_lens=prefix, draft_tokens=draft, target=raw.cuda(), draft_probs=probs,
                mode=mode, seed=3, offset=1,
                sampling=dict(counts=counts, grammar=grammar.cuda(), temperature=temp.cuda()))
    old_counts, old = counts.clone(), [t.clone() for t in cache]
    if captured:
        graph = step.capture(**args)
        counts.copy_(old_counts)
        for t, o in zip(cache, old):
            t.copy_(o)
        graph.replay()
    else:
        step.run(**args)
    torch.cuda.synchronize()
    assert step.st_process.view(reps, 5).cpu().eq(torch.tensor([7, 0, 0, 0, 3])).all()
    assert step.st_accept.view(reps, 5).cpu().eq(torch.tensor([7, 7, 0, 7, 3])).all()
    failed = torch.tensor([True, True, False, True, True] * reps).cuda()
    assert step.out_tokens[failed].eq(-1).all() and step.accept_len[failed].eq(0).all()
    assert step.new_lens[failed].eq(prefix[failed] + 1).all()
    assert torch.equal(counts[failed], old_counts[failed])
    for t, o in zip(cache, old):
        rows = table[failed].view(-1).long()
        assert torch.equal(t[rows], o[rows])
    good = ~failed
    emitted = step.out_tokens[good]
    assert emitted[:, 0].eq(5).all() and step.st_counts.eq(0).all()
    want = old_counts[good].clone()
    want.scatter_add_(1, emitted.clamp(min=0).long(), (emitted >= 0).to(torch.int32))
    assert torch.equal(counts[good], want)

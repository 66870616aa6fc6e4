"""Chunks of new tokens on the GPU: chunk_attention and chunk_kv_append against their
definitions in 64 bits, with bounds derived from the roundings the kernels make."""
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


def attend(tv, c, *, out=None, q=None, stream=None, **kw):
    """Runs chunk_attention on a case of chunk_ref (CPU tensors); (out, status)."""
    g = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    q = g["q"] if q is None else q
    T, Hq, d = q.shape
    B = len(c["n"])
    out = torch.full_like(g["q"], 7.0) if out is None else out
    status = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    ws = torch.full((max(16, tv.chunk_attention_workspace(T, B, Hq, c["k_cache"].shape[1], d, q.dtype)),),
                    0xFF, dtype=torch.uint8, device="cuda")
    tv.chunk_attention(q, g["k_cache"], g["v_cache"], g["table"], g["q_start"], g["prefix"], out,
                       status, ws, **kw)
    torch.cuda.synchronize()
    return out.cpu(), status.cpu()


def check(tv, c, **kw):
    out, status = attend(tv, c, **kw)
    assert status.eq(0).all(), status
    ref, A, S = R.attention(c, **kw)
    tol = R.attention_tolerance(c, ref, A, S, c["q"].shape[2])
    err = (out.double() - ref).abs()
    assert torch.isfinite(out.double()).all()
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max()))


# (n, P) per sequence: single tokens, tile borders of rows and keys, empty sequences, long ones
LENGTHS = [
    ([1], [0]),
    ([1], [300]),
    ([1, 1, 1, 1, 1], [0, 15, 127, 128, 1000]),
    ([0, 3, 0, 17, 1, 0], [5, 0, 0, 250, 129, 7]),
    ([64, 65, 31], [0, 63, 512]),
    ([257], [1]),
    ([200, 1, 333], [77, 2049, 0]),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("heads,d,bs", [((8, 2), 128, 16), ((7, 1), 64, 32), ((4, 4), 128, 48)])
@pytest.mark.parametrize("case", range(len(LENGTHS)))
def test_attention_lengths(tv, dtype, heads, d, bs, case):
    n, P = LENGTHS[case]
    check(tv, R.cache_case(n, P, Hq=heads[0], Hkv=heads[1], d=d, bs=bs, dtype=dtype, seed=case))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window", [1, 2, 17, 128, 200, 4000])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_attention_window_and_cap(tv, dtype, window, cap):
    n, P = [1, 140, 0, 33, 300], [700, 0, 9, 513, 260]
    for heads, d in (((8, 2), 128), ((6, 2), 64)):
        c = R.cache_case(n, P, Hq=heads[0], Hkv=heads[1], d=d, bs=16, dtype=dtype, seed=window)
        check(tv, c, window=window, softcap=cap)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cap", [1e-42, 1e-30, 0.01, 3.0, 1000.0, 1e6, 1e20, 1e31])
def test_attention_caps_of_any_size(tv, dtype, cap):
    """Scores far below, around and far above the cap, in the same tile."""
    for heads, d in (((4, 2), 64), ((4, 1), 128)):
        c = R.cache_case([150, 1], [100, 300], Hq=heads[0], Hkv=heads[1], d=d, bs=16, dtype=dtype, seed=5)
        c["q"] *= torch.tensor([0.1, 1.0, 4.0])[torch.arange(151) % 3][:, None, None].to(dtype)
        check(tv, c, softcap=cap)


@pytest.mark.parametrize("d", [32, 96, 160, 224, 256])
def test_attention_f32_head_sizes(tv, d):
    check(tv, R.cache_case([70, 1], [33, 400], Hq=4, Hkv=2, d=d, bs=8, dtype=torch.float32, seed=d))


@pytest.mark.parametrize("heads", [(1, 1), (24, 1), (28, 4), (128, 1), (160, 1)])
def test_attention_query_heads_per_kv_head(tv, heads):
    """Including more query heads per kv head than a row tile of 128 holds."""
    c = R.cache_case([5, 1, 40], [30, 260, 0], Hq=heads[0], Hkv=heads[1], d=64, bs=16,
                     dtype=torch.bfloat16, seed=heads[0])
    check(tv, c)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_large_scores(tv, dtype):
    """Scores of some hundreds: the running maximum is raised again and again."""
    c = R.cache_case([150, 2], [300, 900], Hq=8, Hkv=2, d=64, bs=16, dtype=dtype, seed=3)
    c["k_cache"] *= torch.linspace(0.1, 6.0, c["k_cache"].shape[0])[:, None, None, None].to(dtype)
    check(tv, c, scale=1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_strided_rows_and_rows_of_no_sequence(tv, dtype):
    c = R.cache_case([20, 3], [40, 5], Hq=4, Hkv=2, d=64, bs=16, dtype=dtype, seed=8)
    T = 23
    wide = torch.full((T + 9, 4 + 3, 64), float("nan"), dtype=dtype)   # q inside a fused row, more rows
    wide[2:T + 2, 2:6] = c["q"]
    q = wide.cuda()[:, 2:6]
    out = torch.full((T + 9, 6, 64), 5.0, dtype=dtype, device="cuda")[:, 1:5]
    ref, A, S = R.attention(c)
    tol = R.attention_tolerance(c, ref, A, S, 64)
    c["q_start"] = c["q_start"] + 2
    got, status = attend(tv, c, q=q, out=out)
    assert status.eq(0).all()
    assert ((got[2:T + 2].double() - ref).abs() <= tol).all()
    assert got[:2].eq(5.0).all() and got[T + 2:].eq(5.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_values_outside_a_rows_keys(tv, dtype, bad):
    """Rows of the cache past the last token, freed blocks before the window, and later
    tokens of the same chunk hold NaN or infinity: only rows that attend to them show it."""
    n, P, window, bs = [90, 1], [200, 333], 64, 16
    first = [max(0, (p - window + 1)) // bs for p in P]
    c = R.cache_case(n, P, Hq=4, Hkv=2, d=64, bs=bs, dtype=dtype, seed=5, first_block=first)
    used = torch.zeros(c["k_cache"].shape[0], bs, dtype=torch.bool)
    for b in range(2):
        for t in range(max(0, P[b] - window + 1), P[b] + n[b]):
            used[c["table"][b, t // bs].long(), t % bs] = True
    for name in ("k_cache", "v_cache"):
        c[name].permute(0, 2, 1, 3)[~used] = bad
    check(tv, c, window=window)
    # a later token of the chunk, and the oldest key of the first tokens' windows
    spot = [(0, 200 + 40), (0, 200 - window + 1 + 3)]
    for b, t in spot:
        c["v_cache"][c["table"][b, t // bs].long(), :, t % bs, 7] = bad
    out, status = attend(tv, c, window=window)
    assert status.eq(0).all()
    ref, A, S = R.attention(c, window=window)
    clean = torch.isfinite(ref)
    assert torch.equal(clean, torch.isfinite(out.double()))
    # column 7 of the rows that see one of the two keys, and nothing else
    assert int((~clean).sum()) == 4 * (50 + 4)
    tol = R.attention_tolerance(c, ref, A, S, 64)
    assert ((out.double() - ref).abs()[clean] <= tol[clean]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_masked_keys_not_finite(tv, dtype):
    """Keys (not values) of later tokens hold NaN."""
    c = R.cache_case([70], [50], Hq=4, Hkv=1, d=64, bs=16, dtype=dtype, seed=6)
    t = 50 + 30
    c["k_cache"][c["table"][0, t // 16].long(), :, t % 16] = float("nan")
    out, _ = attend(tv, c)
    ref, A, S = R.attention(c)
    tol = R.attention_tolerance(c, ref, A, S, 64)
    assert ((out[:30].double() - ref[:30]).abs() <= tol[:30]).all()
    assert out[30:].isnan().all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_bad_sequences(tv, dtype):
    n, P = [40, 3, 0, 65, 1, 2], [100, 20, 4, 9, 30, 8]
    c = R.cache_case(n, P, Hq=4, Hkv=2, d=64, bs=16, dtype=dtype, seed=9)
    ref, A, S = R.attention(c)
    tol = R.attention_tolerance(c, ref, A, S, 64)
    c["table"][0, 3] = c["k_cache"].shape[0]     # block past the cache
    c["prefix"][1] = -1                          # negative length
    c["prefix"][3] = c["table"].shape[1] * 16    # past the block table
    c["table"][4, 0] = -1                        # missing block
    out, status = attend(tv, c)
    assert status.tolist() == [3, 3, 0, 3, 3, 0]
    at = c["q_start"].tolist()
    for b in range(6):
        rows = slice(at[b], at[b + 1])
        if status[b]:
            assert out[rows].eq(0).all(), b
        else:
            assert ((out[rows].double() - ref[rows]).abs() <= tol[rows]).all(), b
    # blocks outside what is needed may hold anything
    c = R.cache_case([5], [100], Hq=4, Hkv=2, d=64, bs=16, dtype=dtype, seed=9)
    c["table"] = torch.cat([c["table"], torch.full((1, 3), 1 << 30, dtype=torch.int32)], 1)
    check(tv, c)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("starts", [[0, 5, 4, 9], [-1, 5, 6, 9], [0, 5, 6, 10], [3, 2, 6, 9]])
def test_attention_bad_row_ranges(tv, dtype, starts):
    c = R.cache_case([5, 1, 3], [10, 20, 30], Hq=4, Hkv=2, d=64, bs=16, dtype=dtype, seed=1)
    c["q_start"] = torch.tensor(starts, dtype=torch.int32)
    out, status = attend(tv, c)
    assert status.eq(3).all() and out.eq(7.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_is_the_same_twice_and_in_a_graph(tv, dtype):
    c = R.cache_case([200, 1, 33], [700, 1500, 0], Hq=8, Hkv=2, d=64, bs=16, dtype=dtype, seed=4)
    first, _ = attend(tv, c)
    again, _ = attend(tv, c)
    assert torch.equal(first, again)
    g = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    out = torch.zeros_like(g["q"])
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(16, tv.chunk_attention_workspace(234, 3, 8, 2, 64, dtype)), dtype=torch.uint8, device="cuda")
    args = (g["q"], g["k_cache"], g["v_cache"], g["table"], g["q_start"], g["prefix"], out, status, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tv.chunk_attention(*args, stream=torch.cuda.current_stream())
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), first)
    # other lengths in the same buffers: the schedule is made on the device
    c["n"], c["P"] = [1, 200, 33], [1200, 600, 0]
    c["q_start"] = torch.tensor([0, 1, 201, 234], dtype=torch.int32)
    c["prefix"] = torch.tensor(c["P"], dtype=torch.int32)
    tab = torch.full_like(c["table"], -1)
    need = [-(-(a + b) // 16) for a, b in zip(c["n"], c["P"])]
    order = torch.randperm(c["k_cache"].shape[0], generator=torch.Generator().manual_seed(1)).to(torch.int32)
    assert sum(need) <= len(order) and max(need) <= tab.shape[1]
    k = 0
    for b, m in enumerate(need):
        tab[b, :m] = order[k:k + m]
        k += m
    c["table"] = tab
    for name in ("table", "q_start", "prefix"):
        g[name].copy_(c[name])
    graph.replay()
    torch.cuda.synchronize()
    ref, A, S = R.attention(c)
    tol = R.attention_tolerance(c, ref, A, S, 64)
    assert ((out.cpu().double() - ref).abs() <= tol).all()


def test_attention_on_another_stream(tv):
    c = R.cache_case([100], [300], Hq=8, Hkv=2, d=128, bs=16, dtype=torch.bfloat16, seed=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check(tv, c)
    g = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    out, status = torch.zeros_like(g["q"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(16, tv.chunk_attention_workspace(100, 1, 8, 2, 128)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    tv.chunk_attention(g["q"], g["k_cache"], g["v_cache"], g["table"], g["q_start"], g["prefix"],
                       out, status, ws, stream=s)
    s.synchronize()
    ref, A, S = R.attention(c)
    assert ((out.cpu().double() - ref).abs() <= R.attention_tolerance(c, ref, A, S, 128)).all()


def test_attention_many_sequences(tv):
    """More sequences than threads of a CTA, most of them short."""
    rng = np.random.default_rng(0)
    n = [int(x) for x in rng.integers(0, 4, 700)]
    P = [int(x) for x in rng.integers(0, 90, 700)]
    check(tv, R.cache_case(n, P, Hq=2, Hkv=1, d=64, bs=16, dtype=torch.bfloat16, seed=10))


@pytest.mark.parametrize("heads,d", [((2, 2), 32), ((4, 1), 64), ((6, 2), 96), ((8, 1), 128), ((5, 5), 128),
                                     ((4, 2), 160), ((4, 1), 256), ((8, 1), 256), ((9, 1), 64)])
@pytest.mark.parametrize("window,cap", [(0, 0.0), (1, 0.0), (100, 5.0)])
def test_decoding_f32(tv, heads, d, window, cap):
    """About one token per sequence: none, one and several; keys from one on, in one part or many."""
    n = [1, 0, 1, 1, 3, 1, 1, 0, 2, 1]
    P = [0, 5, 1, 15, 16, 255, 256, 0, 1000, 5000]
    check(tv, R.cache_case(n, P, Hq=heads[0], Hkv=heads[1], d=d, bs=16, dtype=torch.float32, seed=d),
          window=window, softcap=cap)


@pytest.mark.parametrize("B", [1, 2, 40, 300])
def test_decoding_f32_batches(tv, B):
    rng = np.random.default_rng(B)
    P = [int(x) for x in rng.integers(0, 3000 if B < 300 else 200, B)]
    check(tv, R.cache_case([1] * B, P, Hq=8, Hkv=2, d=64, bs=8, dtype=torch.float32, seed=B))


def test_decoding_f32_bad_sequences(tv):
    """A bad block, a prefix past the table, rows of no sequence; keys with NaN beyond the last."""
    c = R.cache_case([1, 1, 1, 1], [40, 600, 3, 70], Hq=4, Hkv=2, d=64, bs=16, dtype=torch.float32, seed=1)
    ref, A, S = R.attention(c)
    tol = R.attention_tolerance(c, ref, A, S, 64)
    for b in range(4):
        blk, row = int(c["table"][b][(c["P"][b] + 1) // 16]), (c["P"][b] + 1) % 16
        if row:
            c["k_cache"][blk, :, row:], c["v_cache"][blk, :, row:] = float("nan"), float("inf")
    c["table"][1, 20] = c["k_cache"].shape[0]
    c["prefix"][3] = 16 * c["table"].shape[1]
    c["q"] = torch.cat([c["q"][:1], c["q"], c["q"][:2]])
    c["q_start"] = c["q_start"] + 1
    out, status = attend(tv, c)
    assert status.tolist() == [0, 3, 0, 3]
    for b in (0, 2):
        assert ((out[b + 1].double() - ref[b]).abs() <= tol[b]).all()
    assert out[[2, 4]].eq(0).all() and out[[0, 5, 6]].eq(7.0).all()
    c["q_start"] = torch.tensor([0, 2, 1, 3, 4], dtype=torch.int32)
    out, status = attend(tv, c)
    assert status.eq(3).all() and out.eq(7.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_blocks_past_32_bits(tv, dtype):
    """Blocks at both ends of caches of more than 2^31 elements: appended and attended."""
    Hq, Hkv, d, bs = 8, 4, 128, 32
    c = append_case([70, 1], [40, 200], Hq=Hq, Hkv=Hkv, d=d, bs=bs, dtype=dtype, seed=12)
    used = c["k_cache"].shape[0]
    blocks = 2 ** 31 // (Hkv * bs * d) + 100
    far = [b if b % 2 else blocks - 1 - b for b in range(used)]
    idx = torch.tensor(far, device="cuda")
    big = [torch.empty((blocks, Hkv, bs, d), dtype=dtype, device="cuda") for _ in range(2)]
    assert big[0].numel() > 2 ** 31
    for t, n in zip(big, ("k_cache", "v_cache")):
        t[idx] = c[n].cuda()
    small = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    table = small["table"]
    moved = torch.where(table >= 0, idx.to(torch.int32)[table.clamp(min=0).long()], table)
    rope, outs = tv.rope_table(128), []
    for k_cache, v_cache, tab in ((small["k_cache"], small["v_cache"], table), (*big, moved)):
        qkv = small["qkv"].clone()
        q, out = qkv[:, :Hq], torch.zeros((71, Hq, d), dtype=dtype, device="cuda")
        st = torch.full((2, 2), -9, dtype=torch.int32, device="cuda")
        ws = torch.zeros(max(16, tv.chunk_attention_workspace(71, 2, Hq, Hkv, d, dtype)), dtype=torch.uint8, device="cuda")
        tv.chunk_kv_append(q, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], k_cache, v_cache, tab,
                           small["q_start"], small["prefix"], st[0], rope=rope)
        tv.chunk_attention(q, k_cache, v_cache, tab, small["q_start"], small["prefix"], out, st[1], ws)
        torch.cuda.synchronize()
        assert st.eq(0).all()
        outs.append(out)
    assert torch.equal(outs[0], outs[1])
    for t, n in zip(big, ("k_cache", "v_cache")):
        assert torch.equal(t[idx], small[n])


def test_attention_refusals(tv):
    c = R.cache_case([5], [10], Hq=4, Hkv=2, d=64, bs=16, dtype=torch.bfloat16)
    g = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    out, st = torch.zeros_like(g["q"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    call = lambda **k: tv.chunk_attention(  # noqa: E731
        *[k.get(n, v) for n, v in (("q", g["q"]), ("kc", g["k_cache"]), ("vc", g["v_cache"]),
                                   ("table", g["table"]), ("q_start", g["q_start"]),
                                   ("prefix", g["prefix"]), ("out", out), ("st", st), ("ws", ws))])
    with pytest.raises(TypeError):
        call(q=g["q"].float())
    with pytest.raises(ValueError):
        call(q=g["q"].transpose(0, 1))
    with pytest.raises(ValueError):
        call(q_start=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        call(vc=g["v_cache"][:2])
    with pytest.raises(ValueError):
        call(table=g["table"].cpu())
    with pytest.raises(tv.TreeVerifyError):      # block size 8: no bfloat16 kernel
        call(kc=torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16, device="cuda"),
             vc=torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(tv.TreeVerifyError):
        call(q=g["q"][:, :3], out=out[:, :3])    # 3 query heads, 2 kv heads
    if tv.chunk_attention_workspace(5, 1, 4, 2, 64):
        with pytest.raises(tv.TreeVerifyError):
            call(ws=ws[:16])


# ------------------------------------------------------------------ append

ROPES = [None, dict(dim=64, theta=10000.0), dict(dim=32, theta=500000.0, interleaved=True),
         dict(dim=64, theta=1e6, scaling="linear", factor=4.0),
         dict(dim=32, theta=500000.0, scaling="bands", factor=8.0, original_len=8192, low=1.0, high=4.0),
         dict(dim=64, theta=10000.0, interleaved=True, scaling="ramp", factor=16.0, original_len=4096,
              low=1.0, high=32.0)]


def append_case(n, P, *, Hq, Hkv, d, bs, dtype, seed):
    c = R.cache_case(n, P, Hq=Hq, Hkv=Hkv, d=d, bs=bs, dtype=dtype, seed=seed)
    g = torch.Generator().manual_seed(seed + 100)
    c["qkv"] = torch.randn((sum(n), Hq + 2 * Hkv, d), generator=g).to(dtype)
    return c


def run_append(tv, c, Hq, Hkv, rope, positions=None, with_q=True):
    g = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    qkv = g["qkv"]
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    q_out = torch.full((qkv.shape[0], Hq, qkv.shape[2]), 7.0, dtype=qkv.dtype, device="cuda")
    status = torch.full((len(c["n"]),), -9, dtype=torch.int32, device="cuda")
    tv.chunk_kv_append(q if with_q else None, k, v, g["k_cache"], g["v_cache"], g["table"],
                       g["q_start"], g["prefix"], status, q_out=q_out if with_q else None,
                       rope=None if rope is None else tv.rope_table(**rope),
                       positions=None if positions is None else positions.cuda())
    torch.cuda.synchronize()
    return q_out.cpu(), g["k_cache"].cpu(), g["v_cache"].cpu(), status.cpu()


def expected_append(c, Hq, Hkv, rope, positions=None):
    """Rotated queries and the two caches (float64), and which slots were written."""
    T = c["qkv"].shape[0]
    seq = torch.repeat_interleave(torch.arange(len(c["n"])), torch.tensor(c["n"]))
    slot = c["prefix"].long()[seq] + torch.arange(T) - c["q_start"].long()[seq]
    pos = slot if positions is None else positions.long()
    q, k, v = (c["qkv"][:, a:b].double() for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    if rope is not None:
        f, amp = R.frequencies(rope["dim"], rope["theta"], rope.get("scaling", "none"),
                               rope.get("factor", 1.0), rope.get("original_len", 0), rope.get("low", 1.0),
                               rope.get("high", 4.0))
        q, k = (R.rotate(x, pos, f, amp, rope.get("interleaved", False)) for x in (q, k))
    kc, vc = c["k_cache"].double(), c["v_cache"].double()
    blk, row = c["table"][seq, slot // c["bs"]].long(), slot % c["bs"]
    kc[blk, :, row], vc[blk, :, row] = k, v
    return q, kc, vc


def rope_tolerance(x, d, dtype, far):
    """Rotation in float32 (u = 2^-24): the turns per position are rounded to 2^-53 of themselves,
    so the angle of position `far` is off by at most 2 pi far 2^-53 and by the float32 rounding of
    a fraction of a turn (pi u); sincospi is good to 2 u; two products, a sum, the
    amplitude: 4 u more, all relative to the pair's length, at most sqrt(2) max |x|.  The last
    rounding is half a step of the output type."""
    u = 2.0 ** -24
    pair = 1.5 * 1.5 * float(x.abs().max())
    step = 2.0 ** -8 if dtype == torch.bfloat16 else u
    return pair * (10 * u + 8 * far * 2.0 ** -53) + x.abs() * step * 1.01


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rope", range(len(ROPES)))
@pytest.mark.parametrize("shape", [(8, 2, 64, 16), (3, 1, 128, 8), (4, 4, 96, 48)])
def test_append(tv, dtype, rope, shape):
    Hq, Hkv, d, bs = shape
    n, P = [1, 0, 37, 16, 1, 5], [0, 3, 15, 100000, 31, 64]
    c = append_case(n, P, Hq=Hq, Hkv=Hkv, d=d, bs=bs, dtype=dtype, seed=rope)
    q_out, kc, vc, status = run_append(tv, c, Hq, Hkv, ROPES[rope])
    assert status.eq(0).all()
    q, k, v = expected_append(c, Hq, Hkv, ROPES[rope])
    assert torch.equal(vc.double(), v)
    if ROPES[rope] is None:
        assert torch.equal(q_out.double(), q) and torch.equal(kc.double(), k)
    assert ((q_out.double() - q).abs() <= rope_tolerance(q, d, dtype, 100000)).all()
    assert ((kc.double() - k).abs() <= rope_tolerance(k, d, dtype, 100000)).all()
    # slots of no new token, and columns that are not rotated, keep their bits
    keep = k == c["k_cache"].double()
    assert torch.equal(kc[keep], c["k_cache"][keep])


@pytest.mark.parametrize("T", [700, 5000, 33000])
def test_append_long_and_positions(tv, T):
    """More rows than a CTA, and (33000) than the limit from which a kernel checks first;
    positions of their own."""
    n, P = [T - 300, 300], [11, 4000]
    rope = dict(dim=64, theta=500000.0)
    c = append_case(n, P, Hq=4, Hkv=2, d=64, bs=16, dtype=torch.bfloat16, seed=T)
    pos = torch.randint(0, 1 << 30, (T,), generator=torch.Generator().manual_seed(0)).to(torch.int32)
    q_out, kc, vc, status = run_append(tv, c, 4, 2, rope, pos)
    assert status.eq(0).all()
    q, k, v = expected_append(c, 4, 2, rope, pos)
    assert torch.equal(vc.double(), v)
    # the reference's own angle in float64 is off by about pos * 2^-53 radians twice over
    assert ((q_out.double() - q).abs() <= rope_tolerance(q, 64, torch.bfloat16, 1 << 30)).all()
    assert ((kc.double() - k).abs() <= rope_tolerance(k, 64, torch.bfloat16, 1 << 30)).all()


@pytest.mark.parametrize("T", [60, 4000, 33000])
def test_append_bad_sequences_stay_untouched(tv, T):
    n, P = [20, T - 45, 0, 5, 10, 10], [3, 40, 1, 7, 12, 500]
    c = append_case(n, P, Hq=2, Hkv=1, d=64, bs=16, dtype=torch.bfloat16, seed=T)
    want = expected_append(c, 2, 1, None)
    c["table"][0, 1] = -1
    c["prefix"][3] = -5
    pos = torch.arange(T, dtype=torch.int32)
    pos[c["q_start"][4] + 9] = -1
    q_out, kc, vc, status = run_append(tv, c, 2, 1, None, pos)
    assert status.tolist() == [3, 0, 0, 3, 3, 0]
    at = c["q_start"].tolist()
    for b in (0, 3, 4):
        assert q_out[at[b]:at[b + 1]].eq(7.0).all()
    for b in (1, 5):
        assert torch.equal(q_out[at[b]:at[b + 1]].double(), want[0][at[b]:at[b + 1]])
        t = torch.arange(P[b], P[b] + n[b])
        blk, row = c["table"][b][t // 16].long(), t % 16
        assert torch.equal(kc[blk, :, row].double(), want[1][blk, :, row])
    changed = (kc != c["k_cache"]).any(-1).any(1).sum()
    assert int(changed) == n[1] + n[5]
    # a bad q_start: nothing is written
    for starts in ([0, 20, 10, T, T, T, T], [0] * 6 + [T + 1]):
        c["q_start"] = torch.tensor(starts, dtype=torch.int32)
        q_out, kc, vc, status = run_append(tv, c, 2, 1, None)
        assert status.eq(3).all() and q_out.eq(7.0).all()
        assert torch.equal(kc, c["k_cache"]) and torch.equal(vc, c["v_cache"])


def test_append_in_place_and_without_queries(tv):
    c = append_case([30], [2], Hq=4, Hkv=2, d=64, bs=16, dtype=torch.float32, seed=0)
    rope = dict(dim=64, theta=10000.0)
    want_q, want_k, _ = expected_append(c, 4, 2, rope)
    _, kc, _, status = run_append(tv, c, 4, 2, rope, with_q=False)
    assert status.eq(0).all()
    assert ((kc.double() - want_k).abs() <= rope_tolerance(want_k, 64, torch.float32, 100)).all()
    g = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    q = g["qkv"][:, :4]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tv.chunk_kv_append(q, g["qkv"][:, 4:6], g["qkv"][:, 6:], g["k_cache"], g["v_cache"], g["table"],
                       g["q_start"], g["prefix"], st, rope=tv.rope_table(**rope))
    assert ((q.cpu().double() - want_q).abs() <= rope_tolerance(want_q, 64, torch.float32, 100)).all()
    assert torch.equal(g["qkv"][:, 4:].cpu(), c["qkv"][:, 4:])


def test_append_matches_tree_append(tv):
    """A tree's keys through chunk_kv_append with positions P + depth: the rows that
    tree_kv_append writes, to one unit in the last place."""
    B, N, Hkv, d, bs = 3, 7, 2, 128, 16
    par = torch.tensor([[-1, 0, 0, 1, 1, 2, 2]] * B, dtype=torch.int32).cuda()
    mask = torch.zeros((B, N), dtype=torch.int64, device="cuda")
    depth = torch.zeros((B, N), dtype=torch.int32, device="cuda")
    st = torch.zeros(B, dtype=torch.int32, device="cuda")
    tv.tree_mask_build(par, mask, depth, st)
    c = append_case([N] * B, [100, 5, 33], Hq=2, Hkv=Hkv, d=d, bs=bs, dtype=torch.bfloat16, seed=1)
    pos = (c["prefix"][:, None] + depth.cpu()).reshape(-1).to(torch.int32)
    _, kc, vc, status = run_append(tv, c, 2, Hkv, dict(dim=d, theta=10000.0), pos)
    assert status.eq(0).all()
    g = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    k, v = (g["qkv"][:, a:a + Hkv].reshape(B, N, Hkv, d).contiguous() for a in (2, 2 + Hkv))
    tv.tree_kv_append(k, v, depth, g["k_cache"], g["v_cache"], g["table"], g["prefix"], st, rope_theta=10000.0)
    assert torch.equal(vc, g["v_cache"].cpu())
    a, b = kc.float(), g["k_cache"].cpu().float()
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-6).all()


def test_append_refusals(tv):
    c = append_case([4], [2], Hq=4, Hkv=2, d=64, bs=16, dtype=torch.bfloat16, seed=0)
    g = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, v = g["qkv"][:, :4], g["qkv"][:, 4:6], g["qkv"][:, 6:]
    tail = (g["k_cache"], g["v_cache"], g["table"], g["q_start"], g["prefix"], st)
    with pytest.raises(ValueError):
        tv.chunk_kv_append(None, k, v, *tail, q_out=q)
    with pytest.raises(TypeError):
        tv.chunk_kv_append(q, k, v.float(), *tail)
    with pytest.raises(TypeError):
        tv.chunk_kv_append(q, k, v, *tail, rope=dict(dim=64))
    with pytest.raises(ValueError):
        tv.chunk_kv_append(q, k, v, *tail, positions=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(tv.TreeVerifyError):      # more rotated columns than the head has
        tv.chunk_kv_append(q, k, v, *tail, rope=tv.rope_table(128))
    with pytest.raises(tv.TreeVerifyError):      # 24 columns: half a rotation is no 16-byte vector
        tv.chunk_kv_append(q, k, v, *tail, rope=tv.rope_table(24))
    with pytest.raises(ValueError):              # expanded rows: 0 apart
        tv.chunk_kv_append(q, k[:1].expand(4, 2, 64), v[:, :1], *tail)
    with pytest.raises(tv.TreeVerifyError):
        tv.chunk_kv_append(q, k[:1].expand(4, 2, 64), v, *tail)

"""Attention over an 8-bit cache on the GPU against its definition in 64 bits.  What the codes stand
for is exact in bfloat16, so the bounds are those of chunk_attention."""
import pytest
import torch

import chunk_ref as R
import q8_ref as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import eagle_speculative_decoding_parent_gb300 as m
    return m


def attend(tv, c, *, out=None, q=None, mask=None, **kw):
    """Runs chunk_attention_q8 on a case of q8_ref (CPU tensors); (out, status)."""
    g = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    q = g["q"] if q is None else q
    T, Hq, d = q.shape
    B = len(c["n"])
    out = torch.full_like(g["q"], 7.0) if out is None else out
    status = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    ws = torch.full((max(16, tv.chunk_attention_q8_workspace(T, B, Hq, c["k_cache"].shape[1], d)),),
                    0xFF, dtype=torch.uint8, device="cuda")
    tv.chunk_attention_q8(q, g["k_cache"], g["v_cache"], g["k_scale"], g["v_scale"], g["table"],
                          g["q_start"], g["prefix"], out, status, ws,
                          mask=None if mask is None else mask.cuda(), **kw)
    torch.cuda.synchronize()
    return out.cpu(), status.cpu()


def check(tv, c, **kw):
    out, status = attend(tv, c, **kw)
    assert status.eq(0).all(), status
    ref, A, S = Q.attention(c, **kw)
    tol = R.attention_tolerance(c, ref, A, S, c["q"].shape[2])
    err = (out.double() - ref).abs()
    assert torch.isfinite(out.double()).all()
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max()))


LENGTHS = [
    ([1], [0]),
    ([1], [300]),
    ([1, 1, 1, 1, 1], [0, 15, 127, 128, 1000]),
    ([0, 3, 0, 17, 1, 0], [5, 0, 0, 250, 129, 7]),
    ([64, 65, 31], [0, 63, 512]),
    ([257], [1]),
    ([200, 1, 333], [77, 2049, 0]),
    ([6] * 40, [(b * 37) % 700 for b in range(40)]),
]


@pytest.mark.parametrize("heads,d,bs", [((8, 2), 128, 16), ((7, 1), 64, 32), ((4, 4), 128, 48)])
@pytest.mark.parametrize("case", range(len(LENGTHS)))
def test_lengths(tv, heads, d, bs, case):
    n, P = LENGTHS[case]
    check(tv, Q.cache_case(n, P, Hq=heads[0], Hkv=heads[1], d=d, bs=bs, seed=case))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 64), (17, 4), (128, 16), (200, 33), (700, 5),
                                          (4000, 64), (0, 9)])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_window_sinks_and_cap(tv, window, sinks, cap):
    n, P = [1, 140, 0, 33, 300, 1], [700, 0, 9, 513, 260, 30]
    for heads, d, bs in (((8, 2), 128, 16), ((6, 2), 64, 48), ((2, 2), 64, 16)):
        c = Q.cache_case(n, P, Hq=heads[0], Hkv=heads[1], d=d, bs=bs, seed=window)
        check(tv, c, window=window, sinks=sinks, softcap=cap)


@pytest.mark.parametrize("heads,d,bs", [((8, 2), 128, 16), ((16, 1), 64, 32), ((3, 3), 128, 16), ((64, 1), 128, 16)])
@pytest.mark.parametrize("n,P", [([26] * 9, [b * 61 for b in range(9)]), ([1, 64, 0, 33, 60, 2], [0, 0, 4, 700, 127, 128]),
                                 ([7], [2048])])
def test_trees(tv, heads, d, bs, n, P):
    c = Q.cache_case(n, P, Hq=heads[0], Hkv=heads[1], d=d, bs=bs, seed=len(n))
    check(tv, c, mask=Q.trees(n, 3))
    # any bits: those above a row's own node do not count, a row may see nothing of the tree
    g = torch.Generator().manual_seed(1)
    any_bits = torch.randint(-(1 << 63), (1 << 63) - 1, (sum(n),), generator=g) & \
        torch.randint(-(1 << 63), (1 << 63) - 1, (sum(n),), generator=g)
    any_bits[::5] = 0
    check(tv, c, mask=any_bits, softcap=25.0)


@pytest.mark.parametrize("heads", [(1, 1), (24, 1), (28, 4), (128, 1)])
def test_query_heads_per_kv_head(tv, heads):
    check(tv, Q.cache_case([5, 1, 40], [30, 260, 0], Hq=heads[0], Hkv=heads[1], d=64, bs=16, seed=heads[0]))

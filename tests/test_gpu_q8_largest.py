"""The largest numbers in an 8-bit cache: a scale of 2^120 and codes up to 256, which stand for 2^128, no
bfloat16.  They reach the rows that attend to them and no others.  (Weights are up to 2^8 before they are
divided by their sum, so that 2^8 times such a value is beyond float32, in which the sums are: rows that attend
to them may be infinite or, of both signs, NaN, and are not looked at.  Few rows per sequence are summed in
codes, and are.)"""
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


def plant(c, which, n, P, bs):
    """In each sequence's last block, and one that some windows hold: (the case, what rows see of it)."""
    codes, scale = c[which + "_cache"].view(torch.uint8), c[which + "_scale"]
    at = {}
    for b in range(3):
        for t in (P[b] + n[b] - 1, P[b] - 18):
            blk = int(c["table"][b, t // bs])
            scale[blk] = 2.0 ** 120
            big = (codes[blk] & 0x7F) > 0x70                     # the block's others: up to 128
            codes[blk] = torch.where(big, (codes[blk] & 0x80) | 0x70, codes[blk])
            codes[blk, :, t % bs, 7] = 0x78 if t % 2 else 0xF8
            at.setdefault(b, set()).add(t // bs)
    return at


@pytest.mark.parametrize("n", [[1, 3, 2], [40, 64, 9]])
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 32), (64, 16)])
def test_values_of_256(tv, n, d, bs):
    P = [150, 37, 260]
    looked = 0
    for kw in (dict(), dict(window=20), dict(window=33, sinks=5), dict(mask=Q.trees(n, 5))):
        c = Q.cache_case(n, P, Hq=8, Hkv=2, d=d, bs=bs, seed=n[0] + d)
        at = plant(c, "v", n, P, bs)
        out, status = attend(tv, c, **kw)
        assert status.eq(0).all()
        ref, A, S = Q.attention(c, **kw)
        tol = R.attention_tolerance(c, ref, A, S, d)
        start = c["q_start"].tolist()
        for b in range(3):
            seen = Q.seen_keys(c, b, kw.get("window", 0), kw.get("sinks", 0), kw.get("mask"))
            far = torch.zeros(n[b], dtype=torch.bool)
            for lb in at[b]:
                far |= seen[:, lb * bs:(lb + 1) * bs].any(1)
            rows = start[b] + (torch.arange(n[b]) if max(n) < 4 else (~far).nonzero().view(-1))
            looked += rows.numel()
            # results beyond the largest bfloat16, 2^128 (1 - 2^-8), within what is allowed may be infinite
            got, want, most = out[rows].double(), ref[rows], tol[rows]
            over = torch.isinf(got) & (want.abs() + most >= 2.0 ** 128 * (1 - 2.0 ** -8))
            assert bool(((got - want).abs() <= most)[~over].all())
    assert looked >= 6


@pytest.mark.parametrize("n", [[1, 3, 2], [40, 64, 9]])
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 32), (64, 16)])
def test_keys_of_256(tv, n, d, bs):
    """A key's 2^128 against a query's zero is nothing.  (Queries small enough for float32 products.)"""
    P = [150, 37, 260]
    for kw in (dict(), dict(window=20), dict(window=33, sinks=5), dict(mask=Q.trees(n, 5))):
        c = Q.cache_case(n, P, Hq=8, Hkv=2, d=d, bs=bs, seed=n[0] + d)
        plant(c, "k", n, P, bs)
        c["q"] *= 2.0 ** -8
        c["q"][..., 7] = 0.0
        out, status = attend(tv, c, scale=2.0 ** -118, **kw)
        assert status.eq(0).all()
        ref, A, S = Q.attention(c, scale=2.0 ** -118, **kw)
        assert bool(((out.double() - ref).abs() <= R.attention_tolerance(c, ref, A, S, d)).all())

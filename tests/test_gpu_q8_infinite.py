"""Query rows with infinities over an 8-bit cache with capped scores, which the cap makes finite: plus or minus
the cap, or NaN where an infinity meets a zero or another of the other sign."""
import pytest
import torch

import chunk_ref as R
import q8_ref as Q
from test_gpu_q8 import attend

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import eagle_speculative_decoding_parent_gb300 as m
    return m


@pytest.mark.parametrize("n", [[1, 3, 2], [40, 64, 9], [300, 5, 40]])
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 32), (128, 48)])
def test_infinite_queries_under_a_cap(tv, n, d, bs):
    P, cap = [150, 37, 260], 20.0
    for kw in (dict(), dict(window=33), dict(window=33, sinks=5), dict(mask=True)):
        if kw.get("mask"):
            if max(n) > 64:
                continue
            kw["mask"] = Q.trees(n, 5)
        c = Q.cache_case(n, P, Hq=8, Hkv=2, d=d, bs=bs, seed=n[0] + d)
        codes = c["k_cache"].view(torch.uint8)
        codes[(codes & 0x7F) == 0] = 0x01                        # (zeros are placed below)
        T = sum(n)
        odd = torch.zeros((T, 8), dtype=torch.bool)
        q = c["q"]
        for r, h, put in [(0, 0, {3: INF}), (0, 5, {d - 1: -INF}), (1, 7, {0: INF, 1: INF}), (2, 1, {40: INF, 63: -INF}),
                          (3, 2, {17: INF}), (T - 1, 3, {d // 2: -INF}), (T - 1, 6, {5: INF}), (T // 2, 4, {c: INF for c in range(d)}),
                          (T - 2, 0, {8: INF, 9: float("nan")})]:
            for col, x in put.items():
                q[r, h, col] = x
            odd[r, h] = True
        # a zero in the column of row 3's infinity, at a key of the last sequence's prefix, and of the last
        # row's, at the last key
        at = lambda b, t: (int(c["table"][b, t // bs]), slice(None), t % bs)  # noqa: E731
        codes[at(2, P[2] - 20)][:, 17] = 0x80
        codes[at(2, P[2] + n[2] - 1)][:, 5] = 0x00
        # and a NaN among the keys, that some rows see
        codes[at(1, P[1] + 1)][0, 9] = 0x7F
        out, status = attend(tv, c, softcap=cap, **kw)
        assert status.eq(0).all()
        ref, A, _ = Q.attention(c, softcap=cap, **kw)
        # (an infinite score is the cap itself: as far off as one of its size at most)
        fine = torch.where(torch.isfinite(q), q, 0.0)
        _, _, S = Q.attention(dict(c, q=fine), softcap=cap, **kw)
        S = torch.where(odd | ~torch.isfinite(S), cap, S)
        tol = R.attention_tolerance(c, ref, A, S, d)
        nan = ref.isnan()
        assert bool((~nan.any(-1))[odd].any()) and bool(nan.any(-1)[odd].any())
        assert torch.equal(out.isnan(), nan)
        assert bool(((out.double() - ref).abs() <= tol)[~nan].all())

"""Waits that run out in chunk_attention.  The test-only variable TV_TEST_WAITS_RUN_OUT = "w" or
"w@c" makes the first wait for work or data of warp w (of CTA c alone) count as run out: nothing
hangs, copies and products in flight are still waited for, and the status has to say that the rows
are not right."""
import pytest
import torch

import chunk_ref as R
from test_gpu_chunk import attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import eagle_speculative_decoding_parent_gb300 as m
    return m


def matches(c, out, status, keep, **kw):
    """Rows of the sequences `keep` are right and their status is TV_OK."""
    ref, A, S = R.attention(c, **kw)
    tol = R.attention_tolerance(c, ref, A, S, c["q"].shape[2])
    at = c["q_start"].tolist()
    for b in keep:
        rows = slice(at[b], at[b + 1])
        assert status[b] == 0 and ((out[rows].double() - ref[rows]).abs() <= tol[rows]).all(), b


CASES = [dict(n=[1], P=[300], Hq=8, Hkv=2, d=128),
         dict(n=[0, 200, 1, 0, 33, 300], P=[5, 700, 1500, 3, 0, 90], Hq=8, Hkv=2, d=64),
         dict(n=[1 + b % 3 for b in range(400)], P=[b % 80 for b in range(400)], Hq=2, Hkv=1, d=128)]


# warps 0 - 7: softmax; 8: products; 9: K/V copies; 10: Q tiles; 11: scheduler
@pytest.mark.parametrize("warp", [0, 6, 8, 9, 10, 11])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_every_cta_of_the_bfloat16_kernel(tv, monkeypatch, warp, case):
    c = R.cache_case(bs=16, dtype=torch.bfloat16, seed=warp, **CASES[case])
    kw = dict(softcap=30.0) if case == 1 else {}
    monkeypatch.setenv("TV_TEST_WAITS_RUN_OUT", str(warp))
    _, status = attend(tv, c, **kw)
    assert status.tolist() == [6 if n else 0 for n in c["n"]]
    monkeypatch.delenv("TV_TEST_WAITS_RUN_OUT")
    out, status = attend(tv, c, **kw)
    matches(c, out, status, range(len(c["n"])), **kw)


@pytest.mark.parametrize("warp", [3, 8, 9, 10, 11])
@pytest.mark.parametrize("cta", [0, 7, 100])
def test_one_cta_of_the_bfloat16_kernel(tv, monkeypatch, warp, cta):
    """Only the sequences with work on that CTA are affected, and none of them says TV_OK."""
    c = R.cache_case([1, 120, 40] * 20, [900, 50, 333] * 20, Hq=8, Hkv=4, d=64, bs=16,
                     dtype=torch.bfloat16, seed=cta)
    monkeypatch.setenv("TV_TEST_WAITS_RUN_OUT", f"{warp}@{cta}")
    out, status = attend(tv, c)
    late = (status == 6).nonzero().view(-1).tolist()
    assert late == list(range(late[0], late[-1] + 1)) and len(late) < 10
    matches(c, out, status, [b for b in range(60) if b not in late])


@pytest.mark.parametrize("n,P", [([1, 1, 0, 1], [40, 900, 7, 3000]), ([70, 0, 300, 1], [33, 2, 500, 1200])])
def test_float32_kernels(tv, monkeypatch, n, P):
    c = R.cache_case(n, P, Hq=4, Hkv=2, d=64, bs=16, dtype=torch.float32, seed=1)
    monkeypatch.setenv("TV_TEST_WAITS_RUN_OUT", "0")
    _, status = attend(tv, c)
    assert status.tolist() == [6 if k else 0 for k in n]
    monkeypatch.delenv("TV_TEST_WAITS_RUN_OUT")
    out, status = attend(tv, c)
    matches(c, out, status, range(4))

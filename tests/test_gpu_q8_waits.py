"""Waits that run out in chunk_attention_q8: TV_TEST_WAITS_RUN_OUT, as in test_gpu_waits.py."""
import pytest
import torch

import q8_ref as Q
from test_gpu_q8 import attend
from test_gpu_q8_edges import matches

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import eagle_speculative_decoding_parent_gb300 as m
    return m


FEW = [dict(n=[1], P=[300]), dict(n=[0, 2, 1, 0, 3, 1], P=[5, 700, 1500, 3, 0, 90])]
MORE = [dict(n=[40], P=[300]), dict(n=[0, 200, 1, 0, 33, 300], P=[5, 700, 1500, 3, 0, 90])]


# warps 0 - 7: softmax; 8: products; 9: copies; 10: Q tiles; 11: scheduler; 12 - 15: widening
@pytest.mark.parametrize("warp", [0, 6, 8, 9, 10, 11, 12, 15])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("case", range(len(MORE)))
def test_every_cta(tv, monkeypatch, warp, case, d):
    for which in (MORE, FEW) if warp == 0 else (MORE,):        # (few rows per sequence: any warp stands for all)
        c = Q.cache_case(bs=16, Hq=8, Hkv=2, d=d, seed=warp, **which[case])
        kw = dict(softcap=30.0) if case == 1 else {}
        monkeypatch.setenv("TV_TEST_WAITS_RUN_OUT", str(warp))
        _, status = attend(tv, c, **kw)
        assert status.tolist() == [6 if n else 0 for n in c["n"]]
        monkeypatch.delenv("TV_TEST_WAITS_RUN_OUT")
        out, status = attend(tv, c, **kw)
        matches(c, out, status, **kw)


@pytest.mark.parametrize("warp", [3, 8, 9, 10, 11, 13])
@pytest.mark.parametrize("cta", [0, 7, 100])
def test_one_cta(tv, monkeypatch, warp, cta):
    """Only the sequences with work on that CTA are affected, and none of them says TV_OK."""
    for n in ([30, 120, 40] * 20,) + (([1, 2, 1] * 20,) if warp == 3 else ()):
        c = Q.cache_case(n, [900, 50, 333] * 20, Hq=8, Hkv=4, d=128, bs=16, seed=cta)
        monkeypatch.setenv("TV_TEST_WAITS_RUN_OUT", f"{warp}@{cta}")
        out, status = attend(tv, c)
        monkeypatch.delenv("TV_TEST_WAITS_RUN_OUT")
        late = (status == 6).nonzero().view(-1).tolist()
        assert late == list(range(late[0], late[-1] + 1)) and len(late) < 10
        matches(c, out, status, [b for b in range(60) if b not in late])

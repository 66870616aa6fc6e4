"""chunk_attention where its arithmetic meets infinities."""
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


def put(c, name, b, t, column, x):
    c[name][c["table"][b, t // c["bs"]].long(), :, t % c["bs"], column] = x


# ------------------------------------------------------------------ infinite values

@pytest.mark.parametrize("heads,d", [((4, 2), 64), ((8, 1), 128), ((4, 1), 256)])
@pytest.mark.parametrize("window", [0, 77])
def test_decoding_f32_infinite_values(tv, heads, d, window):
    """A value of infinity among a token's keys makes that column infinite, wherever the key lies
    in the kernel's steps and parts: the last key, and 31 others spread over the row."""
    n, P = [1] * 6, [0, 5, 31, 200, 999, 3000]
    c = R.cache_case(n, P, Hq=heads[0], Hkv=heads[1], d=d, bs=16, dtype=torch.float32, seed=d + window)
    for b, p in enumerate(P):
        first = max(0, p - window + 1) if window else 0
        keys = p + 1 - first
        for j in range(32):                     # column j: the last key of the j-th 32nd
            put(c, "v_cache", b, first + max(1, keys * (j + 1) // 32) - 1, j, float("inf"))
    out, status = attend(tv, c, window=window)
    assert status.eq(0).all()
    assert out[:, :, :32].eq(float("inf")).all()
    c["v_cache"] = torch.where(c["v_cache"].isinf(), torch.zeros(()), c["v_cache"])
    ref, A, S = R.attention(c, window=window)
    tol = R.attention_tolerance(c, ref, A, S, d)
    assert ((out.double() - ref).abs() <= tol)[:, :, 32:].all()

"""chunk_attention at the edges: infinite values and scores, caps far above the scores, windows past
32 bits."""
import pytest
import torch

import chunk_ref as R
from test_gpu_chunk import attend, check

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


# ------------------------------------------------------------------ scores of -infinity

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,P,window", [([1], [0], 0), ([1], [2500], 0), ([1, 90, 1, 300], [40, 0, 0, 700], 1),
                                        ([200], [1000], 0), ([3, 70], [0, 300], 0)])
def test_rows_whose_every_score_is_minus_infinity(tv, dtype, n, P, window):
    """The softmax of such a row has no value: NaN, in every form of the kernels; rows that see
    some other key are as if the keys at -infinity were not there."""
    c = R.cache_case(n, P, Hq=4, Hkv=1, d=64, bs=16, dtype=dtype, seed=len(n) + n[0])
    c["q"][..., 0] = c["q"][..., 0].abs() + 0.1
    for b in range(len(n)):
        # every key up to that of the sequence's middle row
        for t in range(P[b] + n[b] // 2 + 1):
            put(c, "k_cache", b, t, 0, float("-inf"))
    out, status = attend(tv, c, window=window)
    assert status.eq(0).all()
    ref, A, _ = R.attention(c, window=window)
    assert torch.equal(out.isnan(), ref.isnan())
    seen = ~ref.isnan()
    assert seen.any() == any(a > 1 for a in n) and ref.isnan().any()
    k = dict(c, k_cache=torch.where(c["k_cache"].isinf(), torch.zeros((), dtype=dtype), c["k_cache"]))
    _, _, S = R.attention(k, window=window)     # (the keys at -infinity have weight 0, not a rounding)
    tol = R.attention_tolerance(c, ref, A, S, 64)
    assert ((out.double() - ref).abs() <= tol)[seen].all()


# ------------------------------------------------------------------ caps far above the scores

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cap", [30.0, 1e4, 2e6, 1e7, 1e8, 1e9])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_thousands_below_a_far_cap(tv, dtype, cap, d):
    """Scores of 2,400 to 2,404 and a cap of thousands of times that: a score keeps float32's
    precision, which a difference of numbers as large as the cap would not.  Few keys per row, so
    that errors do not average out.  The products are exact: one column gives 2,400, one the
    sixteenths behind it, the rest zero."""
    c = R.cache_case([1, 6, 9], [5, 0, 3], Hq=4, Hkv=2, d=d, bs=16, dtype=dtype, seed=d)
    g = torch.Generator().manual_seed(int(cap) % 1000)
    c["q"].zero_()
    c["q"][..., 0], c["q"][..., 9] = 32.0, 1.0
    c["k_cache"].zero_()
    c["k_cache"][..., 0] = 75.0
    c["k_cache"][..., 9] = (torch.randint(0, 64, c["k_cache"].shape[:3], generator=g) / 16).to(dtype)
    check(tv, c, scale=1.0, softcap=cap)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scores_of_zero_with_the_largest_scale_over_cap(tv, dtype):
    """scale / cap past float32's range: a score of 0 stays 0."""
    c = R.cache_case([40], [30], Hq=4, Hkv=2, d=64, bs=16, dtype=dtype, seed=1)
    c["q"][1::2] = 0.0
    c["q"][::2] = 1.0
    c["k_cache"][:] = 1.0
    check(tv, c, scale=1e12, softcap=1e-30)


# ------------------------------------------------------------------ windows past 32 bits

@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, -2 ** 32 + 5])
def test_windows_past_32_bits_are_none(tv, window):
    c = R.cache_case([40, 1], [30, 200], Hq=4, Hkv=2, d=64, bs=16, dtype=torch.bfloat16, seed=1)
    out, status = attend(tv, c, window=window)
    assert status.eq(0).all()
    assert torch.equal(out, attend(tv, c)[0])

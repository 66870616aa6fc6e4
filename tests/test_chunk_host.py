"""Host side of the operators on chunks and logits (CPU only): argument checks, which run
before anything touches a GPU, and rotary tables against their formulas."""
import ctypes
import math
import os
import shutil

import pytest

import chunk_ref as R

P, I, I64, F, D, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                       ctypes.c_size_t)
NZ = P(64)          # a non-null, 16-byte aligned pointer that nothing reads


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    bm = __graft_entry__._build_module()
    if not os.path.exists(bm.LIB) and not shutil.which("nvcc"):
        pytest.skip("library not built and nvcc unavailable")
    return ctypes.CDLL(bm.build())


class Table(ctypes.Structure):
    _fields_ = [("dim", I), ("interleaved", I), ("amplitude", F), ("reserved", I),
                ("turn", ctypes.c_uint64 * 128)]


def table(lib, dim, interleaved=0, theta=10000.0, scaling=0, factor=1.0, old=0.0, low=0.0, high=0.0, amp=0.0):
    t = Table()
    f = lib.rope_table_init
    f.argtypes = [P, I, I, D, I, D, D, D, D, D]
    return f(ctypes.addressof(t), dim, interleaved, theta, scaling, factor, old, low, high, amp), t


@pytest.mark.parametrize("scaling", ["none", "linear", "bands", "ramp"])
@pytest.mark.parametrize("dim,theta,factor,old", [(64, 10000.0, 4.0, 4096), (128, 500000.0, 8.0, 8192),
                                                  (2, 10000.0, 2.0, 100), (256, 1e6, 40.0, 32768)])
def test_rope_tables(lib, scaling, dim, theta, factor, old):
    low, high = 1.0, 32.0 if scaling == "ramp" else 4.0
    rc, t = table(lib, dim, 1, theta, ["none", "linear", "bands", "ramp"].index(scaling), factor, old)
    assert rc == 0 and t.dim == dim and t.interleaved == 1
    f, amp = R.frequencies(dim, theta, scaling, factor, old, low, high)
    assert abs(t.amplitude - amp) <= 2.0 ** -23 * amp
    for j in range(dim // 2):
        want = float(f[j]) / (2 * math.pi)
        # pow and the products in float64: within a few units in the last place of each other
        assert abs(t.turn[j] / 2.0 ** 64 - want) <= 16 * 2.0 ** -53 * want + 2.0 ** -64


def test_rope_table_refusals(lib):
    nan, inf = float("nan"), float("inf")
    assert table(lib, 64)[0] == 0
    for bad in (dict(dim=0), dict(dim=3), dict(dim=258), dict(dim=64, theta=1.0), dict(dim=64, theta=nan),
                dict(dim=64, scaling=4), dict(dim=64, scaling=1, factor=0.5), dict(dim=64, scaling=1, factor=inf),
                dict(dim=64, scaling=2, factor=2.0), dict(dim=64, scaling=3, factor=2.0, old=nan),
                dict(dim=64, scaling=3, factor=2.0, old=4096.0, low=8.0, high=4.0), dict(dim=64, amp=inf)):
        assert table(lib, **bad)[0] == 1, bad


def append(lib, *, T=4, B=1, Hq=8, Hkv=2, d=64, q=NZ, q_out=NZ, stride=None, rope=None, bs=16, blocks=9, mb=4,
           dt=1, q_start=NZ, k=NZ):
    f = lib.chunk_kv_append
    f.argtypes = [P, I64, P, I64, P, I64, P, I, P, P, I, I, I, I, P, P, I64, P, P, P, I, I, I, I, P, P]
    s = (Hq + 2 * Hkv) * d if stride is None else stride
    return f(q, s, k, s, NZ, s, None, T, q_start, NZ, B, Hq, Hkv, d, None if rope is None else ctypes.addressof(rope),
             q_out, s, NZ, NZ, NZ, mb, bs, blocks, dt, NZ, None)


def test_append_host_checks(lib):
    assert append(lib, B=0) == 0                        # empty batch: nothing to do
    assert append(lib, dt=7) == 1
    for bad in (dict(T=-1), dict(B=-1), dict(Hkv=0), dict(d=0), dict(bs=0), dict(blocks=0), dict(mb=0)):
        assert append(lib, **bad) == 1, bad
    assert append(lib, q=None) == 1                     # an output without queries
    assert append(lib, q_out=None) == 1
    assert append(lib, q_start=None) == 1 and append(lib, k=None) == 1
    assert append(lib, stride=100) == 1                 # rows that overlap
    assert append(lib, q=P(8)) == 1                     # misaligned
    assert append(lib, d=12) == 4                       # 24-byte heads
    assert append(lib, stride=12 * 64 + 4) == 4         # rows off the 16-byte grid
    _, t = table(lib, 128)
    assert append(lib, rope=t) == 1                     # rotates more than the head
    _, t = table(lib, 24)
    assert append(lib, rope=t) == 4


def attend(lib, *, T=4, B=1, Hq=8, Hkv=2, d=64, stride=512, bs=16, blocks=9, mb=4, dt=1, cap=0.0, q=NZ,
           ws=NZ, ws_bytes=1 << 40):
    f = lib.chunk_attention
    f.argtypes = [P, I64, P, P, P, I, P, P, I, I, I, I, I, I, I, I, F, F, I, P, I64, P, P, SZ, P]
    return f(q, stride, NZ, NZ, NZ, mb, NZ, NZ, T, B, Hq, Hkv, d, bs, blocks, dt, 0.0, cap, 0, NZ, stride, NZ,
             ws, ws_bytes, None)


def test_attention_host_checks(lib):
    assert attend(lib, B=0) == 0
    for bad in (dict(dt=5), dict(T=-1), dict(B=-2), dict(Hq=7), dict(mb=0), dict(bs=0), dict(blocks=0),
                dict(cap=float("nan")), dict(cap=float("inf")), dict(q=None), dict(q=P(4)), dict(stride=500)):
        assert attend(lib, **bad) == 1, bad
    for bad in (dict(d=96), dict(bs=8), dict(stride=516), dict(dt=0, d=48), dict(dt=0, d=288)):
        assert attend(lib, **bad) == 4, bad
    ws = lib.chunk_attention_workspace
    ws.restype, ws.argtypes = SZ, [I] * 6
    assert ws(0, 1, 8, 2, 64, 1) == 0 and ws(4, 1, 7, 2, 64, 1) == 0
    need = ws(4, 1, 8, 2, 64, 0)
    if need:
        assert attend(lib, dt=0, ws=None) == 8 and attend(lib, dt=0, ws_bytes=need - 1) == 8


def test_counts_host_checks(lib):
    f = lib.token_counts_update
    f.argtypes = [P, P, P, I, I, I, I, I, P, P]
    call = lambda total=6, B=2, V=10, counts=NZ, tokens=NZ, starts=None: f(  # noqa: E731
        counts, tokens, starts, total, B, V, 0, 0, NZ, None)
    assert call(B=0) == 0
    assert call(B=-1) == 1 and call(V=0) == 1 and call(V=(1 << 24) + 1) == 1 and call(total=-1) == 1
    assert call(total=5) == 1                           # rows of unequal length without starts
    assert call(counts=None) == 1 and call(tokens=None) == 1


def test_logits_host_checks(lib):
    f = lib.tree_logits_process
    f.argtypes = [P, I, I, I, I] + [P] * 10 + [I, P, P, P]
    call = lambda B=2, N=4, V=10, dt=0, logits=NZ, mask=None, tokens=None, counts=None, rep=None: f(  # noqa: E731
        logits, dt, B, N, V, None, mask, tokens, counts, None, None, rep, None, None, None, 1, NZ, NZ, None)
    assert call(B=0) == 0
    assert call(B=-1) == 1 and call(N=0) == 1 and call(N=65) == 1 and call(V=0) == 1 and call(dt=3) == 1
    assert call(logits=None) == 1
    assert call(mask=NZ) == 1 and call(tokens=NZ) == 1  # one without the other
    assert call(rep=NZ) == 1                            # a penalty without a history

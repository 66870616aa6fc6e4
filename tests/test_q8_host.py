"""Host side of the operators on 8-bit caches and of sampling (CPU only): the argument checks, which
run before anything touches a GPU, and the binding's."""
import ctypes

import pytest
import torch

from test_chunk_host import I, I64, F, NZ, P, SZ, lib, table  # noqa: F401


def append(lib, *, T=4, B=1, Hq=8, Hkv=2, d=64, q=NZ, q_out=NZ, stride=None, rope=None, bs=16, blocks=9, mb=4,  # noqa: F811
           q_start=NZ, k=NZ, kc=NZ, ks=NZ, vs=NZ, status=NZ):
    f = lib.chunk_kv_append_q8
    f.argtypes = [P, I64, P, I64, P, I64, P, I, P, P, I, I, I, I, P, P, I64, P, P, P, P, P, I, I, I, P, P]
    s = (Hq + 2 * Hkv) * d if stride is None else stride
    return f(q, s, k, s, NZ, s, None, T, q_start, NZ, B, Hq, Hkv, d, None if rope is None else ctypes.addressof(rope),
             q_out, s, kc, NZ, ks, vs, NZ, mb, bs, blocks, status, None)


def test_append(lib):  # noqa: F811
    assert append(lib, B=0) == 0
    for bad in (dict(T=-1), dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(d=0), dict(bs=0), dict(blocks=0), dict(mb=0),
                dict(q=None), dict(q_out=None), dict(q_start=None), dict(k=None), dict(kc=None), dict(ks=None), dict(vs=None),
                dict(status=None), dict(stride=100), dict(q=P(8)), dict(kc=P(72))):
        assert append(lib, **bad) == 1, bad
    for bad in (dict(d=96), dict(d=256), dict(bs=8), dict(bs=24), dict(stride=12 * 64 + 4), dict(Hq=1 << 25, d=64)):
        assert append(lib, **bad) == 4, bad
    _, t = table(lib, 128)
    assert append(lib, rope=t) == 1                     # rotates more than the head
    _, t = table(lib, 24)
    assert append(lib, rope=t) == 4


def attend(lib, *, T=4, B=1, Hq=8, Hkv=2, d=64, stride=512, bs=16, blocks=9, mb=4, cap=0.0, window=0, sinks=0, mask=None,  # noqa: F811
           q=NZ, kc=NZ, ks=NZ, vs=NZ, out=NZ, status=NZ, ws=NZ, ws_bytes=1 << 40):
    f = lib.chunk_attention_q8
    f.argtypes = [P, I64, P, P, P, P, P, I, P, P, P, I, I, I, I, I, I, I, F, F, I, I, P, I64, P, P, SZ, P]
    return f(q, stride, kc, NZ, ks, vs, NZ, mb, NZ, NZ, mask, T, B, Hq, Hkv, d, bs, blocks, 0.0, cap, window, sinks,
             out, stride, status, ws, ws_bytes, None)


def test_attention(lib):  # noqa: F811
    assert attend(lib, B=0) == 0
    for bad in (dict(T=-1), dict(B=-2), dict(Hq=7), dict(Hq=0), dict(Hkv=0), dict(mb=0), dict(bs=0), dict(blocks=0),
                dict(cap=float("nan")), dict(cap=float("inf")), dict(q=None), dict(q=P(4)), dict(out=P(24)), dict(kc=P(8)),
                dict(stride=500), dict(ks=None), dict(vs=None), dict(kc=None), dict(out=None), dict(status=None),
                dict(sinks=-1), dict(sinks=65), dict(mask=NZ, window=5)):
        assert attend(lib, **bad) == 1, bad
    for bad in (dict(d=96), dict(d=32), dict(bs=8), dict(bs=20), dict(stride=516), dict(Hq=129, Hkv=1, stride=129 * 64)):
        assert attend(lib, **bad) == 4, bad
    # without a GPU its size is not known, and no workspace is needed before there is one
    ws = lib.chunk_attention_q8_workspace
    ws.restype, ws.argtypes = SZ, [I] * 5
    for none in ((0, 1, 8, 2, 64), (4, 0, 8, 2, 64), (4, 1, 7, 2, 64), (4, 1, 8, 2, 96), (4, 1, 0, 0, 64)):
        assert ws(*none) == 0, none
    for T, B in ((4, 1), (1000, 1)):
        need = ws(T, B, 8, 2, 64)
        if need:
            assert attend(lib, T=T, B=B, ws=None) == 8 and attend(lib, T=T, B=B, ws_bytes=need - 1) == 8
            assert attend(lib, T=T, B=B, ws=P(72)) == 8


def compact(lib, *, layers=1, stride=None, sstride=None, mb=4, most=3, B=1, Hkv=2, d=64, bs=16, blocks=9, kc=NZ, ks=NZ, vs=NZ,  # noqa: F811
            path=NZ, accept=NZ, new=NZ, status=NZ):
    f = lib.kv_compact_q8
    f.argtypes = [P, P, P, P, I, I64, I64, P, I, P, P, P, I, I, I, I, I, I, P, P, P, P, P]
    return f(kc, NZ, ks, vs, layers, blocks * Hkv * bs * d if stride is None else stride,
             blocks * Hkv if sstride is None else sstride, NZ, mb, NZ, path, accept, most, B, Hkv, d, bs, blocks, new, None,
             None, status, None)


def test_compact(lib):  # noqa: F811
    assert compact(lib, B=0) == 0 and compact(lib, layers=0) == 0
    for bad in (dict(B=-1), dict(Hkv=0), dict(d=0), dict(bs=0), dict(blocks=0), dict(mb=0), dict(most=0), dict(layers=-1),
                dict(stride=-16), dict(sstride=-1), dict(layers=2, stride=16), dict(layers=2, sstride=1), dict(kc=None),
                dict(ks=None), dict(vs=None), dict(path=None), dict(accept=None), dict(new=None), dict(status=None),
                dict(kc=P(8)), dict(layers=2, stride=9 * 2 * 16 * 64 + 8)):
        assert compact(lib, **bad) == 1, bad
    for bad in (dict(d=96), dict(bs=8), dict(bs=40)):
        assert compact(lib, **bad) == 4, bad


def test_sample(lib):  # noqa: F811
    f = lib.logits_sample
    f.argtypes = [P, I, I, I, I] + [P] * 9 + [P]
    call = lambda dt=0, B=1, N=1, V=10, logits=NZ, uniform=NZ, tokens=NZ, probs=None, status=NZ: f(  # noqa: E731
        logits, dt, B, N, V, None, uniform, None, None, None, None, tokens, probs, status, None)
    assert call(B=0) == 0
    for bad in (dict(dt=2), dict(dt=-1), dict(B=-1), dict(N=0), dict(N=65), dict(V=0), dict(V=(1 << 24) + 1), dict(logits=None),
                dict(uniform=None), dict(tokens=None), dict(status=None), dict(probs=NZ)):
        assert call(**bad) == 1, bad


# ------------------------------------------------------------------ the binding

@pytest.fixture()
def tv(lib, monkeypatch):  # noqa: F811
    import eagle_speculative_decoding_parent_gb300 as m
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return m


def test_binding(tv):
    """Shapes, types and devices are looked at before the call is made."""
    bf = dict(dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    q, k = torch.zeros((4, 8, 64), **bf), torch.zeros((4, 2, 64), **bf)
    c, s = torch.zeros((9, 2, 16, 64)).to(torch.float8_e4m3fn), torch.ones((9, 2))
    t, qs, st = torch.zeros((1, 4), **i32), torch.tensor([0, 4], **i32), torch.zeros(1, **i32)
    wrong = (TypeError, ValueError)
    for bad in (dict(k=k[0]), dict(k=k.float()), dict(q=q[:3]), dict(q=None, q_out=q), dict(kc=c.float()), dict(ks=s[:8]),
                dict(ks=s.double()), dict(t=t.long()), dict(qs=qs[:1]), dict()):
        a = dict(dict(q=q, k=k, kc=c, ks=s, t=t, qs=qs, q_out=None), **bad)
        with pytest.raises(wrong):                      # (the last: tensors on the CPU)
            tv.chunk_kv_append_q8(a["q"], a["k"], k, a["kc"], c, a["ks"], s, a["t"], a["qs"], st, st, q_out=a["q_out"])
    for bad in (dict(q=q[0]), dict(q=q.float()), dict(kc=c[0]), dict(sinks=65), dict(sinks=-1), dict(mask=t), dict()):
        a = dict(dict(q=q, kc=c, sinks=0, mask=None), **bad)
        with pytest.raises(wrong):
            tv.chunk_attention_q8(a["q"], a["kc"], c, s, s, t, qs, st, q, st, None, sinks=a["sinks"], mask=a["mask"])
    for bad in (dict(kc=c[0]), dict(path=st), dict(t=t[0]), dict()):
        a = dict(dict(kc=c, path=t, t=t), **bad)
        with pytest.raises(wrong):
            tv.kv_compact_q8(a["kc"], c, s, s, a["t"], st, a["path"], st, st, st)
    x, u = torch.zeros((2, 1, 10)), torch.zeros((2, 1))
    tok = torch.zeros((2, 1), **i32)
    for bad in (dict(x=x[0]), dict(x=x.double()), dict(u=u[0]), dict(tok=tok.long()), dict()):
        a = dict(dict(x=x, u=u, tok=tok), **bad)
        with pytest.raises(wrong):
            tv.logits_sample(a["x"], a["u"], a["tok"], tok)

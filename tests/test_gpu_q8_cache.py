"""Appending to an 8-bit cache, and moving accepted rows in it, on the GPU against their definitions."""
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


def new_rows(c, Hkv, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    T, _, d = c["q"].shape
    f = lambda: (torch.randn((T, Hkv, d), generator=g) * spread).bfloat16()  # noqa: E731
    return f(), f()


def append(tv, c, k, v, *, q=None, rope=None, positions=None, q_out=None, status=None):
    """Runs chunk_kv_append_q8; (caches and scales after it on the CPU, q_out, status)."""
    g = {x: y.cuda() for x, y in c.items() if isinstance(y, torch.Tensor)}
    status = torch.full((len(c["n"]),), -9, dtype=torch.int32, device="cuda")
    tv.chunk_kv_append_q8(None if q is None else q, k.cuda() if not k.is_cuda else k, v.cuda() if not v.is_cuda else v,
                          g["k_cache"], g["v_cache"], g["k_scale"], g["v_scale"], g["table"],
                          g["q_start"], g["prefix"], status, q_out=q_out, rope=rope,
                          positions=None if positions is None else positions.cuda())
    torch.cuda.synchronize()
    return {x: g[x].cpu() for x in ("k_cache", "v_cache", "k_scale", "v_scale")}, status.cpu()


# An angle is a fraction of a turn rounded to float32 (at most 2^-25 half turns, 9.4e-8 radians), cos
# and sin are off by two units in the last place (1.2e-7), times the amplitude, two products and a
# sum are rounded (2^-24 each): at most 2^-21 of |x| + |y| times the amplitude.
ROTATED = 2.0 ** -21


def check_codes(got, want, exact, err, scale):
    """Codes [blocks, H, bs, d] are those of numbers within err of the exact ones."""
    differ = got != want
    assert differ.float().mean() < 1e-3
    a, b = (x.view(Q.E4M3).double() * scale[..., None, None] for x in (got, want))
    step = torch.exp2(torch.floor(torch.log2((exact / scale[..., None, None]).abs().clamp_min(2.0 ** -6))) - 3) * scale[..., None, None]
    # where the exact number lies within err of the border between two codes
    ok = ((a - exact).abs() <= step / 2 + err) & ((a - b).abs() <= step * 1.01)
    assert bool(ok[differ].all())


SEQS = [([1], [0]), ([1, 1, 1], [15, 16, 31]), ([0, 3, 0, 17, 1, 0], [5, 0, 0, 250, 129, 7]),
        ([26] * 5, [512, 7, 100, 33, 64]), ([200, 1, 333], [77, 2049, 0]), ([5] * 40, list(range(40)))]


@pytest.mark.parametrize("heads,d,bs", [((8, 2), 128, 16), ((7, 1), 64, 32), ((4, 4), 128, 48), ((6, 3), 64, 128)])
@pytest.mark.parametrize("case", range(len(SEQS)))
@pytest.mark.parametrize("rope", ["none", "half", "interleaved", "part"])
def test_append(tv, heads, d, bs, case, rope):
    n, P = SEQS[case]
    c = Q.cache_case(n, P, Hq=heads[0], Hkv=heads[1], d=d, bs=bs, seed=case)
    k, v = new_rows(c, heads[1], case, spread=[1.0, 40.0, 0.01][case % 3])
    pos = torch.cat([torch.arange(b, a + b) for a, b in zip(n, P)])
    table, exact = None, k.double()
    q_exact, err = c["q"].double(), torch.zeros_like(exact)
    if rope != "none":
        m = 48 if rope == "part" else d
        table = tv.rope_table(m, theta=500000.0, interleaved=rope == "interleaved", scaling="ramp", factor=4.0,
                              original_len=8192)
        f, amp = R.frequencies(m, 500000.0, "ramp", 4.0, 8192, 1.0, 32.0)
        exact, q_exact = (R.rotate(x, pos, f, amp, rope == "interleaved") for x in (k, c["q"]))
        i = (slice(0, m, 2), slice(1, m, 2)) if rope == "interleaved" else (slice(0, m // 2), slice(m // 2, m))
        s = (k[..., i[0]].abs() + k[..., i[1]].abs()).double() * amp * ROTATED
        err[..., i[0]], err[..., i[1]] = s, s
    q = c["q"].cuda()
    q_out = torch.full_like(q, 9.0)
    got, status = append(tv, c, k, v, q=q, rope=table, q_out=q_out)
    assert status.eq(0).all()
    for x, rows, e in (("k", exact, err), ("v", v.double(), torch.zeros_like(exact))):
        code, scale = Q.append(c, x, rows)
        assert torch.equal(got[x + "_scale"].double(), scale)
        have = got[x + "_cache"].view(torch.uint8)
        if x == "v":
            assert torch.equal(have, code)
        else:
            numbers = code.view(Q.E4M3).double() * scale[..., None, None]
            wide = torch.zeros_like(numbers)
            for b in range(len(n)):
                for i in range(n[b]):
                    at, r = int(c["table"][b, (P[b] + i) // bs]), (P[b] + i) % bs
                    numbers[at, :, r] = rows[int(c["q_start"][b]) + i]
                    wide[at, :, r] = e[int(c["q_start"][b]) + i]
            check_codes(have, code, numbers, wide, scale)
    # queries: one rounding to bfloat16 behind the float32 rotation
    w = R.rotate(c["q"].abs(), pos * 0, torch.zeros(1, dtype=torch.float64), 1.0, False)
    bound = q_exact.abs() * 2.0 ** -8 * 1.01 + 4 * ROTATED * float(w.amax())
    assert bool(((q_out.cpu().double() - q_exact).abs() <= bound).all())


def test_append_moves_earlier_codes_to_a_larger_scale(tv):
    """Blocks whose scale grows by 2^1 .. 2^12: exact above the subnormal codes, rounded below; and
    blocks whose scale is larger than the new rows need keep it."""
    for j, (d, bs) in enumerate([(128, 16), (64, 48)]):
        c = Q.cache_case([3] * 6, [b * 17 + 5 for b in range(6)], Hq=2, Hkv=2, d=d, bs=bs, seed=j, scales=(-12, 3))
        for x in ("k", "v"):                                     # every code there is
            codes = torch.arange(c[x + "_cache"].numel(), dtype=torch.int64) % 256
            c[x + "_cache"] = codes.to(torch.uint8).view(c[x + "_cache"].shape).view(Q.E4M3)
        k, v = new_rows(c, 2, 5, spread=30.0)
        got, status = append(tv, c, k, v)
        assert status.eq(0).all()
        for x, rows in (("k", k), ("v", v)):
            code, scale = Q.append(c, x, rows.double())
            assert torch.equal(got[x + "_scale"].double(), scale)
            have, nan = got[x + "_cache"].view(torch.uint8), (code & 0x7F) == 0x7F
            assert torch.equal(have[~nan], code[~nan]) and bool(((have[nan] & 0x7F) == 0x7F).all())


def test_append_odd_values(tv):
    """Zeros, the largest and smallest numbers, infinities and NaN (neither counts for the scale)."""
    c = Q.cache_case([16, 16, 16, 16, 2], [0, 16, 32, 0, 7], Hq=2, Hkv=1, d=64, bs=16, seed=2)
    T = 66
    k, v = torch.zeros((T, 1, 64)).bfloat16(), torch.zeros((T, 1, 64)).bfloat16()
    k[16:32] = 3.3e38
    k[32:48] = 1e-38
    k[48:64] = torch.linspace(-5, 5, 1024).view(16, 1, 64)
    k[50, 0, 3], k[51, 0, 9], k[52, 0, 1] = float("inf"), float("-inf"), float("nan")
    v[20, 0, 5], v[64, 0, 2] = float("nan"), 448.0
    v[0:16] = 449.0
    got, status = append(tv, c, k, v)
    assert status.eq(0).all()
    for x, rows in (("k", k), ("v", v)):
        code, scale = Q.append(c, x, rows.double())
        assert torch.equal(got[x + "_scale"].double(), scale)
        have, nan = got[x + "_cache"].view(torch.uint8), (code & 0x7F) == 0x7F
        assert torch.equal(have[~nan] & 0x7F, code[~nan] & 0x7F) and bool(((have[nan] & 0x7F) == 0x7F).all())
        zero = (code & 0x7F) == 0
        assert torch.equal(have[~nan & ~zero], code[~nan & ~zero])


def test_append_step_by_step(tv):
    """A prompt in chunks and then single tokens: blocks fill step by step and stay what they stand
    for, within a rounding of each growth."""
    n = [37, 3, 1, 1, 60, 1, 16, 1]
    c = Q.cache_case([sum(n)], [0], Hq=2, Hkv=2, d=128, bs=16, seed=4)
    k, v = new_rows(c, 2, 9)
    k *= torch.linspace(0.1, 8.0, sum(n))[:, None, None].bfloat16()
    at = 0
    full = {x: c[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale")}
    for m in n:
        step = dict(c, **full, n=[m], P=[at], q=c["q"][:m], q_start=torch.tensor([0, m], dtype=torch.int32),
                    prefix=torch.tensor([at], dtype=torch.int32))
        want = {x: Q.append(step, x, y[at:at + m].double()) for x, y in (("k", k), ("v", v))}
        full, status = append(tv, step, k[at:at + m], v[at:at + m])
        assert status.eq(0).all()
        for x in ("k", "v"):
            assert torch.equal(full[x + "_cache"].view(torch.uint8), want[x][0])
            assert torch.equal(full[x + "_scale"].double(), want[x][1])
        at += m


def test_append_refuses_and_leaves_alone(tv):
    n, P = [5, 4, 6, 3, 2, 0], [10, 20, 0, 3, 40, -1]
    c = Q.cache_case(n, [max(0, p) for p in P], Hq=2, Hkv=2, d=64, bs=16, seed=6)
    c["P"], c["prefix"] = P, torch.tensor(P, dtype=torch.int32)
    c["table"][1, 1] = 10 ** 6
    c["prefix"][3] = -2
    c["prefix"][4] = c["table"].shape[1] * 16 - 1
    k, v = new_rows(c, 2, 1)
    pos = torch.arange(sum(n), dtype=torch.int32)
    pos[10] = -1                                                 # of the third sequence
    q = torch.full((sum(n), 2, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    q_out = torch.full_like(q, 9.0)
    got, status = append(tv, c, k, v, q=q, q_out=q_out, positions=pos)
    assert status.tolist() == [0, 3, 3, 3, 3, 3]
    only = dict(c, n=[5, 0, 0, 0, 0, 0])
    for x, rows in (("k", k), ("v", v)):
        code, scale = Q.append(only, x, rows.double())
        assert torch.equal(got[x + "_cache"].view(torch.uint8), code) and torch.equal(got[x + "_scale"].double(), scale)
    assert bool((q_out[:5] == 2.0).all()) and bool((q_out[5:] == 9.0).all())
    # a bad q_start: nothing is written
    bad = dict(c, q_start=torch.tensor([0, 5, 4, 15, 18, 20, 20], dtype=torch.int32))
    got, status = append(tv, bad, k, v, positions=pos)
    assert status.eq(3).all()
    for x in ("k_cache", "v_cache", "k_scale", "v_scale"):
        assert torch.equal(got[x].view(torch.uint8), c[x].view(torch.uint8))


def test_append_views_of_one_projection_and_rows_of_no_sequence(tv):
    c = Q.cache_case([20, 3], [40, 5], Hq=4, Hkv=2, d=64, bs=16, seed=8)
    T = 23
    wide = torch.randn((T + 9, 8, 64), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    q, k, v = wide[:, :4], wide[:, 4:6], wide[:, 6:]
    before = wide.clone()
    shifted = dict(c, q_start=c["q_start"] + 2)
    table = tv.rope_table(64)
    got, status = append(tv, shifted, k, v, q=q, rope=table)     # queries in place
    assert status.eq(0).all()
    f, amp = R.frequencies(64, 10000.0, "none", 1.0, 0, 0, 0)
    pos = torch.cat([torch.arange(40, 60), torch.arange(5, 8)])
    code, scale = Q.append(c, "v", before[2:T + 2, 6:].double().cpu())
    assert torch.equal(got["v_cache"].view(torch.uint8), code) and torch.equal(got["v_scale"].double(), scale)
    want = R.rotate(before[2:T + 2, :4].cpu(), pos, f, amp, False)
    assert bool(((wide[2:T + 2, :4].cpu().double() - want).abs() <= want.abs() * 2.0 ** -8 + 1e-5).all())
    assert torch.equal(wide[:2], before[:2]) and torch.equal(wide[T + 2:], before[T + 2:])
    assert torch.equal(wide[:, 4:], before[:, 4:])


def test_append_long(tv):
    """More rows than the CTAs check for themselves."""
    n, P = [33000, 5], [9, 100]
    c = Q.cache_case(n, P, Hq=1, Hkv=1, d=64, bs=16, seed=1)
    k, v = new_rows(c, 1, 2)
    got, status = append(tv, c, k, v)
    assert status.eq(0).all()
    for x, rows in (("k", k), ("v", v)):
        code, scale = Q.append(c, x, rows.double())
        assert torch.equal(got[x + "_cache"].view(torch.uint8), code) and torch.equal(got[x + "_scale"].double(), scale)
    c["table"][0, 2000] = -7
    got, status = append(tv, c, k, v)
    assert status.tolist() == [3, 0]
    assert torch.equal(got["k_cache"].view(torch.uint8)[c["table"][0, :1999].long()],
                       c["k_cache"].view(torch.uint8)[c["table"][0, :1999].long()])


# ------------------------------------------------------------------ moving accepted rows

def compact(tv, c, path, accept, **kw):
    g = {x: y.cuda() for x, y in c.items() if isinstance(y, torch.Tensor)}
    B, most = path.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    new, status = torch.full((B,), -9, **i32), torch.full((B,), -9, **i32)
    src, dst = (torch.full((B, most), -9, dtype=torch.int64, device="cuda") for _ in range(2))
    tv.kv_compact_q8(g["k_cache"], g["v_cache"], g["k_scale"], g["v_scale"], g["table"], g["prefix"],
                     path.cuda(), accept.cuda(), new, status, src_slots=src, dst_slots=dst)
    torch.cuda.synchronize()
    return {x: g[x].cpu() for x in ("k_cache", "v_cache", "k_scale", "v_scale")}, new.cpu(), status.cpu(), src.cpu(), dst.cpu()


@pytest.mark.parametrize("d,bs,Hkv", [(128, 16, 8), (64, 32, 1), (128, 48, 3)])
@pytest.mark.parametrize("N,most", [(26, 7), (60, 60), (64, 64), (6, 6)])
def test_compact(tv, d, bs, Hkv, N, most):
    g = torch.Generator().manual_seed(N)
    P = [0, 5, 16, 100, 31, 513]
    c = Q.cache_case([N] * len(P), P, Hq=Hkv, Hkv=Hkv, d=d, bs=bs, seed=N, scales=(-11, -1))
    path, accept = torch.full((len(P), most), -1, dtype=torch.int32), torch.zeros(len(P), dtype=torch.int32)
    for b in range(len(P)):
        a = int(torch.randint(0, most, (1,), generator=g)) if b else most - 1
        accept[b] = a
        path[b, :a + 1] = torch.randperm(N, generator=g)[:a + 1].sort().values if b != 2 else torch.arange(a + 1)
        path[b, 0] = 0
    got, new, status, src, dst = compact(tv, c, path, accept)
    assert status.eq(0).all() and new.tolist() == [p + int(a) + 1 for p, a in zip(P, accept)]
    for x in ("k", "v"):
        code, scale = Q.compact(c, x, path, accept)
        assert torch.equal(got[x + "_scale"].double(), scale)
        have = got[x + "_cache"].view(torch.uint8)
        zero = (code & 0x7F) == 0
        assert torch.equal(have[~zero], code[~zero]) and bool(((have[zero] & 0x7F) == 0).all())
    for b in range(len(P)):
        for j in range(most):
            want = [-1, -1]
            if j <= accept[b]:
                want = [int(c["table"][b, (P[b] + t) // bs]) * bs + (P[b] + t) % bs for t in (int(path[b, j]), j)]
            assert [int(src[b, j]), int(dst[b, j])] == want


def test_compact_layers_and_the_same_node_twice(tv):
    c = Q.cache_case([12, 12], [3, 40], Hq=2, Hkv=2, d=64, bs=16, seed=5)
    layers = [Q.cache_case([12, 12], [3, 40], Hq=2, Hkv=2, d=64, bs=16, seed=5 + i, scales=(-8 + i, -1)) for i in range(3)]
    stack = dict(c)
    for x in ("k_cache", "v_cache", "k_scale", "v_scale"):
        stack[x] = torch.stack([l[x].view(torch.uint8) if "cache" in x else l[x] for l in layers])
        if "cache" in x:
            stack[x] = stack[x].view(Q.E4M3)
    path = torch.tensor([[0, 7, 7, 9], [0, 1, 1, -1]], dtype=torch.int32)
    accept = torch.tensor([3, 2], dtype=torch.int32)
    got, _, status, _, _ = compact(tv, stack, path, accept)
    assert status.eq(0).all()
    for i, l in enumerate(layers):
        for x in ("k", "v"):
            code, scale = Q.compact(dict(l, table=c["table"]), x, path, accept)
            have = got[x + "_cache"][i].view(torch.uint8)
            assert torch.equal(got[x + "_scale"][i].double(), scale)
            assert torch.equal(have.view(Q.E4M3).float(), code.view(Q.E4M3).float())


def test_compact_refuses_and_leaves_alone(tv):
    c = Q.cache_case([8] * 5, [3, 10, 20, 5, 9], Hq=2, Hkv=2, d=64, bs=16, seed=5)
    path = torch.tensor([[0, 2, 3, -1]] * 5, dtype=torch.int32)
    accept = torch.tensor([2, 4, 2, 2, -1], dtype=torch.int32)
    path[2, 1] = -1
    c["table"][3, 0] = 10 ** 6
    got, new, status, src, _ = compact(tv, c, path, accept)
    assert status.tolist() == [0, 3, 3, 3, 3] and new.tolist() == [6, 10, 20, 5, 9]
    assert bool((src[1:] == -1).all())
    only = dict(c, P=[3])
    for x in ("k", "v"):
        code, scale = Q.compact(only, x, path, accept)
        assert torch.equal(got[x + "_cache"].view(torch.uint8), code) and torch.equal(got[x + "_scale"].double(), scale)

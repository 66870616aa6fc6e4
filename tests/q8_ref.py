"""Plain definitions in 64 bits of the operators on 8-bit caches and of sampling, and seeded inputs
for them.  No code of the library is used."""
import math

import torch

import chunk_ref as R

E4M3 = torch.float8_e4m3fn
SMALL = -100                     # exponent of the smallest scale


def values(cache, scale):
    """What e4m3 codes [blocks, heads, bs, d] with their scales stand for, float64."""
    return cache.view(torch.uint8).view(E4M3).float().double() * scale.double()[..., None, None]


def to_code(y):
    """float64 to the nearest e4m3 code (ties to even), as uint8; infinities and NaN to 0x7f.  |y| has
    to be at most 448 otherwise."""
    a = y.abs()
    ok = torch.isfinite(y)
    assert bool((a[ok] <= 448).all())
    a = torch.where(ok, a, 0.0)
    e = torch.floor(torch.log2(a.clamp_min(2.0 ** -6)))
    m = torch.round(a / torch.exp2(e - 3))                       # 8 .. 16, below the normal ones 0 .. 8
    code = torch.where(a < 2.0 ** -6, m, (e + 6) * 8 + m).to(torch.uint8)
    code = torch.where(y.signbit(), code | 0x80, code)
    return torch.where(ok, code, torch.tensor(0x7F, dtype=torch.uint8))


def need(a):
    """The smallest 2^e >= 2^SMALL with a <= 448 2^e, for each of a (float64)."""
    p = torch.exp2(torch.arange(SMALL, 125, dtype=torch.float64))
    return p[(a[..., None] > 448.0 * p).sum(-1)]


def cache_case(n, P, *, Hq, Hkv, d, bs, seed=0, spare=3, first_block=None, scales=(-9, -4)):
    """chunk_ref.cache_case with an 8-bit cache: every code but NaN, mostly of normal numbers."""
    c = R.cache_case(n, P, Hq=Hq, Hkv=Hkv, d=d, bs=bs, dtype=torch.bfloat16, seed=seed, spare=spare,
                     first_block=first_block)
    g = torch.Generator().manual_seed(seed + 1000)
    for x in ("k", "v"):
        shape = c[x + "_cache"].shape
        c[x + "_cache"] = (torch.randn(shape, generator=g) * 90).clamp(-448, 448).to(E4M3)
        c[x + "_scale"] = torch.exp2(torch.randint(*scales, shape[:2], generator=g).float())
    return c


def trees(n, seed):
    """Ancestor bits of random trees of n[b] nodes, row by row: int64 [sum(n)]."""
    g = torch.Generator().manual_seed(seed)
    rows = []
    for a in n:
        for i in range(a):
            par = int(torch.randint(0, i, (1,), generator=g)) if i else 0
            rows.append((rows[len(rows) - i + par] if i else 0) | (1 << i))
    return torch.tensor([r - (1 << 64) if r >= 1 << 63 else r for r in rows], dtype=torch.int64)


def seen_keys(c, b, window, sinks, mask):
    """bool [n, P + n]: the keys that the rows of sequence b attend to."""
    n, P, lo = c["n"][b], c["P"][b], int(c["q_start"][b])
    t, at = torch.arange(P + n), torch.arange(P, P + n)[:, None]
    seen = t[None] <= at
    if window > 0:
        seen = seen & ((t[None] > at - window) | (t[None] < sinks))
    if mask is not None:
        for a in range(n):
            bit = (mask[lo:lo + n] >> a) & 1
            seen[:, P + a] &= bit.bool()
    return seen


def attention(c, *, scale=0.0, softcap=0.0, window=0, sinks=0, mask=None):
    """(out, A, S) as chunk_ref.attention; rows without a key are zero."""
    T, Hq, d = c["q"].shape
    Hkv, bs = c["k_cache"].shape[1], c["bs"]
    G = Hq // Hkv
    scale = scale if scale > 0 else 1.0 / math.sqrt(d)
    out = torch.zeros((T, Hq, d), dtype=torch.float64)
    A, S = torch.zeros_like(out), torch.zeros((T, Hq), dtype=torch.float64)
    k, v = (values(c[x + "_cache"], c[x + "_scale"]) for x in ("k", "v"))
    for b, n in enumerate(c["n"]):
        if n == 0:
            continue
        lo = int(c["q_start"][b])
        seen = seen_keys(c, b, window, sinks, mask)
        some = seen.any(0).nonzero().view(-1)                      # (other blocks may be gone)
        seen = seen[:, some]
        blk, row = c["table"][b][some // bs].long(), some % bs
        for g in range(Hkv):
            K, V = k[blk, g, row], v[blk, g, row]
            Q = c["q"][lo:lo + n, g * G:(g + 1) * G].double()
            s = torch.einsum("ihd,td->iht", Q, K) * scale
            if softcap > 0:
                s = softcap * torch.tanh(s / softcap)
            s = s.masked_fill(~seen[:, None], -math.inf)
            p = torch.softmax(s, -1)
            p = torch.where(seen.any(1)[:, None, None], p, 0.0)
            p = torch.where(seen[:, None], p, 0.0)
            odd = ~torch.isfinite(V).all(1)                        # values that reach only who sees them
            fine = torch.where(odd[:, None], 0.0, V)
            for to, X in ((out, fine), (A, fine.abs())):
                to[lo:lo + n, g * G:(g + 1) * G] = torch.einsum("iht,td->ihd", p, X)
            for t in odd.nonzero().view(-1).tolist():
                out[lo:lo + n, g * G:(g + 1) * G] += torch.where(seen[:, t, None, None], p[:, :, t, None] * V[t], 0.0)
            m = torch.einsum("ihd,td->iht", Q.abs(), K.abs()) * scale
            if some.numel():
                S[lo:lo + n, g * G:(g + 1) * G] = torch.where(seen[:, None], m, 0.0).amax(-1)
    return out, A, S


def append(c, name, rows):
    """The cache and scales [codes uint8, scales float64] after rows [T, heads, d] (float64: what is
    quantised) have been appended to case c; block by block."""
    code, scale = c[name + "_cache"].view(torch.uint8).clone(), c[name + "_scale"].double().clone()
    bs = c["bs"]
    for b, (n, P) in enumerate(zip(c["n"], c["P"])):
        for lb in range(P // bs, (P + n - 1) // bs + 1) if n else ():
            at = int(c["table"][b, lb])
            lo, hi = max(P, lb * bs), min(P + n, (lb + 1) * bs)
            x = rows[int(c["q_start"][b]) + lo - P:int(c["q_start"][b]) + hi - P].transpose(0, 1)   # [H, new, d]
            s = need(torch.where(torch.isfinite(x), x.abs(), 0.0).amax((1, 2)))
            r0, r1 = lo - lb * bs, hi - lb * bs
            if r0:
                s = torch.maximum(s, scale[at])
                was = code[at, :, :r0].view(E4M3).double()
                code[at, :, :r0] = to_code(was * (scale[at] / s)[:, None, None])
            code[at, :, r0:r1] = to_code(x / s[:, None, None])
            scale[at] = s
    return code, scale


def compact(c, name, path, accept):
    """[codes uint8, scales float64] after the accepted paths have been moved."""
    code, scale = c[name + "_cache"].view(torch.uint8).clone(), c[name + "_scale"].double().clone()
    was, had, bs = code.clone(), scale.clone(), c["bs"]
    for b, P in enumerate(c["P"]):
        A, block = int(accept[b]), c["table"][b].tolist()
        for lb in range(P // bs, (P + A) // bs + 1):
            js = [j for j in range(A + 1) if (P + j) // bs == lb]
            to, keep = block[lb], max(0, P - lb * bs)
            s = torch.stack([had[block[(P + int(path[b, j])) // bs]] for j in js]).amax(0)
            if keep:
                s = torch.maximum(s, had[to])
                code[to, :, :keep] = to_code(was[to, :, :keep].view(E4M3).double() * (had[to] / s)[:, None, None])
            for j in js:
                src = P + int(path[b, j])
                x = was[block[src // bs], :, src % bs].view(E4M3).double() * had[block[src // bs]][:, None]
                code[to, :, (P + j) % bs] = to_code(x / s[:, None])
            scale[to] = s
    return code, scale


def sample_sets(x, temp, k, top_p, min_p):
    """(weights, kept, near): exact weights of a row x (1-D), what the filters keep, and the entries
    whose keeping hangs on a sum within 2^-30 of a border."""
    x = x.double()
    V = x.numel()
    w = torch.zeros(V, dtype=torch.float64)
    near = torch.zeros(V, dtype=torch.bool)
    order = torch.argsort(x, descending=True, stable=True)
    if temp == 0:
        w[order[0]] = 1.0
        return w, w > 0, near
    w = torch.exp((x - x.max()) / temp)
    kept = torch.zeros(V, dtype=torch.bool)
    first = order[:k] if 0 < k < V else order
    ww = w[first]
    before = torch.cumsum(ww, 0) - ww
    goal = top_p * float(ww.sum())
    take = (before < goal) | (top_p >= 1.0)
    take[0] = True
    if top_p < 1.0:
        near[first[(before - goal).abs() <= 2.0 ** -30 * float(ww.sum())]] = True
    kept[first[take]] = True
    near |= (w - min_p).abs() <= 2.0 ** -36
    return w, kept & (w >= min_p), near

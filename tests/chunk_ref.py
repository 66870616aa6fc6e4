"""Plain definitions in 64 bits of the operators on chunks of new tokens and on a tree's
logits, and seeded inputs for them.  No code of the library is used."""
import math

import torch


def cache_case(n, P, *, Hq, Hkv, d, bs, dtype, seed=0, spare=3, first_block=None):
    """A paged cache with shuffled blocks for sequences of n new tokens after P cached ones.
    first_block: per sequence, the first block that exists (earlier table entries are -1)."""
    g = torch.Generator().manual_seed(seed)
    need = [max(1, -(-(a + b) // bs)) for a, b in zip(n, P)]
    first = [0] * len(n) if first_block is None else first_block
    total = sum(need) + spare
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(n), max(need)), -1, dtype=torch.int32)
    k = 0
    for b, m in enumerate(need):
        for j in range(first[b], m):
            table[b, j] = order[k]
            k += 1
    T = sum(n)
    start = [0]
    for a in n:
        start.append(start[-1] + a)
    f = lambda *s: torch.randn(s, generator=g).to(dtype)  # noqa: E731
    return dict(n=list(n), P=list(P), bs=bs, table=table, q_start=torch.tensor(start, dtype=torch.int32),
                prefix=torch.tensor(P, dtype=torch.int32), q=f(T, Hq, d),
                k_cache=f(total, Hkv, bs, d), v_cache=f(total, Hkv, bs, d))


def attention(c, *, scale=0.0, softcap=0.0, window=0):
    """(out, A, S) in float64: the outputs, sum_t p_t |v_t| per output, and the largest
    scale * sum_j |q_j k_j| over visible keys of each (row, head)."""
    T, Hq, d = c["q"].shape
    Hkv, bs = c["k_cache"].shape[1], c["bs"]
    G = Hq // Hkv
    scale = scale if scale > 0 else 1.0 / math.sqrt(d)
    out = torch.zeros((T, Hq, d), dtype=torch.float64)
    A, S = torch.zeros_like(out), torch.zeros((T, Hq), dtype=torch.float64)
    for b, n in enumerate(c["n"]):
        if n == 0:
            continue
        P, lo = c["P"][b], int(c["q_start"][b])
        t0 = max(0, P - window + 1) if window > 0 else 0
        t = torch.arange(t0, P + n)
        blk, row = c["table"][b][t // bs].long(), t % bs
        at = torch.arange(P, P + n)[:, None]
        seen = (t[None] <= at) & ((t[None] > at - window) if window > 0 else True)
        for g in range(Hkv):
            K, V = c["k_cache"][blk, g, row].double(), c["v_cache"][blk, g, row].double()
            Q = c["q"][lo:lo + n, g * G:(g + 1) * G].double()
            s = torch.einsum("ihd,td->iht", Q, K) * scale
            if softcap > 0:
                s = softcap * torch.tanh(s / softcap)
            s = s.masked_fill(~seen[:, None], -math.inf)
            p = torch.softmax(s, -1)
            # a key outside a row's set contributes nothing, whatever its value holds
            dot = lambda w, X: torch.where(  # noqa: E731
                torch.isfinite(X).all(), torch.einsum("iht,td->ihd", w, torch.nan_to_num(X)),
                (torch.where(seen[:, None, :, None], w[..., None] * X[None, None], 0.0)).sum(2)
                if not torch.isfinite(X).all() else 0.0)
            out[lo:lo + n, g * G:(g + 1) * G] = dot(p, V)
            A[lo:lo + n, g * G:(g + 1) * G] = dot(p, V.abs())
            m = torch.einsum("ihd,td->iht", Q.abs(), K.abs()) * scale
            S[lo:lo + n, g * G:(g + 1) * G] = torch.where(seen[:, None], m, 0.0).amax(-1)
    return out, A, S


def attention_tolerance(c, out, A, S, d):
    """Elementwise bound on the error of a kernel that keeps sums and softmax statistics in
    float32 and rounds only the weights (bfloat16 caches) and the output.
    u = 2^-24.  A score is a float32 dot product of d terms and at most four more roundings: off
    by at most (d + 4) u S.  That moves a weight by the same factor, once in the numerator and
    once in the sum; the sums over L keys add L u each, the exponential 2^-21.
    bfloat16: a weight is rounded by at most 2^-8 of itself, the output by 2^-8 of itself."""
    u = 2.0 ** -24
    L = max(a + b for a, b in zip(c["n"], c["P"]))
    rel = 2 * (d + 4) * u * S[..., None] + 2 * L * u + 2.0 ** -20
    if c["q"].dtype == torch.bfloat16:
        return A * (rel + 2.0 ** -8 * 1.01) + out.abs() * 2.0 ** -8 * 1.01 + 1e-30
    return A * rel + out.abs() * 2.0 ** -24 + 1e-30


def frequencies(dim, theta, scaling, factor, original_len, low, high):
    """Radians per position of each pair, and the amplitude."""
    fs, amp = [], 1.0
    if scaling == "ramp":
        e = lambda n: dim * math.log(original_len / (2 * math.pi * n)) / (2 * math.log(theta))  # noqa: E731
        a, z = max(0, math.floor(e(high))), min(dim - 1, math.ceil(e(low)))
        amp = 0.1 * math.log(factor) + 1.0
    for j in range(dim // 2):
        f = theta ** (-2.0 * j / dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "bands":
            k = min(1.0, max(0.0, (original_len * f / (2 * math.pi) - low) / (high - low)))
            f *= k + (1 - k) / factor
        elif scaling == "ramp":
            s = min(1.0, max(0.0, (j - a) / max(z - a, 0.001)))
            f = f * (1 - s) + f / factor * s
        fs.append(f)
    return torch.tensor(fs, dtype=torch.float64), amp


def rotate(x, pos, freq, amp, interleaved):
    """x [T, H, d] rotated by pos [T] in its first 2 * len(freq) columns, float64."""
    x = x.double().clone()
    m = 2 * len(freq)
    a = pos.double()[:, None] * freq
    co, si = (a.cos() * amp)[:, None], (a.sin() * amp)[:, None]
    i = (slice(0, m, 2), slice(1, m, 2)) if interleaved else (slice(0, m // 2), slice(m // 2, m))
    u, v = x[..., i[0]].clone(), x[..., i[1]].clone()
    x[..., i[0]] = u * co - v * si
    x[..., i[1]] = v * co + u * si
    return x


def logits(z, *, mask=None, tokens=None, counts=None, bias=None, grammar=None, rep=None,
           freq=None, pres=None, temp=None, probs=False):
    """Processed rows [B, N, V] in float64."""
    B, N, V = z.shape
    out = z.double().clone()
    for b in range(B):
        for i in range(N):
            r = out[b, i]
            if bias is not None:
                r = r + bias[b].double()
            if counts is not None:
                n = (counts[b].long() & 0x7FFFFFFF).clone()
                if mask is not None:
                    for c in range(1, N):
                        if (int(mask[b, i]) >> c) & 1:
                            n[int(tokens[b, c])] += 1
                told = (n > 0) | (counts[b] < 0)
                k = float(rep[b]) if rep is not None else 1.0
                r = torch.where(told, torch.where(r > 0, r / k, r * k), r)
                if freq is not None:
                    r = r - float(freq[b]) * n
                if pres is not None:
                    r = r - float(pres[b]) * (n > 0)
            if temp is not None:
                r = r / float(temp[b])
            if grammar is not None:
                x = torch.arange(V)
                ok = (grammar[b, i].long()[x // 32] >> (x % 32)) & 1
                r = torch.where(ok == 1, r, torch.tensor(-math.inf, dtype=torch.float64))
            if probs:
                if bool((r == -math.inf).all()):
                    r = torch.zeros_like(r)
                else:
                    r = torch.softmax(r, -1)
            out[b, i] = r
    return out

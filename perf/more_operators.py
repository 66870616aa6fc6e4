"""Cases of a serving step over an 8-bit cache and of sampling, and their plain forms.

Four operators, on the paged caches, ragged chunks and trees that the framework's
calls use.  The cache holds e4m3 codes with one power-of-two scale per block of
tokens and kv head (keys and values apart):

* ``append``: new tokens' queries and keys rotated by their positions, keys and values
  quantised into the cache's blocks, whose scales grow with what comes in;
* ``attend``: the attention of those tokens over the cache: prompt chunks, single
  tokens, chains, trees; windows, first tokens that stay visible, capped scores;
* ``compact``: the accepted path of each tree moved to contiguous positions;
* ``sample``: temperature, top-k, top-p and min-p on the target model's rows: the token
  that a given uniform number draws, and the filtered distribution.

``run`` computes them with elementary torch operations, or (``own``) through
the framework's entry points.
"""
import math
import random

import torch

own = False

GB = 1 << 30
E4M3 = torch.float8_e4m3fn
TOP = 448.0                  # the largest code
SMALL = -100                 # exponent of the smallest scale


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # the smallest call: one new token of one short conversation
        dict(name="attend_one_token", op="attend", heads=32, kv_heads=8, dim=128, block=16, batch=1,
             new_lo=1, new_hi=1, prefix_lo=300, prefix_hi=300, window=0, sinks=0, cap=0.0,
             tree=False, shape=1),
        # plain decoding of a full batch: every sequence one token, long ragged prefixes
        dict(name="attend_decode_b64", op="attend", heads=32, kv_heads=8, dim=128, block=16,
             batch=64, new_lo=1, new_hi=1, prefix_lo=512, prefix_hi=8192, window=0, sinks=0,
             cap=0.0, tree=False, shape=2),
        # verification of chains of five drafts in a large batch
        dict(name="attend_chains_b128", op="attend", heads=32, kv_heads=8, dim=128, block=16,
             batch=128, new_lo=6, new_hi=6, prefix_lo=1024, prefix_hi=4096, window=0, sinks=0,
             cap=0.0, tree=False, shape=3),
        # verification of trees of 26 nodes
        dict(name="attend_trees_b32", op="attend", heads=32, kv_heads=8, dim=128, block=16,
             batch=32, new_lo=26, new_hi=26, prefix_lo=512, prefix_hi=8192, window=0, sinks=0,
             cap=0.0, tree=True, shape=4),
        # layers with a sliding window, a few first tokens that stay visible and capped scores:
        # chunks of odd lengths beside sequences that decode, head size 64, larger blocks
        dict(name="attend_window_sinks", op="attend", heads=16, kv_heads=2, dim=64, block=32,
             batch=5, new_lo=1, new_hi=1200, prefix_lo=1000, prefix_hi=8000, window=1024, sinks=4,
             cap=30.0, tree=False, shape=5),
        # the largest: one chunk of a long prompt over what came before it
        dict(name="attend_long_chunk", op="attend", heads=28, kv_heads=4, dim=128, block=16,
             batch=1, new_lo=4096, new_hi=4096, prefix_lo=12281, prefix_hi=12281, window=0,
             sinks=0, cap=0.0, tree=False, shape=6),
        # the nodes of a batch of trees behind blocks that are partly filled, positions by depth
        dict(name="append_trees", op="append", heads=32, kv_heads=8, dim=128, block=16, batch=32,
             new_lo=26, new_hi=26, prefix_lo=512, prefix_hi=8192, layout="half", rotate=128,
             scaling="none", factor=1.0, by_depth=True, shape=7),
        # prompt chunks: interleaved pairs in half of the head, scaled for a long context
        dict(name="append_prompts", op="append", heads=28, kv_heads=4, dim=128, block=16, batch=4,
             new_lo=1000, new_hi=4100, prefix_lo=0, prefix_hi=90000, layout="interleaved",
             rotate=64, scaling="ramp", factor=8.0, by_depth=False, shape=8),
        # the accepted paths of a batch of trees, in the caches of a few layers
        dict(name="compact_b32", op="compact", layers=4, kv_heads=8, dim=128, block=16, batch=32,
             nodes=26, depth=6, prefix_lo=512, prefix_hi=8192, shape=9),
        # one tree of 60 nodes, every layer of a model at once
        dict(name="compact_b1_layers", op="compact", layers=32, kv_heads=8, dim=128, block=16,
             batch=1, nodes=60, depth=6, prefix_lo=2048, prefix_hi=2048, shape=23),
        # the next token of every sequence of a decoding batch, half-precision rows, all filters
        dict(name="sample_decode_b64", op="sample", dtype="bf16", batch=64, nodes=1, vocab=128256,
             top_k=50, top_p=0.9, min_p=0.02, temp=0.8, probs=False, shape=11),
        # the distributions that the acceptance of a batch of trees reads, after top-p
        dict(name="sample_trees_probs", op="sample", dtype="f32", batch=32, nodes=26, vocab=128256,
             top_k=0, top_p=0.95, min_p=0.0, temp=0.7, probs=True, shape=12),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 2)))) - 1))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "compact", "sample", "sample"])
    shape = rng.randrange(1 << 30)
    if op == "sample":
        c = dict(op=op, dtype=rng.choice(["f32", "f32", "bf16"]), batch=_log_int(rng, 1, 64),
                 nodes=rng.choice([1, 1, _log_int(rng, 1, 64)]),
                 vocab=rng.choice([128256, 152064, _log_int(rng, 1000, 260000)]),
                 top_k=rng.choice([0, 0, 1, 20, 50, _log_int(rng, 1, 5000)]),
                 top_p=rng.choice([1.0, 0.8, 0.9, 0.95, rng.uniform(0.05, 0.999)]),
                 min_p=rng.choice([0.0, 0.0, 0.02, rng.uniform(0.001, 0.5)]),
                 temp=rng.choice([0.6, 0.8, 1.0, rng.uniform(0.2, 2.0), 0.0]),
                 probs=rng.choice([True, False]), shape=shape)
        while c["batch"] * c["nodes"] * c["vocab"] > 32 * 26 * 128256:
            if c["batch"] > c["nodes"]:
                c["batch"] //= 2
            else:
                c["nodes"] //= 2
        return c
    block = rng.choice([16, 16, 32, 48, 128])
    if op == "compact":
        nodes = _log_int(rng, 2, 64)
        c = dict(op=op, layers=_log_int(rng, 1, 32), kv_heads=rng.choice([8, 4, 2, 1, 5]),
                 dim=rng.choice([64, 128, 128]), block=block, batch=_log_int(rng, 1, 128), nodes=nodes,
                 depth=rng.randrange(1, min(nodes, 9)), prefix_lo=0, prefix_hi=_log_int(rng, 1, 16000),
                 shape=shape)
        while c["layers"] * c["batch"] > 256:
            c["layers"] = max(1, c["layers"] // 2)
            c["batch"] = max(1, c["batch"] // 2)
        return c
    heads, kv_heads = rng.choice([(32, 8), (28, 4), (16, 2), (8, 8), (6, 2), (24, 1), (2, 1)])
    c = dict(op=op, heads=heads, kv_heads=kv_heads, dim=rng.choice([64, 128, 128]), block=block,
             batch=_log_int(rng, 1, 64), shape=shape)
    far = _log_int(rng, 0, 16000)
    c["prefix_lo"], c["prefix_hi"] = rng.choice([0, far // 4, far]), far
    kind = rng.choice(["chunk", "chunk", "window", "tree"])
    top = _log_int(rng, 1, 64 if kind == "tree" else 4096)
    c["new_lo"], c["new_hi"] = rng.choice([0, 1, max(1, top // 3)]), top
    if op == "attend":
        c["tree"] = kind == "tree"
        c["window"] = _log_int(rng, 1, 4000) if kind == "window" else 0
        c["sinks"] = rng.choice([0, 1, 4, 16, _log_int(rng, 1, 64)]) if kind == "window" else 0
        c["cap"] = rng.choice([0.0, 0.0, rng.uniform(5.0, 60.0)])
    else:
        c["layout"] = rng.choice(["half", "interleaved"])
        c["rotate"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2, 32])
        c["scaling"] = rng.choice(["none", "linear", "ramp", "bands"])
        c["factor"] = 1.0 if c["scaling"] == "none" else rng.uniform(1.5, 16.0)
        c["by_depth"] = rng.choice([False, True])
    # no more work than the largest listed cases of the operator
    while True:
        w = work(c)
        if sum(_lens(c)[0]) == 0:
            c["new_hi"] = c["new_lo"] = 1
        elif w["flops"] > 6e11 or w["bytes"] > 0.25 * GB:
            if c["batch"] > 4 or (c["new_hi"] <= 64 and c["batch"] > 1):
                c["batch"] = c["batch"] // 2
            else:
                c["new_hi"] = max(1, c["new_hi"] // 2)
                c["new_lo"] = min(c["new_lo"], c["new_hi"])
        else:
            return c


def _lens(c):
    """New tokens and prefix lengths of the sequences: the case's own, whatever the seed."""
    r = random.Random(c["shape"])
    lo, hi = (c["nodes"], c["nodes"]) if c["op"] == "compact" else (c["new_lo"], c["new_hi"])
    n = [_log_int(r, lo, hi) for _ in range(c["batch"])]
    p = [_log_int(r, c["prefix_lo"], c["prefix_hi"]) for _ in n]
    return n, p


def _paths(c):
    """Accepted paths of a compact case: a chain's start, then nodes behind the path's length (a
    tree labelled breadth-first), so that compacting twice is compacting once."""
    r = random.Random(c["shape"] + 1)
    paths = []
    for _ in range(c["batch"]):
        a = r.randrange(0, c["depth"] + 1)
        same = r.randrange(0, a + 1) if a + 1 + a < c["nodes"] else a
        paths.append(list(range(same + 1)) + sorted(r.sample(range(a + 1, c["nodes"]), a - same)))
    return paths


def work(case):
    c = case
    if c["op"] == "sample":
        cells = c["batch"] * c["nodes"] * c["vocab"]
        b = cells * ((4 if c["dtype"] == "f32" else 2) + (4 if c["probs"] else 0))
        return {"bytes": b + c["batch"] * c["nodes"] * 8, "flops": 3.0 * cells}
    if c["op"] == "compact":
        moved = sum(1 for p in _paths(c) for j, x in enumerate(p) if j != x)
        return {"bytes": 4 * c["layers"] * c["kv_heads"] * c["dim"] * moved + 12 * c["batch"], "flops": 0}
    n, p = _lens(c)
    h, g, d = c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "append":
        blocks = sum(-(-(a + b) // c["block"]) - b // c["block"] for a, b in zip(n, p) if a)
        return {"bytes": max(1, sum(n) * (4 * h + 6 * g) * d + 8 * blocks * g),
                "flops": sum(n) * (h + g) * c["rotate"] * 3.0}
    pairs = keys = 0
    for ni, pi in zip(n, p):
        if ni == 0:
            continue
        if c["window"]:
            w = c["window"]
            full = max(0, min(ni, pi + ni - w))    # tokens whose window is full
            rest = ni - full
            pairs += full * w + rest * pi + rest * (rest + 1) // 2
            pairs += sum(min(c["sinks"], max(0, pi + i - w + 1)) for i in range(ni)) if c["sinks"] else 0
            keys += min(pi + ni, w + ni - 1 + c["sinks"])
        else:
            # (of a tree's nodes each sees some of those before it: counted as half of them)
            pairs += ni * pi + (ni * (ni + 1) // (4 if c["tree"] else 2))
            keys += pi + ni
    return {"bytes": max(1, 4 * sum(n) * h * d + 2 * keys * g * d + 8 * keys * g // c["block"]),
            "flops": 4.0 * pairs * h * d}


# --------------------------------------------------------------------------
# what a user's program has in hand
# --------------------------------------------------------------------------

def _pages(c, n, p):
    """Block table of a paged cache, blocks in shuffled order: attention reads every sequence
    whole; where tokens are only appended or moved, the blocks before them are given back."""
    r = random.Random(c["shape"] + 2)
    last = [max(1, -(-(a + b) // c["block"])) for a, b in zip(n, p)]
    first = [0 if c["op"] == "attend" else min(b // c["block"], t - 1) for b, t in zip(p, last)]
    order = list(range(sum(last) - sum(first)))
    r.shuffle(order)
    order = torch.tensor(order, dtype=torch.int32, device="cuda")
    table = torch.full((len(n), max(last)), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(max(last), device="cuda")
    lo, hi = (torch.tensor(t, device="cuda")[:, None] for t in (first, last))
    table[(at >= lo) & (at < hi)] = order
    return table, order.numel()


def _starts(n):
    s = [0]
    for a in n:
        s.append(s[-1] + a)
    return s


def _codes(shape, gen):
    """Codes as a quantised block holds them: normal numbers whose largest is near the top."""
    flat = torch.empty(shape, dtype=torch.uint8, device="cuda")
    part = flat.view(-1)
    for i in range(0, part.numel(), 1 << 28):              # (float32 numbers of a part at once)
        x = torch.randn(min(1 << 28, part.numel() - i), generator=gen, device="cuda").mul_(96.0)
        part[i:i + x.numel()] = x.clamp_(-TOP, TOP).to(E4M3).view(torch.uint8)
    return flat.view(E4M3)


def _scales(shape, gen):
    e = torch.randint(-8, -5, shape, generator=gen, device="cuda")
    return torch.ldexp(torch.ones(shape, device="cuda"), e)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    i32 = dict(dtype=torch.int32, device="cuda")
    if c["op"] == "sample":
        s = _prepare_sample(c, gen, i32)
    elif c["op"] == "compact":
        s = _prepare_compact(c, gen, i32)
    else:
        s = _prepare_tokens(c, gen, i32)
    s["c"] = c
    if own:
        import eagle_speculative_decoding_parent_gb300 as tv
        s["tv"] = tv
        if c["op"] == "attend":
            need = tv.chunk_attention_q8_workspace(s["q"].shape[0], c["batch"], c["heads"],
                                                   c["kv_heads"], c["dim"])
            s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        if c["op"] == "append":
            s["rope"] = tv.rope_table(c["rotate"], theta=500000.0, interleaved=c["layout"] != "half",
                                      scaling=c["scaling"], factor=c["factor"],
                                      original_len=8192)
    return s


def _prepare_tokens(c, gen, i32):
    n, p = _lens(c)
    h, g, d = c["heads"], c["kv_heads"], c["dim"]
    table, blocks = _pages(c, n, p)
    starts = _starts(n)
    T = starts[-1]
    s = {"n": n, "p": p, "starts": starts, "table": table, "q_start": torch.tensor(starts, **i32),
         "prefix": torch.tensor(p, **i32), "status": torch.zeros(c["batch"], **i32)}
    for x in ("k", "v"):
        s[x + "_cache"] = _codes((blocks, g, c["block"], d), gen)
        s[x + "_scale"] = _scales((blocks, g), gen)
    # position of each token in its sequence, and the sequence it belongs to
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), torch.tensor(n, device="cuda"))
    at = torch.arange(T, device="cuda") - s["q_start"][:-1].long()[seq]
    s["seq"], s["at"] = seq, at
    s["slot"] = s["prefix"].long()[seq] + at
    if c["op"] == "attend":
        s["q"] = torch.randn((T, h, d), generator=gen, device="cuda", dtype=torch.bfloat16)
        s["out"] = torch.empty((T, h, d), device="cuda", dtype=torch.bfloat16)
        s["mask"] = None
        if c["tree"]:
            # random trees in topological order, as ancestor bits
            N = max(n)
            parent = (torch.rand((c["batch"], N), generator=gen, device="cuda") * torch.arange(N, device="cuda")).long()
            rel = torch.eye(N, dtype=torch.bool, device="cuda").expand(c["batch"], N, N).clone()
            for i in range(1, N):
                rel[:, i] |= rel[torch.arange(c["batch"], device="cuda"), parent[:, i]]
            bits = torch.ones((), dtype=torch.int64, device="cuda") << torch.arange(N, device="cuda")
            s["mask"] = (rel * bits).sum(2)[seq, at]
        return s
    # queries, keys and values as a fused projection leaves them: views of one row
    qkv = torch.randn((T, h + 2 * g, d), generator=gen, device="cuda", dtype=torch.bfloat16)
    s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + g], qkv[:, h + g:]
    s["q_out"] = torch.empty((T, h, d), device="cuda", dtype=torch.bfloat16)
    s["positions"] = None
    if c["by_depth"]:
        depth = torch.minimum(at, torch.randint(0, 7, (T,), generator=gen, device="cuda"))
        s["positions"] = (s["prefix"].long()[seq] + depth).to(torch.int32)
    return s


def _prepare_compact(c, gen, i32):
    n, p = _lens(c)
    table, blocks = _pages(c, n, p)
    paths, most = _paths(c), c["depth"] + 1
    s = {"n": n, "p": p, "table": table, "prefix": torch.tensor(p, **i32), "paths": paths,
         "path": torch.tensor([x + [-1] * (most - len(x)) for x in paths], **i32),
         "accept_len": torch.tensor([len(x) - 1 for x in paths], **i32),
         "new_lens": torch.zeros(c["batch"], **i32), "status": torch.zeros(c["batch"], **i32)}
    for x in ("k", "v"):
        s[x + "_cache"] = _codes((c["layers"], blocks, c["kv_heads"], c["block"], c["dim"]), gen)
        s[x + "_scale"] = _scales((c["layers"], blocks, c["kv_heads"]), gen)
    return s


def _prepare_sample(c, gen, i32):
    B, N, V = c["batch"], c["nodes"], c["vocab"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    f32 = dict(dtype=torch.float32, device="cuda")
    s = {"logits": torch.randn((B, N, V), generator=gen, device="cuda", dtype=dt).mul_(3.0),
         "uniform": torch.rand((B, N), generator=gen, device="cuda"),
         "tokens": torch.empty((B, N), **i32), "status": torch.zeros((B, N), **i32),
         "probs": torch.empty((B, N, V), **f32) if c["probs"] else None}
    # each sequence's own settings: some leave a filter out, or take the best token
    r = random.Random(c["shape"] + 3)
    temp = [r.choice([c["temp"], c["temp"], 1.0]) for _ in range(B)]
    s["temp"] = torch.tensor(temp, **f32)
    s["top_k"] = torch.tensor([r.choice([c["top_k"], c["top_k"], 2 * c["top_k"]]) for _ in range(B)], **i32)
    s["top_p"] = torch.tensor([r.choice([c["top_p"], c["top_p"], 1.0]) for _ in range(B)], **f32)
    s["min_p"] = torch.tensor([r.choice([c["min_p"], c["min_p"], 0.0]) for _ in range(B)], **f32)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    s, c = state, state["c"]
    if c["op"] == "attend":
        if own:
            s["tv"].chunk_attention_q8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"],
                                       s["v_scale"], s["table"], s["q_start"], s["prefix"],
                                       s["out"], s["status"], s["workspace"], softcap=c["cap"],
                                       window=c["window"], sinks=c["sinks"], mask=s["mask"])
            return s["out"]
        return _attend(s, c)
    if c["op"] == "append":
        if own:
            s["tv"].chunk_kv_append_q8(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                                       s["k_scale"], s["v_scale"], s["table"], s["q_start"],
                                       s["prefix"], s["status"], q_out=s["q_out"],
                                       rope=s["rope"], positions=s["positions"])
        else:
            _append(s, c)
        return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"],
                "v_scale": s["v_scale"]}
    if c["op"] == "compact":
        if own:
            s["tv"].kv_compact_q8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                  s["table"], s["prefix"], s["path"], s["accept_len"],
                                  s["new_lens"], s["status"])
        else:
            _compact(s, c)
        return {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"],
                "v_scale": s["v_scale"], "lens": s["new_lens"]}
    if own:
        s["tv"].logits_sample(s["logits"], s["uniform"], s["tokens"], s["status"],
                              temperature=s["temp"], top_k=s["top_k"], top_p=s["top_p"],
                              min_p=s["min_p"], probs=s["probs"])
    else:
        _sample(s, c)
    return {"tokens": s["tokens"], "probs": s["probs"]} if c["probs"] else {"tokens": s["tokens"]}


def _values(cache, scale, pages):
    """What the blocks of S sequences hold: [S, heads, positions, d] in 32 bits."""
    x = cache.view(torch.uint8)[pages].view(E4M3).float() * scale[pages][..., None, None]
    return x.transpose(2, 3).flatten(1, 2).transpose(1, 2)


def _attend_rows(s, c, b, n):
    """Softmax attention of the n tokens of each of the sequences b."""
    h, g, d, S = c["heads"], c["kv_heads"], c["dim"], len(b)
    w = h // g
    most = max(-(-(s["p"][i] + n) // c["block"]) for i in b)
    b = torch.tensor(b, device="cuda")
    prefix = s["prefix"][b].long()
    pages = s["table"][b, :most].clamp_min(0).long()
    rows = s["q_start"][b].long()[:, None] + torch.arange(n, device="cuda")
    k, v = (_values(s[x + "_cache"], s[x + "_scale"], pages) for x in ("k", "v"))
    at = (prefix[:, None] + torch.arange(n, device="cuda"))[..., None]   # [S, n, 1]
    keys = torch.arange(k.shape[2], device="cuda")
    seen = keys <= at
    if c["window"]:
        seen = seen & ((keys > at - c["window"]) | (keys < c["sinks"]))
    if s["mask"] is not None:
        node = (keys - prefix[:, None, None]).clamp(0, 63)
        seen = seen & ((keys < prefix[:, None, None]) | ((s["mask"][rows][..., None] >> node) & 1 > 0))
    q = s["q"][rows].float().view(S, n, g, w, d).permute(0, 2, 3, 1, 4).reshape(S, g, w * n, d)
    x = (q @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(S, g, w, n, -1)
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    o = (x.view(S, g, w * n, -1) @ v) / x.sum(-1).view(S, g, w * n, 1)
    return rows, o.view(S, g, w, n, d).permute(0, 3, 1, 2, 4).reshape(S, n, h, d)


def _attend(s, c):
    out = torch.empty_like(s["q"])
    # sequences with equally many new tokens together, few enough to hold their scores
    for n in sorted(set(s["n"]) - {0}):
        b = [i for i, a in enumerate(s["n"]) if a == n]
        step = max(1, (1 << 31) // (n * c["heads"] * (max(s["p"][i] for i in b) + n)))
        for i in range(0, len(b), step):
            rows, o = _attend_rows(s, c, b[i:i + step], n)
            out[rows] = o.to(out.dtype)
    return out


def _frequencies(c):
    """Radians per position of each rotated pair, in 64 bits, and the factor on cos and sin."""
    dim, theta, old, factor = c["rotate"], 500000.0, 8192, c["factor"]
    j = torch.arange(dim // 2, dtype=torch.float64, device="cuda")
    f = theta ** (-2.0 * j / dim)
    if c["scaling"] == "linear":
        return f / factor, 1.0
    if c["scaling"] == "bands":
        # long waves slowed down, short ones kept, a blend between the two borders
        turns = old * f / (2.0 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return f * (keep + (1.0 - keep) / factor), 1.0
    if c["scaling"] == "ramp":
        # a linear ramp over the pairs between 32 turns and one turn of the old context
        edge = [dim * math.log(old / (t * 2.0 * math.pi)) / (2.0 * math.log(theta)) for t in (32.0, 1.0)]
        lo, hi = max(0, math.floor(edge[0])), min(dim - 1, math.ceil(edge[1]))
        slow = ((j - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return f * (1.0 - slow) + f / factor * slow, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _rotate(x, cos, sin, c):
    m, half = c["rotate"], c["rotate"] // 2
    y = x.float().clone()
    a, b = (slice(0, half), slice(half, m)) if c["layout"] == "half" else (slice(0, m, 2), slice(1, m, 2))
    u, v = y[..., a].clone(), y[..., b].clone()
    y[..., a] = u * cos - v * sin
    y[..., b] = v * cos + u * sin
    return y


def _need(top):
    """The smallest power of two (from 2^-100 on) times which the largest code reaches top."""
    m, e = torch.frexp(top)                                # top = m 2^e, m in [1/2, 1)
    e = e.long() - 9 + (m > TOP / 512.0)
    return torch.where(top > 0, torch.ldexp(torch.ones_like(top), e.clamp_min(SMALL)), 2.0 ** SMALL)


def _put(s, c, name, x):
    """Quantises the rows x [T, heads, d] into their blocks."""
    cache, scale = s[name + "_cache"].view(torch.uint8), s[name + "_scale"]
    block = s["table"][s["seq"], s["slot"] // c["block"]].long()
    top = torch.zeros_like(scale).index_reduce_(0, block, x.abs().amax(-1), "amax")
    new = _need(top)
    # blocks that hold earlier tokens too keep at least their scale; their codes follow it
    b = torch.tensor([i for i, (a, p) in enumerate(zip(s["n"], s["p"])) if a and p % c["block"]],
                     dtype=torch.int64, device="cuda")
    p = s["prefix"][b].long()
    old = s["table"][b, p // c["block"]].long()
    new[old] = torch.maximum(new[old], scale[old])
    kept = (torch.arange(c["block"], device="cuda") < (p % c["block"])[:, None])[:, None, :, None]
    was = cache[old]
    now = (was.view(E4M3).float() * (scale[old] / new[old])[..., None, None]).to(E4M3)
    cache[old] = torch.where(kept, now.view(torch.uint8), was)
    cache[block, :, s["slot"] % c["block"]] = (x / new[block][..., None]).to(E4M3).view(torch.uint8)
    scale[block] = new[block]


def _append(s, c):
    f, amp = _frequencies(c)
    pos = s["slot"] if s["positions"] is None else s["positions"]
    angle = pos.double()[:, None] * f
    cos, sin = ((t * amp).float()[:, None] for t in (angle.cos(), angle.sin()))
    _put(s, c, "k", _rotate(s["k"], cos, sin, c))
    _put(s, c, "v", s["v"].float())
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c))


def _compact(s, c):
    bs = c["block"]
    A, path, p = s["accept_len"].long(), s["path"].long(), s["prefix"].long()[:, None]
    s["new_lens"].copy_(s["prefix"] + s["accept_len"] + 1)
    j = torch.arange(path.shape[1], device="cuda")
    live = (j <= A[:, None]).flatten()
    src, dst = (p + path).flatten()[live], (p + j).flatten()[live]
    seq = torch.arange(c["batch"], device="cuda").repeat_interleave(path.shape[1])[live]
    sb, db = s["table"][seq, src // bs].long(), s["table"][seq, dst // bs].long()
    # the blocks in which positions before the root stay
    part = (s["prefix"] % bs) > 0
    kb = s["table"][torch.arange(c["batch"], device="cuda"), s["prefix"].long() // bs].long()[part]
    kept = (torch.arange(bs, device="cuda") < (s["prefix"][part] % bs)[:, None])[:, None, :, None]
    for x in ("k", "v"):
        cache, scale = s[x + "_cache"].view(torch.uint8), s[x + "_scale"]
        rows, was = cache[:, sb, :, src % bs], scale[:, sb]            # rows [moved, layers, heads, d]
        new = torch.zeros_like(scale).index_reduce_(1, db, was, "amax")
        new[:, kb] = torch.maximum(new[:, kb], scale[:, kb])
        old = cache[:, kb]
        now = (old.view(E4M3).float() * (scale[:, kb] / new[:, kb])[..., None, None]).to(E4M3)
        cache[:, kb] = torch.where(kept, now.view(torch.uint8), old)
        ratio = (was / new[:, db]).transpose(0, 1)
        cache[:, db, :, dst % bs] = (rows.view(E4M3).float() * ratio[..., None]).to(E4M3).view(torch.uint8)
        scale[:, db] = new[:, db]


def _sample(s, c):
    B, N, V = c["batch"], c["nodes"], c["vocab"]
    x = s["logits"].float().view(B * N, V)
    temp, k, top_p, min_p = (s[t].repeat_interleave(N)[:, None] for t in ("temp", "top_k", "top_p", "min_p"))
    # best first, equal ones by their index; the weights in 64 bits, as sums next to a border are
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = (x - x[:, :1]).double().div_(torch.where(temp > 0, temp, 1.0).double()).exp_()
    rank = torch.arange(V, device="cuda")
    keep = rank < torch.where(temp > 0, torch.where(k > 0, k, V), 1)
    w = torch.where(keep, w, 0.0)
    before = torch.cumsum(w, 1) - w
    total = w.sum(1, keepdim=True)
    keep = (before < top_p.double() * total) | (top_p >= 1.0) | (rank == 0)
    w = torch.where(keep & (w >= min_p.double()), w, 0.0)
    w = torch.zeros_like(w).scatter_(1, order, w)                      # by index again
    mass = torch.cumsum(w, 1)
    total = mass[:, -1:]
    token = torch.searchsorted(mass, s["uniform"].view(-1, 1).double() * total, right=True)
    # (a cumulated sum that rounds down may stay below the last border)
    last = V - 1 - (w > 0).flip(1).to(torch.uint8).argmax(1, keepdim=True)
    s["tokens"].copy_(torch.minimum(token, last).view(B, N))
    if c["probs"]:
        s["probs"].copy_((w / total).view(B, N, V))


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    return {"attend": _attend_exact, "append": _append_exact, "compact": _compact_exact,
            "sample": _sample_exact}[c["op"]](s, c)


def _attend_exact(s, c):
    h, g, d = c["heads"], c["kv_heads"], c["dim"]
    out = torch.zeros((s["starts"][-1], h, d), dtype=torch.float64, device="cuda")
    low = torch.tensor(-math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["n"]):
        p, lo = s["p"][b], s["starts"][b]
        if n == 0:
            continue
        t = torch.arange(p + n, device="cuda")
        block, row = s["table"][b][t // c["block"]].long(), t % c["block"]
        code = {x: s[x + "_cache"].view(torch.uint8)[block, :, row].view(E4M3).double() for x in ("k", "v")}
        key, val = (code[x] * s[x + "_scale"][block].double()[..., None] for x in ("k", "v"))
        for kv in range(g):
            own_heads = slice(kv * (h // g), (kv + 1) * (h // g))
            for i in range(0, n, 1024):                    # query rows at once
                here = torch.arange(i, min(n, i + 1024), device="cuda")
                z = torch.einsum("ihd,td->iht", s["q"][lo + here, own_heads].double(), key[:, kv])
                z = z / d ** 0.5
                if c["cap"] > 0:
                    z = torch.tanh(z / c["cap"]) * c["cap"]
                me = p + here[:, None]
                ok = t[None] <= me
                if c["window"] > 0:
                    ok = ok & ((t[None] > me - c["window"]) | (t[None] < c["sinks"]))
                if s["mask"] is not None:
                    for node in range(n):
                        hides = torch.div(s["mask"][lo + here], 2 ** node, rounding_mode="floor") % 2 == 0
                        ok[:, p + node] = ok[:, p + node] & ~hides
                z = torch.where(ok[:, None], z, low)
                out[lo + here, own_heads] = torch.einsum("iht,td->ihd", torch.softmax(z, -1), val[:, kv])
    return out


def _to_code(y):
    """The nearest e4m3 number of |y| <= 448, ties to even, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3.0)
    return torch.round(y / step) * step


def _least(top):
    """The least scale for values up to top, by counting up the powers of two that are too small."""
    fits = torch.arange(SMALL, 121, dtype=torch.float64, device="cuda").exp2()
    return fits[(top[..., None] > TOP * fits).sum(-1)]


def _append_exact(s, c):
    m = c["rotate"]
    old, theta, k = 8192.0, 500000.0, c["factor"]
    rate, amp = [], 1.0
    for j in range(m // 2):
        f = math.pow(theta, -2.0 * j / m)
        if c["scaling"] == "linear":
            f /= k
        elif c["scaling"] == "bands":
            wave = 2.0 * math.pi / f
            if wave > old / 1.0:
                f /= k
            elif wave > old / 4.0:
                mix = (old / wave - 1.0) / 3.0
                f = (1.0 - mix) * f / k + mix * f
        elif c["scaling"] == "ramp":
            first = max(0, math.floor(m * math.log(old / (64.0 * math.pi)) / (2.0 * math.log(theta))))
            last = min(m - 1, math.ceil(m * math.log(old / (2.0 * math.pi)) / (2.0 * math.log(theta))))
            r = min(1.0, max(0.0, (j - first) / (last - first if last > first else 0.001)))
            f = f * (1.0 - r) + r * f / k
            amp = 0.1 * math.log(k) + 1.0
        rate.append(f)
    pos = (s["slot"] if s["positions"] is None else s["positions"].long()).double()
    turn = torch.polar(torch.full((1,), amp, dtype=torch.float64, device="cuda"),
                       torch.outer(pos, torch.tensor(rate, dtype=torch.float64, device="cuda")))[:, None]

    def spun(x):
        x = x.double()
        pairs = x[..., :m].unflatten(-1, (2, m // 2)).transpose(-1, -2) if c["layout"] == "half" else x[..., :m].unflatten(-1, (m // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.transpose(-1, -2).flatten(-2) if c["layout"] == "half" else z.flatten(-2)
        return torch.cat([z, x[..., m:]], -1)

    found = {"q": spun(s["q"])}
    for name, rows in (("k", spun(s["k"])), ("v", s["v"].double())):
        code = s[name + "_cache"].double()
        scale = s[name + "_scale"].double()
        # sequence by sequence, block by block
        for b, (n, p) in enumerate(zip(s["n"], s["p"])):
            for lb in range(p // c["block"], -(-(p + n) // c["block"]) if n else 0):
                lo, hi = max(p, lb * c["block"]), min(p + n, (lb + 1) * c["block"])
                at, x = int(s["table"][b, lb]), rows[s["starts"][b] + lo - p:s["starts"][b] + hi - p]
                least = _least(x.abs().amax((0, 2)))
                r0, r1 = lo - lb * c["block"], hi - lb * c["block"]
                if r0 > 0:
                    least = torch.maximum(least, scale[at])
                    code[at, :, :r0] = _to_code(code[at, :, :r0] * (scale[at] / least)[:, None, None])
                code[at, :, r0:r1] = _to_code(x.transpose(0, 1) / least[:, None, None])
                scale[at] = least
        found[name], found[name + "_scale"] = code, scale
    return found


def _compact_exact(s, c):
    found = {"lens": torch.tensor([p + len(x) for p, x in zip(s["p"], s["paths"])], dtype=torch.int32, device="cuda")}
    bs = c["block"]
    for name in ("k", "v"):
        code, scale = s[name + "_cache"].double(), s[name + "_scale"].double()
        was, had = code.clone(), scale.clone()
        for b, (p, path) in enumerate(zip(s["p"], s["paths"])):
            block = s["table"][b].tolist()
            for lb in range(p // bs, (p + len(path) - 1) // bs + 1):
                to = block[lb]
                js = [j for j in range(len(path)) if (p + j) // bs == lb]
                new = torch.stack([had[:, block[(p + path[j]) // bs]] for j in js]).amax(0)
                keep = max(0, p - lb * bs)
                if keep:
                    new = torch.maximum(new, had[:, to])
                    code[:, to, :, :keep] = _to_code(was[:, to, :, :keep] * (had[:, to] / new)[..., None, None])
                for j in js:
                    src = p + path[j]
                    x = was[:, block[src // bs], :, src % bs] * had[:, block[src // bs]][..., None]
                    code[:, to, :, (p + j) % bs] = _to_code(x / new[..., None])
                scale[:, to] = new
        found[name], found[name + "_scale"] = code, scale
    return found


def _sample_exact(s, c):
    B, N, V = c["batch"], c["nodes"], c["vocab"]
    tokens = torch.zeros((B, N), dtype=torch.int32, device="cuda")
    probs = torch.zeros((B, N, V), dtype=torch.float64, device="cuda") if c["probs"] else None
    settings = [s[t].tolist() for t in ("temp", "top_k", "top_p", "min_p")]
    for b in range(B):
        temp, k, top_p, min_p = (t[b] for t in settings)
        z = s["logits"][b].double()
        for i in range(N):
            best = torch.argmax(z[i])
            row = z[i] - z[i, best]
            if temp == 0.0:
                row = torch.where(torch.arange(V, device="cuda") == best, 0.0, -math.inf).double()
                k, top_p, min_p = 0, 1.0, 0.0
            else:
                row = row / temp
            w = torch.exp(row)
            order = torch.argsort(row, descending=True, stable=True)
            order = order[:k] if 0 < k < V else order
            if top_p < 1.0:
                mass = torch.cumsum(w[order], 0)
                order = order[:int((mass < top_p * w[order].sum()).sum()) + 1]
            order = order[w[order] >= min_p]
            only = torch.zeros_like(w)
            only[order] = w[order]
            ids = torch.sort(order[w[order] > 0]).values
            edge = torch.cumsum(w[ids], 0)
            tokens[b, i] = ids[min(int((edge <= s["uniform"][b, i].double() * edge[-1]).sum()), ids.numel() - 1)]
            if c["probs"]:
                probs[b, i] = only / edge[-1]
    return {"tokens": tokens, "probs": probs} if c["probs"] else {"tokens": tokens}
